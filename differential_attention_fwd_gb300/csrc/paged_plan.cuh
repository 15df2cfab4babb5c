// paged_plan.cuh -- how the attention over a paged cache is cut into work, shared by
// its kernels and the pass that merges their partial results.
//
// The lengths are on the device, so the host launches a fixed number of workers (blocks,
// groups of warps, or warps) and every one finds its own share.  A unit is (sequence,
// key/value head, row chunk) with the sequence's tiles of KT keys; the units' tiles are
// laid end to end, sequence by sequence, and of `total` tiles every worker takes
// total / G in a row, or one more, whatever the lengths (fewer workers where there are
// fewer tiles).  A boundary that falls within `snap` tiles of a unit's end moves there:
// so little work is not worth a unit in two parts, unless it is much of a share.
//
// A worker's range falls into segments, each of one unit.  A segment that holds its whole
// unit is finished by its worker; one that does not leaves a partial result: in slot
// 2 c + 1 if the unit starts in it (it is then the worker's last), else in slot 2 c (the
// worker's first).  So the workspace grows with the workers and not with the batch, and a
// merging pass has at most one unit a worker to join.
#pragma once

#include "kernels.h"
#include "paged.h"
#include "ptx.cuh"

namespace diffattn {

// A sequence's lengths as the kernels use them.
struct PagedSeq {
    int n_new;          // query rows of each head
    int64_t before;     // tokens before them
    int total;          // keys
    bool bad;           // lengths outside the table: rows of NaN (n_new and total are stand-ins)
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int b) {
    PagedSeq s;
    s.n_new = p.q_lengths ? p.q_lengths[b] : p.Tq;
    s.before = p.lengths[b];
    s.total = 0;
    s.bad = false;
    if (s.n_new == 0) return s;
    const int64_t total = s.before + s.n_new;
    if (s.n_new < 0 || s.n_new > p.Tq || s.before < 0 || total > p.max_pages * p.page || total > INT32_MAX / 2) {
        s.bad = true;
        s.n_new = p.Tq;
        s.before = 0;
        s.total = 1;
    } else {
        s.total = (int)total;
    }
    return s;
}

__device__ __forceinline__ int paged_seq_tiles(const PagedSeq& s, int kt) { return (s.total + kt - 1) / kt; }

// The page of a key's slot, or -1 if its table entry is out of range.  `key` is below
// the sequence's total, so the entry exists.
__device__ __forceinline__ int paged_page(const PagedParams& p, int b, int index) {
    const int32_t pg = __ldg(p.table + b * p.table_stride + index);
    return pg >= 0 && pg < p.num_pages ? pg : -1;
}

// The division of a launch.  All counts are below 2^31 (checked on the host).
struct PagedShares {
    int total;          // tiles of all units
    int workers;        // that take tiles
    int each, more;     // `more` of them take each + 1 tiles, the others each
    int snap;
    __device__ __forceinline__ void set(int t, int most, int most_snap) {
        total = t;
        workers = min(most, t);
        each = workers ? t / workers : 0;
        more = t - each * workers;
        snap = min(most_snap, each / 4);
    }
    // Where worker c's share begins before it is moved to a unit's end; `total` for a
    // worker that takes none.
    __device__ __forceinline__ int bound(int c) const { return c < workers ? c * each + min(c, more) : total; }
    // The last worker whose share begins at `tile` or before.
    __device__ __forceinline__ int worker_at(int tile) const {
        const int turn = more * (each + 1);
        return tile < turn ? tile / (each + 1) : more + (tile - turn) / each;
    }
};

// Where a worker's range starts: the launch's tile, its sequence, and its place among the
// sequence's tiles (all of them: the range starts with the next sequence that has any).
struct PagedStart {
    int tile, b, local;
};

// What a block knows of its workers, in shared memory.
template <int NW>
struct PagedBlock {
    PagedShares shares;
    PagedStart start[NW + 1];       // of its workers, and of the one after them
};

// The tiles and active units before and in each thread's sequences.  Every thread of the
// block calls this; `scratch`: 2 * THREADS / 32 ints in shared memory.
struct PagedScan {
    int b0, b1;         // the thread's sequences,
    int at, sum;        // the tiles before them and in them
    int tiles;          // of a unit of its last sequence with any
    int total, units;   // of the launch
};
template <int THREADS>
__device__ __forceinline__ PagedScan paged_scan(const PagedParams& p, int kt, int extra, int* scratch) {
    constexpr int WARPS = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per_seq = p.Hk * p.row_chunks;
    const int per = (p.B + THREADS - 1) / THREADS;
    PagedScan s;
    s.b0 = min(p.B, tid * per);
    s.b1 = min(p.B, s.b0 + per);
    s.sum = s.tiles = 0;
    int active = 0;
    for (int b = s.b0; b < s.b1; ++b) {
        const int tiles = paged_seq_tiles(paged_seq(p, b), kt);
        s.sum += tiles ? (tiles + extra) * per_seq : 0;
        active += tiles ? per_seq : 0;
        s.tiles = tiles ? tiles : s.tiles;
    }
    int incl = s.sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    active = __reduce_add_sync(0xffffffffu, active);
    if (lane == 31) {
        scratch[warp] = incl;
        scratch[WARPS + warp] = active;
    }
    __syncthreads();
    int before = 0;
    s.total = s.units = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += scratch[w];
        s.total += scratch[w];
        s.units += scratch[WARPS + w];
    }
    s.at = before + incl - s.sum;
    return s;
}

// Where the block's `nw` <= NW workers start, of `most` in the launch, and the one after.
// Every thread calls this, and it ends with a barrier.
template <int NW>
__device__ __forceinline__ void paged_locate(const PagedParams& p, const PagedScan& s, int kt, int extra, int nw, int most,
                                             int snap, PagedBlock<NW>* out) {
    const int tid = threadIdx.x;
    const int units = p.Hk * p.row_chunks;
    PagedShares sh;
    sh.set(s.total, most, snap);
    if (tid == 0) out->shares = sh;
    if (tid <= nw && sh.bound(blockIdx.x * nw + tid) >= s.total) out->start[tid] = PagedStart{s.total, p.B, 0};
    for (int w = 0; w <= nw; ++w) {
        const int first = sh.bound(blockIdx.x * nw + w);
        if (first >= s.total || first < s.at || first >= s.at + s.sum) continue;
        int at = s.at;
        for (int b = s.b0; b < s.b1; ++b) {
            // with a sequence a thread its tiles are known
            int tiles = s.b1 - s.b0 == 1 ? s.tiles : paged_seq_tiles(paged_seq(p, b), kt);
            if (tiles == 0) continue;
            tiles += extra;
            if (first < at + tiles * units) {
                const int off = (first - at) % tiles;       // in its unit
                const int move = off <= extra + sh.snap ? -off : tiles - off <= sh.snap ? tiles - off : 0;
                out->start[w] = PagedStart{first + move, b, first + move - at};
                break;
            }
            at += tiles * units;
        }
    }
    __syncthreads();
}

// A worker's segments in turn.
struct PagedCursor {
    int left;                   // tiles of the worker's range not yet handed out
    int local;                  // place among the sequence's tiles
    int worker;
    int b;
    int hk, rc;                 // the segment's unit: key/value head and row chunk
    int tile0, n;               // the segment's tiles within the unit,
    int step;                   // and how many they count as
    int tiles;                  // the unit's
    PagedSeq s;

    // The `w`-th worker of the block, worker c of the launch.
    template <int NW>
    __device__ __forceinline__ void begin(const PagedParams& p, const PagedBlock<NW>& blk, int w, int c, int kt, int extra) {
        worker = c;
        left = blk.start[w + 1].tile - blk.start[w].tile;
        b = blk.start[w].b;
        local = blk.start[w].local;
        if (left <= 0) return;
        s = paged_seq(p, b);
        tiles = paged_seq_tiles(s, kt);
        enter(p, kt, extra);
    }
    __device__ __forceinline__ void enter(const PagedParams& p, int kt, int extra) {
        if (local == (tiles + extra) * p.Hk * p.row_chunks) {
            local = 0;
            do {
                if (++b >= p.B) { left = 0; return; }   // never with tiles left
                s = paged_seq(p, b);
            } while (s.n_new == 0);
            tiles = paged_seq_tiles(s, kt);
        }
        const int counts = tiles + extra, unit = local / counts, off = local - unit * counts;
        step = min(left, counts - off);
        tile0 = max(0, off - extra);
        n = off + step - extra - tile0;
        hk = unit / p.row_chunks;
        rc = unit - hk * p.row_chunks;
    }
    __device__ __forceinline__ bool done() const { return left <= 0; }
    __device__ __forceinline__ void next(const PagedParams& p, int kt, int extra) {
        left -= step;
        local += step;
        if (left > 0) enter(p, kt, extra);
    }
    __device__ __forceinline__ bool whole() const { return n == tiles; }
    __device__ __forceinline__ int slot() const { return 2 * worker + (tile0 == 0 ? 1 : 0); }
    // One thread of the worker, at each of its segments, and no_join once before them:
    // leaves word for the merging pass.  A unit that starts here and does not end here is
    // this range's last, and the workers that go on with it are those whose bounds fall
    // into it and were not moved to its ends.  `end`: where this range ends.
    __device__ __forceinline__ static void no_join(const PagedParams& p, int c) { p.joins[c].parts = 0; }
    __device__ __forceinline__ void join(const PagedParams& p, const PagedShares& sh, int end, int extra) const {
        if (tile0 != 0 || whole()) return;
        const int u1 = end - step + tiles + extra;
        p.joins[worker] = PagedJoin{sh.worker_at(u1 - sh.snap - 1) - worker + 1, b, hk * p.row_chunks + rc, s.n_new};
    }
    // The segment's tiles that some row of its chunk may see: later ones hold only
    // keys behind the chunk's last query.
    __device__ __forceinline__ int live_tiles(const PagedParams& p, int kt) const {
        if (s.bad) return 0;
        const int row0 = rc * p.chunk_rows;
        int64_t last = s.total - 1;
        if (!p.mask && row0 / p.head_rows == (row0 + p.chunk_rows - 1) / p.head_rows)   // rows of one head
            last = min(last, s.before + min(row0 % p.head_rows + p.chunk_rows, s.n_new) - 1);
        const int64_t need = last / kt + 1 - tile0;
        return (int)(need < 0 ? 0 : need < n ? need : n);
    }
};

// Row r of a unit: head and query, and whether it is one (not padding).
struct PagedRow {
    int h, q;
    bool live;
};
__device__ __forceinline__ PagedRow paged_row(const PagedParams& p, int hk, int rc, int r, int n_new) {
    const int row = rc * p.chunk_rows + r;
    const int hh = row / p.head_rows;
    PagedRow x;
    x.q = row - hh * p.head_rows;
    x.h = hk * p.group + hh;
    x.live = hh < p.group && x.q < n_new;
    return x;
}

// Which of the new tokens each lane's row q sees, as bits (tree; Tq <= 64), for the lanes
// below N whose row is live; the others get 0.  The whole warp calls this: it reads one
// row after another, a byte a lane, all of them at once (a row a thread, byte by byte,
// took 3 to 5 us at a segment's start).
template <int N>
__device__ __forceinline__ uint64_t paged_mask_bits(const PagedParams& p, int b, int q, bool live, int n_new, int lane) {
    const uint8_t* m = p.mask + b * p.mask_stride[0];
    uint64_t bits = 0;
    constexpr int AT_ONCE = N < 16 ? N : 16;
    const int c0 = min(lane, n_new - 1), c1 = min(lane + 32, n_new - 1);
    const uint32_t has0 = n_new >= 32 ? ~0u : (1u << n_new) - 1;
    const uint32_t has1 = n_new <= 32 ? 0u : n_new >= 64 ? ~0u : (1u << (n_new - 32)) - 1;
    const int64_t at = live ? q * p.mask_stride[1] : 0;
    for (int r0 = 0; r0 < N; r0 += AT_ONCE) {
        // no branch around a load, so that none waits for another
        uint8_t x[AT_ONCE][2];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const int64_t row = __shfl_sync(0xffffffffu, at, r0 + i);
            x[i][0] = m[row + c0];
            x[i][1] = m[row + c1];
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const uint32_t lo = __ballot_sync(0xffffffffu, x[i][0] != 0), hi = __ballot_sync(0xffffffffu, x[i][1] != 0);
            if (lane == r0 + i && live) bits = (uint64_t)(hi & has1) << 32 | (lo & has0);
        }
    }
    return bits;
}

// One row's output from O_b and l_b of both branches: columns lane + 32 j, j < J, or
// J lane + j where ROWWISE.
template <int J, bool ROWWISE = false>
__device__ __forceinline__ void paged_finish_row(const PagedParams& p, float lam, int b, int h, int q, int lane,
                                                 const float (&o1)[J], float l1, const float (&o2)[J], float l2) {
    const float i1 = l1 == 0.f ? 0.f : 1.f / l1;       // a row that saw nothing gives 0
    const float i2 = l2 == 0.f ? 0.f : 1.f / l2;
    const auto col = [&](int j) { return ROWWISE ? J * lane + j : lane + 32 * j; };
    float y[J];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        // the branches rounded alike, so that alike branches cancel exactly at lambda = 1
        y[j] = fmaf(-lam, __fmul_rn(o2[j], i2), __fmul_rn(o1[j], i1));
        if (col(j) >= p.Dv) y[j] = 0.f;
        sum += y[j];
    }
    if (p.norm != kNormNone) {
        float mean = 0.f;
        if (p.norm == kNormGroup) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            mean = sum / p.Dv;
        }
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (col(j) < p.Dv) {
                y[j] -= mean;
                ss = fmaf(y[j], y[j], ss);
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = 1.0f / sqrtf(ss / p.Dv + p.norm_eps);
#pragma unroll
        for (int j = 0; j < J; ++j) y[j] *= r;
    }
    const int64_t at = b * p.s_o[0] + h * p.s_o[1] + q * p.s_o[2];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = col(j);
        if (c >= p.Dv) continue;
        float v = y[j];
        if (p.norm_weight) v *= p.norm_weight[(int64_t)h * p.Dv + c];
        if (p.norm_bias) v += p.norm_bias[(int64_t)h * p.Dv + c];
        v *= p.out_scale;
        y[j] = v;
        if (ROWWISE && p.o4) continue;
        if (p.bf16) static_cast<__nv_bfloat16*>(p.out)[at + c] = __float2bfloat16_rn(v);
        else static_cast<float*>(p.out)[at + c] = v;
    }
    if constexpr (ROWWISE) {                    // bf16, all columns live
        if (p.o4)
#pragma unroll
            for (int j = 0; j < J; j += 2)
                *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + at + col(j)) = pack_bf16x2(y[j], y[j + 1]);
    }
}

}  // namespace diffattn
