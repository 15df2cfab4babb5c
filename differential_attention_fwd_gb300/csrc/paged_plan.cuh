// paged_plan.cuh -- how the attention over a paged cache is cut into work, shared by
// its kernels and the pass that merges their partial results.
//
// The lengths are on the device, so the host launches a fixed grid and every block
// finds its own share.  A unit is (sequence, key/value head, row chunk) with the
// sequence's tiles of KT keys; the units' tiles are laid end to end, sequence by
// sequence, and of `total` tiles block c takes c * total / G .. (c + 1) * total / G,
// G = min(grid, total): equal to within one tile, whatever the lengths.  A block's
// range falls into segments, each of one unit.  A segment that holds its whole unit
// is finished by its block; one that does not leaves a partial result: in slot
// 2 c + 1 if the unit starts in it (it is then the block's last), else in slot 2 c
// (the block's first).  So the workspace grows with the grid and not with the batch,
// and the merging pass takes one block a boundary.
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

__device__ __forceinline__ int64_t paged_seq_tiles(const PagedSeq& s, int kt) { return (s.total + kt - 1) / kt; }

// The page of a key's slot, or -1 if its table entry is out of range.  `key` is below
// the sequence's total, so the entry exists.
__device__ __forceinline__ int paged_page(const PagedParams& p, int b, int index) {
    const int32_t pg = __ldg(p.table + b * p.table_stride + index);
    return pg >= 0 && pg < p.num_pages ? pg : -1;
}

struct PagedStart {
    int64_t total;      // tiles of all units
    int64_t first;      // the block's first tile,
    int b;              // its sequence, and
    int64_t local;      // its place among the sequence's tiles
};

// Every thread of the block calls this; `scratch` holds THREADS / 32 + 1 int64_t and
// a PagedStart in shared memory.
template <int THREADS>
__device__ __forceinline__ PagedStart paged_start(const PagedParams& p, int kt, int64_t* scratch, PagedStart* result) {
    constexpr int WARPS = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t units = (int64_t)p.Hk * p.row_chunks;
    const int per = (p.B + THREADS - 1) / THREADS;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b) sum += paged_seq_tiles(paged_seq(p, b), kt) * units;
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += scratch[w];
        total += scratch[w];
    }
    int64_t at = before + incl - sum;          // tiles before this thread's sequences
    const int64_t grid = total < gridDim.x ? total : (int64_t)gridDim.x;
    const int64_t first = blockIdx.x < grid ? blockIdx.x * total / grid : total;
    if (tid == 0) *result = PagedStart{total, total, p.B, 0};
    __syncthreads();
    for (int b = b0; b < b1; ++b) {
        const int64_t n = paged_seq_tiles(paged_seq(p, b), kt) * units;
        if (first >= at && first < at + n) *result = PagedStart{total, first, b, first - at};
        at += n;
    }
    __syncthreads();
    return *result;
}

// A block's segments in turn.
struct PagedCursor {
    int64_t left;               // tiles of the block's range not yet handed out
    int local;                  // place among the sequence's tiles (fewer than 2^31: checked on the host)
    int b, unit;                // unit of the sequence (hk * row_chunks + row chunk)
    int hk, rc;
    int tile0, n;               // the segment's tiles within the unit
    int tiles;                  // the unit's
    PagedSeq s;

    __device__ __forceinline__ void begin(const PagedParams& p, const PagedStart& st, int kt) {
        const int64_t grid = st.total < gridDim.x ? st.total : (int64_t)gridDim.x;
        left = blockIdx.x < grid ? (blockIdx.x + 1) * st.total / grid - st.first : 0;
        b = st.b;
        local = (int)st.local;
        if (left > 0) load(p, kt);
    }
    __device__ __forceinline__ void load(const PagedParams& p, int kt) {
        s = paged_seq(p, b);
        tiles = (int)paged_seq_tiles(s, kt);
        cut(p);
    }
    __device__ __forceinline__ void cut(const PagedParams& p) {
        unit = local / tiles;
        tile0 = local - unit * tiles;
        n = (int)(left < tiles - tile0 ? left : tiles - tile0);
        hk = unit / p.row_chunks;
        rc = unit - hk * p.row_chunks;
    }
    __device__ __forceinline__ bool done() const { return left <= 0; }
    __device__ __forceinline__ void next(const PagedParams& p, int kt) {
        left -= n;
        local += n;
        if (left <= 0) return;
        if (local == tiles * p.Hk * p.row_chunks) {
            local = 0;
            do {
                if (++b >= p.B) { left = 0; return; }   // never with tiles left
                s = paged_seq(p, b);
            } while (s.n_new == 0);
            tiles = (int)paged_seq_tiles(s, kt);
        }
        cut(p);
    }
    __device__ __forceinline__ bool whole() const { return n == tiles; }
    __device__ __forceinline__ int slot() const { return 2 * (int)blockIdx.x + (tile0 == 0 ? 1 : 0); }
    // One thread of the block, at each of its segments and once before them: leaves word
    // for the merging pass.  The unit's last tile is in the block before the first one
    // that begins at its end or later.
    __device__ __forceinline__ void no_join(const PagedParams& p) const { p.joins[blockIdx.x].parts = 0; }
    __device__ __forceinline__ void join(const PagedParams& p, int64_t total) const {
        if (tile0 != 0 || whole()) return;
        const int64_t grid = total < gridDim.x ? total : (int64_t)gridDim.x;
        // the block's range ends with this segment: the unit goes on at tile `end` of the
        // launch, and ends `rest` tiles later
        const int64_t end = (int64_t)(blockIdx.x + 1) * total / grid, last = end + (tiles - n) - 1;
        int64_t c = last * grid / total;                // a block that begins at `last` or before
        while (c + 1 < grid && (c + 1) * total / grid <= last) ++c;
        while (c * total / grid > last) --c;
        p.joins[blockIdx.x] = PagedJoin{(int)(c - blockIdx.x) + 1, b, unit, s.n_new};
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

// Which of the new tokens row q sees, as bits (tree; Tq <= 64).
__device__ __forceinline__ uint64_t paged_mask_bits(const PagedParams& p, int b, int q, int n_new) {
    const uint8_t* m = p.mask + b * p.mask_stride[0] + q * p.mask_stride[1];
    uint64_t bits = 0;
    for (int j = 0; j < n_new; ++j) bits |= (uint64_t)(m[j] != 0) << j;
    return bits;
}

// One row's output from O_b and l_b of both branches: columns lane + 32 j, j < J.
template <int J>
__device__ __forceinline__ void paged_finish_row(const PagedParams& p, float lam, int b, int h, int q, int lane,
                                                 const float (&o1)[J], float l1, const float (&o2)[J], float l2) {
    const float i1 = l1 == 0.f ? 0.f : 1.f / l1;       // a row that saw nothing gives 0
    const float i2 = l2 == 0.f ? 0.f : 1.f / l2;
    float y[J];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        // the branches rounded alike, so that alike branches cancel exactly at lambda = 1
        y[j] = fmaf(-lam, __fmul_rn(o2[j], i2), __fmul_rn(o1[j], i1));
        if (lane + 32 * j >= p.Dv) y[j] = 0.f;
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
            if (lane + 32 * j < p.Dv) {
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
        const int c = lane + 32 * j;
        if (c >= p.Dv) continue;
        float v = y[j];
        if (p.norm_weight) v *= p.norm_weight[(int64_t)h * p.Dv + c];
        if (p.norm_bias) v += p.norm_bias[(int64_t)h * p.Dv + c];
        v *= p.out_scale;
        if (p.bf16) static_cast<__nv_bfloat16*>(p.out)[at + c] = __float2bfloat16_rn(v);
        else static_cast<float*>(p.out)[at + c] = v;
    }
}

}  // namespace diffattn
