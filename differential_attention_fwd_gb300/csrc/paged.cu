// paged.cu -- differential attention over a paged key/value cache: the pass that
// merges partial results, and the CUDA-core kernel, which takes every type, width and
// page size (the tensor-core kernels in paged_mma.cu and paged_tc.cu take bf16 with a
// value width of 128).
//
// CUDA-core kernel: a block of 128 threads streams a unit's keys in tiles of 32 through
// two stages of shared memory (cp.async, one tile ahead).  Per tile: each thread takes
// one key of one branch against half of the unit's rows; each warp forms the running
// maxima, weights and sums of its rows with a lane a key; then a thread takes one output
// column (two for Dv > 128) of both branches and all rows over its share of the keys.
// Everything is float32, as the float32 cache's results are.  A tile that reaches into
// the new tokens or past the end marks hidden keys by a negative weight, which the
// sums leave out: a hidden key's value may hold anything.
//
// Bound, where it is used (float32 caches and other widths of small models), by latency: 4
// sequences of up to 2900 keys, 3 tokens, 4 key/value heads, D = 32 take 22.2 us.  Of those
// 1.6 go to the lengths and the division, 2.8 to the first queries, 2 to a page and its keys,
// 2.5 to each of two tiles, 1.3 to the block's sums, and 6 to the merging pass; HBM would
// take 2.3.  At length by shared memory and the exchanges of the softmax: 9 tokens, 16
// heads, 4 sequences of up to 8348 take 128 us, 0.21 of the copy rate.
#include "paged_plan.cuh"
#include "kernels.h"
#include "pdl.cuh"

namespace diffattn {
namespace paged {

constexpr int THREADS = 128;
constexpr int WARPS = THREADS / 32;
constexpr int KT = 32;
constexpr int MAX_RC = 16;
constexpr int SNAP = 2;
constexpr int EXTRA = 1;                        // what a unit's start costs, in tiles

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// 16 bytes of shared memory as floats.
__device__ __forceinline__ void load16(const float* p, float* x) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float* x) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Shared memory of the CUDA-core kernel.  Key rows are 16 bytes longer than their
// data, so that threads of one quarter warp read 16 bytes of eight rows from
// different banks; widths are rounded up to 16 bytes with zeros.
struct Layout {
    int dpad;           // D rounded up to 16 bytes, elements
    int krow, vrow;     // row strides, elements
    int stage;          // bytes
    int off_q, off_p, off_stat, total;
};
// Floats of a key's weights: 4 x an odd number, so that keys of 32 lanes spread over the banks.
__host__ __device__ constexpr int weights_row(int rc) { return rc > 1 && rc % 4 == 0 ? 2 * rc + 4 : 2 * rc; }
__host__ __device__ inline Layout simt_layout(int D, int Dv, int es, int rc, bool shared) {
    const int v = 16 / es;
    Layout l;
    l.dpad = (D + v - 1) / v * v;
    l.krow = l.dpad + v;
    l.vrow = (Dv + v - 1) / v * v;
    l.stage = KT * ((shared ? 1 : 2) * l.krow + l.vrow) * es;
    // the stages also hold the merged O of a segment: [2][rc][Dv] floats
    const int stages = 2 * l.stage > 8 * rc * Dv ? 2 * l.stage : 8 * rc * Dv;
    l.off_q = (stages + 15) / 16 * 16;                          // float [2][rc][dpad]
    l.off_p = l.off_q + 2 * rc * l.dpad * 4;                    // float [KT][weights_row(rc)]
    l.off_stat = l.off_p + KT * weights_row(rc) * 4;                     // float m, l, alpha [2 rc]
    l.total = l.off_stat + 3 * 2 * rc * 4;
    return l;
}

// TWO: value widths above 128 (a thread has two columns).  Without, four blocks an SM, whose
// latencies hide one another: 9 rows a key/value head (4 sequences of up to 8348 keys, 16
// heads, D = 32, float32) take 272 us with two, which 255 registers leave, 151 with four.
template <typename T, int RC, bool TWO, bool X>
__global__ void __launch_bounds__(THREADS, TWO ? 1 : kSimtBlocksPerSm)
paged_simt_kernel(const PagedParams p) {
    constexpr int V = 16 / sizeof(T), PS = weights_row(RC);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int scan[2 * WARPS];
    __shared__ PagedBlock<1> blk;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = p.D, Dv = p.Dv;
    const bool shared = p.k_shared != 0;
    const Layout L = simt_layout(D, Dv, sizeof(T), RC, shared);
    float* qs = reinterpret_cast<float*>(smem + L.off_q);
    float* ps = reinterpret_cast<float*>(smem + L.off_p);
    float* st_m = reinterpret_cast<float*>(smem + L.off_stat);
    float* st_l = st_m + 2 * RC;
    float* st_a = st_l + 2 * RC;
    pdl_wait();                     // before the merging pass may start, which writes too
    pdl_launch_dependents();
    paged_locate<1, X>(p, paged_scan<THREADS, X>(p, KT, EXTRA, scan), KT, EXTRA, 1, p.workers, SNAP, &blk);
    const float lam = paged_lambda<X>(p);

    // output columns of this thread: c0, and c0 + 128 for Dv > 128; its keys: kg, kg + KG, ...
    const int CG = Dv <= 32 ? 32 : Dv <= 64 ? 64 : 128;
    const int KG = THREADS / CG;
    const int c0 = tid % CG, kg = tid / CG;

    PagedCursor<X> cur;
    if (tid == 0) PagedCursor<X>::no_join(p, blockIdx.x);
    for (cur.begin(p, blk, 0, blockIdx.x, KT, EXTRA); !cur.done(); cur.next(p, KT, EXTRA)) {
        const int live = cur.live_tiles(p, KT);
        const int n_new = cur.s.n_new;
        if (tid == 0) cur.join(p, blk.shares, blk.start[1].tile, EXTRA);
        bool bad = cur.s.bad;
        // The page of the row that a thread stages of a tile (four threads a key row), a tile
        // ahead; the first two beside the queries.
        auto look = [&](int tile) -> int {
            const int key = (cur.tile0 + tile) * KT + (tid >> 2);
            return tile < live && key < cur.s.total ? paged_page<X>(p, cur.b, key / p.page) : -2;
        };
        int page = look(0), next = look(1);
        // the rows' queries and state
#pragma unroll
        for (int j0 = 0; j0 < 2 * RC; j0 += WARPS) {
            const int j = j0 + warp, br = j / RC, r = j % RC;      // a warp a row
            if (j >= 2 * RC) break;
            const PagedRow x = paged_row(p, cur.hk, cur.rc, r, n_new);
            const T* src = br ? static_cast<const T*>(p.q2) + cur.b * p.s_q2[0] + x.h * p.s_q2[1] + x.q * p.s_q2[2]
                              : static_cast<const T*>(p.q1) + cur.b * p.s_q1[0] + x.h * p.s_q1[1] + x.q * p.s_q1[2];
            for (int c = lane; c < L.dpad; c += 32) qs[j * L.dpad + c] = x.live && c < D ? to_float<T>(src[c]) : 0.f;
        }
        if (tid < 2 * RC) { st_m[tid] = -INFINITY; st_l[tid] = 0.f; }
        constexpr int COLS = TWO ? 2 : 1;
        float acc[COLS][2][RC];
#pragma unroll
        for (int i = 0; i < COLS; ++i)
#pragma unroll
            for (int r = 0; r < RC; ++r) acc[i][0][r] = acc[i][1][r] = 0.f;

        // A row past the sequence's end or on a page outside the cache is zeros (the latter
        // makes the segment's rows NaN).
        auto stage = [&](int tile, int buf, int page) {
            const int r = tid >> 2, c4 = tid & 3;
            const int key = (cur.tile0 + tile) * KT + r;
            T* k1 = reinterpret_cast<T*>(smem + buf * L.stage) + r * L.krow;
            T* k2 = k1 + KT * L.krow;
            T* v = reinterpret_cast<T*>(smem + buf * L.stage) + (shared ? 1 : 2) * KT * L.krow + r * L.vrow;
            if (page == -1) { bad = true; atomicOr(p.status, kStatusIndex); }
            const int64_t slot = key % p.page;
            const T* g1 = static_cast<const T*>(p.k1) + page * p.s_k1[0] + cur.hk * p.s_k1[1] + slot * p.s_k1[2];
            const T* g2 = static_cast<const T*>(p.k2) + page * p.s_k2[0] + cur.hk * p.s_k2[1] + slot * p.s_k2[2];
            const T* gv = static_cast<const T*>(p.v) + page * p.s_v[0] + cur.hk * p.s_v[1] + slot * p.s_v[2];
            if (page >= 0 && p.vec16) {
                for (int c = c4 * V; c < D; c += 4 * V) {
                    cp_async16(k1 + c, g1 + c);
                    if (!shared) cp_async16(k2 + c, g2 + c);
                }
                for (int c = c4 * V; c < Dv; c += 4 * V) cp_async16(v + c, gv + c);
            } else {
                for (int c = c4; c < L.dpad; c += 4) {
                    k1[c] = page >= 0 && c < D ? g1[c] : T(0.f);
                    if (!shared) k2[c] = page >= 0 && c < D ? g2[c] : T(0.f);
                }
                for (int c = c4; c < L.vrow; c += 4) v[c] = page >= 0 && c < Dv ? gv[c] : T(0.f);
            }
        };
        if (live > 0) stage(0, 0, page);
        cp_async_commit();
        page = next;
        for (int i = 0; i < live; ++i) {
            if (i + 1 < live) stage(i + 1, (i + 1) & 1, page);
            cp_async_commit();
            page = look(i + 2);
            cp_async_wait<1>();
            __syncthreads();
            const T* kt = reinterpret_cast<const T*>(smem + (i & 1) * L.stage);
            const T* vt = kt + (shared ? 1 : 2) * KT * L.krow;
            const int key0 = (cur.tile0 + i) * KT;
            const bool edge = key0 + KT > cur.s.before;      // some row may not see some key
            // ---- scores: key `lane` of branch (warp & 1), rows of half (warp >> 1)
            {
                constexpr int HALF = RC > 1 ? RC / 2 : 1;
                const int br = warp & 1, r0 = (warp >> 1) * HALF;
                if (RC > 1 || warp < 2) {
                    const T* kr = kt + (br && !shared ? KT * L.krow : 0) + lane * L.krow;
                    const float* q = qs + (br * RC + r0) * L.dpad;
                    float s[HALF];
#pragma unroll
                    for (int r = 0; r < HALF; ++r) s[r] = 0.f;
                    for (int c = 0; c < L.dpad; c += V) {
                        float x[V];
                        load16(kr + c, x);
#pragma unroll
                        for (int r = 0; r < HALF; ++r)
#pragma unroll
                            for (int e = 0; e < V; e += 4) {     // four queries a read, the same for all lanes
                                const float4 y = *reinterpret_cast<const float4*>(q + r * L.dpad + c + e);
                                s[r] = fmaf(y.x, x[e], s[r]);
                                s[r] = fmaf(y.y, x[e + 1], s[r]);
                                s[r] = fmaf(y.z, x[e + 2], s[r]);
                                s[r] = fmaf(y.w, x[e + 3], s[r]);
                            }
                    }
#pragma unroll
                    for (int r = 0; r < HALF; ++r) ps[lane * PS + br * RC + r0 + r] = s[r] * p.scale_log2;
                }
            }
            __syncthreads();
            // ---- weights: a warp takes rows (branch, r) warp, warp + 4, ..., all at once: one
            // after another their shuffles' latencies would be most of the tile's time
            {
                constexpr int NJ = (2 * RC + WARPS - 1) / WARPS;
                float s[NJ], top[NJ], w[NJ], sum[NJ], m0[NJ];
                bool seen[NJ];
#pragma unroll
                for (int k = 0; k < NJ; ++k) {
                    const int j = min(warp + k * WARPS, 2 * RC - 1);
                    s[k] = ps[lane * PS + j];
                    seen[k] = true;
                    if (edge) {
                        const PagedRow x = paged_row(p, cur.hk, cur.rc, j % RC, n_new);
                        const int64_t d = key0 + lane - cur.s.before;      // place among the new tokens
                        seen[k] = key0 + lane < cur.s.total && x.live &&
                                  (d < 0 || (p.mask ? p.mask[cur.b * p.mask_stride[0] + x.q * p.mask_stride[1] + d] != 0
                                                    : d <= x.q));
                        if (!seen[k]) s[k] = -INFINITY;
                    }
                    top[k] = s[k];
                    m0[k] = st_m[j];
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                    for (int k = 0; k < NJ; ++k) top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], o));
#pragma unroll
                for (int k = 0; k < NJ; ++k) {
                    top[k] = fmaxf(m0[k], top[k]);
                    w[k] = s[k] == -INFINITY ? 0.f : exp2f(s[k] - top[k]);   // NaN scores stay NaN
                    sum[k] = w[k];
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                    for (int k = 0; k < NJ; ++k) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
                __syncwarp();
#pragma unroll
                for (int k = 0; k < NJ; ++k) {
                    const int j = warp + k * WARPS;
                    if (j >= 2 * RC) break;
                    ps[lane * PS + j] = seen[k] ? w[k] : -1.f;
                    if (lane == 0) {
                        const float a = m0[k] == top[k] ? 1.f : exp2f(m0[k] - top[k]);
                        st_m[j] = top[k];
                        st_l[j] = st_l[j] * a + sum[k];
                        st_a[j] = a;
                    }
                }
            }
            __syncthreads();
            // ---- O = alpha O + P V
            if (c0 < Dv) {
#pragma unroll
                for (int r = 0; r < RC; ++r) {
                    const float a1 = st_a[r], a2 = st_a[RC + r];
#pragma unroll
                    for (int i = 0; i < COLS; ++i) {
                        acc[i][0][r] *= a1;
                        acc[i][1][r] *= a2;
                    }
                }
                const bool second = TWO && c0 + 128 < Dv;
                auto value = [&](int t, float (&x)[COLS], float (&w)[2 * RC]) {
                    x[0] = to_float<T>(vt[t * L.vrow + c0]);
                    if constexpr (TWO) x[1] = second ? to_float<T>(vt[t * L.vrow + c0 + 128]) : 0.f;
                    if constexpr (RC > 1) {
#pragma unroll
                        for (int r = 0; r < 2 * RC; r += 4)
                            *reinterpret_cast<float4*>(w + r) = *reinterpret_cast<const float4*>(ps + t * PS + r);
                    } else {
                        w[0] = ps[t * PS];
                        w[1] = ps[t * PS + 1];
                    }
                };
                if (!edge) {
                    // two keys at a time, so that one's reads pass while the other's are used
#pragma unroll 2
                    for (int t = kg; t < KT; t += KG) {
                        float x[COLS], w[2 * RC];
                        value(t, x, w);
#pragma unroll
                        for (int i = 0; i < COLS; ++i)
#pragma unroll
                            for (int r = 0; r < RC; ++r) {
                                acc[i][0][r] = fmaf(w[r], x[i], acc[i][0][r]);
                                acc[i][1][r] = fmaf(w[RC + r], x[i], acc[i][1][r]);
                            }
                    }
                } else {
#pragma unroll 1
                    for (int t = kg; t < KT; t += KG) {
                        float x[COLS], w[2 * RC];
                        value(t, x, w);
#pragma unroll
                        for (int r = 0; r < RC; ++r) {
                            if (w[r] < 0.f) continue;               // hidden
#pragma unroll
                            for (int i = 0; i < COLS; ++i) {
                                acc[i][0][r] = fmaf(w[r], x[i], acc[i][0][r]);
                                acc[i][1][r] = fmaf(w[RC + r], x[i], acc[i][1][r]);
                            }
                        }
                    }
                }
            }
            __syncthreads();        // the stage and the weights are free again
        }
        bad = __syncthreads_or(bad);
        cp_async_wait<0>();
        __syncthreads();
        // ---- the key groups' sums, in order, then the rows out
        float* om = reinterpret_cast<float*>(smem);         // [2][RC][Dv]
        for (int k = 0; k < KG; ++k) {
            if (kg == k && c0 < Dv) {
#pragma unroll
                for (int r = 0; r < RC; ++r)
#pragma unroll
                    for (int br = 0; br < 2; ++br) {
                        float* o = om + (br * RC + r) * Dv + c0;
                        o[0] = k ? o[0] + acc[0][br][r] : acc[0][br][r];
                        if constexpr (TWO)                                      // one key group then
                            if (c0 + 128 < Dv) o[128] = acc[1][br][r];
                    }
            }
            __syncthreads();
        }
        const int stride = paged_part_floats(Dv), width = paged_part_width(Dv);
        for (int r = warp; r < RC; r += WARPS) {
            const PagedRow x = paged_row(p, cur.hk, cur.rc, r, n_new);
            if (!x.live) continue;
            const float l1 = bad ? __int_as_float(0x7fc00000) : st_l[r];
            const float l2 = bad ? __int_as_float(0x7fc00000) : st_l[RC + r];
            if (cur.whole()) {
                float o1[8], o2[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = lane + 32 * j;
                    o1[j] = c < Dv ? om[r * Dv + c] : 0.f;
                    o2[j] = c < Dv ? om[(RC + r) * Dv + c] : 0.f;
                }
                paged_finish_row<8>(p, lam, cur.b, x.h, x.q, lane, o1, l1, o2, l2);
            } else {
                float* part = p.part + ((int64_t)cur.slot() * p.chunk_rows + r) * stride;
                if (lane == 0) {
                    part[0] = st_m[r];
                    part[1] = l1;
                    part[2] = st_m[RC + r];
                    part[3] = l2;
                }
                for (int c = lane; c < Dv; c += 32) {
                    part[4 + c] = om[r * Dv + c];
                    part[4 + width + c] = om[(RC + r) * Dv + c];
                }
            }
        }
        if (cur.s.bad && tid == 0) atomicOr(p.status, kStatusIndex);
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Merging pass: the units that workers c of the first pass started and did not finish.
// With partial maxima m_i (log2 units), sums l_i and O_i:
//     M = max m_i,  l = sum 2^(m_i - M) l_i,  O = sum 2^(m_i - M) O_i.
// A row is taken by one warp, or with many parts (a long sequence over many blocks) by
// two, four or all eight, each adding its share of them: the time is the latency of
// reading the parts from L2, which then overlap.  The order of the sums is fixed.
// ---------------------------------------------------------------------------
constexpr int C_WARPS = 8;
constexpr int kJoinsPerBlock = 4;

// Zeros for the rows past a sequence's queries, a warp a row.
__device__ __forceinline__ void zero_rest(const PagedParams& p, int warp, int warps, int lane) {
    const int64_t rows = (int64_t)p.B * p.H * p.Tq;
    for (int64_t i = warp; i < rows; i += warps) {
        const int64_t bh = i / p.Tq;
        const int q = (int)(i - bh * p.Tq), b = (int)(bh / p.H), h = (int)(bh - (int64_t)b * p.H);
        if (q < paged_seq<false>(p, b).n_new) continue;
        const int64_t at = b * p.s_o[0] + h * p.s_o[1] + q * p.s_o[2];
        for (int c = lane; c < p.Dv; c += 32) {
            if (p.bf16) static_cast<__nv_bfloat16*>(p.out)[at + c] = __float2bfloat16_rn(0.f);
            else static_cast<float*>(p.out)[at + c] = 0.f;
        }
    }
}

// J columns a lane; VEC: J = 4 of them in a row, for a value width of 128 in bf16 (two
// 16-byte reads a part instead of eight of 4 bytes).  AHEAD: parts read at once.  Four for
// units of up to 16 rows, which may have many parts and leave the SMs empty (one sequence
// of 517 keys: 14.1 us in all with two, 13.2 with four); two for those of 128, whose rows
// want the warps that fewer registers allow (61 tokens over 16 x 8192: 117.5, 118.2 with four).
template <int J, bool VEC, int AHEAD, bool X>
__global__ void __launch_bounds__(C_WARPS * 32, J > 4 ? 2 : AHEAD > 2 ? 3 : 4)
paged_combine_kernel(const PagedParams p) {
    __shared__ float share[C_WARPS][2 * 32 * J];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    // before the first pass is over: it does not touch these rows
    if (!X && p.zero_rest)
        zero_rest(p, (blockIdx.y * gridDim.x + blockIdx.x) * C_WARPS + warp, gridDim.x * gridDim.y * C_WARPS, lane);
    pdl_wait();
    const float lam = paged_lambda<X>(p);
    const int stride = paged_part_floats(p.Dv), width = paged_part_width(p.Dv);
    // the words of this block's workers, all at once: most of them say that there is nothing
    int4 joins[kJoinsPerBlock];
#pragma unroll
    for (int k = 0; k < kJoinsPerBlock; ++k) {
        const int c = blockIdx.x * p.join_block + k * p.join_step;
        joins[k] = c < p.workers ? *reinterpret_cast<const int4*>(p.joins + c) : make_int4(0, 0, 0, 0);
    }
#pragma unroll 1
    for (int k = 0; k < kJoinsPerBlock; ++k) {
        const int c = blockIdx.x * p.join_block + k * p.join_step;
        const int4 join = k == 0 ? joins[0] : k == 1 ? joins[1] : k == 2 ? joins[2] : joins[3];
        const int parts = join.x, b = join.y, unit = join.z, n_new = join.w;
        if (parts == 0) continue;
        const int hk = unit / p.row_chunks, rc = unit - hk * p.row_chunks;
        const int W = parts <= 4 ? 1 : parts <= 8 ? 2 : parts <= 16 ? 4 : C_WARPS;
        const int sub = warp % W;
        const int step = gridDim.y * (C_WARPS / W);
        for (int r0 = blockIdx.y * (C_WARPS / W); r0 < p.chunk_rows; r0 += step) {
            const int r = r0 + warp / W;
            const PagedRow x = paged_row(p, hk, rc, r, n_new);
            const bool live = x.live && r < p.chunk_rows;
            auto part_of = [&](int i) {
                const int64_t slot = i == 0 ? 2 * c + 1 : 2 * (c + i);
                return p.part + (slot * p.chunk_rows + r) * stride;
            };
            float o[2][J], l[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < J; ++j) o[0][j] = o[1][j] = 0.f;
            if (live) {
                // Loads first, and all that fit: the pass is the latency of L2, met once if
                // no load waits for another's value.  So no branch on a weight either (a
                // part that saw nothing holds zeros).
                float4 v[AHEAD][2][(J + 3) / 4];
                float4 st[AHEAD];
                auto load = [&](int i, int k) {
                    const float* src = part_of(min(i, parts - 1));
                    st[k] = *reinterpret_cast<const float4*>(src);
#pragma unroll
                    for (int br = 0; br < 2; ++br) {
                        const float* at = src + 4 + br * width;
                        if constexpr (VEC) {
                            v[k][br][0] = *reinterpret_cast<const float4*>(at + 4 * lane);
                        } else {
                            float* f = reinterpret_cast<float*>(v[k][br]);
#pragma unroll
                            for (int j = 0; j < J; ++j) f[j] = at[min(lane + 32 * j, p.Dv - 1)];
                        }
                    }
                };
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) load(sub + k * W, k);
                float m[2], m1, m2;
                // where nothing was seen m_i is -inf, and l_i 0 (or NaN: a bad page) as it is
                auto add_l = [&](float4 s4) {
                    l[0] += s4.y * (s4.x == -INFINITY ? 1.f : exp2f(s4.x - m1));
                    l[1] += s4.w * (s4.z == -INFINITY ? 1.f : exp2f(s4.z - m2));
                };
                if (parts == 2) {               // the most common: every lane has both
                    m[0] = fmaxf(st[0].x, st[1].x);
                    m[1] = fmaxf(st[0].z, st[1].z);
                    m1 = m[0] == -INFINITY ? 0.f : m[0];
                    m2 = m[1] == -INFINITY ? 0.f : m[1];
                    add_l(st[0]);
                    add_l(st[1]);
                } else {
                    const float4 own = *reinterpret_cast<const float4*>(part_of(min(lane, parts - 1)));
                    m[0] = own.x;
                    m[1] = own.z;
                    for (int i = lane + 32; i < parts; i += 32) {
                        const float4 s4 = *reinterpret_cast<const float4*>(part_of(i));
                        m[0] = fmaxf(m[0], s4.x);
                        m[1] = fmaxf(m[1], s4.z);
                    }
#pragma unroll
                    for (int k = 16; k > 0; k >>= 1) {
                        m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], k));
                        m[1] = fmaxf(m[1], __shfl_xor_sync(0xffffffffu, m[1], k));
                    }
                    m1 = m[0] == -INFINITY ? 0.f : m[0];
                    m2 = m[1] == -INFINITY ? 0.f : m[1];
                    for (int i = lane; i < parts; i += 32)
                        add_l(i < 32 ? own : *reinterpret_cast<const float4*>(part_of(i)));
#pragma unroll
                    for (int k = 16; k > 0; k >>= 1) {
                        l[0] += __shfl_xor_sync(0xffffffffu, l[0], k);
                        l[1] += __shfl_xor_sync(0xffffffffu, l[1], k);
                    }
                }
                for (int i = sub; i < parts; i += AHEAD * W) {
                    if (i > sub) {
#pragma unroll
                        for (int k = 0; k < AHEAD; ++k) load(i + k * W, k);
                    }
#pragma unroll
                    for (int k = 0; k < AHEAD; ++k) {
                        if (i + k * W >= parts) continue;
                        const float w[2] = {exp2f(st[k].x - m1), exp2f(st[k].z - m2)};
#pragma unroll
                        for (int br = 0; br < 2; ++br) {
                            const float* f = reinterpret_cast<const float*>(v[k][br]);
#pragma unroll
                            for (int j = 0; j < J; ++j) o[br][j] = fmaf(w[br], f[j], o[br][j]);
                        }
                    }
                }
            }
            if (W > 1) {
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    share[warp][32 * j + lane] = o[0][j];
                    share[warp][32 * (J + j) + lane] = o[1][j];
                }
                __syncthreads();
                if (sub == 0)
                    for (int w = 1; w < W; ++w)
#pragma unroll
                        for (int j = 0; j < J; ++j) {
                            o[0][j] += share[warp + w][32 * j + lane];
                            o[1][j] += share[warp + w][32 * (J + j) + lane];
                        }
            }
            if (live && sub == 0) paged_finish_row<J, VEC>(p, lam, b, x.h, x.q, lane, o[0], l[0], o[1], l[1]);
            if (W > 1) __syncthreads();
        }
    }
}

template <bool X>
auto combine_kernel(const PagedParams& p, int most) {
    return p.Dv == 128 && p.bf16 ? (most > 16 ? paged_combine_kernel<4, true, 2, X> : paged_combine_kernel<4, true, 4, X>)
           : p.Dv <= 128         ? paged_combine_kernel<4, false, 4, X>
                                 : paged_combine_kernel<8, false, 2, X>;
}

template <typename T, int RC>
int launch_rc(const PagedParams& p, cudaStream_t stream) {
    const Layout L = simt_layout(p.D, p.Dv, sizeof(T), RC, p.k_shared != 0);
    const auto kernel = p.cross ? (p.Dv > 128 ? paged_simt_kernel<T, RC, true, true> : paged_simt_kernel<T, RC, false, true>)
                        : p.Dv > 128 ? paged_simt_kernel<T, RC, true, false>
                                     : paged_simt_kernel<T, RC, false, false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L.total) != cudaSuccess) return -1;
    return pdl_launch(kernel, dim3(p.workers), THREADS, L.total, stream, p);
}

template <typename T>
int launch_t(const PagedParams& p, cudaStream_t stream) {
    switch (p.chunk_rows) {
        case 1: return launch_rc<T, 1>(p, stream);
        case 2: return launch_rc<T, 2>(p, stream);
        case 4: return launch_rc<T, 4>(p, stream);
        case 6: return launch_rc<T, 6>(p, stream);
        case 8: return launch_rc<T, 8>(p, stream);
        case 12: return launch_rc<T, 12>(p, stream);
        case 16: return launch_rc<T, 16>(p, stream);
        default: return -1;
    }
}

}  // namespace paged

int paged_simt_rows(int64_t rows) {
    for (int r : {1, 2, 4, 6, 8, 12})
        if (rows <= r) return r;
    return paged::MAX_RC;
}

int paged_simt_blocks(int D, int Dv, int es, int rows) {
    const int fit = 227 * 1024 / (paged::simt_layout(D, Dv, es, rows, false).total + 1024 + 256);
    const int most = Dv > 128 ? 2 : kSimtBlocksPerSm;
    return fit < 1 ? 1 : fit < most ? fit : most;
}

int launch_paged_combine(const PagedParams& params, cudaStream_t stream) {
    PagedParams p = params;
    // At most every unit is shared, and a block whose words say that there is nothing still
    // costs its launch: with 16 units of 456 workers, 3648 blocks took 13 us, 912 take 7.
    // So a block reads four words in a row where the units are fewer than the workers' quarter,
    // and four far apart where three quarters of the workers may not exist (paged_mma.cu, whose
    // warps are workers by themselves only where the units are many).
    const int64_t units = (int64_t)p.B * p.Hk * p.row_chunks;
    const bool sparse = p.sparse_joins && 2 * units >= p.solo_workers;
    if (p.sparse_joins && !sparse) p.workers /= kMmaWarps;
    const int words = sparse || 4 * units <= p.workers ? paged::kJoinsPerBlock : 1;
    const int blocks = (p.workers + words - 1) / words;
    p.join_block = sparse ? 1 : words;
    p.join_step = sparse ? blocks : words > 1 ? 1 : p.workers;
    // Along the rows: a block a row where all blocks fit at once (few units, which may have
    // many parts: then all of a block's warps share a row's), at least a row a warp.  One unit
    // of 24 rows in 152 parts: 74 us in all with three blocks, 25 with 24.
    const int joins = (int)(units < p.workers ? units : p.workers), fit = p.solo_workers / 2;
    const int most = p.chunk_rows, least = most <= 16 ? most : (most + paged::C_WARPS - 1) / paged::C_WARPS;
    const int rows = fit / joins < least ? least : fit / joins > most ? most : fit / joins;
    const auto kernel = p.cross ? paged::combine_kernel<true>(p, most) : paged::combine_kernel<false>(p, most);
    return pdl_launch(kernel, dim3((unsigned)blocks, (unsigned)rows), paged::C_WARPS * 32, 0, stream, p);
}

int launch_paged_simt(const PagedParams& p, cudaStream_t stream) {
    const int rc = p.bf16 ? paged::launch_t<__nv_bfloat16>(p, stream) : paged::launch_t<float>(p, stream);
    return rc == 0 ? launch_paged_combine(p, stream) : rc;
}

}  // namespace diffattn
