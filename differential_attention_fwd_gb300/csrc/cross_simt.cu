// cross_simt.cu -- differential attention over an encoder's states on the CUDA cores,
// forward and backward: any D <= 128 and Dv <= 256, float32 (exact float32 arithmetic) and
// bf16, any layout.  Sequence b has its first n_b of Tk states.
//
//     S_b = Q_b K_b^T / sqrt(D) over the n states,  A_b = softmax(S_b)
//     O   = (A_1 - lambda A_2) V                    (a row with no state: 0)
//     dP  = dO V^T,   Dd_b = rowsum(A_b dP)
//     dS_1 = A_1 (dP - Dd_1),  dS_2 = -lambda A_2 (dP - Dd_2)
//     dQ_b = dS_b K_b / sqrt(D),  dK_b = dS_b^T Q_b / sqrt(D),  dV = (A_1 - lambda A_2)^T dO
//     dlambda = -sum Dd_2
//
// Blocks of 256 threads work on tiles of 32 query rows and 32 states in shared memory, in
// float32: the forward and the dQ kernel walk the states for 32 rows of a head, the dK/dV
// kernel walks the rows of every query head of its key/value head for 32 states.  A
// thread's part of each product is a small tile of registers (2 x 4 scores; 2 x 4 to 8 x 4
// of an output), so that a float4 read of shared memory feeds 5 to 10 multiplications.
// What lies behind a sequence's states is never read: those rows of the tiles are zeros,
// and their weights 0.
//
// Bound by the reads of shared memory that feed the products: 16 x 16 heads of 64, 512 rows over
// 1500 states, bf16: 6.4 ms, 23.5 TFLOP/s (the tensor cores take 0.12 ms).  Small calls are chains
// of latencies: 3 x 6 over 3 heads of 32, float32, 77 rows over 129 states: forward 19.7 us, dQ 19.6, dK
// and dV 41.3.
//
// Dd comes from the forward's saved results in float32 (Dd_2 = dO . (A_2 V), Dd_1 = dO .
// (O + lambda A_2 V)); in bf16 their rounding would stay in every dS of the row, so the dQ
// kernel walks the states twice and sums A_b dP first.
#include "block.h"
#include "kernels.h"
#include "pdl.cuh"
#include "rows.cuh"

#include <cmath>

namespace diffattn {
namespace xsimt {

constexpr int THREADS = 256;
constexpr int BM = 32;          // query rows of a tile
constexpr int BN = 32;          // states of a tile
constexpr int LP = BM + 4;      // row stride of the score tiles
// Stages of the operands that a block walks: float32 tiles arrive while the last is worked on.
template <typename T>
constexpr int STAGES = sizeof(T) == 4 ? 2 : 1;

// Sizes by class: 0: D <= 32, Dv <= 64; 1: D <= 64, Dv <= 128; 2: D <= 128, Dv <= 256.
template <int S>
struct Size {
    static constexpr int D = 32 << S, DV = 64 << S;
    // products of width Dv over all threads: CV threads of NV float4 columns, RV rows each
    static constexpr int CV = S == 0 ? 16 : 32, NV = DV / 4 / CV, RV = BM / (THREADS / CV);
    // products of width D, a branch on each half: CD threads of a float4, RD rows each
    static constexpr int CD = D / 4, RD = BM / (THREADS / 2 / CD);
};

__host__ __device__ constexpr int padded(int n) { return (n + 3) / 4 * 4 + 4; }

// 4 or 16 bytes from global to shared memory by cp.async, or zeros.
template <int BYTES>
__device__ __forceinline__ void async_copy(float* dst, const void* src, bool there) {
    const int n = there ? BYTES : 0;
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// `count` rows of `width` elements into 32 rows of `ld` floats; the other rows, and the columns
// up to 4 past the width's multiple of 4, are zeros.  float32 goes by cp.async, so that a tile
// arrives while the last one is worked on (async_wait, then a barrier); bf16 through registers,
// four pieces of a row at a time.  vec: rows of whole 16-byte pieces on 16-byte boundaries.
template <typename T>
__device__ __forceinline__ void load_rows(float* dst, int ld, const T* src, int64_t stride, int count, int width, bool vec) {
    constexpr int V = 16 / sizeof(T);
    const int step = vec ? V : 1, pieces = width / step;
    // lanes of a row: a power of two, as many as it has pieces, 32 at most
    const int lanes = pieces > 16 ? 32 : pieces > 8 ? 16 : pieces > 4 ? 8 : 4;
    const int sub = threadIdx.x & (lanes - 1);
    const int rows = THREADS / lanes;
    if constexpr (sizeof(T) == 4) {
        for (int r = threadIdx.x / lanes; r < 32; r += rows) {
            const T* row = src + (int64_t)(r < count ? r : 0) * stride;
            for (int c = sub; c < pieces; c += lanes) {
                if (vec) async_copy<16>(dst + r * ld + 4 * c, row + 4 * c, r < count);
                else async_copy<4>(dst + r * ld + c, row + c, r < count);
            }
            for (int c = width + sub; c < ld; c += lanes) dst[r * ld + c] = 0.f;
        }
    } else {
        for (int r = threadIdx.x / lanes; r < 32; r += rows) {
            const T* row = src + (int64_t)(r < count ? r : 0) * stride;
            float* to = dst + r * ld;
            for (int c0 = sub; c0 < pieces; c0 += 4 * lanes) {
                if (vec) {
                    uint4 x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[i] = r < count && c0 + i * lanes < pieces ? *reinterpret_cast<const uint4*>(row + V * (c0 + i * lanes))
                                                                   : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (c0 + i * lanes >= pieces) break;
                        uint64_t f[4];
                        Vec<__nv_bfloat16>::unpack(x[i], f);
                        float4* at = reinterpret_cast<float4*>(to + V * (c0 + i * lanes));
                        at[0] = make_float4(f2_lo(f[0]), f2_hi(f[0]), f2_lo(f[1]), f2_hi(f[1]));
                        at[1] = make_float4(f2_lo(f[2]), f2_hi(f[2]), f2_lo(f[3]), f2_hi(f[3]));
                    }
                } else {
                    float x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[i] = r < count && c0 + i * lanes < pieces ? Vec<T>::get(row[c0 + i * lanes]) : 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c0 + i * lanes < pieces) to[c0 + i * lanes] = x[i];
                }
            }
            for (int c = width + sub; c < ld; c += lanes) to[c] = 0.f;
        }
    }
}

// Whether rows of this width, base and strides are whole 16-byte pieces.
template <typename T>
__device__ __forceinline__ bool pieces16(const void* p, const int64_t (&s)[3], int width) {
    return ((reinterpret_cast<uintptr_t>(p) | (uint64_t)(s[0] * sizeof(T)) | (uint64_t)(s[1] * sizeof(T)) |
             (uint64_t)(s[2] * sizeof(T)) | (uint64_t)(width * sizeof(T))) & 15) == 0;
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float s) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s))));
}

// Scores of both branches, branch b by half b of the block: dst[branch] is [state][row]
// where `by_state`, else [row][state].
__device__ __forceinline__ void scores(const float* q, const float* k, int ld, int D, float* dst, bool by_state) {
    const int br = threadIdx.x >> 7, t = threadIdx.x & 127, r = t >> 3, c = t & 7;
    q += br * BM * ld;
    k += br * BN * ld;
    float s[2][4] = {};
    for (int d = 0; d < D; d += 4) {
        float4 x[2], y[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) x[i] = *reinterpret_cast<const float4*>(q + (r + 16 * i) * ld + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(k + (c + 8 * j) * ld + d);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = dot4(x[i], y[j], s[i][j]);
    }
    dst += br * BN * LP;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = r + 16 * i, key = c + 8 * j;
            dst[by_state ? key * LP + row : row * LP + key] = s[i][j];
        }
}

// dO V^T of a tile by the whole block, laid out as scores'.
__device__ __forceinline__ void products(const float* g, const float* v, int ld, int Dv, float* dst, bool by_state) {
    const int r = threadIdx.x >> 4, c = threadIdx.x & 15;
    float s[2][2] = {};
    for (int d = 0; d < Dv; d += 4) {
        float4 x[2], y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[i] = *reinterpret_cast<const float4*>(g + (r + 16 * i) * ld + d);
            y[i] = *reinterpret_cast<const float4*>(v + (c + 16 * i) * ld + d);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) s[i][j] = dot4(x[i], y[j], s[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = r + 16 * i, key = c + 16 * j;
            dst[by_state ? key * LP + row : row * LP + key] = s[i][j];
        }
}

// acc[i][n] += sum over k < 32 of w[k][r0 + i] x[k][columns of n], w with rows of LP.
template <int R, int N>
__device__ __forceinline__ void accumulate(const float* w, int r0, const float* x, int ld, int c0, int step, int width,
                                           float4 (&acc)[R][N]) {
    static_assert(R == 2 || R % 4 == 0, "rows of a thread");
#pragma unroll 4
    for (int k = 0; k < 32; ++k) {
        float a[R];
        if constexpr (R == 2) {
            const float2 t = *reinterpret_cast<const float2*>(w + k * LP + r0);
            a[0] = t.x;
            a[1] = t.y;
        } else {
#pragma unroll
            for (int i = 0; i < R; i += 4) {
                const float4 t = *reinterpret_cast<const float4*>(w + k * LP + r0 + i);
                a[i] = t.x;
                a[i + 1] = t.y;
                a[i + 2] = t.z;
                a[i + 3] = t.w;
            }
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if (c0 + n * step >= width) break;
            const float4 y = *reinterpret_cast<const float4*>(x + k * ld + c0 + n * step);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                acc[i][n].x = fmaf(a[i], y.x, acc[i][n].x);
                acc[i][n].y = fmaf(a[i], y.y, acc[i][n].y);
                acc[i][n].z = fmaf(a[i], y.z, acc[i][n].z);
                acc[i][n].w = fmaf(a[i], y.w, acc[i][n].w);
            }
        }
    }
}

// Four columns of a dense or strided row, as many as there are.
template <typename T>
__device__ __forceinline__ void put4(T* row, int c, int width, float4 x, float s) {
    const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (c + i < width) row[c + i] = Vec<T>::put(v[i] * s);
}

// What the rounding to T leaves.
template <typename T>
__device__ __forceinline__ float4 left(float4 x) {
    const auto f = [](float v) { return v - Vec<T>::get(Vec<T>::put(v)); };
    return make_float4(f(x.x), f(x.y), f(x.z), f(x.w));
}

// A block's 32 query rows: batch, head, key/value head and first row.
struct Rows {
    int b, h, hk, q0, count;
};
__device__ __forceinline__ Rows rows_of(const CrossParams& p) {
    const int tiles = (p.Tq + BM - 1) / BM;
    const int bh = blockIdx.x / tiles;
    Rows r;
    r.b = bh / p.H;
    r.h = bh - r.b * p.H;
    r.hk = r.h / p.group;
    r.q0 = (blockIdx.x - bh * tiles) * BM;
    r.count = min(BM, p.Tq - r.q0);
    return r;
}

// A head's rows in global memory, and how they are read.
template <typename T>
struct Source {
    const T* at;
    int64_t stride;
    int width;
    bool vec;
    __device__ __forceinline__ Source(const void* x, const int64_t (&s)[3], int b, int h, int w)
        : at(static_cast<const T*>(x) + b * s[0] + h * s[1]), stride(s[2]), width(w), vec(pieces16<T>(x, s, w)) {}
    __device__ __forceinline__ void load(float* dst, int ld, int row, int count) const {
        load_rows(dst, ld, at + row * stride, stride, count, width, vec);
    }
};

// A sequence's states, tile by tile.
template <typename T>
struct States {
    Source<T> k1, k2, v;
    int n, ld, lv;
    __device__ __forceinline__ States(const CrossParams& p, int b, int hk, int n_, int ld_, int lv_)
        : k1(p.k1, p.s_k1, b, hk, p.D), k2(p.k2, p.s_k2, b, hk, p.D), v(p.v, p.s_v, b, hk, p.Dv), n(n_), ld(ld_), lv(lv_) {}
    __device__ __forceinline__ void fetch(float* to, int k0) const {
        const int live = min(BN, n - k0);
        k1.load(to, ld, k0, live);
        k2.load(to + BN * ld, ld, k0, live);
        v.load(to + 2 * BN * ld, lv, k0, live);
        async_commit();
    }
    // Before the first tile, and for each: where tile k0 is, with the next one on its way.
    __device__ __forceinline__ void begin(float* kv) const {
        if (STAGES<T> == 2) fetch(kv, 0);
    }
    __device__ __forceinline__ float* next(float* kv, int stage, int k0) const {
        if (STAGES<T> == 1) {
            __syncthreads();                    // the last tile has been read
            fetch(kv, k0);
            __syncthreads();
            return kv;
        }
        const int now = (k0 / BN) & 1;
        async_wait();
        __syncthreads();                        // the tile is there, and the last one has been read
        if (k0 + BN < n) fetch(kv + (now ^ 1) * stage, k0 + BN);
        return kv + now * stage;
    }
};

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <typename T, int S>
__global__ void __launch_bounds__(THREADS)
cross_fwd_kernel(const CrossParams p) {
    using Z = Size<S>;
    extern __shared__ __align__(16) float sm[];
    const int ld = padded(p.D), lv = padded(p.Dv);
    float* qs = sm;                             // [branch][row][ld]
    float* kv = qs + 2 * BM * ld;               // [stage]: keys [branch][state][ld], values [state][lv]
    const int stage = 2 * BN * ld + BN * lv;
    float* ps = kv + STAGES<T> * stage;         // [branch][state][LP]
    float* fix = ps + 2 * BN * LP;              // [branch][row]: the tile's rescaling, then 1 / l
    pdl_wait();
    pdl_launch_dependents();
    const Rows r = rows_of(p);
    const CrossLen len = cross_len(p.lengths, r.b, p.Tk);
    if (len.bad && threadIdx.x == 0) atomicOr(p.status, kStatusIndex);
    Source<T>(p.q1, p.s_q1, r.b, r.h, p.D).load(qs, ld, r.q0, r.count);
    Source<T>(p.q2, p.s_q2, r.b, r.h, p.D).load(qs + BM * ld, ld, r.q0, r.count);
    // the softmax: four threads a row and branch
    const int br = threadIdx.x >> 7, row = (threadIdx.x >> 2) & 31, sub = threadIdx.x & 3;
    float m = -INFINITY, l = 0.f;
    // the output: RV rows by NV float4 columns a thread
    const int r0 = threadIdx.x / Z::CV * Z::RV, c0 = threadIdx.x % Z::CV * 4;
    float4 o1[Z::RV][Z::NV] = {}, o2[Z::RV][Z::NV] = {};
    const States<T> states(p, r.b, r.hk, len.n, ld, lv);
    if (len.n > 0) states.begin(kv);
    for (int k0 = 0; k0 < len.n; k0 += BN) {
        const int live = min(BN, len.n - k0);
        const float* ks = states.next(kv, stage, k0);
        const float* vs = ks + 2 * BN * ld;
        scores(qs, ks, ld, p.D, ps, true);
        __syncthreads();
        {
            float* w = ps + br * BN * LP + row;
            float s[8], top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[j] = sub + 4 * j < live ? w[(sub + 4 * j) * LP] * p.scale : -INFINITY;
                top = fmaxf(top, s[j]);
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float next = fmaxf(m, top);
            const float base = next == -INFINITY ? 0.f : next;      // every score so far is -inf
            const float a = expf(m - base);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[j] = sub + 4 * j < live ? expf(s[j] - base) : 0.f;
                sum += s[j];
                w[(sub + 4 * j) * LP] = s[j];
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            l = l * a + sum;
            m = next;
            if (sub == 0) fix[br * BM + row] = a;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < Z::RV; ++i) {
            const float a1 = fix[r0 + i], a2 = fix[BM + r0 + i];
#pragma unroll
            for (int n = 0; n < Z::NV; ++n) {
                o1[i][n].x *= a1; o1[i][n].y *= a1; o1[i][n].z *= a1; o1[i][n].w *= a1;
                o2[i][n].x *= a2; o2[i][n].y *= a2; o2[i][n].z *= a2; o2[i][n].w *= a2;
            }
        }
        accumulate<Z::RV, Z::NV>(ps, r0, vs, lv, c0, 4 * Z::CV, p.Dv, o1);
        accumulate<Z::RV, Z::NV>(ps + BN * LP, r0, vs, lv, c0, 4 * Z::CV, p.Dv, o2);
    }
    async_wait();                               // (the queries, where there was no state)
    __syncthreads();
    const float nan = __int_as_float(0x7fc00000);
    if (sub == 0) {
        fix[br * BM + row] = len.bad ? nan : l == 0.f ? 0.f : 1.0f / l;      // no weight at all: 0
        if (p.lse && row < r.count)
            p.lse[(((int64_t)r.b * p.H + r.h) * p.Tq + r.q0 + row) * 2 + br] = len.bad ? nan : m + logf(l);
    }
    __syncthreads();
    const float lam = lambda_of(p.lambda_dev, p.lambda_bf16, p.lambda);
    T* out2 = p.out2 ? static_cast<T*>(p.out2) + r.b * p.s_o[0] + r.h * p.s_o[1] + r.q0 * p.s_o[2] : nullptr;
    // dense rows of what the roundings of O and A_2 V leave
    T* rest = p.rests ? static_cast<T*>(p.rests) + (((int64_t)r.b * p.H + r.h) * p.Tq + r.q0) * p.Dv : nullptr;
    T* rest2 = rest + (int64_t)p.B * p.H * p.Tq * p.Dv;
#pragma unroll
    for (int i = 0; i < Z::RV; ++i) {
        const float i1 = fix[r0 + i], i2 = fix[BM + r0 + i];
#pragma unroll
        for (int n = 0; n < Z::NV; ++n) {
            const int c = c0 + n * 4 * Z::CV;
            if (c >= p.Dv) break;
            const float4 x = o1[i][n], y = o2[i][n];
            const float4 b = make_float4(__fmul_rn(y.x, i2), __fmul_rn(y.y, i2), __fmul_rn(y.z, i2), __fmul_rn(y.w, i2));
            // the branches rounded alike, so that alike branches cancel exactly at lambda = 1
            *reinterpret_cast<float4*>(kv + (r0 + i) * lv + c) =
                make_float4(fmaf(-lam, b.x, __fmul_rn(x.x, i1)), fmaf(-lam, b.y, __fmul_rn(x.y, i1)),
                            fmaf(-lam, b.z, __fmul_rn(x.z, i1)), fmaf(-lam, b.w, __fmul_rn(x.w, i1)));
            if (out2 && r0 + i < r.count) put4(out2 + (r0 + i) * p.s_o[2], c, p.Dv, b, 1.f);
            if (rest && r0 + i < r.count) put4(rest2 + (int64_t)(r0 + i) * p.Dv, c, p.Dv, left<T>(b), 1.f);
        }
    }
    __syncthreads();
    // the epilogue, a warp a row
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = warp; i < r.count; i += THREADS / 32) {
        const float* y = kv + i * lv;
        float mu = 0.f, rs = 1.f;
        if (p.norm != kNormNone) {
            if (p.norm == kNormGroup) {
                float sum = 0.f;
                for (int c = lane; c < p.Dv; c += 32) sum += y[c];
                mu = group_sum<32>(sum) / p.Dv;
            }
            float ss = 0.f;
            for (int c = lane; c < p.Dv; c += 32) ss = fmaf(y[c] - mu, y[c] - mu, ss);
            rs = 1.0f / sqrtf(group_sum<32>(ss) / p.Dv + p.norm_eps);
        }
        T* dst = static_cast<T*>(p.out) + r.b * p.s_o[0] + r.h * p.s_o[1] + (r.q0 + i) * p.s_o[2];
        for (int c = lane; c < p.Dv; c += 32) {
            float x = (y[c] - mu) * rs;
            if (p.norm_weight) x *= __ldg(p.norm_weight + (int64_t)r.h * p.Dv + c);
            if (p.norm_bias) x += __ldg(p.norm_bias + (int64_t)r.h * p.Dv + c);
            dst[c] = Vec<T>::put(x * p.out_scale);
            if (rest) rest[(int64_t)i * p.Dv + c] = Vec<T>::put(x * p.out_scale - Vec<T>::get(dst[c]));
        }
    }
}

// ---------------------------------------------------------------------------
// dQ, and the rows' Dd
// ---------------------------------------------------------------------------
template <typename T, int S>
__global__ void __launch_bounds__(THREADS)
cross_dq_kernel(const CrossParams p) {
    using Z = Size<S>;
    constexpr bool TWICE = sizeof(T) == 2;
    extern __shared__ __align__(16) float sm[];
    const int ld = padded(p.D), lv = padded(p.Dv);
    float* qs = sm;
    float* gs = qs + 2 * BM * ld;               // [row][lv]
    float* kv = gs + BM * lv;
    const int stage = 2 * BN * ld + BN * lv;
    float* ps = kv + STAGES<T> * stage;         // [branch][state][LP]: scores, then dS
    float* ds = ps + 2 * BN * LP;               // [state][LP]: dP
    pdl_wait();
    pdl_launch_dependents();
    const Rows r = rows_of(p);
    const CrossLen len = cross_len(p.lengths, r.b, p.Tk);
    if (len.bad && threadIdx.x == 0) atomicOr(p.status, kStatusIndex);
    if (blockIdx.x == 0 && threadIdx.x == 0) p.counters[2] = 0;
    Source<T>(p.q1, p.s_q1, r.b, r.h, p.D).load(qs, ld, r.q0, r.count);
    Source<T>(p.q2, p.s_q2, r.b, r.h, p.D).load(qs + BM * ld, ld, r.q0, r.count);
    const Source<T> grads(p.dout, p.s_do, r.b, r.h, p.Dv);
    grads.load(gs, lv, r.q0, r.count);
    const float lam = lambda_of(p.lambda_dev, p.lambda_bf16, p.lambda);
    const int br = threadIdx.x >> 7, row = (threadIdx.x >> 2) & 31, sub = threadIdx.x & 3;
    const int64_t at = ((int64_t)r.b * p.H + r.h) * p.Tq + r.q0 + row;
    const float lse = row < r.count ? p.lse[at * 2 + br] : 0.f;
    float dd = 0.f;
    if (!TWICE && row < r.count && len.n > 0) {
        // from the saved results, four threads a row
        const int64_t o = r.b * p.s_o[0] + r.h * p.s_o[1] + (r.q0 + row) * p.s_o[2];
        const T* o1 = static_cast<const T*>(p.out) + o;
        const T* o2 = static_cast<const T*>(p.out2) + o;
        const T* g = grads.at + (r.q0 + row) * grads.stride;
        for (int c = sub; c < p.Dv; c += 4) {
            const float x = Vec<T>::get(o2[c]);
            dd = fmaf(Vec<T>::get(g[c]), br ? x : fmaf(lam, x, Vec<T>::get(o1[c])), dd);
        }
    }
    if (!TWICE) {
        dd += __shfl_xor_sync(0xffffffffu, dd, 1);
        dd += __shfl_xor_sync(0xffffffffu, dd, 2);
    }
    const int half = threadIdx.x & 127, r0 = half / Z::CD * Z::RD, c0 = half % Z::CD * 4;
    float4 acc[Z::RD][1] = {};
    const States<T> states(p, r.b, r.hk, len.n, ld, lv);
    for (int sweep = TWICE ? 0 : 1; sweep < 2; ++sweep) {
        if (len.n > 0) states.begin(kv);
        for (int k0 = 0; k0 < len.n; k0 += BN) {
            const int live = min(BN, len.n - k0);
            const float* ks = states.next(kv, stage, k0);
            const float* vs = ks + 2 * BN * ld;
            scores(qs, ks, ld, p.D, ps, true);
            products(gs, vs, lv, p.Dv, ds, true);
            __syncthreads();
            float* w = ps + br * BN * LP + row;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int key = sub + 4 * j;
                const float a = key < live && row < r.count ? expf(w[key * LP] * p.scale - lse) : 0.f;
                const float dp = ds[key * LP + row];
                if (sweep == 0) dd = fmaf(a, dp, dd);
                else w[key * LP] = (br ? -lam : 1.f) * a * (dp - dd);
            }
            if (sweep == 0) continue;
            __syncthreads();
            accumulate<Z::RD, 1>(ps + br * BN * LP, r0, ks + br * BN * ld, ld, c0, 0, p.D, acc);
        }
        if (sweep == 0) {
            dd += __shfl_xor_sync(0xffffffffu, dd, 1);
            dd += __shfl_xor_sync(0xffffffffu, dd, 2);
        }
    }
    async_wait();
    const float nan = __int_as_float(0x7fc00000);
    if (sub == 0 && row < r.count) {
        p.stats[at * 4 + br] = lse;
        p.stats[at * 4 + 2 + br] = len.bad ? nan : dd;
    }
    T* dq = static_cast<T*>(br ? p.dq2 : p.dq1);
    if (!dq || c0 >= p.D) return;
#pragma unroll
    for (int i = 0; i < Z::RD; ++i)
        if (r0 + i < r.count)
            put4(dq + (((int64_t)r.b * p.H + r.h) * p.Tq + r.q0 + r0 + i) * p.D, c0, p.D, acc[i][0], len.bad ? nan : p.scale);
}

// ---------------------------------------------------------------------------
// dK and dV
// ---------------------------------------------------------------------------
template <typename T, int S>
__global__ void __launch_bounds__(THREADS)
cross_dkdv_kernel(const CrossParams p) {
    using Z = Size<S>;
    extern __shared__ __align__(16) float sm[];
    const int ld = padded(p.D), lv = padded(p.Dv);
    float* ks = sm;                             // [branch][state][ld]
    float* vs = ks + 2 * BN * ld;               // [state][lv]
    float* rows_at = vs + BN * lv;              // [stage]: queries [branch][row][ld], dO [row][lv]
    const int stage = 2 * BM * ld + BM * lv;
    float* ps = rows_at + STAGES<T> * stage;    // [branch][row][LP]: scores, then dS
    float* ds = ps + 2 * BM * LP;               // [row][LP]: dP, then W = A_1 - lambda A_2
    const int tiles = (p.Tk + BN - 1) / BN;
    const int bh = blockIdx.x / tiles, b = bh / p.Hk, hk = bh - b * p.Hk;
    const int k0 = (blockIdx.x - bh * tiles) * BN, count = min(BN, p.Tk - k0);
    pdl_wait();
    pdl_launch_dependents();
    const CrossLen len = cross_len(p.lengths, b, p.Tk);
    const int live = max(0, min(count, len.n - k0));
    const float lam = lambda_of(p.lambda_dev, p.lambda_bf16, p.lambda);
    const int half = threadIdx.x & 127, br = threadIdx.x >> 7;
    const int rd = half / Z::CD * Z::RD, cd = half % Z::CD * 4;
    const int rv = threadIdx.x / Z::CV * Z::RV, cv = threadIdx.x % Z::CV * 4;
    float4 dk[Z::RD][1] = {}, dv[Z::RV][Z::NV] = {};
    if (live > 0) {
        Source<T>(p.k1, p.s_k1, b, hk, p.D).load(ks, ld, k0, live);
        Source<T>(p.k2, p.s_k2, b, hk, p.D).load(ks + BN * ld, ld, k0, live);
        Source<T>(p.v, p.s_v, b, hk, p.Dv).load(vs, lv, k0, live);
        const int per_head = (p.Tq + BM - 1) / BM, total = p.group * per_head;
        auto fetch = [&](float* to, int i) {
            const int h = hk * p.group + i / per_head, q0 = i % per_head * BM, rows = min(BM, p.Tq - q0);
            Source<T>(p.q1, p.s_q1, b, h, p.D).load(to, ld, q0, rows);
            Source<T>(p.q2, p.s_q2, b, h, p.D).load(to + BM * ld, ld, q0, rows);
            Source<T>(p.dout, p.s_do, b, h, p.Dv).load(to + 2 * BM * ld, lv, q0, rows);
            async_commit();
        };
        if (STAGES<T> == 2) fetch(rows_at, 0);
        for (int i = 0; i < total; ++i) {
            const int h = hk * p.group + i / per_head, q0 = i % per_head * BM, rows = min(BM, p.Tq - q0);
            const float* qs = rows_at + (STAGES<T> == 2 ? (i & 1) * stage : 0);
            const float* gs = qs + 2 * BM * ld;
            if (STAGES<T> == 2) {
                async_wait();
                __syncthreads();                // the rows are there, and the last ones have been read
                if (i + 1 < total) fetch(rows_at + ((i & 1) ^ 1) * stage, i + 1);
            } else {
                __syncthreads();
                fetch(rows_at, i);
                __syncthreads();
            }
            scores(qs, ks, ld, p.D, ps, false);
            products(gs, vs, lv, p.Dv, ds, false);
            __syncthreads();
            const int row = threadIdx.x >> 3;
            float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row < rows)
                st = *reinterpret_cast<const float4*>(p.stats + (((int64_t)b * p.H + h) * p.Tq + q0 + row) * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = (threadIdx.x & 7) + 8 * j, at = row * LP + key;
                const bool seen = row < rows && key < live;
                const float a1 = seen ? expf(ps[at] * p.scale - st.x) : 0.f;
                const float a2 = seen ? lam * expf(ps[BM * LP + at] * p.scale - st.y) : 0.f;
                const float dp = ds[at];
                ps[at] = a1 * (dp - st.z);
                ps[BM * LP + at] = -a2 * (dp - st.w);
                ds[at] = a1 - a2;
            }
            __syncthreads();
            accumulate<Z::RV, Z::NV>(ds, rv, gs, lv, cv, 4 * Z::CV, p.Dv, dv);
            accumulate<Z::RD, 1>(ps + br * BM * LP, rd, qs + br * BM * ld, ld, cd, 0, p.D, dk);
        }
    }
    const float fill = len.bad ? __int_as_float(0x7fc00000) : 1.f;
    const int64_t at = ((int64_t)b * p.Hk + hk) * p.Tk + k0;
#pragma unroll
    for (int i = 0; i < Z::RV; ++i)
#pragma unroll
        for (int n = 0; n < Z::NV; ++n)
            if (rv + i < count && cv + n * 4 * Z::CV < p.Dv)
                put4(static_cast<T*>(p.dv) + (at + rv + i) * p.Dv, cv + n * 4 * Z::CV, p.Dv, dv[i][n], fill);
    if (p.k_shared) {                           // one tensor: the branches' gradients before the rounding
        __syncthreads();
        if (br == 1 && cd < p.D)
#pragma unroll
            for (int i = 0; i < Z::RD; ++i) *reinterpret_cast<float4*>(rows_at + (rd + i) * ld + cd) = dk[i][0];
        __syncthreads();
        if (br == 0 && cd < p.D)
#pragma unroll
            for (int i = 0; i < Z::RD; ++i) {
                const float4 x = *reinterpret_cast<const float4*>(rows_at + (rd + i) * ld + cd);
                dk[i][0] = make_float4(dk[i][0].x + x.x, dk[i][0].y + x.y, dk[i][0].z + x.z, dk[i][0].w + x.w);
            }
        if (br == 1) return;
    }
    if (cd >= p.D) return;
#pragma unroll
    for (int i = 0; i < Z::RD; ++i)
        if (rd + i < count)
            put4(static_cast<T*>(br ? p.dk2 : p.dk1) + (at + rd + i) * p.D, cd, p.D, dk[i][0], fill * p.scale);
}

// ---------------------------------------------------------------------------
// dlambda: blocks sum their shares of the rows, the last of them the blocks' sums; the order
// of either is fixed.  One launch (two were 10 us of the host's time).
// ---------------------------------------------------------------------------
constexpr int LAMBDA_THREADS = 256;
__device__ __forceinline__ float block_sum(float s, float* part) {
    s = group_sum<32>(s);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    float t = 0.f;
    if (threadIdx.x == 0)
        for (int w = 0; w < LAMBDA_THREADS / 32; ++w) t += part[w];
    return t;
}
__global__ void __launch_bounds__(LAMBDA_THREADS)
cross_dlambda_kernel(const CrossParams p, float sign) {
    __shared__ float part[LAMBDA_THREADS / 32];
    __shared__ bool last;
    pdl_wait();
    const int64_t rows = (int64_t)p.B * p.H * p.Tq, per = (rows + gridDim.x - 1) / gridDim.x;
    const int64_t r1 = min(rows, (blockIdx.x + 1) * per);
    float s = 0.f;
    for (int64_t r = blockIdx.x * per + threadIdx.x; r < r1; r += LAMBDA_THREADS) s += p.stats[r * 4 + 3];
    const float mine = block_sum(s, part);
    if (threadIdx.x == 0) {
        p.lambda_parts[blockIdx.x] = mine;
        __threadfence();
        last = atomicAdd(p.counters + 2, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    s = threadIdx.x < gridDim.x ? *static_cast<volatile float*>(p.lambda_parts + threadIdx.x) : 0.f;
    const float total = sign * block_sum(s, part);
    if (threadIdx.x != 0) return;
    if (p.lambda_bf16) *static_cast<__nv_bfloat16*>(p.dlambda) = __float2bfloat16_rn(total);
    else *static_cast<float*>(p.dlambda) = total;
}
static_assert(kLambdaBlocks <= LAMBDA_THREADS, "a block's sum a thread");

template <typename K>
int launch_smem(K kernel, int64_t blocks, int floats, const CrossParams& p, cudaStream_t stream) {
    if (blocks > INT32_MAX ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, floats * 4) != cudaSuccess)
        return -1;
    return pdl_launch(kernel, dim3((unsigned)blocks), THREADS, (size_t)floats * 4, stream, p);
}

template <typename T, int S>
int launch(const CrossParams& p, bool backward, cudaStream_t stream) {
    const int ld = padded(p.D), lv = padded(p.Dv);
    const int64_t row_blocks = (int64_t)p.B * p.H * ((p.Tq + BM - 1) / BM);
    const int walked = STAGES<T> * (2 * BN * ld + BN * lv);
    if (!backward) return launch_smem(cross_fwd_kernel<T, S>, row_blocks, 2 * BM * ld + walked + 2 * BN * LP + 2 * BM, p, stream);
    const int floats = 2 * BM * ld + BM * lv + walked + 3 * BN * LP;
    if (launch_smem(cross_dq_kernel<T, S>, row_blocks, floats, p, stream) != 0) return -1;
    if (!p.dv) return 0;
    return launch_smem(cross_dkdv_kernel<T, S>, (int64_t)p.B * p.Hk * ((p.Tk + BN - 1) / BN), floats, p, stream);
}

template <typename T>
int launch_type(const CrossParams& p, bool backward, cudaStream_t stream) {
    if (p.D <= 32 && p.Dv <= 64) return launch<T, 0>(p, backward, stream);
    if (p.D <= 64 && p.Dv <= 128) return launch<T, 1>(p, backward, stream);
    return launch<T, 2>(p, backward, stream);
}

}  // namespace xsimt

int launch_cross_dlambda(const CrossParams& p, float sign, cudaStream_t stream) {
    const int64_t blocks = ((int64_t)p.B * p.H * p.Tq + 1023) / 1024;
    return pdl_launch(xsimt::cross_dlambda_kernel, dim3((unsigned)(blocks < kLambdaBlocks ? blocks : kLambdaBlocks)),
                      xsimt::LAMBDA_THREADS, 0, stream, p, sign);
}

int launch_cross_simt(const CrossParams& p, cudaStream_t stream) {
    return p.bf16 ? xsimt::launch_type<__nv_bfloat16>(p, false, stream) : xsimt::launch_type<float>(p, false, stream);
}

int launch_cross_simt_bwd(const CrossParams& p, cudaStream_t stream) {
    return p.bf16 ? xsimt::launch_type<__nv_bfloat16>(p, true, stream) : xsimt::launch_type<float>(p, true, stream);
}

}  // namespace diffattn
