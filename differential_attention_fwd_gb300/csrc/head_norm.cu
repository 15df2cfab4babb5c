// head_norm.cu -- the norm of each head's output and its gradients (diffattn_head_norm,
// diffattn_head_norm_bwd): the attention's output epilogue as an operator of its own.
//
// For a row x of C channels of head h, with mu = mean(x) (0 for the RMS norm),
// r = (mean((x - mu)^2) + eps)^-1/2 and h^ = (x - mu) r:
//
//     y  = s (w h^ + b)                        w, b [H, C], s the output's scale
//     g  = s w dy
//     dx = r (g - mean(g) - h^ mean(g h^))     (without mean(g) for the RMS norm)
//     dw = s sum over rows of dy h^,           db = s sum over rows of dy
//
// The mean comes off before the squares are summed (values far from 0 keep their digits),
// and the backward forms mu and r again from the x that it reads anyway.  float32
// arithmetic, one rounding of y and dx at the end.
//
// The passes are bound by HBM: x in, y out; x and dy in, dx out.  A group of lanes holds a
// row, twice 16 bytes a lane (the exchanges of the row's sums are a third of the backward's
// instructions with 16), so the row stays in registers and the only exchanges are its sums.
// A block works on one head, whose weights stay in registers, and takes ROWS rows a group at a
// time: their loads go out together.  In the backward every block walks a chunk of the tokens,
// each lane adding up dw and db of its own channels, and leaves one partial row of each: the
// sums' order is fixed, without atomics.
//
// 2 x 8192 tokens, 16 heads of 128, bf16, layer norm: forward 22.6 us (5.9 TB/s), backward 36.8
// us (5.5 TB/s) and 3.5 us for dw and db; with 16 bytes a lane 27 and 50 us.  One token of 16
// sequences: 3.2 us, a launch's latency.
#include "block.h"
#include "pdl.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace diffattn {
namespace hnorm {

constexpr int THREADS = 256;
constexpr int MAX_C = 256;
constexpr int ROWS = 2;             // of a group, loaded together
constexpr int BWD_ROWS = 2;
constexpr int BWD_AN_SM = 2;
constexpr int CH = 2;               // pieces of 16 bytes a lane
constexpr int BWD_BLOCKS = 304;     // of the backward, about: the two that each of 152 SMs holds

// The lanes' part of a row: CH pieces of 16 bytes, V elements each, piece j of lane g at
// element (g + j G) V.
template <typename T, int G>
struct Part {
    static constexpr int V = Vec<T>::N;
    static constexpr int P = CH * V / 2;    // pairs
    int at[CH];
    bool live[CH];
    __device__ __forceinline__ Part(int g, int C) {
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            at[j] = (g + j * G) * V;
            live[j] = at[j] < C;
        }
    }
    __device__ __forceinline__ void load(const T* row, bool there, uint4 (&raw)[CH]) const {
#pragma unroll
        for (int j = 0; j < CH; ++j)
            raw[j] = there && live[j] ? *reinterpret_cast<const uint4*>(row + at[j]) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ static void unpack(const uint4 (&raw)[CH], uint64_t (&x)[P]) {
#pragma unroll
        for (int j = 0; j < CH; ++j) Vec<T>::unpack(raw[j], x + j * V / 2);
    }
    __device__ __forceinline__ void store(T* row, const uint64_t (&x)[P]) const {
#pragma unroll
        for (int j = 0; j < CH; ++j)
            if (live[j]) *reinterpret_cast<uint4*>(row + at[j]) = Vec<T>::pack(x + j * V / 2);
    }
    // float32 weights of the lane's channels, or `none` for each
    __device__ __forceinline__ void weights(const float* w, float none, uint64_t (&x)[P]) const {
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            if (w && live[j]) {
                load_pairs<V>(w + at[j], x + j * V / 2);
            } else {
#pragma unroll
                for (int e = 0; e < V / 2; ++e) x[j * V / 2 + e] = f2_pack(none, none);
            }
        }
    }
    // x - mean(x) in place (channels that a row does not have stay 0)
    __device__ __forceinline__ void center(uint64_t (&x)[P], float inv_C) const {
        const float mu = group_sum<G>(pair_sum<P>(x)) * inv_C;
        const uint64_t m = f2_pack(mu, mu);
#pragma unroll
        for (int j = 0; j < CH; ++j)
            if (live[j])
#pragma unroll
                for (int e = 0; e < V / 2; ++e) x[j * V / 2 + e] = f2_sub(x[j * V / 2 + e], m);
    }
};

template <int P>
__device__ __forceinline__ float dot(const uint64_t (&a)[P], const uint64_t (&b)[P]) {
    uint64_t s = f2_mul(a[0], b[0]);
#pragma unroll
    for (int e = 1; e < P; ++e) s = f2_fma(a[e], b[e], s);
    return f2_lo(s) + f2_hi(s);
}

template <typename T, int G>
__global__ void __launch_bounds__(THREADS)
head_norm_kernel(const HeadNormParams p) {
    using L = Part<T, G>;
    constexpr int GROUPS = THREADS / G;
    const L part(threadIdx.x % G, p.C);
    const int h = blockIdx.y;
    const int tok0 = blockIdx.x * (GROUPS * ROWS) + threadIdx.x / G;
    pdl_wait();
    pdl_launch_dependents();
    uint4 raw[ROWS][CH];
    int64_t to[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int tok = tok0 + i * GROUPS;
        const bool in = tok < p.tokens;
        const int b = in ? p.by_T.div(tok) : 0, t = in ? tok - b * p.T : 0;
        part.load(static_cast<const T*>(p.x) + b * p.sx[0] + h * p.sx[1] + t * p.sx[2], in, raw[i]);
        to[i] = in ? b * p.sy[0] + h * p.sy[1] + t * p.sy[2] : -1;
    }
    uint64_t w[L::P], bias[L::P];
    part.weights(p.w ? p.w + (int64_t)h * p.C : nullptr, 1.f, w);
    part.weights(p.b ? p.b + (int64_t)h * p.C : nullptr, 0.f, bias);
    const uint64_t s2 = f2_pack(p.scale, p.scale);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        uint64_t x[L::P];
        L::unpack(raw[i], x);
        if (p.group) part.center(x, p.inv_C);
        const float r = rsqrtf(group_sum<G>(dot(x, x)) * p.inv_C + p.eps);
        const uint64_t r2 = f2_pack(r, r);
#pragma unroll
        for (int e = 0; e < L::P; ++e) x[e] = f2_mul(f2_fma(f2_mul(x[e], r2), w[e], bias[e]), s2);
        if (to[i] >= 0) part.store(static_cast<T*>(p.y) + to[i], x);
    }
}

template <typename T, int G>
__global__ void __launch_bounds__(THREADS, BWD_AN_SM)
head_norm_bwd_kernel(const HeadNormParams p) {
    using L = Part<T, G>;
    constexpr int GROUPS = THREADS / G;
    constexpr int V = L::V;
    __shared__ float red[2][THREADS / 32][32 * CH * V];     // [dw, db][warp][lane's channels]
    const L part(threadIdx.x % G, p.C);
    const int h = blockIdx.y;
    pdl_wait();
    pdl_launch_dependents();
    uint64_t w[L::P], dw[L::P], db[L::P];
    part.weights(p.w ? p.w + (int64_t)h * p.C : nullptr, 1.f, w);
    const uint64_t s2 = f2_pack(p.scale, p.scale);
#pragma unroll
    for (int e = 0; e < L::P; ++e) {
        w[e] = f2_mul(w[e], s2);
        dw[e] = db[e] = 0;
    }
    const int end = min(p.tokens, (blockIdx.x + 1) * p.per_chunk);
    for (int tok0 = blockIdx.x * p.per_chunk + threadIdx.x / G; tok0 - (int)(threadIdx.x / G) < end; tok0 += GROUPS * BWD_ROWS) {
        uint4 rx[BWD_ROWS][CH], rg[BWD_ROWS][CH];
        int64_t to[BWD_ROWS];
#pragma unroll
        for (int i = 0; i < BWD_ROWS; ++i) {
            const int tok = tok0 + i * GROUPS;
            const bool in = tok < end;
            const int b = in ? p.by_T.div(tok) : 0, t = in ? tok - b * p.T : 0;
            part.load(static_cast<const T*>(p.x) + b * p.sx[0] + h * p.sx[1] + t * p.sx[2], in, rx[i]);
            part.load(static_cast<const T*>(p.dy) + b * p.sdy[0] + h * p.sdy[1] + t * p.sdy[2], in, rg[i]);
            to[i] = in ? b * p.sdx[0] + h * p.sdx[1] + t * p.sdx[2] : -1;
        }
#pragma unroll
        for (int i = 0; i < BWD_ROWS; ++i) {
            uint64_t x[L::P], dy[L::P], g[L::P];
            L::unpack(rx[i], x);
            L::unpack(rg[i], dy);
            if (p.group) part.center(x, p.inv_C);
#pragma unroll
            for (int e = 0; e < L::P; ++e) g[e] = f2_mul(dy[e], w[e]);
            const float r = rsqrtf(group_sum<G>(dot(x, x)) * p.inv_C + p.eps);
            const uint64_t r2 = f2_pack(r, r);
            const float gh = group_sum<G>(dot(g, x)) * p.inv_C * r;         // mean(g h^)
            const float gm = p.group ? group_sum<G>(pair_sum<L::P>(g)) * p.inv_C : 0.f;
            const uint64_t ngh = f2_pack(-gh, -gh), ngm = f2_pack(-gm, -gm);
#pragma unroll
            for (int e = 0; e < L::P; ++e) {
                const uint64_t hat = f2_mul(x[e], r2);
                dw[e] = f2_fma(dy[e], hat, dw[e]);
                db[e] = f2_add(db[e], dy[e]);
                x[e] = f2_mul(f2_fma(hat, ngh, f2_add(g[e], ngm)), r2);
            }
            if (to[i] >= 0 && p.dx) part.store(static_cast<T*>(p.dx) + to[i], x);
        }
    }
    if (!p.dw && !p.db) return;
    // the groups of a warp by shuffles, then the warps in turn
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < 2 * L::P; ++i) {
        float a = i & 1 ? f2_hi(dw[i / 2]) : f2_lo(dw[i / 2]), c = i & 1 ? f2_hi(db[i / 2]) : f2_lo(db[i / 2]);
#pragma unroll
        for (int o = G; o < 32; o <<= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            c += __shfl_xor_sync(0xffffffffu, c, o);
        }
        const int j = i / V, at = ((lane % G) + j * G) * V + i % V;
        if (lane < G) {
            red[0][warp][at] = a;
            red[1][warp][at] = c;
        }
    }
    __syncthreads();
    float* out = p.partial + ((int64_t)blockIdx.x * p.H + h) * 2 * p.C;
    for (int c = threadIdx.x; c < 2 * p.C; c += THREADS) {
        const int k = c >= p.C, at = c - k * p.C;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < THREADS / 32; ++j) sum += red[k][j][at];
        out[c] = sum;
    }
}

// Any width up to 256, any alignment: a warp a row.
constexpr int E = MAX_C / 32;

__device__ __forceinline__ float any_row(const HeadNormParams& p, float (&x)[E], int lane) {
    if (p.group) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s += x[e];
        const float mu = group_sum<32>(s) / p.C;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (lane + 32 * e < p.C) x[e] -= mu;
    }
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) ss = fmaf(x[e], x[e], ss);
    return 1.0f / sqrtf(group_sum<32>(ss) / p.C + p.eps);
}

template <typename T>
__global__ void __launch_bounds__(THREADS)
head_norm_any_kernel(const HeadNormParams p) {
    const int lane = threadIdx.x % 32, h = blockIdx.y;
    pdl_wait();
    pdl_launch_dependents();
    const int tok = blockIdx.x * (THREADS / 32) + threadIdx.x / 32;
    if (tok >= p.tokens) return;
    const int b = tok / p.T, t = tok - b * p.T;
    const T* src = static_cast<const T*>(p.x) + b * p.sx[0] + h * p.sx[1] + t * p.sx[2];
    T* dst = static_cast<T*>(p.y) + b * p.sy[0] + h * p.sy[1] + t * p.sy[2];
    float x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = lane + 32 * e < p.C ? Vec<T>::get(src[lane + 32 * e]) : 0.f;
    const float r = any_row(p, x, lane);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = lane + 32 * e;
        if (c >= p.C) continue;
        const float w = p.w ? p.w[(int64_t)h * p.C + c] : 1.f, bias = p.b ? p.b[(int64_t)h * p.C + c] : 0.f;
        dst[c] = Vec<T>::put(fmaf(x[e] * r, w, bias) * p.scale);
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS)
head_norm_bwd_any_kernel(const HeadNormParams p) {
    constexpr int WARPS = THREADS / 32;
    __shared__ float red[2][WARPS][MAX_C];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, h = blockIdx.y;
    pdl_wait();
    pdl_launch_dependents();
    float w[E], dw[E] = {}, db[E] = {};
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = p.scale * (p.w && lane + 32 * e < p.C ? p.w[(int64_t)h * p.C + lane + 32 * e] : 1.f);
    const int end = min(p.tokens, (blockIdx.x + 1) * p.per_chunk);
    for (int tok = blockIdx.x * p.per_chunk + warp; tok < end; tok += WARPS) {
        const int b = tok / p.T, t = tok - b * p.T;
        const T* xs = static_cast<const T*>(p.x) + b * p.sx[0] + h * p.sx[1] + t * p.sx[2];
        const T* gs = static_cast<const T*>(p.dy) + b * p.sdy[0] + h * p.sdy[1] + t * p.sdy[2];
        float x[E], dy[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const bool in = lane + 32 * e < p.C;
            x[e] = in ? Vec<T>::get(xs[lane + 32 * e]) : 0.f;
            dy[e] = in ? Vec<T>::get(gs[lane + 32 * e]) : 0.f;
        }
        const float r = any_row(p, x, lane);
        float gx = 0.f, gs_ = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            gx = fmaf(w[e] * dy[e], x[e], gx);
            gs_ = fmaf(w[e], dy[e], gs_);
        }
        const float gh = group_sum<32>(gx) / p.C * r;
        const float gm = p.group ? group_sum<32>(gs_) / p.C : 0.f;
        T* dx = p.dx ? static_cast<T*>(p.dx) + b * p.sdx[0] + h * p.sdx[1] + t * p.sdx[2] : nullptr;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float hat = x[e] * r;
            dw[e] = fmaf(dy[e], hat, dw[e]);
            db[e] += dy[e];
            if (dx && lane + 32 * e < p.C) dx[lane + 32 * e] = Vec<T>::put((w[e] * dy[e] - gm - hat * gh) * r);
        }
    }
    if (!p.dw && !p.db) return;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        red[0][warp][lane + 32 * e] = dw[e];
        red[1][warp][lane + 32 * e] = db[e];
    }
    __syncthreads();
    float* out = p.partial + ((int64_t)blockIdx.x * p.H + h) * 2 * p.C;
    for (int c = threadIdx.x; c < 2 * p.C; c += THREADS) {
        const int k = c >= p.C, at = c - k * p.C;
        float sum = 0.f;
        for (int j = 0; j < WARPS; ++j) sum += red[k][j][at];
        out[c] = sum;
    }
}

// dw and db from the blocks' partial rows, in a fixed order: 32 channels of a head's pair
// of rows a block, the chunks spread over its warps.
constexpr int RED_WARPS = 16;
__global__ void __launch_bounds__(32 * RED_WARPS)
head_norm_dw_kernel(const HeadNormParams p) {
    __shared__ float red[RED_WARPS][32];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, h = blockIdx.x;
    const int c = blockIdx.y * 32 + lane;           // of the 2 C
    float sum = 0.f;
    if (c < 2 * p.C)
#pragma unroll 4
        for (int k = warp; k < p.chunks; k += RED_WARPS) sum += p.partial[((int64_t)k * p.H + h) * 2 * p.C + c];
    red[warp][lane] = sum;
    __syncthreads();
    if (warp != 0 || c >= 2 * p.C) return;
    float total = 0.f;
#pragma unroll
    for (int j = 0; j < RED_WARPS; ++j) total += red[j][lane];
    float* out = c < p.C ? p.dw : p.db;
    if (out) out[(int64_t)h * p.C + (c < p.C ? c : c - p.C)] = total * p.scale;
}

template <typename T, int G>
int launch_one(const HeadNormParams& p, bool backward, cudaStream_t stream) {
    constexpr int PER = THREADS / G * ROWS;
    if (backward)
        return pdl_launch(head_norm_bwd_kernel<T, G>, dim3((unsigned)p.chunks, (unsigned)p.H), THREADS, 0, stream, p);
    return pdl_launch(head_norm_kernel<T, G>, dim3((unsigned)((p.tokens + PER - 1) / PER), (unsigned)p.H), THREADS, 0,
                      stream, p);
}

// Lanes of a row: the fewest, a power of two, that hold it in two pieces each.
int lanes_of(const HeadNormParams& p) {
    const int pieces = p.C / (p.bf16 ? 8 : 4);
    return pieces <= 8 ? 4 : pieces <= 16 ? 8 : pieces <= 32 ? 16 : 32;
}

template <typename T>
int launch_type(const HeadNormParams& p, bool backward, cudaStream_t stream) {
    if (!p.fast) {
        const auto kernel = backward ? head_norm_bwd_any_kernel<T> : head_norm_any_kernel<T>;
        const unsigned blocks = backward ? (unsigned)p.chunks : (unsigned)((p.tokens + THREADS / 32 - 1) / (THREADS / 32));
        return pdl_launch(kernel, dim3(blocks, (unsigned)p.H), THREADS, 0, stream, p);
    }
    switch (lanes_of(p)) {
        case 4: return launch_one<T, 4>(p, backward, stream);
        case 8: return launch_one<T, 8>(p, backward, stream);
        case 16: return launch_one<T, 16>(p, backward, stream);
    }
    return launch_one<T, 32>(p, backward, stream);
}

int launch(const HeadNormParams& p, bool backward, cudaStream_t stream) {
    return p.bf16 ? launch_type<__nv_bfloat16>(p, backward, stream) : launch_type<float>(p, backward, stream);
}

}  // namespace hnorm

// Blocks along the tokens: about BWD_BLOCKS over all heads, each with whole steps.
void plan_head_norm_bwd(HeadNormParams* p) {
    const int step = p->fast ? hnorm::THREADS / hnorm::lanes_of(*p) * hnorm::BWD_ROWS : hnorm::THREADS / 32;
    const int64_t steps = ((int64_t)p->tokens + step - 1) / step, most = (hnorm::BWD_BLOCKS + p->H - 1) / p->H;
    const int64_t each = (steps + most - 1) / most;
    p->per_chunk = (int)(each * step);
    p->chunks = (int)((steps + each - 1) / each);
}

size_t head_norm_bwd_floats(int64_t H, int64_t C) { return (size_t)((hnorm::BWD_BLOCKS + H) * 2 * C); }

int launch_head_norm(const HeadNormParams& p, cudaStream_t stream) { return hnorm::launch(p, false, stream); }

int launch_head_norm_bwd(const HeadNormParams& p, cudaStream_t stream) {
    if (hnorm::launch(p, true, stream) != 0) return -1;
    if (!p.dw && !p.db) return 0;
    return pdl_launch(hnorm::head_norm_dw_kernel, dim3((unsigned)p.H, (unsigned)((2 * p.C + 31) / 32)),
                      32 * hnorm::RED_WARPS, 0, stream, p);
}

}  // namespace diffattn
