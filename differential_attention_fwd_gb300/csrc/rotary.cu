// rotary.cu -- norm of each query and key head and the position rotation in one
// pass over the rows (diffattn_rotary, its backward, and diffattn_paged_append,
// which writes the rotated keys and the values into a paged cache).
//
// For a head row x of width D at position p, with r = (mean(x^2) + eps)^-1/2 and
// weights w (r = w = 1 without the norm):
//
//     n = x r w,   y_a = n_a cos - n_b sin,   y_b = n_b cos + n_a sin
//
// for the pairs (a, b) = (i, i + R/2), or (2i, 2i + 1) when interleaved, of the
// first R elements; the rest is n.  cos and sin come from tables by position: their
// angles need more than 32 bits at far positions, which the table's maker spends
// once.  All arithmetic is in float32, with one rounding of y at the end.
//
// The pass is bound by HBM: x in, y out.  A group of D / (2 V) lanes holds one row,
// V = 16 bytes of elements twice a lane: the two halves of its pairs, so a pair never
// leaves its lane and the only exchange is the sum of squares.  A group walks several
// heads of one token with the token's cosines and sines in registers, since the
// table row (4 R bytes) is as large as a bf16 head row: read for each head from L2 it
// would be as much traffic as x itself.
#include "paged.h"
#include "ptx.cuh"

namespace diffattn {
namespace rot {

constexpr int THREADS = 256;
constexpr int MAX_D = 128;

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ void load(const float* p, float* x) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    }
    __device__ static __forceinline__ void store(float* p, const float* x) {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    }
    __device__ static __forceinline__ float get(float v) { return v; }
    __device__ static __forceinline__ float put(float v) { return v; }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static __forceinline__ void load(const __nv_bfloat16* p, float* x) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static __forceinline__ void store(__nv_bfloat16* p, const float* x) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                  pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
    __device__ static __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    __device__ static __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};

// The token (b, t): its position, and in the paged cache its page and slot.
struct Token {
    bool live;          // to be processed (padding of a ragged batch is not)
    bool ok;            // position and page are inside the table and the cache
    int64_t pos, page, slot;
};

__device__ __forceinline__ Token find_token(const RotaryParams& p, int b, int t, bool paged) {
    Token k{true, true, t, 0, 0};
    if (paged) {
        const int64_t before = p.lengths[b];
        k.live = p.new_lengths ? t < p.new_lengths[b] : true;
        if (!k.live) return k;
        const int64_t at = before + t;
        const int64_t pg = at / p.page;
        k.pos = at;
        k.slot = at - pg * p.page;
        k.ok = before >= 0 && pg < p.max_pages;
        if (k.ok) {
            k.page = p.table[b * p.table_stride + pg];
            k.ok = k.page >= 0 && k.page < p.num_pages;
        }
    }
    if (p.pos) {
        const int64_t i = b * p.pos_stride[0] + t * p.pos_stride[1];
        k.pos = p.pos64 ? static_cast<const int64_t*>(p.pos)[i] : static_cast<const int32_t*>(p.pos)[i];
    }
    if (p.R > 0 && (k.pos < 0 || k.pos >= p.table_rows)) k.ok = false;
    return k;
}

// Stream and first head of a head block.
__device__ __forceinline__ int find_stream(const RotaryParams& p, int block, int* head0) {
    int i = 0;
    for (; i < p.n - 1; ++i) {
        const int nb = (p.s[i].heads + p.heads_per_block - 1) / p.heads_per_block;
        if (block < nb) break;
        block -= nb;
    }
    *head0 = block * p.heads_per_block;
    return i;
}

// Element offsets of a lane's two chunks, and whether its pairs are rotated: with
// pairs (i, i + R/2) the first R / (2 V) lanes hold chunks g and g + R / (2 V), the
// others two chunks of the unrotated rest; interleaved, every lane holds 2 V
// consecutive elements.  Either way the lane's pairs are V g .. V g + V - 1.
template <int V, bool INTER>
__device__ __forceinline__ bool chunk_offsets(int g, int R, int* a, int* b) {
    const int rc = R / (2 * V);
    const bool turn = g < rc;
    if (INTER || !turn) {
        *a = 2 * g * V;
        *b = *a + V;
    } else {
        *a = g * V;
        *b = (g + rc) * V;
    }
    return turn;
}

// One row's pairs (e0, e1) from its two chunks and back.
template <int V, bool INTER>
__device__ __forceinline__ void to_pairs(const float* c, float* e0, float* e1) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        e0[i] = INTER ? c[2 * i] : c[i];
        e1[i] = INTER ? c[2 * i + 1] : c[V + i];
    }
}
template <int V, bool INTER>
__device__ __forceinline__ void from_pairs(const float* e0, const float* e1, float* c) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        c[INTER ? 2 * i : i] = e0[i];
        c[INTER ? 2 * i + 1 : V + i] = e1[i];
    }
}

template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// cos and sin of the lane's V pairs (1 and 0 where nothing turns).
template <int V>
__device__ __forceinline__ void load_turn(const RotaryParams& p, int64_t pos, int g, bool turn, float* cs, float* sn) {
    if (turn) {
        const int64_t at = pos * (p.R / 2) + g * V;
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 c = *reinterpret_cast<const float4*>(p.cos + at + i);
            const float4 s = *reinterpret_cast<const float4*>(p.sin + at + i);
            cs[i] = c.x; cs[i + 1] = c.y; cs[i + 2] = c.z; cs[i + 3] = c.w;
            sn[i] = s.x; sn[i + 1] = s.y; sn[i + 2] = s.z; sn[i + 3] = s.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) { cs[i] = 1.f; sn[i] = 0.f; }
    }
}

// ---------------------------------------------------------------------------
// forward and append
// ---------------------------------------------------------------------------
template <typename T, int G, bool INTER>
__global__ void __launch_bounds__(THREADS)
rotary_kernel(const RotaryParams p) {
    constexpr int V = Vec<T>::N;
    constexpr int TOKENS = THREADS / G;
    const int g = threadIdx.x % G;
    int head0;
    const int si = find_stream(p, blockIdx.y, &head0);
    const RowStream& s = p.s[si];
    const int head1 = min(s.heads, head0 + p.heads_per_block);
    const bool paged = s.kind != kRowsDense;
    // the lanes of a group share a token; a group past the last token only takes
    // part in the warp's shuffles
    const int64_t tok = (int64_t)blockIdx.x * TOKENS + threadIdx.x / G;
    const bool in = tok < (int64_t)p.B * p.T;
    const int b = in ? (int)(tok / p.T) : 0;
    const int t = in ? (int)(tok - (int64_t)b * p.T) : 0;
    Token k = find_token(p, b, t, paged);
    k.live = k.live && in;
    if (k.live && !k.ok && g == 0) atomicOr(p.status, kStatusIndex);
    const bool write = k.live && (k.ok || !paged);
    const T* x0 = static_cast<const T*>(s.x) + b * s.sx[0] + t * s.sx[2];
    T* y0 = static_cast<T*>(s.y) + (paged ? k.page * s.sy[0] + k.slot * s.sy[2] : b * s.sy[0] + t * s.sy[2]);
    if (s.kind == kRowsCopy) {
        if (!write) return;
        for (int h = head0; h < head1; ++h)
            for (int c = g * V; c < s.width; c += G * V)
                *reinterpret_cast<uint4*>(y0 + h * s.sy[1] + c) =
                    *reinterpret_cast<const uint4*>(x0 + h * s.sx[1] + c);
        return;
    }
    int oa, ob;
    const bool turn = chunk_offsets<V, INTER>(g, p.R, &oa, &ob);
    float cs[V], sn[V];
    load_turn<V>(p, k.pos, g, turn && k.live && k.ok, cs, sn);
    const float fill = k.ok ? 0.f : __int_as_float(0x7fc00000);   // a position outside the table: NaN
    float w[2 * V];
    const bool weighted = p.norm && s.weight;
    if (weighted && s.w_stride == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            Vec<float>::load(s.weight + oa + i, w + i);
            Vec<float>::load(s.weight + ob + i, w + V + i);
        }
    }
#pragma unroll 2
    for (int h = head0; h < head1; ++h) {
        float c[2 * V] = {};
        if (k.live) {
            Vec<T>::load(x0 + h * s.sx[1] + oa, c);
            Vec<T>::load(x0 + h * s.sx[1] + ob, c + V);
        }
        if (p.norm) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) ss = fmaf(c[i], c[i], ss);
            const float r = 1.0f / sqrtf(group_sum<G>(ss) / p.D + p.eps);
            if (weighted) {
                if (s.w_stride) {
#pragma unroll
                    for (int i = 0; i < V; i += 4) {
                        Vec<float>::load(s.weight + h * s.w_stride + oa + i, w + i);
                        Vec<float>::load(s.weight + h * s.w_stride + ob + i, w + V + i);
                    }
                }
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) c[i] *= r * w[i];
            } else {
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) c[i] *= r;
            }
        }
        float e0[V], e1[V];
        to_pairs<V, INTER>(c, e0, e1);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float u = e0[i] * cs[i] - e1[i] * sn[i] + fill;
            e1[i] = e1[i] * cs[i] + e0[i] * sn[i] + fill;
            e0[i] = u;
        }
        from_pairs<V, INTER>(e0, e1, c);
        if (write) {
            Vec<T>::store(y0 + h * s.sy[1] + oa, c);
            Vec<T>::store(y0 + h * s.sy[1] + ob, c + V);
        }
    }
}

// Any width up to 128, any alignment: a warp a row.
template <typename T>
__global__ void __launch_bounds__(THREADS)
rotary_any_kernel(const RotaryParams p) {
    constexpr int WARPS = THREADS / 32;
    __shared__ float rows[WARPS][MAX_D];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    float* row = rows[warp];
    int head0;
    const int si = find_stream(p, blockIdx.y, &head0);      // one head a block here
    const RowStream& s = p.s[si];
    const bool paged = s.kind != kRowsDense;
    const int64_t tok = (int64_t)blockIdx.x * WARPS + warp;
    if (tok >= (int64_t)p.B * p.T) return;
    const int b = (int)(tok / p.T);
    const int t = (int)(tok - (int64_t)b * p.T);
    const Token k = find_token(p, b, t, paged);
    if (!k.live) return;
    if (!k.ok && lane == 0) atomicOr(p.status, kStatusIndex);
    if (!k.ok && paged) return;
    const T* x = static_cast<const T*>(s.x) + b * s.sx[0] + head0 * s.sx[1] + t * s.sx[2];
    T* y = static_cast<T*>(s.y) + head0 * s.sy[1] +
           (paged ? k.page * s.sy[0] + k.slot * s.sy[2] : b * s.sy[0] + t * s.sy[2]);
    if (s.kind == kRowsCopy) {
        for (int i = lane; i < s.width; i += 32) y[i] = x[i];
        return;
    }
    if (!k.ok) {
        for (int i = lane; i < p.D; i += 32) y[i] = Vec<T>::put(__int_as_float(0x7fc00000));
        return;
    }
    float ss = 0.f;
    for (int i = lane; i < p.D; i += 32) {
        const float v = Vec<T>::get(x[i]);
        row[i] = v;
        ss = fmaf(v, v, ss);
    }
    const float r = p.norm ? 1.0f / sqrtf(group_sum<32>(ss) / p.D + p.eps) : 1.f;
    if (p.norm) {
        const float* w = s.weight ? s.weight + head0 * s.w_stride : nullptr;
        for (int i = lane; i < p.D; i += 32) row[i] *= w ? r * w[i] : r;
    }
    __syncwarp();
    const int half = p.R / 2;
    for (int i = lane; i < p.D; i += 32) {
        float v = row[i];
        if (i < p.R) {
            const int j = p.interleaved ? i / 2 : (i < half ? i : i - half);
            const bool first = p.interleaved ? (i & 1) == 0 : i < half;
            const float other = row[p.interleaved ? i ^ 1 : (first ? i + half : i - half)];
            const float cs = p.cos[k.pos * half + j], sn = p.sin[k.pos * half + j];
            v = first ? v * cs - other * sn : v * cs + other * sn;
        }
        y[i] = Vec<T>::put(v);
    }
}

// ---------------------------------------------------------------------------
// backward: with u = R(p)^T dy (the rotation by the negative angle),
//     dw = sum over rows of u x r,
//     dx = r (w u - x r^2 mean(w u x)).
// Reads x and dy, writes dx: bound by HBM.  A block walks a chunk of the tokens and
// a few heads, one when the weights differ by head; each lane keeps the dw of its own
// 2 V channels in registers, and a block leaves one partial row, so the sum's order
// is fixed and no atomics are needed.
// ---------------------------------------------------------------------------
template <typename T, int G, bool INTER>
__global__ void __launch_bounds__(THREADS)
rotary_bwd_kernel(const RotaryParams p) {
    constexpr int V = Vec<T>::N;
    constexpr int GROUPS = THREADS / G;
    constexpr int D = G * 2 * V;
    __shared__ float red[GROUPS * D];
    const int g = threadIdx.x % G, group = threadIdx.x / G;
    int head0;
    const int si = find_stream(p, blockIdx.y, &head0);
    const RowStream& s = p.s[si];
    const int head1 = min(s.heads, head0 + p.heads_per_block);
    int oa, ob;
    const bool turn = chunk_offsets<V, INTER>(g, p.R, &oa, &ob);
    const bool weighted = p.norm && s.weight;
    float w[2 * V], dw[2 * V];
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) { w[i] = 1.f; dw[i] = 0.f; }
    if (weighted && s.w_stride == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            Vec<float>::load(s.weight + oa + i, w + i);
            Vec<float>::load(s.weight + ob + i, w + V + i);
        }
    }
    const int64_t tokens = (int64_t)p.B * p.T;
    // every group of the block makes the same number of steps: the sums below are
    // warp-wide
    for (int64_t base = (int64_t)blockIdx.x * GROUPS; base < tokens; base += (int64_t)gridDim.x * GROUPS) {
        const int64_t tok = base + group;
        const bool in = tok < tokens;
        const int b = in ? (int)(tok / p.T) : 0;
        const int t = in ? (int)(tok - (int64_t)b * p.T) : 0;
        const Token k = find_token(p, b, t, false);
        if (in && !k.ok && g == 0) atomicOr(p.status, kStatusIndex);
        float cs[V], sn[V];
        load_turn<V>(p, k.pos, g, turn && in && k.ok, cs, sn);
        const float fill = k.ok ? 0.f : __int_as_float(0x7fc00000);
        const T* x0 = static_cast<const T*>(s.x) + b * s.sx[0] + t * s.sx[2];
        const T* g0 = static_cast<const T*>(s.g) + b * s.sg[0] + t * s.sg[2];
        T* y0 = static_cast<T*>(s.y) + b * s.sy[0] + t * s.sy[2];
#pragma unroll 2
        for (int h = head0; h < head1; ++h) {
            float x[2 * V] = {}, u[2 * V] = {};
            if (in) {
                if (p.norm) {
                    Vec<T>::load(x0 + h * s.sx[1] + oa, x);
                    Vec<T>::load(x0 + h * s.sx[1] + ob, x + V);
                }
                Vec<T>::load(g0 + h * s.sg[1] + oa, u);
                Vec<T>::load(g0 + h * s.sg[1] + ob, u + V);
            }
            float e0[V], e1[V];
            to_pairs<V, INTER>(u, e0, e1);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float v = e0[i] * cs[i] + e1[i] * sn[i] + fill;
                e1[i] = e1[i] * cs[i] - e0[i] * sn[i] + fill;
                e0[i] = v;
            }
            from_pairs<V, INTER>(e0, e1, u);
            if (p.norm) {
                if (weighted && s.w_stride) {
#pragma unroll
                    for (int i = 0; i < V; i += 4) {
                        Vec<float>::load(s.weight + h * s.w_stride + oa + i, w + i);
                        Vec<float>::load(s.weight + h * s.w_stride + ob + i, w + V + i);
                    }
                }
                float ss = 0.f, sx = 0.f;
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) {
                    ss = fmaf(x[i], x[i], ss);
                    sx = fmaf(w[i] * u[i], x[i], sx);
                }
                const float r = 1.0f / sqrtf(group_sum<G>(ss) / p.D + p.eps);
                const float m = group_sum<G>(sx) / p.D * r * r;
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) {
                    dw[i] = fmaf(u[i] * r, x[i], dw[i]);
                    u[i] = r * (w[i] * u[i] - x[i] * m);
                }
            }
            if (in) {
                Vec<T>::store(y0 + h * s.sy[1] + oa, u);
                Vec<T>::store(y0 + h * s.sy[1] + ob, u + V);
            }
        }
    }
    if (!p.norm || !p.dw[s.grad_slot]) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        red[group * D + oa + i] = dw[i];
        red[group * D + ob + i] = dw[V + i];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += THREADS) {
        float sum = 0.f;
        for (int j = 0; j < GROUPS; ++j) sum += red[j * D + c];
        p.partial[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * D + c] = sum;
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS)
rotary_bwd_any_kernel(const RotaryParams p) {
    constexpr int WARPS = THREADS / 32;
    constexpr int E = MAX_D / 32;
    __shared__ float rows[WARPS][MAX_D];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    float* row = rows[warp];
    int head0;
    const int si = find_stream(p, blockIdx.y, &head0);      // one head a block here
    const RowStream& s = p.s[si];
    const float* w = p.norm && s.weight ? s.weight + head0 * s.w_stride : nullptr;
    const int half = p.R / 2;
    const int64_t tokens = (int64_t)p.B * p.T;
    float dw[E] = {};
    for (int64_t tok = (int64_t)blockIdx.x * WARPS + warp; tok < tokens; tok += (int64_t)gridDim.x * WARPS) {
        const int b = (int)(tok / p.T);
        const int t = (int)(tok - (int64_t)b * p.T);
        const Token k = find_token(p, b, t, false);
        if (!k.ok && lane == 0) atomicOr(p.status, kStatusIndex);
        const T* x = static_cast<const T*>(s.x) + b * s.sx[0] + head0 * s.sx[1] + t * s.sx[2];
        const T* gr = static_cast<const T*>(s.g) + b * s.sg[0] + head0 * s.sg[1] + t * s.sg[2];
        T* y = static_cast<T*>(s.y) + b * s.sy[0] + head0 * s.sy[1] + t * s.sy[2];
        for (int i = lane; i < p.D; i += 32) row[i] = Vec<T>::get(gr[i]);
        __syncwarp();
        float u[E], xv[E], ss = 0.f, sx = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = lane + 32 * e;
            u[e] = xv[e] = 0.f;
            if (i >= p.D) continue;
            float v = row[i];
            if (!k.ok) {
                v = __int_as_float(0x7fc00000);
            } else if (i < p.R) {
                const int j = p.interleaved ? i / 2 : (i < half ? i : i - half);
                const bool first = p.interleaved ? (i & 1) == 0 : i < half;
                const float other = row[p.interleaved ? i ^ 1 : (first ? i + half : i - half)];
                const float cs = p.cos[k.pos * half + j], sn = p.sin[k.pos * half + j];
                v = first ? v * cs + other * sn : v * cs - other * sn;
            }
            u[e] = v;
            if (p.norm) {
                xv[e] = Vec<T>::get(x[i]);
                ss = fmaf(xv[e], xv[e], ss);
                sx = fmaf((w ? w[i] : 1.f) * v, xv[e], sx);
            }
        }
        __syncwarp();                   // the next token's row overwrites this one
        if (p.norm) {
            const float r = 1.0f / sqrtf(group_sum<32>(ss) / p.D + p.eps);
            const float m = group_sum<32>(sx) / p.D * r * r;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = lane + 32 * e;
                dw[e] = fmaf(u[e] * r, xv[e], dw[e]);
                u[e] = r * ((w && i < p.D ? w[i] : 1.f) * u[e] - xv[e] * m);
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (lane + 32 * e < p.D) y[lane + 32 * e] = Vec<T>::put(u[e]);
    }
    if (!p.norm || !p.dw[s.grad_slot]) return;
#pragma unroll
    for (int e = 0; e < E; ++e) row[lane + 32 * e] = dw[e];
    __syncthreads();
    for (int c = threadIdx.x; c < p.D; c += THREADS) {
        float sum = 0.f;
        for (int j = 0; j < WARPS; ++j) sum += rows[j][c];
        p.partial[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * p.D + c] = sum;
    }
}

// dw from the blocks' partial rows: one block an output row (a head, or all of them),
// the q weight's rows first.  Eight parts of the partials, then their sum: a fixed order.
constexpr int RED_PARTS = 8;
__global__ void __launch_bounds__(RED_PARTS * MAX_D)
rotary_dw_kernel(const RotaryParams p, int q_rows) {
    __shared__ float red[RED_PARTS][MAX_D];
    const int slot = (int)blockIdx.x < q_rows ? 0 : 1;
    const int out_row = slot ? blockIdx.x - q_rows : blockIdx.x;
    const int c = threadIdx.x % MAX_D, part = threadIdx.x / MAX_D;
    float sum = 0.f;
    int block0 = 0;
    for (int i = 0; i < p.n; ++i) {
        const int nb = (p.s[i].heads + p.heads_per_block - 1) / p.heads_per_block;
        if (p.s[i].grad_slot == slot && c < p.D) {
            const int first = p.dw_stride[slot] ? block0 + out_row : block0;
            const int last = p.dw_stride[slot] ? first + 1 : block0 + nb;
            const float* src = p.partial + (int64_t)first * p.chunks * p.D + c;
            const int n = (last - first) * p.chunks;
            for (int j = part; j < n; j += RED_PARTS) sum += src[(int64_t)j * p.D];
        }
        block0 += nb;
    }
    red[part][c] = sum;
    __syncthreads();
    if (part == 0 && c < p.D) {
        float total = 0.f;
#pragma unroll
        for (int i = 0; i < RED_PARTS; ++i) total += red[i][c];
        p.dw[slot][out_row * p.dw_stride[slot] + c] = total;
    }
}

template <typename T, bool INTER>
int launch_fast(const RotaryParams& p, bool backward, cudaStream_t stream) {
    constexpr int V = Vec<T>::N;
    const int G = p.D / (2 * V);
    const int64_t tokens = (int64_t)p.B * p.T;
    const dim3 grid((unsigned)(backward ? p.chunks : (tokens * G + THREADS - 1) / THREADS), (unsigned)p.head_blocks);
#define DIFFATTN_ROTARY(GG)                                                               \
    if (G == GG) {                                                                        \
        if (backward) rotary_bwd_kernel<T, GG, INTER><<<grid, THREADS, 0, stream>>>(p);   \
        else rotary_kernel<T, GG, INTER><<<grid, THREADS, 0, stream>>>(p);                \
        return cudaGetLastError() == cudaSuccess ? 0 : -1;                                \
    }
    DIFFATTN_ROTARY(2)
    DIFFATTN_ROTARY(4)
    DIFFATTN_ROTARY(8)
    if constexpr (sizeof(T) == 4) { DIFFATTN_ROTARY(16) }
#undef DIFFATTN_ROTARY
    return -1;
}

int launch(const RotaryParams& p, bool backward, cudaStream_t stream) {
    if (p.fast) {
        if (p.bf16) return p.interleaved ? launch_fast<__nv_bfloat16, true>(p, backward, stream)
                                         : launch_fast<__nv_bfloat16, false>(p, backward, stream);
        return p.interleaved ? launch_fast<float, true>(p, backward, stream)
                             : launch_fast<float, false>(p, backward, stream);
    }
    constexpr int WARPS = THREADS / 32;
    const int64_t tokens = (int64_t)p.B * p.T;
    const dim3 grid((unsigned)(backward ? p.chunks : (tokens + WARPS - 1) / WARPS), (unsigned)p.head_blocks);
    if (backward) {
        if (p.bf16) rotary_bwd_any_kernel<__nv_bfloat16><<<grid, THREADS, 0, stream>>>(p);
        else rotary_bwd_any_kernel<float><<<grid, THREADS, 0, stream>>>(p);
    } else {
        if (p.bf16) rotary_any_kernel<__nv_bfloat16><<<grid, THREADS, 0, stream>>>(p);
        else rotary_any_kernel<float><<<grid, THREADS, 0, stream>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

void set_head_blocks(RotaryParams* p, int hpb) {
    p->heads_per_block = hpb;
    p->head_blocks = 0;
    for (int i = 0; i < p->n; ++i) p->head_blocks += (p->s[i].heads + hpb - 1) / hpb;
}

}  // namespace rot

// Enough blocks for a few waves of every SM, then as many heads a block as that
// leaves (16 at most: the registers that hold the token's cosines are paid for by then).
void plan_rotary(RotaryParams* p, int num_sms) {
    int heads = 0;
    for (int i = 0; i < p->n; ++i) heads += p->s[i].heads;
    int hpb = 1;
    if (p->fast) {
        const int lanes = p->D / (p->bf16 ? 16 : 8);
        const int64_t blocks = ((int64_t)p->B * p->T * lanes + rot::THREADS - 1) / rot::THREADS * heads;
        const int64_t want = blocks / (16ll * num_sms);
        hpb = want < 1 ? 1 : want > 16 ? 16 : (int)want;
    }
    rot::set_head_blocks(p, hpb);
}

// The backward's blocks must not depend on the GPU: the workspace is sized for them.
void plan_rotary_bwd(RotaryParams* p) {
    const bool per_head = p->norm && ((p->dw[0] && p->dw_stride[0]) || (p->dw[1] && p->dw_stride[1]));
    rot::set_head_blocks(p, !p->fast || per_head ? 1 : 4);
    const int groups = p->fast ? rot::THREADS / (p->D / (p->bf16 ? 16 : 8)) : rot::THREADS / 32;
    const int64_t steps = ((int64_t)p->B * p->T + groups - 1) / groups;
    int64_t chunks = (2432 + p->head_blocks - 1) / p->head_blocks;
    p->chunks = (int)(chunks < steps ? chunks : steps);
}

int launch_rotary(const RotaryParams& p, cudaStream_t stream) { return rot::launch(p, false, stream); }

int launch_rotary_bwd(const RotaryParams& p, cudaStream_t stream) {
    if (rot::launch(p, true, stream) != 0) return -1;
    if (!p.norm || (!p.dw[0] && !p.dw[1])) return 0;
    int heads[2] = {0, 0};
    for (int i = 0; i < p.n; ++i) heads[p.s[i].grad_slot] = p.s[i].heads;
    const int q_rows = !p.dw[0] ? 0 : p.dw_stride[0] ? heads[0] : 1;
    const int k_rows = !p.dw[1] ? 0 : p.dw_stride[1] ? heads[1] : 1;
    rot::rotary_dw_kernel<<<q_rows + k_rows, rot::RED_PARTS * rot::MAX_D, 0, stream>>>(p, q_rows);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace diffattn
