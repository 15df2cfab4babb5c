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
//
// Measured: 2 x 8192 tokens of 64 heads of 64 in bf16 take 51.5 us (5.3 TB/s, 0.78 of the
// copy rate; half of an SM's issue slots are arithmetic and conversions, see Vec); a decode
// step of 16 tokens 2.8 us and an append of as many 2.9, a launch's latency; 4 x 2047 tokens
// appended with 8 heads of 128 15.5 us (3.7 TB/s: a fourth of it is the grid's start and
// end).  The kernels start while the stream's last one ends and wait for it before they
// read (calls among others: 18.5 to 16.0 us for that append).
#include "paged.h"
#include "ptx.cuh"
#include "pdl.cuh"

namespace diffattn {
namespace rot {

constexpr int THREADS = 256;
constexpr int MAX_D = 128;
constexpr int BWD_STEPS = 3;    // rows of each group of lanes in an item of the backward,
constexpr int BWD_STAGES = 3;   // and rows on their way
// Blocks of the backward for any layout, and partial rows that they leave, in all: a number of its
// own (16 for each of 152 SMs), since the workspace's size must not depend on the current device.
constexpr int BWD_ANY_BLOCKS = 2432;

// 16 bytes of elements, N of them, as N / 2 packed pairs of floats (two elements an
// instruction: at an SM's share of the HBM rate the arithmetic is half of the time).
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ void unpack(uint4 v, uint64_t* x) {
        x[0] = f2_from_bits(v.x, v.y);
        x[1] = f2_from_bits(v.z, v.w);
    }
    __device__ static __forceinline__ uint4 pack(const uint64_t* x) {
        return make_uint4((uint32_t)x[0], (uint32_t)(x[0] >> 32), (uint32_t)x[1], (uint32_t)(x[1] >> 32));
    }
    __device__ static __forceinline__ float get(float v) { return v; }
    __device__ static __forceinline__ float put(float v) { return v; }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static __forceinline__ void unpack(uint4 v, uint64_t* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = f2_from_bits(w[i] << 16, w[i] & 0xffff0000u);
    }
    __device__ static __forceinline__ uint4 pack(const uint64_t* x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(f2_lo(x[i]), f2_hi(x[i]));
        return make_uint4(w[0], w[1], w[2], w[3]);
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

// V floats as V / 2 packed pairs.
template <int V>
__device__ __forceinline__ void load_pairs(const float* p, uint64_t* x) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
        x[2 * i] = f2_from_bits(v.x, v.y);
        x[2 * i + 1] = f2_from_bits(v.z, v.w);
    }
}

// Turn the lane's V pairs of elements, c[0 .. V/2) from its first chunk and c[V/2 .. V)
// from its second, by the angles with these cosines and sines (negated for the backward).
template <int V, bool INTER>
__device__ __forceinline__ void rotate(uint64_t* c, const uint64_t* cs, const uint64_t* sn, bool back) {
    if constexpr (INTER) {
        // both elements of a pair are in one register pair
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float co = i & 1 ? f2_hi(cs[i / 2]) : f2_lo(cs[i / 2]);
            const float s0 = i & 1 ? f2_hi(sn[i / 2]) : f2_lo(sn[i / 2]), si = back ? -s0 : s0;
            const float a = f2_lo(c[i]), b = f2_hi(c[i]);
            c[i] = f2_pack(a * co - b * si, b * co + a * si);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const uint64_t a = c[i], b = c[V / 2 + i];
            const uint64_t p = f2_mul(a, sn[i]), q = f2_mul(b, sn[i]);
            if (back) {
                c[i] = f2_fma(a, cs[i], q);
                c[V / 2 + i] = f2_sub(f2_mul(b, cs[i]), p);
            } else {
                c[i] = f2_sub(f2_mul(a, cs[i]), q);
                c[V / 2 + i] = f2_fma(b, cs[i], p);
            }
        }
    }
}

// Sum of both halves of V packed pairs.
template <int V>
__device__ __forceinline__ float pair_sum(const uint64_t* x) {
    uint64_t s = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) s = f2_add(s, x[i]);
    return f2_lo(s) + f2_hi(s);
}

template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// ---------------------------------------------------------------------------
// forward and append
//
// A thread's loads are what hides the HBM's latency: four heads' chunks (128 bytes) go
// out together, the first four before the token's position is even known, since the
// chain position - table row - arithmetic is as long as theirs.
// ---------------------------------------------------------------------------
constexpr int AHEAD = 4;        // heads

template <typename T, int G, bool INTER>
__global__ void __launch_bounds__(THREADS, 3)
rotary_kernel(const RotaryParams p) {
    constexpr int V = Vec<T>::N;
    constexpr int TOKENS = THREADS / G;
    const int g = threadIdx.x % G;
    pdl_wait();
    pdl_launch_dependents();
    int head0;
    const int si = find_stream(p, blockIdx.y, &head0);
    const RowStream& s = p.s[si];
    const int head1 = min(s.heads, head0 + p.heads_per_block);
    const bool paged = s.kind != kRowsDense;
    // the lanes of a group share a token; a group past the last token only takes
    // part in the warp's shuffles
    const int tok = blockIdx.x * TOKENS + threadIdx.x / G;
    const bool in = tok < p.B * p.T;
    const int b = in ? p.by_T.div(tok) : 0;
    const int t = in ? tok - b * p.T : 0;
    const T* x0 = static_cast<const T*>(s.x) + b * s.sx[0] + t * s.sx[2];
    if (s.kind == kRowsCopy) {
        const Token k = find_token(p, b, t, true);
        if (in && k.live && !k.ok && g == 0) atomicOr(p.status, kStatusIndex);
        if (!in || !k.live || !k.ok) return;
        T* y0 = static_cast<T*>(s.y) + k.page * s.sy[0] + k.slot * s.sy[2];
        // two heads and two chunks at a time
        for (int h = head0; h < head1; h += 2)
            for (int c = g * V; c < s.width; c += 2 * G * V) {
                uint4 v[2][2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (h + i < head1 && c + j * G * V < s.width)
                            v[i][j] = *reinterpret_cast<const uint4*>(x0 + (h + i) * s.sx[1] + c + j * G * V);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (h + i < head1 && c + j * G * V < s.width)
                            *reinterpret_cast<uint4*>(y0 + (h + i) * s.sy[1] + c + j * G * V) = v[i][j];
            }
        return;
    }
    int oa, ob;
    const bool turn = chunk_offsets<V, INTER>(g, p.R, &oa, &ob);
    uint4 raw[AHEAD][2];
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
            if (in && h + i < head1) {
                raw[i][0] = *reinterpret_cast<const uint4*>(x0 + (h + i) * s.sx[1] + oa);
                raw[i][1] = *reinterpret_cast<const uint4*>(x0 + (h + i) * s.sx[1] + ob);
            }
        }
    };
    load(head0);
    Token k = find_token(p, b, t, paged);
    k.live = k.live && in;
    if (k.live && !k.ok && g == 0) atomicOr(p.status, kStatusIndex);
    const bool write = k.live && (k.ok || !paged);
    T* y0 = static_cast<T*>(s.y) + (paged ? k.page * s.sy[0] + k.slot * s.sy[2] : b * s.sy[0] + t * s.sy[2]);
    uint64_t cs[V / 2], sn[V / 2];
    const bool turned = turn && k.live && k.ok;
    if (turned) {
        load_pairs<V>(p.cos + k.pos * (p.R / 2) + g * V, cs);
        load_pairs<V>(p.sin + k.pos * (p.R / 2) + g * V, sn);
    }
    const bool weighted = p.norm && s.weight;
    for (int h0 = head0; h0 < head1; h0 += AHEAD) {
        if (h0 > head0) load(h0);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int h = h0 + i;
            if (h >= head1) break;
            uint64_t c[V];
            Vec<T>::unpack(raw[i][0], c);
            Vec<T>::unpack(raw[i][1], c + V / 2);
            if (p.norm) {
                uint64_t sq[V];
#pragma unroll
                for (int e = 0; e < V; ++e) sq[e] = f2_mul(c[e], c[e]);
                // (off by 2 units in the last place at most: float32 rows 1.5e-7 where a root and
                // a division give 1.2e-7)
                const float r = rsqrtf(group_sum<G>(pair_sum<V>(sq)) * p.inv_D + p.eps);
                const uint64_t r2 = f2_pack(r, r);
                if (weighted) {             // from L1: the registers are worth more blocks an SM
                    uint64_t w[V];
                    load_pairs<V>(s.weight + h * s.w_stride + oa, w);
                    load_pairs<V>(s.weight + h * s.w_stride + ob, w + V / 2);
#pragma unroll
                    for (int e = 0; e < V; ++e) c[e] = f2_mul(c[e], f2_mul(r2, w[e]));
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) c[e] = f2_mul(c[e], r2);
                }
            }
            if (turned) rotate<V, INTER>(c, cs, sn, false);
            if (!k.ok) {                    // a position outside the tables
#pragma unroll
                for (int e = 0; e < V; ++e) c[e] = 0x7fc000007fc00000ull;
            }
            if (write) {
                *reinterpret_cast<uint4*>(y0 + h * s.sy[1] + oa) = Vec<T>::pack(c);
                *reinterpret_cast<uint4*>(y0 + h * s.sy[1] + ob) = Vec<T>::pack(c + V / 2);
            }
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
    pdl_wait();
    pdl_launch_dependents();
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
// Reads x and dy, writes dx: bound by HBM.  An item is one head over a chunk of tokens
// (BWD_STEPS rows for each group of lanes); the items are laid out head by head, chunk by
// chunk, and every block, two an SM, takes an equal run of them.  A chunk's cosines and
// sines stay in shared memory for its heads: read for each head from L2 they were as much
// traffic as dy, behind the position's own latency.  Rows of x and dy come by cp.async,
// BWD_STAGES ahead, each thread's own (96 KB an SM on their way; one row ahead in registers
// kept the HBM at 2.8 TB/s), and so do an item's weights.  Each lane keeps the dw of its
// own 2 V channels in registers, and an item leaves one partial row: the sum's order is
// fixed, without atomics.
// ---------------------------------------------------------------------------
// Shared memory of a backward block, in floats: ring, tables, sums, weights, flags.
struct BwdLayout {
    int turns, red, weights, fine, total;
};
__host__ __device__ constexpr BwdLayout bwd_layout(int groups, int D, int R) {
    BwdLayout l{};
    l.turns = BWD_STAGES * 4 * THREADS * 4;                 // ring: [stage][x, x, dy, dy][thread] of 16 bytes
    l.red = l.turns + BWD_STEPS * groups * R;               // [token of the chunk][cos R/2, sin R/2]
    l.weights = l.red + THREADS / 32 * D;                   // [warp][D]
    l.fine = l.weights + 2 * D;                             // [item & 1][D]
    l.total = l.fine + BWD_STEPS * groups;                  // int [token]: its position is in the tables
    return l;
}

template <typename T, int G, bool INTER>
__global__ void __launch_bounds__(THREADS, 2)
rotary_bwd_kernel(const RotaryParams p) {
    constexpr int V = Vec<T>::N;
    constexpr int GROUPS = THREADS / G;
    constexpr int D = G * 2 * V;
    extern __shared__ __align__(16) float smem_f[];
    const BwdLayout L = bwd_layout(GROUPS, D, p.R);
    uint4* ring = reinterpret_cast<uint4*>(smem_f);
    float* turns = smem_f + L.turns;
    float* red = smem_f + L.red;
    float* weights = smem_f + L.weights;
    int* fine = reinterpret_cast<int*>(smem_f + L.fine);
    const int tid = threadIdx.x, g = tid % G, group = tid / G;
    const int lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();
    const int half = p.R / 2;
    const int tokens = p.B * p.T;
    const int items = p.chunks * p.heads;                   // checked on the host to fit
    const int row0 = (int)((int64_t)blockIdx.x * items / gridDim.x) * BWD_STEPS;
    const int row1 = (int)((int64_t)(blockIdx.x + 1) * items / gridDim.x) * BWD_STEPS;
    int oa, ob;
    const bool turn = chunk_offsets<V, INTER>(g, p.R, &oa, &ob);
    uint64_t dw[V];

    // Row i of this group: its stream and head, and its token; b < 0: there is none.
    struct Row {
        int item, step, si, h, b, t;
    };
    auto row_of = [&](int i) {
        Row r;
        r.item = i / BWD_STEPS;
        r.step = i - r.item * BWD_STEPS;
        const int chunk = p.by_heads.div(r.item);
        r.h = r.item - chunk * p.heads;
        for (r.si = 0; r.h >= p.s[r.si].heads; ++r.si) r.h -= p.s[r.si].heads;
        const int tok = (chunk * BWD_STEPS + r.step) * GROUPS + group;
        r.b = tok < tokens ? p.by_T.div(tok) : -1;
        r.t = tok - r.b * p.T;
        return r;
    };
    auto load = [&](int i) {
        if (i < row1) {
            const Row r = row_of(i);
            const RowStream& s = p.s[r.si];
            uint4* at = ring + (i % BWD_STAGES) * 4 * THREADS + tid;
            if (r.b >= 0) {
                if (p.norm) {
                    const T* x = static_cast<const T*>(s.x) + r.b * s.sx[0] + r.h * s.sx[1] + r.t * s.sx[2];
                    cp_async16(at, x + oa);
                    cp_async16(at + THREADS, x + ob);
                }
                const T* gr = static_cast<const T*>(s.g) + r.b * s.sg[0] + r.h * s.sg[1] + r.t * s.sg[2];
                cp_async16(at + 2 * THREADS, gr + oa);
                cp_async16(at + 3 * THREADS, gr + ob);
            }
            if (r.step == 0 && s.weight && tid < D / 4)
                cp_async16(weights + (r.item & 1) * D + 4 * tid, s.weight + r.h * s.w_stride + 4 * tid);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // The tables of a chunk's tokens; the caller has the barriers.
    auto enter = [&](int chunk) {
        const int tok0 = chunk * (BWD_STEPS * GROUPS), per = max(half / 4, 1);
        for (int i = tid; i < BWD_STEPS * GROUPS * per; i += THREADS) {
            const int k = i / per, c = (i - k * per) * 4;
            if (tok0 + k >= tokens) continue;
            const int b = p.by_T.div(tok0 + k);
            const Token at = find_token(p, b, tok0 + k - b * p.T, false);
            if (c == 0) {
                fine[k] = at.ok;
                if (!at.ok) atomicOr(p.status, kStatusIndex);
            }
            if (!at.ok || half == 0) continue;
            *reinterpret_cast<float4*>(turns + k * p.R + c) = *reinterpret_cast<const float4*>(p.cos + at.pos * half + c);
            *reinterpret_cast<float4*>(turns + k * p.R + half + c) = *reinterpret_cast<const float4*>(p.sin + at.pos * half + c);
        }
    };
    // The item's partial row: sums of the groups in a fixed order.  (The next write of `red`
    // comes after the next item's first barrier.)
    auto leave = [&](int item) {
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) {
            float v = i & 1 ? f2_hi(dw[i / 2]) : f2_lo(dw[i / 2]);
#pragma unroll
            for (int o = G; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane < G) red[warp * D + (i < V ? oa + i : ob + i - V)] = v;
        }
        __syncthreads();
        for (int c = tid; c < D; c += THREADS) {
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < THREADS / 32; ++j) sum += red[j * D + c];
            p.partial[(int64_t)item * D + c] = sum;         // [chunk][head]
        }
    };
#pragma unroll
    for (int i = 0; i < BWD_STAGES - 1; ++i) load(row0 + i);
    int chunk = -1;
    for (int i = row0; i < row1; ++i) {
        load(i + BWD_STAGES - 1);
        const Row r = row_of(i);
        const RowStream& s = p.s[r.si];
        asm volatile("cp.async.wait_group %0;" ::"n"(BWD_STAGES - 1) : "memory");
        if (r.step == 0) {                  // a new item: its weights are there, and its tables
#pragma unroll
            for (int e = 0; e < V; ++e) dw[e] = 0;
            __syncthreads();
            if (p.by_heads.div(r.item) != chunk) {
                enter(chunk = p.by_heads.div(r.item));
                __syncthreads();
            }
        }
        const uint4* at = ring + (i % BWD_STAGES) * 4 * THREADS + tid;
        const int k = r.step * GROUPS + group;
        const bool none = r.b < 0;
        uint64_t x[V], u[V];
        Vec<T>::unpack(at[2 * THREADS], u);
        Vec<T>::unpack(at[3 * THREADS], u + V / 2);
        if (turn) {
            uint64_t cs[V / 2], sn[V / 2];
            load_pairs<V>(turns + k * p.R + g * V, cs);
            load_pairs<V>(turns + k * p.R + half + g * V, sn);
            rotate<V, INTER>(u, cs, sn, true);
        }
        if (none || !fine[k]) {                             // no token: nothing; no position: NaN
#pragma unroll
            for (int e = 0; e < V; ++e) u[e] = none ? 0ull : 0x7fc000007fc00000ull;
        }
        if (p.norm) {
            Vec<T>::unpack(at[0], x);
            Vec<T>::unpack(at[THREADS], x + V / 2);
            if (none) {
#pragma unroll
                for (int e = 0; e < V; ++e) x[e] = 0ull;
            }
            uint64_t g2[V], s1 = 0, s2 = 0;                 // w u, and the sums of x x and w u x
            if (s.weight) {
                load_pairs<V>(weights + (r.item & 1) * D + oa, g2);
                load_pairs<V>(weights + (r.item & 1) * D + ob, g2 + V / 2);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                g2[e] = s.weight ? f2_mul(g2[e], u[e]) : u[e];
                s1 = f2_fma(x[e], x[e], s1);
                s2 = f2_fma(g2[e], x[e], s2);
            }
            const float rr = rsqrtf(group_sum<G>(f2_lo(s1) + f2_hi(s1)) * p.inv_D + p.eps);
            const float m = -(group_sum<G>(f2_lo(s2) + f2_hi(s2)) * p.inv_D * rr * rr * rr);
            const uint64_t rr2 = f2_pack(rr, rr), m2 = f2_pack(m, m);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                dw[e] = f2_fma(f2_mul(u[e], rr2), x[e], dw[e]);
                u[e] = f2_fma(x[e], m2, f2_mul(g2[e], rr2));
            }
        }
        if (!none) {
            T* y = static_cast<T*>(s.y) + r.b * s.sy[0] + r.h * s.sy[1] + r.t * s.sy[2];
            *reinterpret_cast<uint4*>(y + oa) = Vec<T>::pack(u);
            *reinterpret_cast<uint4*>(y + ob) = Vec<T>::pack(u + V / 2);
        }
        if (r.step == BWD_STEPS - 1 && p.norm && p.dw[s.grad_slot]) leave(r.item);
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
    pdl_launch_dependents();
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
    // one head a block: its number among all heads is the block's
    for (int c = threadIdx.x; c < p.D; c += THREADS) {
        float sum = 0.f;
        for (int j = 0; j < WARPS; ++j) sum += rows[j][c];
        p.partial[((int64_t)blockIdx.x * p.heads + blockIdx.y) * p.D + c] = sum;
    }
}

// dw from the blocks' partial rows: a block an output row (a head, or all of them), the q
// weight's rows first, with the partial rows spread over its warps and lanes' columns.  The
// order of the sums is fixed.
constexpr int RED_THREADS = 1024;
__global__ void __launch_bounds__(RED_THREADS)
rotary_dw_kernel(const RotaryParams p, int q_rows) {
    __shared__ float red[RED_THREADS];
    pdl_wait();
    const int slot = (int)blockIdx.x < q_rows ? 0 : 1;
    const int out_row = slot ? blockIdx.x - q_rows : blockIdx.x;
    const bool by_head = p.dw_stride[slot] != 0;
    const int cols = p.D <= 32 ? 32 : p.D <= 64 ? 64 : 128, parts = RED_THREADS / cols;
    const int c = threadIdx.x % cols, part = threadIdx.x / cols;
    float sum = 0.f;
    int heads = 0;
    for (int i = 0; i < p.n; ++i) {
        if (p.s[i].grad_slot == slot && c < p.D) {
            const int rows = by_head ? 1 : p.s[i].heads, first = heads + (by_head ? out_row : 0);
            const int n = rows * p.chunks;
#pragma unroll 8
            for (int j = part; j < n; j += parts) {
                const int chunk = j / rows;
                sum += p.partial[((int64_t)chunk * p.heads + first + j - chunk * rows) * p.D + c];
            }
        }
        heads += p.s[i].heads;
    }
    red[threadIdx.x] = sum;
    __syncthreads();
    if (part == 0 && c < p.D) {
        float total = 0.f;
        for (int i = 0; i < parts; ++i) total += red[i * cols + c];
        p.dw[slot][out_row * p.dw_stride[slot] + c] = total;
    }
}

template <typename T, int G, bool INTER>
int launch_bwd(const RotaryParams& p, dim3 grid, cudaStream_t stream) {
    constexpr int D = G * 2 * Vec<T>::N, GROUPS = THREADS / G;
    const auto bytes = [](int R) { return bwd_layout(GROUPS, D, R).total * 4; };
    if (cudaFuncSetAttribute(rotary_bwd_kernel<T, G, INTER>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(D)) !=
        cudaSuccess)
        return -1;
    rotary_bwd_kernel<T, G, INTER><<<grid, THREADS, bytes(p.R), stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <typename T, bool INTER>
int launch_fast(const RotaryParams& p, bool backward, cudaStream_t stream) {
    constexpr int V = Vec<T>::N;
    const int G = p.D / (2 * V);
    const int64_t tokens = (int64_t)p.B * p.T;
    const dim3 grid((unsigned)(backward ? p.head_blocks : (tokens * G + THREADS - 1) / THREADS),
                    backward ? 1u : (unsigned)p.head_blocks);
#define DIFFATTN_ROTARY(GG)                                                               \
    if (G == GG) {                                                                        \
        if (backward) return launch_bwd<T, GG, INTER>(p, grid, stream);                   \
        return pdl_launch(rotary_kernel<T, GG, INTER>, grid, THREADS, 0, stream, p);      \
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
    if (!backward)
        return pdl_launch(p.bf16 ? rotary_any_kernel<__nv_bfloat16> : rotary_any_kernel<float>, grid, THREADS, 0, stream, p);
    if (p.bf16) rotary_bwd_any_kernel<__nv_bfloat16><<<grid, THREADS, 0, stream>>>(p);
    else rotary_bwd_any_kernel<float><<<grid, THREADS, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

void set_head_blocks(RotaryParams* p, int hpb) {
    p->heads_per_block = hpb;
    p->head_blocks = 0;
    for (int i = 0; i < p->n; ++i) p->head_blocks += (p->s[i].heads + hpb - 1) / hpb;
}

}  // namespace rot

// As many heads a block as leave a few blocks for every SM (16 at most: the registers that
// hold the token's cosines are paid for by then), in whole batches of loads.
void plan_rotary(RotaryParams* p, int num_sms) {
    int heads = 0;
    for (int i = 0; i < p->n; ++i) heads += p->s[i].heads;
    int hpb = 1;
    if (p->fast) {
        const int lanes = p->D / (p->bf16 ? 16 : 8);
        const int64_t blocks = ((int64_t)p->B * p->T * lanes + rot::THREADS - 1) / rot::THREADS * heads;
        const int64_t want = blocks / (8ll * num_sms);
        hpb = want < 1 ? 1 : want < rot::AHEAD ? (int)want : want > 16 ? 16 : (int)want / rot::AHEAD * rot::AHEAD;
    }
    rot::set_head_blocks(p, hpb);
}

// The backward's items (see rotary_bwd_kernel), and its blocks: two an SM (head_blocks).
void plan_rotary_bwd(RotaryParams* p, int num_sms) {
    p->heads = 0;
    for (int i = 0; i < p->n; ++i) p->heads += p->s[i].heads;
    p->by_heads.set((uint32_t)p->heads);
    const int64_t tokens = (int64_t)p->B * p->T;
    if (!p->fast) {                         // a head a block, and chunks in strides
        rot::set_head_blocks(p, 1);
        const int64_t steps = (tokens + 7) / 8, chunks = (rot::BWD_ANY_BLOCKS + p->heads - 1) / p->heads;
        p->chunks = (int)(chunks < steps ? chunks : steps);
        return;
    }
    const int per = rot::THREADS / (p->D / (p->bf16 ? 16 : 8)) * rot::BWD_STEPS;
    p->chunks = (int)((tokens + per - 1) / per);
    const int64_t items = (int64_t)p->chunks * p->heads;
    p->head_blocks = (int)(items < 2 * num_sms ? items : 2 * num_sms);
}

size_t rotary_bwd_floats(int64_t B, int64_t T, int64_t D, int64_t heads) {
    // at most: chunks of the fewest tokens a block takes (16 groups a step), a row a head
    const int64_t chunks = (B * T + 16 * rot::BWD_STEPS - 1) / (16 * rot::BWD_STEPS);
    const int64_t fast = chunks * heads, any = rot::BWD_ANY_BLOCKS + heads;
    return (size_t)((fast > any ? fast : any) * D);
}

int launch_rotary(const RotaryParams& p, cudaStream_t stream) { return rot::launch(p, false, stream); }

int launch_rotary_bwd(const RotaryParams& p, cudaStream_t stream) {
    if (rot::launch(p, true, stream) != 0) return -1;
    if (!p.norm || (!p.dw[0] && !p.dw[1])) return 0;
    int heads[2] = {0, 0};
    for (int i = 0; i < p.n; ++i) heads[p.s[i].grad_slot] = p.s[i].heads;
    const int q_rows = !p.dw[0] ? 0 : p.dw_stride[0] ? heads[0] : 1;
    const int k_rows = !p.dw[1] ? 0 : p.dw_stride[1] ? heads[1] : 1;
    return pdl_launch(rot::rotary_dw_kernel, dim3((unsigned)(q_rows + k_rows)), rot::RED_THREADS, 0, stream, p, q_rows);
}

}  // namespace diffattn
