// paged_mma.cu -- differential attention over a paged cache for up to 16 query rows a
// key/value head (single tokens, a few, small trees): bf16, value width 128, Q/K width
// 64 or 128, pages of a multiple of 16 slots.
//
// Bound by HBM: a key costs 4 D + 256 bytes (2 D + 256 with shared keys) and 4 (D + 128)
// operations a row, 192 FLOP a byte short of what the tensor cores could do even at 16
// rows.  So the design is about never leaving the memory idle:
//   - One producer warp streams the block's tiles of 64 keys through TMA into a ring
//     that takes most of shared memory, across unit boundaries, two or more tiles ahead.
//     A lane a page: box i of a tile is the part of it in one page.
//   - Four consumer warps take 16 keys of each tile each, and run on their own: a warp
//     keeps its own running maximum, sum and O (16 rows x 128 columns of both branches,
//     128 registers a thread), so a tile needs no barrier but the ring's two.  They meet
//     once a segment, when the four partial results are merged in the stage that was
//     read last.
//   - Two blocks an SM: one streams while the other starts or merges a segment.
//   - The products are warp-level (m16n8k16): at this size they are a quarter of the
//     time that the tile's bytes take, and P goes from the score's accumulators to the
//     next product's operand in registers.  A tcgen05 product would want 128 keys as its
//     M and P through shared memory with two block-wide barriers a tile (the layout of
//     the dense decode, 0.83 of the copy rate).
//
// Weights are 2^(s - m) against a running maximum that moves only when some weight would
// pass 2^8; they are rounded to bf16 for the product with V (half a step of 2^-8, as
// everywhere on the tensor cores), while their sum is taken unrounded in float32.
#include "paged_plan.cuh"
#include "kernels.h"
#include "pdl.cuh"

namespace diffattn {
namespace pmma {

constexpr int CONSUMERS = 4;                    // warps
// A second warpgroup for the producer (three of its warps idle), which gives registers to
// the consumers: 128 x 216 + 128 x 40 = 256 x 128, what the block is launched with.
constexpr int THREADS = 256;
constexpr int BLOCKS_PER_SM = kMmaBlocksPerSm;
constexpr uint32_t REGS_CONSUMER = 216, REGS_PRODUCER = 40;
static_assert(128 * REGS_CONSUMER + 128 * REGS_PRODUCER <= THREADS * 128, "register split");
constexpr int KT = kMmaTile;
constexpr int SLICE = KT / CONSUMERS;           // keys of a warp
constexpr int NR = 16;                          // rows of a unit
constexpr int DV = 128;
constexpr int PANEL = KT * 128;                 // 8 KB: 64 keys x 64 columns

template <int HD, bool KS>
struct Cfg {
    static constexpr int KP = HD / 64;                          // panels of a key tile
    static constexpr int NK = KS ? 1 : 2;
    static constexpr int STAGE = (NK * KP + 2) * PANEL;         // 24, 32 or 48 KB
    static constexpr int NST = 96 * 1024 / STAGE;
    static constexpr int OFF_V = NK * KP * PANEL;
    static constexpr int OFF_Q = NST * STAGE;                   // [branch][panel] 16 rows x 128 bytes
    static constexpr int Q_PANEL = NR * 128;
    static constexpr int OFF_STAT = OFF_Q + 2 * KP * Q_PANEL;   // float [warp][m, l][branch][row]
    static constexpr int OFF_BAR = OFF_STAT + CONSUMERS * 2 * 2 * NR * 4;
    static constexpr int OFF_MISC = OFF_BAR + 2 * NST * 8;      // abort, bad flags by stage
    static constexpr int SMEM = OFF_MISC + 64 + 1024;
    static constexpr int ROUND = STAGE / CONSUMERS / (2 * DV * 4);  // rows merged at once
    static_assert(BLOCKS_PER_SM * (SMEM + 256 + 1024) <= 228 * 1024, "shared memory");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16-byte chunk c of row r in the 128-byte swizzled layout that TMA writes.
__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ bool bf16x2_finite(uint32_t w) {
    return (w & 0x7f80u) != 0x7f80u && (w & 0x7f800000u) != 0x7f800000u;
}

// Bits of the slice's 16 keys, from k0 on, that a row sees (bit d of `tree`: new token d).
__device__ __forceinline__ uint32_t slice_mask(const PagedParams& p, const PagedSeq& s, int k0, bool live, int q,
                                               uint64_t tree) {
    if (!live) return 0;
    const int64_t off = s.before - k0;                  // keys of the slice before the new tokens, < 16
    uint32_t m;
    if (p.mask) {
        m = off <= 0 ? (uint32_t)(tree >> -off) : ((uint32_t)tree << off) | ((1u << off) - 1);
    } else {
        const int64_t n = off + q + 1;
        m = n <= 0 ? 0 : n >= SLICE ? 0xffffu : (1u << n) - 1;
    }
    const int n = s.total - k0;
    return m & (n >= SLICE ? 0xffffu : (1u << n) - 1);
}

template <int HD, bool KS>
__global__ void __launch_bounds__(THREADS, BLOCKS_PER_SM)
paged_mma_kernel(const __grid_constant__ CUtensorMap tm_k1, const __grid_constant__ CUtensorMap tm_k2,
                 const __grid_constant__ CUtensorMap tm_v, const PagedParams p, const int box_rows) {
    using C = Cfg<HD, KS>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int64_t scan[THREADS / 32 + 1];
    __shared__ PagedStart start_s;
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* empty = full + C::NST;
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
    volatile uint32_t* bad_stage = abort_flag + 1;              // [NST]
    float* stat = reinterpret_cast<float*>(smem + C::OFF_STAT);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const AbortState ab{abort_flag, p.status};
    pdl_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < C::NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], CONSUMERS);
            bad_stage[i] = 0;
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    const PagedStart start = paged_start<THREADS>(p, KT, scan, &start_s);     // its barriers order the above
    PagedCursor cur;

    if (warp >= CONSUMERS) {
        // ---------------------------------------------------------------- producer
        regs_dec<REGS_PRODUCER>();
        if (warp > CONSUMERS) return;
        cur.begin(p, start, KT);
        if (lane == 0) {
            tma_prefetch_desc(&tm_k1);
            tma_prefetch_desc(&tm_k2);
            tma_prefetch_desc(&tm_v);
        }
        if (lane == 0) cur.no_join(p);
        const int boxes = KT / box_rows;
        uint32_t armed = 0;                     // tiles issued
        int st = 0;
        uint32_t ph = 1;                        // the first pass over the ring finds it free
        bool ok = true;
        for (; ok && !cur.done(); cur.next(p, KT)) {
            const int live = cur.live_tiles(p, KT);
            if (lane == 0) cur.join(p, start_s.total);
            // the page of this lane's box, one tile ahead
            auto look = [&](int i) -> int {
                const int key = (cur.tile0 + i) * KT + lane * box_rows;
                if (i >= live || lane >= boxes || key >= cur.s.total) return -2;        // nothing to load
                return paged_page(p, cur.b, key / p.page);
            };
            int page = look(0);
            for (int i = 0; i < live; ++i) {
                const int now = page;
                page = look(i + 1);
                if (!(ok = mbar_wait_warp(&empty[st], ph, ab))) break;
                const unsigned have = __ballot_sync(0xffffffffu, now >= 0);
                const bool bad = __any_sync(0xffffffffu, now == -1);
                if (lane == 0) {
                    if (bad) atomicOr(p.status, kStatusIndex);
                    bad_stage[st] = bad;
                    const uint32_t bytes = __popc(have) * box_rows * 128 * (C::NK * C::KP + 2);
                    if (bytes) mbar_arrive_expect_tx(&full[st], bytes);
                    else mbar_arrive(&full[st]);
                }
                __syncwarp();
                if (now >= 0) {
                    const int key = (cur.tile0 + i) * KT + lane * box_rows;
                    const int slot = key % p.page;
                    uint8_t* dst = smem + st * C::STAGE + lane * box_rows * 128;
#pragma unroll
                    for (int pn = 0; pn < C::KP; ++pn) {
                        tma_load_4d(dst + pn * PANEL, &tm_k1, &full[st], pn * 64, slot, cur.hk, now);
                        if (!KS) tma_load_4d(dst + (C::KP + pn) * PANEL, &tm_k2, &full[st], pn * 64, slot, cur.hk, now);
                    }
                    tma_load_4d(dst + C::OFF_V, &tm_v, &full[st], 0, slot, cur.hk, now);
                    tma_load_4d(dst + C::OFF_V + PANEL, &tm_v, &full[st], 64, slot, cur.hk, now);
                }
                ++armed;
                if (++st == C::NST) { st = 0; ph ^= 1; }
            }
        }
        // no copy may be in flight when the block ends: wait for the last phase of each stage
        for (uint32_t t = armed > C::NST ? armed - C::NST : 0; t < armed; ++t)
            mbar_wait_teardown(&full[t % C::NST], (t / C::NST) & 1u, 200ull * 1000ull * 1000ull);
        return;
    }

    // -------------------------------------------------------------------- consumers
    regs_inc<REGS_CONSUMER>();
    cur.begin(p, start, KT);
    const float sl2 = p.scale_log2;
    const float lam = p.lambda_dev ? __ldg(p.lambda_dev) : p.lambda;
    const int r0 = lane >> 2;                   // this thread's rows r0 and r0 + 8
    // lane addresses of the ldmatrix operands within the warp's 16 rows of a panel
    const int krow = warp * SLICE + (lane & 7) + ((lane >> 4) << 3), kch = (lane >> 3) & 1;
    const int vrow = warp * SLICE + (lane & 7) + (((lane >> 3) & 1) << 3), vch = lane >> 4;
    const int qrow = (lane & 7) + (((lane >> 3) & 1) << 3), qch = lane >> 4;
    int st = 0;
    uint32_t ph = 0;
    bool ok = true;                             // after a failed wait: no more work, but every barrier
    for (; !cur.done(); cur.next(p, KT)) {
        const int live = cur.live_tiles(p, KT);
        const PagedSeq s = cur.s;
        bool bad = s.bad;
        if (bad && tid == 0) atomicOr(p.status, kStatusIndex);
        // ---- the unit's queries, zeros for padding rows
        for (int i = tid; i < NR * 2 * (HD / 8); i += 32 * CONSUMERS) {
            const int c = i % (HD / 8), br = i / (HD / 8) & 1, r = i / (HD / 4);
            const PagedRow x = paged_row(p, cur.hk, cur.rc, r, s.n_new);
            uint4 w = make_uint4(0, 0, 0, 0);
            if (x.live && r < p.chunk_rows) {
                const __nv_bfloat16* src =
                    br ? static_cast<const __nv_bfloat16*>(p.q2) + cur.b * p.s_q2[0] + x.h * p.s_q2[1] + x.q * p.s_q2[2]
                       : static_cast<const __nv_bfloat16*>(p.q1) + cur.b * p.s_q1[0] + x.h * p.s_q1[1] + x.q * p.s_q1[2];
                src += c * 8;
                if (p.q16) {
                    w = *reinterpret_cast<const uint4*>(src);
                } else {
                    const uint16_t* e = reinterpret_cast<const uint16_t*>(src);
                    w = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16,
                                   e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
                }
            }
            *reinterpret_cast<uint4*>(smem + C::OFF_Q + (br * C::KP + (c >> 3)) * C::Q_PANEL + sw128(r, c & 7)) = w;
        }
        named_bar_sync(1, 32 * CONSUMERS);
        const PagedRow ra = paged_row(p, cur.hk, cur.rc, r0, s.n_new);
        const PagedRow rb = paged_row(p, cur.hk, cur.rc, r0 + 8, s.n_new);
        const bool la = ra.live && r0 < p.chunk_rows, lb = rb.live && r0 + 8 < p.chunk_rows;
        uint64_t ta = 0, tb = 0;
        if (p.mask && (cur.tile0 + live) * KT > s.before) {
            if (la) ta = paged_mask_bits(p, cur.b, ra.q, s.n_new);
            if (lb) tb = paged_mask_bits(p, cur.b, rb.q, s.n_new);
        }
        float o[2][DV / 8][4];
        float m[2][2], l[2][2];
#pragma unroll
        for (int br = 0; br < 2; ++br) {
            m[br][0] = m[br][1] = -INFINITY;
            l[br][0] = l[br][1] = 0.f;
#pragma unroll
            for (int n = 0; n < DV / 8; ++n) o[br][n][0] = o[br][n][1] = o[br][n][2] = o[br][n][3] = 0.f;
        }
        for (int i = 0; i < live; ++i) {
            ok = ok && mbar_wait_warp(&full[st], ph, ab);
            if (bad_stage[st]) bad = true;
            const int k0 = (cur.tile0 + i) * KT + warp * SLICE;
            const uint32_t stage = sbase + st * C::STAGE;
            if (ok && k0 < s.total) {
                // ---- S_b = Q_b K_b^T, 16 rows x 16 keys
                float sc[2][2][4];
#pragma unroll
                for (int br = 0; br < 2; ++br)
#pragma unroll
                    for (int n = 0; n < 2; ++n) sc[br][n][0] = sc[br][n][1] = sc[br][n][2] = sc[br][n][3] = 0.f;
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    uint32_t kf[4];
#pragma unroll
                    for (int br = 0; br < 2; ++br) {
                        if (br == 0 || !KS)
                            ldsm4(stage + (br * C::KP + (kk >> 2)) * PANEL + sw128(krow, 2 * (kk & 3) + kch), kf);
                        uint32_t qf[4];         // read again for each slice: registers hold O
                        ldsm4(sbase + C::OFF_Q + (br * C::KP + (kk >> 2)) * C::Q_PANEL + sw128(qrow, 2 * (kk & 3) + qch), qf);
                        mma16816(sc[br][0], qf, kf[0], kf[1]);
                        mma16816(sc[br][1], qf, kf[2], kf[3]);
                    }
                }
                // ---- P = 2^(S - m): element e of part n is row r0 + 8 (e >> 1), key 8 n + 2 (lane & 3) + (e & 1)
                const bool edge = k0 + SLICE > s.before;
                uint32_t seen[2] = {0xffffu, 0xffffu};
                if (edge) {
                    seen[0] = slice_mask(p, s, k0, la, ra.q, ta);
                    seen[1] = slice_mask(p, s, k0, lb, rb.q, tb);
                }
                float pr[2][2][4];
                bool big = false;
#pragma unroll
                for (int br = 0; br < 2; ++br)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const bool vis = seen[e >> 1] >> (8 * n + 2 * (lane & 3) + (e & 1)) & 1u;
                            const float x = vis ? sc[br][n][e] * sl2 : -INFINITY;
                            sc[br][n][e] = x;
                            pr[br][n][e] = vis ? ex2_approx(x - m[br][e >> 1]) : 0.f;
                            big |= !(pr[br][n][e] <= 256.f);
                        }
                if (__any_sync(0xffffffffu, big)) {
#pragma unroll
                    for (int br = 0; br < 2; ++br)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float x = fmaxf(fmaxf(sc[br][0][2 * h], sc[br][0][2 * h + 1]),
                                            fmaxf(sc[br][1][2 * h], sc[br][1][2 * h + 1]));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                            const float mn = fmaxf(m[br][h], x);
                            const float a = m[br][h] == mn ? 1.f : ex2_approx(m[br][h] - mn);
                            m[br][h] = mn;
                            l[br][h] *= a;
#pragma unroll
                            for (int n = 0; n < 2; ++n)
#pragma unroll
                                for (int e = 2 * h; e < 2 * h + 2; ++e)
                                    pr[br][n][e] = sc[br][n][e] == -INFINITY ? 0.f : ex2_approx(sc[br][n][e] - mn);
#pragma unroll
                            for (int n = 0; n < DV / 8; ++n) {
                                o[br][n][2 * h] *= a;
                                o[br][n][2 * h + 1] *= a;
                            }
                        }
                }
                uint32_t pa[2][4];
#pragma unroll
                for (int br = 0; br < 2; ++br) {
                    l[br][0] += (pr[br][0][0] + pr[br][0][1]) + (pr[br][1][0] + pr[br][1][1]);
                    l[br][1] += (pr[br][0][2] + pr[br][0][3]) + (pr[br][1][2] + pr[br][1][3]);
                    pa[br][0] = pack_bf16x2(pr[br][0][0], pr[br][0][1]);
                    pa[br][1] = pack_bf16x2(pr[br][0][2], pr[br][0][3]);
                    pa[br][2] = pack_bf16x2(pr[br][1][0], pr[br][1][1]);
                    pa[br][3] = pack_bf16x2(pr[br][1][2], pr[br][1][3]);
                }
                if (edge) {
                    // Values that a row does not see may be anything, and the product's 0 x NaN
                    // is NaN.  Rows past the end become zeros; elsewhere a value that is not
                    // finite is taken out of the tile and added here to the rows that see it.
                    uint8_t* vt = smem + st * C::STAGE + C::OFF_V + warp * SLICE * 128;
                    for (int j = 0; j < 8; ++j) {
                        const int key = 2 * j + (lane >> 4), c = lane & 15;
                        uint8_t* at = vt + (c >> 3) * PANEL + sw128(key, c & 7);
                        uint4 w = *reinterpret_cast<uint4*>(at);
                        const bool past = k0 + key >= s.total;
                        const bool fix = past || !(bf16x2_finite(w.x) && bf16x2_finite(w.y) && bf16x2_finite(w.z) &&
                                                   bf16x2_finite(w.w));
                        unsigned todo = __ballot_sync(0xffffffffu, fix && !past);
                        while (todo) {
                            const int from = __ffs(todo) - 1;
                            todo &= todo - 1;
                            const uint32_t v4[4] = {__shfl_sync(0xffffffffu, w.x, from), __shfl_sync(0xffffffffu, w.y, from),
                                                    __shfl_sync(0xffffffffu, w.z, from), __shfl_sync(0xffffffffu, w.w, from)};
                            const int fk = 2 * j + (from >> 4);             // key, and first column
                            const int fc = (from & 15) * 8;
                            const int src = (lane & ~3) | ((fk & 7) >> 1);
                            float pk[2][2];
#pragma unroll
                            for (int br = 0; br < 2; ++br)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const float x0 = (fk & 1) ? pr[br][0][2 * h + 1] : pr[br][0][2 * h];
                                    const float x1 = (fk & 1) ? pr[br][1][2 * h + 1] : pr[br][1][2 * h];
                                    pk[br][h] = __shfl_sync(0xffffffffu, fk >= 8 ? x1 : x0, src);
                                }
                            // this thread's columns of the eight: 2 (lane & 3) and the next
                            const uint32_t pair = (lane & 3) == 0 ? v4[0] : (lane & 3) == 1 ? v4[1] : (lane & 3) == 2 ? v4[2] : v4[3];
                            const float vv[2] = {__uint_as_float(pair << 16), __uint_as_float(pair & 0xffff0000u)};
#pragma unroll
                            for (int n = 0; n < DV / 8; ++n)
                                if (n == fc / 8)
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        if (!isfinite(vv[e & 1]) && (seen[e >> 1] >> fk & 1u)) {
                                            o[0][n][e] = fmaf(pk[0][e >> 1], vv[e & 1], o[0][n][e]);
                                            o[1][n][e] = fmaf(pk[1][e >> 1], vv[e & 1], o[1][n][e]);
                                        }
                        }
                        if (fix) {
                            auto clean = [&](uint32_t x) -> uint32_t {
                                if (past) return 0;
                                if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
                                if ((x & 0x7f800000u) == 0x7f800000u) x &= 0x0000ffffu;
                                return x;
                            };
                            *reinterpret_cast<uint4*>(at) = make_uint4(clean(w.x), clean(w.y), clean(w.z), clean(w.w));
                        }
                    }
                    fence_proxy_async_smem();           // before TMA writes the stage again
                    __syncwarp();
                }
                // ---- O_b += P_b V, both branches from one read of V
#pragma unroll
                for (int n = 0; n < DV / 16; ++n) {
                    uint32_t vf[4];
                    ldsm4_t(stage + C::OFF_V + (n >> 2) * PANEL + sw128(vrow, 2 * (n & 3) + vch), vf);
#pragma unroll
                    for (int br = 0; br < 2; ++br) {
                        mma16816(o[br][2 * n], pa[br], vf[0], vf[1]);
                        mma16816(o[br][2 * n + 1], pa[br], vf[2], vf[3]);
                    }
                }
            }
            if (i + 1 < live) {                 // the segment's last stage is freed after the merge
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st]);
                if (++st == C::NST) { st = 0; ph ^= 1; }
            }
        }
        // ---- merge the warps: their maxima and sums, then O in rounds of ROUND rows through
        // the stage that was read last
#pragma unroll
        for (int br = 0; br < 2; ++br)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x = l[br][h];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if (bad) x = __int_as_float(0x7fc00000);
                if ((lane & 3) == 0) {
                    stat[(warp * 2 + 0) * 2 * NR + br * NR + r0 + 8 * h] = m[br][h];
                    stat[(warp * 2 + 1) * 2 * NR + br * NR + r0 + 8 * h] = x;
                }
            }
        named_bar_sync(1, 32 * CONSUMERS);      // every warp is done with the stage, too
        // Unscaled: this runs once a segment, cold, so it costs by its instructions.
        float* buf = reinterpret_cast<float*>(smem + st * C::STAGE);     // [warp][row of the round][branch][DV]
        for (int row0 = 0; row0 < p.chunk_rows; row0 += C::ROUND) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = r0 + 8 * h - row0;
                if (live == 0 || r < 0 || r >= C::ROUND || !(h ? lb : la)) continue;
                float* dst = buf + (warp * C::ROUND + r) * 2 * DV + 2 * (lane & 3);
#pragma unroll
                for (int br = 0; br < 2; ++br)
#pragma unroll
                    for (int n = 0; n < DV / 8; ++n)
                        *reinterpret_cast<float2*>(dst + br * DV + 8 * n) = make_float2(o[br][n][2 * h], o[br][n][2 * h + 1]);
            }
            named_bar_sync(1, 32 * CONSUMERS);
            for (int r = warp; r < C::ROUND && row0 + r < p.chunk_rows; r += CONSUMERS) {
                const PagedRow x = paged_row(p, cur.hk, cur.rc, row0 + r, s.n_new);
                if (!x.live) continue;
                float mt[2], lt[2], wt[2][CONSUMERS], a[2][DV / 32];
#pragma unroll
                for (int br = 0; br < 2; ++br) {
                    const float* ms = stat + br * NR + row0 + r;
                    mt[br] = fmaxf(fmaxf(ms[0], ms[4 * NR]), fmaxf(ms[8 * NR], ms[12 * NR]));
                    lt[br] = 0.f;
#pragma unroll
                    for (int w = 0; w < CONSUMERS; ++w) {
                        const float mw = ms[w * 4 * NR], lw = ms[(w * 4 + 2) * NR];
                        wt[br][w] = mw == -INFINITY ? 0.f : ex2_approx(mw - mt[br]);
                        lt[br] += mw == -INFINITY ? lw : lw * wt[br][w];       // 0 or NaN where nothing was seen
                    }
#pragma unroll
                    for (int j = 0; j < DV / 32; ++j) a[br][j] = 0.f;
                }
                if (live > 0) {
#pragma unroll
                    for (int w = 0; w < CONSUMERS; ++w)
#pragma unroll
                        for (int br = 0; br < 2; ++br)
#pragma unroll
                            for (int j = 0; j < DV / 32; ++j)
                                a[br][j] = fmaf(wt[br][w], buf[((w * C::ROUND + r) * 2 + br) * DV + lane + 32 * j], a[br][j]);
                }
                if (cur.whole()) {
                    paged_finish_row<DV / 32>(p, lam, cur.b, x.h, x.q, lane, a[0], lt[0], a[1], lt[1]);
                } else {
                    float* part = p.part + ((int64_t)cur.slot() * p.chunk_rows + row0 + r) * (4 + 2 * DV);
                    if (lane == 0) *reinterpret_cast<float4*>(part) = make_float4(mt[0], lt[0], mt[1], lt[1]);
#pragma unroll
                    for (int br = 0; br < 2; ++br)
#pragma unroll
                        for (int j = 0; j < DV / 32; ++j) part[4 + br * DV + lane + 32 * j] = a[br][j];
                }
            }
            fence_proxy_async_smem();
            named_bar_sync(1, 32 * CONSUMERS);
        }
        if (live > 0) {
            if (lane == 0) mbar_arrive(&empty[st]);
            if (++st == C::NST) { st = 0; ph ^= 1; }
        }
    }
}

template <int HD, bool KS>
int launch_hd(const CUtensorMap* maps, const PagedParams& p, int box_rows, cudaStream_t stream) {
    constexpr int smem = Cfg<HD, KS>::SMEM;
    if (cudaFuncSetAttribute(paged_mma_kernel<HD, KS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return -1;
    paged_mma_kernel<HD, KS><<<p.grid, THREADS, smem, stream>>>(maps[0], maps[1], maps[2], p, box_rows);
    return cudaGetLastError() == cudaSuccess ? launch_paged_combine(p, stream) : -1;
}

}  // namespace pmma

int launch_paged_mma(const CUtensorMap* maps, const PagedParams& p, int box_rows, cudaStream_t stream) {
    if (p.D == 64) return p.k_shared ? pmma::launch_hd<64, true>(maps, p, box_rows, stream)
                                     : pmma::launch_hd<64, false>(maps, p, box_rows, stream);
    return p.k_shared ? pmma::launch_hd<128, true>(maps, p, box_rows, stream)
                      : pmma::launch_hd<128, false>(maps, p, box_rows, stream);
}

}  // namespace diffattn
