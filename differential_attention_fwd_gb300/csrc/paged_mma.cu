// paged_mma.cu -- differential attention over a paged cache for up to 16 query rows a
// key/value head (single tokens, a few, small trees): bf16, value width 128, Q/K width
// 64 or 128, pages of a multiple of 16 slots.
//
// Bound by HBM: a key costs 4 D + 256 bytes (2 D + 256 with shared keys) and 4 (D + 128)
// operations a row, 192 FLOP a byte short of what the tensor cores could do even at 16
// rows.  So the design is about never leaving the memory idle:
//   - A warp takes 16 keys at a time and keeps its rows' running maximum, sum and O (16
//     rows x 128 columns of both branches, 128 registers a thread) for itself, so a tile
//     needs no barrier.
//   - A second warp streams its slices of 16 keys through TMA into a ring of its own,
//     across unit boundaries.  A slice lies in one page.  Two blocks of four such pairs
//     an SM keep 130 to 190 KB in flight, more than the HBM rate times its latency.
//   - SMs stream at different rates (the slowest 20 % behind the fastest), which is what
//     is left of a long call: blocks end between 99 and 119 us of 120.  Twice the blocks in
//     waves cost more by their starts (133 us).
//   - With many units (a batch of short sequences) a worker is one warp, which writes its
//     rows from its registers at a unit's end.  With few, four warps share a worker's
//     tiles of 64 keys and merge their results in shared memory at its end, so that the
//     merging pass has a quarter of the parts.  (2048 units of 100 keys: 78 us with four
//     warps a worker, whose merge takes 2 us a unit, 51 with one, 36 with what followed.
//     16 units of 16384: 33 us with four, 42 with one, the difference in the merging pass.)
//   - The products are warp-level (m16n8k16): P goes from the score's accumulators to the
//     next product's operand in registers, and no warp waits for another.  A tcgen05
//     product would want 128 keys as its M and P through shared memory with two block-wide
//     barriers a tile (the layout of the dense decode, 0.83 of the copy rate).
//
// Weights are 2^(s - m) against a running maximum that moves only when some weight would
// pass 2^8.  They go to the product with V as two bf16 parts, the rounded weight and what
// the rounding left (2^-16 together): with one part the branches' difference was off by
// 2.1e-3 of itself, more than the output's own rounding (1.7e-3).  The second product passes
// while the tile's bytes arrive; where it does not quite, at 4 rows of head width 128, it costs 5 %.
//
// Measured, both launches: 16 sequences of up to 8192 keys, 16 heads, D = 64, 710 MB of
// cache: 122 us, 0.86 of the copy rate; 4 of 65536, 8 key/value heads, shared keys, D = 128:
// 118 us, 0.89; one of 517: 12.7 us, the latency of the two launches, the lengths, a page
// and its keys in turn.  A warp is busy with a slice of 16 keys for 2,500 cycles of the
// 3,000 that HBM allows it, which is what is left of mid-length calls (64 x 1000, 16 heads:
// 78 us of 49): the next step is the products' other order, keys as their 16 rows.
#include "paged_plan.cuh"
#include "kernels.h"
#include "pdl.cuh"

namespace diffattn {
namespace pmma {

constexpr int WARPS = kMmaWarps;                // pairs of warps of a block; two blocks an SM
// The producers' warpgroup gives registers to the consumers': 128 x 216 + 128 x 40 =
// 256 x 128, what the block is launched with.
constexpr int THREADS = 2 * 32 * WARPS;
constexpr uint32_t REGS_CONSUMER = 216, REGS_PRODUCER = 40;
static_assert(128 * REGS_CONSUMER + 128 * REGS_PRODUCER <= THREADS * 128, "register split");
constexpr int KT = kMmaTile;                    // keys of a tile: four slices
constexpr int SLICE = 16;
constexpr int NR = 16;                          // rows of a unit
constexpr int DV = 128;
constexpr int PANEL = SLICE * 128;              // 2 KB: 16 keys x 64 columns
constexpr int SNAP = 1;                         // tiles at a unit's end that are not worth another part
constexpr int EXTRA = 1;                        // what a unit's start costs, in tiles

// Shared memory: a ring for each pair, the queries (one warp a worker: WARP_ROWS a warp;
// else 16 rows of the block, and the maxima and sums of its warps), barriers.
template <int HD, bool KS>
struct Cfg {
    static constexpr int KP = HD / 64;                          // panels of a key tile
    static constexpr int NK = KS ? 1 : 2;
    static constexpr int STAGE = (NK * KP + 2) * PANEL;         // 6, 8 or 12 KB
    static constexpr int NST = 24 * 1024 / STAGE;               // 4, 3 or 2
    static constexpr int RING = NST * STAGE;
    static constexpr int OFF_V = NK * KP * PANEL;
    static constexpr int WARP_ROWS = paged_solo_rows(HD);
    static_assert(WARP_ROWS <= 8, "a warp alone has one row a thread: HR = 1");
    static constexpr int Q_PANEL = NR * 128;                    // [branch][panel] 16 rows x 128 bytes of the block,
    static constexpr int Q_WARP = 2 * KP * WARP_ROWS * 128;     // or WARP_ROWS x 128 bytes of a warp
    static constexpr int OFF_Q = WARPS * RING;
    static constexpr int OFF_STAT = OFF_Q + WARPS * Q_WARP;     // float [warp][m, l][branch][row]
    static constexpr int OFF_BAR = OFF_STAT + WARPS * 4 * NR * 4;   // [warp] full [NST], empty [NST]
    static constexpr int OFF_MISC = OFF_BAR + WARPS * 2 * NST * 8;  // abort, bad flags [warp][NST]
    static constexpr int SMEM = OFF_MISC + 4 + WARPS * NST * 4 + 1024;
    static constexpr int ROUND = STAGE / (2 * DV * 4);          // rows merged at once
    static_assert(2 * KP * Q_PANEL <= WARPS * Q_WARP, "the block's queries");
    static_assert(2 * (SMEM + 512 + 1024) <= 228 * 1024, "shared memory");
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

// HR: 1 for units of up to 8 rows, whose threads have no second row, else 2.
template <int HD, bool KS, int HR>
__global__ void __launch_bounds__(THREADS, 2)
paged_mma_kernel(const __grid_constant__ CUtensorMap tm_k1, const __grid_constant__ CUtensorMap tm_k2,
                 const __grid_constant__ CUtensorMap tm_v, const PagedParams p) {
    using C = Cfg<HD, KS>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int scan[2 * THREADS / 32];
    __shared__ PagedBlock<WARPS> blk;
    uint8_t* smem_block = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem_block + C::OFF_MISC);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int w = warp % WARPS;                 // the pair
    uint8_t* ring = smem_block + w * C::RING;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem_block + C::OFF_BAR) + w * 2 * C::NST;
    uint64_t* empty = full + C::NST;
    volatile uint32_t* bad_stage = abort_flag + 1 + w * C::NST;
    const AbortState ab{abort_flag, p.status};
    if (warp < WARPS && lane < C::NST) {
        mbar_init(&full[lane], 1);
        mbar_init(&empty[lane], 1);
        bad_stage[lane] = 0;
        if (tid == 0) *abort_flag = 0;
        fence_mbar_init();
    }
    pdl_wait();                                 // before the merging pass may start, which writes too
    pdl_launch_dependents();
    // One warp a worker where that makes at most two workers a unit, and if the unit's rows
    // allow it.  (The barriers in here order the above.)
    const PagedScan found = paged_scan<THREADS>(p, KT, EXTRA, scan);
    const bool solo = HR == 1 && p.chunk_rows <= C::WARP_ROWS && 2ll * found.units >= p.solo_workers;
    const int nw = solo ? WARPS : 1;                            // workers of the block
    paged_locate<WARPS>(p, found, KT, EXTRA, nw, gridDim.x * nw, SNAP, &blk);
    const int mine = solo ? w : 0;
    const int worker = blockIdx.x * nw + mine;
    // the warp's slices in a tile: all four, or one
    const int slices = solo ? KT / SLICE : 1, slice0 = solo ? 0 : w;
    PagedCursor cur;

    if (warp >= WARPS) {
        // ---------------------------------------------------------------- producer
        regs_dec<REGS_PRODUCER>();
        cur.begin(p, blk, mine, worker, KT, EXTRA);
        const bool scribe = lane == 0 && (solo || w == 0);
        if (lane == 0) {
            tma_prefetch_desc(&tm_k1);
            tma_prefetch_desc(&tm_k2);
            tma_prefetch_desc(&tm_v);
        }
        if (scribe) {
            PagedCursor::no_join(p, worker);
            // the words of workers that there are not
            if (!solo)
                for (int c = gridDim.x + worker; c < p.workers; c += gridDim.x) PagedCursor::no_join(p, c);
        }
        uint32_t armed = 0;                     // slices issued
        int st = 0;
        uint32_t ph = 1;                        // the first pass over the ring finds it free
        bool ok = true;
        for (; ok && !cur.done(); cur.next(p, KT, EXTRA)) {
            const int live = cur.live_tiles(p, KT) * slices;
            if (scribe) cur.join(p, blk.shares, blk.start[mine + 1].tile, EXTRA);
            int page = 0;                       // of slice i0 + lane, looked up 32 at a time
            for (int i = 0; i < live; ++i) {
                // slice i of the warp: the key it starts with
                auto key_of = [&](int k) { return solo ? cur.tile0 * KT + k * SLICE : (cur.tile0 + k) * KT + slice0 * SLICE; };
                if ((i & 31) == 0) {
                    const int key = key_of(i + lane);
                    page = -2;                  // nothing to load
                    if (i + lane < live && key < cur.s.total) page = paged_page(p, cur.b, key / p.page);
                }
                const int now = __shfl_sync(0xffffffffu, page, i & 31);
                if (!(ok = mbar_wait_warp(&empty[st], ph, ab))) break;
                if (lane == 0) {
                    bad_stage[st] = now == -1;
                    if (now < 0) {
                        if (now == -1) atomicOr(p.status, kStatusIndex);
                        mbar_arrive(&full[st]);
                    } else {
                        mbar_arrive_expect_tx(&full[st], C::STAGE);
                        const int slot = key_of(i) % p.page;
                        uint8_t* dst = ring + st * C::STAGE;
#pragma unroll
                        for (int pn = 0; pn < C::KP; ++pn) {
                            tma_load_4d(dst + pn * PANEL, &tm_k1, &full[st], pn * 64, slot, cur.hk, now);
                            if (!KS) tma_load_4d(dst + (C::KP + pn) * PANEL, &tm_k2, &full[st], pn * 64, slot, cur.hk, now);
                        }
                        tma_load_4d(dst + C::OFF_V, &tm_v, &full[st], 0, slot, cur.hk, now);
                        tma_load_4d(dst + C::OFF_V + PANEL, &tm_v, &full[st], 64, slot, cur.hk, now);
                    }
                }
                __syncwarp();
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
    cur.begin(p, blk, mine, worker, KT, EXTRA);
    const float sl2 = p.scale_log2;
    const int r0 = lane >> 2;                   // this thread's rows r0 and r0 + 8
    // the worker's queries: [branch][panel] rows of 128 bytes
    const int q_panel = solo ? C::WARP_ROWS * 128 : C::Q_PANEL;
    uint8_t* qs = smem_block + C::OFF_Q + (solo ? w * C::Q_WARP : 0);
    float* stat = reinterpret_cast<float*>(smem_block + C::OFF_STAT);
    // lane addresses of the ldmatrix operands; alone, the other rows read the first ones again
    const int krow = (lane & 7) + ((lane >> 4) << 3), kch = (lane >> 3) & 1;
    const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vch = lane >> 4;
    const int qrow = solo ? lane & (C::WARP_ROWS - 1) : (lane & 7) + (((lane >> 3) & 1) << 3), qch = lane >> 4;
    const uint32_t sring = smem_u32(ring), sq = smem_u32(qs);
    int st = 0;
    uint32_t ph = 0;
    bool ok = true;                             // after a failed wait: no more work, but every barrier
    for (; !cur.done(); cur.next(p, KT, EXTRA)) {
        const int live = cur.live_tiles(p, KT) * slices;
        const PagedSeq s = cur.s;
        bool bad = s.bad;
        if (bad && lane == 0) atomicOr(p.status, kStatusIndex);
        // ---- the unit's queries, zeros for padding rows
        {
            constexpr int QCH = HD / 8;         // 16-byte chunks of a row
            const int threads = solo ? 32 : WARPS * 32, t0 = solo ? lane : tid;
            const int c = t0 % (2 * QCH) % QCH, br = t0 % (2 * QCH) / QCH;
            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(br ? p.q2 : p.q1) + c * 8;
            const int64_t sb = br ? p.s_q2[0] : p.s_q1[0], sh = br ? p.s_q2[1] : p.s_q1[1], sq_ = br ? p.s_q2[2] : p.s_q1[2];
            src += cur.b * sb;
            const int rows = solo ? C::WARP_ROWS : NR, step = threads / (2 * QCH);
#pragma unroll 4
            for (int r = t0 / (2 * QCH); r < rows; r += step) {
                const PagedRow x = paged_row(p, cur.hk, cur.rc, r, s.n_new);
                uint4 v = make_uint4(0, 0, 0, 0);
                if (x.live && r < p.chunk_rows) {
                    const __nv_bfloat16* at = src + x.h * sh + x.q * sq_;
                    if (p.q16) {
                        v = *reinterpret_cast<const uint4*>(at);
                    } else {
                        const uint16_t* e = reinterpret_cast<const uint16_t*>(at);
                        v = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16,
                                       e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
                    }
                }
                *reinterpret_cast<uint4*>(qs + (br * C::KP + (c >> 3)) * q_panel + sw128(r, c & 7)) = v;
            }
        }
        if (solo) __syncwarp();
        else named_bar_sync(1, WARPS * 32);
        const PagedRow ra = paged_row(p, cur.hk, cur.rc, r0, s.n_new);
        const PagedRow rb = paged_row(p, cur.hk, cur.rc, r0 + 8, s.n_new);
        const bool la = ra.live && r0 < p.chunk_rows, lb = rb.live && r0 + 8 < p.chunk_rows;
        uint64_t ta = 0, tb = 0;
        if (p.mask && (int64_t)(cur.tile0 + cur.n) * KT > s.before) {
            // lane r reads row r's, then each thread takes its two rows'
            const PagedRow x = paged_row(p, cur.hk, cur.rc, lane & 15, s.n_new);
            const uint64_t bits = paged_mask_bits<NR>(p, cur.b, x.q, x.live && (lane & 15) < p.chunk_rows, s.n_new, lane);
            ta = __shfl_sync(0xffffffffu, bits, r0);
            tb = __shfl_sync(0xffffffffu, bits, r0 + 8);
        }
        float o[2][DV / 8][4];
        float m[2][HR], l[2][HR];
#pragma unroll
        for (int br = 0; br < 2; ++br) {
#pragma unroll
            for (int h = 0; h < HR; ++h) {
                m[br][h] = -INFINITY;
                l[br][h] = 0.f;
            }
#pragma unroll
            for (int n = 0; n < DV / 8; ++n) o[br][n][0] = o[br][n][1] = o[br][n][2] = o[br][n][3] = 0.f;
        }
        for (int i = 0; i < live; ++i) {
            ok = ok && mbar_wait_warp(&full[st], ph, ab);
            const int k0 = solo ? cur.tile0 * KT + i * SLICE : (cur.tile0 + i) * KT + slice0 * SLICE;
            const uint32_t stage = sring + st * C::STAGE;
            if (bad_stage[st]) {
                bad = true;                     // nothing was loaded
            } else if (ok && k0 < s.total) {
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
                        ldsm4(sq + (br * C::KP + (kk >> 2)) * q_panel + sw128(qrow, 2 * (kk & 3) + qch), qf);
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
                float pr[2][2][2 * HR];
                bool big = false;
#pragma unroll
                for (int br = 0; br < 2; ++br)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 2 * HR; ++e) {
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
                        for (int h = 0; h < HR; ++h) {
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
                                if (HR == 1) {          // second parts
                                    o[br][n][2] *= a;
                                    o[br][n][3] *= a;
                                }
                            }
                        }
                }
                // The weights' two parts.  A warp alone has up to 8 rows, and its second parts go
                // into the product's other 8: half of the products (2048 units of 100 keys: 37.5
                // to 36 us; 1024 of 1000: 80.6 to 78.3).  Four warps together have the time, and
                // are better off with a steady pace: SMs that wait for nothing but HBM take it
                // from one another (V2 head, 4 x 65536: 118 us, 124 with half of the products).
                uint32_t pa[2][4], pb[2][4];
#pragma unroll
                for (int br = 0; br < 2; ++br) {
#pragma unroll
                    for (int h = 0; h < HR; ++h) {
                        l[br][h] += (pr[br][0][2 * h] + pr[br][0][2 * h + 1]) + (pr[br][1][2 * h] + pr[br][1][2 * h + 1]);
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const float a = pr[br][n][2 * h], b = pr[br][n][2 * h + 1];
                            const uint32_t hi = pack_bf16x2(a, b);
                            const uint32_t lo = pack_bf16x2(a - __uint_as_float(hi << 16),      // what the rounding left
                                                            b - __uint_as_float(hi & 0xffff0000u));
                            pa[br][2 * n + h] = hi;
                            pb[br][2 * n + h] = lo;
                            if (HR == 1) {
                                pa[br][2 * n + 1] = solo ? lo : 0;
                                pb[br][2 * n + 1] = 0;
                            }
                        }
                    }
                }
                if (edge) {
                    // Values that a row does not see may be anything, and the product's 0 x NaN
                    // is NaN.  Rows past the end become zeros; elsewhere a value that is not
                    // finite is taken out of the tile and added here to the rows that see it.
                    uint8_t* vt = ring + st * C::STAGE + C::OFF_V;
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
                            float pk[2][HR];
#pragma unroll
                            for (int br = 0; br < 2; ++br)
#pragma unroll
                                for (int h = 0; h < HR; ++h) {
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
                                    for (int e = 0; e < 2 * HR; ++e)
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
                        if (HR == 2 || !solo) {
                            mma16816(o[br][2 * n], pb[br], vf[0], vf[1]);
                            mma16816(o[br][2 * n + 1], pb[br], vf[2], vf[3]);
                        }
                    }
                }
            }
            if (solo || i + 1 < live) {         // a shared unit's last stage is freed after its merge
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st]);
                if (++st == C::NST) { st = 0; ph ^= 1; }
            }
        }
        if (HR == 1 && solo) {
#pragma unroll
            for (int br = 0; br < 2; ++br)
#pragma unroll
                for (int n = 0; n < DV / 8; ++n) {
                    o[br][n][0] += o[br][n][2];
                    o[br][n][1] += o[br][n][3];
                }
        }
#pragma unroll
        for (int br = 0; br < 2; ++br)
#pragma unroll
            for (int h = 0; h < HR; ++h) {
                l[br][h] += __shfl_xor_sync(0xffffffffu, l[br][h], 1);
                l[br][h] += __shfl_xor_sync(0xffffffffu, l[br][h], 2);
                if (bad || !ok) l[br][h] = __int_as_float(0x7fc00000);
            }
        if (!solo) {
            // ---- merge the block's warps: their maxima and sums, then O in rounds of ROUND
            // rows through the stages that were read last.  Cold code, once a segment: it
            // costs by its instructions, so O goes out unscaled.
#pragma unroll
            for (int br = 0; br < 2; ++br)
#pragma unroll
                for (int h = 0; h < HR; ++h)
                    if ((lane & 3) == 0) {
                        stat[(w * 2 + 0) * 2 * NR + br * NR + r0 + 8 * h] = m[br][h];
                        stat[(w * 2 + 1) * 2 * NR + br * NR + r0 + 8 * h] = l[br][h];
                    }
            // [row of the round][branch][DV], each warp's in its own ring
            float* buf = reinterpret_cast<float*>(ring + st * C::STAGE);
            // where the others have theirs: all have walked as many stages
            const float* bufs = reinterpret_cast<const float*>(smem_block + st * C::STAGE);
            for (int row0 = 0; row0 < p.chunk_rows; row0 += C::ROUND) {
#pragma unroll
                for (int h = 0; h < HR; ++h) {
                    const int r = r0 + 8 * h - row0;
                    if (live == 0 || r < 0 || r >= C::ROUND || !(h ? lb : la)) continue;
                    float* dst = buf + r * 2 * DV + 2 * (lane & 3);
#pragma unroll
                    for (int br = 0; br < 2; ++br)
#pragma unroll
                        for (int n = 0; n < DV / 8; ++n)
                            *reinterpret_cast<float2*>(dst + br * DV + 8 * n) = make_float2(o[br][n][2 * h], o[br][n][2 * h + 1]);
                }
                named_bar_sync(1, WARPS * 32);
                for (int r = w; r < C::ROUND && row0 + r < p.chunk_rows; r += WARPS) {
                    const PagedRow x = paged_row(p, cur.hk, cur.rc, row0 + r, s.n_new);
                    if (!x.live) continue;
                    float mt[2], lt[2], wt[2][WARPS], a[2][DV / 32];
#pragma unroll
                    for (int br = 0; br < 2; ++br) {
                        const float* ms = stat + br * NR + row0 + r;
                        mt[br] = fmaxf(fmaxf(ms[0], ms[4 * NR]), fmaxf(ms[8 * NR], ms[12 * NR]));
                        lt[br] = 0.f;
#pragma unroll
                        for (int k = 0; k < WARPS; ++k) {
                            const float mw = ms[k * 4 * NR], lw = ms[(k * 4 + 2) * NR];
                            wt[br][k] = mw == -INFINITY ? 0.f : ex2_approx(mw - mt[br]);
                            lt[br] += mw == -INFINITY ? lw : lw * wt[br][k];       // 0 or NaN where nothing was seen
                        }
#pragma unroll
                        for (int j = 0; j < DV / 32; ++j) a[br][j] = 0.f;
                    }
                    if (live > 0) {
#pragma unroll
                        for (int k = 0; k < WARPS; ++k)
#pragma unroll
                            for (int br = 0; br < 2; ++br)
#pragma unroll
                                for (int j = 0; j < DV / 32; ++j)
                                    a[br][j] = fmaf(wt[br][k], bufs[k * (C::RING / 4) + (r * 2 + br) * DV + lane + 32 * j], a[br][j]);
                    }
                    if (cur.whole()) {
                        const float lam = p.lambda_dev ? __ldg(p.lambda_dev) : p.lambda;
                        paged_finish_row<DV / 32>(p, lam, cur.b, x.h, x.q, lane, a[0], lt[0], a[1], lt[1]);
                    } else {
                        float* part = p.part + ((int64_t)cur.slot() * p.chunk_rows + row0 + r) * paged_part_floats(DV);
                        if (lane == 0) *reinterpret_cast<float4*>(part) = make_float4(mt[0], lt[0], mt[1], lt[1]);
#pragma unroll
                        for (int br = 0; br < 2; ++br)
#pragma unroll
                            for (int j = 0; j < DV / 32; ++j) part[4 + br * DV + lane + 32 * j] = a[br][j];
                    }
                }
                fence_proxy_async_smem();       // before TMA writes the stages again
                named_bar_sync(1, WARPS * 32);
            }
            if (live > 0) {
                if (lane == 0) mbar_arrive(&empty[st]);
                if (++st == C::NST) { st = 0; ph ^= 1; }
            }
            continue;
        }
        // ---- alone: the rows out of the registers, finished, or as a partial result
        if (!cur.whole()) {
            float* part = p.part + ((int64_t)cur.slot() * p.chunk_rows + r0) * paged_part_floats(DV);
            if (la) {
                if ((lane & 3) == 0) *reinterpret_cast<float4*>(part) = make_float4(m[0][0], l[0][0], m[1][0], l[1][0]);
#pragma unroll
                for (int br = 0; br < 2; ++br)
#pragma unroll
                    for (int n = 0; n < DV / 8; ++n)
                        *reinterpret_cast<float2*>(part + 4 + br * DV + 8 * n + 2 * (lane & 3)) =
                            make_float2(o[br][n][0], o[br][n][1]);
            }
            __syncwarp();                   // before the next unit's queries overwrite these
            continue;
        }
        const PagedRow x = ra;
        const float lam = p.lambda_dev ? __ldg(p.lambda_dev) : p.lambda;
        const float i1 = l[0][0] == 0.f ? 0.f : 1.f / l[0][0], i2 = l[1][0] == 0.f ? 0.f : 1.f / l[1][0];
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < DV / 8; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                o[0][n][e] = fmaf(-lam, __fmul_rn(o[1][n][e], i2), __fmul_rn(o[0][n][e], i1));
                sum += o[0][n][e];
            }
        if (p.norm != kNormNone) {          // of the row's four threads
            float mean = 0.f, ss = 0.f;
            if (p.norm == kNormGroup) {
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                mean = sum / DV;
            }
#pragma unroll
            for (int n = 0; n < DV / 8; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    o[0][n][e] -= mean;
                    ss = fmaf(o[0][n][e], o[0][n][e], ss);
                }
            ss += __shfl_xor_sync(0xffffffffu, ss, 1);
            ss += __shfl_xor_sync(0xffffffffu, ss, 2);
            const float r = 1.0f / sqrtf(ss / DV + p.norm_eps);
#pragma unroll
            for (int n = 0; n < DV / 8; ++n) {
                o[0][n][0] *= r;
                o[0][n][1] *= r;
            }
        }
        const int64_t at = cur.b * p.s_o[0] + x.h * p.s_o[1] + x.q * p.s_o[2] + 2 * (lane & 3);
        const int64_t ch = (int64_t)x.h * DV + 2 * (lane & 3);
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + at;
        if (la) {
#pragma unroll
            for (int n = 0; n < DV / 8; ++n) {
                float y0 = o[0][n][0], y1 = o[0][n][1];
                if (p.norm_weight) { y0 *= p.norm_weight[ch + 8 * n]; y1 *= p.norm_weight[ch + 8 * n + 1]; }
                if (p.norm_bias) { y0 += p.norm_bias[ch + 8 * n]; y1 += p.norm_bias[ch + 8 * n + 1]; }
                y0 *= p.out_scale;
                y1 *= p.out_scale;
                if (p.o4) {
                    *reinterpret_cast<uint32_t*>(out + 8 * n) = pack_bf16x2(y0, y1);
                } else {
                    out[8 * n] = __float2bfloat16_rn(y0);
                    out[8 * n + 1] = __float2bfloat16_rn(y1);
                }
            }
        }
        __syncwarp();                           // before the next unit's queries overwrite these
    }
}

template <int HD, bool KS, int HR>
int launch_rows(const CUtensorMap* maps, const PagedParams& p, cudaStream_t stream) {
    constexpr int smem = Cfg<HD, KS>::SMEM;
    // workers are warps where one warp may be one
    const int blocks = p.workers / (p.chunk_rows <= Cfg<HD, KS>::WARP_ROWS ? WARPS : 1);
    if (cudaFuncSetAttribute(paged_mma_kernel<HD, KS, HR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return -1;
    const int rc = pdl_launch(paged_mma_kernel<HD, KS, HR>, dim3(blocks), THREADS, smem, stream, maps[0], maps[1], maps[2], p);
    return rc == 0 ? launch_paged_combine(p, stream) : rc;
}

template <int HD, bool KS>
int launch_hd(const CUtensorMap* maps, const PagedParams& p, cudaStream_t stream) {
    return p.chunk_rows <= 8 ? launch_rows<HD, KS, 1>(maps, p, stream) : launch_rows<HD, KS, 2>(maps, p, stream);
}

}  // namespace pmma

int launch_paged_mma(const CUtensorMap* maps, const PagedParams& p, cudaStream_t stream) {
    if (p.D == 64) return p.k_shared ? pmma::launch_hd<64, true>(maps, p, stream)
                                     : pmma::launch_hd<64, false>(maps, p, stream);
    return p.k_shared ? pmma::launch_hd<128, true>(maps, p, stream)
                      : pmma::launch_hd<128, false>(maps, p, stream);
}

}  // namespace diffattn
