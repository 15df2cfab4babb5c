// paged_tc.cu -- differential attention over a paged cache for more than 16 query rows a
// key/value head (trees of drafted tokens, chunks of a prefill): bf16, value width 128,
// Q/K width 64 or 128, pages of a multiple of 16 slots, on tcgen05.
//
// A unit is up to 128 query rows of the heads that share a key/value head: each head's
// new tokens, padded to a multiple of 8 rows, one head after another in the MMA's M, so
// that a tree of 61 tokens of two heads fills one tile and its cache is read once.  Per
// 64 keys: S_b = Q_b K_b^T (M = 128, N = 64) into one of two TMEM buffers a branch, the
// weights by one warpgroup a branch (a row a thread, lazily moved maximum), written over
// S_b as bf16, and O_b += P_b V.  The work is cut by the lengths on the device (see
// paged_plan.cuh), and every role walks the block's segments on its own.
//
// What bounds it: the hand-offs between the weights' warps and the tensor core.  A tile of
// 64 keys takes 1,900 cycles.  Its operands are 1,540 cycles of shared memory at 128 bytes
// a cycle with head width 128 (96 KB of Q and K for the scores, 64 KB of V for both parts
// of both branches' weights, 32 KB of copies), 1,150 with 64; the weights' warps are busy
// for 1,500; HBM would take 1,000.  Timed with parts left out (16 sequences of 8192 keys, 64
// tokens; head width 128 on 8 key/value heads, 64 on 16): all 155 and 249 us, half of the
// products 149 and 242, no arithmetic between scores and weights 139 and 207, the cache in
// L2 147 and 246.  Sixteen warps for the weights in place of eight, half of a tile's keys
// each with a barrier a pair, took 6 % longer, and 4 % with everything unrolled over 64 keys
// (the warps then wait for instructions).  The row count hardly matters: 98 us with 9 tokens
// (ragged, 8 heads), 116 with 64.  Chunks of 512 and 1024 tokens run at 600 to 630 TFLOP/s.
//
// Warp roles (384 threads):
//   warps 0-3, 4-7   weights and results of branch 1, 2 (TMEM lanes 0-127)
//   warp 8           TMA producer: a lane a page of the tile
//   warps 9, 10      MMA issue for branch 1, 2; warp 9 allocates TMEM
//   warp 11          makes the values of tiles that reach into the new tokens safe
//
// A product with a weight of zero is not zero where the value is NaN or infinite, and the
// cache behind a sequence's end, or a drafted token that a row does not see, may hold
// either.  So in those tiles (the last one or two of a sequence) warp 11 puts zeros for
// rows past the end, and for single values that are not finite it puts zeros and marks
// the key; the results' warps then add such a value to the rows that see its key.
#include <cfloat>

#include "paged_plan.cuh"
#include "kernels.h"
#include "pdl.cuh"

namespace diffattn {
namespace ptc {

constexpr int BM = 128;
constexpr int KT = 64;
constexpr int DV = 128;
constexpr int SNAP = 3;
constexpr int EXTRA = 6;                        // what a unit's start costs, in tiles
constexpr int THREADS = 384;
// launched at 168 registers a thread: 256 x 200 + 128 x 104 = 384 x 168
constexpr uint32_t REGS_SOFTMAX = 200, REGS_OTHER = 104;
static_assert(256 * REGS_SOFTMAX + 128 * REGS_OTHER <= THREADS * 168, "register split");
constexpr uint32_t Q_PANEL = BM * 128;          // 16 KB
constexpr uint32_t K_PANEL = KT * 128;          // 8 KB: 64 keys x 64 columns
constexpr uint32_t V_BYTES = 2 * K_PANEL;
constexpr int VST = 5;                          // value stages
constexpr int KST_MAX = 5;
constexpr int SEGS = 8;                         // segments whose flags are kept apart
constexpr int FLAGS = 18;                       // tiles that reach into the new tokens: (1024 + 63) / 64 + 1
// A finite stand-in for the maximum of a row that has seen nothing: no score is lower.
constexpr float NOTHING = -FLT_MAX;
// What the sum of 32 weights may reach before the maximum m is looked at again.  The exponent s *
// scale - m is one fused operation, so the highest score's is not 0 but what m's own rounding left:
// nothing up to 2^24, but from 2^31 on an infinity or no weight at all.  Beyond 2^24 the limit is
// below any sum, and the weights are formed again with the product rounded as m was.  (Two
// operations for every score: 3 % of the time of 64 tokens over 16 x 8192, for scores that no
// ordinary head has.)
__device__ __forceinline__ float sum_limit(float m) { return fabsf(m) < 16777216.f || m == NOTHING ? 256.f : -1.f; }

template <int HD, bool KS>
struct Cfg {
    static constexpr int KP = HD / 64;
    static constexpr int NK = KS ? 1 : 2;
    static constexpr uint32_t Q_BYTES = KP * Q_PANEL;               // a branch
    static constexpr uint32_t K_BYTES = KP * K_PANEL;               // a branch's key tile
    static constexpr uint32_t K_STAGE = NK * K_BYTES;               // 8, 16 or 32 KB
    static constexpr int KST = HD == 128 && !KS ? 2 : KST_MAX;
    static constexpr uint32_t OFF_K = 2 * Q_BYTES;
    static constexpr uint32_t OFF_V = OFF_K + KST * K_STAGE;
    static constexpr uint32_t OFF_BAR = OFF_V + VST * V_BYTES;
};

enum : int {
    B_Q_FULL, B_Q_EMPTY,
    B_K_FULL, B_K_EMPTY = B_K_FULL + KST_MAX,
    B_V_FULL = B_K_EMPTY + KST_MAX, B_V_EMPTY = B_V_FULL + VST, B_V_SAFE = B_V_EMPTY + VST,
    B_S_FULL = B_V_SAFE + VST,                  // [branch][buffer]
    B_P_FULL = B_S_FULL + 4,                    // [branch][buffer]
    B_PV_DONE = B_P_FULL + 4,                   // [branch]
    B_O_FULL = B_PV_DONE + 2, B_O_EMPTY,
    B_ROWS,                                     // sums exchanged between the warpgroups
    B_FINAL,                                    // [branch]
    NUM_BARS = B_FINAL + 2
};
constexpr uint32_t REL_TMEM = NUM_BARS * 8;
constexpr uint32_t REL_ABORT = REL_TMEM + 4;
constexpr uint32_t REL_BAD = REL_ABORT + 4;                         // uint32 [SEGS]
constexpr uint32_t REL_FLAGS = (REL_BAD + SEGS * 4 + 7) & ~7u;      // uint64 [SEGS][FLAGS]
constexpr uint32_t REL_ANY = REL_FLAGS + SEGS * FLAGS * 8;          // uint32 [SEGS]
constexpr uint32_t REL_END = REL_ANY + SEGS * 4;
template <int HD, bool KS>
constexpr uint32_t smem_bytes() { return Cfg<HD, KS>::OFF_BAR + REL_END + 1024; }
static_assert(smem_bytes<128, true>() <= 232448 - 256 && smem_bytes<64, false>() <= 232448 - 256 &&
              smem_bytes<128, false>() <= 232448 - 256, "shared memory");

constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TM_O = 256;
constexpr uint32_t IDESC_S = idesc_bf16_f32(BM, KT, 0, 0);
constexpr uint32_t IDESC_PV = idesc_bf16_f32(BM, DV, 0, 1);
__device__ __forceinline__ uint32_t tm_s(int br, int buf) { return br * 128 + buf * 64; }

__device__ __forceinline__ bool bf16_finite(uint32_t half) { return (half & 0x7f80u) != 0x7f80u; }

// 16 rows x 32 columns of TMEM: of each 8 columns, words 4 i .. 4 i + 3 of lane t are row
// t / 4, columns 2 (t % 4) and the next, and the same of row t / 4 + 8.
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr) : "memory");
}

// Maximum of 32 scores, in three chains.
__device__ __forceinline__ float half_max(const uint32_t (&s)[32]) {
    auto f = [&](int i) { return __uint_as_float(s[i]); };
    float a = fmaxf(f(0), f(1)), b = f(2), c = f(3);
#pragma unroll
    for (int i = 4; i < 28; i += 6) {
        a = fmax3(a, f(i), f(i + 1));
        b = fmax3(b, f(i + 2), f(i + 3));
        c = fmax3(c, f(i + 4), f(i + 5));
    }
    a = fmax3(a, f(28), f(29));
    b = fmax3(b, f(30), f(31));
    return fmax3(a, b, c);
}
// A pair of weights as two bf16 parts, what the first leaves in the second.
__device__ __forceinline__ void split2(uint64_t w, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16x2(f2_lo(w), f2_hi(w));
    const uint64_t d = f2_sub(w, f2_pack(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)));
    lo = pack_bf16x2(f2_lo(d), f2_hi(d));
}
// P = 2^(s * scale_log2 - m) for 32 scores, and the sum of P.  Rounded to one bf16, P would
// put an error of 2e-3 of the result's size into long caches, where the means of the two
// branches cancel; so it is the sum of two: pk[0..15] and what is left, pk[16..31], 2^-16 together
// (and as much once more for a tile's first half where the maximum moves in its second).
__device__ __forceinline__ float half_weights(const uint32_t (&s)[32], float sl2, float m, uint32_t (&pk)[32]) {
    const uint64_t scale2 = f2_pack(sl2, sl2);
    const uint64_t negm2 = f2_pack(-m, -m);
    uint64_t rsum[2] = {0, 0};
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        const uint64_t x = f2_fma(f2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), scale2, negm2);
        const uint64_t w = f2_pack(ex2_approx(f2_lo(x)), ex2_approx(f2_hi(x)));
        rsum[c & 1] = f2_add(rsum[c & 1], w);
        split2(w, pk[c], pk[16 + c]);
    }
    const uint64_t r = f2_add(rsum[0], rsum[1]);
    return f2_lo(r) + f2_hi(r);
}

// A bf16 pair with zeros for what is not finite.
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
    if (!bf16_finite(w)) w &= 0xffff0000u;
    if (!bf16_finite(w >> 16)) w &= 0x0000ffffu;
    return w;
}
// 16-byte chunk c (of 16) of a key's value row in a staged tile.
__device__ __forceinline__ uint4* value_at(uint8_t* vt, int key, int c) {
    return reinterpret_cast<uint4*>(vt + (c >> 3) * K_PANEL + key * 128 + (((c & 7) ^ (key & 7)) << 4));
}

// Bits of the 64 keys from k0 on that a row sees (bit d of `tree`: new token d).
__device__ __forceinline__ uint64_t tile_mask(const PagedParams& p, const PagedSeq& s, int k0, int q, uint64_t tree) {
    auto low = [](int64_t n) -> uint64_t { return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1; };
    const int64_t off = s.before - k0;          // keys of the tile before the new tokens, < 64
    uint64_t m;
    if (p.mask) m = off <= 0 ? (off <= -64 ? 0 : tree >> -off) : (tree << off) | low(off);
    else m = low(off + q + 1);
    return m & low((int64_t)s.total - k0);
}

template <int HD, bool KS>
__global__ void __launch_bounds__(THREADS, 1)
paged_tc_kernel(const __grid_constant__ CUtensorMap tm_q1, const __grid_constant__ CUtensorMap tm_q2,
                const __grid_constant__ CUtensorMap tm_k1, const __grid_constant__ CUtensorMap tm_k2,
                const __grid_constant__ CUtensorMap tm_v, const PagedParams p, const int box_rows, const int q_box) {
    using C = Cfg<HD, KS>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int scan[2 * THREADS / 32];
    __shared__ PagedBlock<1> blk;
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + REL_TMEM);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_BAR + REL_ABORT);
    volatile uint32_t* bad_seg = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_BAR + REL_BAD);
    volatile uint64_t* flags = reinterpret_cast<volatile uint64_t*>(smem + C::OFF_BAR + REL_FLAGS);
    volatile uint32_t* any_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_BAR + REL_ANY);
    const uint32_t warp = warp_id();
    const uint32_t lane = threadIdx.x & 31;
    const AbortState ab{abort_flag, p.status};
    if (threadIdx.x < NUM_BARS) {
        const int i = threadIdx.x;
        int arrivals = 1;
        if ((i >= B_K_EMPTY && i < B_K_EMPTY + KST_MAX) || i == B_Q_EMPTY || i == B_O_FULL) arrivals = 2;   // both products
        if (i >= B_V_EMPTY && i < B_V_EMPTY + VST) arrivals = 3;        // and warp 11
        if (i >= B_P_FULL && i < B_P_FULL + 4) arrivals = 4;            // a branch's warps
        if (i == B_O_EMPTY || i == B_ROWS) arrivals = 8;                // both branches'
        mbar_init(&bars[i], arrivals);
        if (i < SEGS) bad_seg[i] = any_flag[i] = 0;
        if (i == 0) *abort_flag = 0;
        fence_mbar_init();
    }
    // rows of the query tiles that no head fills stay zero: their scores must be finite
    for (uint32_t i = threadIdx.x; i < 2 * C::Q_BYTES / 16; i += THREADS)
        reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (warp == 9) {
        tmem_alloc(tmem_ptr, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    pdl_wait();                                 // before the merging pass may start, which writes too
    pdl_launch_dependents();
    paged_locate<1>(p, paged_scan<THREADS>(p, KT, EXTRA, scan), KT, EXTRA, 1, p.workers, SNAP, &blk);    // with their barriers
    tc_fence_after();
    const uint32_t tmem_base = *tmem_ptr;
    const uint64_t lim = 200ull * 1000ull * 1000ull;
    PagedCursor cur;

    if (warp >= 8) {
        regs_dec<REGS_OTHER>();
        cur.begin(p, blk, 0, blockIdx.x, KT, EXTRA);
        if (warp == 8) {
            // ------------------------------------------------------------ producer
            if (lane == 0) {
                tma_prefetch_desc(&tm_q1);
                tma_prefetch_desc(&tm_q2);
                tma_prefetch_desc(&tm_k1);
                tma_prefetch_desc(&tm_k2);
                tma_prefetch_desc(&tm_v);
            }
            constexpr int Q_LEAD = (C::KST < VST ? C::KST : VST) - 1;   // tiles that may go ahead of their queries
            const int boxes = KT / box_rows;
            uint32_t kst = 0, kph = 1, vst = 0, vph = 1, nk = 0, nv = 0, nq = 0;
            bool ok = true;
            if (lane == 0) PagedCursor::no_join(p, blockIdx.x);
            int seg = -1;                       // segments with tiles, as every role counts them
            for (; ok && !cur.done(); cur.next(p, KT, EXTRA)) {
                const int live = cur.live_tiles(p, KT);
                if (cur.s.bad && lane == 0) atomicOr(p.status, kStatusIndex);
                if (lane == 0) cur.join(p, blk.shares, blk.start[1].tile, EXTRA);
                if (live == 0) continue;
                ++seg;
                if (lane == 0) bad_seg[seg % SEGS] = 0;
                // the unit's queries: a box a head and panel, once the last segment's scores are done
                bool have_q = false;
                auto load_q = [&](bool wait) -> bool {
                    if (nq > 0) {
                        const uint32_t par = (nq - 1) & 1;
                        if (wait) {
                            if (!mbar_wait_warp(&bars[B_Q_EMPTY], par, ab)) return false;
                        } else if (!__all_sync(0xffffffffu, mbar_test(&bars[B_Q_EMPTY], par))) {
                            return true;
                        }
                    }
                    have_q = true;
                    ++nq;
                    if (lane == 0) {
                        const int row0 = cur.rc * p.chunk_rows;
                        const int h0 = row0 / p.head_rows, q0 = row0 % p.head_rows;
                        const int heads = min((p.chunk_rows + p.head_rows - 1) / p.head_rows, p.group - h0);
                        mbar_arrive_expect_tx(&bars[B_Q_FULL], heads * C::KP * 2 * q_box * 128);
                        for (int h = 0; h < heads; ++h)
#pragma unroll
                            for (int pn = 0; pn < C::KP; ++pn) {
                                uint8_t* dst = smem + pn * Q_PANEL + h * p.head_rows * 128;
                                tma_load_4d(dst, &tm_q1, &bars[B_Q_FULL], pn * 64, q0, cur.hk * p.group + h0 + h, cur.b);
                                tma_load_4d(dst + C::Q_BYTES, &tm_q2, &bars[B_Q_FULL], pn * 64, q0,
                                            cur.hk * p.group + h0 + h, cur.b);
                            }
                    }
                    __syncwarp();
                    return true;
                };
                auto look = [&](int i) -> int {     // the page of this lane's box
                    const int key = (cur.tile0 + i) * KT + (int)lane * box_rows;
                    if (i >= live || (int)lane >= boxes || key >= cur.s.total) return -2;
                    return paged_page(p, cur.b, key / p.page);
                };
                int page = look(0);
                for (int i = 0; i < live; ++i) {
                    const int now = page;
                    page = look(i + 1);
                    if (!have_q && !(ok = load_q(i >= Q_LEAD))) break;
                    const int key = (cur.tile0 + i) * KT + (int)lane * box_rows;
                    const int slot = key % p.page;
                    const unsigned have = __ballot_sync(0xffffffffu, now >= 0);
                    if (__any_sync(0xffffffffu, now == -1) && lane == 0) {
                        bad_seg[seg % SEGS] = 1;
                        atomicOr(p.status, kStatusIndex);
                    }
                    const uint32_t rows = __popc(have) * box_rows;
                    if (!(ok = mbar_wait_warp(&bars[B_K_EMPTY + kst], kph, ab))) break;
                    if (lane == 0) {
                        if (rows) mbar_arrive_expect_tx(&bars[B_K_FULL + kst], rows * 128 * C::KP * C::NK);
                        else mbar_arrive(&bars[B_K_FULL + kst]);
                    }
                    __syncwarp();
                    if (now >= 0) {
                        uint8_t* dst = smem + C::OFF_K + kst * C::K_STAGE + lane * box_rows * 128;
#pragma unroll
                        for (int pn = 0; pn < C::KP; ++pn) {
                            tma_load_4d(dst + pn * K_PANEL, &tm_k1, &bars[B_K_FULL + kst], pn * 64, slot, cur.hk, now);
                            if (!KS)
                                tma_load_4d(dst + C::K_BYTES + pn * K_PANEL, &tm_k2, &bars[B_K_FULL + kst], pn * 64, slot,
                                            cur.hk, now);
                        }
                    }
                    ++nk;
                    if (++kst == (uint32_t)C::KST) { kst = 0; kph ^= 1; }
                    if (!(ok = mbar_wait_warp(&bars[B_V_EMPTY + vst], vph, ab))) break;
                    if (lane == 0) {
                        if (rows) mbar_arrive_expect_tx(&bars[B_V_FULL + vst], rows * 128 * 2);
                        else mbar_arrive(&bars[B_V_FULL + vst]);
                    }
                    __syncwarp();
                    if (now >= 0) {
                        uint8_t* dst = smem + C::OFF_V + vst * V_BYTES + lane * box_rows * 128;
                        tma_load_4d(dst, &tm_v, &bars[B_V_FULL + vst], 0, slot, cur.hk, now);
                        tma_load_4d(dst + K_PANEL, &tm_v, &bars[B_V_FULL + vst], 64, slot, cur.hk, now);
                    }
                    ++nv;
                    if (++vst == (uint32_t)VST) { vst = 0; vph ^= 1; }
                }
                if (ok && !have_q) ok = load_q(true);
            }
            // no copy may be in flight when the block ends
            if (nq) mbar_wait_teardown(&bars[B_Q_FULL], (nq - 1) & 1, lim);
            for (uint32_t t = nk > (uint32_t)C::KST ? nk - C::KST : 0; t < nk; ++t)
                mbar_wait_teardown(&bars[B_K_FULL + t % C::KST], (t / C::KST) & 1, lim);
            for (uint32_t t = nv > (uint32_t)VST ? nv - VST : 0; t < nv; ++t)
                mbar_wait_teardown(&bars[B_V_FULL + t % VST], (t / VST) & 1, lim);
            __syncwarp();
        } else if (warp == 11) {
            // ------------------------------------------- values that must not be multiplied
            uint32_t vst = 0, vph = 0;
            bool ok = true;
            int seg = -1;
            for (; ok && !cur.done(); cur.next(p, KT, EXTRA)) {
                const int live = cur.live_tiles(p, KT);
                if (live == 0) continue;
                ++seg;
                const int edge0 = (int)(cur.s.before / KT);         // the first tile with a new token
                if (lane < FLAGS) flags[(seg % SEGS) * FLAGS + lane] = 0;
                if (lane == 0) any_flag[seg % SEGS] = 0;
                __syncwarp();
                for (int i = 0; i < live; ++i) {
                    const int tile = cur.tile0 + i;
                    if (!(ok = mbar_wait_warp(&bars[B_V_FULL + vst], vph, ab))) break;
                    if (tile >= edge0) {
                        uint8_t* vt = smem + C::OFF_V + vst * V_BYTES;
                        // eight reads at a time; what is found is almost always nothing
                        uint32_t lo = 0, hi = 0;            // keys with a value that is not finite
                        for (int j0 = 0; j0 < KT / 2; j0 += 8) {
                            uint4 x[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                x[j] = *value_at(vt, 2 * (j0 + j) + (int)(lane >> 4), lane & 15);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const int key = 2 * (j0 + j) + (int)(lane >> 4);
                                const bool past = tile * KT + key >= cur.s.total;
                                const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
                                // an exponent of ones carries into the sign's place
                                uint32_t ones = 0;
#pragma unroll
                                for (int e = 0; e < 4; ++e) ones |= (w[e] & 0x7f807f80u) + 0x00800080u;
                                const bool odd = (ones & 0x80008000u) != 0;
                                if (past) {
                                    *value_at(vt, key, lane & 15) = make_uint4(0, 0, 0, 0);
                                } else if (odd) {
                                    *value_at(vt, key, lane & 15) = make_uint4(finite_only(w[0]), finite_only(w[1]),
                                                                               finite_only(w[2]), finite_only(w[3]));
                                    if (key < 32) lo |= 1u << key;
                                    else hi |= 1u << (key - 32);
                                }
                            }
                        }
                        lo = __reduce_or_sync(0xffffffffu, lo);
                        hi = __reduce_or_sync(0xffffffffu, hi);
                        if ((lo | hi) && lane == 0 && tile - edge0 < FLAGS) {
                            flags[(seg % SEGS) * FLAGS + tile - edge0] = (uint64_t)hi << 32 | lo;
                            any_flag[seg % SEGS] = 1;
                        }
                        fence_proxy_async_smem();
                        __threadfence_block();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars[B_V_SAFE + vst]);
                    }
                    // every stage passes here, so that this warp never falls a phase behind
                    if (lane == 0) mbar_arrive(&bars[B_V_EMPTY + vst]);
                    if (++vst == (uint32_t)VST) { vst = 0; vph ^= 1; }
                }
            }
        } else {
            // --------------------------------------------- MMA issue, one warp a branch
            const int br = warp - 9;
            if (elect_one()) {
                const uint64_t qdesc = sdesc_sw128(smem_u32(smem + br * C::Q_BYTES), 16, 1024);
                const uint64_t kdesc = sdesc_sw128(smem_u32(smem + C::OFF_K + (KS ? 0 : br) * C::K_BYTES), 16, 1024);
                const uint64_t vdesc = sdesc_sw128(smem_u32(smem + C::OFF_V), K_PANEL, 1024);
                const uint32_t d_o = tmem_base + TM_O + br * 128;
                uint32_t kst = 0, kph = 0, vst = 0, vph = 0, qph = 0, oeph = 0, pph = 0, safeph = 0;
                bool ok = true, first = true;
                auto issue_s = [&](uint32_t stage, int buf) {
                    const uint32_t d = tmem_base + tm_s(br, buf);
                    const uint64_t kd = kdesc + ((stage * C::K_STAGE) >> 4);
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk) {
                        const uint32_t pn = kk >> 2, ks = kk & 3;
                        mma_ss(d, qdesc + pn * (Q_PANEL >> 4) + 2 * ks, kd + pn * (K_PANEL >> 4) + 2 * ks, IDESC_S, kk > 0);
                    }
                    mma_commit(&bars[B_S_FULL + 2 * br + buf]);
                    mma_commit(&bars[B_K_EMPTY + stage]);
                };
                for (; ok && !cur.done(); cur.next(p, KT, EXTRA)) {
                    const int n = cur.live_tiles(p, KT);
                    if (n == 0) continue;
                    const int edge0 = (int)(cur.s.before / KT);
                    if (!(ok = mbar_wait(&bars[B_Q_FULL], qph, ab))) break;
                    qph ^= 1;
                    for (int t = 0; t < 2 && t < n; ++t) {
                        if (!(ok = mbar_wait(&bars[B_K_FULL + kst], kph, ab))) break;
                        tc_fence_after();
                        issue_s(kst, t);
                        if (++kst == (uint32_t)C::KST) { kst = 0; kph ^= 1; }
                    }
                    if (!ok) break;
                    if (n <= 2) mma_commit(&bars[B_Q_EMPTY]);
                    for (int j = 0; j < n; ++j) {
                        const int buf = j & 1;
                        if (!(ok = mbar_wait(&bars[B_V_FULL + vst], vph, ab))) break;
                        if (cur.tile0 + j >= edge0) {
                            if (!(ok = mbar_wait(&bars[B_V_SAFE + vst], (safeph >> vst) & 1u, ab))) break;
                            safeph ^= 1u << vst;
                        }
                        if (j + 2 < n && !(ok = mbar_wait(&bars[B_K_FULL + kst], kph, ab))) break;
                        if (j == 0 && !first) {
                            if (!(ok = mbar_wait(&bars[B_O_EMPTY], oeph, ab))) break;
                            oeph ^= 1;
                        }
                        if (!(ok = mbar_wait(&bars[B_P_FULL + 2 * br + buf], (pph >> buf) & 1u, ab))) break;
                        pph ^= 1u << buf;
                        tc_fence_after();
                        const uint64_t vd = vdesc + ((vst * V_BYTES) >> 4);
#pragma unroll
                        for (int kk = 0; kk < KT / 8; ++kk)     // a half: 32 keys' first parts, then their second ones
                            mma_ts(d_o, tmem_base + tm_s(br, buf) + kk * 8, vd + 128 * (kk / 4 * 2 + kk % 2), IDESC_PV,
                                   (j > 0 || kk > 0) ? 1u : 0u);
                        mma_commit(&bars[B_PV_DONE + br]);
                        mma_commit(&bars[B_V_EMPTY + vst]);
                        if (++vst == (uint32_t)VST) { vst = 0; vph ^= 1; }
                        if (j + 2 < n) {
                            issue_s(kst, buf);
                            if (++kst == (uint32_t)C::KST) { kst = 0; kph ^= 1; }
                            if (j + 3 == n) mma_commit(&bars[B_Q_EMPTY]);
                        }
                    }
                    if (!ok) break;
                    mma_commit(&bars[B_O_FULL]);
                    first = false;
                }
                mma_commit(&bars[B_FINAL + br]);        // before TMEM is freed
                mbar_wait_teardown(&bars[B_FINAL + br], 0, lim);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------ weights and results
        regs_inc<REGS_SOFTMAX>();
        cur.begin(p, blk, 0, blockIdx.x, KT, EXTRA);
        const int br = warp >> 2;
        const uint32_t quad = warp & 3;
        const int row = quad * 32 + lane;
        const uint32_t lane_base = tmem_base + ((quad * 32u) << 16);
        const uint32_t tO = lane_base + TM_O + br * 128;     // this branch's O
        const float sl2 = p.scale_log2;
        const float lam = p.lambda_dev ? __ldg(p.lambda_dev) : p.lambda;
        uint32_t sph = 0, ofph = 0, wph = 0;
        uint32_t pv_count = 0;
        bool ok = true;
        int seg = -1;
        for (; ok && !cur.done(); cur.next(p, KT, EXTRA)) {
            const int live = cur.live_tiles(p, KT);
            if (live > 0) ++seg;
            const PagedSeq s = cur.s;
            const PagedRow x = paged_row(p, cur.hk, cur.rc, row, s.n_new);
            const bool mine = x.live && row < p.chunk_rows;
            uint64_t tree = 0;
            if (p.mask && (int64_t)(cur.tile0 + live) * KT > s.before)
                tree = paged_mask_bits<32>(p, cur.b, x.q, mine, s.n_new, lane);
            float m_run = NOTHING, l = 0.f, limit = 256.f;
            for (int j = 0; j < live; ++j) {
                const int buf = j & 1;
                const uint32_t tS = lane_base + tm_s(br, buf);
                if (!(ok = mbar_wait_warp(&bars[B_S_FULL + 2 * br + buf], (sph >> buf) & 1u, ab))) break;
                sph ^= 1u << buf;
                tc_fence_after();
                const int k0 = (cur.tile0 + j) * KT;
                const bool edge = k0 + KT > s.before;
                const uint64_t vis = edge && mine ? tile_mask(p, s, k0, x.q, tree) : 0;
                // A loop over the tile's halves that stays one: each 32 keys' weights go over
                // their scores, 16 columns a part.  Unrolled, it waited for instructions a fifth
                // of the time (61 tokens over 16 x 8192: 125 us, 121 as a loop).
#pragma unroll 1
                for (int h = 0; ok && h < 2; ++h) {
                    uint32_t sc[32], pk[32];
                    tmem_ld32(tS + 32 * h, sc);
                    tmem_wait_ld();
                    if (edge) {
                        const uint32_t seen = (uint32_t)(vis >> (32 * h));
#pragma unroll
                        for (int c = 0; c < 32; ++c) sc[c] = (seen >> c & 1u) ? sc[c] : 0xff800000u;
                    }
                    const bool first = j == 0 && h == 0;
                    if (first) {
                        m_run = fmaxf(half_max(sc) * sl2, NOTHING);
                        limit = sum_limit(m_run);
                    }
                    float tsum = half_weights(sc, sl2, m_run, pk);
                    if (__any_sync(0xffffffffu, !(tsum <= limit))) {
                        const float mxs = half_max(sc) * sl2;
                        const bool move = __any_sync(0xffffffffu, mxs > m_run + 8.0f);
                        float alpha = 1.f;
                        if (move) {
                            const float m_new = fmaxf(m_run, mxs);
                            alpha = ex2_approx(m_run - m_new);
                            l *= alpha;
                            m_run = m_new;
                            limit = sum_limit(m_run);
                        }
                        if (move || __any_sync(0xffffffffu, limit < 0.f)) {
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                sc[c] = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(sc[c]), sl2), -m_run));
                            tsum = half_weights(sc, 1.f, 0.f, pk);
                        }
                        if (move) {
                            uint32_t o[32];
                            if (h == 1) {       // the first half's weights
                                tmem_wait_st();
                                tmem_ld32(tS, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    auto both = [&](uint32_t a, uint32_t b) { return (__uint_as_float(a) + __uint_as_float(b)) * alpha; };
                                    split2(f2_pack(both(o[i] << 16, o[16 + i] << 16),
                                                   both(o[i] & 0xffff0000u, o[16 + i] & 0xffff0000u)), o[i], o[16 + i]);
                                }
                                tmem_st32(tS, o);
                            }
                            if (j > 0) {        // and O
                                ok = mbar_wait_warp(&bars[B_PV_DONE + br], (pv_count + j - 1) & 1u, ab);
                                tc_fence_after();
#pragma unroll 1
                                for (int c4 = 0; ok && c4 < 4; ++c4) {
                                    tmem_ld32(tO + c4 * 32, o);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                                    tmem_st32(tO + c4 * 32, o);
                                }
                            }
                        }
                    }
                    tmem_st32(tS + 32 * h, pk);
                    l += tsum;
                }
                if (!ok) break;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_P_FULL + 2 * br + buf]);
            }
            if (!ok) break;
            pv_count += live;
            if (live > 0) {
                if (!(ok = mbar_wait_warp(&bars[B_O_FULL], ofph, ab))) break;
                ofph ^= 1;
                tc_fence_after();
            }
            // Every exchange between the warps is a phase of one barrier.
            auto exchange = [&]() -> bool {
                __threadfence_block();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_ROWS]);
                const bool got = mbar_wait_warp(&bars[B_ROWS], wph, ab);
                wph ^= 1;
                return got;
            };
            // a segment without tiles: the last one's exchanges must be over before its places
            // are written again (with tiles, the weights' barriers see to that)
            if (live == 0 && !(ok = exchange())) break;
            if (s.bad || (live > 0 && bad_seg[seg % SEGS])) l = __int_as_float(0x7fc00000);
            const bool odd = live > 0 && any_flag[seg % SEGS] != 0;
            float* part = p.part + ((int64_t)cur.slot() * p.chunk_rows + row) * paged_part_floats(DV);
            if (mine) *reinterpret_cast<float2*>(part + 2 * br) = make_float2(m_run, l);
            // O may be overwritten once every warp has read its share of it
            auto release_o = [&]() {
                if (live == 0) return;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_O_EMPTY]);
            };
            if (!cur.whole() || odd) {
                // ---- a partial result: this branch's 128 columns of the row, read from TMEM so
                // that four lanes hold 32 bytes of a row: a row a lane is 32 lines a store (4 us a
                // segment), and turning that by shuffles took as long.  Loops that stay loops,
                // here and below: this code runs once or twice a block, and its first fetch is
                // what it costs (17 us for the first segment with everything unrolled).
                const unsigned rows = __ballot_sync(0xffffffffu, mine);
                float* at = p.part + ((int64_t)cur.slot() * p.chunk_rows + quad * 32 + (lane >> 2)) * paged_part_floats(DV) + 4 +
                            br * DV + 2 * (lane & 3);
#pragma unroll 1
                for (int i = 0; i < 2 * DV / 32; ++i) {
                    const int r0 = i & 1 ? 16 : 0, c = (i >> 1) * 32;
                    uint32_t o[16] = {};
                    if (live > 0) {
                        tmem_ld_rows16(tO + ((uint32_t)r0 << 16) + c, o);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (rows >> (r0 + 8 * k + (lane >> 2)) & 1u)
#pragma unroll
                            for (int n = 0; n < 4; ++n)
                                *reinterpret_cast<float2*>(at + (r0 + 8 * k) * paged_part_floats(DV) + c + 8 * n) =
                                    make_float2(__uint_as_float(o[4 * n + 2 * k]), __uint_as_float(o[4 * n + 2 * k + 1]));
                }
                release_o();
                if (odd) {
                    // to the row, the values that are not finite of keys that it sees
                    __syncwarp();
                    const int edge0 = (int)(s.before / KT);
#pragma unroll 1
                    for (int f = 0; mine && f < FLAGS; ++f) {
                        uint64_t keys = flags[(seg % SEGS) * FLAGS + f];
                        if (keys) keys &= tile_mask(p, s, (edge0 + f) * KT, x.q, tree);
                        while (keys) {
                            const int key = (edge0 + f) * KT + __ffsll(keys) - 1;
                            keys &= keys - 1;
                            const int page = paged_page(p, cur.b, key / p.page);
                            if (page < 0) continue;
                            const uint16_t* v = reinterpret_cast<const uint16_t*>(
                                static_cast<const __nv_bfloat16*>(p.v) + page * p.s_v[0] + cur.hk * p.s_v[1] +
                                (int64_t)(key % p.page) * p.s_v[2]);
#pragma unroll 1
                            for (int c = 0; c < DV; ++c)
                                if (!bf16_finite(v[c])) part[4 + br * DV + c] += __uint_as_float((uint32_t)v[c] << 16);
                        }
                    }
                }
                if (!cur.whole()) continue;
                // a whole unit with such a value is finished from the workspace
                if (!(ok = exchange())) break;
#pragma unroll 1
                for (int r = warp; r < p.chunk_rows; r += 8) {
                    const PagedRow y = paged_row(p, cur.hk, cur.rc, r, s.n_new);
                    if (!y.live) continue;
                    const volatile float* src = p.part + ((int64_t)cur.slot() * p.chunk_rows + r) * paged_part_floats(DV);
                    float o1[DV / 32], o2[DV / 32];
#pragma unroll
                    for (int i = 0; i < DV / 32; ++i) {
                        o1[i] = src[4 + lane + 32 * i];
                        o2[i] = src[4 + DV + lane + 32 * i];
                    }
                    paged_finish_row<DV / 32>(p, lam, cur.b, y.h, y.q, lane, o1, src[1], o2, src[3]);
                }
                if (!(ok = exchange())) break;
                continue;
            }
            // ---- a whole unit: this warpgroup takes 64 columns of both branches' O.  The
            // other's sums come through the row's place in the workspace: shared memory is full.
            if (!(ok = exchange())) break;
            const volatile float* sums = part;
            float i1 = 0.f, i2 = 0.f;
            if (mine) {
                const float l1 = sums[1], l2 = sums[3];
                i1 = l1 == 0.f ? 0.f : 1.f / l1;            // a row that saw nothing gives 0
                i2 = l2 == 0.f ? 0.f : 1.f / l2;
            }
            const int c0 = br * 64;
            float y[64];
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
                uint32_t o1[32] = {}, o2[32] = {};
                if (live > 0) {
                    tmem_ld32(lane_base + TM_O + c0 + c, o1);
                    tmem_ld32(lane_base + TM_O + 128 + c0 + c, o2);
                    tmem_wait_ld();
                }
                if (c == 32) release_o();
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    y[c + i] = fmaf(-lam, __fmul_rn(__uint_as_float(o2[i]), i2), __fmul_rn(__uint_as_float(o1[i]), i1));
                    sum += y[c + i];
                }
            }
            if (p.norm != kNormNone) {
                float mean = 0.f;
                if (p.norm == kNormGroup) {
                    if (mine) part[4 + br] = sum;
                    if (!(ok = exchange())) break;
                    if (mine) mean = (sums[4] + sums[5]) / DV;
                }
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    y[i] -= mean;
                    ss = fmaf(y[i], y[i], ss);
                }
                if (mine) part[6 + br] = ss;
                if (!(ok = exchange())) break;
                if (mine) {
                    const float r = 1.0f / sqrtf((sums[6] + sums[7]) / DV + p.norm_eps);
#pragma unroll
                    for (int i = 0; i < 64; ++i) y[i] *= r;
                }
            }
            if (mine) {
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + cur.b * p.s_o[0] + x.h * p.s_o[1] + x.q * p.s_o[2] + c0;
                const float* wt = p.norm_weight ? p.norm_weight + (int64_t)x.h * DV + c0 : nullptr;
                const float* bias = p.norm_bias ? p.norm_bias + (int64_t)x.h * DV + c0 : nullptr;
#pragma unroll
                for (int i = 0; i < 64; i += 8) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[e] = y[i + e];
                        if (wt) v[e] *= wt[i + e];
                        if (bias) v[e] += bias[i + e];
                        v[e] *= p.out_scale;
                    }
                    if (p.o16) {
                        *reinterpret_cast<uint4*>(out + i) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                                        pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) out[i + e] = __float2bfloat16_rn(v[e]);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem_base, TMEM_COLS);
}

template <int HD, bool KS>
int launch_hd(const CUtensorMap* m, const PagedParams& p, int box_rows, int q_box, cudaStream_t stream) {
    constexpr uint32_t smem = smem_bytes<HD, KS>();
    if (cudaFuncSetAttribute(paged_tc_kernel<HD, KS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return -1;
    const int rc = pdl_launch(paged_tc_kernel<HD, KS>, dim3(p.workers), THREADS, smem, stream, m[3], m[4], m[0], m[1], m[2],
                              p, box_rows, q_box);
    return rc == 0 ? launch_paged_combine(p, stream) : rc;
}

}  // namespace ptc

int launch_paged_tc(const CUtensorMap* maps, const PagedParams& p, int box_rows, int q_box, cudaStream_t stream) {
    if (p.D == 64) return p.k_shared ? ptc::launch_hd<64, true>(maps, p, box_rows, q_box, stream)
                                     : ptc::launch_hd<64, false>(maps, p, box_rows, q_box, stream);
    return p.k_shared ? ptc::launch_hd<128, true>(maps, p, box_rows, q_box, stream)
                      : ptc::launch_hd<128, false>(maps, p, box_rows, q_box, stream);
}

}  // namespace diffattn
