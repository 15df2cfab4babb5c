// cross_bwd_tc.cu -- backward of differential attention over an encoder's states on the
// sm_103a tensor cores (bf16, V width 128; D = 64 with one key tensor or two, or the DIFF V2
// head D = 128 with one).  Sequence b has its first n_b of Tk states; Tq query rows.
//
//   A_b  = 2^(S_b log2(e) / sqrt(D) - lse_b)            S_b = Q_b K_b^T
//   dP   = dO V^T,     Dd_b = rowsum(A_b dP)
//   dS_1 = A_1 (dP - Dd_1)          dS_2 = -lambda A_2 (dP - Dd_2)
//   dQ_b = dS_b K_b / sqrt(D)       dK_b = dS_b^T Q_b / sqrt(D)
//   dV   = (A_1 - lambda A_2)^T dO  dlambda = -sum Dd_2
//
// stats holds each row's negated log2-sum-exps and, from the forward's saved results, its
// negated Dd_b.  Two kernels, as in the backward of self-attention (bwd_tc.cu), both
// persistent (one CTA an SM, items claimed from a counter, since sequences are of different
// lengths) with a TMA producer, an MMA-issuing thread and two warpgroups that turn scores
// into their gradients:
//
// dq: item (b, h, 128 query rows in TMEM lanes); a warpgroup a branch; per 64 states S_1, S_2
//   and dP, then dQ_b += dS_b K_b with dS_b in TMEM.
//   D = 64: two score buffers, dS_b written over S_b; dO in TMEM as dP's A operand.
//   D = 128: the dQ accumulators take 256 columns, so there is one score buffer, which the
//   warpgroups release as soon as it is in registers, dS_b has columns of its own and dO
//   is read from shared memory.
//   The warpgroups also sum A_b dP in float32: the row's Dd_b without the roundings of O,
//   which the dK/dV kernel and dlambda take.  dS itself needs Dd before that sum is known (but
//   over a single tile, where the sum comes first), and takes the saved one.  An error of Dd is
//   every dS's of the row, and dQ's times the keys' weighted mean: from bf16 results alone (2^-8 of
//   |dO| |O|) it was 13 % of dQ over 4096 states where keys and values have offsets of 2 and 1 of
//   their spread.  So the forward also leaves the rests of its roundings (18 us of 390 there, 9 here):
//   0.4 %, what dS's own rounding leaves of so much cancellation.
// dkdv: item (b, key/value head, 128 states in TMEM lanes, a split of the query rows where there
//   are few such tiles); over every 64 query rows of the group's heads: S_1^T, S_2^T, dP^T, then
//   dV += W^T dO, dK_b += dS_b^T Q_b (one accumulator for both branches where they share their
//   keys: one rounding).  States behind the sequence's own are lanes whose results are replaced
//   by zeros.
//
// Bound by the elementwise warps, at D = 64 in both (dq 1,500 cycles a tile against 770 of the
// tensor core; dkdv 2,150 against 1,020), and at D = 128 in dkdv; dq there by its operand reads
// from shared memory and the hand-offs of its one score buffer.  2 x 16 heads of 64, 4096 rows
// over 4096 states: 334 us and 474 us, with the V2 head (8 key/value heads) 523 and 686: 850 and
// 909 TFLOP/s of the products that a backward needs.
//
// dS_b and W = A_1 - lambda A_2 are rounded once, to bf16, for their products: errors of their own for
// each element, 2.4e-3 of a gradient with its own rounding.  Where alike branches share their keys,
// dK is the difference of two products that cancel, and off by 7e-3 of what is left; second parts of
// both dS would be two of the dK/dV kernel's seven products again.
//
// What a batch's padding holds must not reach a sum: in dq the rows of K and V behind a
// sequence's last state would meet weights of 0, and 0 times NaN is NaN, so a warp turns
// them into zeros in shared memory before the products read them.  (In dkdv such rows are
// TMEM lanes of their own.)
//
// Every mbarrier wait is bounded (ptx.cuh).
#include "block.h"
#include "item_ring.cuh"
#include "kernels.h"
#include "pdl.cuh"
#include "ptx.cuh"
#include "rows.cuh"

#include <cmath>

namespace diffattn {
namespace xbwd {

constexpr int VD = 128;
constexpr int NUM_THREADS = 384;
constexpr uint32_t REGS_WORK = 200;
constexpr uint32_t REGS_OTHER = 104;
static_assert(256 * REGS_WORK + 128 * REGS_OTHER <= NUM_THREADS * 168, "register split");
constexpr int RING = 4;                            // work items in flight
constexpr uint32_t TMEM_COLS = 512;
constexpr uint64_t TEARDOWN_NS = 200ull * 1000ull * 1000ull;

// Descriptor offset of the k-step kk (16 columns) of a K-major operand in panels of 64 columns.
__device__ __forceinline__ uint32_t kstep(int kk, uint32_t panel) { return (kk >> 2) * (panel >> 4) + 2 * (kk & 3); }

__device__ __forceinline__ uint4 pack8(const uint32_t* x, float s) {
    return make_uint4(pack_bf16x2(__uint_as_float(x[0]) * s, __uint_as_float(x[1]) * s),
                      pack_bf16x2(__uint_as_float(x[2]) * s, __uint_as_float(x[3]) * s),
                      pack_bf16x2(__uint_as_float(x[4]) * s, __uint_as_float(x[5]) * s),
                      pack_bf16x2(__uint_as_float(x[6]) * s, __uint_as_float(x[7]) * s));
}

// Items head by head in groups of `group` heads (whose operands share the L2), within a
// group tile by tile.
__device__ __forceinline__ void locate(int idx, int heads, int tiles, int group, int* head, int* tile) {
    const int per = group * tiles;
    const int g0 = idx / per * group;
    const int size = min(group, heads - g0);
    const int w = idx - g0 * tiles;
    *tile = w / size;
    *head = g0 + (w - *tile * size);
}

// ---------------------------------------------------------------------------
// The rows' statistics from the forward's saved results: Dd_2 = dO . (A_2 V), Dd_1 = dO . (O +
// lambda A_2 V), stored negated with the log2-sum-exps.  RESTS: with what the results' rounding left
// (two bf16 together, 2^-16).  16 lanes a row, 16 bytes a lane, two rows a group: HBM, 28 to 30 us at
// 131,000 rows with the rests, 0.85 to 0.9 of the copy rate (19 without).
// ---------------------------------------------------------------------------
constexpr int PREP_THREADS = 256;
constexpr int PREP_ROWS = 2;            // of a group of lanes, loaded together
template <bool RESTS>
__global__ void __launch_bounds__(PREP_THREADS, RESTS ? 4 : 6)
cross_prep_kernel(const CrossTcParams p) {
    constexpr int GROUPS = PREP_THREADS / 16, N = RESTS ? 5 : 3;
    const int g = threadIdx.x % 16, h = blockIdx.y % p.H, b = blockIdx.y / p.H;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 3) p.sched[threadIdx.x] = 0;
    const int q0 = blockIdx.x * (GROUPS * PREP_ROWS) + threadIdx.x / 16;
    const float lam = lambda_of(p.lambda_dev, p.lambda_bf16, p.lambda);
    const int64_t second = (int64_t)p.B * p.H * p.Tq * VD;      // of the rests
    uint4 raw[PREP_ROWS][N];
#pragma unroll
    for (int i = 0; i < PREP_ROWS; ++i) {
        const int q = q0 + i * GROUPS;
        const int64_t o = b * p.s_o[0] + h * p.s_o[1] + q * p.s_o[2] + 8 * g;
        const int64_t d = b * p.s_do[0] + h * p.s_do[1] + q * p.s_do[2] + 8 * g;
        const int64_t row = ((int64_t)b * p.H + h) * p.Tq + q;
#pragma unroll
        for (int j = 0; j < N; ++j) raw[i][j] = make_uint4(0, 0, 0, 0);
        if (q < p.Tq) {
            raw[i][0] = *reinterpret_cast<const uint4*>(p.dout + d);
            raw[i][1] = *reinterpret_cast<const uint4*>(p.out + o);
            raw[i][2] = *reinterpret_cast<const uint4*>(p.out2 + o);
            if constexpr (RESTS) {
                raw[i][3] = *reinterpret_cast<const uint4*>(p.rests + row * VD + 8 * g);
                raw[i][4] = *reinterpret_cast<const uint4*>(p.rests + second + row * VD + 8 * g);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < PREP_ROWS; ++i) {
        const int q = q0 + i * GROUPS;
        uint64_t x[N][4];
#pragma unroll
        for (int j = 0; j < N; ++j) Vec<__nv_bfloat16>::unpack(raw[i][j], x[j]);
        uint64_t d0 = 0, d2 = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            d0 = f2_fma(x[0][e], x[1][e], d0);
            d2 = f2_fma(x[0][e], x[2][e], d2);
            if constexpr (RESTS) {
                d0 = f2_fma(x[0][e], x[3][e], d0);
                d2 = f2_fma(x[0][e], x[4][e], d2);
            }
        }
        const float s0 = group_sum<16>(f2_lo(d0) + f2_hi(d0)), s2 = group_sum<16>(f2_lo(d2) + f2_hi(d2));
        if (g != 0 || q >= p.Tq) continue;
        const int64_t row = ((int64_t)b * p.H + h) * p.Tq + q;
        const float2 lse = *reinterpret_cast<const float2*>(p.lse + row * 2);
        constexpr float LOG2E = 1.4426950408889634f;
        *reinterpret_cast<float4*>(p.stats + row * 4) = make_float4(-lse.x * LOG2E, -lse.y * LOG2E, -fmaf(lam, s2, s0), -s2);
    }
}

// ===========================================================================
// dq kernel
// ===========================================================================
namespace dq {

constexpr int BM = 128;            // query rows of an item (TMEM lanes)
constexpr int BN = 64;             // states of a tile
constexpr int KSTAGES_MAX = 4;
constexpr int VSTAGES = 3;
constexpr uint32_t Q_PANEL = BM * 128;             // 64 columns of 128 rows
constexpr uint32_t T_PANEL = BN * 128;             // and of 64
constexpr uint32_t V_BYTES = 2 * T_PANEL;

template <int HD>
struct Cfg {
    static constexpr bool TWO = HD == 64;          // two score buffers, dO in TMEM
    static constexpr int PANELS = HD / 64;
    static constexpr uint32_t Q_BYTES = PANELS * Q_PANEL;
    static constexpr uint32_t K_BYTES = PANELS * T_PANEL;
    static constexpr int KSTAGES = HD == 64 ? 4 : 3;
    static constexpr uint32_t K_STAGE = HD == 64 ? 2 * K_BYTES : K_BYTES;
    static constexpr uint32_t OFF_Q1 = 0, OFF_Q2 = Q_BYTES, OFF_DO = 2 * Q_BYTES;
    static constexpr uint32_t OFF_K = OFF_DO + 2 * Q_PANEL;
    static constexpr uint32_t OFF_V = OFF_K + KSTAGES * K_STAGE;
    static constexpr uint32_t OFF_BAR = OFF_V + VSTAGES * V_BYTES;
    // TMEM columns
    static constexpr uint32_t TM_DP = TWO ? 256 : 128, TM_DO = 320, TM_DS = 192;
    static constexpr uint32_t TM_DQ = TWO ? 384 : 256;
    static constexpr uint32_t IDESC_DQ = idesc_bf16_f32(BM, HD, 0, 1);     // dS (TMEM) x K (MN-major)
};
constexpr uint32_t IDESC_S = idesc_bf16_f32(BM, BN, 0, 0);                 // Q x K^T, dO x V^T

enum : int {
    Q_FULL, Q_EMPTY,
    K_FULL, K_EMPTY = K_FULL + KSTAGES_MAX, K_CLEAN = K_EMPTY + KSTAGES_MAX,
    V_FULL = K_CLEAN + KSTAGES_MAX, V_EMPTY = V_FULL + VSTAGES, V_CLEAN = V_EMPTY + VSTAGES,
    S_FULL = V_CLEAN + VSTAGES,     // [buffer]
    DS_FULL = S_FULL + 2,           // [buffer], 8 warps
    DS_FREE = DS_FULL + 2,          // one score buffer: the dQ product has read dS
    DP_FREE,                        // 8 warps: a tile's dP (one score buffer: and scores) in registers
    DQ_FULL, DQ_EMPTY,              // DQ_EMPTY: 8 warps
    DO_READY, DO_FREE,              // dO in TMEM: 4 warps; the item's last dP product done
    FINAL, ITEM_FULL, ITEM_EMPTY = ITEM_FULL + RING, NUM_BARS = ITEM_EMPTY + RING
};
constexpr int CHAINS = 2;           // of a row's sum of A_b dP
constexpr int CONSUMERS = 10;       // of the items: the MMA thread, 8 warps, the cleaning warp
constexpr uint32_t REL_TMEM = NUM_BARS * 8, REL_ABORT = REL_TMEM + 4, REL_RING = REL_ABORT + 4, REL_END = REL_RING + RING * 4;
template <int HD>
constexpr uint32_t smem_bytes() { return Cfg<HD>::OFF_BAR + REL_END + 1024; }
static_assert(smem_bytes<64>() <= 232448 && smem_bytes<128>() <= 232448, "shared memory budget");

struct Item {
    int b, h, qt, len, n;
    bool bad;
};
__device__ __forceinline__ Item decode(int idx, const CrossTcParams& p) {
    Item it;
    int head;
    locate(idx, p.B * p.H, p.nq128, p.group_q, &head, &it.qt);
    it.b = head / p.H;
    it.h = head - it.b * p.H;
    const CrossLen len = cross_len(p.lengths, it.b, p.Tk);
    it.len = len.n;
    it.bad = len.bad;
    it.n = (len.n + BN - 1) / BN;
    return it;
}

template <int HD>
__global__ void __launch_bounds__(NUM_THREADS, 1)
diffattn_cross_dq_kernel(const __grid_constant__ CUtensorMap tm_q1, const __grid_constant__ CUtensorMap tm_k1,
                         const __grid_constant__ CUtensorMap tm_q2, const __grid_constant__ CUtensorMap tm_k2,
                         const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                         const CrossTcParams p) {
    using C = Cfg<HD>;
    constexpr bool TWO = C::TWO;
    // The dK/dV kernel may take each SM as soon as this kernel's CTA there has finished; it
    // waits for the whole grid before it reads the rows' Dd.
    pdl_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + REL_TMEM);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_BAR + REL_ABORT);
    const uint32_t warp = warp_id(), lane = threadIdx.x & 31;
    const AbortState ab{abort_flag, p.status};
    const int total = p.B * p.H * p.nq128;
    const bool shared = HD == 128 || p.k_shared;
    const bool cleaned = p.lengths != nullptr;

    if (threadIdx.x == 0) {
        mbar_init(&bars[Q_FULL], 1);
        mbar_init(&bars[Q_EMPTY], 1);
        for (int s = 0; s < C::KSTAGES; ++s) {
            mbar_init(&bars[K_FULL + s], 1);
            mbar_init(&bars[K_EMPTY + s], 1);
            mbar_init(&bars[K_CLEAN + s], 1);
        }
        for (int s = 0; s < VSTAGES; ++s) {
            mbar_init(&bars[V_FULL + s], 1);
            mbar_init(&bars[V_EMPTY + s], 1);
            mbar_init(&bars[V_CLEAN + s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[S_FULL + i], 1);
            mbar_init(&bars[DS_FULL + i], 8);
        }
        mbar_init(&bars[DS_FREE], 1);
        mbar_init(&bars[DP_FREE], 8);
        mbar_init(&bars[DQ_FULL], 1);
        mbar_init(&bars[DQ_EMPTY], 8);
        mbar_init(&bars[DO_READY], 4);
        mbar_init(&bars[DO_FREE], 1);
        mbar_init(&bars[FINAL], 1);
        for (int i = 0; i < RING; ++i) {
            mbar_init(&bars[ITEM_FULL + i], 1);
            mbar_init(&bars[ITEM_EMPTY + i], CONSUMERS);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(tmem_ptr, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_ptr;
    const ItemRing<RING> ring{bars + ITEM_FULL, bars + ITEM_EMPTY, reinterpret_cast<volatile int*>(smem + C::OFF_BAR + REL_RING),
                              &ab};

    if (warp >= 8) {
        regs_dec<REGS_OTHER>();
        if (warp == 8) {
            // ------------------------------------------------------ producer
            if (elect_one()) {
                uint32_t kst = 0, kph = 0, vst = 0, vph = 0, qph = 0;
                uint32_t armed_q = 0, armed_k[KSTAGES_MAX] = {}, armed_v[VSTAGES] = {};
                bool ok = true;
                for (int k = 0; ok; ++k) {
                    int idx = (int)atomicAdd(p.sched, 1u);
                    if (idx >= total) idx = -1;
                    if (!(ok = ring.put(k, idx)) || idx < 0) break;
                    const Item it = decode(idx, p);
                    if (it.bad) atomicOr(p.status, kStatusIndex);
                    if (it.n == 0) continue;
                    const int hk = it.h / p.group;
                    if (armed_q > 0) {
                        if (!(ok = mbar_wait(&bars[Q_EMPTY], qph, ab))) break;
                        qph ^= 1;
                    }
                    mbar_arrive_expect_tx(&bars[Q_FULL], 2 * C::Q_BYTES + 2 * Q_PANEL);
#pragma unroll
                    for (int pn = 0; pn < C::PANELS; ++pn) {
                        tma_load_4d(smem + C::OFF_Q1 + pn * Q_PANEL, &tm_q1, &bars[Q_FULL], pn * 64, it.qt * BM, it.h, it.b);
                        tma_load_4d(smem + C::OFF_Q2 + pn * Q_PANEL, &tm_q2, &bars[Q_FULL], pn * 64, it.qt * BM, it.h, it.b);
                    }
#pragma unroll
                    for (int pn = 0; pn < 2; ++pn)
                        tma_load_4d(smem + C::OFF_DO + pn * Q_PANEL, &tm_do, &bars[Q_FULL], pn * 64, it.qt * BM, it.h, it.b);
                    ++armed_q;
                    for (int j = 0; j < it.n; ++j) {
                        if (!(ok = mbar_wait(&bars[K_EMPTY + kst], kph ^ 1, ab))) break;
                        // the MMA thread waits for the cleaning of some tiles only: no phase may be skipped
                        if (cleaned && !(ok = mbar_wait(&bars[K_CLEAN + kst], kph ^ 1, ab))) break;
                        uint8_t* kd = smem + C::OFF_K + kst * C::K_STAGE;
                        mbar_arrive_expect_tx(&bars[K_FULL + kst], (shared ? 1 : 2) * C::K_BYTES);
#pragma unroll
                        for (int pn = 0; pn < C::PANELS; ++pn) {
                            tma_load_4d(kd + pn * T_PANEL, &tm_k1, &bars[K_FULL + kst], pn * 64, j * BN, hk, it.b);
                            if (!shared)
                                tma_load_4d(kd + C::K_BYTES + pn * T_PANEL, &tm_k2, &bars[K_FULL + kst], pn * 64, j * BN, hk, it.b);
                        }
                        ++armed_k[kst];
                        if (++kst == C::KSTAGES) { kst = 0; kph ^= 1; }
                        if (!(ok = mbar_wait(&bars[V_EMPTY + vst], vph ^ 1, ab))) break;
                        if (cleaned && !(ok = mbar_wait(&bars[V_CLEAN + vst], vph ^ 1, ab))) break;
                        uint8_t* vd = smem + C::OFF_V + vst * V_BYTES;
                        mbar_arrive_expect_tx(&bars[V_FULL + vst], V_BYTES);
                        tma_load_4d(vd, &tm_v, &bars[V_FULL + vst], 0, j * BN, hk, it.b);
                        tma_load_4d(vd + T_PANEL, &tm_v, &bars[V_FULL + vst], 64, j * BN, hk, it.b);
                        ++armed_v[vst];
                        if (++vst == VSTAGES) { vst = 0; vph ^= 1; }
                    }
                }
                if (armed_q) mbar_wait_teardown(&bars[Q_FULL], (armed_q - 1) & 1, TEARDOWN_NS);
                for (int s = 0; s < C::KSTAGES; ++s)
                    if (armed_k[s]) mbar_wait_teardown(&bars[K_FULL + s], (armed_k[s] - 1) & 1, TEARDOWN_NS);
                for (int s = 0; s < VSTAGES; ++s)
                    if (armed_v[s]) mbar_wait_teardown(&bars[V_FULL + s], (armed_v[s] - 1) & 1, TEARDOWN_NS);
            }
            __syncwarp();
        } else if (warp == 9) {
            // ------------------------------------------------------ MMA issue
            if (elect_one()) {
                const uint64_t q1d = sdesc_sw128(smem_u32(smem + C::OFF_Q1), 16, 1024);
                const uint64_t q2d = sdesc_sw128(smem_u32(smem + C::OFF_Q2), 16, 1024);
                const uint64_t dod = sdesc_sw128(smem_u32(smem + C::OFF_DO), 16, 1024);
                const uint64_t kkd = sdesc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);         // K-major
                const uint64_t kmd = sdesc_sw128(smem_u32(smem + C::OFF_K), T_PANEL, 1024);    // MN-major
                const uint64_t vd = sdesc_sw128(smem_u32(smem + C::OFF_V), 16, 1024);
                const uint32_t k2off = shared ? 0 : C::K_BYTES >> 4;
                uint32_t kc = 0;            // key tiles of earlier items
                uint32_t vst = 0, vph = 0, qph = 0, dqph = 0, dsph = 0;
                int items = 0;              // items with states so far
                bool ok = true;
                // S_1 and S_2 of key tile kt into buffer buf, then dP into its one buffer
                auto issue_s = [&](uint32_t kt, int buf, bool first_tile, bool last_tile) -> bool {
                    const uint32_t ks = kt % C::KSTAGES, kp = (kt / C::KSTAGES) & 1u;
                    if (!mbar_wait(&bars[K_FULL + ks], kp, ab) || !mbar_wait(&bars[V_FULL + vst], vph, ab)) return false;
                    if (cleaned && last_tile && (!mbar_wait(&bars[K_CLEAN + ks], kp, ab) || !mbar_wait(&bars[V_CLEAN + vst], vph, ab)))
                        return false;
                    if (!TWO && kt > 0 && !mbar_wait(&bars[DP_FREE], (kt - 1) & 1u, ab)) return false;
                    tc_fence_after();
                    const uint32_t d = tmem_base + buf * 128;
                    const uint64_t k1 = kkd + ((ks * C::K_STAGE) >> 4);
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk) {
                        mma_ss(d, q1d + kstep(kk, Q_PANEL), k1 + kstep(kk, T_PANEL), IDESC_S, kk > 0);
                        mma_ss(d + 64, q2d + kstep(kk, Q_PANEL), k1 + k2off + kstep(kk, T_PANEL), IDESC_S, kk > 0);
                    }
                    if (TWO) {
                        if (kt > 0 && !mbar_wait(&bars[DP_FREE], (kt - 1) & 1u, ab)) return false;
                        if (first_tile && !mbar_wait(&bars[DO_READY], (uint32_t)items & 1u, ab)) return false;
                        tc_fence_after();
                    }
                    const uint64_t v0 = vd + ((vst * V_BYTES) >> 4);
#pragma unroll
                    for (int kk = 0; kk < VD / 16; ++kk) {
                        if constexpr (TWO)
                            mma_ts(tmem_base + C::TM_DP, tmem_base + C::TM_DO + kk * 8, v0 + kstep(kk, T_PANEL), IDESC_S, kk > 0);
                        else
                            mma_ss(tmem_base + C::TM_DP, dod + kstep(kk, Q_PANEL), v0 + kstep(kk, T_PANEL), IDESC_S, kk > 0);
                    }
                    mma_commit(&bars[S_FULL + buf]);
                    mma_commit(&bars[V_EMPTY + vst]);
                    if (TWO && last_tile) mma_commit(&bars[DO_FREE]);
                    if (last_tile) mma_commit(&bars[Q_EMPTY]);
                    if (++vst == VSTAGES) { vst = 0; vph ^= 1; }
                    return true;
                };
                for (int k = 0; ok; ++k) {
                    int idx = -1;
                    if (!(ok = ring.get_one(k, idx)) || idx < 0) break;
                    const int n = decode(idx, p).n;
                    if (n == 0) continue;
                    if (!(ok = mbar_wait(&bars[Q_FULL], qph, ab))) break;
                    qph ^= 1;
                    for (int t = 0; t < (TWO ? 2 : 1) && t < n && ok; ++t) ok = issue_s(kc + t, t, t == 0, t == n - 1);
                    if (!ok) break;
                    for (int j = 0; j < n; ++j) {
                        const uint32_t kt = kc + j;
                        if (!TWO && j + 1 < n && !(ok = issue_s(kt + 1, 0, false, j + 2 == n))) break;
                        // two buffers: tile j's is j & 1, and their phases go by the items' tiles
                        const int buf = TWO ? j & 1 : 0;
                        if (!(ok = mbar_wait(&bars[DS_FULL + buf], TWO ? (dsph >> buf) & 1u : kt & 1u, ab))) break;
                        dsph ^= 1u << buf;
                        if (j == 0 && items > 0) {
                            if (!(ok = mbar_wait(&bars[DQ_EMPTY], dqph, ab))) break;
                            dqph ^= 1;
                        }
                        tc_fence_after();
                        const uint32_t ks = kt % C::KSTAGES;
                        const uint64_t k1 = kmd + ((ks * C::K_STAGE) >> 4);
                        const uint32_t a1 = tmem_base + (TWO ? buf * 128 : C::TM_DS), a2 = a1 + (TWO ? 64 : 32);
#pragma unroll
                        for (int kk = 0; kk < BN / 16; ++kk) {
                            const uint32_t acc = (j > 0 || kk > 0) ? 1u : 0u;
                            mma_ts(tmem_base + C::TM_DQ, a1 + kk * 8, k1 + 128 * kk, C::IDESC_DQ, acc);
                            mma_ts(tmem_base + C::TM_DQ + HD, a2 + kk * 8, k1 + k2off + 128 * kk, C::IDESC_DQ, acc);
                        }
                        mma_commit(&bars[K_EMPTY + ks]);
                        if (!TWO) mma_commit(&bars[DS_FREE]);
                        if (TWO && j + 2 < n && !(ok = issue_s(kt + 2, buf, false, j + 3 == n))) break;
                    }
                    if (!ok) break;
                    mma_commit(&bars[DQ_FULL]);
                    kc += n;
                    ++items;
                }
                mma_commit(&bars[FINAL]);
                mbar_wait_teardown(&bars[FINAL], 0, TEARDOWN_NS);
            }
            __syncwarp();
        } else if (warp == 10) {
            // -------------------------------- rows behind a sequence's last state
            uint32_t kst = 0, kph = 0, vst = 0, vph = 0;
            int idx = -1;
            for (int k = 0; ring.get(k, idx) && idx >= 0; ++k) {
                if (!cleaned) continue;
                const Item it = decode(idx, p);
                bool ok = true;
                for (int j = 0; j < it.n; ++j) {
                    const int live = it.len - j * BN;
                    const bool dirty = live < BN && it.len < p.Tk;
                    // rows of 128 bytes in each panel: the swizzle stays inside a row
                    auto clean = [&](uint8_t* t, int panels) {
                        for (int pn = 0; pn < panels; ++pn)
                            for (int i = live * 8 + lane; i < BN * 8; i += 32)
                                reinterpret_cast<uint4*>(t + pn * T_PANEL)[i] = make_uint4(0, 0, 0, 0);
                    };
                    if (!(ok = mbar_wait_warp(&bars[K_FULL + kst], kph, ab))) break;
                    if (dirty) {
                        clean(smem + C::OFF_K + kst * C::K_STAGE, shared ? C::PANELS : 2 * C::PANELS);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive(&bars[K_CLEAN + kst]);
                    if (++kst == C::KSTAGES) { kst = 0; kph ^= 1; }
                    if (!(ok = mbar_wait_warp(&bars[V_FULL + vst], vph, ab))) break;
                    if (dirty) {
                        clean(smem + C::OFF_V + vst * V_BYTES, 2);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive(&bars[V_CLEAN + vst]);
                    if (++vst == VSTAGES) { vst = 0; vph ^= 1; }
                }
                if (!ok) break;
            }
        }
    } else {
        regs_inc<REGS_WORK>();
        // --------------------------------------- dS, the rows' Dd and the dQ epilogue
        const int br = warp >> 2;
        const uint32_t quad = warp & 3;
        const int row = quad * 32 + lane;
        const uint32_t lane_base = tmem_base + ((quad * 32u) << 16);
        const float lam = lambda_of(p.lambda_dev, p.lambda_bf16, p.lambda);
        const float coef = br ? -lam : 1.0f;
        const uint64_t sl2x2 = f2_pack(p.scale_log2, p.scale_log2), coef2 = f2_pack(coef, coef);
        uint32_t sph = 0, dqph = 0, cnt = 0;        // cnt: tiles so far
        int items = 0;
        bool ok = true;
        int idx = -1;
        for (int k = 0; (ok = ring.get(k, idx)) && idx >= 0; ++k) {
            const Item it = decode(idx, p);
            const int q = it.qt * BM + row;
            const bool live = q < p.Tq;
            const int64_t at = ((int64_t)it.b * p.H + it.h) * p.Tq + q;
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(br ? p.dq2 : p.dq1);
            if (dst) dst += at * HD;
            if (it.n == 0) {                    // no state: zeros (NaN for a bad length)
                const float fill = it.bad ? __int_as_float(0x7fc00000) : 0.f;
                if (live) p.stats[at * 4 + 2 + br] = fill;
                if (live && dst) {
                    const uint32_t w = pack_bf16x2(fill, fill);
#pragma unroll
                    for (int i = 0; i < HD / 8; ++i) *reinterpret_cast<uint4*>(dst + 8 * i) = make_uint4(w, w, w, w);
                }
                continue;
            }
            float nlse = 0.f, ndd = 0.f;        // -lse_b and -Dd_b of this row
            if (live) {
                const float4 st = *reinterpret_cast<const float4*>(p.stats + at * 4);
                nlse = br ? st.y : st.x;
                ndd = br ? st.w : st.z;
            }
            if (TWO && br == 0) {
                // the item's dO rows into TMEM, once they have landed and the last item's dP is done
                if (!(ok = mbar_wait_warp(&bars[Q_FULL], (uint32_t)items & 1u, ab))) break;
                if (items > 0 && !(ok = mbar_wait_warp(&bars[DO_FREE], (uint32_t)(items - 1) & 1u, ab))) break;
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // 64 columns: row `row` of the 128-byte swizzled half, chunk c at c ^ (row % 8)
                    const uint8_t* src = smem + C::OFF_DO + h * Q_PANEL + row * 128;
                    uint32_t w[32];
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const uint4 x = *reinterpret_cast<const uint4*>(src + ((c ^ (row & 7)) * 16));
                        w[4 * c] = x.x;
                        w[4 * c + 1] = x.y;
                        w[4 * c + 2] = x.z;
                        w[4 * c + 3] = x.w;
                    }
                    tmem_st32(lane_base + C::TM_DO + 32 * h, w);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[DO_READY]);
            }
            const uint64_t nlse2 = f2_pack(nlse, nlse);
            uint64_t cndd2 = f2_pack(coef * ndd, coef * ndd);
            uint64_t sum2[CHAINS] = {};         // of A_b dP
            for (int j = 0; j < it.n; ++j, ++cnt) {
                const int buf = TWO ? j & 1 : 0;
                const uint32_t tS = lane_base + buf * 128 + br * 64;
                if (!(ok = mbar_wait_warp(&bars[S_FULL + buf], (sph >> buf) & 1u, ab))) break;
                sph ^= 1u << buf;
                tc_fence_after();
                uint32_t s[64], dp[64];
                tmem_ld32(tS, &s[0]);
                tmem_ld32(tS + 32, &s[32]);
                tmem_ld32(lane_base + C::TM_DP, &dp[0]);
                tmem_ld32(lane_base + C::TM_DP + 32, &dp[32]);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[DP_FREE]);
                const int lim = it.len - j * BN;        // columns from it on are no states
                if (lim < BN) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) s[c] = c < lim ? s[c] : 0xff800000u;
                }
                if (it.n == 1) {                        // one tile: the row's exact Dd comes first
                    uint64_t t[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const uint64_t x = f2_fma(f2_from_bits(s[2 * c], s[2 * c + 1]), sl2x2, nlse2);
                        t[c & 3] = f2_fma(f2_pack(ex2_approx(f2_lo(x)), ex2_approx(f2_hi(x))), f2_from_bits(dp[2 * c], dp[2 * c + 1]),
                                          t[c & 3]);
                    }
                    const uint64_t sum = f2_add(f2_add(t[0], t[1]), f2_add(t[2], t[3]));
                    const float x = -coef * (f2_lo(sum) + f2_hi(sum));
                    cndd2 = f2_pack(x, x);
                }
                // one run of code for the compiler to order, in phases of independent operations in
                // place in the score registers: the exponents, the exponentials, the row's sum, dS_b =
                // coef A_b (dP - Dd_b).  (A branch between the phases, for the mask or the exact Dd,
                // took a fifth of the kernel's time.)
                uint32_t pk[32];
                constexpr int CH = 4;          // column pairs of a step
                auto exps = [&](int c0) {
#pragma unroll
                    for (int c = c0; c < c0 + CH; ++c) {
                        const uint64_t x = f2_fma(f2_from_bits(s[2 * c], s[2 * c + 1]), sl2x2, nlse2);
                        s[2 * c] = __float_as_uint(ex2_approx(f2_lo(x)));
                        s[2 * c + 1] = __float_as_uint(ex2_approx(f2_hi(x)));
                    }
                };
                exps(0);
#pragma unroll
                for (int c0 = 0; c0 < 32; c0 += CH) {
                    if (c0 + CH < 32) exps(c0 + CH);
#pragma unroll
                    for (int c = c0; c < c0 + CH; ++c) {
                        const uint64_t a = f2_from_bits(s[2 * c], s[2 * c + 1]), d = f2_from_bits(dp[2 * c], dp[2 * c + 1]);
                        sum2[c % CHAINS] = f2_fma(a, d, sum2[c % CHAINS]);
                        const uint64_t z = f2_mul(a, f2_fma(d, coef2, cndd2));
                        pk[c] = pack_bf16x2(f2_lo(z), f2_hi(z));
                    }
                }
                if (!TWO && cnt > 0 && !(ok = mbar_wait_warp(&bars[DS_FREE], (cnt - 1) & 1u, ab))) break;
                tmem_st32(TWO ? tS : lane_base + C::TM_DS + br * 32, pk);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[DS_FULL + buf]);
            }
            if (!ok) break;
            ++items;
            if (live) {
                uint64_t t = sum2[0];
#pragma unroll
                for (int i = 1; i < CHAINS; ++i) t = f2_add(t, sum2[i]);
                p.stats[at * 4 + 2 + br] = -(f2_lo(t) + f2_hi(t));
            }
            // dQ_b = scale * (dS_b K_b)
            if (!(ok = mbar_wait_warp(&bars[DQ_FULL], dqph, ab))) break;
            dqph ^= 1;
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < HD / 64; ++h) {
                uint32_t g[64];
                tmem_ld32(lane_base + C::TM_DQ + br * HD + h * 64, &g[0]);
                tmem_ld32(lane_base + C::TM_DQ + br * HD + h * 64 + 32, &g[32]);
                tmem_wait_ld();
                if (live && dst)
#pragma unroll
                    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(dst + h * 64 + 8 * i) = pack8(&g[8 * i], p.scale);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[DQ_EMPTY]);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem_base, TMEM_COLS);
}

}  // namespace dq

// ===========================================================================
// dkdv kernel
// ===========================================================================
namespace dkdv {

constexpr int BM = 128;            // states of an item (TMEM lanes)
constexpr int BN = 64;             // query rows of a tile
constexpr int QSTAGES_MAX = 4;
constexpr uint32_t K_PANEL = BM * 128;
constexpr uint32_t Q_PANEL = BN * 128;

template <int HD>
struct Cfg {
    static constexpr int PANELS = HD / 64;
    static constexpr uint32_t K_BYTES = PANELS * K_PANEL;
    static constexpr uint32_t Q_BYTES = PANELS * Q_PANEL;
    // rings of (Q1, Q2) and of dO: what fits (D = 128: a third stage of both does not)
    static constexpr int QSTAGES = HD == 64 ? 4 : 3, GSTAGES = HD == 64 ? 4 : 2;
    static constexpr uint32_t Q_STAGE = 2 * Q_BYTES, G_STAGE = 2 * Q_PANEL;
    // D = 128: one key tensor
    static constexpr uint32_t OFF_K1 = 0, OFF_K2 = HD == 64 ? K_BYTES : 0;
    static constexpr uint32_t OFF_V = HD == 64 ? 2 * K_BYTES : K_BYTES;
    static constexpr uint32_t OFF_QS = OFF_V + 2 * K_PANEL;
    // dS_2^T [128 states x 64 rows] as a K-major operand (W^T and dS_1^T go to TMEM)
    static constexpr uint32_t OFF_GS = OFF_QS + QSTAGES * Q_STAGE;
    static constexpr uint32_t OFF_PK = OFF_GS + GSTAGES * G_STAGE;
    // per elementwise warp: the statistics of its 32 query rows by quantity
    static constexpr uint32_t OFF_SCR = OFF_PK + BM * 128;
    static constexpr uint32_t OFF_BAR = OFF_SCR + 8 * 4 * 32 * 4;
    static constexpr uint32_t IDESC_DK = idesc_bf16_f32(BM, HD, 0, 1);     // dS^T x Q (MN-major)
};
// TMEM: S1^T, S2^T, dP^T; dV, dK1 (D = 128: dK), dK2; the operands W^T and dS1^T
constexpr uint32_t TM_S1 = 0, TM_S2 = 64, TM_DP = 128, TM_DV = 192, TM_DK1 = 320, TM_DK2 = 384, TM_W = 448, TM_DS1 = 480;
constexpr uint32_t IDESC_S = idesc_bf16_f32(BM, BN, 0, 0);         // K x Q^T, V x dO^T
constexpr uint32_t IDESC_DV = idesc_bf16_f32(BM, VD, 0, 1);        // W^T (TMEM) x dO (MN-major)

enum : int {
    KV_FULL, KV_EMPTY, Q_FULL, Q_EMPTY = Q_FULL + QSTAGES_MAX, G_FULL = Q_EMPTY + QSTAGES_MAX,
    G_EMPTY = G_FULL + QSTAGES_MAX, S_FULL = G_EMPTY + QSTAGES_MAX,
    S_FREE,                         // 8 warps: scores in registers
    DS_FULL,                        // 8 warps: operands written
    PK_FREE,                        // the operands have been read
    ACC_FULL, ACC_EMPTY,            // ACC_EMPTY: 8 warps
    FINAL, ITEM_FULL, ITEM_EMPTY = ITEM_FULL + RING, NUM_BARS = ITEM_EMPTY + RING
};
constexpr int CONSUMERS = 9;        // of the items: the MMA thread and 8 warps
constexpr uint32_t REL_TMEM = NUM_BARS * 8, REL_ABORT = REL_TMEM + 4, REL_RING = REL_ABORT + 4, REL_END = REL_RING + RING * 4;
template <int HD>
constexpr uint32_t smem_bytes() { return Cfg<HD>::OFF_BAR + REL_END + 1024; }
static_assert(smem_bytes<64>() <= 232448 && smem_bytes<128>() <= 232448, "shared memory budget");

struct Item {
    int b, hk, kt, len;
    int split;      // of the query tiles of all the group's heads,
    int t0, n;      // the split's first one and its tiles
    bool bad;
};
__device__ __forceinline__ Item decode(int idx, const CrossTcParams& p) {
    Item it;
    int head;
    locate(idx, p.B * p.Hk, p.nk128 * p.splits, p.group_k, &head, &it.kt);
    it.split = it.kt % p.splits;
    it.kt /= p.splits;
    it.b = head / p.Hk;
    it.hk = head - it.b * p.Hk;
    const CrossLen len = cross_len(p.lengths, it.b, p.Tk);
    it.len = len.n;
    it.bad = len.bad;
    const int64_t tiles = (int64_t)p.group * p.nq64;
    it.t0 = (int)(tiles * it.split / p.splits);
    it.n = it.kt * BM < len.n ? (int)(tiles * (it.split + 1) / p.splits) - it.t0 : 0;
    return it;
}

template <int HD>
__global__ void __launch_bounds__(NUM_THREADS, 1)
diffattn_cross_dkdv_kernel(const __grid_constant__ CUtensorMap tm_q1, const __grid_constant__ CUtensorMap tm_k1,
                           const __grid_constant__ CUtensorMap tm_q2, const __grid_constant__ CUtensorMap tm_k2,
                           const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                           const CrossTcParams p) {
    using C = Cfg<HD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + REL_TMEM);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_BAR + REL_ABORT);
    const uint32_t warp = warp_id(), lane = threadIdx.x & 31;
    const AbortState ab{abort_flag, p.status};
    const int total = p.B * p.Hk * p.nk128 * p.splits;
    const bool shared = HD == 128 || p.k_shared;

    if (threadIdx.x == 0) {
        mbar_init(&bars[KV_FULL], 1);
        mbar_init(&bars[KV_EMPTY], 1);
        for (int s = 0; s < C::QSTAGES; ++s) {
            mbar_init(&bars[Q_FULL + s], 1);
            mbar_init(&bars[Q_EMPTY + s], 1);
        }
        for (int s = 0; s < C::GSTAGES; ++s) {
            mbar_init(&bars[G_FULL + s], 1);
            mbar_init(&bars[G_EMPTY + s], 1);
        }
        mbar_init(&bars[S_FULL], 1);
        mbar_init(&bars[S_FREE], 8);
        mbar_init(&bars[DS_FULL], 8);
        mbar_init(&bars[PK_FREE], 1);
        mbar_init(&bars[ACC_FULL], 1);
        mbar_init(&bars[ACC_EMPTY], 8);
        mbar_init(&bars[FINAL], 1);
        for (int i = 0; i < RING; ++i) {
            mbar_init(&bars[ITEM_FULL + i], 1);
            mbar_init(&bars[ITEM_EMPTY + i], CONSUMERS);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(tmem_ptr, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_ptr;
    const ItemRing<RING> ring{bars + ITEM_FULL, bars + ITEM_EMPTY, reinterpret_cast<volatile int*>(smem + C::OFF_BAR + REL_RING),
                              &ab};

    if (warp >= 8) {
        regs_dec<REGS_OTHER>();
        if (warp == 8) {
            // ------------------------------------------------------ producer
            if (elect_one()) {
                uint32_t qs = 0, qph = 0, gs = 0, gph = 0, kvph = 0;
                uint32_t armed_kv = 0, armed_q[QSTAGES_MAX] = {}, armed_g[QSTAGES_MAX] = {};
                bool ok = true;
                for (int k = 0; ok; ++k) {
                    int idx = (int)atomicAdd(p.sched + 1, 1u);
                    if (idx >= total) idx = -1;
                    if (!(ok = ring.put(k, idx)) || idx < 0) break;
                    const Item it = decode(idx, p);
                    if (it.n == 0) continue;
                    if (armed_kv > 0) {
                        if (!(ok = mbar_wait(&bars[KV_EMPTY], kvph, ab))) break;
                        kvph ^= 1;
                    }
                    const int k0 = it.kt * BM;
                    mbar_arrive_expect_tx(&bars[KV_FULL], (shared ? 1 : 2) * C::K_BYTES + 2 * K_PANEL);
#pragma unroll
                    for (int pn = 0; pn < C::PANELS; ++pn) {
                        tma_load_4d(smem + C::OFF_K1 + pn * K_PANEL, &tm_k1, &bars[KV_FULL], pn * 64, k0, it.hk, it.b);
                        if (!shared)
                            tma_load_4d(smem + C::OFF_K2 + pn * K_PANEL, &tm_k2, &bars[KV_FULL], pn * 64, k0, it.hk, it.b);
                    }
#pragma unroll
                    for (int pn = 0; pn < 2; ++pn)
                        tma_load_4d(smem + C::OFF_V + pn * K_PANEL, &tm_v, &bars[KV_FULL], pn * 64, k0, it.hk, it.b);
                    ++armed_kv;
                    int h = it.hk * p.group + it.t0 / p.nq64, qt = it.t0 % p.nq64;
                    for (int t = 0; t < it.n && ok; ++t) {
                        if (!(ok = mbar_wait(&bars[Q_EMPTY + qs], qph ^ 1, ab))) break;
                        uint8_t* st = smem + C::OFF_QS + qs * C::Q_STAGE;
                        const int q0 = qt * BN;
                        mbar_arrive_expect_tx(&bars[Q_FULL + qs], C::Q_STAGE);
#pragma unroll
                        for (int pn = 0; pn < C::PANELS; ++pn) {
                            tma_load_4d(st + pn * Q_PANEL, &tm_q1, &bars[Q_FULL + qs], pn * 64, q0, h, it.b);
                            tma_load_4d(st + C::Q_BYTES + pn * Q_PANEL, &tm_q2, &bars[Q_FULL + qs], pn * 64, q0, h, it.b);
                        }
                        ++armed_q[qs];
                        if (++qs == C::QSTAGES) { qs = 0; qph ^= 1; }
                        if (!(ok = mbar_wait(&bars[G_EMPTY + gs], gph ^ 1, ab))) break;
                        mbar_arrive_expect_tx(&bars[G_FULL + gs], C::G_STAGE);
#pragma unroll
                        for (int pn = 0; pn < 2; ++pn)
                            tma_load_4d(smem + C::OFF_GS + gs * C::G_STAGE + pn * Q_PANEL, &tm_do, &bars[G_FULL + gs], pn * 64,
                                        q0, h, it.b);
                        ++armed_g[gs];
                        if (++gs == C::GSTAGES) { gs = 0; gph ^= 1; }
                        if (++qt == p.nq64) { qt = 0; ++h; }
                    }
                }
                if (armed_kv) mbar_wait_teardown(&bars[KV_FULL], (armed_kv - 1) & 1, TEARDOWN_NS);
                for (int s = 0; s < C::QSTAGES; ++s)
                    if (armed_q[s]) mbar_wait_teardown(&bars[Q_FULL + s], (armed_q[s] - 1) & 1, TEARDOWN_NS);
                for (int s = 0; s < C::GSTAGES; ++s)
                    if (armed_g[s]) mbar_wait_teardown(&bars[G_FULL + s], (armed_g[s] - 1) & 1, TEARDOWN_NS);
            }
            __syncwarp();
        } else if (warp == 9) {
            // ------------------------------------------------------ MMA issue
            if (elect_one()) {
                const uint64_t k1d = sdesc_sw128(smem_u32(smem + C::OFF_K1), 16, 1024);
                const uint64_t k2d = shared ? k1d : sdesc_sw128(smem_u32(smem + C::OFF_K2), 16, 1024);
                const uint64_t vd = sdesc_sw128(smem_u32(smem + C::OFF_V), 16, 1024);
                const uint64_t qk = sdesc_sw128(smem_u32(smem + C::OFF_QS), 16, 1024);         // K-major
                const uint64_t qm = sdesc_sw128(smem_u32(smem + C::OFF_QS), Q_PANEL, 1024);    // MN-major
                const uint64_t gk = sdesc_sw128(smem_u32(smem + C::OFF_GS), 16, 1024);
                const uint64_t gm = sdesc_sw128(smem_u32(smem + C::OFF_GS), Q_PANEL, 1024);
                const uint64_t pkd = sdesc_sw128(smem_u32(smem + C::OFF_PK), 16, 1024);        // K-major
                const uint32_t dk2 = tmem_base + (shared ? TM_DK1 : TM_DK2);
                uint32_t kvph = 0, accph = 0;
                uint32_t tiles = 0;       // query tiles whose scores were issued (whole launch)
                uint32_t done = 0;        // query tiles whose dV/dK products were issued
                bool ok = true, first = true;
                // S_1^T, S_2^T, dP^T of the next query tile; the previous tile's scores must have
                // been read out of TMEM
                auto issue_s = [&](bool last) -> bool {
                    const uint32_t qs = tiles % C::QSTAGES, gs = tiles % C::GSTAGES;
                    if (tiles > 0 && !mbar_wait(&bars[S_FREE], (tiles - 1) & 1u, ab)) return false;
                    if (!mbar_wait(&bars[Q_FULL + qs], (tiles / C::QSTAGES) & 1u, ab)) return false;
                    tc_fence_after();
                    const uint64_t sb = qk + ((qs * C::Q_STAGE) >> 4), gb = gk + ((gs * C::G_STAGE) >> 4);
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk) {
                        mma_ss(tmem_base + TM_S1, k1d + kstep(kk, K_PANEL), sb + kstep(kk, Q_PANEL), IDESC_S, kk > 0);
                        mma_ss(tmem_base + TM_S2, k2d + kstep(kk, K_PANEL), sb + (C::Q_BYTES >> 4) + kstep(kk, Q_PANEL), IDESC_S, kk > 0);
                    }
                    if (!mbar_wait(&bars[G_FULL + gs], (tiles / C::GSTAGES) & 1u, ab)) return false;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < VD / 16; ++kk)
                        mma_ss(tmem_base + TM_DP, vd + kstep(kk, K_PANEL), gb + kstep(kk, Q_PANEL), IDESC_S, kk > 0);
                    mma_commit(&bars[S_FULL]);
                    if (last) mma_commit(&bars[KV_EMPTY]);
                    ++tiles;
                    return true;
                };
                for (int k = 0; ok; ++k) {
                    int idx = -1;
                    if (!(ok = ring.get_one(k, idx)) || idx < 0) break;
                    const int n = decode(idx, p).n;
                    if (n == 0) continue;
                    if (!(ok = mbar_wait(&bars[KV_FULL], kvph, ab))) break;
                    kvph ^= 1;
                    if (!(ok = issue_s(n == 1))) break;
                    for (int t = 0; t < n; ++t) {
                        // the next tile's scores overlap this tile's elementwise work
                        if (t + 1 < n && !(ok = issue_s(t + 2 == n))) break;
                        if (!(ok = mbar_wait(&bars[DS_FULL], done & 1u, ab))) break;
                        if (t == 0 && !first) {
                            if (!(ok = mbar_wait(&bars[ACC_EMPTY], accph, ab))) break;
                            accph ^= 1;
                        }
                        tc_fence_after();
                        const uint32_t qs = done % C::QSTAGES, gs = done % C::GSTAGES;
                        const uint64_t sb = qm + ((qs * C::Q_STAGE) >> 4), gb = gm + ((gs * C::G_STAGE) >> 4);
#pragma unroll
                        for (int kk = 0; kk < BN / 16; ++kk) {
                            const uint32_t acc = (t > 0 || kk > 0) ? 1u : 0u;
                            mma_ts(tmem_base + TM_DV, tmem_base + TM_W + kk * 8, gb + 128 * kk, IDESC_DV, acc);
                            mma_ts(tmem_base + TM_DK1, tmem_base + TM_DS1 + kk * 8, sb + 128 * kk, C::IDESC_DK, acc);
                            mma_ss(dk2, pkd + 2 * kk, sb + (C::Q_BYTES >> 4) + 128 * kk, C::IDESC_DK, shared ? 1u : acc);
                        }
                        mma_commit(&bars[PK_FREE]);
                        mma_commit(&bars[Q_EMPTY + qs]);
                        mma_commit(&bars[G_EMPTY + gs]);
                        ++done;
                    }
                    if (!ok) break;
                    mma_commit(&bars[ACC_FULL]);
                    first = false;
                }
                mma_commit(&bars[FINAL]);
                mbar_wait_teardown(&bars[FINAL], 0, TEARDOWN_NS);
            }
            __syncwarp();
        }
    } else {
        regs_inc<REGS_WORK>();
        // ---------------------------------- dS^T, W^T and the dK/dV epilogue
        const int half = warp >> 2;          // query columns [32*half, 32*half + 32)
        const uint32_t quad = warp & 3;
        const int row = quad * 32 + lane;    // state within the tile
        const uint32_t lane_base = tmem_base + ((quad * 32u) << 16);
        const uint32_t c0 = 32 * half;
        const float lam = lambda_of(p.lambda_dev, p.lambda_bf16, p.lambda);
        // |lambda| goes into branch 2's exponents, -sign(lambda) into its Dd and the two sums: no
        // product with lambda is left (2 x 16 heads x 4096 rows over 4096 states: 946 -> 927 thousand cycles)
        const float log_lam = log2f(fabsf(lam)), nsgn = lam < 0.f ? 1.f : -1.f;
        const uint64_t sl2x2 = f2_pack(p.scale_log2, p.scale_log2), nsgn2 = f2_pack(nsgn, nsgn);
        uint32_t accph = 0, qc = 0;          // qc: query tiles consumed (whole launch)
        // the rows' exact Dd are the dQ kernel's
        pdl_wait();
        // Statistics of the warp's 32 query columns: lane l loads column l's one tile ahead (zeros
        // past Tq) and, when the tile starts, writes them to the warp's scratch by quantity, so
        // that the packed arithmetic reads those of four columns with one load.
        float* scr = reinterpret_cast<float*>(smem + C::OFF_SCR) + warp * 128;
        const float4* pl = reinterpret_cast<const float4*>(scr);
        auto stats_of = [&](int b, int h, int qt) -> float4 {
            const int q = qt * BN + (int)c0 + (int)lane;
            if (q >= p.Tq) return make_float4(0.f, 0.f, 0.f, 0.f);
            return *(reinterpret_cast<const float4*>(p.stats) + (((int64_t)b * p.H + h) * p.Tq + q));
        };
        bool ok = true;
        int idx = -1;
        for (int k = 0; (ok = ring.get(k, idx)) && idx >= 0; ++k) {
            const Item it = decode(idx, p);
            const int key = it.kt * BM + row;
            const int64_t krow = ((int64_t)it.b * p.Hk + it.hk) * p.Tk + key;
            __nv_bfloat16* dv = static_cast<__nv_bfloat16*>(p.dv) + krow * VD + 64 * half;
            __nv_bfloat16* dk = HD == 128 ? static_cast<__nv_bfloat16*>(p.dk1) + krow * HD + 64 * half
                                          : static_cast<__nv_bfloat16*>(half ? p.dk2 : p.dk1) + krow * HD;
            const bool has_dk = HD == 128 || half == 0 || !shared;
            if (p.splits == 1 && key >= it.len && key < p.Tk) {     // not the sequence's: zeros (NaN for a bad length)
                const uint32_t w = it.bad ? 0x7fc07fc0u : 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    *reinterpret_cast<uint4*>(dv + 8 * i) = make_uint4(w, w, w, w);
                    if (has_dk) *reinterpret_cast<uint4*>(dk + 8 * i) = make_uint4(w, w, w, w);
                }
            }
            if (it.n == 0) continue;
            int h = it.hk * p.group + it.t0 / p.nq64, qt = it.t0 % p.nq64;
            float4 nst = stats_of(it.b, h, qt);
            for (int t = 0; t < it.n; ++t, ++qc) {
                const int qbase = qt * BN + (int)c0;
                if (++qt == p.nq64) { qt = 0; ++h; }
                __syncwarp();               // the previous tile's reads of the scratch are done
                scr[lane] = nst.x;
                scr[32 + lane] = nst.y + log_lam;
                scr[64 + lane] = nst.z;
                scr[96 + lane] = nsgn * nst.w;
                __syncwarp();
                if (t + 1 < it.n) nst = stats_of(it.b, h, qt);
                if (!(ok = mbar_wait_warp(&bars[S_FULL], qc & 1u, ab))) break;
                tc_fence_after();
                uint32_t s1[32], s2[32], dp[32];
                tmem_ld32(lane_base + TM_S1 + c0, s1);
                tmem_ld32(lane_base + TM_S2 + c0, s2);
                tmem_ld32(lane_base + TM_DP + c0, dp);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[S_FREE]);
                uint32_t w1[16], w2[16], w3[16];
                const int qlim = p.Tq - qbase;              // columns from it on are no query rows
                if (qlim < 32) {
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        s1[c] = c < qlim ? s1[c] : 0xff800000u;
                        s2[c] = c < qlim ? s2[c] : 0xff800000u;
                    }
                }
                auto exps = [&](int c0) {
#pragma unroll
                    for (int c = c0; c < c0 + 4; c += 4) {
                        const float4 l1 = pl[c / 4], l2 = pl[8 + c / 4];
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            const int cc = c + 2 * hh;
                            const uint64_t L1 = hh ? f2_pack(l1.z, l1.w) : f2_pack(l1.x, l1.y);
                            const uint64_t L2 = hh ? f2_pack(l2.z, l2.w) : f2_pack(l2.x, l2.y);
                            const uint64_t x1 = f2_fma(f2_from_bits(s1[cc], s1[cc + 1]), sl2x2, L1);
                            const uint64_t x2 = f2_fma(f2_from_bits(s2[cc], s2[cc + 1]), sl2x2, L2);
                            s1[cc] = __float_as_uint(ex2_approx(f2_lo(x1)));
                            s1[cc + 1] = __float_as_uint(ex2_approx(f2_hi(x1)));
                            s2[cc] = __float_as_uint(ex2_approx(f2_lo(x2)));
                            s2[cc + 1] = __float_as_uint(ex2_approx(f2_hi(x2)));
                        }
                    }
                };
                exps(0);
#pragma unroll
                for (int b0 = 0; b0 < 32; b0 += 4) {
                    if (b0 + 4 < 32) exps(b0 + 4);
#pragma unroll
                    for (int c = b0; c < b0 + 4; c += 4) {
                        const float4 e1 = pl[16 + c / 4], e2 = pl[24 + c / 4];
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            const int cc = c + 2 * hh;
                            const uint64_t E1 = hh ? f2_pack(e1.z, e1.w) : f2_pack(e1.x, e1.y);
                            const uint64_t E2 = hh ? f2_pack(e2.z, e2.w) : f2_pack(e2.x, e2.y);
                            const uint64_t a1 = f2_from_bits(s1[cc], s1[cc + 1]);
                            const uint64_t a2 = f2_from_bits(s2[cc], s2[cc + 1]);      // |lambda| A_2
                            const uint64_t dp2 = f2_from_bits(dp[cc], dp[cc + 1]);
                            const uint64_t d1 = f2_mul(a1, f2_add(dp2, E1));
                            const uint64_t d2 = f2_mul(a2, f2_fma(dp2, nsgn2, E2));
                            const uint64_t w = f2_fma(a2, nsgn2, a1);
                            w1[cc / 2] = pack_bf16x2(f2_lo(d1), f2_hi(d1));
                            w2[cc / 2] = pack_bf16x2(f2_lo(d2), f2_hi(d2));
                            w3[cc / 2] = pack_bf16x2(f2_lo(w), f2_hi(w));
                        }
                    }
                }
                // the previous tile's dV/dK products must have read the operands
                if (qc > 0 && !(ok = mbar_wait_warp(&bars[PK_FREE], (qc - 1) & 1u, ab))) break;
                tmem_st16(lane_base + TM_W + 16 * half, w3);
                tmem_st16(lane_base + TM_DS1 + 16 * half, w1);
                // row `row`, queries [c0, c0 + 32) = 16-byte chunks 4*half .. 4*half + 3, swizzled by
                // the row's place in its 8-row group
                uint8_t* prow = smem + C::OFF_PK + row * 128;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint4*>(prow + (((4 * half + i) ^ (row & 7)) * 16)) =
                        make_uint4(w2[4 * i], w2[4 * i + 1], w2[4 * i + 2], w2[4 * i + 3]);
                fence_proxy_async_smem();
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[DS_FULL]);
            }
            if (!ok) break;
            // epilogue: warpgroup 0 writes dV columns 0-63, warpgroup 1 columns 64-127, and each a
            // part of dK: its branch's, or its half of the width, or (D = 64 with one key tensor)
            // warpgroup 0 all of it
            if (!(ok = mbar_wait_warp(&bars[ACC_FULL], accph, ab))) break;
            accph ^= 1;
            tc_fence_after();
            uint32_t gv[64], gk[64];
            tmem_ld32(lane_base + TM_DV + 64 * half, &gv[0]);
            tmem_ld32(lane_base + TM_DV + 64 * half + 32, &gv[32]);
            tmem_ld32(lane_base + TM_DK1 + 64 * half, &gk[0]);
            tmem_ld32(lane_base + TM_DK1 + 64 * half + 32, &gk[32]);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[ACC_EMPTY]);
            if (p.splits > 1) {         // partial sums, for the pass that joins them
                constexpr int W = VD + 2 * 64;
                float* part = p.parts + ((int64_t)it.split * p.B * p.Hk * p.Tk + krow) * W;
                if (key < it.len) {
#pragma unroll
                    for (int i = 0; i < 64; i += 4) {
                        *reinterpret_cast<uint4*>(part + 64 * half + i) = make_uint4(gv[i], gv[i + 1], gv[i + 2], gv[i + 3]);
                        *reinterpret_cast<uint4*>(part + VD + 64 * half + i) = make_uint4(gk[i], gk[i + 1], gk[i + 2], gk[i + 3]);
                    }
                }
            } else if (key < it.len) {
#pragma unroll
                for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(dv + 8 * i) = pack8(&gv[8 * i], 1.f);
                if (has_dk)
#pragma unroll
                    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(dk + 8 * i) = pack8(&gk[8 * i], p.scale);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem_base, TMEM_COLS);
}

// The splits' partial sums joined, in their order: a thread 8 of a state's 256 columns (dV, then
// dK_1 and dK_2 or the D = 128 columns of dK).
constexpr int JOIN_THREADS = 256;
template <int HD>
__global__ void __launch_bounds__(JOIN_THREADS)
cross_join_kernel(const CrossTcParams p) {
    pdl_wait();
    constexpr int W = VD + 2 * 64;
    const int64_t rows = (int64_t)p.B * p.Hk * p.Tk;
    const int64_t row = (int64_t)blockIdx.x * (JOIN_THREADS / 32) + threadIdx.x / 32;
    if (row >= rows) return;
    const int c = (threadIdx.x % 32) * 8;
    const int b = (int)(row / ((int64_t)p.Hk * p.Tk)), key = (int)(row % p.Tk);
    const CrossLen len = cross_len(p.lengths, b, p.Tk);
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.dv) + row * VD + c;
    if (c >= VD) {
        if (HD == 128) dst = static_cast<__nv_bfloat16*>(p.dk1) + row * HD + (c - VD);
        else if (c < VD + 64) dst = static_cast<__nv_bfloat16*>(p.dk1) + row * HD + (c - VD);
        else if (p.dk2) dst = static_cast<__nv_bfloat16*>(p.dk2) + row * HD + (c - VD - 64);
        else return;
    }
    if (key >= len.n) {
        const uint32_t w = len.bad ? 0x7fc07fc0u : 0u;
        *reinterpret_cast<uint4*>(dst) = make_uint4(w, w, w, w);
        return;
    }
    float x[8] = {};
    for (int s = 0; s < p.splits; ++s) {
        const float* part = p.parts + (s * rows + row) * W + c;
        const float4 a = *reinterpret_cast<const float4*>(part), d = *reinterpret_cast<const float4*>(part + 4);
        x[0] += a.x; x[1] += a.y; x[2] += a.z; x[3] += a.w;
        x[4] += d.x; x[5] += d.y; x[6] += d.z; x[7] += d.w;
    }
    const float f = c >= VD ? p.scale : 1.f;
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0] * f, x[1] * f), pack_bf16x2(x[2] * f, x[3] * f),
                                                pack_bf16x2(x[4] * f, x[5] * f), pack_bf16x2(x[6] * f, x[7] * f));
}

}  // namespace dkdv

template <int HD>
int launch(const CUtensorMap* maps, const CrossTcParams& p, int num_sms, cudaStream_t stream) {
    if (cudaFuncSetAttribute(dq::diffattn_cross_dq_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)dq::smem_bytes<HD>()) != cudaSuccess ||
        cudaFuncSetAttribute(dkdv::diffattn_cross_dkdv_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)dkdv::smem_bytes<HD>()) != cudaSuccess)
        return -1;
    const int dq_items = p.B * p.H * p.nq128, kv_items = p.B * p.Hk * p.nk128 * p.splits;
    constexpr int PER = PREP_THREADS / 16 * PREP_ROWS;
    const auto prep = p.rests ? cross_prep_kernel<true> : cross_prep_kernel<false>;
    prep<<<dim3((p.Tq + PER - 1) / PER, p.B * p.H), PREP_THREADS, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return -1;
    dq::diffattn_cross_dq_kernel<HD><<<dq_items < num_sms ? dq_items : num_sms, NUM_THREADS, dq::smem_bytes<HD>(), stream>>>(
        maps[0], maps[1], maps[2], maps[3], maps[4], maps[5], p);
    if (cudaGetLastError() != cudaSuccess) return -1;
    if (!p.dv) return 0;
    // One CTA of either kernel takes a whole SM's registers, so they never share one.
    if (pdl_launch(dkdv::diffattn_cross_dkdv_kernel<HD>, dim3(kv_items < num_sms ? kv_items : num_sms), NUM_THREADS,
                   dkdv::smem_bytes<HD>(), stream, maps[6], maps[7], maps[8], maps[9], maps[10], maps[11], p) != 0)
        return -1;
    if (p.splits == 1) return 0;
    constexpr int ROWS = dkdv::JOIN_THREADS / 32;
    const int64_t rows = (int64_t)p.B * p.Hk * p.Tk;
    return pdl_launch(dkdv::cross_join_kernel<HD>, dim3((unsigned)((rows + ROWS - 1) / ROWS)), dkdv::JOIN_THREADS, 0, stream, p);
}

}  // namespace xbwd

// Items of all of a head's query rows keep 152 SMs busy when there are many; few leave the last
// round of items half empty.  The estimate, in tiles of 64 rows (about 0.9 us): the rounds of
// items, 4 tiles for an item's start and end, and the partial sums' way to HBM and back.
int cross_bwd_splits(int64_t B, int64_t Hk, int64_t group, int64_t Tq, int64_t Tk) {
    constexpr double SMS = 152;
    const double items = (double)B * Hk * ((Tk + 127) / 128), tiles = (double)group * ((Tq + 63) / 64);
    int best = 1;
    double least = 0;
    for (int s = 1; s <= 8; ++s) {
        if (s > 1 && tiles < 4 * s) break;
        const double join = s > 1 ? (double)s * B * Hk * Tk * 256 * 4 * 2 / 4.5e12 / 0.9e-6 + 3 : 0;
        const double t = std::ceil(items * s / SMS) * (std::ceil(tiles / s) + 4) + join;
        if (s == 1 || t < least) {
            least = t;
            best = s;
        }
    }
    return best;
}

int launch_cross_bwd_tc(const CUtensorMap* maps, const CrossTcParams& p, int head_dim, int num_sms, cudaStream_t stream) {
    if (head_dim == 64) return xbwd::launch<64>(maps, p, num_sms, stream);
    if (head_dim == 128 && p.k_shared) return xbwd::launch<128>(maps, p, num_sms, stream);
    return -1;
}

}  // namespace diffattn
