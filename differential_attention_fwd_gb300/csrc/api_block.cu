// api_block.cu -- the C ABI of the operators of a cross-attention block: argument checks
// and launches.
#include "block.h"
#include "diffattn.h"
#include "kernels.h"

#include <cmath>
#include <cstdint>

namespace diffattn {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool nonneg(const int64_t s[3]) { return s[0] >= 0 && s[1] >= 0 && s[2] >= 0; }
// Rows of sizes n that start on 16-byte boundaries (a dimension of one is not stepped).
bool rows16(const void* p, const int64_t n[3], const int64_t s[3], int64_t es) {
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && s[i] * es % 16 != 0) return false;
    return aligned16(p);
}
// Whether rows of these sizes and strides have a place each (a stride of 0 gives many one).
bool apart(const int64_t n[3], const int64_t s[3]) {
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && s[i] == 0) return false;
    return true;
}
void copy3(int64_t dst[3], const int64_t src[3]) {
    for (int i = 0; i < 3; ++i) dst[i] = src[i];
}

int check_norm(const diffattn_norm_desc* d) {
    if (!d || d->B < 1 || d->H < 1 || d->T < 1 || d->C < 1 || d->C > 256 ||
        (d->dtype != DIFFATTN_BF16 && d->dtype != DIFFATTN_F32) ||
        (d->norm != DIFFATTN_NORM_RMS && d->norm != DIFFATTN_NORM_GROUP) || !std::isfinite(d->eps) || d->eps <= 0.f ||
        !std::isfinite(d->out_scale) || !nonneg(d->x_stride) || !nonneg(d->y_stride) || !nonneg(d->dy_stride) ||
        !nonneg(d->dx_stride))
        return DIFFATTN_ERR_INVALID;
    // token indices, and those of a last block's rows past them, in 31 bits
    constexpr int64_t kMaxTokens = 1 << 30;
    if (d->H > 65535 || d->B > kMaxTokens || d->T > kMaxTokens || d->B * d->T > kMaxTokens) return DIFFATTN_ERR_UNSUPPORTED;
    return DIFFATTN_OK;
}

void fill_norm(HeadNormParams* p, const diffattn_norm_desc& d, const void* x, const float* w, const float* b) {
    p->B = (int)d.B;
    p->H = (int)d.H;
    p->T = (int)d.T;
    p->C = (int)d.C;
    p->tokens = (int)(d.B * d.T);
    p->by_T.set((uint32_t)d.T);
    p->bf16 = d.dtype == DIFFATTN_BF16;
    p->group = d.norm == DIFFATTN_NORM_GROUP;
    p->eps = d.eps;
    p->scale = d.out_scale;
    p->inv_C = 1.0f / (float)d.C;
    p->x = x;
    p->w = w;
    p->b = b;
    copy3(p->sx, d.x_stride);
    const int64_t n[3] = {d.B, d.H, d.T}, es = p->bf16 ? 2 : 4;
    p->fast = d.C * es % 16 == 0 && rows16(x, n, d.x_stride, es) && (!w || aligned16(w)) && (!b || aligned16(b));
}

// ---------------------------------------------------------------------------
// attention over an encoder's states
// ---------------------------------------------------------------------------
int64_t group_of(const diffattn_cross_desc& d) { return d.kv_group > 1 ? d.kv_group : 1; }
int64_t width_of(const diffattn_cross_desc& d) { return d.Dv == 0 ? 2 * d.D : d.Dv; }

int check_cross(const diffattn_cross_desc* d) {
    if (!d || d->B < 1 || d->H < 1 || d->Tq < 1 || d->Tk < 1 || d->D < 1 || d->D > 128 || d->Dv < 0 ||
        (d->dtype != DIFFATTN_BF16 && d->dtype != DIFFATTN_F32) || d->kv_group < 0 ||
        (d->lambda_dtype != DIFFATTN_BF16 && d->lambda_dtype != DIFFATTN_F32) || d->reserved != 0)
        return DIFFATTN_ERR_INVALID;
    if (width_of(*d) > 256 || d->H % group_of(*d) != 0 || !nonneg(d->q1_stride) || !nonneg(d->k1_stride) ||
        !nonneg(d->q2_stride) || !nonneg(d->k2_stride) || !nonneg(d->v_stride) || !nonneg(d->o_stride) ||
        !nonneg(d->dout_stride))
        return DIFFATTN_ERR_INVALID;
    // rows, states, and the tiles of 32 of either, in 31 bits
    const double tiles = (double)d->B * d->H * ((double)(d->Tq > d->Tk ? d->Tq : d->Tk) / 32 + 2);
    if (d->Tq > INT32_MAX / 2 || d->Tk > INT32_MAX / 2 || d->B > INT32_MAX || d->H > INT32_MAX || tiles > INT32_MAX)
        return DIFFATTN_ERR_UNSUPPORTED;
    return DIFFATTN_OK;
}

bool same3(const int64_t a[3], const int64_t b[3]) { return a[0] == b[0] && a[1] == b[1] && a[2] == b[2]; }

void fill_cross(CrossParams* p, const diffattn_cross_desc& d, const void* q1, const void* k1, const void* q2, const void* k2,
                const void* v, const int32_t* lengths, float lambda, const void* lambda_dev) {
    p->B = (int)d.B;
    p->H = (int)d.H;
    p->group = (int)group_of(d);
    p->Hk = p->H / p->group;
    p->Tq = (int)d.Tq;
    p->Tk = (int)d.Tk;
    p->D = (int)d.D;
    p->Dv = (int)width_of(d);
    p->bf16 = d.dtype == DIFFATTN_BF16;
    p->k_shared = k1 == k2 && same3(d.k1_stride, d.k2_stride);
    p->scale = (float)(1.0 / std::sqrt((double)d.D));
    p->lambda = lambda;
    p->lambda_dev = static_cast<const float*>(lambda_dev);
    p->lambda_bf16 = d.lambda_dtype == DIFFATTN_BF16;
    p->lengths = lengths;
    p->q1 = q1;
    p->k1 = k1;
    p->q2 = q2;
    p->k2 = k2;
    p->v = v;
    copy3(p->s_q1, d.q1_stride);
    copy3(p->s_k1, d.k1_stride);
    copy3(p->s_q2, d.q2_stride);
    copy3(p->s_k2, d.k2_stride);
    copy3(p->s_v, d.v_stride);
    copy3(p->s_o, d.o_stride);
    copy3(p->s_do, d.dout_stride);
}

bool workspace_ok(const void* workspace, size_t bytes, size_t need) {
    return need == 0 || (workspace && aligned16(workspace) && bytes >= need);
}

int64_t cross_rows(const diffattn_cross_desc& d) { return d.B * d.H * d.Tq; }

// Strides that TMA takes, of the dimensions that are stepped.
bool tma_rows(const void* p, const int64_t n[3], const int64_t s[3]) {
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (s[i] % 8 != 0 || s[i] <= 0 || s[i] >= (int64_t(1) << 38))) return false;
    return aligned16(p);
}

// Whether the tensor cores take the shape: bf16, value width 128, Q/K width 64 or 128.
bool tc_shape(const diffattn_cross_desc& d) {
    return d.dtype == DIFFATTN_BF16 && width_of(d) == 128 && (d.D == 64 || d.D == 128);
}
// The longest sequence that they take: the dK/dV kernel's blocks may wait for as long as the dQ
// kernel walks one (0.8 us for 64 states), and a wait ends after 2 s.
constexpr int64_t kMaxTiledStates = 1 << 26;
// And the call's layout.
bool tc_inputs(const diffattn_cross_desc& d, const void* q1, const void* k1, const void* q2, const void* k2, const void* v) {
    const int64_t nq[3] = {d.B, d.H, d.Tq}, nk[3] = {d.B, d.H / group_of(d), d.Tk};
    return tc_shape(d) && d.Tk <= kMaxTiledStates && tma_rows(q1, nq, d.q1_stride) && tma_rows(q2, nq, d.q2_stride) && tma_rows(k1, nk, d.k1_stride) &&
           tma_rows(k2, nk, d.k2_stride) && tma_rows(v, nk, d.v_stride);
}

// A short head's rows, a power of two and at least 8 (what a swizzled tile's rows repeat in), and
// how many heads of a group the tensor-core forward's items take together: as few as leave one
// item an SM, if they fit into 128 rows.  16 sequences of 1500 states, 32 rows of 16 over 4 heads:
// 24 us with two heads an item, 43 with one.
int short_rows_log2(int64_t Tq) {
    int s = 3;
    while (s < 7 && (int64_t(1) << s) < Tq) ++s;
    return s;
}
int packed_heads(int64_t B, int64_t H, int64_t group, int64_t Tq) {
    int pack = 1;
    for (int64_t n = 2; n <= group && (n << short_rows_log2(Tq)) <= 128 && Tq <= 64 && B * H / pack > 152; ++n)
        if (group % n == 0) pack = (int)n;
    return pack;
}

// What the tensor-core forward takes for sequences of Tk states, about, in us.
double whole_us(int64_t B, int64_t H, int64_t group, int64_t Tq, int64_t Tk, int64_t D) {
    const double items = (double)B * H / packed_heads(B, H, group, Tq) * ((Tq + 127) / 128), tiles = (double)((Tk + 63) / 64);
    return 5 + std::ceil(items / 152) * tiles * (D == 64 ? 0.70 : 0.96);
}

// Whether the kernels of the paged cache take a serving call.  They divide the states of all
// sequences evenly over the SMs and join the parts in a second launch, where the forward's
// blocks each walk a whole sequence for 128 rows.  By estimates, in us, for lengths of Tk, from
// what either measured (bf16; the forward, then the split):
//   one sequence, 16 heads of 64, 32 rows:   77 states 6.3, 15.0; 1500 22.0, 19.3; 6000 71, 28
//   16 sequences, the same:                  77 states 11.1, 21.7; 1500 47, 69; 6000 158, 175
//   16 sequences, 16 heads, one row:         1500 states 46.3, 44.3; of two thirds on average 36.0, 38.1
//   16 sequences, 16 over 4 heads, one row:  77 states 8.0, 14.1; 1500 24.2, 23.3; 6000 74, 48
//   the same, 32 rows:                       77 states 8.0, 20.9; 1500 24.9, 41; 6000 75, 69
//   the V2 head, 16 over 8 heads, 64 rows:   77 states 6.7, 16.7; 1500 25.7, 28.7; 6000 95, 33
//   16 sequences, the same:                  1500 states 33.3, 56; 6000 106, 115
//   4 sequences, 64 over 4 heads, 4 rows:    3000 states 40.3, 25.7
// Up to 16 rows a key/value head the split is bound by HBM, beyond by its products and starts.
bool wants_split(const diffattn_cross_desc& d) {
    if (!cross_paged_ok(d)) return false;
    constexpr double SMS = 152;
    const int64_t rows = group_of(d) * d.Tq, Hk = d.H / group_of(d);
    const double tiles = (double)((d.Tk + 63) / 64);
    if (!tc_shape(d)) {
        // CUDA cores: blocks of 32 rows of a head (about 1.5 us a tile of 32 states) against shares
        // of all tiles, 4 to an SM (3 us for 16 rows)
        const double items = (double)d.B * d.H * ((d.Tq + 31) / 32), units = (double)d.B * Hk * ((rows + 15) / 16);
        const double whole = 6 + std::ceil(items / (2 * SMS)) * 2 * tiles * 1.5;
        return 20 + units * 2 * tiles / (4 * SMS) * 3 < whole;
    }
    const double bytes = (double)d.B * Hk * d.Tk * 512;     // of a state's keys (the V2 head's: one tensor) and value
    const double least = 5 + bytes / 5.0e6, by_tiles = whole_us(d.B, d.H, group_of(d), d.Tq, d.Tk, d.D);
    const double whole = by_tiles > least ? by_tiles : least;
    if (rows <= 16) return 12.5 + bytes / 5.6e6 * (rows > 8 ? 1.5 : 1.0) < whole;
    const int64_t head_rows = (d.Tq + 7) / 8 * 8;
    const double chunks = d.Tq <= 128 ? std::ceil(group_of(d) / std::floor(128.0 / head_rows))
                                      : (double)group_of(d) * ((d.Tq + 127) / 128);
    const double units = d.B * Hk * chunks;
    return (d.D == 64 ? 18 : 26) + units * tiles / SMS * 1.2 + units * 0.08 < whole;
}

// A few rows, of a shape for the tensor cores but in a layout that TMA does not take, are split
// on the CUDA cores: 16 sequences of 1500 states, one row of 4 heads, all reading one sequence's
// states: 33 us, where copies for the tensor cores take 64 (and for 4 rows each 70, against 77).
bool few_rows(const diffattn_cross_desc& d) { return tc_shape(d) && group_of(d) * d.Tq <= 4 && cross_paged_ok(d); }

// Heads that the persistent kernels work on at a time, each streaming `bytes`: about 48 MiB of
// them (they then share the L2), with an item of `tiles` for every SM.
int heads_at_once(int64_t heads, int64_t bytes, int64_t tiles, int sms) {
    int64_t g = (48ll << 20) / (bytes > 0 ? bytes : 1);
    const int64_t least = (sms + tiles - 1) / tiles;
    if (g < least) g = least;
    return (int)(g < 1 ? 1 : g > heads ? heads : g);
}

// Maps of Q1, K1, Q2, K2, V and a tensor of O's shape, with boxes of 64 columns and so many rows.
int cross_maps(CUtensorMap* m, const CrossParams& p, const void* o, const int64_t so[3], int q_rows, int k_rows, int o_rows) {
    const int64_t qd[4] = {p.D, p.Tq, p.H, p.B}, kd[4] = {p.D, p.Tk, p.Hk, p.B};
    const int64_t vd[4] = {p.Dv, p.Tk, p.Hk, p.B}, od[4] = {p.Dv, p.Tq, p.H, p.B};
    return encode_map_4d(&m[0], p.q1, qd, p.s_q1, 64, q_rows) == DIFFATTN_OK &&
                   encode_map_4d(&m[1], p.k1, kd, p.s_k1, 64, k_rows) == DIFFATTN_OK &&
                   encode_map_4d(&m[2], p.q2, qd, p.s_q2, 64, q_rows) == DIFFATTN_OK &&
                   encode_map_4d(&m[3], p.k2, kd, p.s_k2, 64, k_rows) == DIFFATTN_OK &&
                   encode_map_4d(&m[4], p.v, vd, p.s_v, 64, k_rows) == DIFFATTN_OK &&
                   encode_map_4d(&m[5], o, od, so, 64, o_rows) == DIFFATTN_OK
               ? DIFFATTN_OK
               : DIFFATTN_ERR_CUDA;
}

// The forward on the tensor cores; `counter`: 64 bytes of workspace.
int forward_tc(const CrossParams& c, int sms, void* counter, cudaStream_t stream) {
    TcParams p{};
    p.pack = packed_heads(c.B, c.H, c.group, c.Tq);
    p.item_heads = c.H / p.pack;
    p.pack_shift = p.pack > 1 ? short_rows_log2(c.Tq) : 7;
    CUtensorMap maps[6];
    const int rows = 1 << p.pack_shift;
    if (cross_maps(maps, c, c.out, c.s_o, rows, 64, rows < 32 ? rows : 32) != DIFFATTN_OK) return DIFFATTN_ERR_CUDA;
    p.B = c.B;
    p.H = c.H;
    p.T = c.Tq;
    p.Tk = c.Tk;
    p.nq = (c.Tq + 127) / 128;
    p.nk = (c.Tk + 63) / 64;
    p.total_items = c.B * p.item_heads * p.nq;
    p.group = heads_at_once((int64_t)c.B * p.item_heads, (int64_t)c.Tk * ((c.k_shared ? 1 : 2) * c.D + c.Dv) * 2, p.nq, sms);
    p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)c.D));
    p.lambda = c.lambda;
    p.lambda_dev = c.lambda_dev;
    p.lambda_bf16 = c.lambda_bf16;
    p.out = static_cast<__nv_bfloat16*>(c.out);
    p.o_sB = c.s_o[0];
    p.o_sH = c.s_o[1];
    p.o_sT = c.s_o[2];
    p.status = c.status;
    p.norm = c.norm;
    p.norm_eps = c.norm_eps;
    p.norm_weight = c.norm_weight;
    p.norm_bias = c.norm_bias;
    p.out_scale = c.out_scale;
    p.kv_group = c.group;
    p.k_shared = c.k_shared;
    p.out2 = static_cast<__nv_bfloat16*>(c.out2);
    p.lse = c.lse;
    p.rests = static_cast<__nv_bfloat16*>(c.rests);
    p.lengths = c.lengths;
    const int grid = p.total_items < sms ? p.total_items : sms;
    // Long calls claim their items from a counter, since sequences differ in length.  To zero it
    // takes 7 us between the stream's kernels, so short ones deal them out.
    if (p.total_items > sms && whole_us(c.B, c.H, c.group, c.Tq, c.Tk, c.D) > 60) {
        p.sched = static_cast<uint32_t*>(counter);
        if (cudaMemsetAsync(counter, 0, 64, stream) != cudaSuccess) return DIFFATTN_ERR_CUDA;
    }
    return launch_cross_tc(maps, p, c.D, grid, stream) == 0 ? DIFFATTN_OK : DIFFATTN_ERR_CUDA;
}

// The backward on the tensor cores; `parts`: workspace for the splits' partial sums.
int backward_tc(const CrossParams& c, int sms, float* parts, cudaStream_t stream) {
    CUtensorMap maps[12];
    if (cross_maps(maps, c, c.dout, c.s_do, 128, 64, 128) != DIFFATTN_OK ||
        cross_maps(maps + 6, c, c.dout, c.s_do, 64, 128, 64) != DIFFATTN_OK)
        return DIFFATTN_ERR_CUDA;
    CrossTcParams p{};
    p.B = c.B;
    p.H = c.H;
    p.Hk = c.Hk;
    p.group = c.group;
    p.Tq = c.Tq;
    p.Tk = c.Tk;
    p.nq128 = (c.Tq + 127) / 128;
    p.nq64 = (c.Tq + 63) / 64;
    p.nk128 = (c.Tk + 127) / 128;
    p.k_shared = c.k_shared;
    p.group_q = heads_at_once((int64_t)c.B * c.H, (int64_t)c.Tk * ((c.k_shared ? 1 : 2) * c.D + c.Dv) * 2, p.nq128, sms);
    p.group_k = heads_at_once((int64_t)c.B * c.Hk, (int64_t)c.Tq * c.group * (2 * c.D + c.Dv) * 2, p.nk128, sms);
    p.scale = c.scale;
    p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)c.D));
    p.lambda = c.lambda;
    p.lambda_dev = c.lambda_dev;
    p.lambda_bf16 = c.lambda_bf16;
    p.lengths = c.lengths;
    p.status = c.status;
    p.sched = c.counters;
    p.out = static_cast<const __nv_bfloat16*>(c.out);
    p.out2 = static_cast<const __nv_bfloat16*>(c.out2);
    p.rests = static_cast<const __nv_bfloat16*>(c.rests);
    p.dout = static_cast<const __nv_bfloat16*>(c.dout);
    copy3(p.s_o, c.s_o);
    copy3(p.s_do, c.s_do);
    p.lse = c.lse;
    p.stats = c.stats;
    p.splits = cross_bwd_splits(c.B, c.Hk, c.group, c.Tq, c.Tk);
    p.parts = parts;
    p.dq1 = c.dq1;
    p.dq2 = c.dq2;
    p.dk1 = c.dk1;
    p.dk2 = c.dk2;
    p.dv = c.dv;
    return launch_cross_bwd_tc(maps, p, c.D, sms, stream) == 0 ? DIFFATTN_OK : DIFFATTN_ERR_CUDA;
}

}  // namespace
}  // namespace diffattn

using namespace diffattn;

extern "C" {

size_t diffattn_cross_workspace_bytes(const diffattn_cross_desc* desc) {
    if (check_cross(desc) != DIFFATTN_OK) return 0;
    const size_t paged = wants_split(*desc) || few_rows(*desc) ? cross_paged_bytes(*desc) : 0;
    return paged > 64 ? paged : 64;     // or an item counter
}

size_t diffattn_cross_bwd_workspace_bytes(const diffattn_cross_desc* desc) {
    if (check_cross(desc) != DIFFATTN_OK) return 0;
    // the rows' statistics, partial sums of dlambda and item counters; the tensor cores' partial
    // sums of dK and dV
    size_t floats = cross_rows(*desc) * 4 + kLambdaBlocks + 4;
    if (tc_shape(*desc)) {
        const int64_t Hk = desc->H / group_of(*desc);
        const int splits = cross_bwd_splits(desc->B, Hk, group_of(*desc), desc->Tq, desc->Tk);
        if (splits > 1) floats += (size_t)splits * desc->B * Hk * desc->Tk * 256;
    }
    return floats * sizeof(float);
}

int diffattn_cross_fwd(const diffattn_cross_desc* desc, const void* q1, const void* k1, const void* q2, const void* k2,
                       const void* v, const int32_t* kv_lengths, float lambda, const void* lambda_dev,
                       const diffattn_epilogue* epi, void* out, void* out2, float* lse, void* workspace,
                       size_t workspace_bytes, diffattn_stream_t stream) {
    return diffattn_cross_fwd_ex(desc, q1, k1, q2, k2, v, kv_lengths, lambda, lambda_dev, epi, out, out2, lse, nullptr,
                                 workspace, workspace_bytes, stream);
}

int diffattn_cross_fwd_ex(const diffattn_cross_desc* desc, const void* q1, const void* k1, const void* q2, const void* k2,
                          const void* v, const int32_t* kv_lengths, float lambda, const void* lambda_dev,
                          const diffattn_epilogue* epi, void* out, void* out2, float* lse, void* rests, void* workspace,
                          size_t workspace_bytes, diffattn_stream_t stream) {
    int rc = check_cross(desc);
    if (rc != DIFFATTN_OK) return rc;
    const diffattn_cross_desc& d = *desc;
    const int64_t rows[3] = {d.B, d.H, d.Tq};
    if (!q1 || !k1 || !q2 || !k2 || !v || !out || (out2 != nullptr) != (lse != nullptr) || !apart(rows, d.o_stride))
        return DIFFATTN_ERR_INVALID;
    if (rests && (!out2 || d.dtype != DIFFATTN_BF16 || !aligned16(rests))) return DIFFATTN_ERR_INVALID;
    if (!lambda_dev && !std::isfinite(lambda)) return DIFFATTN_ERR_INVALID;
    diffattn_epilogue e;
    rc = check_epilogue(epi, &e);
    if (rc != DIFFATTN_OK) return rc;
    if (e.norm == DIFFATTN_NORM_NONE && (e.weight || e.bias)) return DIFFATTN_ERR_INVALID;
    if (out2 && (e.norm != DIFFATTN_NORM_NONE || e.out_scale != 1.f)) return DIFFATTN_ERR_INVALID;
    if (!workspace_ok(workspace, workspace_bytes, diffattn_cross_workspace_bytes(desc))) return DIFFATTN_ERR_INVALID;
    CrossParams p{};
    fill_cross(&p, d, q1, k1, q2, k2, v, kv_lengths, lambda, lambda_dev);
    p.out = out;
    p.out2 = out2;
    p.lse = lse;
    p.rests = rests;
    p.norm = e.norm;
    p.norm_eps = e.eps;
    p.norm_weight = e.weight;
    p.norm_bias = e.bias;
    p.out_scale = e.out_scale;
    int sms = 0;
    rc = device_info(&p.status, &sms);
    if (rc != DIFFATTN_OK) return rc;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool tc = tc_inputs(d, q1, k1, q2, k2, v) && tma_rows(out, rows, d.o_stride) && (!out2 || aligned16(out2));
    if (!out2 && (wants_split(d) || (!tc && few_rows(d))))
        return cross_paged(d, q1, k1, q2, k2, v, kv_lengths, lambda, p.lambda_dev, e, out, workspace, workspace_bytes, st);
    if (tc)
        return forward_tc(p, sms, workspace, st);
    return launch_cross_simt(p, st) == 0 ? DIFFATTN_OK : DIFFATTN_ERR_CUDA;
}

int diffattn_cross_bwd(const diffattn_cross_desc* desc, const void* q1, const void* k1, const void* q2, const void* k2,
                       const void* v, const int32_t* kv_lengths, float lambda, const void* lambda_dev, const void* out,
                       const void* out2, const float* lse, const void* dout, void* dq1, void* dk1, void* dq2, void* dk2,
                       void* dv, void* dlambda, void* workspace, size_t workspace_bytes, diffattn_stream_t stream) {
    return diffattn_cross_bwd_ex(desc, q1, k1, q2, k2, v, kv_lengths, lambda, lambda_dev, out, out2, lse, nullptr, dout, dq1,
                                 dk1, dq2, dk2, dv, dlambda, workspace, workspace_bytes, stream);
}

int diffattn_cross_bwd_ex(const diffattn_cross_desc* desc, const void* q1, const void* k1, const void* q2, const void* k2,
                          const void* v, const int32_t* kv_lengths, float lambda, const void* lambda_dev, const void* out,
                          const void* out2, const float* lse, const void* rests, const void* dout, void* dq1, void* dk1,
                          void* dq2, void* dk2, void* dv, void* dlambda, void* workspace, size_t workspace_bytes,
                          diffattn_stream_t stream) {
    int rc = check_cross(desc);
    if (rc != DIFFATTN_OK) return rc;
    const diffattn_cross_desc& d = *desc;
    if (rests && (d.dtype != DIFFATTN_BF16 || !aligned16(rests))) return DIFFATTN_ERR_INVALID;
    if (!q1 || !k1 || !q2 || !k2 || !v || !out || !out2 || !lse || !dout) return DIFFATTN_ERR_INVALID;
    if (!lambda_dev && !std::isfinite(lambda)) return DIFFATTN_ERR_INVALID;
    if (!dq1 && !dq2 && !dv && !dlambda) return DIFFATTN_ERR_INVALID;
    if ((dk1 != nullptr) != (dv != nullptr) || (dk2 && !dk1)) return DIFFATTN_ERR_INVALID;
    if (!workspace_ok(workspace, workspace_bytes, diffattn_cross_bwd_workspace_bytes(desc))) return DIFFATTN_ERR_INVALID;
    CrossParams p{};
    fill_cross(&p, d, q1, k1, q2, k2, v, kv_lengths, lambda, lambda_dev);
    if (dk1 && !dk2 && !p.k_shared) return DIFFATTN_ERR_INVALID;
    if (dk1) p.k_shared = !dk2;
    p.out = const_cast<void*>(out);
    p.out2 = const_cast<void*>(out2);
    p.lse = const_cast<float*>(lse);
    p.rests = const_cast<void*>(rests);
    p.dout = dout;
    p.dq1 = dq1;
    p.dk1 = dk1;
    p.dq2 = dq2;
    p.dk2 = dk2;
    p.dv = dv;
    p.stats = static_cast<float*>(workspace);
    p.dlambda = dlambda;
    p.lambda_parts = p.stats + cross_rows(d) * 4;
    p.counters = reinterpret_cast<uint32_t*>(p.lambda_parts + kLambdaBlocks);
    int sms = 0;
    rc = device_info(&p.status, &sms);
    if (rc != DIFFATTN_OK) return rc;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // two key tensors 128 wide leave no TMEM for their gradients' accumulators
    const int64_t rows[3] = {d.B, d.H, d.Tq};
    const bool tc = tc_inputs(d, q1, k1, q2, k2, v) && tma_rows(dout, rows, d.dout_stride) && tma_rows(out, rows, d.o_stride) &&
                    aligned16(out2) && (d.D == 64 || p.k_shared) && d.B * d.H <= 65535 &&
                    aligned16(dq1) && aligned16(dk1) && aligned16(dq2) && aligned16(dk2) && aligned16(dv);
    if (tc) {
        rc = backward_tc(p, sms, p.lambda_parts + kLambdaBlocks + 4, st);
        if (rc != DIFFATTN_OK) return rc;
    } else if (launch_cross_simt_bwd(p, st) != 0) {
        return DIFFATTN_ERR_CUDA;
    }
    if (!dlambda) return DIFFATTN_OK;
    // the tensor-core path's rows hold -Dd_2
    return launch_cross_dlambda(p, tc ? 1.0f : -1.0f, st) == 0 ? DIFFATTN_OK : DIFFATTN_ERR_CUDA;
}

int diffattn_head_norm(const diffattn_norm_desc* desc, const void* x, const float* weight, const float* bias, void* y,
                       diffattn_stream_t stream) {
    const int rc = check_norm(desc);
    if (rc != DIFFATTN_OK) return rc;
    const diffattn_norm_desc& d = *desc;
    const int64_t n[3] = {d.B, d.H, d.T};
    if (!x || !y || !apart(n, d.y_stride)) return DIFFATTN_ERR_INVALID;
    HeadNormParams p{};
    fill_norm(&p, d, x, weight, bias);
    p.y = y;
    copy3(p.sy, d.y_stride);
    if (!rows16(y, n, d.y_stride, p.bf16 ? 2 : 4)) p.fast = 0;
    return launch_head_norm(p, reinterpret_cast<cudaStream_t>(stream)) == 0 ? DIFFATTN_OK : DIFFATTN_ERR_CUDA;
}

size_t diffattn_head_norm_bwd_workspace_bytes(const diffattn_norm_desc* desc) {
    if (check_norm(desc) != DIFFATTN_OK) return 0;
    return head_norm_bwd_floats(desc->H, desc->C) * sizeof(float);
}

int diffattn_head_norm_bwd(const diffattn_norm_desc* desc, const void* x, const float* weight, const void* dy, void* dx,
                           float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                           diffattn_stream_t stream) {
    const int rc = check_norm(desc);
    if (rc != DIFFATTN_OK) return rc;
    const diffattn_norm_desc& d = *desc;
    const int64_t n[3] = {d.B, d.H, d.T};
    if (!x || !dy || (!dx && !dweight && !dbias) || (dx && !apart(n, d.dx_stride))) return DIFFATTN_ERR_INVALID;
    if ((dweight || dbias) && (!workspace || !aligned16(workspace) ||
                               workspace_bytes < diffattn_head_norm_bwd_workspace_bytes(desc)))
        return DIFFATTN_ERR_INVALID;
    HeadNormParams p{};
    fill_norm(&p, d, x, weight, nullptr);
    p.dy = dy;
    p.dx = dx;
    copy3(p.sdy, d.dy_stride);
    copy3(p.sdx, d.dx_stride);
    p.dw = dweight;
    p.db = dbias;
    p.partial = static_cast<float*>(workspace);
    const int64_t es = p.bf16 ? 2 : 4;
    if (!rows16(dy, n, d.dy_stride, es) || (dx && !rows16(dx, n, d.dx_stride, es))) p.fast = 0;
    plan_head_norm_bwd(&p);
    return launch_head_norm_bwd(p, reinterpret_cast<cudaStream_t>(stream)) == 0 ? DIFFATTN_OK : DIFFATTN_ERR_CUDA;
}

}  // extern "C"
