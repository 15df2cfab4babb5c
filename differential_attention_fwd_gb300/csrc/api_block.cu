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
        (d->dtype != DIFFATTN_BF16 && d->dtype != DIFFATTN_F32) || d->kv_group < 0)
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
                const void* v, const int32_t* lengths, float lambda, const float* lambda_dev) {
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
    p->lambda_dev = lambda_dev;
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

}  // namespace
}  // namespace diffattn

using namespace diffattn;

extern "C" {

size_t diffattn_cross_workspace_bytes(const diffattn_cross_desc* desc) {
    if (check_cross(desc) != DIFFATTN_OK) return 0;
    return 16;
}

size_t diffattn_cross_bwd_workspace_bytes(const diffattn_cross_desc* desc) {
    if (check_cross(desc) != DIFFATTN_OK) return 0;
    // the rows' statistics, and partial sums of dlambda
    return (size_t)(cross_rows(*desc) * 4 + 128) * sizeof(float);
}

int diffattn_cross_fwd(const diffattn_cross_desc* desc, const void* q1, const void* k1, const void* q2, const void* k2,
                       const void* v, const int32_t* kv_lengths, float lambda, const float* lambda_dev,
                       const diffattn_epilogue* epi, void* out, void* out2, float* lse, void* workspace,
                       size_t workspace_bytes, diffattn_stream_t stream) {
    int rc = check_cross(desc);
    if (rc != DIFFATTN_OK) return rc;
    const diffattn_cross_desc& d = *desc;
    const int64_t rows[3] = {d.B, d.H, d.Tq};
    if (!q1 || !k1 || !q2 || !k2 || !v || !out || (out2 != nullptr) != (lse != nullptr) || !apart(rows, d.o_stride))
        return DIFFATTN_ERR_INVALID;
    if (!lambda_dev && !std::isfinite(lambda)) return DIFFATTN_ERR_INVALID;
    diffattn_epilogue e;
    rc = check_epilogue(epi, &e);
    if (rc != DIFFATTN_OK) return rc;
    if (out2 && (e.norm != DIFFATTN_NORM_NONE || e.weight || e.bias || e.out_scale != 1.f)) return DIFFATTN_ERR_INVALID;
    if (!workspace_ok(workspace, workspace_bytes, diffattn_cross_workspace_bytes(desc))) return DIFFATTN_ERR_INVALID;
    CrossParams p{};
    fill_cross(&p, d, q1, k1, q2, k2, v, kv_lengths, lambda, lambda_dev);
    p.out = out;
    p.out2 = out2;
    p.lse = lse;
    p.norm = e.norm;
    p.norm_eps = e.eps;
    p.norm_weight = e.weight;
    p.norm_bias = e.bias;
    p.out_scale = e.out_scale;
    int sms = 0;
    rc = device_info(&p.status, &sms);
    if (rc != DIFFATTN_OK) return rc;
    return launch_cross_simt(p, reinterpret_cast<cudaStream_t>(stream)) == 0 ? DIFFATTN_OK : DIFFATTN_ERR_CUDA;
}

int diffattn_cross_bwd(const diffattn_cross_desc* desc, const void* q1, const void* k1, const void* q2, const void* k2,
                       const void* v, const int32_t* kv_lengths, float lambda, const float* lambda_dev, const void* out,
                       const void* out2, const float* lse, const void* dout, void* dq1, void* dk1, void* dq2, void* dk2,
                       void* dv, float* dlambda, void* workspace, size_t workspace_bytes, diffattn_stream_t stream) {
    int rc = check_cross(desc);
    if (rc != DIFFATTN_OK) return rc;
    const diffattn_cross_desc& d = *desc;
    if (!q1 || !k1 || !q2 || !k2 || !v || !out || !out2 || !lse || !dout) return DIFFATTN_ERR_INVALID;
    if (!lambda_dev && !std::isfinite(lambda)) return DIFFATTN_ERR_INVALID;
    if (!dq1 && !dq2 && !dv && !dlambda) return DIFFATTN_ERR_INVALID;
    if ((dk1 != nullptr) != (dv != nullptr) || (dk2 && !dk1)) return DIFFATTN_ERR_INVALID;
    if (!workspace_ok(workspace, workspace_bytes, diffattn_cross_bwd_workspace_bytes(desc))) return DIFFATTN_ERR_INVALID;
    CrossParams p{};
    fill_cross(&p, d, q1, k1, q2, k2, v, kv_lengths, lambda, lambda_dev);
    if (dk1 && !dk2 && !p.k_shared) return DIFFATTN_ERR_INVALID;
    p.k_shared = dk1 && !dk2;
    p.out = const_cast<void*>(out);
    p.out2 = const_cast<void*>(out2);
    p.lse = const_cast<float*>(lse);
    p.dout = dout;
    p.dq1 = dq1;
    p.dk1 = dk1;
    p.dq2 = dq2;
    p.dk2 = dk2;
    p.dv = dv;
    p.stats = static_cast<float*>(workspace);
    int sms = 0;
    rc = device_info(&p.status, &sms);
    if (rc != DIFFATTN_OK) return rc;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (launch_cross_simt_bwd(p, st) != 0) return DIFFATTN_ERR_CUDA;
    if (!dlambda) return DIFFATTN_OK;
    return launch_bwd_dlambda(p.stats, cross_rows(d), -1.0f, dlambda, st) == 0 ? DIFFATTN_OK : DIFFATTN_ERR_CUDA;
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
