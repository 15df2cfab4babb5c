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

}  // namespace
}  // namespace diffattn

using namespace diffattn;

extern "C" {

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
