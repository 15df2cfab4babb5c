// api_paged.cu -- the C ABI of the operators around a paged key/value cache: argument
// checks, plans and launches.
#include "diffattn.h"
#include "kernels.h"
#include "paged.h"

#include <cmath>
#include <cstdint>

namespace diffattn {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool nonneg(const int64_t s[3]) { return s[0] >= 0 && s[1] >= 0 && s[2] >= 0; }
bool rows16(const void* p, const int64_t s[3], int64_t es) {
    return aligned16(p) && s[0] * es % 16 == 0 && s[1] * es % 16 == 0 && s[2] * es % 16 == 0;
}
void copy3(int64_t dst[3], const int64_t src[3]) {
    for (int i = 0; i < 3; ++i) dst[i] = src[i];
}
bool dtype_ok(int32_t d) { return d == DIFFATTN_BF16 || d == DIFFATTN_F32; }

// The checks of a rotary descriptor that need no tensors.
int check_rotary(const diffattn_rotary_desc* d, const float* cos, const float* sin, bool tables) {
    // H and Hk count where their tensors are left out too: the backward's workspace goes by both
    if (!d || d->B < 1 || d->T < 1 || d->D < 1 || d->D > 128 || d->H < 0 || d->Hk < 0 || !dtype_ok(d->dtype))
        return DIFFATTN_ERR_INVALID;
    if (d->rotary_dim < 0 || d->rotary_dim > d->D || d->rotary_dim % 2 != 0) return DIFFATTN_ERR_INVALID;
    if (d->norm != DIFFATTN_NORM_NONE && d->norm != DIFFATTN_NORM_RMS) return DIFFATTN_ERR_INVALID;
    if (d->norm != DIFFATTN_NORM_NONE && !(std::isfinite(d->eps) && d->eps > 0.f)) return DIFFATTN_ERR_INVALID;
    if (tables && d->rotary_dim > 0 && (!cos || !sin || d->table_rows < 1)) return DIFFATTN_ERR_INVALID;
    if (d->pos_stride[0] < 0 || d->pos_stride[1] < 0) return DIFFATTN_ERR_INVALID;
    if ((d->q_weight_stride != 0 && d->q_weight_stride != d->D) ||
        (d->k_weight_stride != 0 && d->k_weight_stride != d->D))
        return DIFFATTN_ERR_INVALID;
    // token indices, and those of a last block's threads past them, in 31 bits
    constexpr int64_t kMaxTokens = 1 << 30;
    if (d->B > kMaxTokens || d->T > kMaxTokens || d->B * d->T > kMaxTokens) return DIFFATTN_ERR_UNSUPPORTED;
    // rows of the backward's kernels are counted in 31 bits
    if (2.0 * (d->B * d->T / 16 + 16) * ((double)d->H + (double)d->Hk) > INT32_MAX)
        return DIFFATTN_ERR_UNSUPPORTED;
    return DIFFATTN_OK;
}

void fill_rotary(RotaryParams* p, const diffattn_rotary_desc& d, const float* cos, const float* sin,
                 const void* positions) {
    p->B = (int)d.B;
    p->T = (int)d.T;
    p->by_T.set((uint32_t)d.T);
    p->D = (int)d.D;
    p->R = d.rotary_dim;
    p->bf16 = d.dtype == DIFFATTN_BF16;
    p->interleaved = d.interleaved != 0;
    p->norm = d.norm == DIFFATTN_NORM_RMS;
    p->eps = d.eps;
    p->inv_D = 1.0f / (float)d.D;       // exact where the vector kernel takes D
    p->cos = cos;
    p->sin = sin;
    p->table_rows = d.table_rows;
    p->pos = positions;
    p->pos64 = d.pos64 != 0;
    p->pos_stride[0] = d.pos_stride[0];
    p->pos_stride[1] = d.pos_stride[1];
    // the vector kernel: a row is 2, 4, 8 (float32: 16) lanes of twice 16 bytes
    const int v = p->bf16 ? 8 : 4;
    const int lanes = p->D % (2 * v) == 0 ? p->D / (2 * v) : 0;
    p->fast = (lanes == 2 || lanes == 4 || lanes == 8 || (lanes == 16 && !p->bf16)) && p->R % (2 * v) == 0 &&
              (p->R == 0 || (aligned16(cos) && aligned16(sin)));
}

// One of Q1, K1, Q2, K2 as a stream; false if its arguments do not fit.
bool add_stream(RotaryParams* p, const void* x, const int64_t sx[3], int64_t heads, void* y, const float* w,
                int64_t w_stride, int slot) {
    if (!x && !y) return true;
    if (!x || !y || heads < 1 || !nonneg(sx)) return false;
    RowStream& s = p->s[p->n++];
    s.x = x;
    s.y = y;
    copy3(s.sx, sx);
    s.sy[2] = p->D;
    s.sy[1] = (int64_t)p->T * p->D;
    s.sy[0] = s.sy[1] * heads;
    s.heads = (int)heads;
    s.width = p->D;
    s.kind = kRowsDense;
    s.weight = w;
    s.w_stride = w_stride;
    s.g = nullptr;
    s.grad_slot = slot;
    const int es = p->bf16 ? 2 : 4;
    if (!rows16(x, sx, es) || !aligned16(y) || (w && !aligned16(w))) p->fast = 0;
    return true;
}

constexpr int64_t kMaxHeads = 65535;

int build_rotary(RotaryParams* p, const diffattn_rotary_desc* d, const void* q1, const void* k1, const void* q2,
                 const void* k2, const float* qw, const float* kw, const float* cos, const float* sin,
                 const void* positions, void* yq1, void* yk1, void* yq2, void* yk2) {
    const int rc = check_rotary(d, cos, sin, true);
    if (rc != DIFFATTN_OK) return rc;
    if ((qw || kw) && d->norm == DIFFATTN_NORM_NONE) return DIFFATTN_ERR_INVALID;
    if (d->H > kMaxHeads || d->Hk > kMaxHeads || 2 * (d->H + d->Hk) > kMaxHeads) return DIFFATTN_ERR_UNSUPPORTED;
    fill_rotary(p, *d, cos, sin, positions);
    if (!add_stream(p, q1, d->q1_stride, d->H, yq1, qw, d->q_weight_stride, 0) ||
        !add_stream(p, k1, d->k1_stride, d->Hk, yk1, kw, d->k_weight_stride, 1) ||
        !add_stream(p, q2, d->q2_stride, d->H, yq2, qw, d->q_weight_stride, 0) ||
        !add_stream(p, k2, d->k2_stride, d->Hk, yk2, kw, d->k_weight_stride, 1) || p->n == 0)
        return DIFFATTN_ERR_INVALID;
    return DIFFATTN_OK;
}

size_t rotary_bwd_bytes(const diffattn_rotary_desc* d) {
    return rotary_bwd_floats(d->B, d->T, d->D, 2 * (d->H + d->Hk)) * sizeof(float);
}

int check_pages(const diffattn_pages* g) {
    if (!g || g->num_pages < 1 || g->page_size < 1 || g->max_pages < 1 || g->block_table_stride < 0 ||
        !nonneg(g->k1_stride) || !nonneg(g->k2_stride) || !nonneg(g->v_stride))
        return DIFFATTN_ERR_INVALID;
    if (g->num_pages > INT32_MAX || g->page_size > (1 << 20) || g->max_pages > INT32_MAX)
        return DIFFATTN_ERR_UNSUPPORTED;
    return DIFFATTN_OK;
}

// Whether rows of these sizes and strides have a place each (a stride of 0 gives many one).
bool apart(const int64_t n[3], const int64_t s[3]) {
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && s[i] == 0) return false;
    return true;
}

bool same3(const int64_t a[3], const int64_t b[3]) { return a[0] == b[0] && a[1] == b[1] && a[2] == b[2]; }

// ---------------------------------------------------------------------------
// attention over the paged cache
// ---------------------------------------------------------------------------
struct PagedPlan {
    int chunk_rows = 0, head_rows = 0, row_chunks = 0, tile = 0, workers = 0;
    size_t bytes = 0;
};

int check_paged(const diffattn_paged_desc* d, const diffattn_pages* g) {
    if (!d || d->B < 1 || d->H < 1 || d->Tq < 1 || d->D < 1 || d->D > 128 || !dtype_ok(d->dtype))
        return DIFFATTN_ERR_INVALID;
    const int64_t dv = d->Dv == 0 ? 2 * d->D : d->Dv;
    const int64_t group = d->kv_group > 1 ? d->kv_group : 1;
    if (d->kv_group < 0 || d->H % group != 0 || dv < 1 || dv > 256 || !nonneg(d->q1_stride) ||
        !nonneg(d->q2_stride) || !nonneg(d->o_stride) || d->mask_stride[0] < 0 || d->mask_stride[1] < 0 ||
        d->zero_rest < 0 || d->zero_rest > 1 || d->reserved != 0)
        return DIFFATTN_ERR_INVALID;
    const int rc = check_pages(g);
    if (rc != DIFFATTN_OK) return rc;
    // the tiles of all units in 31 bits, 16 keys a tile and 16 rows a unit at least
    const double keys = (double)g->max_pages * g->page_size, rows = (double)group * d->Tq;
    if (keys > INT32_MAX / 2 || d->B * (keys / 16 + 8) * (double)(d->H / group) * (rows / 16 + 1) > INT32_MAX)
        return DIFFATTN_ERR_UNSUPPORTED;
    if (d->Tq > 1024 || d->B > (1 << 24) || d->H > (1 << 20) || d->B * d->H > (1ll << 31) / 1024)
        return DIFFATTN_ERR_UNSUPPORTED;
    return DIFFATTN_OK;
}

size_t part_bytes(const PagedPlan& n, int64_t dv) {
    return n.workers * sizeof(PagedJoin) + (size_t)2 * n.workers * n.chunk_rows * paged_part_floats((int)dv) * sizeof(float);
}

// `workers`, or fewer if there cannot be that many tiles.
int fewer(const diffattn_paged_desc& d, const diffattn_pages& g, const PagedPlan* n, int workers) {
    const int64_t group = d.kv_group > 1 ? d.kv_group : 1;
    const double tiles = (double)d.B * (d.H / group) * n->row_chunks * ((double)g.max_pages * g.page_size / n->tile + 1);
    return tiles < workers ? (int)tiles : workers;
}

// The plan of the CUDA-core kernel; its blocks are what `sms` multiprocessors hold at
// once.
void plan_simt(const diffattn_paged_desc& d, const diffattn_pages& g, int sms, PagedPlan* n) {
    const int64_t dv = d.Dv == 0 ? 2 * d.D : d.Dv;
    const int64_t group = d.kv_group > 1 ? d.kv_group : 1;
    n->head_rows = (int)d.Tq;
    n->chunk_rows = paged_simt_rows(group * d.Tq);
    n->row_chunks = (int)((group * d.Tq + n->chunk_rows - 1) / n->chunk_rows);
    n->tile = 32;
    n->workers = fewer(d, g, n, sms * paged_simt_blocks((int)d.D, (int)dv, d.dtype == DIFFATTN_BF16 ? 2 : 4, n->chunk_rows));
    n->bytes = part_bytes(*n, dv);
}

// Strides that TMA takes, of the dimensions that are stepped.
bool tma_strides(const int64_t n[3], const int64_t s[3]) {
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (s[i] % 8 != 0 || s[i] <= 0 || s[i] >= (int64_t(1) << 38))) return false;
    return true;
}

// Whether the tensor-core kernels take the shape and the cache's layout: bf16, value
// width 128, Q/K width 64 or 128, pages of a multiple of 16 slots, and strides (with the
// bases, checked at the call) that TMA takes.
bool tc_shape(const diffattn_paged_desc& d, const diffattn_pages& g) {
    if (d.dtype != DIFFATTN_BF16 || (d.Dv == 0 ? 2 * d.D : d.Dv) != 128 || (d.D != 64 && d.D != 128) ||
        g.page_size % 16 != 0)
        return false;
    const int64_t n[3] = {g.num_pages, d.H / (d.kv_group > 1 ? d.kv_group : 1), g.page_size};
    return tma_strides(n, g.k1_stride) && tma_strides(n, g.k2_stride) && tma_strides(n, g.v_stride);
}

// The plan of the tensor-core kernel for up to 16 rows.
void plan_mma(const diffattn_paged_desc& d, const diffattn_pages& g, int sms, PagedPlan* n) {
    const int64_t group = d.kv_group > 1 ? d.kv_group : 1;
    const int64_t rows = group * d.Tq;
    n->head_rows = (int)d.Tq;
    n->row_chunks = (int)((rows + kMmaRows - 1) / kMmaRows);
    n->chunk_rows = (int)((rows + n->row_chunks - 1) / n->row_chunks);
    n->tile = kMmaTile;
    n->workers = sms * kMmaBlocks * (n->chunk_rows <= paged_solo_rows((int)d.D) ? kMmaWarps : 1);
    n->bytes = part_bytes(*n, 128);
}

// The tcgen05 kernel, for more than 16 rows: the 16-row kernel reads the cache once for each
// 16 of them.  Measured on both sides (16 sequences of up to 8192 keys; D = 128 with 8
// key/value heads and shared keys, D = 64 with 16): 16 rows take 86 and 139 us there and 100 and
// 170 here, 18 to 32 rows 128 to 139 and 232 to 245 there, 98 and 168 here.
bool wants_tc(const diffattn_paged_desc& d) {
    const int64_t group = d.kv_group > 1 ? d.kv_group : 1;
    return group * d.Tq > kMmaRows;
}
// Its plan: whole heads in units of up to 128 rows, each head's tokens padded to a multiple of 8.
void plan_tc(const diffattn_paged_desc& d, const diffattn_pages& g, int sms, PagedPlan* n) {
    const int64_t group = d.kv_group > 1 ? d.kv_group : 1;
    if (d.Tq <= kTcRows) {
        n->head_rows = (int)((d.Tq + 7) / 8 * 8);
        int64_t heads = kTcRows / n->head_rows;
        if (heads > group) heads = group;
        n->row_chunks = (int)((group + heads - 1) / heads);
        heads = (group + n->row_chunks - 1) / n->row_chunks;        // evenly filled
        n->chunk_rows = (int)heads * n->head_rows;
    } else {
        n->head_rows = (int)((d.Tq + kTcRows - 1) / kTcRows * kTcRows);
        n->chunk_rows = kTcRows;
        n->row_chunks = (int)(group * (n->head_rows / kTcRows));
    }
    n->tile = kTcTile;
    n->workers = fewer(d, g, n, sms);
    n->bytes = part_bytes(*n, 128);
}

int device_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 152;                 // no GPU: a size to plan with
    }
    return sms;
}

}  // namespace
}  // namespace diffattn

using namespace diffattn;

extern "C" {

int diffattn_rotary(const diffattn_rotary_desc* desc, const void* q1, const void* k1, const void* q2,
                    const void* k2, const float* q_weight, const float* k_weight, const float* cos,
                    const float* sin, const void* positions, void* q1_out, void* k1_out, void* q2_out,
                    void* k2_out, diffattn_stream_t stream) {
    RotaryParams p{};
    int rc = build_rotary(&p, desc, q1, k1, q2, k2, q_weight, k_weight, cos, sin, positions, q1_out, k1_out,
                          q2_out, k2_out);
    if (rc != DIFFATTN_OK) return rc;
    int sms = 0;
    rc = device_info(&p.status, &sms);
    if (rc != DIFFATTN_OK) return rc;
    plan_rotary(&p, sms);
    return launch_rotary(p, reinterpret_cast<cudaStream_t>(stream)) == 0 ? DIFFATTN_OK : DIFFATTN_ERR_CUDA;
}

size_t diffattn_rotary_bwd_workspace_bytes(const diffattn_rotary_desc* desc) {
    if (check_rotary(desc, nullptr, nullptr, false) != DIFFATTN_OK || desc->H > kMaxHeads ||
        desc->Hk > kMaxHeads)
        return 0;
    return rotary_bwd_bytes(desc);
}

int diffattn_rotary_bwd(const diffattn_rotary_desc* desc, const void* q1, const void* k1, const void* q2,
                        const void* k2, const float* q_weight, const float* k_weight, const float* cos,
                        const float* sin, const void* positions, const void* dq1_out, const void* dk1_out,
                        const void* dq2_out, const void* dk2_out, void* dq1, void* dk1, void* dq2, void* dk2,
                        float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                        diffattn_stream_t stream) {
    if (!desc) return DIFFATTN_ERR_INVALID;
    diffattn_rotary_desc d = *desc;
    const void* x[4] = {q1, k1, q2, k2};
    const void* g[4] = {dq1_out, dk1_out, dq2_out, dk2_out};
    int64_t* sx[4] = {d.q1_stride, d.k1_stride, d.q2_stride, d.k2_stride};
    const int64_t* sg[4] = {d.q1_grad_stride, d.k1_grad_stride, d.q2_grad_stride, d.k2_grad_stride};
    for (int i = 0; i < 4; ++i) {
        if (!x[i] && g[i] && d.norm == DIFFATTN_NORM_NONE) {
            // a rotation's gradient does not depend on the rows, and the kernels do not read them
            x[i] = g[i];
            copy3(sx[i], sg[i]);
        }
        if ((x[i] != nullptr) != (g[i] != nullptr)) return DIFFATTN_ERR_INVALID;
    }
    RotaryParams p{};
    int rc = build_rotary(&p, &d, x[0], x[1], x[2], x[3], q_weight, k_weight, cos, sin, positions, dq1, dk1, dq2, dk2);
    if (rc != DIFFATTN_OK) return rc;
    for (int i = 0, n = 0; i < 4; ++i) {
        if (!x[i]) continue;
        if (!nonneg(sg[i])) return DIFFATTN_ERR_INVALID;
        p.s[n].g = g[i];
        copy3(p.s[n].sg, sg[i]);
        if (!rows16(g[i], sg[i], p.bf16 ? 2 : 4)) p.fast = 0;
        ++n;
    }
    if ((dq_weight || dk_weight) && d.norm == DIFFATTN_NORM_NONE) return DIFFATTN_ERR_INVALID;
    if ((dq_weight && !q1 && !q2) || (dk_weight && !k1 && !k2)) return DIFFATTN_ERR_INVALID;
    if (!workspace || workspace_bytes < rotary_bwd_bytes(&d) || !aligned16(workspace)) return DIFFATTN_ERR_INVALID;
    p.partial = static_cast<float*>(workspace);
    p.dw[0] = dq_weight;
    p.dw[1] = dk_weight;
    p.dw_stride[0] = d.q_weight_stride;
    p.dw_stride[1] = d.k_weight_stride;
    int sms = 0;
    rc = device_info(&p.status, &sms);
    if (rc != DIFFATTN_OK) return rc;
    plan_rotary_bwd(&p, sms);
    return launch_rotary_bwd(p, reinterpret_cast<cudaStream_t>(stream)) == 0 ? DIFFATTN_OK : DIFFATTN_ERR_CUDA;
}

int diffattn_paged_append(const diffattn_rotary_desc* desc, int64_t Dv, const int64_t v_stride[3],
                          const diffattn_pages* pages, const void* k1, const void* k2, const void* v,
                          const float* k_weight, const float* cos, const float* sin, const void* positions,
                          const int32_t* lengths, const int32_t* new_lengths, const int32_t* block_table,
                          void* k1_cache, void* k2_cache, void* v_cache, diffattn_stream_t stream) {
    if (!desc) return DIFFATTN_ERR_INVALID;
    diffattn_rotary_desc d = *desc;
    d.H = 0;                            // not read
    int rc = check_rotary(&d, cos, sin, true);
    if (rc != DIFFATTN_OK) return rc;
    rc = check_pages(pages);
    if (rc != DIFFATTN_OK) return rc;
    const int64_t dv = Dv == 0 ? 2 * d.D : Dv;
    if (dv < 1 || dv > 256 || d.Hk < 1 || !v_stride || !nonneg(v_stride) || !k1 || !v || !lengths || !block_table ||
        !k1_cache || !v_cache || (k_weight && d.norm == DIFFATTN_NORM_NONE))
        return DIFFATTN_ERR_INVALID;
    if (3 * d.Hk > kMaxHeads) return DIFFATTN_ERR_UNSUPPORTED;
    const bool shared = (!k2 && !k2_cache) || (k2 == k1 && k2_cache == k1_cache &&
                                               same3(d.k1_stride, d.k2_stride) &&
                                               same3(pages->k1_stride, pages->k2_stride));
    if (!shared && (!k2 || !k2_cache || k2_cache == k1_cache)) return DIFFATTN_ERR_INVALID;
    const int64_t slots[3] = {pages->num_pages, d.Hk, pages->page_size};
    if (v_cache == k1_cache || v_cache == k2_cache || !apart(slots, pages->k1_stride) || !apart(slots, pages->v_stride) ||
        (!shared && !apart(slots, pages->k2_stride)))
        return DIFFATTN_ERR_INVALID;
    RotaryParams p{};
    fill_rotary(&p, d, cos, sin, positions);
    const int es = p.bf16 ? 2 : 4;
    if (!add_stream(&p, k1, d.k1_stride, d.Hk, k1_cache, k_weight, d.k_weight_stride, 1) ||
        (!shared && !add_stream(&p, k2, d.k2_stride, d.Hk, k2_cache, k_weight, d.k_weight_stride, 1)) ||
        !add_stream(&p, v, v_stride, d.Hk, v_cache, nullptr, 0, 1))
        return DIFFATTN_ERR_INVALID;
    for (int i = 0; i < p.n; ++i) {
        const int64_t* s = i == p.n - 1 ? pages->v_stride : i == 0 ? pages->k1_stride : pages->k2_stride;
        copy3(p.s[i].sy, s);
        p.s[i].kind = i == p.n - 1 ? kRowsCopy : kRowsPaged;
        if (!rows16(p.s[i].y, s, es)) p.fast = 0;
    }
    p.s[p.n - 1].width = (int)dv;
    if (dv * es % 16 != 0) p.fast = 0;
    p.lengths = lengths;
    p.new_lengths = new_lengths;
    p.table = block_table;
    p.table_stride = pages->block_table_stride;
    p.max_pages = pages->max_pages;
    p.num_pages = pages->num_pages;
    p.page = pages->page_size;
    int sms = 0;
    rc = device_info(&p.status, &sms);
    if (rc != DIFFATTN_OK) return rc;
    plan_rotary(&p, sms);
    return launch_rotary(p, reinterpret_cast<cudaStream_t>(stream)) == 0 ? DIFFATTN_OK : DIFFATTN_ERR_CUDA;
}

size_t diffattn_paged_workspace_bytes(const diffattn_paged_desc* desc, const diffattn_pages* pages) {
    if (check_paged(desc, pages) != DIFFATTN_OK) return 0;
    PagedPlan n;
    const int sms = device_sms();
    plan_simt(*desc, *pages, sms, &n);
    size_t bytes = n.bytes;
    if (tc_shape(*desc, *pages)) {
        plan_mma(*desc, *pages, sms, &n);
        if (n.bytes > bytes) bytes = n.bytes;
        if (wants_tc(*desc)) {
            plan_tc(*desc, *pages, sms, &n);
            if (n.bytes > bytes) bytes = n.bytes;
        }
    }
    return bytes;
}

int diffattn_paged_decode(const diffattn_paged_desc* desc, const diffattn_pages* pages, const void* q1,
                          const void* k1_cache, const void* q2, const void* k2_cache, const void* v_cache,
                          const int32_t* block_table, const int32_t* lengths, const int32_t* q_lengths,
                          const uint8_t* tree_mask, float lambda, const float* lambda_dev,
                          const diffattn_epilogue* epi, void* out, void* workspace, size_t workspace_bytes,
                          diffattn_stream_t stream) {
    int rc = check_paged(desc, pages);
    if (rc != DIFFATTN_OK) return rc;
    if (!q1 || !k1_cache || !q2 || !k2_cache || !v_cache || !block_table || !lengths || !out)
        return DIFFATTN_ERR_INVALID;
    if (tree_mask && desc->Tq > 64) return DIFFATTN_ERR_INVALID;
    if (!lambda_dev && !std::isfinite(lambda)) return DIFFATTN_ERR_INVALID;
    diffattn_epilogue e;
    rc = check_epilogue(epi, &e);
    if (rc != DIFFATTN_OK) return rc;
    if (!workspace || !aligned16(workspace)) return DIFFATTN_ERR_INVALID;
    const diffattn_paged_desc& d = *desc;
    const int64_t rows[3] = {d.B, d.H, d.Tq};
    if (!apart(rows, d.o_stride)) return DIFFATTN_ERR_INVALID;
    const int64_t es = d.dtype == DIFFATTN_BF16 ? 2 : 4;
    PagedParams p{};
    int sms = 0;
    rc = device_info(&p.status, &sms);
    if (rc != DIFFATTN_OK) return rc;
    PagedPlan n;
    const bool tc = tc_shape(d, *pages) && aligned16(k1_cache) && aligned16(k2_cache) && aligned16(v_cache);
    // the queries go through TMA too, from 16-byte aligned rows
    const bool tcgen = tc && wants_tc(d) && aligned16(q1) && aligned16(q2) && tma_strides(rows, d.q1_stride) &&
                       tma_strides(rows, d.q2_stride);
    if (tcgen) plan_tc(d, *pages, sms, &n);
    else if (tc) plan_mma(d, *pages, sms, &n);
    else plan_simt(d, *pages, sms, &n);
    if (workspace_bytes < n.bytes) return DIFFATTN_ERR_INVALID;
    p.B = (int)d.B;
    p.H = (int)d.H;
    p.group = d.kv_group > 1 ? d.kv_group : 1;
    p.Hk = p.H / p.group;
    p.Tq = (int)d.Tq;
    p.D = (int)d.D;
    p.Dv = (int)(d.Dv == 0 ? 2 * d.D : d.Dv);
    p.bf16 = d.dtype == DIFFATTN_BF16;
    p.k_shared = k1_cache == k2_cache && same3(pages->k1_stride, pages->k2_stride);
    p.page = (int)pages->page_size;
    p.max_pages = pages->max_pages;
    p.num_pages = pages->num_pages;
    p.q1 = q1;
    p.q2 = q2;
    p.k1 = k1_cache;
    p.k2 = k2_cache;
    p.v = v_cache;
    p.out = out;
    copy3(p.s_q1, d.q1_stride);
    copy3(p.s_q2, d.q2_stride);
    copy3(p.s_o, d.o_stride);
    copy3(p.s_k1, pages->k1_stride);
    copy3(p.s_k2, pages->k2_stride);
    copy3(p.s_v, pages->v_stride);
    p.table = block_table;
    p.table_stride = pages->block_table_stride;
    p.lengths = lengths;
    p.q_lengths = q_lengths;
    p.zero_rest = q_lengths && d.zero_rest;
    p.mask = tree_mask;
    p.mask_stride[0] = d.mask_stride[0];
    p.mask_stride[1] = d.mask_stride[1];
    p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)d.D));
    p.lambda = lambda;
    p.lambda_dev = lambda_dev;
    p.norm = e.norm;
    p.norm_eps = e.eps;
    p.norm_weight = e.weight;
    p.norm_bias = e.bias;
    p.out_scale = e.out_scale;
    p.vec16 = p.D * es % 16 == 0 && p.Dv * es % 16 == 0 && rows16(p.k1, p.s_k1, es) && rows16(p.k2, p.s_k2, es) &&
              rows16(p.v, p.s_v, es);
    p.q16 = rows16(q1, d.q1_stride, es) && rows16(q2, d.q2_stride, es);
    p.o4 = (reinterpret_cast<uintptr_t>(out) | (uintptr_t)(d.o_stride[0] * es) | (uintptr_t)(d.o_stride[1] * es) |
            (uintptr_t)(d.o_stride[2] * es)) % 4 == 0;
    p.o16 = rows16(out, d.o_stride, es);
    p.joins = static_cast<PagedJoin*>(workspace);
    p.part = reinterpret_cast<float*>(p.joins + n.workers);
    p.head_rows = n.head_rows;
    p.chunk_rows = n.chunk_rows;
    p.row_chunks = n.row_chunks;
    p.workers = n.workers;
    p.sparse_joins = tc && !tcgen && n.chunk_rows <= paged_solo_rows(p.D);
    p.solo_workers = sms * kMmaBlocks * kMmaWarps;
    if (tc) {
        // boxes that stay inside one page and divide the tile
        int box = tcgen ? kTcTile : 16;          // a slice of the 16-row kernel
        while (p.page % box != 0) box /= 2;
        CUtensorMap maps[5];
        const int64_t kd[4] = {p.D, p.page, p.Hk, p.num_pages}, vd[4] = {p.Dv, p.page, p.Hk, p.num_pages};
        if (encode_map_4d(&maps[0], p.k1, kd, p.s_k1, 64, box) != DIFFATTN_OK ||
            encode_map_4d(&maps[1], p.k2, kd, p.s_k2, 64, box) != DIFFATTN_OK ||
            encode_map_4d(&maps[2], p.v, vd, p.s_v, 64, box) != DIFFATTN_OK)
            return DIFFATTN_ERR_CUDA;
        if (tcgen) {
            const int q_box = p.head_rows < kTcRows ? p.head_rows : kTcRows;
            const int64_t qd[4] = {p.D, p.Tq, p.H, p.B};
            if (encode_map_4d(&maps[3], q1, qd, p.s_q1, 64, q_box) != DIFFATTN_OK ||
                encode_map_4d(&maps[4], q2, qd, p.s_q2, 64, q_box) != DIFFATTN_OK)
                return DIFFATTN_ERR_CUDA;
            return launch_paged_tc(maps, p, box, q_box, reinterpret_cast<cudaStream_t>(stream)) == 0 ? DIFFATTN_OK
                                                                                                     : DIFFATTN_ERR_CUDA;
        }
        return launch_paged_mma(maps, p, reinterpret_cast<cudaStream_t>(stream)) == 0 ? DIFFATTN_OK
                                                                                           : DIFFATTN_ERR_CUDA;
    }
    return launch_paged_simt(p, reinterpret_cast<cudaStream_t>(stream)) == 0 ? DIFFATTN_OK : DIFFATTN_ERR_CUDA;
}

}  // extern "C"
