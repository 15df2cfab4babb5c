// block.h -- internal interface of the operators of a cross-attention block: attention over
// an encoder's states and the norm of each head's output.  Not part of the public ABI.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "diffattn.h"
#include "paged.h"

namespace diffattn {

// The norm of head rows x [B, H, T, C], forward and backward.
struct HeadNormParams {
    int B, H, T, C;
    int tokens;                 // B * T
    FastDiv by_T;
    int bf16, group;            // group: the mean is taken off first
    float eps, scale, inv_C;
    const void* x;
    void* y;
    const void* dy;
    void* dx;                   // nullptr: not wanted
    int64_t sx[3], sy[3], sdy[3], sdx[3];
    const float* w;             // [H, C], nullptr = 1
    const float* b;             // [H, C], nullptr = 0
    float* dw;                  // [H, C], nullptr: not wanted
    float* db;
    float* partial;             // [chunks][H][2][C]
    int fast;                   // 16-byte rows: the vector kernel
    int chunks, per_chunk;      // backward: blocks along the tokens, and the tokens of each
};

int launch_head_norm(const HeadNormParams& p, cudaStream_t stream);
int launch_head_norm_bwd(const HeadNormParams& p, cudaStream_t stream);
void plan_head_norm_bwd(HeadNormParams* p);
size_t head_norm_bwd_floats(int64_t H, int64_t C);

// Attention over an encoder's states, forward and backward.  Gradients are dense: dq
// [B, H, Tq, D], dk [B, Hk, Tk, D], dv [B, Hk, Tk, Dv].
struct CrossParams {
    int B, H, Hk, group, Tq, Tk, D, Dv;
    int bf16;
    int k_shared;               // K1 and K2 are one tensor, and dk1 takes both branches' gradient
    float scale;                // 1 / sqrt(D)
    float lambda;
    const float* lambda_dev;
    int lambda_bf16;            // it points to a bf16, and so does dlambda
    const int32_t* lengths;     // [B], nullptr: Tk each
    uint32_t* status;
    const void* q1; const void* k1; const void* q2; const void* k2; const void* v;
    void* out;
    int64_t s_q1[3], s_k1[3], s_q2[3], s_k2[3], s_v[3], s_o[3];
    int norm;                   // the output epilogue
    float norm_eps;
    const float* norm_weight;
    const float* norm_bias;
    float out_scale;
    void* out2;                 // training: A_2 V with out's strides,
    float* lse;                 // and [B, H, Tq, 2] log-sum-exps (natural), -inf without a key
    void* rests;                // bf16: dense [2][B, H, Tq, Dv], what the rounding of out and out2 left; or nullptr
    // backward
    const void* dout;
    int64_t s_do[3];
    void* dq1; void* dq2; void* dk1; void* dk2; void* dv;   // nullptr: not wanted
    float* stats;               // [B, H, Tq, 4]: log-sum-exps, Dd_1, Dd_2
    void* dlambda;              // nullptr: not wanted
    float* lambda_parts;        // [kLambdaBlocks]
    uint32_t* counters;         // two of items, then one of dlambda's blocks
};

#ifdef __CUDACC__
// A sequence's states, and whether its length is outside 0 .. Tk (then 0 states, and
// everything of the sequence is NaN).
struct CrossLen {
    int n;
    bool bad;
};
__device__ __forceinline__ CrossLen cross_len(const int32_t* lengths, int b, int Tk) {
    const int n = lengths ? __ldg(lengths + b) : Tk;
    const bool bad = n < 0 || n > Tk;
    return {bad ? 0 : n, bad};
}
#endif

// Parameters of the tensor-core backward (bf16, Dv = 128, D = 64, or 128 with one key tensor).
struct CrossTcParams {
    int B, H, Hk, group, Tq, Tk;
    int nq128, nq64, nk128;     // tiles along Tq and Tk
    int group_q, group_k;       // heads, and key/value heads, that are worked on at a time
    int k_shared;
    float scale, scale_log2;
    float lambda;
    const float* lambda_dev;
    int lambda_bf16;
    const int32_t* lengths;
    uint32_t* status;
    uint32_t* sched;            // 2 item counters, and dlambda's
    const __nv_bfloat16* out; const __nv_bfloat16* out2; const __nv_bfloat16* dout;
    const __nv_bfloat16* rests; // [2][B, H, Tq, 128] of out and out2, or nullptr
    int64_t s_o[3], s_do[3];
    const float* lse;
    float* stats;               // rows of -lse_1, -lse_2 (log2), -Dd_1, -Dd_2
    int splits;                 // of the query rows of a tile of states
    float* parts;               // [splits][B, Hk, Tk][256] where there are several
    void* dq1; void* dq2; void* dk1; void* dk2; void* dv;
};
// How many splits, for sizes alone.
int cross_bwd_splits(int64_t B, int64_t Hk, int64_t group, int64_t Tq, int64_t Tk);
int launch_cross_bwd_tc(const CUtensorMap* maps /*dq: q1,k1,q2,k2,v,do; dkdv: the same*/, const CrossTcParams& p,
                        int head_dim, int num_sms, cudaStream_t stream);

// dlambda = sign * (the sum of the rows' last statistic), after either backward.
constexpr int kLambdaBlocks = 128;
int launch_cross_dlambda(const CrossParams& p, float sign, cudaStream_t stream);

// The CUDA-core kernels: any D <= 128, Dv <= 256, type and layout.
int launch_cross_simt(const CrossParams& p, cudaStream_t stream);
int launch_cross_simt_bwd(const CrossParams& p, cudaStream_t stream);

}  // namespace diffattn
