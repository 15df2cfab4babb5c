// block.h -- internal interface of the operators of a cross-attention block: attention over
// an encoder's states and the norm of each head's output.  Not part of the public ABI.
#pragma once

#include <cstdint>
#include <cuda.h>
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

}  // namespace diffattn
