// tile_softmax.cuh -- one thread's share of a 64-key score tile (a query row): the row
// maximum, and the weights with their sum.  Shared by the forward and the attention over
// a paged cache.
#pragma once

#include "ptx.cuh"

namespace diffattn {
namespace tc {

// Row max of one thread's 64 scores (four independent chains of
// three-input maxima).
__device__ __forceinline__ float tile_row_max(const float (&s)[64]) {
    float mx0 = s[0], mx1 = s[1], mx2 = s[2], mx3 = s[3];
#pragma unroll
    for (int c = 4; c < 60; c += 8) {
        mx0 = fmax3(mx0, s[c], s[c + 1]);
        mx1 = fmax3(mx1, s[c + 2], s[c + 3]);
        mx2 = fmax3(mx2, s[c + 4], s[c + 5]);
        mx3 = fmax3(mx3, s[c + 6], s[c + 7]);
    }
    mx0 = fmax3(mx0, s[60], s[61]);
    mx1 = fmax3(mx1, s[62], s[63]);
    return fmax3(mx0, mx1, fmaxf(mx2, mx3));
}

// P = 2^(s * scale_log2 - m) for one thread's 64 scores, two columns per
// packed operation: P rounded to bf16 pairs into pk, and the sum of the
// unrounded P returned.
__device__ __forceinline__ float tile_exp2(const float (&s)[64], float sl2, float m, uint32_t (&pk)[32]) {
    const uint64_t scale2 = f2_pack(sl2, sl2);
    const uint64_t negm2 = f2_pack(-m, -m);
    uint64_t rsum[4] = {0, 0, 0, 0};     // four short addition chains
#pragma unroll
    for (int c = 0; c < 32; ++c) {
        const uint64_t x = f2_fma(f2_pack(s[2 * c], s[2 * c + 1]), scale2, negm2);
        const float p0 = ex2_approx(f2_lo(x));
        const float p1 = ex2_approx(f2_hi(x));
        rsum[c & 3] = f2_add(rsum[c & 3], f2_pack(p0, p1));
        pk[c] = pack_bf16x2(p0, p1);
    }
    const uint64_t r = f2_add(f2_add(rsum[0], rsum[1]), f2_add(rsum[2], rsum[3]));
    return f2_lo(r) + f2_hi(r);
}

}  // namespace tc
}  // namespace diffattn
