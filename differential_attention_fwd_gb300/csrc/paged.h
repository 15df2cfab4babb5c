// paged.h -- internal interface of the operators around a paged key/value cache:
// norm and rotation of queries and keys, appending to the cache, and attention over
// it.  Not part of the public ABI.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "diffattn.h"

namespace diffattn {

// What a stream of head rows is for.
enum : int {
    kRowsDense = 0,     // norm and rotation, dense rows out
    kRowsPaged = 1,     // norm and rotation into the paged cache
    kRowsCopy = 2,      // values: copied into the paged cache
};

// One tensor of head rows that the rotation kernel walks: x [B, heads, T, width]
// by strides; y by strides (dense: [0] = B, [1] = head, [2] = T; paged: [0] = page,
// [1] = head, [2] = slot in the page).
struct RowStream {
    const void* x;
    void* y;
    int64_t sx[3], sy[3];
    int heads, width, kind;
    const float* weight;        // [D] or [heads, D], nullptr = 1
    int64_t w_stride;           // 0 or D
    // backward only: gradient of y (strides sg), and where y above takes dx
    const void* g;
    int64_t sg[3];
    int grad_slot;              // 0: q weight, 1: k weight
};

// Division of numbers below 2^31 by a divisor that the host knows.
struct FastDiv {
    uint32_t mul;
    int shift;
    void set(uint32_t d) {
        shift = 0;
        while ((1ull << shift) < d) ++shift;
        mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int div(int n) const {
        return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift);
    }
#endif
};

struct RotaryParams {
    RowStream s[4];
    int n;                      // streams
    int B, T, D, R;             // R rotated elements of each row (0: none)
    FastDiv by_T, by_heads;
    int bf16, interleaved, norm;
    float eps, inv_D;
    const float* cos;           // [table_rows, R / 2]
    const float* sin;
    int64_t table_rows;
    const void* pos;            // nullptr: the slot (paged) or t
    int pos64;
    int64_t pos_stride[2];      // B, T
    int axes;                   // 0: a position a token; else so many, the pairs in sections,
    int axis_end[DIFFATTN_MAX_AXES];    // each turned by its own axis's: where they end
    int64_t axis_stride;        // of a token's positions
    // the paged cache
    const int32_t* lengths;     // [B] tokens before the call
    const int32_t* new_lengths; // [B] or nullptr (T each)
    const int32_t* table;       // [B, max_pages]
    int64_t table_stride;
    int64_t max_pages, num_pages, page;
    uint32_t* status;
    int fast;                   // 16-byte rows: the vector kernel
    int heads_per_block;
    int head_blocks;            // of all streams (backward, vector kernel: blocks in all)
    // backward
    int chunks;                 // of the tokens
    int heads;                  // of all streams
    float* partial;             // [chunks][heads][D]
    float* dw[2];               // q and k weight gradients, nullptr: not wanted
    int64_t dw_stride[2];       // 0: [D], summed over heads; D: [heads, D]
};

int launch_rotary(const RotaryParams& p, cudaStream_t stream);
int launch_rotary_bwd(const RotaryParams& p, cudaStream_t stream);
// Heads a block walks, and the blocks along tokens and heads, for p's sizes.
void plan_rotary(RotaryParams* p, int num_sms);
void plan_rotary_bwd(RotaryParams* p, int num_sms);
// Floats of the weight gradients' partial rows, at most, for `heads` heads in all.
size_t rotary_bwd_floats(int64_t B, int64_t T, int64_t D, int64_t heads);

// A unit that worker c started and did not finish, for the merging pass: its parts are
// in slots 2 c + 1, 2 (c + 1), ... 2 (c + parts - 1).  parts = 0: there is none.
struct alignas(16) PagedJoin {
    int parts, b, unit, n_new;
};

// Attention over the paged cache.
struct PagedParams {
    int B, H, Hk, group, Tq, D, Dv;
    int bf16;
    int k_shared;
    int page;                   // slots of a page
    int64_t max_pages, num_pages;
    const void* q1; const void* q2;
    const void* k1; const void* k2; const void* v;
    void* out;
    int64_t s_q1[3], s_q2[3], s_o[3];
    int64_t s_k1[3], s_k2[3], s_v[3];   // page, head, slot
    const int32_t* table;       // nullptr: sequence b is page b
    int64_t table_stride;
    const int32_t* lengths;
    int cross;                  // over an encoder's states: every row sees the lengths[b] keys (nullptr: a
                                // page's) and no other
    const int32_t* q_lengths;   // nullptr: Tq each
    const uint8_t* mask;        // tree: [B, Tq, Tq] bytes, nullptr: causal
    int64_t mask_stride[2];
    float scale_log2, lambda;
    const float* lambda_dev;
    int lambda_bf16;            // it points to a bf16
    int norm;
    float norm_eps;
    const float* norm_weight;
    const float* norm_bias;
    float out_scale;
    uint32_t* status;
    // The query rows of a key/value head: its heads' head_rows rows each, Tq or more
    // (then the rest is padding), cut into row_chunks units of chunk_rows.
    int head_rows;
    int row_chunks;
    int chunk_rows;
    int vec16;                  // rows of the caches are 16-byte aligned,
    int q16;                    // and of the queries
    int o4, o16;                // output rows are 4-byte, 16-byte aligned
    int solo_workers;           // warps of the launch: one is a worker where units are many
    int workers;                // that share the first pass, at most
    int sparse_joins;           // a quarter of them may be all there are
    int zero_rest;              // rows past a sequence's queries are zeroed
    int join_block, join_step;  // merging pass: its block b takes words b join_block + k join_step
    float* part;                // [2 * workers][chunk_rows][paged_part_floats(Dv)]
    struct PagedJoin* joins;    // [workers] what the merging pass has to do
};

// Floats of one row's partial result: m_1, l_1, m_2, l_2, O_1 and O_2, each O's width
// rounded up to even so that rows stay 16-byte aligned.
__host__ __device__ constexpr int paged_part_width(int Dv) { return (Dv + 1) / 2 * 2; }
__host__ __device__ constexpr int paged_part_floats(int Dv) { return 4 + 2 * paged_part_width(Dv); }

int launch_paged_simt(const PagedParams& p, cudaStream_t stream);
// Rows of a unit of the CUDA-core kernel, for `rows` query rows a key/value head.
int paged_simt_rows(int64_t rows);
constexpr int kSimtBlocksPerSm = 4;
// Blocks of it that an SM holds at once (elements of `es` bytes, `rows` of a unit).
int paged_simt_blocks(int D, int Dv, int es, int rows);
// The tensor-core kernel of up to 16 rows a unit: maps of K1, K2 and V with boxes of
// 64 columns x 16 slots.
constexpr int kMmaRows = 16;
constexpr int kMmaTile = 64;
constexpr int kMmaWarps = 4;            // of a block: as many workers, or one
constexpr int kMmaBlocks = 2;           // an SM
// Most rows of a unit that one warp takes alone (their queries are in its shared memory).
__host__ __device__ constexpr int paged_solo_rows(int D) { return D == 64 ? 8 : 4; }
int launch_paged_mma(const CUtensorMap* maps, const PagedParams& p, cudaStream_t stream);
// The tcgen05 kernel of up to 128 rows a unit: maps of K1, K2, V (boxes of 64 columns x
// box_rows slots), Q1 and Q2 (boxes of 64 columns x q_box tokens).
constexpr int kTcRows = 128;
constexpr int kTcTile = 64;
int launch_paged_tc(const CUtensorMap* maps, const PagedParams& p, int box_rows, int q_box, cudaStream_t stream);
// Merges the partial results of the units that several blocks share.
int launch_paged_combine(const PagedParams& p, cudaStream_t stream);

// Attention over an encoder's states on the kernels of the paged cache (api_paged.cu): whether they
// take the sizes, the workspace for them, and the call (k, v: the states, as pages of Tk slots).
bool cross_paged_ok(const diffattn_cross_desc& d);
size_t cross_paged_bytes(const diffattn_cross_desc& d);
int cross_paged(const diffattn_cross_desc& d, const void* q1, const void* k1, const void* q2, const void* k2,
                const void* v, const int32_t* lengths, float lambda, const float* lambda_dev,
                const diffattn_epilogue& e, void* out, void* workspace, size_t workspace_bytes, cudaStream_t stream);

// Checks an output epilogue and fills in what a NULL one means (api.cu).
int check_epilogue(const diffattn_epilogue* epi, diffattn_epilogue* e);
// The C-ABI layer's view of the current device (api.cu).
int device_info(uint32_t** status, int* num_sms);
// 4-D bf16 tensor map with 128-byte swizzling: dims {inner, rows, heads, outer},
// element strides {outer, heads, rows} as in the descriptors.
int encode_map_4d(CUtensorMap* m, const void* base, const int64_t dims[4], const int64_t s[3],
                  uint32_t box_inner, uint32_t box_rows);

}  // namespace diffattn
