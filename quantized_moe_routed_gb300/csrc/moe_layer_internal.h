// moe_layer_internal.h -- launch interface between the host sides of the layer operators
// (moe_layer.cu, moe_speculate.cu) and their kernels.  Not part of the ABI.
#pragma once
#include "moe_layer.h"
#include "moe_speculate.h"

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace moe {

// moe_norm.cu
struct NormParams {
    const void *x;
    long long x_stride;
    const uint16_t *r;
    uint16_t *r_out;
    const uint16_t *w;
    uint16_t *y;
    uint8_t *q;
    float *q_scale;
    float eps;
    int T, H, x_f32;
};
cudaError_t launch_norm(const NormParams &p, cudaStream_t st);

// moe_linear.cu
struct LinearParams {
    const uint8_t *q, *s;
    const float *ts;
    const uint16_t *x;
    long long x_stride;
    void *y;
    int N, K, T, y_bf16;
};
constexpr int kLinearMaxT = 24;  // tokens of one pass over the weights
cudaError_t launch_linear(const LinearParams &p, int num_sms, cudaStream_t st);

// moe_linear_tc.cu: many rows, K a multiple of 256, s and its rows 16-byte aligned
struct LinearTcPlan {
    int rows, tiles, blocks;  // rows of a tile, tiles of a block, blocks along the rows
};
struct LinearTcParams {
    CUtensorMap tm_q;  // boxes of 128 bytes, swizzled, plan.rows high
    LinearParams l;
    int rows, tiles;
    long long timeout_ns;
};
LinearTcPlan linear_tc_plan(const LinearParams &p, int num_sms);
cudaError_t launch_linear_tc(const LinearTcParams &p, int blocks, cudaStream_t st);

// The cache's pages, and one step's sequences (fields as in moe_layer.h).
struct KvParams {
    CUtensorMap tm_k;  // a page's k as 64 rows of head_dim bytes, swizzled over the row (128 or 64 bytes)
    uint8_t *k, *v;
    float *ks, *vs;
    const float *rope;
    int n_pages, q_heads, kv_heads, D;
    int rot_dim, rot_inter, rope_positions;
    const int32_t *q_off, *kv_len, *pages;
    int max_pages, B, N, max_q;
    uint32_t *ctrl;  // workspace control block: word 2 holds the error bits
};
constexpr uint32_t kErrBadIndex = 16u;

// moe_kv_append.cu
struct AppendParams {
    KvParams c;
    const uint16_t *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    uint16_t *q_out;
    const int32_t *parent = nullptr;  // the new tokens are trees (moe_speculate.h): [N], else null
};
cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t st);

// moe_kv_attend.cu: tiles of 8 or 16 rows
struct AttendParams {
    KvParams c;
    const uint16_t *q;
    uint16_t *o;
    long long q_stride;
    float scale_log2;   // softmax scale times log2(e)
    uint32_t *count;    // [grid] arrivals at the tiles that start in a CTA and end in a later one
    float *part;        // [2 * grid] partial results (attend_part_floats each)
    long long timeout_ns;
    const int32_t *parent = nullptr;  // as in AppendParams
};
constexpr int kAttendMaxRows = 128;  // query rows of the largest tile
__host__ __device__ inline size_t attend_part_floats(int D) { return static_cast<size_t>(kAttendMaxRows) * (D + 2); }
cudaError_t launch_kv_attend_rows(const AttendParams &p, int tile_rows, int num_sms, int smem_optin, cudaStream_t st);
// moe_kv_attend_tc.cu: tiles of 128 rows
cudaError_t launch_kv_attend_tc(const AttendParams &p, int num_sms, cudaStream_t st);

// moe_kv_move.cu
struct CompactParams {
    KvParams c;
    const int32_t *keep, *n_keep;
    int max_keep;
    int32_t *kv_len_out;
};
cudaError_t launch_kv_compact(const CompactParams &p, cudaStream_t st);
struct ForkParams {
    KvParams c;  // kv_len, pages, max_pages, B: the sequences that children go on from
    const int32_t *src, *fresh;
    int C;
    int32_t *kv_len_out, *pages_out;
};
cudaError_t launch_kv_fork(const ForkParams &p, cudaStream_t st);

// moe_sample.cu
cudaError_t launch_sample(const moe_sample_desc &d, int num_sms, cudaStream_t st);

}  // namespace moe
