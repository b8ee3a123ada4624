// Launchers of the readout operators (group_norm.hip, dropout.hip, cross_attn_*.hip) and of the decoder
// operators (embedding.hip, rms_norm.hip, causal_attn_*.hip), called by capi_readout.cpp and
// capi_decoder.cpp with checked arguments.
#pragma once

#include <cstddef>
#include <cstdint>

#include <hip/hip_runtime.h>

#include "oeq.h"

namespace oeq {
namespace readout {

struct DropoutArgs {
    int64_t rows, cols;
    const void *x, *residual;  // residual may be NULL
    void *out;
    int64_t ld_x, ld_residual, ld_out;
    uint32_t threshold;
    float scale;
    const int64_t *rng;
};
hipError_t dropout(oeq_dtype dtype, const DropoutArgs &a, hipStream_t stream);

struct GroupNormArgs {
    int64_t rows;
    int32_t n_struct, channels, groups, silu;
    const int32_t *ptr;
    const void *x;
    int64_t ld_x;
    const float *weight, *bias;  // either may be NULL (ones, zeros)
    float eps;
    float *mean, *rstd;  // written by the forward, read by the backward
    void *out;           // forward
    int64_t ld_out;
    const void *grad_out;  // backward
    int64_t ld_grad_out;
    void *grad_x;
    int64_t ld_grad_x;
    float *grad_weight, *grad_bias;
    void *workspace;
};
struct GroupNormBytes {
    size_t fwd, bwd;
};
// Workspace bytes, and the workgroups of the largest launch.
GroupNormBytes group_norm_workspace(int64_t rows, int32_t n_struct, int32_t channels, int32_t groups);
int64_t group_norm_blocks(int64_t rows, int32_t n_struct, int32_t channels, int32_t groups);
hipError_t group_norm_fwd(oeq_dtype dtype, const GroupNormArgs &a, hipStream_t stream);
hipError_t group_norm_bwd(oeq_dtype dtype, const GroupNormArgs &a, hipStream_t stream);

struct EmbeddingArgs {
    int64_t table_rows, cols, rows;
    const void *index;
    int wide;  // the index has 64 bits, else 32
    float scale;
    const void *table;  // forward
    int64_t ld_table;
    void *out;
    int64_t ld_out;
    const void *grad_out;  // backward
    int64_t ld_grad_out;
    void *grad_table;
    int64_t ld_grad_table;
    void *workspace;
};
// Workspace bytes of the backward, and the workgroups of its largest launch.
size_t embedding_workspace(int64_t table_rows, int64_t cols, int64_t rows);
int64_t embedding_blocks(int64_t table_rows, int64_t cols, int64_t rows);
hipError_t embedding_fwd(oeq_dtype dtype, const EmbeddingArgs &a, hipStream_t stream);
hipError_t embedding_bwd(oeq_dtype dtype, const EmbeddingArgs &a, hipStream_t stream);

constexpr int64_t kRmsMostCols = 16384;
struct RmsNormArgs {
    int64_t rows;
    int32_t cols;
    float eps;
    const void *x, *residual;  // forward; residual may be NULL
    int64_t ld_x, ld_residual;
    const float *weight;  // may be NULL (ones)
    void *sum;            // written by the forward where there is a residual; read by the backward
    int64_t ld_sum;
    void *out;
    int64_t ld_out;
    float *out_scale;  // not NULL: out is e4m3, with a scale a row
    float *rstd;       // written by the forward (may be NULL), read by the backward
    const void *grad_out, *grad_sum;  // backward; grad_sum may be NULL
    int64_t ld_grad_out, ld_grad_sum;
    void *grad_x;  // may be NULL
    int64_t ld_grad_x;
    float *grad_weight;  // may be NULL
    void *workspace;
};
// Workspace bytes of the backward, and the workgroups of the forward.
size_t rms_norm_workspace(int64_t rows, int32_t cols);
int64_t rms_norm_blocks(int64_t rows, int32_t cols);
hipError_t rms_norm_fwd(oeq_dtype dtype, const RmsNormArgs &a, hipStream_t stream);
hipError_t rms_norm_bwd(oeq_dtype dtype, const RmsNormArgs &a, hipStream_t stream);

struct AttnArgs {
    int32_t n_struct, heads, kv_heads, share;  // share = heads / kv_heads
    int32_t dim;
    int64_t q_rows, k_rows;
    const int32_t *q_ptr, *k_ptr;
    const int32_t *k_len;     // causal forward: states in use of each structure; may be NULL (all)
    const uint8_t *key_mask;  // may be NULL
    const void *q, *k, *v;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head;  // strides
    float scale;
    uint32_t threshold;  // of the dropout; 0: none
    float keep_scale;
    const int64_t *rng;
    void *out;  // written by the forward, read by the backward
    float *lse;
    const void *grad_out;  // backward
    void *grad_q, *grad_k, *grad_v;
    void *workspace;
};
// Workspace bytes and the workgroups of the largest launch of each direction.
size_t cross_attn_fwd_workspace(oeq_dtype dtype, const AttnArgs &a);
size_t cross_attn_bwd_workspace(oeq_dtype dtype, const AttnArgs &a);
int64_t cross_attn_fwd_blocks(oeq_dtype dtype, const AttnArgs &a);
int64_t cross_attn_bwd_blocks(oeq_dtype dtype, const AttnArgs &a);
hipError_t cross_attn_fwd(oeq_dtype dtype, const AttnArgs &a, hipStream_t stream);
hipError_t cross_attn_bwd(oeq_dtype dtype, const AttnArgs &a, hipStream_t stream);
// The same with the causal limit.
size_t causal_attn_fwd_workspace(oeq_dtype dtype, const AttnArgs &a);
size_t causal_attn_bwd_workspace(oeq_dtype dtype, const AttnArgs &a);
int64_t causal_attn_fwd_blocks(oeq_dtype dtype, const AttnArgs &a);
int64_t causal_attn_bwd_blocks(oeq_dtype dtype, const AttnArgs &a);
hipError_t causal_attn_fwd(oeq_dtype dtype, const AttnArgs &a, hipStream_t stream);
hipError_t causal_attn_bwd(oeq_dtype dtype, const AttnArgs &a, hipStream_t stream);

}  // namespace readout
}  // namespace oeq
