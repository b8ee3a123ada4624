// Launchers of the readout operators (group_norm.hip, dropout.hip, cross_attn_*.hip),
// called by capi_readout.cpp with checked arguments.
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

struct AttnArgs {
    int32_t n_struct, heads, kv_heads, share;  // share = heads / kv_heads
    int32_t dim;
    int64_t q_rows, k_rows;
    const int32_t *q_ptr, *k_ptr;
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

}  // namespace readout
}  // namespace oeq
