// C ABI entry points of the readout operators: group norm, dropout, cross attention.
// Host-side checks only; the kernels are in group_norm.hip, dropout.hip and cross_attn_*.hip.
#include "capi_readout.hpp"

using namespace oeq::capi;

namespace {

oeq_status check_structures(int64_t n_rows, int32_t n_struct, const int32_t *ptr) {
    if (n_rows < 0 || n_struct < 0) return fail(OEQ_ERR_INVALID_ARG, "negative size");
    if (n_rows >= kMaxRows) return fail(OEQ_ERR_UNSUPPORTED, "rows must fit int32");
    if (n_struct == 0 && n_rows != 0) return fail(OEQ_ERR_INVALID_ARG, "rows without structures");
    if (n_struct > 0) {
        if (!ptr) return fail(OEQ_ERR_INVALID_ARG, "the row pointer is NULL");
        OEQ_TRY(check_aligned(ptr, 4, "the row pointer"));
    }
    return OEQ_OK;
}

// ---- group norm -----------------------------------------------------------------------

oeq_status check_groups(int64_t n_rows, int32_t n_struct, int32_t channels, int32_t groups) {
    if (n_rows < 0 || n_struct < 0) return fail(OEQ_ERR_INVALID_ARG, "negative size");
    if (n_rows >= kMaxRows) return fail(OEQ_ERR_UNSUPPORTED, "rows must fit int32");
    if (channels < 1 || groups < 1 || channels % groups)
        return fail(OEQ_ERR_INVALID_ARG, "n_groups must divide n_channels");
    if (channels / groups > 2048) return fail(OEQ_ERR_UNSUPPORTED, "more than 2048 channels in a group");
    if (ro::group_norm_blocks(n_rows, n_struct, channels, groups) >= (int64_t(1) << 24))
        return fail(OEQ_ERR_UNSUPPORTED, "too many structures, groups or channels for one launch");
    return OEQ_OK;
}

oeq_status check_group_norm(oeq_dtype dtype, oeq_act act, const ro::GroupNormArgs &a) {
    OEQ_TRY(check_dtype(dtype));
    if (act != OEQ_ACT_NONE && act != OEQ_ACT_SILU) return fail(OEQ_ERR_INVALID_ARG, "unknown activation");
    OEQ_TRY(check_structures(a.rows, a.n_struct, a.ptr));
    OEQ_TRY(check_groups(a.rows, a.n_struct, a.channels, a.groups));
    if (a.rows > 0 && !a.x) return fail(OEQ_ERR_INVALID_ARG, "x is NULL");
    if (a.n_struct > 0 && (!a.mean || !a.rstd)) return fail(OEQ_ERR_INVALID_ARG, "mean or rstd is NULL");
    if (a.ld_x < a.channels) return fail(OEQ_ERR_INVALID_ARG, "the row stride of x is below n_channels");
    OEQ_TRY(check_aligned(a.x, element_size(dtype), "x"));
    return OEQ_OK;
}

// ---- dropout ------------------------------------------------------------------------------

oeq_status run_dropout(oeq_dtype dtype, ro::DropoutArgs a, double p, hipStream_t stream) {
    OEQ_TRY(check_dtype(dtype));
    if (a.rows < 0 || a.cols < 0) return fail(OEQ_ERR_INVALID_ARG, "negative size");
    if (a.rows >> 32 || a.cols >= kMaxRows)
        return fail(OEQ_ERR_UNSUPPORTED, "rows must be below 2^32 and columns below 2^31");
    OEQ_TRY(drop_of(p, &a.threshold, &a.scale));
    if (!a.rng) return fail(OEQ_ERR_INVALID_ARG, "rng is NULL");
    OEQ_TRY(check_aligned(a.rng, 8, "rng"));
    if (a.rows == 0 || a.cols == 0) return OEQ_OK;
    if (!a.x || !a.out) return fail(OEQ_ERR_INVALID_ARG, "an input or output is NULL");
    if (a.ld_x < a.cols || a.ld_out < a.cols || (a.residual && a.ld_residual < a.cols))
        return fail(OEQ_ERR_INVALID_ARG, "a row stride is below n_cols");
    const size_t es = element_size(dtype);
    OEQ_TRY(check_aligned(a.x, es, "the input"));
    OEQ_TRY(check_aligned(a.out, es, "the output"));
    OEQ_TRY(check_aligned(a.residual, es, "residual"));
    return from_hip(ro::dropout(dtype, a, stream), "dropout");
}

}  // namespace

extern "C" {

oeq_status oeq_group_norm_workspace_size(int64_t n_rows, int32_t n_struct, int32_t n_channels, int32_t n_groups,
                                         size_t *fwd_bytes, size_t *bwd_bytes) {
    return guarded([&]() -> oeq_status {
        OEQ_TRY(check_groups(n_rows, n_struct, n_channels, n_groups));
        const ro::GroupNormBytes need = ro::group_norm_workspace(n_rows, n_struct, n_channels, n_groups);
        if (fwd_bytes) *fwd_bytes = need.fwd;
        if (bwd_bytes) *bwd_bytes = need.bwd;
        return OEQ_OK;
    });
}

oeq_status oeq_group_norm_fwd(oeq_dtype dtype, int64_t n_rows, int32_t n_struct, int32_t n_channels, int32_t n_groups,
                              oeq_act act, double eps, const int32_t *ptr, const void *x, int64_t x_stride,
                              const float *weight, const float *bias, void *out, int64_t out_stride, float *mean,
                              float *rstd, void *workspace, size_t workspace_bytes, void *stream) {
    return guarded([&]() -> oeq_status {
        ro::GroupNormArgs a{};
        a.rows = n_rows, a.n_struct = n_struct, a.channels = n_channels, a.groups = n_groups;
        a.silu = act == OEQ_ACT_SILU, a.ptr = ptr, a.x = x, a.ld_x = x_stride, a.weight = weight, a.bias = bias;
        a.eps = static_cast<float>(eps), a.mean = mean, a.rstd = rstd, a.out = out, a.ld_out = out_stride;
        a.workspace = workspace;
        OEQ_TRY(check_group_norm(dtype, act, a));
        if (!(a.eps > 0.f) || !std::isfinite(a.eps)) return fail(OEQ_ERR_INVALID_ARG, "eps must be positive");
        if (n_rows > 0 && !out) return fail(OEQ_ERR_INVALID_ARG, "out is NULL");
        if (out_stride < n_channels) return fail(OEQ_ERR_INVALID_ARG, "the row stride of out is below n_channels");
        OEQ_TRY(check_aligned(out, element_size(dtype), "out"));
        if (n_struct == 0) return OEQ_OK;
        const ro::GroupNormBytes need = ro::group_norm_workspace(n_rows, n_struct, n_channels, n_groups);
        OEQ_TRY(check_workspace(workspace, workspace_bytes, need.fwd));
        return from_hip(ro::group_norm_fwd(dtype, a, static_cast<hipStream_t>(stream)), "group norm");
    });
}

oeq_status oeq_group_norm_bwd(oeq_dtype dtype, int64_t n_rows, int32_t n_struct, int32_t n_channels, int32_t n_groups,
                              oeq_act act, const int32_t *ptr, const void *x, int64_t x_stride, const float *weight,
                              const float *bias, const float *mean, const float *rstd, const void *grad_out,
                              int64_t grad_out_stride, void *grad_x, int64_t grad_x_stride, float *grad_weight,
                              float *grad_bias, void *workspace, size_t workspace_bytes, void *stream) {
    return guarded([&]() -> oeq_status {
        ro::GroupNormArgs a{};
        a.rows = n_rows, a.n_struct = n_struct, a.channels = n_channels, a.groups = n_groups;
        a.silu = act == OEQ_ACT_SILU, a.ptr = ptr, a.x = x, a.ld_x = x_stride, a.weight = weight, a.bias = bias;
        a.mean = const_cast<float *>(mean), a.rstd = const_cast<float *>(rstd);
        a.grad_out = grad_out, a.ld_grad_out = grad_out_stride, a.grad_x = grad_x, a.ld_grad_x = grad_x_stride;
        a.grad_weight = grad_weight, a.grad_bias = grad_bias, a.workspace = workspace;
        OEQ_TRY(check_group_norm(dtype, act, a));
        if (n_rows > 0 && !grad_out) return fail(OEQ_ERR_INVALID_ARG, "grad_out is NULL");
        if (grad_out_stride < n_channels || (grad_x && grad_x_stride < n_channels))
            return fail(OEQ_ERR_INVALID_ARG, "a gradient's row stride is below n_channels");
        OEQ_TRY(check_aligned(grad_out, element_size(dtype), "grad_out"));
        OEQ_TRY(check_aligned(grad_x, element_size(dtype), "grad_x"));
        if (!grad_x && !grad_weight && !grad_bias) return OEQ_OK;
        const ro::GroupNormBytes need = ro::group_norm_workspace(n_rows, n_struct, n_channels, n_groups);
        OEQ_TRY(check_workspace(workspace, workspace_bytes, need.bwd));
        return from_hip(ro::group_norm_bwd(dtype, a, static_cast<hipStream_t>(stream)), "group norm backward");
    });
}

oeq_status oeq_dropout_fwd(oeq_dtype dtype, int64_t n_rows, int64_t n_cols, const void *x, int64_t x_stride,
                           const void *residual, int64_t residual_stride, double p, const int64_t *rng, void *out,
                           int64_t out_stride, void *stream) {
    return guarded([&]() -> oeq_status {
        ro::DropoutArgs a{};
        a.rows = n_rows, a.cols = n_cols, a.x = x, a.ld_x = x_stride, a.residual = residual;
        a.ld_residual = residual_stride, a.rng = rng, a.out = out, a.ld_out = out_stride;
        return run_dropout(dtype, a, p, static_cast<hipStream_t>(stream));
    });
}

oeq_status oeq_dropout_bwd(oeq_dtype dtype, int64_t n_rows, int64_t n_cols, const void *grad_out,
                           int64_t grad_out_stride, double p, const int64_t *rng, void *grad_x, int64_t grad_x_stride,
                           void *stream) {
    return guarded([&]() -> oeq_status {
        ro::DropoutArgs a{};
        a.rows = n_rows, a.cols = n_cols, a.x = grad_out, a.ld_x = grad_out_stride;
        a.rng = rng, a.out = grad_x, a.ld_out = grad_x_stride;
        return run_dropout(dtype, a, p, static_cast<hipStream_t>(stream));
    });
}

oeq_status oeq_cross_attn_workspace_size(const oeq_attn_desc *desc, size_t *fwd_bytes, size_t *bwd_bytes) {
    return guarded([&]() -> oeq_status {
        ro::AttnArgs a;
        OEQ_TRY(attn_args(desc, &a, ro::cross_attn_fwd_blocks, ro::cross_attn_bwd_blocks));
        if (fwd_bytes) *fwd_bytes = a.n_struct && a.q_rows ? ro::cross_attn_fwd_workspace(desc->dtype, a) : 0;
        if (bwd_bytes) *bwd_bytes = a.n_struct ? ro::cross_attn_bwd_workspace(desc->dtype, a) : 0;
        return OEQ_OK;
    });
}

oeq_status oeq_cross_attn_fwd(const oeq_attn_desc *desc, const int32_t *q_ptr, const int32_t *k_ptr, const void *q,
                              const void *k, const void *v, const uint8_t *key_mask, const int64_t *rng, void *out,
                              float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    return guarded([&]() -> oeq_status {
        ro::AttnArgs a;
        OEQ_TRY(attn_args(desc, &a, ro::cross_attn_fwd_blocks, ro::cross_attn_bwd_blocks));
        OEQ_TRY(attn_operands(&a, q_ptr, k_ptr, q, k, v, key_mask, rng));
        if (a.q_rows == 0) return OEQ_OK;
        if (!out || !lse) return fail(OEQ_ERR_INVALID_ARG, "out or lse is NULL");
        OEQ_TRY(check_aligned(out, 16, "out"));
        OEQ_TRY(check_aligned(lse, 4, "lse"));
        OEQ_TRY(check_workspace(workspace, workspace_bytes, ro::cross_attn_fwd_workspace(desc->dtype, a)));
        a.out = out, a.lse = lse, a.workspace = workspace;
        return from_hip(ro::cross_attn_fwd(desc->dtype, a, static_cast<hipStream_t>(stream)), "cross attention");
    });
}

oeq_status oeq_cross_attn_bwd(const oeq_attn_desc *desc, const int32_t *q_ptr, const int32_t *k_ptr, const void *q,
                              const void *k, const void *v, const uint8_t *key_mask, const int64_t *rng,
                              const void *out, const float *lse, const void *grad_out, void *grad_q, void *grad_k,
                              void *grad_v, void *workspace, size_t workspace_bytes, void *stream) {
    return guarded([&]() -> oeq_status {
        ro::AttnArgs a;
        OEQ_TRY(attn_args(desc, &a, ro::cross_attn_fwd_blocks, ro::cross_attn_bwd_blocks));
        OEQ_TRY(attn_operands(&a, q_ptr, k_ptr, q, k, v, key_mask, rng));
        if (a.q_rows && (!out || !lse || !grad_out)) return fail(OEQ_ERR_INVALID_ARG, "out, lse or grad_out is NULL");
        for (const void *p : {out, grad_out, static_cast<const void *>(grad_q), static_cast<const void *>(grad_k),
                              static_cast<const void *>(grad_v)})
            OEQ_TRY(check_aligned(p, 16, "out, grad_out and the gradients"));
        OEQ_TRY(check_aligned(lse, 4, "lse"));
        if (a.n_struct == 0 || (!grad_q && !grad_k && !grad_v)) return OEQ_OK;
        OEQ_TRY(check_workspace(workspace, workspace_bytes, ro::cross_attn_bwd_workspace(desc->dtype, a)));
        a.out = const_cast<void *>(out), a.lse = const_cast<float *>(lse), a.grad_out = grad_out;
        a.grad_q = grad_q, a.grad_k = grad_k, a.grad_v = grad_v, a.workspace = workspace;
        return from_hip(ro::cross_attn_bwd(desc->dtype, a, static_cast<hipStream_t>(stream)),
                        "cross attention backward");
    });
}

}  // extern "C"
