// C ABI entry points of the decoder operators: embedding, root-mean-square norm, causal attention.
// Host-side checks only; the kernels are in embedding.hip, rms_norm.hip and causal_attn_*.hip.
#include "capi_readout.hpp"

using namespace oeq::capi;

namespace {

constexpr int64_t kMostBlocks = int64_t(1) << 24;  // a launch holds fewer than 2^32 threads

// ---- embedding ------------------------------------------------------------------------------

oeq_status check_embedding_sizes(oeq_dtype dtype, int64_t n_table, int64_t n_cols, int64_t n_rows) {
    OEQ_TRY(check_dtype(dtype));
    if (n_table < 0 || n_cols < 0 || n_rows < 0) return fail(OEQ_ERR_INVALID_ARG, "negative size");
    if (n_table >= kMaxRows || n_rows >= kMaxRows)
        return fail(OEQ_ERR_UNSUPPORTED, "table rows and rows must be below 2^31 - 1");
    if (n_cols >= int64_t(1) << 23)  // the second dimension of a launch counts pieces of 256 columns, to 65535
        return fail(OEQ_ERR_UNSUPPORTED, "columns must be below 2^23");
    if (ro::embedding_blocks(n_table, n_cols, n_rows) >= kMostBlocks)
        return fail(OEQ_ERR_UNSUPPORTED, "too many rows or columns for one launch");
    return OEQ_OK;
}

// What both directions take.
oeq_status embedding_args(oeq_dtype dtype, int64_t n_table, int64_t n_cols, int64_t n_rows, const void *index,
                          int32_t index_bytes, double scale, ro::EmbeddingArgs *a) {
    OEQ_TRY(check_embedding_sizes(dtype, n_table, n_cols, n_rows));
    if (index_bytes != 4 && index_bytes != 8) return fail(OEQ_ERR_INVALID_ARG, "index_bytes must be 4 or 8");
    if (n_rows && !index) return fail(OEQ_ERR_INVALID_ARG, "index is NULL");
    OEQ_TRY(check_aligned(index, static_cast<size_t>(index_bytes), "index"));
    if (!std::isfinite(static_cast<float>(scale))) return fail(OEQ_ERR_INVALID_ARG, "scale must be finite");
    a->table_rows = n_table, a->cols = n_cols, a->rows = n_rows, a->index = index, a->wide = index_bytes == 8;
    a->scale = static_cast<float>(scale);
    return OEQ_OK;
}

// ---- rms norm -------------------------------------------------------------------------------

oeq_status check_rms_sizes(int64_t n_rows, int32_t n_cols) {
    if (n_rows < 0) return fail(OEQ_ERR_INVALID_ARG, "negative size");
    if (n_cols < 1) return fail(OEQ_ERR_INVALID_ARG, "n_cols must be positive");
    if (n_cols > ro::kRmsMostCols) return fail(OEQ_ERR_UNSUPPORTED, "more than 16384 columns");
    if (ro::rms_norm_blocks(n_rows, n_cols) >= kMostBlocks)
        return fail(OEQ_ERR_UNSUPPORTED, "too many rows for one launch");
    return OEQ_OK;
}

// A [rows, n_cols] operand of a call with rows.
oeq_status check_rows(const void *p, int64_t stride, int32_t n_cols, size_t size, const char *name) {
    if (!p) return fail(OEQ_ERR_INVALID_ARG, std::string(name) + " is NULL");
    if (stride < n_cols) return fail(OEQ_ERR_INVALID_ARG, std::string("the row stride of ") + name + " is below n_cols");
    return check_aligned(p, size, name);
}

oeq_status causal_args(const oeq_attn_desc *desc, ro::AttnArgs *a) {
    OEQ_TRY(attn_args(desc, a, ro::causal_attn_fwd_blocks, ro::causal_attn_bwd_blocks));
    // the walks count rows up to a tile of keys past a sequence's last query
    if (desc->q_rows + 256 >= (int64_t(1) << 31) / desc->n_heads)
        return fail(OEQ_ERR_UNSUPPORTED, "query rows times heads must stay 256 rows below 2^31");
    return OEQ_OK;
}

}  // namespace

extern "C" {

oeq_status oeq_embedding_fwd(oeq_dtype dtype, int64_t n_table, int64_t n_cols, int64_t n_rows, const void *table,
                             int64_t table_stride, const void *index, int32_t index_bytes, double scale, void *out,
                             int64_t out_stride, void *stream) {
    return guarded([&]() -> oeq_status {
        ro::EmbeddingArgs a{};
        OEQ_TRY(embedding_args(dtype, n_table, n_cols, n_rows, index, index_bytes, scale, &a));
        if (n_rows == 0 || n_cols == 0) return OEQ_OK;
        if (!out || (n_table && !table)) return fail(OEQ_ERR_INVALID_ARG, "table or out is NULL");
        if (table_stride < n_cols || out_stride < n_cols)
            return fail(OEQ_ERR_INVALID_ARG, "a row stride is below n_cols");
        OEQ_TRY(check_aligned(table, element_size(dtype), "table"));
        OEQ_TRY(check_aligned(out, element_size(dtype), "out"));
        a.table = table, a.ld_table = table_stride, a.out = out, a.ld_out = out_stride;
        return from_hip(ro::embedding_fwd(dtype, a, static_cast<hipStream_t>(stream)), "embedding");
    });
}

oeq_status oeq_embedding_workspace_size(oeq_dtype dtype, int64_t n_table, int64_t n_cols, int64_t n_rows,
                                        size_t *bwd_bytes) {
    return guarded([&]() -> oeq_status {
        OEQ_TRY(check_embedding_sizes(dtype, n_table, n_cols, n_rows));
        if (bwd_bytes) *bwd_bytes = n_table && n_cols ? ro::embedding_workspace(n_table, n_cols, n_rows) : 0;
        return OEQ_OK;
    });
}

oeq_status oeq_embedding_bwd(oeq_dtype dtype, int64_t n_table, int64_t n_cols, int64_t n_rows, const void *index,
                             int32_t index_bytes, double scale, const void *grad_out, int64_t grad_out_stride,
                             void *grad_table, int64_t grad_table_stride, void *workspace, size_t workspace_bytes,
                             void *stream) {
    return guarded([&]() -> oeq_status {
        ro::EmbeddingArgs a{};
        OEQ_TRY(embedding_args(dtype, n_table, n_cols, n_rows, index, index_bytes, scale, &a));
        if (n_table == 0 || n_cols == 0) return OEQ_OK;
        if (!grad_table || (n_rows && !grad_out)) return fail(OEQ_ERR_INVALID_ARG, "grad_out or grad_table is NULL");
        if (grad_out_stride < n_cols || grad_table_stride < n_cols)
            return fail(OEQ_ERR_INVALID_ARG, "a row stride is below n_cols");
        OEQ_TRY(check_aligned(grad_out, element_size(dtype), "grad_out"));
        OEQ_TRY(check_aligned(grad_table, element_size(dtype), "grad_table"));
        OEQ_TRY(check_workspace(workspace, workspace_bytes, ro::embedding_workspace(n_table, n_cols, n_rows)));
        a.grad_out = grad_out, a.ld_grad_out = grad_out_stride, a.grad_table = grad_table;
        a.ld_grad_table = grad_table_stride, a.workspace = workspace;
        return from_hip(ro::embedding_bwd(dtype, a, static_cast<hipStream_t>(stream)), "embedding backward");
    });
}

oeq_status oeq_rms_norm_workspace_size(int64_t n_rows, int32_t n_cols, size_t *bwd_bytes) {
    return guarded([&]() -> oeq_status {
        OEQ_TRY(check_rms_sizes(n_rows, n_cols));
        if (bwd_bytes) *bwd_bytes = ro::rms_norm_workspace(n_rows, n_cols);
        return OEQ_OK;
    });
}

oeq_status oeq_rms_norm_fwd(oeq_dtype dtype, int64_t n_rows, int32_t n_cols, double eps, const void *x,
                            int64_t x_stride, const void *residual, int64_t residual_stride, const float *weight,
                            void *sum, int64_t sum_stride, void *out, int64_t out_stride, float *out_scale,
                            float *rstd, void *stream) {
    return guarded([&]() -> oeq_status {
        OEQ_TRY(check_dtype(dtype));
        OEQ_TRY(check_rms_sizes(n_rows, n_cols));
        const float e = static_cast<float>(eps);
        if (!(e > 0.f) || !std::isfinite(e)) return fail(OEQ_ERR_INVALID_ARG, "eps must be positive");
        if (n_rows == 0) return OEQ_OK;
        const size_t size = element_size(dtype);
        OEQ_TRY(check_rows(x, x_stride, n_cols, size, "x"));
        if (residual) {
            OEQ_TRY(check_rows(residual, residual_stride, n_cols, size, "residual"));
            OEQ_TRY(check_rows(sum, sum_stride, n_cols, size, "sum"));
        }
        OEQ_TRY(check_rows(out, out_stride, n_cols, out_scale ? 1 : size, "out"));
        OEQ_TRY(check_aligned(weight, 4, "weight"));
        OEQ_TRY(check_aligned(out_scale, 4, "out_scale"));
        OEQ_TRY(check_aligned(rstd, 4, "rstd"));
        ro::RmsNormArgs a{};
        a.rows = n_rows, a.cols = n_cols, a.eps = e, a.x = x, a.ld_x = x_stride, a.residual = residual;
        a.ld_residual = residual_stride, a.weight = weight, a.sum = sum, a.ld_sum = sum_stride, a.out = out;
        a.ld_out = out_stride, a.out_scale = out_scale, a.rstd = rstd;
        return from_hip(ro::rms_norm_fwd(dtype, a, static_cast<hipStream_t>(stream)), "rms norm");
    });
}

oeq_status oeq_rms_norm_bwd(oeq_dtype dtype, int64_t n_rows, int32_t n_cols, const void *sum, int64_t sum_stride,
                            const float *weight, const float *rstd, const void *grad_out, int64_t grad_out_stride,
                            const void *grad_sum, int64_t grad_sum_stride, void *grad_x, int64_t grad_x_stride,
                            float *grad_weight, void *workspace, size_t workspace_bytes, void *stream) {
    return guarded([&]() -> oeq_status {
        OEQ_TRY(check_dtype(dtype));
        OEQ_TRY(check_rms_sizes(n_rows, n_cols));
        const size_t size = element_size(dtype);
        if (n_rows) {
            OEQ_TRY(check_rows(sum, sum_stride, n_cols, size, "sum"));
            OEQ_TRY(check_rows(grad_out, grad_out_stride, n_cols, size, "grad_out"));
            if (grad_sum) OEQ_TRY(check_rows(grad_sum, grad_sum_stride, n_cols, size, "grad_sum"));
            if (grad_x) OEQ_TRY(check_rows(grad_x, grad_x_stride, n_cols, size, "grad_x"));
            if (!rstd) return fail(OEQ_ERR_INVALID_ARG, "rstd is NULL");
        }
        OEQ_TRY(check_aligned(weight, 4, "weight"));
        OEQ_TRY(check_aligned(rstd, 4, "rstd"));
        OEQ_TRY(check_aligned(grad_weight, 4, "grad_weight"));
        if (!grad_x && !grad_weight) return OEQ_OK;
        if (grad_weight)
            OEQ_TRY(check_workspace(workspace, workspace_bytes, ro::rms_norm_workspace(n_rows, n_cols)));
        ro::RmsNormArgs a{};
        a.rows = n_rows, a.cols = n_cols, a.sum = const_cast<void *>(sum), a.ld_sum = sum_stride, a.weight = weight;
        a.rstd = const_cast<float *>(rstd), a.grad_out = grad_out, a.ld_grad_out = grad_out_stride;
        a.grad_sum = grad_sum, a.ld_grad_sum = grad_sum_stride, a.grad_x = grad_x, a.ld_grad_x = grad_x_stride;
        a.grad_weight = grad_weight, a.workspace = workspace;
        return from_hip(ro::rms_norm_bwd(dtype, a, static_cast<hipStream_t>(stream)), "rms norm backward");
    });
}

oeq_status oeq_causal_attn_workspace_size(const oeq_attn_desc *desc, size_t *fwd_bytes, size_t *bwd_bytes) {
    return guarded([&]() -> oeq_status {
        ro::AttnArgs a;
        OEQ_TRY(causal_args(desc, &a));
        if (fwd_bytes) *fwd_bytes = a.n_struct && a.q_rows ? ro::causal_attn_fwd_workspace(desc->dtype, a) : 0;
        if (bwd_bytes) *bwd_bytes = a.n_struct ? ro::causal_attn_bwd_workspace(desc->dtype, a) : 0;
        return OEQ_OK;
    });
}

oeq_status oeq_causal_attn_fwd(const oeq_attn_desc *desc, const int32_t *q_ptr, const int32_t *k_ptr,
                               const int32_t *k_len, const void *q, const void *k, const void *v,
                               const uint8_t *key_mask, const int64_t *rng, void *out, float *lse, void *workspace,
                               size_t workspace_bytes, void *stream) {
    return guarded([&]() -> oeq_status {
        ro::AttnArgs a;
        OEQ_TRY(causal_args(desc, &a));
        OEQ_TRY(attn_operands(&a, q_ptr, k_ptr, q, k, v, key_mask, rng));
        OEQ_TRY(check_aligned(k_len, 4, "k_len"));
        if (a.q_rows == 0) return OEQ_OK;
        if (!out || !lse) return fail(OEQ_ERR_INVALID_ARG, "out or lse is NULL");
        OEQ_TRY(check_aligned(out, 16, "out"));
        OEQ_TRY(check_aligned(lse, 4, "lse"));
        OEQ_TRY(check_workspace(workspace, workspace_bytes, ro::causal_attn_fwd_workspace(desc->dtype, a)));
        a.k_len = k_len, a.out = out, a.lse = lse, a.workspace = workspace;
        return from_hip(ro::causal_attn_fwd(desc->dtype, a, static_cast<hipStream_t>(stream)), "causal attention");
    });
}

oeq_status oeq_causal_attn_bwd(const oeq_attn_desc *desc, const int32_t *q_ptr, const int32_t *k_ptr, const void *q,
                               const void *k, const void *v, const uint8_t *key_mask, const int64_t *rng,
                               const void *out, const float *lse, const void *grad_out, void *grad_q, void *grad_k,
                               void *grad_v, void *workspace, size_t workspace_bytes, void *stream) {
    return guarded([&]() -> oeq_status {
        ro::AttnArgs a;
        OEQ_TRY(causal_args(desc, &a));
        OEQ_TRY(attn_operands(&a, q_ptr, k_ptr, q, k, v, key_mask, rng));
        if (a.q_rows && (!out || !lse || !grad_out)) return fail(OEQ_ERR_INVALID_ARG, "out, lse or grad_out is NULL");
        for (const void *p : {out, grad_out, static_cast<const void *>(grad_q), static_cast<const void *>(grad_k),
                              static_cast<const void *>(grad_v)})
            OEQ_TRY(check_aligned(p, 16, "out, grad_out and the gradients"));
        OEQ_TRY(check_aligned(lse, 4, "lse"));
        if (a.n_struct == 0 || (!grad_q && !grad_k && !grad_v)) return OEQ_OK;
        OEQ_TRY(check_workspace(workspace, workspace_bytes, ro::causal_attn_bwd_workspace(desc->dtype, a)));
        a.out = const_cast<void *>(out), a.lse = const_cast<float *>(lse), a.grad_out = grad_out;
        a.grad_q = grad_q, a.grad_k = grad_k, a.grad_v = grad_v, a.workspace = workspace;
        return from_hip(ro::causal_attn_bwd(desc->dtype, a, static_cast<hipStream_t>(stream)),
                        "causal attention backward");
    });
}

}  // extern "C"
