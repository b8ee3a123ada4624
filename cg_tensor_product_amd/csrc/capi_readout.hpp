// Checks shared by the entry points of the readout and decoder operators (capi_readout.cpp,
// capi_decoder.cpp).  Host-side only.
#pragma once

#include <cmath>
#include <exception>

#include "capi_internal.hpp"
#include "readout.hpp"

namespace oeq {
namespace capi {

namespace ro = oeq::readout;

constexpr int64_t kMaxRows = std::numeric_limits<int32_t>::max();

// No exception leaves a C entry point.
template <class F>
oeq_status guarded(F &&body) noexcept {
    try {
        return body();
    } catch (const std::exception &e) {
        try {
            return fail(OEQ_ERR_HIP, e.what());
        } catch (...) {
            return OEQ_ERR_HIP;
        }
    } catch (...) {
        return OEQ_ERR_HIP;
    }
}

inline size_t element_size(oeq_dtype dtype) { return dtype == OEQ_F32 ? 4 : 2; }

inline oeq_status check_dtype(oeq_dtype dtype) {
    if (dtype != OEQ_F32 && dtype != OEQ_F16 && dtype != OEQ_BF16)
        return fail(OEQ_ERR_UNSUPPORTED, "dtype must be OEQ_F32, OEQ_F16 or OEQ_BF16");
    return OEQ_OK;
}

inline oeq_status check_aligned(const void *p, size_t to, const char *name) {
    if (reinterpret_cast<uintptr_t>(p) % to)
        return fail(OEQ_ERR_INVALID_ARG, std::string(name) + " must be " + std::to_string(to) + "-byte aligned");
    return OEQ_OK;
}

inline oeq_status check_workspace(const void *workspace, size_t have, size_t need) {
    if (need == 0) return OEQ_OK;
    if (!workspace || have < need)
        return fail(OEQ_ERR_WORKSPACE, "workspace must hold " + std::to_string(need) + " bytes");
    if (reinterpret_cast<uintptr_t>(workspace) % kAlign)
        return fail(OEQ_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    return OEQ_OK;
}

inline oeq_status from_hip(hipError_t e, const char *what) {
    if (e == hipSuccess) return OEQ_OK;
    return fail(OEQ_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

#define OEQ_TRY(expr)                          \
    do {                                       \
        const oeq_status st_ = (expr);         \
        if (st_ != OEQ_OK) return st_;         \
    } while (0)

// The drop threshold and the factor of what is kept.
inline oeq_status drop_of(double p, uint32_t *threshold, float *scale) {
    if (!(p >= 0.0 && p < 1.0)) return fail(OEQ_ERR_INVALID_ARG, "the drop probability must be in [0, 1)");
    const double t = std::floor(65536.0 * p + 0.5);
    *threshold = static_cast<uint32_t>(t > 65535.0 ? 65535.0 : t);
    *scale = static_cast<float>(65536.0 / (65536.0 - *threshold));
    return OEQ_OK;
}

// Sizes and types of a descriptor; fills what the launchers take from it.  The functions give the
// workgroups of the largest launch of each direction.
using Blocks = int64_t(oeq_dtype, const ro::AttnArgs &);
inline oeq_status attn_args(const oeq_attn_desc *d, ro::AttnArgs *a, Blocks *fwd_blocks, Blocks *bwd_blocks) {
    if (!d) return fail(OEQ_ERR_INVALID_ARG, "the descriptor is NULL");
    OEQ_TRY(check_dtype(d->dtype));
    if (d->n_struct < 0 || d->q_rows < 0 || d->k_rows < 0) return fail(OEQ_ERR_INVALID_ARG, "negative size");
    if (d->n_heads < 1 || d->n_kv_heads < 1 || d->n_heads % d->n_kv_heads)
        return fail(OEQ_ERR_INVALID_ARG, "n_kv_heads must divide n_heads");
    if (d->head_dim < 1) return fail(OEQ_ERR_INVALID_ARG, "head_dim must be positive");
    if (d->head_dim % 8 || d->head_dim > 128)
        return fail(OEQ_ERR_UNSUPPORTED, "head_dim must be a multiple of 8 and at most 128");
    if (d->n_struct == 0 && (d->q_rows || d->k_rows)) return fail(OEQ_ERR_INVALID_ARG, "rows without structures");
    constexpr int64_t most = int64_t(1) << 31;
    if (d->q_rows >= most / d->n_heads || d->k_rows >= most - 1024)
        return fail(OEQ_ERR_UNSUPPORTED, "query rows times heads, and states, must be below 2^31");
    if (!(d->scale > 0.0) || !std::isfinite(static_cast<float>(d->scale)) || !(static_cast<float>(d->scale) > 0.f))
        return fail(OEQ_ERR_INVALID_ARG, "scale must be positive and finite");
    *a = ro::AttnArgs{};
    a->n_struct = d->n_struct, a->heads = d->n_heads, a->kv_heads = d->n_kv_heads;
    a->share = d->n_heads / d->n_kv_heads, a->dim = d->head_dim, a->q_rows = d->q_rows, a->k_rows = d->k_rows;
    a->q_row = d->q_stride, a->q_head = d->q_head_stride, a->k_row = d->k_stride, a->k_head = d->k_head_stride;
    a->v_row = d->v_stride, a->v_head = d->v_head_stride, a->scale = static_cast<float>(d->scale);
    OEQ_TRY(drop_of(d->p_drop, &a->threshold, &a->keep_scale));
    const int64_t es = static_cast<int64_t>(element_size(d->dtype));
    for (int64_t stride : {a->q_row, a->q_head, a->k_row, a->k_head, a->v_row, a->v_head})
        if (stride < 0 || stride * es % 16)
            return fail(OEQ_ERR_INVALID_ARG, "strides must be non-negative multiples of 16 bytes");
    constexpr int64_t grid = int64_t(1) << 24;  // a launch holds fewer than 2^32 threads
    if (d->n_struct && (fwd_blocks(d->dtype, *a) >= grid || bwd_blocks(d->dtype, *a) >= grid))
        return fail(OEQ_ERR_UNSUPPORTED, "too many rows and heads for one launch");
    return OEQ_OK;
}

// The operands both directions read.
inline oeq_status attn_operands(ro::AttnArgs *a, const int32_t *q_ptr, const int32_t *k_ptr, const void *q, const void *k,
                                const void *v, const uint8_t *key_mask, const int64_t *rng) {
    if (a->n_struct && (!q_ptr || !k_ptr)) return fail(OEQ_ERR_INVALID_ARG, "a row pointer is NULL");
    if (a->q_rows && !q) return fail(OEQ_ERR_INVALID_ARG, "q is NULL");
    if (a->k_rows && (!k || !v)) return fail(OEQ_ERR_INVALID_ARG, "k or v is NULL");
    if (a->threshold && !rng) return fail(OEQ_ERR_INVALID_ARG, "dropout needs rng");
    OEQ_TRY(check_aligned(q_ptr, 4, "q_ptr"));
    OEQ_TRY(check_aligned(k_ptr, 4, "k_ptr"));
    OEQ_TRY(check_aligned(q, 16, "q"));
    OEQ_TRY(check_aligned(k, 16, "k"));
    OEQ_TRY(check_aligned(v, 16, "v"));
    OEQ_TRY(check_aligned(rng, 8, "rng"));
    a->q_ptr = q_ptr, a->k_ptr = k_ptr, a->q = q, a->k = k, a->v = v, a->key_mask = key_mask, a->rng = rng;
    return OEQ_OK;
}

}  // namespace capi
}  // namespace oeq
