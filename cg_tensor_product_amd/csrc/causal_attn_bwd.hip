// Causal attention backward: workspace, workgroups, and the kernels of the call's type.
#include "causal_attn_bwd.hpp"

namespace oeq {
namespace readout {

size_t causal_attn_bwd_workspace(oeq_dtype, const AttnArgs &a) { return choose(a).bytes; }

int64_t causal_attn_bwd_blocks(oeq_dtype, const AttnArgs &a) {
    const Choice c = choose(a);
    const int64_t walks = c.q_slots * a.kv_heads * c.q_splits + c.k_slots * a.kv_heads * c.k_splits;
    return std::max(walks, delta_slots(a) * a.kv_heads);
}

hipError_t causal_attn_bwd(oeq_dtype dtype, const AttnArgs &a, hipStream_t stream) {
    switch (dtype) {
        case OEQ_F32: return causal_attn_bwd_f32(a, stream);
        case OEQ_F16: return causal_attn_bwd_f16(a, stream);
        case OEQ_BF16: return causal_attn_bwd_bf16(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace readout
}  // namespace oeq
