#include "causal_attn_bwd.hpp"

namespace oeq {
namespace readout {

hipError_t causal_attn_bwd_f32(const AttnArgs &a, hipStream_t stream) { return backward<float, true>(a, choose(a), stream); }

}  // namespace readout
}  // namespace oeq
