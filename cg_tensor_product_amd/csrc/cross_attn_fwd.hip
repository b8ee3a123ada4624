// Cross attention forward (attn_forward.hpp): every query row sees all states of its structure.
#include "attn_forward.hpp"

namespace oeq {
namespace readout {

namespace {

Choice choose(const AttnArgs &a) {
    Choice c{};
    const int64_t rows = a.q_rows * a.share;
    c.split_keys = rows <= 32 * int64_t(a.n_struct);
    c.slots = tile_slots(a.q_rows, a.n_struct, a.share, c.split_keys ? 32 : 128);
    // Splits until the workgroups fill the chip about once (256 compute units; four workgroups each
    // at D <= 32, else two).  4 structures of 1024 query rows and 2048 states, 8 heads over 4:
    // bf16, D = 64 takes 36 us with 512 workgroups, 49 with 768 and 45 with 1024; D = 32 takes
    // 39, 37 and 31 us; fp32, D = 128 takes 303, 400 and 324 us.
    const int64_t fill = 256 * (a.dim <= 32 ? 4 : 2);
    const int64_t base = c.slots * a.kv_heads, most = a.k_rows / a.n_struct / 256;  // 256 keys a split at least
    int64_t splits = (fill + base / 2) / base;
    splits = splits > most ? most : splits;
    c.splits = static_cast<int>(splits < 1 ? 1 : splits > 64 ? 64 : splits);
    c.blocks = base * c.splits;
    return c;
}

}  // namespace

size_t cross_attn_fwd_workspace(oeq_dtype, const AttnArgs &a) { return forward_workspace(a, choose(a), false); }

int64_t cross_attn_fwd_blocks(oeq_dtype, const AttnArgs &a) { return choose(a).blocks; }

hipError_t cross_attn_fwd(oeq_dtype dtype, const AttnArgs &a, hipStream_t stream) {
    switch (dtype) {
        case OEQ_F32: return forward<float, false>(a, choose(a), stream);
        case OEQ_F16: return forward<f16, false>(a, choose(a), stream);
        case OEQ_BF16: return forward<bf16, false>(a, choose(a), stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace readout
}  // namespace oeq
