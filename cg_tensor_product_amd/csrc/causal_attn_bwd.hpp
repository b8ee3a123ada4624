// Causal attention backward (attn_backward.hpp): a query row sees the states up to its own place.  One source file
// a type (causal_attn_bwd_*.hip), which compile in parallel; causal_attn_bwd.hip has the entry points.
#pragma once

#include "attn_backward.hpp"

namespace oeq {
namespace readout {

hipError_t causal_attn_bwd_f32(const AttnArgs &a, hipStream_t stream);
hipError_t causal_attn_bwd_f16(const AttnArgs &a, hipStream_t stream);
hipError_t causal_attn_bwd_bf16(const AttnArgs &a, hipStream_t stream);

namespace {

inline Choice choose(const AttnArgs &a) {
    Choice c{};
    // Twice the workgroups the chip holds at once: walks half as long even out better than their
    // partial sums cost (bf16, D = 64, 4 structures of 1024 query rows and 2048 states: 111 us,
    // 135 with walks of one round).
    const int64_t fill = 1024;
    c.split_keys = a.q_rows * a.share <= 32 * int64_t(a.n_struct);
    c.q_slots = tile_slots(a.q_rows, a.n_struct, a.share, c.split_keys ? 32 : 128);
    c.k_slots = tile_slots(a.k_rows, a.n_struct, 1, kKeyTile);
    const int64_t keys = a.k_rows / a.n_struct, rows = a.q_rows * a.share / a.n_struct;
    const int64_t share = (c.q_slots * a.kv_heads * keys + c.k_slots * a.kv_heads * rows) / fill;
    c.q_splits = splits_of(keys, share);
    c.k_splits = splits_of(rows, share);
    c.part_q = c.q_splits > 1 ? up(static_cast<size_t>(c.q_splits) * a.q_rows * a.heads * a.dim * 4) : 0;
    c.part_k = c.k_splits > 1 ? up(static_cast<size_t>(c.k_splits) * a.k_rows * a.kv_heads * a.dim * 4) : 0;
    c.delta = up(static_cast<size_t>(a.q_rows) * a.heads * 4);
    c.bytes = c.part_q + 2 * c.part_k + c.delta;
    return c;
}

}  // namespace
}  // namespace readout
}  // namespace oeq
