// Causal attention backward (attn_backward.hpp): a query row sees the states up to its own place.  One source file
// a type (causal_attn_bwd_*.hip), which compile in parallel; causal_attn_bwd.hip has the entry points.
//
// Bound as the cross attention's, with a third more for tiles that the limit cuts: 2 x 4096 rows, 16 heads over 4,
// D = 128, fp16, 903 us, 380 TFLOP/s of the minimal five products of the visible scores (1592 us with whole walks);
// 8 sequences of up to 2048 rows, 8 heads over 4 of 64, bf16, 130 us, 8 for delta and 10 for the sum of the pieces.
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
    const int64_t rows = a.q_rows * a.share;
    // As in the forward: shared among the waves, 64 x 120 rows, 8 heads of 32, fp32, take 76 us, not 68, and at D = 128
    // (up to 200 rows) 380, not 303.
    c.split_keys = rows <= 32 * int64_t(a.n_struct);
    c.q_slots = tile_slots(a.q_rows, a.n_struct, a.share, c.split_keys ? 32 : 128);
    c.k_slots = tile_slots(a.k_rows, a.n_struct, 1, kKeyTile);
    // Pieces as in the forward, over both roles; a tile of either walk is about the same work.
    const int64_t n = rows / a.n_struct, m = a.k_rows / a.n_struct;
    const int64_t q_walk = (m > n / a.share ? m - n / a.share / 2 : m / 2) / 32 + 1;
    const int64_t k_walk = (m > n / a.share ? n - n * (n / a.share) / (2 * m) : n / 2) / kRowTile + 1;
    const int64_t total = ((rows / (c.split_keys ? 32 : 128) + 1) * q_walk + (a.k_rows / kKeyTile + 1) * k_walk) * a.kv_heads;
    // Three workgroups a compute unit: 142 us and 7 for the sum at 512, 129 and 13 at 1024 (8 sequences of up to 2048
    // rows, as above), 130 and 10 here.
    const int64_t fill = 768;
    const int64_t longest = std::max(m / 32, n / kRowTile) + 1;
    c.piece = static_cast<int>(std::max<int64_t>(8, std::min((total + fill - 1) / fill, longest)));
    const auto splits = [&](int64_t walk) {
        const int64_t most = walk <= c.piece ? 1 : ((a.n_struct > 1 ? 2 : 1) * walk + c.piece - 1) / c.piece;
        return static_cast<int>(most > 16 ? 16 : most);
    };
    c.q_splits = splits(m / 32 + 1);
    c.k_splits = splits(n / kRowTile + 1);
    c.part_q = c.q_splits > 1 ? up(static_cast<size_t>(c.q_splits) * a.q_rows * a.heads * a.dim * 4) : 0;
    c.part_k = c.k_splits > 1 ? up(static_cast<size_t>(c.k_splits) * a.k_rows * a.kv_heads * a.dim * 4) : 0;
    c.delta = up(static_cast<size_t>(a.q_rows) * a.heads * 4);
    c.q_pieces = c.q_splits > 1 ? c.delta : 0;
    c.k_pieces = c.k_splits > 1 ? up(static_cast<size_t>(a.k_rows) * a.kv_heads * 4) : 0;
    c.bytes = c.part_q + 2 * c.part_k + c.delta + c.q_pieces + c.k_pieces;
    return c;
}

}  // namespace
}  // namespace readout
}  // namespace oeq
