// Causal attention forward (attn_forward.hpp): a query row sees the states up to its own place.
//
// Bound by the matrix unit and the vector unit: 2 x 4096 rows, 16 heads over 4, D = 128, fp16: 172 us, 800 TFLOP/s of
// the visible scores' products (the library's large products reach 1127).  Short sequences are bound by latency
// and by tiles that the limit cuts: 64 of up to 200 rows, 8 heads of 32, fp32, dropout, 34 us.  Single tokens over
// caches are as in the cross attention: 14 us and 4 for the join, two thirds of the copy rate.
#include <algorithm>

#include "attn_forward.hpp"

namespace oeq {
namespace readout {

namespace {

Choice choose(oeq_dtype dtype, const AttnArgs &a) {
    Choice c{};
    const int64_t rows = a.q_rows * a.share;
    // Sharing keys among the waves was slower from 33 rows a sequence on: 64 x 120 rows, 8 heads of 32, fp32, 25 -> 28
    // us, 256 x 60 rows 42 -> 47, D = 128 97 -> 105; only few long walks gain (16 x 800 rows: 108 -> 90).
    c.split_keys = rows <= 32 * int64_t(a.n_struct);
    c.slots = tile_slots(a.q_rows, a.n_struct, a.share, c.split_keys ? 32 : 128);
    const int64_t base = c.slots * a.kv_heads, tile = c.split_keys || (dtype == OEQ_F32 && a.dim > 32) ? 32 : 64;
    // Tiles of all walks, for sequences of the average lengths, and of the longest of these.  A piece is what a
    // workgroup has if the work is spread evenly over the chip, 256 keys at least; sequences of twice the
    // average length are still cut so, longer ones into longer pieces.  (8 sequences of up to 2048 rows, 8 heads over 4
    // of 64, bf16, forward and backward: 179 us, 187 with walks cut evenly into a common number.)
    const int64_t n = a.q_rows / a.n_struct, m = a.k_rows / a.n_struct;
    if (m >= 4 * n) {  // the walks of a sequence are alike: split as in the cross attention
        const int64_t most = m / 256, blocks = 256 * (a.dim <= 32 ? 4 : 2), splits = std::min((blocks + base / 2) / base, most);
        c.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(splits, 64)));
        c.blocks = base * c.splits;
        return c;
    }
    const int64_t longest = m / tile + 1, walk = (m > n ? m - n / 2 : m / 2) / tile + 1;
    const int64_t total = (rows / (c.split_keys ? 32 : 128) + 1) * a.kv_heads * walk, fill = 256 * (a.dim <= 32 ? 3 : 2);
    c.piece = static_cast<int>(std::min(std::max<int64_t>(256 / tile, (total + fill - 1) / fill), longest));
    const int64_t splits = longest <= c.piece ? 1 : ((a.n_struct > 1 ? 2 : 1) * longest + c.piece - 1) / c.piece;
    c.splits = static_cast<int>(splits > 16 ? 16 : splits);
    if (c.splits == 1) c.piece = 0;
    c.blocks = base * c.splits;
    return c;
}

}  // namespace

size_t causal_attn_fwd_workspace(oeq_dtype dtype, const AttnArgs &a) { return forward_workspace(a, choose(dtype, a), true); }

int64_t causal_attn_fwd_blocks(oeq_dtype dtype, const AttnArgs &a) { return choose(dtype, a).blocks; }

hipError_t causal_attn_fwd(oeq_dtype dtype, const AttnArgs &a, hipStream_t stream) {
    switch (dtype) {
        case OEQ_F32: return forward<float, true>(a, choose(dtype, a), stream);
        case OEQ_F16: return forward<f16, true>(a, choose(dtype, a), stream);
        case OEQ_BF16: return forward<bf16, true>(a, choose(dtype, a), stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace readout
}  // namespace oeq
