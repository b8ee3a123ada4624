// Cross attention backward.  With p = exp(scale q k^T - lse) formed again from the saved
// log sums, f the dropout factors (0 or 1 / share kept) and delta = sum_d grad_out out:
//   grad_v = (p f)^T grad_out            dp = (grad_out v^T) f
//   ds = p (dp - delta)                  grad_q = scale ds k,  grad_k = scale ds^T q
// Three kernels and no atomics:
//   k_delta        one pass over out and grad_out;
//   k_grad_keys    a wave owns 32 keys (k, v and both gradients in registers) and walks the
//                  query rows of the structure, all heads that share the keys among them, so
//                  the sum over shared heads needs no further step;
//   k_grad_queries a wave owns 32 query rows and walks the keys, like the forward.
// Scores are formed twice (7 products of the minimal 5); the alternative, one kernel that adds
// into grad_q, needs atomics or a partial grad_q for each tile of keys.  With few workgroups
// the walk is split over workgroups, whose fp32 partial sums a last kernel adds in order.
#include "attn_device.hpp"

namespace oeq {
namespace readout {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kKeyTile = 128;  // keys of a k_grad_keys workgroup
constexpr int kRowTile = 32;   // query rows of a step of its walk

struct Bwd {
    float *delta;      // [query row, head]
    float *part_q;     // [split][query row, head][dim]; NULL: one split, written directly
    float *part_k, *part_v;  // [split][key, key head][dim]
};

// exp2 argument of a row that saw nothing: every probability is zero.
__device__ __forceinline__ float log2_sum(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2E; }

// p from a score; fp32 forms scale s - lse in one rounding, since the difference is small
// against its parts.
template <class T>
__device__ __forceinline__ float probability(float s, float scale, float c, float lse, float lse2) {
    if (sizeof(T) == 4) return __builtin_amdgcn_exp2f(fmaf(s, scale, -lse) * kLog2E);
    return __builtin_amdgcn_exp2f(fmaf(s, c, -lse2));
}

// kDim / 8 (up to a power of two) lanes a row.
template <class T, int kLanes>
__global__ void __launch_bounds__(kThreads) k_delta(AttnArgs a, float *delta) {
    const int64_t n = a.q_rows * a.heads, at = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / kLanes;
    const int d = threadIdx.x % kLanes * 8;
    float v = 0.f;
    if (at < n && d < a.dim) {
        const f32x8 o = to_f32<T>(load8(static_cast<const T *>(a.out) + at * a.dim + d));
        const f32x8 g = to_f32<T>(load8(static_cast<const T *>(a.grad_out) + at * a.dim + d));
#pragma unroll
        for (int j = 0; j < 8; ++j) v = fmaf(o[j], g[j], v);
    }
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) v += __shfl_xor(v, off);
    if (at < n && threadIdx.x % kLanes == 0) delta[at] = v;
}

template <class T, int kDim, bool kDrop>
__global__ void __launch_bounds__(kThreads) k_grad_keys(AttnArgs a, Bwd out, int splits, int64_t slots) {
    constexpr int kRow = kTileRow<T, kDim>, kSteps = kDim / 16, kOut = kDim / 32;
    __shared__ __attribute__((aligned(16))) T q_tile[kRowTile * kRow], g_tile[kRowTile * kRow];
    __shared__ __attribute__((aligned(16))) float row_lse[kRowTile], row_delta[kRowTile];
    __shared__ __attribute__((aligned(16))) uint32_t kept[kDrop ? kWaves : 1][kRowTile];
    const Place w = place_of<kKeyTile>(a, false, splits, slots);
    if (!w.any) return;
    const int lane = threadIdx.x & 63, half = lane >> 5, wave = threadIdx.x >> 6;
    const int key = w.first + wave * 32 + (lane & 31);
    const bool key_ok = key < w.keys;
    const int64_t k_row = w.k_begin + (key_ok ? key : 0);
    const bool seen = key_ok && (!a.key_mask || a.key_mask[k_row]);
    vec8<T> kf[kSteps], vf[kSteps];
    {
        const T *k = static_cast<const T *>(a.k) + k_row * a.k_row + w.kv_head * a.k_head;
        const T *v = static_cast<const T *>(a.v) + k_row * a.v_row + w.kv_head * a.v_head;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int d = 16 * s + 8 * half;
            const bool in = seen && d < a.dim;
            kf[s] = in ? *reinterpret_cast<const vec8<T> *>(k + d) : vec8<T>(T(0.f));
            vf[s] = in ? *reinterpret_cast<const vec8<T> *>(v + d) : vec8<T>(T(0.f));
        }
    }
    Rng g{};
    if (kDrop) g = load_rng(a.rng);
    const float c = a.scale * kLog2E;
    f32x16 gk[kOut] = {}, gv[kOut] = {};

    const int n_tiles = (w.rows + kRowTile - 1) / kRowTile, per = (n_tiles + splits - 1) / splits;
    const int t_end = min(n_tiles, (w.split + 1) * per);
    RowStage<T, kRowTile, kDim, kThreads> q_in, g_in;
    float lse_in = 0.f, delta_in = 0.f;
    auto side_row = [&](int r, int64_t *q_row, int *head) {
        r = min(r, w.rows - 1);
        *q_row = w.q_begin + r / a.share;
        *head = w.kv_head * a.share + r % a.share;
    };
    auto fetch = [&](int t) {
        int64_t q_row;
        int head;
        q_in.fetch(threadIdx.x, a.dim, [&](int row) {
            side_row(t * kRowTile + row, &q_row, &head);
            return static_cast<const T *>(a.q) + q_row * a.q_row + head * a.q_head;
        });
        g_in.fetch(threadIdx.x, a.dim, [&](int row) {
            side_row(t * kRowTile + row, &q_row, &head);
            return static_cast<const T *>(a.grad_out) + (q_row * a.heads + head) * a.dim;
        });
        if (threadIdx.x < kRowTile) {
            side_row(t * kRowTile + threadIdx.x, &q_row, &head);
            const bool in = t * kRowTile + int(threadIdx.x) < w.rows;
            lse_in = in ? a.lse[q_row * a.heads + head] : -INFINITY;  // rows past the end count as unseen
            delta_in = in ? out.delta[q_row * a.heads + head] : 0.f;
        }
    };
    int t = w.split * per;
    if (t < t_end) fetch(t);
    for (; t < t_end; ++t) {
        const int r0 = t * kRowTile;
        const int in_tile = min(kRowTile, w.rows - r0);
        __syncthreads();  // the last tile has been read
        const uint64_t valid = (1ull << in_tile) - 1;
        q_in.store(q_tile, threadIdx.x, a.dim, valid);
        g_in.store(g_tile, threadIdx.x, a.dim, valid);
        if (threadIdx.x < kRowTile) {
            row_lse[threadIdx.x] = lse_in == -INFINITY ? INFINITY : sizeof(T) == 4 ? lse_in : lse_in * kLog2E;
            row_delta[threadIdx.x] = delta_in;
        }
        if (kDrop) {
            // 32 rows x 4 generator blocks of this wave's keys, two a lane; the bits of a row make a word
            int64_t q_row;
            int head;
            side_row(r0 + (lane & 31), &q_row, &head);
            const uint32_t row = static_cast<uint32_t>(q_row * a.heads + head);
            const uint32_t block = static_cast<uint32_t>(w.first + wave * 32) / 8 + 2 * half;
            const uint32_t bits = keep_bits(g, block, row, a.threshold) | keep_bits(g, block + 1, row, a.threshold) << 8;
            reinterpret_cast<uint16_t *>(kept[wave])[(lane & 31) * 2 + half] = static_cast<uint16_t>(bits);
        }
        __syncthreads();
        if (t + 1 < t_end) fetch(t + 1);

        f32x16 s = {}, dp = {};
        const int row = permuted_row(lane & 31);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) s = mma(s, row_operand(q_tile, kRow, row, 16 * i, half), kf[i]);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) dp = mma(dp, row_operand(g_tile, kRow, row, 16 * i, half), vf[i]);
        vec8<T> pf[2], sf[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f32x8 p8, s8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int at = 16 * h + 8 * half + j;  // the row of the tile
                const float l = row_lse[at];
                float p = seen ? probability<T>(s[8 * h + j], a.scale, c, l, l) : 0.f;
                float d = dp[8 * h + j];
                float pk = p;
                if (kDrop) {
                    const bool keep = kept[wave][at] >> (lane & 31) & 1;
                    pk = keep ? p : 0.f;
                    d = keep ? d * a.keep_scale : 0.f;
                }
                p8[j] = pk;
                s8[j] = p * (d - row_delta[at]);
            }
            pf[h] = from_f32<T>(p8);
            sf[h] = from_f32<T>(s8);
        }
#pragma unroll
        for (int d = 0; d < kOut; ++d) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                gv[d] = mma(gv[d], column_operand(g_tile, kRow, 16 * h, 32 * d, lane), pf[h]);
                gk[d] = mma(gk[d], column_operand(q_tile, kRow, 16 * h, 32 * d, lane), sf[h]);
            }
        }
    }
    if (!key_ok) return;
    const int64_t n = a.k_rows * a.kv_heads, at = k_row * a.kv_heads + w.kv_head;
    using V4 = T __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int d = 0; d < kOut; ++d) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int col = 32 * d + 8 * i + 4 * half;
            if (col < a.dim) {
                f32x4 k = {gk[d][4 * i], gk[d][4 * i + 1], gk[d][4 * i + 2], gk[d][4 * i + 3]};
                f32x4 v = {gv[d][4 * i], gv[d][4 * i + 1], gv[d][4 * i + 2], gv[d][4 * i + 3]};
                // a key that is not seen has no gradient, whatever the rows hold
                k = seen ? k * a.scale : f32x4{};
                v = seen ? v * a.keep_scale : f32x4{};
                if (splits > 1) {
                    const int64_t to = (w.split * n + at) * a.dim + col;
                    if (a.grad_k) *reinterpret_cast<f32x4 *>(out.part_k + to) = k;
                    if (a.grad_v) *reinterpret_cast<f32x4 *>(out.part_v + to) = v;
                } else {
                    const int64_t to = at * a.dim + col;
                    if (a.grad_k) *reinterpret_cast<V4 *>(static_cast<T *>(a.grad_k) + to) = __builtin_convertvector(k, V4);
                    if (a.grad_v) *reinterpret_cast<V4 *>(static_cast<T *>(a.grad_v) + to) = __builtin_convertvector(v, V4);
                }
            }
        }
    }
}

template <class T, int kDim, bool kSplitKeys>
struct Tiles {
    static constexpr int kKeys = 32;
    static constexpr int kRow = kTileRow<T, kDim>;
    static constexpr int kRows = kSplitKeys ? 32 : 128;  // query rows of a workgroup
    static constexpr int kStage = kSplitKeys ? 64 : kThreads;
    static constexpr int kTile = kKeys * kRow;
    static constexpr int kLds = (kSplitKeys ? kWaves : 1) * 2 * kTile * int(sizeof(T));
    static constexpr int kJoinRow = kDim + 4;
    static constexpr int kJoin = kSplitKeys ? kWaves * 32 * kJoinRow * 4 : 0;
    static constexpr int kBytes = kLds > kJoin ? kLds : kJoin;
};

// The waves share tiles of keys, or with kSplitKeys (few query rows) take them in turn, as in
// the forward.
template <class T, int kDim, bool kDrop, bool kSplitKeys>
__global__ void __launch_bounds__(kThreads) k_grad_queries(AttnArgs a, Bwd out, int splits, int64_t slots) {
    using C = Tiles<T, kDim, kSplitKeys>;
    constexpr int kKeys = C::kKeys, kRow = C::kRow, kSteps = kDim / 16, kOut = kDim / 32;
    __shared__ __attribute__((aligned(16))) char lds[C::kBytes];
    const Place w = place_of<C::kRows>(a, true, splits, slots);
    if (!w.any) return;
    const int lane = threadIdx.x & 63, half = lane >> 5, wave = threadIdx.x >> 6;
    const int thread = kSplitKeys ? lane : threadIdx.x;
    T *k_tile = reinterpret_cast<T *>(lds) + (kSplitKeys ? wave * 2 * C::kTile : 0), *v_tile = k_tile + C::kTile;
    const int r = w.first + (kSplitKeys ? 0 : wave * 32) + (lane & 31);
    const bool row_ok = r < w.rows;
    const int64_t q_row = w.q_begin + (row_ok ? r / a.share : 0);
    const int head = w.kv_head * a.share + (row_ok ? r % a.share : 0);
    const int64_t at = q_row * a.heads + head;
    vec8<T> qf[kSteps], gf[kSteps];
    {
        const T *q = static_cast<const T *>(a.q) + q_row * a.q_row + head * a.q_head;
        const T *g = static_cast<const T *>(a.grad_out) + at * a.dim;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int d = 16 * s + 8 * half;
            const bool in = row_ok && d < a.dim;
            qf[s] = in ? *reinterpret_cast<const vec8<T> *>(q + d) : vec8<T>(T(0.f));
            gf[s] = in ? *reinterpret_cast<const vec8<T> *>(g + d) : vec8<T>(T(0.f));
        }
    }
    const float lse = row_ok ? a.lse[at] : -INFINITY, lse1 = lse == -INFINITY ? INFINITY : lse, lse2 = log2_sum(lse);
    const float delta = row_ok ? out.delta[at] : 0.f;
    Rng g{};
    if (kDrop) g = load_rng(a.rng);
    const float c = a.scale * kLog2E;
    f32x16 gq[kOut] = {};

    const int n_tiles = (w.keys + kKeys - 1) / kKeys, per = (n_tiles + splits - 1) / splits;
    const int t_end = min(n_tiles, (w.split + 1) * per), t_step = kSplitKeys ? kWaves : 1;
    const T *k_base = static_cast<const T *>(a.k) + w.k_begin * a.k_row + w.kv_head * a.k_head;
    const T *v_base = static_cast<const T *>(a.v) + w.k_begin * a.v_row + w.kv_head * a.v_head;
    const uint8_t *mask = a.key_mask ? a.key_mask + w.k_begin : nullptr;
    RowStage<T, kKeys, kDim, C::kStage> k_in, v_in;
    uint32_t visible = 0;
    auto fetch = [&](int t) {
        const int k0 = t * kKeys, last = w.keys - 1;
        const int key = k0 + (lane & 31);
        visible = key <= last && (!mask || mask[key]);
        k_in.fetch(thread, a.dim, [&](int row) { return k_base + int64_t(min(k0 + row, last)) * a.k_row; });
        v_in.fetch(thread, a.dim, [&](int row) { return v_base + int64_t(min(k0 + row, last)) * a.v_row; });
    };
    int t = w.split * per + (kSplitKeys ? wave : 0);
    if (t < t_end) fetch(t);
    for (; t < t_end; t += t_step) {
        const uint64_t valid = __ballot(visible);
        if (kSplitKeys) wave_sync(); else __syncthreads();
        k_in.store(k_tile, thread, a.dim, valid);
        v_in.store(v_tile, thread, a.dim, valid);
        if (kSplitKeys) wave_sync(); else __syncthreads();
        const int k0 = t * kKeys;
        if (t + t_step < t_end) fetch(t + t_step);
        f32x16 s = {}, dp = {};
        const int row = permuted_row(lane & 31);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) s = mma(s, row_operand(k_tile, kRow, row, 16 * i, half), qf[i]);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) dp = mma(dp, row_operand(v_tile, kRow, row, 16 * i, half), gf[i]);
        vec8<T> sf[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f32x8 s8;
            const uint32_t keep = kDrop ? keep_bits(g, (k0 + 16 * h) / 8 + half, static_cast<uint32_t>(at), a.threshold) : 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int key = 16 * h + 8 * half + j;
                const float p = valid >> key & 1 ? probability<T>(s[8 * h + j], a.scale, c, lse1, lse2) : 0.f;
                float d = dp[8 * h + j];
                if (kDrop) d = (keep >> j & 1) ? d * a.keep_scale : 0.f;
                s8[j] = p * (d - delta);
            }
            sf[h] = from_f32<T>(s8);
        }
#pragma unroll
        for (int d = 0; d < kOut; ++d) {
#pragma unroll
            for (int h = 0; h < 2; ++h) gq[d] = mma(gq[d], column_operand(k_tile, kRow, 16 * h, 32 * d, lane), sf[h]);
        }
    }
    const int64_t n = a.q_rows * a.heads;
    if (!kSplitKeys) {
        if (!row_ok) return;
        using V4 = T __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int d = 0; d < kOut; ++d) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = 32 * d + 8 * i + 4 * half;
                if (col < a.dim) {
                    f32x4 v = {gq[d][4 * i], gq[d][4 * i + 1], gq[d][4 * i + 2], gq[d][4 * i + 3]};
                    v *= a.scale;
                    if (splits > 1)
                        *reinterpret_cast<f32x4 *>(out.part_q + (w.split * n + at) * a.dim + col) = v;
                    else
                        *reinterpret_cast<V4 *>(static_cast<T *>(a.grad_q) + at * a.dim + col) =
                            __builtin_convertvector(v, V4);
                }
            }
        }
        return;
    }
    __syncthreads();
    float *join = reinterpret_cast<float *>(lds), *mine = join + (wave * 32 + (lane & 31)) * C::kJoinRow;
#pragma unroll
    for (int d = 0; d < kOut; ++d) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 v = {gq[d][4 * i], gq[d][4 * i + 1], gq[d][4 * i + 2], gq[d][4 * i + 3]};
            *reinterpret_cast<f32x4 *>(mine + 32 * d + 8 * i + 4 * half) = v;
        }
    }
    __syncthreads();
    const int jr = threadIdx.x >> 3, row = w.first + jr;  // eight threads a row
    if (row >= w.rows) return;
    const int64_t to = (w.q_begin + row / a.share) * a.heads + w.kv_head * a.share + row % a.share;
    for (int col = (threadIdx.x & 7) * 8; col < a.dim; col += 64) {
        f32x8 v = {};
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            const float *from = join + (i * 32 + jr) * C::kJoinRow + col;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += from[j];
        }
        v *= a.scale;
        if (splits > 1)
            store8(out.part_q + (w.split * n + to) * a.dim + col, v);
        else
            store8(static_cast<T *>(a.grad_q) + to * a.dim + col, from_f32<T>(v));
    }
}

// out = sum of `splits` fp32 arrays of n values (a multiple of eight), in order.
template <class T>
__global__ void __launch_bounds__(kThreads) k_add(const float *part, T *out, int64_t n, int splits) {
    const int64_t step = int64_t(gridDim.x) * kThreads * 8;
    for (int64_t i = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * 8; i < n; i += step) {
        f32x8 v = load8(part + i);
        for (int s = 1; s < splits; ++s) v += load8(part + s * n + i);
        store8(out + i, from_f32<T>(v));
    }
}

constexpr size_t up(size_t v) { return (v + 255) / 256 * 256; }

struct Choice {
    bool split_keys;
    int q_splits, k_splits;  // of k_grad_queries (over keys), of k_grad_keys (over rows)
    int64_t q_slots, k_slots;
    size_t delta, part_q, part_k, bytes;  // offsets of the workspace's pieces
    size_t k_bytes;
};

int splits_of(int64_t blocks, int64_t walk) {
    int64_t s = (512 + blocks - 1) / blocks;  // two workgroups a compute unit
    const int64_t most = walk / 256;          // 256 rows of the walk a split at least
    s = s > most ? most : s;
    return static_cast<int>(s < 1 ? 1 : s > 64 ? 64 : s);
}

Choice choose(const AttnArgs &a) {
    Choice c{};
    c.split_keys = a.q_rows * a.share <= 32 * int64_t(a.n_struct);
    c.q_slots = tile_slots(a.q_rows, a.n_struct, a.share, c.split_keys ? 32 : 128);
    c.k_slots = tile_slots(a.k_rows, a.n_struct, 1, kKeyTile);
    c.q_splits = splits_of(c.q_slots * a.kv_heads, a.k_rows / a.n_struct);
    c.k_splits = splits_of(c.k_slots * a.kv_heads, a.q_rows * a.share / a.n_struct);
    c.part_q = up(static_cast<size_t>(a.q_rows) * a.heads * sizeof(float));
    c.part_k = c.part_q + (c.q_splits > 1 ? up(static_cast<size_t>(c.q_splits) * a.q_rows * a.heads * a.dim * 4) : 0);
    c.k_bytes = c.k_splits > 1 ? up(static_cast<size_t>(c.k_splits) * a.k_rows * a.kv_heads * a.dim * 4) : 0;
    c.bytes = c.part_k + 2 * c.k_bytes;
    return c;
}

unsigned grid_of(int64_t blocks) { return static_cast<unsigned>(blocks > (1 << 22) ? 1 << 22 : blocks); }

template <class T, int kDim, bool kDrop>
void launch(const AttnArgs &a, const Choice &c, const Bwd &out, hipStream_t stream) {
    const dim3 threads(kThreads);
    if (a.grad_k || a.grad_v) {
        const dim3 grid(static_cast<unsigned>(c.k_slots * a.kv_heads * c.k_splits));
        k_grad_keys<T, kDim, kDrop><<<grid, threads, 0, stream>>>(a, out, c.k_splits, c.k_slots);
    }
    if (a.grad_q && a.q_rows) {
        const dim3 grid(static_cast<unsigned>(c.q_slots * a.kv_heads * c.q_splits));
        if (c.split_keys)
            k_grad_queries<T, kDim, kDrop, true><<<grid, threads, 0, stream>>>(a, out, c.q_splits, c.q_slots);
        else
            k_grad_queries<T, kDim, kDrop, false><<<grid, threads, 0, stream>>>(a, out, c.q_splits, c.q_slots);
    }
}

template <class T, int kDim>
void launch(const AttnArgs &a, const Choice &c, const Bwd &out, hipStream_t stream) {
    if (a.q_rows) {
        constexpr int kLanes = kDim <= 32 ? 4 : kDim <= 64 ? 8 : 16;
        const int64_t n = a.q_rows * a.heads * kLanes;
        k_delta<T, kLanes><<<dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream>>>(
            a, out.delta);
    }
    if (a.threshold)
        launch<T, kDim, true>(a, c, out, stream);
    else
        launch<T, kDim, false>(a, c, out, stream);
}

template <class T>
hipError_t backward(const AttnArgs &a, hipStream_t stream) {
    const Choice c = choose(a);
    char *ws = static_cast<char *>(a.workspace);
    Bwd out{};
    out.delta = reinterpret_cast<float *>(ws);
    out.part_q = reinterpret_cast<float *>(ws + c.part_q);
    out.part_k = reinterpret_cast<float *>(ws + c.part_k);
    out.part_v = reinterpret_cast<float *>(ws + c.part_k + c.k_bytes);
    if (a.dim <= 32)
        launch<T, 32>(a, c, out, stream);
    else if (a.dim <= 64)
        launch<T, 64>(a, c, out, stream);
    else if (a.dim <= 96)
        launch<T, 96>(a, c, out, stream);
    else
        launch<T, 128>(a, c, out, stream);
    const auto add = [&](const float *part, void *to, int64_t n, int splits) {
        if (to && splits > 1 && n)
            k_add<T><<<dim3(grid_of((n / 8 + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream>>>(
                part, static_cast<T *>(to), n, splits);
    };
    add(out.part_q, a.grad_q, a.q_rows * a.heads * a.dim, c.q_splits);
    add(out.part_k, a.grad_k, a.k_rows * a.kv_heads * a.dim, c.k_splits);
    add(out.part_v, a.grad_v, a.k_rows * a.kv_heads * a.dim, c.k_splits);
    return hipGetLastError();
}

}  // namespace

size_t cross_attn_bwd_workspace(const AttnArgs &a) { return choose(a).bytes; }

int64_t cross_attn_bwd_blocks(const AttnArgs &a) {
    const Choice c = choose(a);
    const int64_t q = c.q_slots * a.kv_heads * c.q_splits, k = c.k_slots * a.kv_heads * c.k_splits;
    return q > k ? q : k;
}

hipError_t cross_attn_bwd(oeq_dtype dtype, const AttnArgs &a, hipStream_t stream) {
    switch (dtype) {
        case OEQ_F32: return backward<float>(a, stream);
        case OEQ_F16: return backward<f16>(a, stream);
        case OEQ_BF16: return backward<bf16>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace readout
}  // namespace oeq
