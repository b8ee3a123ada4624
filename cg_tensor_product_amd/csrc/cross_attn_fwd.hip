// Cross attention forward.  For the visible keys of a query row's structure
//   s = scale q k^T,  lse = log sum exp s,  p = exp(s - lse),  out = (p * keep) v
// in one pass over the keys with a running maximum and sum.
//
// A wave computes S^T = K Q^T tile by tile with its 32 query rows along the lanes, so the
// softmax statistics are one number a lane, and O^T = V^T P^T takes the probabilities
// straight from the score registers (attn_device.hpp).  K and V pass through LDS; V's
// operand is read transposed from it.
//
// Two ways to split the work (kSplitKeys):
//   false: the four waves own 32 query rows each and share tiles of 64 keys;
//   true:  for few query rows (single tokens, small structures) the four waves share 32 rows
//          and take tiles of 32 keys in turn, each through LDS of its own and without
//          barriers; their results are joined in LDS at the end.
// With few workgroups the keys are also split over workgroups; a second kernel joins them.
//
// Large calls are bound by the vector unit (exponentials, the running maximum, the copies of the
// output's rescaling) next to the matrix unit: fp16, 2 x 2048 query rows x 16 heads over 5000
// states, D = 128: 200 us, 840 TFLOP/s; with D = 64 bf16 at 485 TFLOP/s, where an exponential is
// worth half the products.  fp32 runs at the rate of its matrix instructions (115 TFLOP/s, D = 64).
// Single tokens are bound by the read of K and V: 16 x up to 5000 states, 4 key heads of 64, bf16,
// 15 us and 4 for the join.
#include "attn_device.hpp"

namespace oeq {
namespace readout {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;
// The running maximum may lag behind by this many powers of two before the sums are scaled, so that most
// tiles scale nothing (a device known from published attention kernels).
constexpr float kLag = 8.f;

template <class T, int kDim, bool kSplitKeys>
struct Tiles {
    static constexpr int kKeys = kSplitKeys ? 32 : 64;
    static constexpr int kRow = kTileRow<T, kDim>;
    static constexpr int kRows = kSplitKeys ? 32 : 128;  // query rows of a workgroup
    static constexpr int kStage = kSplitKeys ? 64 : kThreads;
    static constexpr int kTile = kKeys * kRow;  // elements of one K or V tile
    static constexpr int kLds = (kSplitKeys ? kWaves : 2) * 2 * kTile * int(sizeof(T));
    static constexpr int kJoinRow = kDim + 4;
    static constexpr int kJoin = kSplitKeys ? kWaves * 32 * (kJoinRow + 2) * 4 : 0;
    static constexpr int kBytes = kLds > kJoin ? kLds : kJoin;
};

struct Partial {
    float *out;  // [split][query row, head][dim], normalised
    float *lse;  // [split][query row, head], in powers of two
};

// f(i, v) with a lane's results of a 32 x 32 block as eight consecutive rows of it from 8 i on (the
// two halves exchange theirs), so that a lane writes 16 bytes of a 16-bit type at once, not 8: 40 x 450
// query rows x 16 heads over 9 states each, D = 80, bf16, 37 -> 33 us.  Lanes l and l + 32 have to be
// active together.
template <class F>
__device__ __forceinline__ void each_eight(f32x16 o, int half, F &&f) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        f32x8 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(o[4 * i + j]), __float_as_uint(o[4 * i + 4 + j]),
                                                            false, false);
            v[j] = __uint_as_float(r[0]);
            v[4 + j] = __uint_as_float(r[1]);
        }
        f(i + half, v);
    }
}

template <class T, int kDim, bool kDrop, bool kSplitKeys>
__global__ void __launch_bounds__(kThreads) k_forward(AttnArgs a, int splits, int64_t slots, Partial partial) {
    using C = Tiles<T, kDim, kSplitKeys>;
    constexpr int kKeys = C::kKeys, kRow = C::kRow, kSteps = kDim / 16, kOut = kDim / 32, kSub = kKeys / 32;
    __shared__ __attribute__((aligned(16))) char lds[C::kBytes];
    const Place w = place_of<C::kRows>(a, blockIdx.x, true, splits, slots);
    if (!w.any) return;
    const int lane = threadIdx.x & 63, half = lane >> 5, wave = threadIdx.x >> 6;
    const int thread = kSplitKeys ? lane : threadIdx.x;
    T *k_tile = reinterpret_cast<T *>(lds) + (kSplitKeys ? wave * 2 * C::kTile : 0), *v_tile = k_tile + C::kTile;

    // this lane's query row
    const int r = w.first + (kSplitKeys ? 0 : wave * 32) + (lane & 31);
    const bool row_ok = r < w.rows;
    const int64_t q_row = w.q_begin + (row_ok ? r / a.share : 0);
    const int head = w.kv_head * a.share + (row_ok ? r % a.share : 0);
    Rng g{};
    if (kDrop) g = load_rng(a.rng);
    const uint32_t drop_row = static_cast<uint32_t>(q_row * a.heads + head);

    const float c = a.scale * kLog2E;
    f32x16 o[kOut] = {};
    float top = -INFINITY, sum = 0.f;  // the running maximum (unscaled) and this half's sum

    // this workgroup's keys, in whole tiles
    const int n_tiles = (w.keys + kKeys - 1) / kKeys, per = (n_tiles + splits - 1) / splits;
    const int t_end = min(n_tiles, (w.split + 1) * per), t_step = kSplitKeys ? kWaves : 1;
    const T *k_base = static_cast<const T *>(a.k) + w.k_begin * a.k_row + w.kv_head * a.k_head;
    const T *v_base = static_cast<const T *>(a.v) + w.k_begin * a.v_row + w.kv_head * a.v_head;
    const uint8_t *mask = a.key_mask ? a.key_mask + w.k_begin : nullptr;

    KeyStage<T, kKeys, kDim, C::kStage> in(thread, a.dim);
    int buffer = 0;

    int t = w.split * per + (kSplitKeys ? wave : 0);
    if (t < t_end) in.fetch(a, k_base, v_base, mask, w.keys, t);
    vec8<T> qf[kSteps];  // a wave without keys needs none
    {
        const T *q = static_cast<const T *>(a.q) + q_row * a.q_row + head * a.q_head;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int d = 16 * s + 8 * half;
            qf[s] = row_ok && d < a.dim && t < t_end ? *reinterpret_cast<const vec8<T> *>(q + d) : vec8<T>(T(0.f));
        }
    }
    for (; t < t_end; t += t_step) {
        if (kSplitKeys) wave_sync();
        const uint64_t valid = in.store(k_tile, v_tile);
        if (kSplitKeys) wave_sync(); else __syncthreads();
        const int k0 = t * kKeys;
        in.fetch(a, k_base, v_base, mask, w.keys, min(t + t_step, t_end - 1));  // at the end, again the last

        f32x16 s[kSub];
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
            s[u] = f32x16{};
            const int row = 32 * u + permuted_row(lane & 31);
#pragma unroll
            for (int i = 0; i < kSteps; ++i) s[u] = mma(s[u], row_operand(k_tile, kRow, row, 16 * i, half), qf[i]);
        }
        if (valid != ~0ull) {
            rare();
#pragma unroll
            for (int u = 0; u < kSub; ++u)
                each_score(static_cast<uint32_t>(valid >> (32 * u)), half,
                           [&](int i, bool used) { s[u][i] = used ? s[u][i] : -INFINITY; });
        }
        float high = s[0][0];
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
#pragma unroll
            for (int i = 0; i < 16; ++i) high = fmaxf(high, s[u][i]);
        }
        high = max_halves(high);
        // top = -inf (nothing seen yet) always moves on; a row that has seen nothing stays there
        if (__any((high - top) * c > kLag || (top == -INFINITY && high > -INFINITY))) {
            rare();
            const float now = fmaxf(top, high);
            const float scale = now == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((top - now) * c);
            sum *= scale;
#pragma unroll
            for (int d = 0; d < kOut; ++d) o[d] *= scale;
            top = now;
        }
        const float shift = top == -INFINITY ? 0.f : top * c;
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
            vec8<T> p[2];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float e = __builtin_amdgcn_exp2f(fmaf(s[u][i], c, -shift));
                sum += e;
                s[u][i] = e;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x8 e;
#pragma unroll
                for (int j = 0; j < 8; ++j) e[j] = s[u][8 * h + j];
                if (kDrop) {
                    const uint32_t keep = keep_bits(g, (k0 + 32 * u + 16 * h) / 8 + half, drop_row, a.threshold);
#pragma unroll
                    for (int j = 0; j < 8; ++j) e[j] = (keep >> j & 1) ? e[j] : 0.f;
                }
                // 16-bit types round p once, as the product takes it: with that out has 1.3 to 1.4 times the
                // error of rounding it alone; the rest as a second term would be half as many products more.
                p[h] = from_f32<T>(e);
            }
#pragma unroll
            for (int d = 0; d < kOut; ++d) {
                o[d] = mma(o[d], column_operand(v_tile, kRow, 32 * u, 32 * d, lane), p[0]);
                o[d] = mma(o[d], column_operand(v_tile, kRow, 32 * u + 16, 32 * d, lane), p[1]);
            }
        }
        // shared tiles have two buffers: one barrier a tile, since no wave is a whole tile ahead
        if (!kSplitKeys) {
            k_tile = reinterpret_cast<T *>(lds) + (buffer ^= 1) * 2 * C::kTile;
            v_tile = k_tile + C::kTile;
        }
    }
    sum = sum_halves(sum);

    const int64_t at = q_row * a.heads + head;
    if (!kSplitKeys) {
        if (!row_ok) return;
        const float lse2 = sum > 0.f || sum != sum ? top * c + __builtin_amdgcn_logf(sum) : -INFINITY;
        const float norm = sum > 0.f || sum != sum ? a.keep_scale / sum : 0.f;
        if (splits > 1) {
            const int64_t to = int64_t(w.split) * a.q_rows * a.heads + at;
            if (half == 0) partial.lse[to] = lse2;
#pragma unroll
            for (int d = 0; d < kOut; ++d) {
                each_eight(o[d], half, [&](int i, f32x8 v) {
                    if (32 * d + 8 * i < a.dim) store8(partial.out + to * a.dim + 32 * d + 8 * i, v * norm);
                });
            }
            return;
        }
        if (half == 0) a.lse[at] = lse2 * kLn2;
        T *out = static_cast<T *>(a.out) + at * a.dim;
#pragma unroll
        for (int d = 0; d < kOut; ++d) {
            each_eight(o[d], half, [&](int i, f32x8 v) {
                if (32 * d + 8 * i < a.dim) store8(out + 32 * d + 8 * i, from_f32<T>(v * norm));
            });
        }
        return;
    }

    // join the four waves: every one has its own maximum, sum and output for the same 32 rows
    __syncthreads();
    float *join = reinterpret_cast<float *>(lds), *join_top = join + kWaves * 32 * C::kJoinRow,
          *join_sum = join_top + kWaves * 32;
    float *mine = join + (wave * 32 + (lane & 31)) * C::kJoinRow;
#pragma unroll
    for (int d = 0; d < kOut; ++d) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 v = {o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
            *reinterpret_cast<f32x4 *>(mine + 32 * d + 8 * i + 4 * half) = v;
        }
    }
    if (half == 0) {
        join_top[wave * 32 + lane] = top;
        join_sum[wave * 32 + lane] = sum;
    }
    __syncthreads();
    const int jr = threadIdx.x >> 3, jc = threadIdx.x & 7, row = w.first + jr;  // eight threads a row
    if (row >= w.rows) return;
    float most = -INFINITY, total = 0.f, weight[kWaves];
#pragma unroll
    for (int i = 0; i < kWaves; ++i) most = fmaxf(most, join_top[i * 32 + jr]);
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        const float m = join_top[i * 32 + jr];
        weight[i] = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m - most) * c);
        // a wave that saw nothing has a zero sum; one that saw a NaN has a NaN
        total += join_sum[i * 32 + jr] * (m == -INFINITY ? 1.f : weight[i]);
    }
    const bool seen = total > 0.f || total != total;
    const float lse2 = seen ? most * c + __builtin_amdgcn_logf(total) : -INFINITY;
    const float norm = seen ? a.keep_scale / total : 0.f;
    const int64_t q_out = (w.q_begin + row / a.share) * a.heads + w.kv_head * a.share + row % a.share;
    const int64_t to = int64_t(w.split) * a.q_rows * a.heads + q_out;
    if (jc == 0) {
        if (splits > 1)
            partial.lse[to] = lse2;
        else
            a.lse[q_out] = lse2 * kLn2;
    }
    for (int col = jc * 8; col < a.dim; col += 64) {
        f32x8 v = {};
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            const float *from = join + (i * 32 + jr) * C::kJoinRow + col;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += from[j] * weight[i];
        }
        v *= norm;
        if (splits > 1)
            store8(partial.out + to * a.dim + col, v);
        else
            store8(static_cast<T *>(a.out) + q_out * a.dim + col, from_f32<T>(v));
    }
}

// Joins the splits: eight columns of one (query row, head) a thread, kLanes threads for the
// columns times kGroups that share the splits.
template <class T, int kLanes, int kGroups>
__global__ void __launch_bounds__(kThreads) k_join(AttnArgs a, int splits, Partial partial) {
    constexpr int kAhead = 4, kRow = kLanes * kGroups;
    const int64_t n = a.q_rows * a.heads, at = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / kRow;
    const int col = threadIdx.x % kLanes * 8, group = threadIdx.x % kRow / kLanes;
    // Rows that no structure holds have no partial results and are not written.  Whole rows of threads
    // end here: the exchanges below stay within one.
    const Span held = span_of(a.q_ptr[0], a.q_ptr[a.n_struct], a.q_rows);
    if (at < held.begin * a.heads || at >= held.end * a.heads) return;
    float most = -INFINITY, total = 0.f, bad = 0.f;
    f32x8 v = {};
    for (int first = group; first < splits; first += kGroups * kAhead) {
        float l[kAhead];
        f32x8 o[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int s = first + i * kGroups;
            l[i] = s < splits ? partial.lse[s * n + at] : -INFINITY;
            o[i] = s < splits && col < a.dim ? load8(partial.out + (s * n + at) * a.dim + col) : f32x8{};
        }
        float high = most;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            high = fmaxf(high, l[i]);
            if (l[i] != l[i]) bad = l[i];  // the maximum leaves a NaN out
        }
        const float scale = most == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(most - high);
        v *= scale;
        total *= scale;
        most = high;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const float weight = l[i] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(l[i] - most);
            v += o[i] * weight;
            total += weight;
        }
    }
    if (kGroups > 1) {
        float high = most;
#pragma unroll
        for (int off = kLanes; off < kRow; off <<= 1) high = fmaxf(high, __shfl_xor(high, off));
        const float scale = most == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(most - high);
        v *= scale;
        total *= scale;
        most = high;
#pragma unroll
        for (int off = kLanes; off < kRow; off <<= 1) {
            total += __shfl_xor(total, off);
            bad += __shfl_xor(bad, off);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += __shfl_xor(v[j], off);
        }
    }
    total += bad;
    if (group != 0 || col >= a.dim) return;
    const bool seen = total > 0.f || total != total;
    if (col == 0) a.lse[at] = seen ? (most + __builtin_amdgcn_logf(total)) * kLn2 : -INFINITY;
    store8(static_cast<T *>(a.out) + at * a.dim + col, from_f32<T>(v * (seen ? 1.f / total : 0.f)));
}

constexpr size_t up(size_t v) { return (v + 255) / 256 * 256; }

struct Choice {
    bool split_keys;
    int splits;
    int64_t slots, blocks;
};

Choice choose(const AttnArgs &a) {
    Choice c;
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

template <class T, int kDim, bool kDrop>
void launch(const AttnArgs &a, const Choice &c, const Partial &partial, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(c.blocks)), threads(kThreads);
    // At 33 to 64 columns of a 16-bit type a compute unit would hold three workgroups, and with about
    // two for each some get three and some one.  LDS that nothing uses keeps them to two there (the
    // 512 workgroups above: 36 us for 43, with dropout 51 for 65; but 23 us for 17 where 768
    // workgroups of 64 structures, many of them empty, can use the third place).  The count has slots
    // without rows in it, so the bound is a rough one: at 560 the two places win (4 x 384 rows: 27 us for 30), at
    // 608 and 640 the three (4 x 1152: 44 for 53), and at 576 either does (4 x 512: 26 for 29 with two;
    // 8 x 512: 43 for 49 with three).
    const unsigned spare = sizeof(T) == 2 && kDim == 64 && c.blocks <= 576 ? 20480 : 0;
    if (c.split_keys)
        k_forward<T, kDim, kDrop, true><<<grid, threads, 0, stream>>>(a, c.splits, c.slots, partial);
    else
        k_forward<T, kDim, kDrop, false><<<grid, threads, spare, stream>>>(a, c.splits, c.slots, partial);
}

template <class T, int kDim>
void launch(const AttnArgs &a, const Choice &c, const Partial &partial, hipStream_t stream) {
    if (a.threshold)
        launch<T, kDim, true>(a, c, partial, stream);
    else
        launch<T, kDim, false>(a, c, partial, stream);
}

size_t partial_out(const AttnArgs &a, const Choice &c) {
    return up(static_cast<size_t>(c.splits) * a.q_rows * a.heads * a.dim * sizeof(float));
}

template <class T>
hipError_t forward(const AttnArgs &a, hipStream_t stream) {
    const Choice c = choose(a);
    Partial partial{};
    if (c.splits > 1) {
        partial.out = static_cast<float *>(a.workspace);
        partial.lse = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + partial_out(a, c));
    }
    if (a.dim <= 32)
        launch<T, 32>(a, c, partial, stream);
    else if (a.dim <= 64)
        launch<T, 64>(a, c, partial, stream);
    else if (a.dim <= 96)
        launch<T, 96>(a, c, partial, stream);
    else
        launch<T, 128>(a, c, partial, stream);
    if (c.splits > 1) {
        const int64_t n = a.q_rows * a.heads;
        const auto join = [&](auto lanes) {
            constexpr int kLanes = decltype(lanes)::value;
            // many splits are shared by the threads of a wave, since they come with few rows
            const int row = c.splits > 4 ? 64 : kLanes;
            const dim3 grid(static_cast<unsigned>((n * row + kThreads - 1) / kThreads));
            if (c.splits > 4)
                k_join<T, kLanes, 64 / kLanes><<<grid, dim3(kThreads), 0, stream>>>(a, c.splits, partial);
            else
                k_join<T, kLanes, 1><<<grid, dim3(kThreads), 0, stream>>>(a, c.splits, partial);
        };
        if (a.dim <= 32)
            join(std::integral_constant<int, 4>());
        else if (a.dim <= 64)
            join(std::integral_constant<int, 8>());
        else
            join(std::integral_constant<int, 16>());
    }
    return hipGetLastError();
}

}  // namespace

size_t cross_attn_fwd_workspace(oeq_dtype, const AttnArgs &a) {
    const Choice c = choose(a);
    if (c.splits == 1) return 0;
    return partial_out(a, c) + up(static_cast<size_t>(c.splits) * a.q_rows * a.heads * sizeof(float));
}

int64_t cross_attn_fwd_blocks(oeq_dtype, const AttnArgs &a) { return choose(a).blocks; }

hipError_t cross_attn_fwd(oeq_dtype dtype, const AttnArgs &a, hipStream_t stream) {
    switch (dtype) {
        case OEQ_F32: return forward<float>(a, stream);
        case OEQ_F16: return forward<f16>(a, stream);
        case OEQ_BF16: return forward<bf16>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace readout
}  // namespace oeq
