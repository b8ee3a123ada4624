// Attention forward: cross (cross_attn_fwd.hip) and causal (causal_attn_fwd.hip).  For the visible keys of a
// query row's structure
//   s = scale q k^T,  lse = log sum exp s,  p = exp(s - lse),  out = (p * keep) v
// in one pass over the keys with a running maximum and sum.
//
// A wave computes S^T = K Q^T tile by tile with its 32 query rows along the lanes, so the
// softmax statistics are one number a lane, and O^T = V^T P^T takes the probabilities
// straight from the score registers (attn_device.hpp).  K and V pass through LDS; V's
// operand is read transposed from it.
//
// Two ways to split the work (kSplitKeys):
//   false: the four waves own 32 query rows each and share tiles of 64 keys (causal fp32 of 32);
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
//
// Causal (kCausal): a workgroup ends with the last key that its last row sees, and only tiles that reach past
// what a wave's first row sees are masked, each lane by its own row.  A key that a row does not see has
// the probability zero there, but its value is in the tile: if it is infinite or NaN, the product
// leaves a NaN.  So a walk whose sums are not finite is done again with care (finite_only, add_others).
#pragma once

#include "attn_device.hpp"

namespace oeq {
namespace readout {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;
// The running maximum may lag behind by this many powers of two before the sums are scaled, so that most
// tiles scale nothing (a device known from published attention kernels).
constexpr float kLag = 8.f;

template <class T, int kDim, bool kSplitKeys, bool kCausal>
struct Tiles {
    // Causal fp32 above 32 columns: half a tile that the limit cuts off is not multiplied, which pays for the
    // barriers (64 sequences of up to 200 rows, 8 heads of 64: 53 -> 46 us, of 128 95 -> 88, 32 x 400 rows of 96 211 ->
    // 181; 16 x 800 rows of 128 338 -> 347, and at D = 32 16 x 800 rows 95 -> 102).
    static constexpr int kKeys = kSplitKeys || (kCausal && sizeof(T) == 4 && kDim > 32) ? 32 : 64;
    static constexpr int kRow = kTileRow<T, kDim>;
    static constexpr int kRows = kSplitKeys ? 32 : 128;  // query rows of a workgroup
    static constexpr int kStage = kSplitKeys ? 64 : kThreads;
    static constexpr int kTile = kKeys * kRow;  // elements of one K or V tile
    static constexpr int kLds = (kSplitKeys ? kWaves : 2) * 2 * kTile * int(sizeof(T));
    static constexpr int kJoinRow = kDim + 4;
    static constexpr int kJoin = kSplitKeys ? kWaves * 32 * (kJoinRow + 2) * 4 : 0;
    static constexpr int kBytes = kLds > kJoin ? kLds : kJoin;
};

// Whether `v` holds in a wave of the workgroup.
__device__ __forceinline__ bool any_wave(bool v) {
    __shared__ int of_wave[kWaves];
    if ((threadIdx.x & 63) == 0) of_wave[threadIdx.x >> 6] = v;
    __syncthreads();
    return of_wave[0] | of_wave[1] | of_wave[2] | of_wave[3];
}

struct Partial {
    float *out;  // [split][query row, head][dim], normalised
    float *lse;  // [split][query row, head], in powers of two
    // causal: walks of different lengths are cut into pieces of about this many tiles, at most `splits` of them (0:
    // all into `splits`); [query row, head]: into how many
    int piece;
    int32_t *pieces;
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

// The waves' rows (or keys) of a workgroup.  kCausal: walks grow from wave to wave, and the workgroups of a compute
// unit, 256 blocks apart, take them in turn forwards and backwards, so that no SIMD has all the long ones.
template <bool kCausal>
__device__ __forceinline__ int part_of(int wave) {
    return kCausal && (blockIdx.x >> 8 & 1) ? kWaves - 1 - wave : wave;
}

// Workgroups that a compute unit is to hold of the causal kernels, where registers allow it.
template <class T, int kDim>
constexpr int kHeld = sizeof(T) == 4 ? 1 : kDim <= 32 ? 3 : 2;

// In pairs: a chain of sixteen additions would be waited for.
__device__ __forceinline__ float sum_of(f32x16 v) {
#pragma unroll
    for (int n = 8; n > 0; n >>= 1) {
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] += v[n + i];
    }
    return v[0];
}

template <class T, int kDim, bool kDrop, bool kSplitKeys, bool kCausal>
__global__ void __launch_bounds__(kThreads, (kCausal ? kHeld<T, kDim> : 1))
    k_forward(AttnArgs a, int splits, int64_t slots, Partial partial) {
    using C = Tiles<T, kDim, kSplitKeys, kCausal>;
    constexpr int kKeys = C::kKeys, kRow = C::kRow, kSteps = kDim / 16, kOut = kDim / 32, kSub = kKeys / 32;
    __shared__ __attribute__((aligned(16))) char lds[C::kBytes];
    const Place w = place_of<C::kRows, kCausal>(a, blockIdx.x, true, splits, slots, partial.piece == 0);
    if (!w.any) return;
    const int lane = threadIdx.x & 63, half = lane >> 5, wave = threadIdx.x >> 6;
    const int thread = kSplitKeys ? lane : threadIdx.x;
    T *k_tile = reinterpret_cast<T *>(lds) + (kSplitKeys ? wave * 2 * C::kTile : 0), *v_tile = k_tile + C::kTile;

    // this lane's query row
    const int base = w.first + (kSplitKeys ? 0 : part_of<kCausal>(wave) * 32), r = base + (lane & 31);
    const bool row_ok = r < w.rows;
    const int64_t q_row = w.q_begin + (row_ok ? r / a.share : 0);
    const int head = w.kv_head * a.share + (row_ok ? r % a.share : 0);
    Rng g{};
    if (kDrop) g = load_rng(a.rng);
    const uint32_t drop_row = static_cast<uint32_t>(q_row * a.heads + head);

    const float c = a.scale * kLog2E;
    f32x16 o[kOut] = {};
    float top = -INFINITY, sum = 0.f;  // the running maximum (unscaled) and this half's sum

    // Causal: the keys that the workgroup's last row sees, and the last that this lane's and the wave's first and
    // last rows do
    int keys = w.keys, limit = 0, wave_first = 0, wave_last = 0;
    if (kCausal) {
        const int off = causal_offset(a, w), most = w.rows - 1;
        keys = max(0, min(keys, min(w.first + C::kRows - 1, most) / a.share + off + 1));
        limit = min(r, most) / a.share + off;
        wave_first = __builtin_amdgcn_readfirstlane(min(base, most) / a.share + off);
        wave_last = __builtin_amdgcn_readfirstlane(min(base + 31, most) / a.share + off);
    }
    // this workgroup's keys, in whole tiles
    const int n_tiles = (keys + kKeys - 1) / kKeys;
    int pieces = splits;
    if (kCausal && partial.piece) {
        pieces = max(1, min(splits, (n_tiles + partial.piece - 1) / partial.piece));
        if (w.split >= pieces) return;
        if (w.split == 0 && threadIdx.x < C::kRows) {
            const int row = w.first + static_cast<int>(threadIdx.x);
            if (row < w.rows)
                partial.pieces[(w.q_begin + row / a.share) * a.heads + w.kv_head * a.share + row % a.share] = pieces;
        }
    }
    const int per = (n_tiles + pieces - 1) / pieces;
    const int t_end = min(n_tiles, (w.split + 1) * per), t_step = kSplitKeys ? kWaves : 1;
    const T *k_base = static_cast<const T *>(a.k) + w.k_begin * a.k_row + w.kv_head * a.k_head;
    const T *v_base = static_cast<const T *>(a.v) + w.k_begin * a.v_row + w.kv_head * a.v_head;
    const uint8_t *mask = a.key_mask ? a.key_mask + w.k_begin : nullptr;

    KeyStage<T, kKeys, kDim, C::kStage> in(thread, a.dim);
    int buffer = 0;

    const int t_begin = w.split * per + (kSplitKeys ? wave : 0);
    int t = t_begin;
    if (t < t_end) in.fetch(a, k_base, v_base, mask, keys, t);
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
        in.fetch(a, k_base, v_base, mask, keys, min(t + t_step, t_end - 1));  // at the end, again the last
        const auto turn = [&]() {
            // shared tiles have two buffers: one barrier a tile, since no wave is a whole tile ahead
            if (!kSplitKeys) {
                k_tile = reinterpret_cast<T *>(lds) + (buffer ^= 1) * 2 * C::kTile;
                v_tile = k_tile + C::kTile;
            }
        };
        if (kCausal && k0 > wave_last) {  // no row of this wave sees any of it
            turn();
            continue;
        }

        f32x16 s[kSub];
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
            s[u] = f32x16{};
            const int row = 32 * u + permuted_row(lane & 31);
#pragma unroll
            for (int i = 0; i < kSteps; ++i) s[u] = mma(s[u], row_operand(k_tile, kRow, row, 16 * i, half), qf[i]);
        }
        // Between the products a wave goes first: with two waves on a SIMD, one's exponentials then run beside the
        // other's products (2 x 4096 rows, 16 heads over 4, D = 128, fp16: 181 -> 172 us)
        if (kCausal) __builtin_amdgcn_s_setprio(1);
        uint64_t used_keys = valid;
        const bool cut = kCausal && k0 + kKeys - 1 > wave_first;  // some row of the wave sees only a part
        if (cut) used_keys &= low_bits(limit - k0 + 1);
        if (valid != ~0ull || cut) {
            rare();
#pragma unroll
            for (int u = 0; u < kSub; ++u)
                each_score(static_cast<uint32_t>(used_keys >> (32 * u)), half,
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
                if (!kCausal) sum += e;
                s[u][i] = e;
            }
            if (kCausal) sum += sum_of(s[u]);
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
        if (kCausal) __builtin_amdgcn_s_setprio(0);
        turn();
    }
    if constexpr (kCausal) {
        if (any_wave(__any(row_ok && !finite(o)))) {
            rare();
            // again with care: the maximum and the sum are known, tiles are neither read ahead nor taken together
#pragma unroll
            for (int d = 0; d < kOut; ++d) o[d] = f32x16{};
            const float shift = top == -INFINITY ? 0.f : top * c;
#pragma unroll 1
            for (t = t_begin; t < t_end; t += t_step) {
                in.fetch(a, k_base, v_base, mask, keys, t);
                if (kSplitKeys) wave_sync(); else __syncthreads();
                const uint64_t valid = in.store(k_tile, v_tile);
                if (kSplitKeys) wave_sync(); else __syncthreads();
                const int k0 = t * kKeys;
                if (k0 > wave_last) continue;
#pragma unroll 1
                for (int u = 0; u < kSub; ++u) {
                    const T *k_sub = k_tile + 32 * u * kRow, *v_sub = v_tile + 32 * u * kRow;
                    const int first = k0 + 32 * u;
                    const uint32_t used = static_cast<uint32_t>(valid >> (32 * u) & low_bits(limit - first + 1));
                    const bool cut = first + 31 > wave_first;
                    f32x16 s = {};
#pragma unroll
                    for (int i = 0; i < kSteps; ++i)
                        s = mma(s, row_operand(k_sub, kRow, permuted_row(lane & 31), 16 * i, half), qf[i]);
                    each_score(used, half, [&](int i, bool in) {
                        s[i] = in ? __builtin_amdgcn_exp2f(fmaf(s[i], c, -shift)) : 0.f;
                    });
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        f32x8 e;
                        const uint32_t keep =
                            kDrop ? keep_bits(g, (first + 16 * h) / 8 + half, drop_row, a.threshold) : 0xFFu;
#pragma unroll
                        for (int j = 0; j < 8; ++j) e[j] = (keep >> j & 1) ? s[8 * h + j] : 0.f;
                        const vec8<T> p = from_f32<T>(e);
#pragma unroll
                        for (int d = 0; d < kOut; ++d) {
                            vec8<T> v = column_operand(v_sub, kRow, 16 * h, 32 * d, lane);
                            if (cut) v = finite_only<T>(v);
                            o[d] = mma(o[d], v, p);
                        }
                    }
                    if (cut) add_others<false>(o, v_sub, kRow, used, half);
                }
            }
        }
    }
    sum = sum_halves(sum);

    const int64_t at = q_row * a.heads + head;
    if (!kSplitKeys) {
        if (!row_ok) return;
        const float lse2 = sum > 0.f || sum != sum ? top * c + __builtin_amdgcn_logf(sum) : -INFINITY;
        const float norm = sum > 0.f || sum != sum ? a.keep_scale / sum : 0.f;
        if (pieces > 1) {
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
        if (pieces > 1)
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
        if (pieces > 1)
            store8(partial.out + to * a.dim + col, v);
        else
            store8(static_cast<T *>(a.out) + q_out * a.dim + col, from_f32<T>(v));
    }
    return;
}

// Joins the splits: eight columns of one (query row, head) a thread, kLanes threads for the
// columns times kGroups that share the splits.
template <class T, int kLanes, int kGroups, bool kCausal>
__global__ void __launch_bounds__(kThreads) k_join(AttnArgs a, int splits, Partial partial) {
    constexpr int kAhead = 4, kRow = kLanes * kGroups;
    const int64_t n = a.q_rows * a.heads, at = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / kRow;
    const int col = threadIdx.x % kLanes * 8, group = threadIdx.x % kRow / kLanes;
    // Rows that no structure holds have no partial results and are not written.  Whole rows of threads
    // end here: the exchanges below stay within one.
    const Span held = span_of(a.q_ptr[0], a.q_ptr[a.n_struct], a.q_rows);
    if (at < held.begin * a.heads || at >= held.end * a.heads) return;
    if (kCausal && partial.piece) {
        // (rows that a row pointer which decreases leaves out have no count: any, within the workspace)
        splits = max(1, min(partial.pieces[at], splits));
        if (splits == 1) return;  // written by its walk
    }
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
    int splits, piece;  // piece: see Partial
    int64_t slots, blocks;
};

template <class T, int kDim, bool kDrop, bool kCausal>
void launch(const AttnArgs &a, const Choice &c, const Partial &partial, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(c.blocks)), threads(kThreads);
    // At 33 to 64 columns of a 16-bit type a compute unit would hold three workgroups, and with about
    // two for each some get three and some one.  LDS that nothing uses keeps them to two there (the
    // 512 workgroups above: 36 us for 43, with dropout 51 for 65; but 23 us for 17 where 768
    // workgroups of 64 structures, many of them empty, can use the third place).  The count has slots
    // without rows in it, so the bound is a rough one: at 560 the two places win (4 x 384 rows: 27 us for 30), at
    // 608 and 640 the three (4 x 1152: 44 for 53), and at 576 either does (4 x 512: 26 for 29 with two;
    // 8 x 512: 43 for 49 with three).
    const unsigned spare = sizeof(T) == 2 && kDim == 64 && c.blocks <= 576 && c.piece == 0 ? 20480 : 0;
    if (c.split_keys)
        k_forward<T, kDim, kDrop, true, kCausal><<<grid, threads, 0, stream>>>(a, c.splits, c.slots, partial);
    else
        k_forward<T, kDim, kDrop, false, kCausal><<<grid, threads, spare, stream>>>(a, c.splits, c.slots, partial);
}

template <class T, int kDim, bool kCausal>
void launch(const AttnArgs &a, const Choice &c, const Partial &partial, hipStream_t stream) {
    if (a.threshold)
        launch<T, kDim, true, kCausal>(a, c, partial, stream);
    else
        launch<T, kDim, false, kCausal>(a, c, partial, stream);
}

inline size_t partial_out(const AttnArgs &a, const Choice &c) {
    return up(static_cast<size_t>(c.splits) * a.q_rows * a.heads * a.dim * sizeof(float));
}
inline size_t partial_lse(const AttnArgs &a, const Choice &c) {
    return up(static_cast<size_t>(c.splits) * a.q_rows * a.heads * sizeof(float));
}

template <class T, bool kCausal>
hipError_t forward(const AttnArgs &a, const Choice &c, hipStream_t stream) {
    Partial partial{};
    if (c.splits > 1) {
        partial.out = static_cast<float *>(a.workspace);
        partial.lse = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + partial_out(a, c));
        partial.pieces = reinterpret_cast<int32_t *>(static_cast<char *>(a.workspace) + partial_out(a, c) + partial_lse(a, c));
        partial.piece = c.piece;
    }
    if (a.dim <= 32)
        launch<T, 32, kCausal>(a, c, partial, stream);
    else if (a.dim <= 64)
        launch<T, 64, kCausal>(a, c, partial, stream);
    else if (a.dim <= 96)
        launch<T, 96, kCausal>(a, c, partial, stream);
    else
        launch<T, 128, kCausal>(a, c, partial, stream);
    if (c.splits > 1) {
        const int64_t n = a.q_rows * a.heads;
        const auto join = [&](auto lanes) {
            constexpr int kLanes = decltype(lanes)::value;
            // many splits are shared by the threads of a wave, since they come with few rows (not where walks have
            // as many as their length asks for)
            const bool share = c.splits > 4 && c.piece == 0;
            const int row = share ? 64 : kLanes;
            const dim3 grid(static_cast<unsigned>((n * row + kThreads - 1) / kThreads));
            if (share)
                k_join<T, kLanes, 64 / kLanes, kCausal><<<grid, dim3(kThreads), 0, stream>>>(a, c.splits, partial);
            else
                k_join<T, kLanes, 1, kCausal><<<grid, dim3(kThreads), 0, stream>>>(a, c.splits, partial);
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

inline size_t forward_workspace(const AttnArgs &a, const Choice &c, bool causal) {
    if (c.splits == 1) return 0;
    return partial_out(a, c) + partial_lse(a, c) + (causal ? up(static_cast<size_t>(a.q_rows) * a.heads * 4) : 0);
}

}  // namespace
}  // namespace readout
}  // namespace oeq
