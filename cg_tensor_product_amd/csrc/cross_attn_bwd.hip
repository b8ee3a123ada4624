// Cross attention backward.  With p = exp(scale q k^T - lse) formed again from the saved
// log sums, f the dropout factors (0 or 1 / share kept) and delta = sum_d grad_out out:
//   grad_v = (p f)^T grad_out            dp = (grad_out v^T) f
//   ds = p (dp - delta)                  grad_q = scale ds k,  grad_k = scale ds^T q
// One kernel in two roles, and no atomics:
//   grad_keys     a wave owns 32 keys (k, v and both gradients in registers) and walks the
//                 query rows of the structure, all heads that share the keys among them, so
//                 the sum over shared heads needs no further step;
//   grad_queries  a wave owns 32 query rows and walks the keys, like the forward.
// Both form delta themselves, from rows that they read anyway and from out.  Where out is
// rounded to 16 bits and a structure has few states (kExactStates), that rounding would be
// most of its gradients' error: there, in one tile of keys, delta is the sum of p dp in fp32.
// Scores are formed twice (7 products of the minimal 5; 10 for 16-bit types with the second terms of
// probabilities and score gradients); the alternative, one walk that adds into grad_q, needs atomics or a partial
// grad_q for each tile of keys.  With few workgroups the walks are split over workgroups, whose
// fp32 partial sums a second kernel adds in order.
//
// Bound by the vector unit next to the matrix unit, fp32 by its matrix instructions: 4 structures of
// 1024 query rows and 2048 states, 8 heads over 4, D = 64: bf16 118 us (364 TFLOP/s of the minimal
// products; 149 us with dropout, whose generator runs in both roles), fp16 120 and 150, fp32 482 us (89
// TFLOP/s).
//
// The product that gives dp starts from -delta / (factor of what is kept) in its accumulators,
// so that a score's gradient is one multiplication, and the factor is applied to the sums.
#include "attn_device.hpp"

namespace oeq {
namespace readout {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kKeyTile = 128;  // keys of a workgroup that owns keys
constexpr int kRowTile = 32;   // query rows of a step of its walk
// Structures of so many states, one tile of one wave, sum p dp for delta.  From the rounded out instead,
// grad_q and grad_k have 3.0 times the error that rounding the result has at 2 states, 2.1 at 4, 1.7 at
// 8, 1.3 at 32 and 1.2 at 64 (1.0 from p dp).  It goes by each structure's length, so its gradients do not
// depend on what else is in its batch.
constexpr int kExactStates = 32;
template <class T>
constexpr bool kExactDelta = sizeof(T) == 2;

// Probabilities and score gradients of 16-bit types go into their products as two terms, the rounded value
// and the rest.  Rounded once, score gradients (with delta's rounding) leave grad_q and grad_k with 1.4 to 1.9
// times the error that rounding the result alone does (10 to 4096 states), probabilities grad_v with 1.4
// to 1.6 times; with the rest it is 1.0 to 1.2 from 64 states on.  For the score gradients that costs 7 % of a
// decoder's training step (8 structures of up to 1024 query rows and 2048 states, 8 heads over 4, D = 64,
// bf16, dropout: 206 -> 221 us), for the probabilities 5 to 8 % of the backward (159 -> 172 us there).
template <class T>
constexpr bool kRest = sizeof(T) == 2;

// fp16 ends at 2^-24 and 65504, and score gradients, about grad_out / states, leave that range at both
// ends.  So they are brought into it by a power of two, chosen ahead of a walk: |grad_out| (|v| + |out|),
// of rows at hand, bounds |dp - delta| within a small factor if the other rows are alike, and p |dp - delta|
// is put where that bound is 2^14; what p = 2^-17 leaves of it still lies 2^22 above the last bit.
//   grad_queries  a power for each row, which is a lane and a column of its sums; p carries it;
//   grad_keys     one for the workgroup: p carries 2^kProbBits (of it grad_v too: probabilities near
//                 2^-16 would keep eight bits, and keep all), the rows of grad_out in LDS the rest.
// Where a walk meets rows so much larger that a score gradient passes 65504, its sums are no longer
// finite (as where an input is not), and it is done again: that of queries with the powers that a walk for
// the largest of each row finds, that of keys with care (kCare): a power for each key, from 2^60 on, falls
// with the tile whose largest reaches 2 so that this one gets 2^-6 .. 2^-5, and the sums are scaled along;
// what is lost is below 2^-19 of the column's largest.  With care from the start large calls take
// 10 % longer (D = 64: each tile waits for the check).
template <class T>
constexpr bool kScaled = std::is_same<T, f16>::value;
constexpr int kMostBits = 60;  // what is below 2^-60 is nothing to a result, and no product with it overflows fp32
template <class T, bool kCare>
constexpr int kProbBits = kScaled<T> ? (kCare ? 15 : 6) : 0;

__device__ __forceinline__ float power(int bits) { return __builtin_ldexpf(1.f, bits); }

// The power that puts a bound, given its square (0: not known), between 2^(to - 1) and 2^to.
__device__ __forceinline__ int bits_ahead(int to, float bound2) {
    return bound2 > 0.f ? min(to - ((__builtin_amdgcn_frexp_expf(bound2) + 1) >> 1), kMostBits) : 0;
}

// The power that brings the largest of a row between 2^13 and 2^14.
__device__ __forceinline__ int bits_for(float most) {
    return most > 0.f ? min(14 - __builtin_amdgcn_frexp_expf(most), kMostBits) : 0;
}

// Whether all sums are finite (they are far from where their own sum would not be).
template <int kOut>
__device__ __forceinline__ bool finite(const f32x16 (&sum)[kOut]) {
    f32x16 all = sum[0];
#pragma unroll
    for (int d = 1; d < kOut; ++d) all += sum[d];
#pragma unroll
    for (int n = 8; n > 0; n >>= 1) {
#pragma unroll
        for (int i = 0; i < n; ++i) all[i] += all[n + i];
    }
    return fabsf(all[0]) < INFINITY;
}
__device__ __forceinline__ float largest(f32x16 v) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]));
    return max_halves(m);
}
// Whether a value reaches 2: below it bit 14 of fp16 is clear.
__device__ __forceinline__ bool reaches_two(const vec8<f16> (&v)[2]) {
    using Words = uint32_t __attribute__((ext_vector_type(4)));
    const Words a = __builtin_bit_cast(Words, v[0]), b = __builtin_bit_cast(Words, v[1]);
    return ((a[0] | a[1] | a[2] | a[3] | b[0] | b[1] | b[2] | b[3]) & 0x40004000u) != 0;
}

// The largest `v` of the workgroup's waves, which all of them have then brought.  Calls of one kCall have
// another barrier between them.
template <int kCall>
__device__ __forceinline__ int max_wave(int v) {
    __shared__ int of_wave[kWaves];
    if ((threadIdx.x & 63) == 0) of_wave[threadIdx.x >> 6] = v;
    __syncthreads();
    return max(max(of_wave[0], of_wave[1]), max(of_wave[2], of_wave[3]));
}

struct Bwd {
    float *part_q;           // [split][query row, head][dim]
    float *part_k, *part_v;  // [split][key, key head][dim]
    int q_splits, k_splits;  // 1: gradients are written directly
    int64_t q_slots, k_slots;
    int64_t key_blocks;  // workgroups that own keys; the rest own query rows
};

// p from a score, times 2^bits where `lse` is less by that; fp32 forms scale s - lse in one
// rounding, since the difference is small against its parts.  `lse` is in powers of two for 16-bit
// types, and +infinity for a row that saw nothing, whose probabilities are zero.
template <class T>
__device__ __forceinline__ float probability(float s, float scale, float c, float lse) {
    if (sizeof(T) == 4) return __builtin_amdgcn_exp2f(fmaf(s, scale, -lse) * kLog2E);
    return __builtin_amdgcn_exp2f(fmaf(s, c, -lse));
}
template <class T>
__device__ __forceinline__ float kept_lse(float lse) {
    return lse == -INFINITY ? INFINITY : sizeof(T) == 4 ? lse : lse * kLog2E;
}

template <class T>
__device__ __forceinline__ float dot(vec8<T> a, vec8<T> b) {
    const f32x8 x = to_f32<T>(a), y = to_f32<T>(b);
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) v = fmaf(x[j], y[j], v);
    return v;
}

// Probabilities or score gradients as operands of a product: the rounded values and the rest.
template <class T>
__device__ __forceinline__ void two_terms(f32x8 v, vec8<T> *value, vec8<T> *rest) {
    *value = from_f32<T>(v);
    if (kRest<T>) *rest = from_f32<T>(v - to_f32<T>(*value));
}

// The step with care: lowers the power where a lane's score gradients `ds` reach 1 with it, scales the sums
// and forms the terms again.  Returns by how much.
template <class T, int kOut>
__device__ __forceinline__ int lower(f32x16 ds, bool used, f32x16 (&sum)[kOut], vec8<T> (&value)[2], vec8<T> (&rest)[2]) {
    const float most = largest(ds);
    const int by = used && most >= 1.f ? -5 - __builtin_amdgcn_frexp_expf(most) : 0;
    const float factor = power(by);
#pragma unroll
    for (int d = 0; d < kOut; ++d) sum[d] *= factor;
    ds *= factor;
    two_terms<T>(__builtin_shufflevector(ds, ds, 0, 1, 2, 3, 4, 5, 6, 7), &value[0], &rest[0]);
    two_terms<T>(__builtin_shufflevector(ds, ds, 8, 9, 10, 11, 12, 13, 14, 15), &value[1], &rest[1]);
    return by;
}

// Four consecutive columns of a gradient, to the fp32 partial sums or the result.
template <class T>
__device__ __forceinline__ void put4(float *part, void *out, int64_t at, f32x4 v) {
    using V4 = T __attribute__((ext_vector_type(4)));
    if (part)
        *reinterpret_cast<f32x4 *>(part + at) = v;
    else
        *reinterpret_cast<V4 *>(static_cast<T *>(out) + at) = __builtin_convertvector(v, V4);
}

__device__ __forceinline__ f32x8 load_lds8(const float *p) {
    const f32x4 a = reinterpret_cast<const f32x4 *>(p)[0], b = reinterpret_cast<const f32x4 *>(p)[1];
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <class T, int kDim>
struct KeyLds {
    static constexpr int kRow = kTileRow<T, kDim>;
    // two buffers, so that a step needs one barrier
    T q[2][kRowTile * kRow], g[2][kRowTile * kRow];
    float lse[2][kRowTile], delta[2][kRowTile];  // delta as the accumulators start from it
    uint32_t kept[kWaves][kRowTile];             // bit = key of the wave
};

// Sum over the 32 lanes of a half: sixteen by rotations, then both sixteens.
__device__ __forceinline__ float sum_half(float v) {
    const auto rotated = [](float x, auto by) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x120 + decltype(by)::value, 0xF, 0xF, true));
    };
    v += rotated(v, std::integral_constant<int, 8>());
    v += rotated(v, std::integral_constant<int, 4>());
    v += rotated(v, std::integral_constant<int, 2>());
    v += rotated(v, std::integral_constant<int, 1>());
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// kExact: the structure has kExactStates keys at most, all of them in the first wave, which forms delta
// from p dp; the other waves only bring rows.  kCare: see kScaled.  Returns false, without results, where the
// walk is to be done again with care.  `tid` is threadIdx.x.
template <class T, int kDim, bool kDrop, bool kExact, bool kCare>
__device__ __forceinline__ bool grad_keys(const AttnArgs &a, const Bwd &out, const Place &w, int tid, KeyLds<T, kDim> &lds) {
    constexpr int kRow = KeyLds<T, kDim>::kRow, kSteps = kDim / 16, kOut = kDim / 32;
    const int lane = tid & 63, half = lane >> 5, wave = tid >> 6;
    const int key = w.first + wave * 32 + (lane & 31);
    const bool key_ok = key < w.keys;
    const int64_t k_row = w.k_begin + (key_ok ? key : 0);
    const bool seen = key_ok && (!a.key_mask || a.key_mask[k_row]);

    using Stage = RowStage<T, kRowTile, kDim, kThreads>;
    Stage q_in(tid, a.dim), g_in(tid, a.dim), o_in(tid, a.dim);
    float lse_in = 0.f;
    const int n_tiles = (w.rows + kRowTile - 1) / kRowTile, per = (n_tiles + out.k_splits - 1) / out.k_splits;
    const int t_end = min(n_tiles, (w.split + 1) * per);
    const auto row_of = [&](int r, int64_t *q_row) {  // rows past the end: the last one
        r = min(r, w.rows - 1);
        const int in = r / a.share, head = w.kv_head * a.share + (r - in * a.share);
        *q_row = w.q_begin + in;
        return head;
    };
    const auto fetch = [&](int t) {
        int64_t at[Stage::kPieces];
#pragma unroll
        for (int i = 0; i < Stage::kPieces; ++i) {
            int64_t q_row;
            const int head = row_of(t * kRowTile + q_in.row + i * Stage::kStep, &q_row);
            at[i] = (q_row * a.heads + head) * a.dim + q_in.d;
            if (q_in.reads)
                q_in.v[i] = *reinterpret_cast<const vec8<T> *>(static_cast<const T *>(a.q) + q_row * a.q_row +
                                                               head * a.q_head + q_in.d);
        }
        if (q_in.reads) {
#pragma unroll
            for (int i = 0; i < Stage::kPieces; ++i) {
                g_in.v[i] = *reinterpret_cast<const vec8<T> *>(static_cast<const T *>(a.grad_out) + at[i]);
                if (!kExact) o_in.v[i] = *reinterpret_cast<const vec8<T> *>(static_cast<const T *>(a.out) + at[i]);
            }
        }
        if (tid < kRowTile) {
            int64_t q_row;
            const int r = t * kRowTile + tid, head = row_of(r, &q_row);
            lse_in = a.lse[q_row * a.heads + head];
        }
    };
    int t = w.split * per;
    if (t < t_end) fetch(t);

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
    const float c = a.scale * kLog2E, start = -1.f / a.keep_scale;
    f32x16 gk[kOut] = {}, gv[kOut] = {};
    constexpr int kProb = kProbBits<T, kCare>;
    int bits = kScaled<T> && kCare ? kMostBits - kProb : 0;  // with kProb the power of gk; not kCare: of grad_out
    if constexpr (kScaled<T> && !kCare) {
        // the rows that this wave brings for the first tile stand for all
        float gg = 0.f, oo = 0.f, vv = 0.f;
        if (t < t_end && q_in.reads) {
#pragma unroll
            for (int i = 0; i < Stage::kPieces; ++i) {
                gg += dot<T>(g_in.v[i], g_in.v[i]);
                oo += dot<T>(o_in.v[i], o_in.v[i]);
            }
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) vv += dot<T>(vf[s], vf[s]);
        // of its keys together, and of the waves the one with the largest bound; grad_out has to fit, too
        gg = sum_halves(sum_half(gg));
        const float bound2 = gg * sum_halves(sum_half(vv + oo));
        const int mine = min(bits_ahead(14 - kProb, bound2), bits_ahead(14, gg));
        bits = -max_wave<0>(__builtin_amdgcn_readfirstlane(-mine));
        bits = max(min(bits, 15), -24);  // what one factor of fp16 can be
    }
    float up = power(bits);

    for (int buffer = 0; t < t_end; ++t, buffer ^= 1) {
        const int r0 = t * kRowTile, in_tile = min(kRowTile, w.rows - r0);
        T *q_tile = lds.q[buffer], *g_tile = lds.g[buffer];
        if (!kExact) {
#pragma unroll
            for (int i = 0; i < Stage::kPieces; ++i) {
                const int row = q_in.row + i * Stage::kStep;
                if (kScaled<T> && !kCare) g_in.v[i] *= static_cast<T>(up);
                float v = q_in.reads ? dot<T>(g_in.v[i], o_in.v[i]) : 0.f;
#pragma unroll
                for (int off = 1; off < Stage::kLanes; off <<= 1) v += __shfl_xor(v, off);
                if (q_in.d == 0 && row < kRowTile) lds.delta[buffer][row] = row < in_tile ? v * start : 0.f;
            }
        }
        // Rows past the end are the last one again, as a row that saw nothing: their probabilities are
        // zero, and NaN only where the last row's are (zeros would give NaN against an infinite state).
        q_in.store(q_tile, true, 0);
        g_in.store(g_tile, true, 0);
        if (tid < kRowTile) {
            const float lse = kept_lse<T>(lse_in) - float(kProb);
            lds.lse[buffer][tid] = tid < in_tile ? lse : INFINITY;
        }
        if (kDrop) {
            // 32 rows x 4 generator blocks of this wave's keys, two a lane; a row's bits make a word
            wave_sync();
            int64_t q_row;
            const int head = row_of(r0 + (lane & 31), &q_row);
            const uint32_t row = static_cast<uint32_t>(q_row * a.heads + head);
            const uint32_t block = static_cast<uint32_t>(w.first + wave * 32) / 8 + 2 * half;
            const uint32_t bits = keep_bits(g, block, row, a.threshold) | keep_bits(g, block + 1, row, a.threshold) << 8;
            reinterpret_cast<uint16_t *>(lds.kept[wave])[(lane & 31) * 2 + half] = static_cast<uint16_t>(bits);
        }
        __syncthreads();
        fetch(min(t + 1, t_end - 1));  // at the end, again the last
        if (kExact && wave > 0) continue;

        f32x16 s = {}, dp = {};
#pragma unroll
        for (int i = 0; i < 4 && !kExact; ++i) {
            const f32x4 d = *reinterpret_cast<const f32x4 *>(lds.delta[buffer] + 16 * (i >> 1) + 8 * half + 4 * (i & 1));
#pragma unroll
            for (int j = 0; j < 4; ++j) dp[4 * i + j] = d[j];
        }
        const int row = permuted_row(lane & 31);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) s = mma(s, row_operand(q_tile, kRow, row, 16 * i, half), kf[i]);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) dp = mma(dp, row_operand(g_tile, kRow, row, 16 * i, half), vf[i]);
        vec8<T> pf[2], pl[2], sf[2], sl[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // rows 16 h + 8 half + j of the tile; none: what dp - delta is where the probability was
            // dropped.  Read again here rather than kept, where that saves spills (D = 96 with dropout
            // 228 -> 209 us; at D = 128, which spills either way, 341 -> 378).
            if (kDim < 128) asm volatile("" ::: "memory");
            const int first = 16 * h + 8 * half;
            f32x8 p8, s8, lse = load_lds8(lds.lse[buffer] + first), none;
            uint32_t kept[8];
            if (kDrop) {
                if (!kExact) none = load_lds8(lds.delta[buffer] + first);
                const uint4 *from = reinterpret_cast<const uint4 *>(lds.kept[wave] + first);
                const uint4 x = from[0], y = from[1];
                kept[0] = x.x, kept[1] = x.y, kept[2] = x.z, kept[3] = x.w;
                kept[4] = y.x, kept[5] = y.y, kept[6] = y.z, kept[7] = y.w;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = 8 * h + j;
                const float p = probability<T>(s[i], a.scale, c, lse[j]);
                if (kExact) {
                    const float seen_p = seen ? p : 0.f;
                    const bool keep = !kDrop || (kept[j] & (1u << (lane & 31)));
                    p8[j] = keep ? seen_p : 0.f;
                    const float d = keep ? dp[i] : 0.f;
                    s8[j] = seen_p * (d - sum_half(seen_p * d) * (1.f / (1 << kProb)));
                } else if (kDrop) {
                    const bool keep = kept[j] & (1u << (lane & 31));
                    p8[j] = keep ? p : 0.f;
                    s8[j] = p * (keep ? dp[i] : none[j]);
                } else {
                    p8[j] = p;
                    s8[j] = p * dp[i];
                }
            }
            two_terms<T>(p8, &pf[h], &pl[h]);
            if (kScaled<T> && kCare) {
                s8 *= up;
#pragma unroll
                for (int j = 0; j < 8; ++j) dp[8 * h + j] = s8[j];
            }
            two_terms<T>(s8, &sf[h], &sl[h]);
        }
        if constexpr (kScaled<T> && kCare) {
            if (__any(seen && reaches_two(sf))) {
                rare();
                bits += lower<T>(dp, seen, gk, sf, sl);
                up = power(bits);
            }
        }
#pragma unroll
        for (int d = 0; d < kOut; ++d) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const vec8<T> go = column_operand(g_tile, kRow, 16 * h, 32 * d, lane);
                gv[d] = mma(gv[d], go, pf[h]);
                if (kRest<T>) gv[d] = mma(gv[d], go, pl[h]);
                const vec8<T> q = column_operand(q_tile, kRow, 16 * h, 32 * d, lane);
                gk[d] = mma(gk[d], q, sf[h]);
                if (kRest<T>) gk[d] = mma(gk[d], q, sl[h]);
            }
        }
    }
    if constexpr (kScaled<T> && !kCare) {
        if (max_wave<1>(__any(seen && !finite(gk)))) return false;
    }
    if (!key_ok) return true;
    const bool split = out.k_splits > 1;
    const int64_t at = (split ? int64_t(w.split) * a.k_rows * a.kv_heads : 0) + k_row * a.kv_heads + w.kv_head;
    const float k_factor = a.scale * a.keep_scale * power(-bits - kProb);
    const float v_factor = a.keep_scale * power(kScaled<T> && !kCare ? -bits - kProb : -kProb);
#pragma unroll
    for (int d = 0; d < kOut; ++d) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int col = 32 * d + 8 * i + 4 * half;
            if (col < a.dim) {
                f32x4 k = {gk[d][4 * i], gk[d][4 * i + 1], gk[d][4 * i + 2], gk[d][4 * i + 3]};
                f32x4 v = {gv[d][4 * i], gv[d][4 * i + 1], gv[d][4 * i + 2], gv[d][4 * i + 3]};
                // a key that is not seen has no gradient, whatever its scores were
                k = seen ? k * k_factor : f32x4{};
                v = seen ? v * v_factor : f32x4{};
                if (a.grad_k) put4<T>(split ? out.part_k : nullptr, a.grad_k, at * a.dim + col, k);
                if (a.grad_v) put4<T>(split ? out.part_v : nullptr, a.grad_v, at * a.dim + col, v);
            }
        }
    }
    return true;
}

template <class T, int kDim, bool kSplitKeys>
struct QueryTiles {
    static constexpr int kKeys = 32;
    static constexpr int kRow = kTileRow<T, kDim>;
    static constexpr int kRows = kSplitKeys ? 32 : 128;  // query rows of a workgroup
    static constexpr int kStage = kSplitKeys ? 64 : kThreads;
    static constexpr int kTile = kKeys * kRow;
    static constexpr int kLds = (kSplitKeys ? kWaves : 2) * 2 * kTile * int(sizeof(T));
    static constexpr int kJoinRow = kDim + 4;
    static constexpr int kJoin = kSplitKeys ? kWaves * 32 * kJoinRow * 4 : 0;
    static constexpr int kBytes = kLds > kJoin ? kLds : kJoin;
};

// The waves share tiles of keys, or with kSplitKeys (few query rows) take them in turn, as in
// the forward.  kExact: the structure has kExactStates keys at most, one tile, and delta is its sum of p dp.
template <class T, int kDim, bool kDrop, bool kSplitKeys, bool kExact>
__device__ __forceinline__ void grad_queries(const AttnArgs &a, const Bwd &out, const Place &w, char *lds) {
    using C = QueryTiles<T, kDim, kSplitKeys>;
    constexpr int kKeys = C::kKeys, kRow = C::kRow, kSteps = kDim / 16, kOut = kDim / 32;
    const int lane = threadIdx.x & 63, half = lane >> 5, wave = threadIdx.x >> 6;
    const int thread = kSplitKeys ? lane : threadIdx.x;
    T *k_tile = reinterpret_cast<T *>(lds) + (kSplitKeys ? wave * 2 * C::kTile : 0), *v_tile = k_tile + C::kTile;

    static_assert(kKeys >= kExactStates, "one tile");
    const int splits = out.q_splits, n_tiles = (w.keys + kKeys - 1) / kKeys, per = (n_tiles + splits - 1) / splits;
    const int t_end = min(n_tiles, (w.split + 1) * per), t_step = kSplitKeys ? kWaves : 1;
    const T *k_base = static_cast<const T *>(a.k) + w.k_begin * a.k_row + w.kv_head * a.k_head;
    const T *v_base = static_cast<const T *>(a.v) + w.k_begin * a.v_row + w.kv_head * a.v_head;
    const uint8_t *mask = a.key_mask ? a.key_mask + w.k_begin : nullptr;
    KeyStage<T, kKeys, kDim, C::kStage> in(thread, a.dim);
    const int t_begin = w.split * per + (kSplitKeys ? wave : 0);
    if (t_begin < t_end) in.fetch(a, k_base, v_base, mask, w.keys, t_begin);

    const int r = w.first + (kSplitKeys ? 0 : wave * 32) + (lane & 31);
    const bool row_ok = r < w.rows;
    const int64_t q_row = w.q_begin + (row_ok ? r / a.share : 0);
    const int head = w.kv_head * a.share + (row_ok ? r % a.share : 0);
    const int64_t at = q_row * a.heads + head;
    vec8<T> qf[kSteps], gf[kSteps];
    float delta = 0.f, gg = 0.f, oo = 0.f;  // of grad_out and out: their product and squares
    {
        const T *q = static_cast<const T *>(a.q) + q_row * a.q_row + head * a.q_head;
        const T *g = static_cast<const T *>(a.grad_out) + at * a.dim, *o = static_cast<const T *>(a.out) + at * a.dim;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int d = 16 * s + 8 * half;
            const bool use = row_ok && d < a.dim && t_begin < t_end;  // a wave without keys needs no rows
            qf[s] = use ? *reinterpret_cast<const vec8<T> *>(q + d) : vec8<T>(T(0.f));
            gf[s] = use ? *reinterpret_cast<const vec8<T> *>(g + d) : vec8<T>(T(0.f));
            if (!kExact && use) {
                const vec8<T> of = *reinterpret_cast<const vec8<T> *>(o + d);
                delta += dot<T>(gf[s], of);
                if (kScaled<T>) gg += dot<T>(gf[s], gf[s]), oo += dot<T>(of, of);
            }
        }
    }
    float none = sum_halves(delta) * (-1.f / a.keep_scale);  // what dp - delta is where p was dropped
    const float lse = kept_lse<T>(row_ok ? a.lse[at] : -INFINITY);
    Rng g{};
    if (kDrop) g = load_rng(a.rng);
    const float c = a.scale * kLog2E;
    f32x16 gq[kOut];
    int bits = kScaled<T> && !kExact ? bits_ahead(14, sum_halves(gg) * sum_halves(oo)) : 0;  // the power of gq

    // kMost: for the largest score gradient of each row alone, without the power
    float most = 0.f;
    const auto walk = [&](auto kind) {
        constexpr bool kMost = decltype(kind)::value;
        const float p_lse = lse - (kScaled<T> && !kMost ? float(bits) : 0.f);
        if (!kSplitKeys) {  // every walk starts with the first buffer, as the count of its tiles does
            k_tile = reinterpret_cast<T *>(lds);
            v_tile = k_tile + C::kTile;
        }
        for (int t = t_begin, buffer = 0; t < t_end; t += t_step) {
            if (kSplitKeys) wave_sync();
            const uint64_t valid = in.store(k_tile, v_tile);
            if (kSplitKeys) wave_sync(); else __syncthreads();
            const int k0 = t * kKeys;
            in.fetch(a, k_base, v_base, mask, w.keys, min(t + t_step, t_end - 1));
            f32x16 s = {}, dp;
#pragma unroll
            for (int i = 0; i < 16; ++i) dp[i] = none;  // kExact: zero
            const int row = permuted_row(lane & 31);
#pragma unroll
            for (int i = 0; i < kSteps; ++i) s = mma(s, row_operand(k_tile, kRow, row, 16 * i, half), qf[i]);
#pragma unroll
            for (int i = 0; i < kSteps; ++i) dp = mma(dp, row_operand(v_tile, kRow, row, 16 * i, half), gf[i]);
            if (valid != ~0ull) {
                rare();
                each_score(static_cast<uint32_t>(valid), half, [&](int i, bool used) { s[i] = used ? s[i] : -INFINITY; });
            }
            vec8<T> sf[2], sl[2];
            uint32_t keep[2] = {};
#pragma unroll
            for (int h = 0; h < 2 && kDrop; ++h)
                keep[h] = keep_bits(g, (k0 + 16 * h) / 8 + half, static_cast<uint32_t>(at), a.threshold);
            if (kExact) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (kDrop) dp[i] = keep[i >> 3] & (1u << (i & 7)) ? dp[i] : 0.f;
                    sum = fmaf(probability<T>(s[i], a.scale, c, lse), dp[i], sum);
                }
                none = -sum_halves(sum);
                dp += none;
                if (kScaled<T>) {  // the one tile's own power
                    f32x16 ds;
#pragma unroll
                    for (int i = 0; i < 16; ++i) ds[i] = probability<T>(s[i], a.scale, c, lse) * dp[i];
                    bits = bits_for(largest(ds));
                    dp *= power(bits);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x8 s8;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float p = probability<T>(s[8 * h + j], a.scale, c, kExact ? lse : p_lse);
                    s8[j] = p * (kExact || !kDrop || (keep[h] & (1u << j)) ? dp[8 * h + j] : none);
                    if (kMost) most = fmaxf(most, fabsf(s8[j]));
                }
                if (!kMost) two_terms<T>(s8, &sf[h], &sl[h]);
            }
            if constexpr (!kMost) {
#pragma unroll
                for (int d = 0; d < kOut; ++d) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const vec8<T> k = column_operand(k_tile, kRow, 16 * h, 32 * d, lane);
                        gq[d] = mma(gq[d], k, sf[h]);
                        if (kRest<T>) gq[d] = mma(gq[d], k, sl[h]);
                    }
                }
            }
            if (!kSplitKeys) {
                k_tile = reinterpret_cast<T *>(lds) + (buffer ^= 1) * 2 * C::kTile;
                v_tile = k_tile + C::kTile;
            }
        }
    };
    for (bool again = false;; again = true) {
#pragma unroll
        for (int d = 0; d < kOut; ++d) gq[d] = f32x16{};
        walk(std::false_type());
        if constexpr (!kScaled<T> || kExact) break;
        const bool lost = max_halves(finite(gq) ? 0.f : 1.f) > 0.f;  // the row, whose columns are in both halves
        const int any = __any(lost);
        if (again || !(kSplitKeys ? any : max_wave<2>(any))) break;
        in.fetch(a, k_base, v_base, mask, w.keys, t_begin);
        walk(std::true_type());
        most = max_halves(most);
        if (lost) bits = bits_for(most);
        if (!kSplitKeys) __syncthreads();  // before the first buffer is written again
        in.fetch(a, k_base, v_base, mask, w.keys, t_begin);
    }
    if (kScaled<T>) {
#pragma unroll
        for (int d = 0; d < kOut; ++d) gq[d] *= power(-bits);
    }
    const bool split = splits > 1;
    const int64_t part = split ? int64_t(w.split) * a.q_rows * a.heads : 0;
    const float factor = a.scale * a.keep_scale;
    if (!kSplitKeys) {
        if (!row_ok) return;
#pragma unroll
        for (int d = 0; d < kOut; ++d) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = 32 * d + 8 * i + 4 * half;
                const f32x4 v = {gq[d][4 * i], gq[d][4 * i + 1], gq[d][4 * i + 2], gq[d][4 * i + 3]};
                if (col < a.dim) put4<T>(split ? out.part_q : nullptr, a.grad_q, (part + at) * a.dim + col, v * factor);
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
    const int jr = threadIdx.x >> 3, jrow = w.first + jr;  // eight threads a row
    if (jrow >= w.rows) return;
    const int64_t to = (w.q_begin + jrow / a.share) * a.heads + w.kv_head * a.share + jrow % a.share;
    for (int col = (threadIdx.x & 7) * 8; col < a.dim; col += 64) {
        f32x8 v = {};
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            const float *from = join + (i * 32 + jr) * C::kJoinRow + col;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += from[j];
        }
        v *= factor;
        if (split)
            store8(out.part_q + (part + to) * a.dim + col, v);
        else
            store8(static_cast<T *>(a.grad_q) + to * a.dim + col, from_f32<T>(v));
    }
}

// Three workgroups a compute unit for fp16 at D = 32 (with dropout, 64 structures of up to 32 rows and 200
// states: 21.5 us for 25.0 with two, before probabilities had two terms), else two, where that does not
// leave too few registers: against one, D = 96 with dropout takes 209 us for 287 and D = 128 240 for 291 (bf16,
// 4 structures of 1024 query rows and 2048 states, 8 heads over 4); fp32 at D = 128 would take 1359 for 1029.
template <class T, int kDim, bool kDrop, bool kSplitKeys>
__global__ void __launch_bounds__(kThreads, (kScaled<T> && kDim <= 32) ? 3 : (sizeof(T) == 2 || kDim <= 64) ? 2 : 1)
    k_backward(AttnArgs a, Bwd out) {
    constexpr int kKeyBytes = int(sizeof(KeyLds<T, kDim>)), kQueryBytes = QueryTiles<T, kDim, kSplitKeys>::kBytes;
    __shared__ __attribute__((aligned(16))) char lds[kKeyBytes > kQueryBytes ? kKeyBytes : kQueryBytes];
    uint32_t block = blockIdx.x;
    if (block < out.key_blocks) {
        KeyLds<T, kDim> &tiles = *reinterpret_cast<KeyLds<T, kDim> *>(lds);
        int tid = threadIdx.x;
        const auto place = [&]() { return place_of<kKeyTile>(a, block, false, out.k_splits, out.k_slots); };
        const Place w = place();
        if (!w.any) return;
        if (kExactDelta<T> && w.keys <= kExactStates) {
            grad_keys<T, kDim, kDrop, kExactDelta<T>, kScaled<T>>(a, out, w, tid, tiles);
        } else if ((kScaled<T> && w.rows <= kRowTile) || !grad_keys<T, kDim, kDrop, false, false>(a, out, w, tid, tiles)) {
            // (a walk of one tile is done with care at once: fp16, 64 structures of up to 32 rows and 200
            // states, D = 32 with dropout 21.2 -> 19.9 us)
            if constexpr (kScaled<T>) {
                // finds its place and its thread anew: kept for this, they would take registers of the other walk
                asm volatile("" : "+s"(block), "+v"(tid));
                grad_keys<T, kDim, kDrop, false, true>(a, out, place(), tid, tiles);
            }
        }
    } else {
        const uint32_t item = block - static_cast<uint32_t>(out.key_blocks);
        const Place w = place_of<QueryTiles<T, kDim, kSplitKeys>::kRows>(a, item, true, out.q_splits, out.q_slots);
        if (!w.any) return;
        if constexpr (kExactDelta<T>) {
            if (w.keys <= kExactStates) return grad_queries<T, kDim, kDrop, kSplitKeys, true>(a, out, w, lds);
        }
        grad_queries<T, kDim, kDrop, kSplitKeys, false>(a, out, w, lds);
    }
}

// out = sum of `splits` fp32 arrays of `rows` rows of `row` values (a multiple of eight), in order, for
// the rows that the structures of `ptr` hold (the others have no partial sums and are not written); up
// to three.
struct Sum {
    const float *part;
    void *out;
    const int32_t *ptr;
    int64_t rows, row;  // row = 0: nothing to do
    int splits;
};
struct Sums {
    Sum job[3];
    int32_t n_struct;
};
template <class T>
__global__ void __launch_bounds__(kThreads) k_add(Sums sums) {
    const int64_t step = int64_t(gridDim.x) * kThreads * 8;
    for (const Sum &j : sums.job) {
        const Span held = span_of(j.ptr[0], j.ptr[sums.n_struct], j.rows);
        const int64_t n = j.rows * j.row, end = held.end * j.row;
        for (int64_t i = held.begin * j.row + (int64_t(blockIdx.x) * kThreads + threadIdx.x) * 8; i < end; i += step) {
            f32x8 v = load8(j.part + i);
#pragma unroll 8
            for (int s = 1; s < j.splits; ++s) v += load8(j.part + s * n + i);
            store8(static_cast<T *>(j.out) + i, from_f32<T>(v));
        }
    }
}

constexpr size_t up(size_t v) { return (v + 255) / 256 * 256; }

struct Choice {
    bool split_keys;
    int q_splits, k_splits;
    int64_t q_slots, k_slots;
    size_t part_q, part_k, bytes;  // bytes of the partial sums; k for each of k and v
};

// Splits of a walk of `walk` rows, so that none is longer than `share`, what a workgroup has if the
// work is spread evenly; 256 rows a split at least.
int splits_of(int64_t walk, int64_t share) {
    if (share < 256) share = 256;
    const int64_t s = (walk + share / 2) / share;
    return static_cast<int>(s < 1 ? 1 : s > 64 ? 64 : s);
}

Choice choose(const AttnArgs &a) {
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
    c.bytes = c.part_q + 2 * c.part_k;
    return c;
}

template <class T, int kDim, bool kDrop>
void launch(const AttnArgs &a, const Choice &c, const Bwd &out, int64_t blocks, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(blocks)), threads(kThreads);
    if (c.split_keys)
        k_backward<T, kDim, kDrop, true><<<grid, threads, 0, stream>>>(a, out);
    else
        k_backward<T, kDim, kDrop, false><<<grid, threads, 0, stream>>>(a, out);
}

template <class T, int kDim>
void launch(const AttnArgs &a, const Choice &c, const Bwd &out, int64_t blocks, hipStream_t stream) {
    if (a.threshold)
        launch<T, kDim, true>(a, c, out, blocks, stream);
    else
        launch<T, kDim, false>(a, c, out, blocks, stream);
}

template <class T>
hipError_t backward(const AttnArgs &a, hipStream_t stream) {
    const Choice c = choose(a);
    char *ws = static_cast<char *>(a.workspace);
    Bwd out{};
    out.part_q = reinterpret_cast<float *>(ws);
    out.part_k = reinterpret_cast<float *>(ws + c.part_q);
    out.part_v = reinterpret_cast<float *>(ws + c.part_q + c.part_k);
    out.q_splits = c.q_splits, out.k_splits = c.k_splits, out.q_slots = c.q_slots, out.k_slots = c.k_slots;
    out.key_blocks = a.grad_k || a.grad_v ? c.k_slots * a.kv_heads * c.k_splits : 0;
    const int64_t blocks = out.key_blocks + (a.grad_q ? c.q_slots * a.kv_heads * c.q_splits : 0);
    if (a.dim <= 32)
        launch<T, 32>(a, c, out, blocks, stream);
    else if (a.dim <= 64)
        launch<T, 64>(a, c, out, blocks, stream);
    else if (a.dim <= 96)
        launch<T, 96>(a, c, out, blocks, stream);
    else
        launch<T, 128>(a, c, out, blocks, stream);
    const int64_t q_row = a.grad_q && c.q_splits > 1 ? int64_t(a.heads) * a.dim : 0;
    const int64_t k_row = c.k_splits > 1 ? int64_t(a.kv_heads) * a.dim : 0;
    const Sums sums = {{{out.part_q, a.grad_q, a.q_ptr, a.q_rows, q_row, c.q_splits},
                        {out.part_k, a.grad_k, a.k_ptr, a.k_rows, a.grad_k ? k_row : 0, c.k_splits},
                        {out.part_v, a.grad_v, a.k_ptr, a.k_rows, a.grad_v ? k_row : 0, c.k_splits}},
                       a.n_struct};
    const int64_t nq = a.q_rows * q_row, nk = a.grad_k || a.grad_v ? a.k_rows * k_row : 0;
    const int64_t most = nq > nk ? nq : nk, grid = (most / 8 + kThreads - 1) / kThreads;
    if (most)
        k_add<T><<<dim3(static_cast<unsigned>(grid > 4096 ? 4096 : grid)), dim3(kThreads), 0, stream>>>(sums);
    return hipGetLastError();
}

}  // namespace

size_t cross_attn_bwd_workspace(oeq_dtype, const AttnArgs &a) { return choose(a).bytes; }

int64_t cross_attn_bwd_blocks(oeq_dtype, const AttnArgs &a) {
    const Choice c = choose(a);
    return c.q_slots * a.kv_heads * c.q_splits + c.k_slots * a.kv_heads * c.k_splits;
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
