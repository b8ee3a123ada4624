// Device pieces shared by the attention kernels (cross and causal): matrix products of 32 x 32 tiles,
// tiles of rows in LDS and how a wave takes operands from them.
//
// One 32 x 32 x 16 step multiplies A [32, 16] by B [16, 32].  Lane l holds, with
// half = l / 32, the elements k = 8 half .. 8 half + 7 of row l % 32 of A, and the same of
// column l % 32 of B.  fp16 and bf16 have it as one instruction; fp32 takes eight
// 32 x 32 x 2 instructions, the j-th over the j-th elements of both halves, so that all
// types share one layout.  Of the result the lane holds column l % 32 and the rows
// 8 (i / 4) + 4 half + i % 4 (i = 0..15).
//
// Score tiles are computed with the rows of A permuted, row m holding key (or query)
// 16 (m / 16) + 8 (m / 4 % 2) + 4 (m / 8 % 2) + m % 4 of the tile.  Then lane l's sixteen
// results are the keys 16 s + 8 half + j (i = 8 s + j): exactly its operand of the next
// product's steps s = 0, 1, so probabilities go from one product into the next in
// registers, and eight consecutive keys share one block of the dropout generator.
#pragma once

#include <type_traits>

#include "readout.hpp"
#include "readout_device.hpp"

namespace oeq {
namespace readout {

using f32x16 = float __attribute__((ext_vector_type(16)));
using i16x4 = short __attribute__((ext_vector_type(4)));
using i16x8 = vec8<short>;

constexpr float kLog2E = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

__device__ __forceinline__ f32x16 mma(f32x16 acc, vec8<bf16> a, vec8<bf16> b) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(f32x16 acc, vec8<f16> a, vec8<f16> b) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, acc, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(f32x16 acc, f32x8 a, f32x8 b) {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], acc, 0, 0, 0);
    return acc;
}

// Elements from one tile row to the next: 16 bytes past the row, an odd number of 16-byte
// pieces, so that 16 consecutive rows start in different banks.
template <class T, int kDim>
constexpr int kTileRow = kDim + 16 / int(sizeof(T));

__device__ __forceinline__ int permuted_row(int m) { return (m & 16) | (m & 4) << 1 | (m & 8) >> 1 | (m & 3); }

// A operand: row `row` of the tile, step d0 / 16.
template <class T>
__device__ __forceinline__ vec8<T> row_operand(const T *tile, int tile_row, int row, int d0, int half) {
    return *reinterpret_cast<const vec8<T> *>(tile + row * tile_row + d0 + 8 * half);
}
template <>
__device__ __forceinline__ f32x8 row_operand<float>(const float *tile, int tile_row, int row, int d0, int half) {
    const f32x4 *p = reinterpret_cast<const f32x4 *>(tile + row * tile_row + d0 + 8 * half);
    const f32x4 a = p[0], b = p[1];
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// A operand from the transposed tile: column d0 + lane % 32, rows row0 + 8 half + j.  The
// 16-bit form is two transposing LDS reads: of each 16 lanes the address of lane i is that of
// four elements, row i / 4, and the lane receives column i of the four rows.
template <class T>
__device__ __forceinline__ vec8<T> column_operand(const T *tile, int tile_row, int row0, int d0, int lane) {
    const int half = lane >> 5, group = lane >> 4 & 1, i = lane & 15;
    const T *p = tile + (row0 + 8 * half + (i >> 2)) * tile_row + d0 + 16 * group + (i & 3) * 4;
    using Lds = __attribute__((address_space(3))) i16x4 *;
    const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p));
    const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p + 4 * tile_row));
    const i16x8 v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(vec8<T>, v);
}
template <>
__device__ __forceinline__ f32x8 column_operand<float>(const float *tile, int tile_row, int row0, int d0, int lane) {
    const float *p = tile + (row0 + 8 * (lane >> 5)) * tile_row + d0 + (lane & 31);
    f32x8 v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = p[j * tile_row];
    return v;
}

// Keeps a branch that is seldom taken a branch: its work is not done ahead and selected.
__device__ __forceinline__ void rare() { asm volatile(""); }

// Rows of a strided operand on their way to LDS: kRows x kDim elements by kThreads threads,
// in pieces of eight, kLanes threads a row.  `fetch` reads the rows, `store` writes them with
// zeros for rows whose bit in `valid` is not set and for columns past the head's dimension.
template <class T, int kRows, int kDim, int kThreads>
struct RowStage {
    static constexpr int kLanes = kDim <= 32 ? 4 : kDim <= 64 ? 8 : 16;
    static constexpr int kStep = kThreads / kLanes;  // rows from one of a thread's pieces to the next
    static constexpr int kPieces = (kRows + kStep - 1) / kStep;
    static_assert(kRows % kStep == 0 || kPieces == 1, "every piece but a lone one is whole");
    vec8<T> v[kPieces];
    int row, d;
    bool reads;  // whether this thread's columns are in the head

    __device__ __forceinline__ RowStage(int thread, int dim)
        : row(thread / kLanes), d(thread % kLanes * 8), reads(d < dim && row < kRows) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) v[i] = vec8<T>(T(0.f));  // columns past the head stay zero
    }

    // The tile's rows, at base + row * stride.  Where they end within the tile, row `last` is read
    // in place of those past it (and dropped by store).  One set of loads serves both: a value
    // that came by two ways would be waited for here, to be copied, and not where it is used.
    __device__ __forceinline__ void fetch(const T *base, int64_t stride, int last) {
        if (!reads) return;
        const T *at = base + row * stride + d;
        int64_t off[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) off[i] = i * (kStep * stride);
        if (last < kRows - 1) {
            rare();
#pragma unroll
            for (int i = 0; i < kPieces; ++i) off[i] = int64_t(min(row + i * kStep, last) - row) * stride;
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) v[i] = *reinterpret_cast<const vec8<T> *>(at + off[i]);
    }
    __device__ __forceinline__ void store(T *tile, bool whole, uint64_t valid) {
        if (d >= kDim || row >= kRows) return;
        if (!whole) {
            rare();
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                if (!(valid >> (row + i * kStep) & 1)) v[i] = vec8<T>(T(0.f));
            }
        }
        T *at = tile + row * kTileRow<T, kDim> + d;
#pragma unroll
        for (int i = 0; i < kPieces; ++i, at += kStep * kTileRow<T, kDim>) {
            if constexpr (sizeof(T) == 4) {
                reinterpret_cast<f32x4 *>(at)[0] = __builtin_shufflevector(v[i], v[i], 0, 1, 2, 3);
                reinterpret_cast<f32x4 *>(at)[1] = __builtin_shufflevector(v[i], v[i], 4, 5, 6, 7);
            } else {
                *reinterpret_cast<vec8<T> *>(at) = v[i];
            }
        }
    }
};

// K and V tiles of one structure and key head on their way to LDS, with the mask of the keys
// that are there and visible.
template <class T, int kKeys, int kDim, int kThreads>
struct KeyStage {
    RowStage<T, kKeys, kDim, kThreads> k, v;
    int there = 0;         // keys of the tile that are there
    uint32_t visible = 1;  // what the mask holds for this lane's key
    __device__ __forceinline__ KeyStage(int thread, int dim) : k(thread, dim), v(thread, dim) {}
    __device__ __forceinline__ void fetch(const AttnArgs &a, const T *k_base, const T *v_base, const uint8_t *mask, int keys,
                                          int t) {
        const int k0 = t * kKeys;
        there = keys - k0;
        if (mask) visible = mask[k0 + min(int(threadIdx.x & (kKeys - 1)), there - 1)];
        k.fetch(k_base + int64_t(k0) * a.k_row, a.k_row, there - 1);
        v.fetch(v_base + int64_t(k0) * a.v_row, a.v_row, there - 1);
    }
    // Writes both tiles and returns which keys are to be used (bit = key of the tile).
    __device__ __forceinline__ uint64_t store(T *k_tile, T *v_tile) {
        const uint64_t valid = __ballot(int(threadIdx.x & (kKeys - 1)) < there && visible);
        k.store(k_tile, valid == ~0ull, valid);
        v.store(v_tile, valid == ~0ull, valid);
        return valid;
    }
};

// f(i, used) for a lane's sixteen scores of the 32 keys whose bits are `valid`.
template <class F>
__device__ __forceinline__ void each_score(uint32_t valid, int half, F &&f) {
    const uint32_t mine = valid >> (8 * half);
#pragma unroll
    for (int i = 0; i < 16; ++i) f(i, (mine & (1u << (16 * (i >> 3) + (i & 7)))) != 0);
}

// Orders a wave's own LDS writes before its reads (LDS serves a wave in order; this keeps the
// compiler from moving them).
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Maximum and sum over the two halves' lanes of a column.
__device__ __forceinline__ float max_halves(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Which structure, key head and rows a workgroup has.  Query rows of one key head are
// numbered r = query * share + head within the share, so heads that share keys share the tile.
struct Place {
    int kv_head, split;
    int64_t q_begin, k_begin;  // first rows of the structure
    int rows, keys;            // query rows times share; keys
    int first;                 // first row (or key) of the tile
    bool any;
};

// kCausal: the longest walks come first, those of the last query rows and of the first keys, for an
// even end (2 x 4096 rows, 16 heads over 4, D = 128, fp16: forward 175 us, 230 with the shortest first, backward 903 and
// 945), and the key heads of a tile follow each other, so that with eight heads, or four, an XCD's
// workgroups read one head's keys.
// `even`: every walk has all its splits, which then follow each other, so that an XCD's workgroups read the same
// part of the keys.  Else the first splits of all walks come first: some walks have fewer, and what does
// not exist is spread over the XCDs.
template <int kTile, bool kCausal = false>
__device__ __forceinline__ Place place_of(const AttnArgs &a, uint32_t item, bool by_query, int splits, int64_t n_slots,
                                          bool even = true) {
    Place p;
    const uint32_t slots = static_cast<uint32_t>(n_slots);
    int64_t slot;
    if (kCausal) {
        const uint32_t kv_heads = static_cast<uint32_t>(a.kv_heads), walks = slots * kv_heads;
        uint32_t rest = item / (even ? static_cast<uint32_t>(splits) : walks);
        p.split = static_cast<int>(even ? item - rest * splits : rest);
        rest = even ? rest : item - rest * walks;
        const uint32_t tile = rest / kv_heads;
        p.kv_head = static_cast<int>(rest - tile * kv_heads);
        slot = by_query ? slots - 1 - tile : tile;
    } else {
        const uint32_t rest = item / static_cast<uint32_t>(splits);
        p.split = static_cast<int>(item - rest * splits);
        p.kv_head = static_cast<int>(rest / slots);
        slot = rest - p.kv_head * slots;
    }
    const Owner at_slot = by_query ? find_structure(a.q_ptr, a.k_ptr, a.n_struct, a.share, kTile, slot)
                                   : find_structure(a.k_ptr, a.q_ptr, a.n_struct, 1, kTile, slot);
    const int32_t *qp = by_query ? at_slot.ptr : at_slot.other, *kp = by_query ? at_slot.other : at_slot.ptr;
    const Span q = span_of(qp[0], qp[1], a.q_rows);
    Span k = span_of(kp[0], kp[1], a.k_rows);
    if (kCausal && a.k_len) {
        const int64_t n = a.k_len[at_slot.index];
        k.end = min(k.end, k.begin + max(n, int64_t(0)));
    }
    p.q_begin = q.begin;
    p.k_begin = k.begin;
    p.rows = static_cast<int>((q.end - q.begin) * a.share);
    p.keys = static_cast<int>(k.end - k.begin);
    const int64_t at = (slot - at_slot.first) * kTile;
    p.first = static_cast<int>(at);
    p.any = at >= 0 && at < (by_query ? p.rows : p.keys);
    return p;
}

// Causal visibility: query i of n sees the keys j <= i + `off`, off = keys - n.  Row r of a workgroup's key head
// is query r / share.
__device__ __forceinline__ int causal_offset(const AttnArgs &a, const Place &w) { return w.keys - w.rows / a.share; }

// The lowest n bits (n < 0: none).
__device__ __forceinline__ uint64_t low_bits(int n) { return n >= 64 ? ~0ull : n <= 0 ? 0 : (1ull << n) - 1; }

// A walk with care, where the causal limit cuts a tile: the products take the tile's infinities and NaNs as zeros
// (`finite_only`), and `add_others` adds them, row by row of the tile, to the sums of the lanes whose bit of `used`
// is set; kNan: as NaN, for a factor of either sign.
template <class T>
__device__ __forceinline__ vec8<T> finite_only(vec8<T> v) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fabsf(v[i]) < INFINITY ? v[i] : 0.f;
        return v;
    } else {
        constexpr short kExponent = std::is_same<T, f16>::value ? 0x7C00 : 0x7F80;
        i16x8 w = __builtin_bit_cast(i16x8, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = (w[i] & kExponent) == kExponent ? short(0) : w[i];
        return __builtin_bit_cast(vec8<T>, w);
    }
}
template <bool kNan, class T, int kOut>
__device__ __forceinline__ void add_others(f32x16 (&sum)[kOut], const T *tile, int tile_row, uint32_t used, int half) {
#pragma unroll 1
    for (int j = 0; j < 32; ++j) {
        const bool sees = used >> j & 1;
        const T *row = tile + j * tile_row + 4 * half;
#pragma unroll
        for (int d = 0; d < kOut; ++d) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = static_cast<float>(row[32 * d + 8 * (i >> 2) + (i & 3)]);
                if (sees && !(fabsf(x) < INFINITY)) sum[d][i] += kNan ? x - x : x;
            }
        }
    }
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

// A kernel's arguments for a function that is not inlined, by LDS: `put` copies them there, `get` takes them out
// again, the same for all lanes.  So walks that are seldom taken (with care) have registers of their own, and
// the kernel's other walks are compiled as if they were not there.
template <class A>
struct Passed {
    static constexpr int kWords = (sizeof(A) + 3) / 4;
    uint32_t word[kWords];
    // by one thread, with a barrier before and after
    __device__ __forceinline__ void put(const A &a) { __builtin_memcpy(word, &a, sizeof a); }
    __device__ __forceinline__ A get() const {
        uint32_t w[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = __builtin_amdgcn_readfirstlane(word[i]);
        A a;
        __builtin_memcpy(&a, w, sizeof a);
        return a;
    }
};

}  // namespace readout
}  // namespace oeq
