// Device pieces shared by the cross-attention kernels: matrix products of 32 x 32 tiles,
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

template <int kTile>
__device__ __forceinline__ Place place_of(const AttnArgs &a, uint32_t item, bool by_query, int splits, int64_t n_slots) {
    Place p;
    const uint32_t slots = static_cast<uint32_t>(n_slots), rest = item / static_cast<uint32_t>(splits);
    p.split = static_cast<int>(item - rest * splits);
    p.kv_head = static_cast<int>(rest / slots);
    const int64_t slot = rest - p.kv_head * slots;
    const Owner at_slot = by_query ? find_structure(a.q_ptr, a.k_ptr, a.n_struct, a.share, kTile, slot)
                                   : find_structure(a.k_ptr, a.q_ptr, a.n_struct, 1, kTile, slot);
    const int32_t *qp = by_query ? at_slot.ptr : at_slot.other, *kp = by_query ? at_slot.other : at_slot.ptr;
    const Span q = span_of(qp[0], qp[1], a.q_rows), k = span_of(kp[0], kp[1], a.k_rows);
    p.q_begin = q.begin;
    p.k_begin = k.begin;
    p.rows = static_cast<int>((q.end - q.begin) * a.share);
    p.keys = static_cast<int>(k.end - k.begin);
    const int64_t at = (slot - at_slot.first) * kTile;
    p.first = static_cast<int>(at);
    p.any = at >= 0 && at < (by_query ? p.rows : p.keys);
    return p;
}

}  // namespace readout
}  // namespace oeq
