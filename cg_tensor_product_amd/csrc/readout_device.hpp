// Device helpers shared by the readout kernels (group_norm.hip, dropout.hip,
// cross_attn_*.hip): element types, the dropout generator and the structure lookup.
#pragma once

#include <cstdint>

#include <hip/hip_runtime.h>

namespace oeq {
namespace readout {

using f16 = _Float16;
using bf16 = __bf16;

// Eight consecutive elements: one 16-byte access of a 16-bit type, two of fp32.
template <class T>
using vec8 = T __attribute__((ext_vector_type(8)));

using f32x4 = float __attribute__((ext_vector_type(4)));
using f32x8 = vec8<float>;

// Loads and stores of eight elements at any element alignment (global memory takes
// unaligned 16-byte accesses).
template <class T>
__device__ __forceinline__ vec8<T> load8(const T *p) {
    vec8<T> v;
    __builtin_memcpy(&v, p, sizeof v);
    return v;
}
template <class T>
__device__ __forceinline__ void store8(T *p, vec8<T> v) {
    __builtin_memcpy(p, &v, sizeof v);
}
template <class T>
__device__ __forceinline__ f32x8 to_f32(vec8<T> v) {
    return __builtin_convertvector(v, f32x8);
}
template <class T>
__device__ __forceinline__ vec8<T> from_f32(f32x8 v) {
    return __builtin_convertvector(v, vec8<T>);
}
// The first n < 8 elements of a row's end; the others are zero.
template <class T>
__device__ __forceinline__ vec8<T> load_part(const T *p, int n) {
    vec8<T> v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : T(0.f);
    return v;
}
template <class T>
__device__ __forceinline__ void store_part(T *p, vec8<T> v, int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = v[i];
}

// ---- dropout generator --------------------------------------------------------
// Philox4x32 with 10 rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC 2011).  Element (row, column) of a call takes the 16-bit part
// column % 8 of the block with counter (column / 8, row, offset low, offset high) and the
// seed as key, and is dropped when the part is below a threshold of 2^16 p.  Sixteen bits
// rather than 32 halve the generator's multiplies, which bound the 16-bit dropout kernels
// (ten rounds of two 32 x 32 -> 64 multiplies a block); p is held to 2^-17.
struct Rng {
    uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ Rng load_rng(const int64_t *state) {
    const uint64_t seed = static_cast<uint64_t>(state[0]), offset = static_cast<uint64_t>(state[1]);
    return {static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32), static_cast<uint32_t>(offset),
            static_cast<uint32_t>(offset >> 32)};
}

__device__ __forceinline__ uint4 philox(const Rng &g, uint32_t block, uint32_t row) {
    uint32_t c0 = block, c1 = row, c2 = g.o0, c3 = g.o1, k0 = g.k0, k1 = g.k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = uint64_t(0xD2511F53u) * c0, b = uint64_t(0xCD9E8D57u) * c2;
        // 0x96: the exclusive or of three words in one instruction
        c0 = __builtin_amdgcn_bitop3_b32(uint32_t(b >> 32), c1, k0, 0x96);
        c1 = uint32_t(b);
        c2 = __builtin_amdgcn_bitop3_b32(uint32_t(a >> 32), c3, k1, 0x96);
        c3 = uint32_t(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// Bit i of the result: column 8 * block + i of the row is kept.
__device__ __forceinline__ uint32_t keep_bits(const Rng &g, uint32_t block, uint32_t row, uint32_t threshold) {
    const uint4 w = philox(g, block, row);
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bits |= uint32_t((v[i] & 0xFFFFu) >= threshold) << (2 * i);
        bits |= uint32_t((v[i] >> 16) >= threshold) << (2 * i + 1);
    }
    return bits;
}

// ---- structures -----------------------------------------------------------------
// The rows of structure b, from a row pointer.  A pointer that leaves [0, n_rows] or
// decreases is cut to it, so that no access leaves the tensors.
struct Span {
    int64_t begin, end;
};
__device__ __forceinline__ Span span_of(int64_t lo, int64_t hi, int64_t n_rows) {
    lo = lo < 0 ? 0 : lo > n_rows ? n_rows : lo;
    hi = hi < lo ? lo : hi > n_rows ? n_rows : hi;
    return {lo, hi};
}
__device__ __forceinline__ Span span_of(const int32_t *ptr, int b, int64_t n_rows) {
    return span_of(int64_t(ptr[b]), int64_t(ptr[b + 1]), n_rows);
}

// Tiles of `tile` rows over ragged structures without a table of their lengths: structure
// b owns the slots from ptr[b] * per / tile + b on (rounded down), `per` tile rows for a row
// of the pointer.  A structure of n rows has floor(n * per / tile) + 1 slots or one more,
// enough for its tiles; a slot past its last tile has no work.
__host__ __device__ __forceinline__ int64_t tile_slots(int64_t n_rows, int n_struct, int64_t per, int64_t tile) {
    return n_rows * per / tile + n_struct;
}

// The structure that owns `slot` of the tiling by `ptr`, with its rows on both sides (`other` is
// the second row pointer).  All 64 lanes of the wave take part (a search with 64 probes a step)
// and get the same answer; the last step's probes bring what the answer is made of, so up to 64
// structures take one round of loads.
struct Owner {
    int32_t ptr[2], other[2];  // the structure's begin and end
    int index;                 // which it is
    int64_t first;             // its first slot
};
__device__ __forceinline__ Owner find_structure(const int32_t *ptr, const int32_t *other, int n_struct, int per, int tile,
                                                int64_t slot) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = n_struct;
    while (n > 64) {
        const int step = (n + 63) / 64;
        const int i = lane * step;
        const bool at_or_below = i < n && int64_t(ptr[lo + i]) * per / tile + (lo + i) <= slot;
        const int count = __popcll(__ballot(at_or_below));
        const int skip = count > 1 ? (count - 1) * step : 0;
        lo += skip;
        n = n - skip < step ? n - skip : step;
    }
    const int i = lo + (lane < n ? lane : n - 1);
    const int32_t p0 = ptr[i], p1 = ptr[i + 1], o0 = other[i], o1 = other[i + 1];
    const int64_t mine = int64_t(p0) * per / tile + i;
    const int count = __popcll(__ballot(lane < n && mine <= slot)), at = count > 1 ? count - 1 : 0;
    Owner w;
    w.ptr[0] = __builtin_amdgcn_readlane(p0, at);
    w.ptr[1] = __builtin_amdgcn_readlane(p1, at);
    w.other[0] = __builtin_amdgcn_readlane(o0, at);
    w.other[1] = __builtin_amdgcn_readlane(o1, at);
    w.index = lo + at;
    w.first = int64_t(w.ptr[0]) * per / tile + (lo + at);
    return w;
}

}  // namespace readout
}  // namespace oeq
