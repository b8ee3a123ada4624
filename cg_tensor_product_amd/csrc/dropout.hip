// Dropout from a counter-based generator: out = residual + x * keep * scale, and with
// x = grad_out and no residual its gradient.  The mask is a function of (seed, offset, row,
// column) and is formed again wherever it is needed, so nothing but the operands moves.
//
// One thread takes the eight columns of one generator block: 16-byte loads of 16-bit types,
// two of them of fp32, so a block's ten rounds serve all its columns.  Bound by memory: 280000 x
// 256, bf16, 49 us (5.8 TB/s, the copy rate, with the vector unit two thirds busy); 5000 x 1152,
// fp32, with a residual 11.9 us.
#include <type_traits>

#include "readout.hpp"
#include "readout_device.hpp"

namespace oeq {
namespace readout {

namespace {

constexpr int kThreads = 256;

template <class T, bool kResidual>
__device__ __forceinline__ void drop8(const DropoutArgs &a, const Rng &g, int64_t row, uint32_t block) {
    const int64_t col = int64_t(block) * 8;
    const T *x = static_cast<const T *>(a.x) + row * a.ld_x + col;
    const T *res = kResidual ? static_cast<const T *>(a.residual) + row * a.ld_residual + col : nullptr;
    T *out = static_cast<T *>(a.out) + row * a.ld_out + col;
    const int n = a.cols - col < 8 ? static_cast<int>(a.cols - col) : 8;
    vec8<T> xv, rv;
    if (n == 8) {
        xv = load8(x);
        if (kResidual) rv = load8(res);
    } else {
        xv = load_part(x, n);
        if (kResidual) rv = load_part(res, n);
    }
    const uint32_t keep = keep_bits(g, block, static_cast<uint32_t>(row), a.threshold);
    f32x8 v = to_f32<T>(xv), r = {};
    if (kResidual) r = to_f32<T>(rv);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        // a dropped element is replaced, not multiplied by zero: it may be inf or NaN
        const float kept = (keep >> j & 1) ? v[j] * a.scale : 0.f;
        v[j] = kResidual ? r[j] + kept : kept;
    }
    const vec8<T> o = from_f32<T>(v);
    if (n == 8)
        store8(out, o);
    else
        store_part(out, o, n);
}

// kWide: more than 2^32 generator blocks in the call, numbered in 64 bits.
template <class T, bool kResidual, bool kWide>
__global__ void __launch_bounds__(kThreads) k_dropout(DropoutArgs a, uint32_t per_row) {
    using Index = typename std::conditional<kWide, uint64_t, uint32_t>::type;
    const Rng g = load_rng(a.rng);
    const Index total = static_cast<Index>(a.rows) * per_row, step = Index(gridDim.x) * kThreads;
    for (Index i = Index(blockIdx.x) * kThreads + threadIdx.x; i < total; i += step) {
        const Index row = i / per_row;
        drop8<T, kResidual>(a, g, static_cast<int64_t>(row), static_cast<uint32_t>(i - row * per_row));
        if (total - i <= step) break;  // before i + step can wrap
    }
}

template <class T, bool kResidual>
hipError_t launch(const DropoutArgs &a, hipStream_t stream) {
    const int64_t per_row = (a.cols + 7) / 8, total = a.rows * per_row;
    int64_t grid = (total + kThreads - 1) / kThreads;
    if (grid > (1 << 23)) grid = 1 << 23;  // a launch holds fewer than 2^32 threads
    const dim3 blocks(static_cast<unsigned>(grid)), threads(kThreads);
    if (total >> 32)
        k_dropout<T, kResidual, true><<<blocks, threads, 0, stream>>>(a, static_cast<uint32_t>(per_row));
    else
        k_dropout<T, kResidual, false><<<blocks, threads, 0, stream>>>(a, static_cast<uint32_t>(per_row));
    return hipGetLastError();
}

template <class T>
hipError_t launch(const DropoutArgs &a, hipStream_t stream) {
    return a.residual ? launch<T, true>(a, stream) : launch<T, false>(a, stream);
}

}  // namespace

hipError_t dropout(oeq_dtype dtype, const DropoutArgs &a, hipStream_t stream) {
    switch (dtype) {
        case OEQ_F32: return launch<float>(a, stream);
        case OEQ_F16: return launch<f16>(a, stream);
        case OEQ_BF16: return launch<bf16>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace readout
}  // namespace oeq
