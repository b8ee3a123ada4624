// Root-mean-square norm with the residual's addition, and its gradient.
//   h = x + residual (rounded to the type: the residual stream)   rstd = 1 / sqrt(mean h^2 + eps)
//   y = h rstd weight      out = y, or e4m3(y / scale) with scale = max |y| / 448 for each row
//   dy = grad_out weight   grad_x = rstd (dy - h rstd mean(dy h rstd)) + grad_sum
//   grad_weight = sum over the rows of grad_out h rstd
//
// A row belongs to 8 to 256 threads, which hold it in registers in pieces of eight columns between the
// reduction and the output, so every operand is read once.  The backward walks strips of rows with
// the columns of grad_weight in registers; its partial sums of the strips are added by a second kernel
// (no atomics).
//
// Bound by HBM: 16384 rows of 1024, bf16, with residual: forward 134 MB in 21 us (6.3 TB/s, the last-level cache holding
// a part), backward 134 MB in 22.6 us and 4.0 for the join; 8191 rows of 4096 to e4m3: 235 MB in 36.8 us (6.4 TB/s).
#include <algorithm>
#include <type_traits>

#include "readout.hpp"
#include "readout_device.hpp"

namespace oeq {
namespace readout {

namespace {

constexpr int kThreads = 256;
constexpr float kMostE4m3 = 448.f;

// A thread's part of a row: kPieces pieces of eight columns, kGroup threads a row.
template <class T, int kGroup, int kPieces>
struct Row {
    vec8<T> v[kPieces];
    static __device__ __forceinline__ int col(int i) { return (i * kGroup + int(threadIdx.x) % kGroup) * 8; }
    // Where all pieces are whole, as in most rows, the loads are in a row: a value that came by two ways
    // would be waited for where they meet, before the next load.
    __device__ __forceinline__ void load(const T *row, int cols) {
        if (cols >= kGroup * kPieces * 8) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) v[i] = load8(row + col(i));
            return;
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int c = col(i), n = cols - c;
            v[i] = n >= 8 ? load8(row + c) : n > 0 ? load_part(row + c, n) : vec8<T>(T(0.f));
        }
    }
};
template <class T>
__device__ __forceinline__ void put(T *row, int c, int cols, vec8<T> v) {
    const int n = cols - c;
    if (n >= 8)
        store8(row + c, v);
    else if (n > 0)
        store_part(row + c, v, n);
}
// Eight weights from column c on; past the row's end, zeros.
__device__ __forceinline__ f32x8 weights(const float *weight, int c, int cols) {
    if (!weight) return f32x8(1.f);
    const int n = cols - c;
    return n >= 8 ? load8(weight + c) : n > 0 ? load_part(weight + c, n) : f32x8{};
}

// Sum (or maximum) over the threads of a row; all of them get it.  kCall numbers the calls of a
// kernel, which have an LDS array each, so that a call needs one barrier.
template <int kGroup, int kCall, bool kMax>
__device__ __forceinline__ float across(float v) {
    constexpr int kIn = kGroup < 64 ? kGroup : 64;
#pragma unroll
    for (int off = 1; off < kIn; off <<= 1) {
        const float o = __shfl_xor(v, off);
        v = kMax ? fmaxf(v, o) : v + o;
    }
    if constexpr (kGroup > 64) {
        __shared__ float of_wave[kGroup / 64];
        if ((threadIdx.x & 63) == 0) of_wave[threadIdx.x >> 6] = v;
        __syncthreads();
        v = of_wave[0];
#pragma unroll
        for (int w = 1; w < kGroup / 64; ++w) v = kMax ? fmaxf(v, of_wave[w]) : v + of_wave[w];
    }
    return v;
}

template <class T, int kGroup, int kPieces>
__device__ __forceinline__ float squares(const Row<T, kGroup, kPieces> &h, float by) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const f32x8 v = to_f32<T>(h.v[i]) * by;
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(v[j], v[j], s);
    }
    return s;
}

template <class T, int kGroup, int kPieces, bool kE4m3>
__global__ void __launch_bounds__(kThreads) k_norm(RmsNormArgs a) {
    const int64_t row = int64_t(blockIdx.x) * (kThreads / kGroup) + threadIdx.x / kGroup;
    const bool in = row < a.rows;  // rows past the end stay for the reductions
    using R = Row<T, kGroup, kPieces>;
    R h;
    const int cols = in ? a.cols : 0;
    h.load(static_cast<const T *>(a.x) + (in ? row * a.ld_x : 0), cols);
    if (a.residual) {
        R r;
        r.load(static_cast<const T *>(a.residual) + (in ? row * a.ld_residual : 0), cols);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            h.v[i] = from_f32<T>(to_f32<T>(h.v[i]) + to_f32<T>(r.v[i]));
            put(static_cast<T *>(a.sum) + (in ? row * a.ld_sum : 0), R::col(i), cols, h.v[i]);
        }
    }
    const float share = 1.f / a.cols;
    const float mean = across<kGroup, 0, false>(squares(h, 1.f)) * share;
    float rstd = 1.f / sqrtf(mean + a.eps);
    // squares that leave fp32 (values past 2^63, or where eps is tiny below 2^-50): again with the row
    // scaled by a power of two.  The condition is the same for all threads of a row, and the barrier
    // of `across` is one workgroup's row.
    const bool high = mean == INFINITY, low = mean < 0x1p-100f && a.eps < 0x1p-60f;
    if (kGroup > 64 ? high || low : __any(high || low)) {
        const float by = high ? 0x1p-80f : 0x1p60f;
        const float scaled = across<kGroup, 1, false>(squares(h, by)) * share;
        if (high || low) rstd = by / sqrtf(scaled + a.eps * by * by);
    }
    if (in && a.rstd && threadIdx.x % kGroup == 0) a.rstd[row] = rstd;

    if constexpr (!kE4m3) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const f32x8 y = to_f32<T>(h.v[i]) * rstd * weights(a.weight, R::col(i), cols);
            put(static_cast<T *>(a.out) + (in ? row * a.ld_out : 0), R::col(i), cols, from_f32<T>(y));
        }
    } else {
        f32x8 y[kPieces];
        float most = 0.f, bad = 0.f;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            y[i] = to_f32<T>(h.v[i]) * rstd * weights(a.weight, R::col(i), cols);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                most = fmaxf(most, fabsf(y[i][j]));
                bad = y[i][j] != y[i][j] ? y[i][j] : bad;  // the maximum leaves a NaN out
            }
        }
        most = across<kGroup, 2, true>(most);
        bad = across<kGroup, 3, false>(bad);
        // a row of zeros has a scale all the same, so that it can be divided by
        const float scale = fmaxf(most, 0x1p-100f) / kMostE4m3 + bad, inverse = 1.f / scale;
        if (in && threadIdx.x % kGroup == 0) a.out_scale[row] = scale;
        uint8_t *out = static_cast<uint8_t *>(a.out) + (in ? row * a.ld_out : 0);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            // |y / scale| is at most 448 and a rounding, which e4m3 rounds to 448
            const f32x8 q = y[i] * inverse;
            int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
            lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
            int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
            hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
            const uint64_t bytes = uint64_t(uint32_t(hi)) << 32 | uint32_t(lo);
            const int c = R::col(i), n = cols - c;
            if (n >= 8) {
                __builtin_memcpy(out + c, &bytes, 8);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < n) out[c + j] = static_cast<uint8_t>(bytes >> (8 * j));
            }
        }
    }
}

// Strips of rows: a workgroup's rows are blockIdx.x, + gridDim.x, ... in steps of kThreads / kGroup rows.
template <class T, int kGroup, int kPieces>
__global__ void __launch_bounds__(kThreads) k_norm_grad(RmsNormArgs a, float *part) {
    constexpr int kRows = kThreads / kGroup;
    using R = Row<T, kGroup, kPieces>;
    const int cols = a.cols, mine = threadIdx.x / kGroup;
    const float share = 1.f / cols;
    f32x8 gw[kPieces] = {}, w[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) w[i] = weights(a.weight, R::col(i), cols);
    const int64_t steps = (a.rows + kRows - 1) / kRows;
    for (int64_t step = blockIdx.x; step < steps; step += gridDim.x) {
        const int64_t row = step * kRows + mine;
        const bool in = row < a.rows;
        const int n = in ? cols : 0;
        R h, g, more;
        h.load(static_cast<const T *>(a.sum) + (in ? row * a.ld_sum : 0), n);
        g.load(static_cast<const T *>(a.grad_out) + (in ? row * a.ld_grad_out : 0), n);
        if (a.grad_sum) more.load(static_cast<const T *>(a.grad_sum) + (in ? row * a.ld_grad_sum : 0), n);
        const float rstd = in ? a.rstd[row] : 0.f;
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const f32x8 hat = to_f32<T>(h.v[i]) * rstd, go = to_f32<T>(g.v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dot = fmaf(go[j] * w[i][j], hat[j], dot);
                gw[i][j] = fmaf(go[j], hat[j], gw[i][j]);
            }
        }
        if (!a.grad_x) continue;
        if (kGroup > 64) __syncthreads();  // the step before has read its sums
        dot = across<kGroup, 0, false>(dot) * share;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const f32x8 hat = to_f32<T>(h.v[i]) * rstd, go = to_f32<T>(g.v[i]);
            f32x8 d;
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = rstd * fmaf(-hat[j], dot, go[j] * w[i][j]);
            if (a.grad_sum) d += to_f32<T>(more.v[i]);
            put(static_cast<T *>(a.grad_x) + (in ? row * a.ld_grad_x : 0), R::col(i), n, from_f32<T>(d));
        }
    }
    if (!part) return;
    float *to = part + int64_t(blockIdx.x) * cols;
    if constexpr (kRows == 1) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) put(to, R::col(i), cols, gw[i]);
    } else {
        constexpr int kWide = kGroup * kPieces * 8;
        __shared__ float sums[kRows * kWide];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) store8(sums + mine * kWide + R::col(i), gw[i]);
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += kThreads) {
            float s = 0.f;
            for (int r = 0; r < kRows; ++r) s += sums[r * kWide + c];
            to[c] = s;
        }
    }
}

// grad_weight from the partial sums of `strips` strips: 16 columns a workgroup, 64 threads for each.
constexpr int kJoinThreads = 1024, kJoinCols = 16;
__global__ void __launch_bounds__(kJoinThreads) k_join_strips(const float *part, int strips, int cols, float *grad_weight) {
    constexpr int kShares = kJoinThreads / kJoinCols;
    __shared__ double sums[kShares][kJoinCols];
    const int lane = threadIdx.x % kJoinCols, share = threadIdx.x / kJoinCols, c = blockIdx.x * kJoinCols + lane;
    double s = 0.;
    if (c < cols) {
#pragma unroll 16
        for (int i = share; i < strips; i += kShares) s += part[int64_t(i) * cols + c];
    }
    sums[share][lane] = s;
    __syncthreads();
    if (share || c >= cols) return;
    for (int i = 1; i < kShares; ++i) s += sums[i][lane];
    grad_weight[c] = static_cast<float>(s);
}

// f(kGroup, kPieces) for the smallest group and pieces that hold a row: up to two pieces a thread in a
// wave, then a workgroup.
template <class F>
hipError_t with_shape(int cols, F &&f) {
    using std::integral_constant;
    const auto go = [&](auto group, auto pieces) { return f(group, pieces); };
    if (cols <= 64) return go(integral_constant<int, 8>(), integral_constant<int, 1>());
    if (cols <= 128) return go(integral_constant<int, 16>(), integral_constant<int, 1>());
    if (cols <= 256) return go(integral_constant<int, 32>(), integral_constant<int, 1>());
    if (cols <= 512) return go(integral_constant<int, 64>(), integral_constant<int, 1>());
    if (cols <= 1024) return go(integral_constant<int, 64>(), integral_constant<int, 2>());
    if (cols <= 2048) return go(integral_constant<int, 256>(), integral_constant<int, 1>());
    if (cols <= 4096) return go(integral_constant<int, 256>(), integral_constant<int, 2>());
    if (cols <= 8192) return go(integral_constant<int, 256>(), integral_constant<int, 4>());
    return go(integral_constant<int, 256>(), integral_constant<int, 8>());
}

int group_of(int cols) {
    return cols <= 64 ? 8 : cols <= 128 ? 16 : cols <= 256 ? 32 : cols <= 1024 ? 64 : 256;
}

int64_t strips_of(int64_t rows, int32_t cols) {
    const int64_t steps = (rows + kThreads / group_of(cols) - 1) / (kThreads / group_of(cols));
    return std::min<int64_t>(steps, 1024);
}

template <class T>
hipError_t forward(const RmsNormArgs &a, hipStream_t stream) {
    return with_shape(a.cols, [&](auto group, auto pieces) {
        constexpr int kGroup = decltype(group)::value, kPieces = decltype(pieces)::value, kRows = kThreads / kGroup;
        const dim3 blocks(static_cast<unsigned>((a.rows + kRows - 1) / kRows)), threads(kThreads);
        if (a.out_scale)
            k_norm<T, kGroup, kPieces, true><<<blocks, threads, 0, stream>>>(a);
        else
            k_norm<T, kGroup, kPieces, false><<<blocks, threads, 0, stream>>>(a);
        return hipGetLastError();
    });
}

template <class T>
hipError_t backward(const RmsNormArgs &a, hipStream_t stream) {
    const int64_t strips = strips_of(a.rows, a.cols);
    float *part = a.grad_weight ? static_cast<float *>(a.workspace) : nullptr;
    if (strips) {
        const hipError_t e = with_shape(a.cols, [&](auto group, auto pieces) {
            constexpr int kGroup = decltype(group)::value, kPieces = decltype(pieces)::value;
            const dim3 blocks(static_cast<unsigned>(strips));
            k_norm_grad<T, kGroup, kPieces><<<blocks, dim3(kThreads), 0, stream>>>(a, part);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
    }
    if (a.grad_weight)
        k_join_strips<<<dim3((a.cols + kJoinCols - 1) / kJoinCols), dim3(kJoinThreads), 0, stream>>>(
            part, static_cast<int>(strips), a.cols, a.grad_weight);
    return hipGetLastError();
}

}  // namespace

int64_t rms_norm_blocks(int64_t rows, int32_t cols) {
    const int64_t in_block = kThreads / group_of(cols);
    return (rows + in_block - 1) / in_block;
}

size_t rms_norm_workspace(int64_t rows, int32_t cols) {
    return (static_cast<size_t>(strips_of(rows, cols)) * cols * 4 + 255) / 256 * 256;
}

hipError_t rms_norm_fwd(oeq_dtype dtype, const RmsNormArgs &a, hipStream_t stream) {
    switch (dtype) {
        case OEQ_F32: return forward<float>(a, stream);
        case OEQ_F16: return forward<f16>(a, stream);
        case OEQ_BF16: return forward<bf16>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

hipError_t rms_norm_bwd(oeq_dtype dtype, const RmsNormArgs &a, hipStream_t stream) {
    switch (dtype) {
        case OEQ_F32: return backward<float>(a, stream);
        case OEQ_F16: return backward<f16>(a, stream);
        case OEQ_BF16: return backward<bf16>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace readout
}  // namespace oeq
