// Group norm over the rows of each structure, channels last, with an optional SiLU.
//
// Structure b has the rows [ptr[b], ptr[b+1]); group g has the C / G channels from g C / G
// on.  Over the n = rows * C / G elements of (b, g):
//   mean, var = the mean and the (biased) variance, rstd = 1 / sqrt(var + eps)
//   xhat = (x - mean) rstd,  z = xhat w + b,  y = z or z / (1 + exp(-z))
// and with dz = grad_out * dy/dz, dh = dz w:
//   grad_w = sum dz xhat, grad_b = sum dz (over all rows)
//   grad_x = rstd (dh - mean(dh) - xhat mean(dh xhat))
// An empty structure has mean 0 and rstd 0.
//
// Everything here is bound by memory.  A workgroup owns (structure, split of its rows, slab
// of whole groups, about 64 channels): lanes run along the channels in pieces of eight, so a
// row of the slab is one 128- or 256-byte access, and the sums over the rows are each
// thread's own until one reduction at the end.  Structures of few rows take one split, whose
// workgroup computes the sums and then applies them (the second read comes from its cache);
// with more splits the partial sums go through the workspace to a joining kernel and a third
// one applies them.  No atomics: every result is bitwise repeatable.
//
// Sums are fp32 in a thread and fp64 from there on.  The variance is summed about the
// channel's value in the split's first row, so it does not cancel against a large mean.
#include <type_traits>

#include "readout.hpp"
#include "readout_device.hpp"

namespace oeq {
namespace readout {

namespace {

constexpr int kThreads = 256;
constexpr int kSlab = 64;         // channels of a slab, where a group is not wider
constexpr int kSplitRows = 256;   // rows a split has at least, on average
constexpr int kMostSplits = 256;

struct Shape {
    int cg;         // channels of a group
    int gps;        // groups of a slab
    int n_slabs;
    int cols;       // threads along a slab's channels (a power of two)
    int splits;
};

Shape shape_of(int64_t rows, int32_t n_struct, int32_t channels, int32_t groups) {
    Shape s;
    s.cg = channels / groups;
    s.gps = s.cg >= kSlab ? 1 : kSlab / s.cg;
    if (s.gps > groups) s.gps = groups;
    s.n_slabs = (groups + s.gps - 1) / s.gps;
    s.gps = (groups + s.n_slabs - 1) / s.n_slabs;
    s.cols = 1;
    while (s.cols * 8 < s.gps * s.cg) s.cols *= 2;
    int64_t splits = (rows / n_struct + kSplitRows - 1) / kSplitRows;
    s.splits = static_cast<int>(splits < 1 ? 1 : splits > kMostSplits ? kMostSplits : splits);
    return s;
}

__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * z));
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
    return v;
}

// What a thread works on: the channels [c, c + n) (n <= 8, none for n <= 0) of the rows
// begin + lane, begin + lane + lanes, ... of its split.
struct Part {
    int64_t begin, end;
    int c, n, lane, lanes, c0, width, g0, n_groups;
};

__device__ __forceinline__ Part part_of(const GroupNormArgs &a, const Shape &s, int b, int split, int slab) {
    Part p;
    const Span rows = span_of(a.ptr, b, a.rows);
    const int64_t len = rows.end - rows.begin;
    p.begin = rows.begin + len * split / s.splits;
    p.end = rows.begin + len * (split + 1) / s.splits;
    p.g0 = slab * s.gps;
    p.n_groups = a.groups - p.g0 < s.gps ? a.groups - p.g0 : s.gps;
    p.c0 = p.g0 * s.cg;
    p.width = p.n_groups * s.cg;
    const int col = threadIdx.x & (s.cols - 1);
    p.c = p.c0 + col * 8;
    p.n = p.width - col * 8 < 8 ? p.width - col * 8 : 8;
    p.lane = threadIdx.x / s.cols;
    p.lanes = kThreads / s.cols;
    return p;
}

template <class T>
__device__ __forceinline__ f32x8 fetch(const void *base, int64_t ld, int64_t row, const Part &p) {
    const T *at = static_cast<const T *>(base) + row * ld + p.c;
    return to_f32<T>(p.n == 8 ? load8(at) : load_part(at, p.n));
}
template <class T>
__device__ __forceinline__ void put(void *base, int64_t ld, int64_t row, const Part &p, f32x8 v) {
    T *at = static_cast<T *>(base) + row * ld + p.c;
    const vec8<T> o = from_f32<T>(v);
    if (p.n == 8)
        store8(at, o);
    else
        store_part(at, o, p.n);
}
__device__ __forceinline__ f32x8 channel_values(const float *v, const Part &p, float without) {
    f32x8 o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = v && j < p.n ? v[p.c + j] : without;
    return o;
}

// Sums two values per channel over the rows' threads; afterwards sums[i][c - c0] holds them.
// `sums` has room for kThreads * 8 values a piece.
__device__ __forceinline__ void channel_sums(f32x8 u, f32x8 v, const Part &p, int cols, float (*sums)[kThreads * 8]) {
    for (int off = cols; off < 64; off <<= 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            u[j] += __shfl_xor(u[j], off);
            v[j] += __shfl_xor(v[j], off);
        }
    }
    // waves that hold the same channels are added in order through LDS
    const int per_set = cols > 64 ? cols / 64 : 1, sets = 4 / per_set, wave = threadIdx.x >> 6;
    const int col = threadIdx.x & (cols - 1), set = wave / per_set;
    if (p.lane % (cols < 64 ? 64 / cols : 1) == 0 && p.n > 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sums[0][set * cols * 8 + col * 8 + j] = u[j];
            sums[1][set * cols * 8 + col * 8 + j] = v[j];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.width; c += kThreads) {
        for (int k = 1; k < sets; ++k) {
            sums[0][c] += sums[0][k * cols * 8 + c];
            sums[1][c] += sums[1][k * cols * 8 + c];
        }
    }
    __syncthreads();
}

// Mean and sum of squared deviations of each group of the slab over the part's rows, left in
// group_mean / group_m2 (LDS, by group of the slab).
template <class T>
__device__ __forceinline__ void statistics(const GroupNormArgs &a, const Shape &s, const Part &p,
                                           float (*sums)[kThreads * 8], double *group_mean, double *group_m2) {
    const int64_t n = p.end - p.begin;
    f32x8 shift = {}, u = {}, v = {};
    if (p.n > 0 && n > 0) {
        shift = fetch<T>(a.x, a.ld_x, p.begin, p);
#pragma unroll 4
        for (int64_t r = p.begin + p.lane; r < p.end; r += p.lanes) {
            const f32x8 d = fetch<T>(a.x, a.ld_x, r, p) - shift;
            u += d;
            v += d * d;
        }
    }
    channel_sums(u, v, p, s.cols, sums);
    const int lane = threadIdx.x & 63;
    for (int g = threadIdx.x >> 6; g < p.n_groups; g += kThreads / 64) {
        double mean = 0, m2 = 0;
        if (n > 0) {
            const T *first = static_cast<const T *>(a.x) + p.begin * a.ld_x + p.c0 + g * s.cg;
            for (int c = lane; c < s.cg; c += 64)
                mean += double(static_cast<float>(first[c])) + double(sums[0][g * s.cg + c]) / double(n);
            mean = wave_sum(mean) / s.cg;
            for (int c = lane; c < s.cg; c += 64) {
                const double total = sums[0][g * s.cg + c];
                const double off = double(static_cast<float>(first[c])) + total / double(n) - mean;
                const double own = double(sums[1][g * s.cg + c]) - total * total / double(n);
                m2 += own + double(n) * off * off;
            }
            m2 = wave_sum(m2);
        }
        if (lane == 0) {
            group_mean[g] = mean;
            group_m2[g] = m2;
        }
    }
    __syncthreads();
}

__device__ __forceinline__ float rstd_of(double m2, double n, float eps) {
    const double var = m2 > 0 || !(m2 == m2) ? m2 / n : 0;  // rounding can leave a small negative sum
    return n > 0 ? static_cast<float>(1.0 / sqrt(var + double(eps))) : 0.f;
}

template <class T, bool kSilu>
__device__ __forceinline__ void apply_forward(const GroupNormArgs &a, const Part &p, f32x8 mean, f32x8 rstd) {
    if (p.n <= 0) return;
    const f32x8 w = channel_values(a.weight, p, 1.f) * rstd, bias = channel_values(a.bias, p, 0.f);
#pragma unroll 4
    for (int64_t r = p.begin + p.lane; r < p.end; r += p.lanes) {
        f32x8 z = (fetch<T>(a.x, a.ld_x, r, p) - mean) * w + bias;
        if (kSilu) {
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] *= sigmoid(z[j]);
        }
        put<T>(a.out, a.ld_out, r, p, z);
    }
}

// One split: statistics and output in one launch.
template <class T, bool kSilu>
__global__ void __launch_bounds__(kThreads) k_forward(GroupNormArgs a, Shape s) {
    __shared__ float sums[2][kThreads * 8];
    __shared__ double group_mean[kSlab], group_m2[kSlab];
    const int b = blockIdx.x / s.n_slabs;
    const Part p = part_of(a, s, b, 0, blockIdx.x % s.n_slabs);
    statistics<T>(a, s, p, sums, group_mean, group_m2);
    const double n = double(p.end - p.begin) * s.cg;
    f32x8 mean = {}, rstd = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j < p.n) {
            const int g = (p.c + j - p.c0) / s.cg;
            mean[j] = static_cast<float>(group_mean[g]);
            rstd[j] = rstd_of(group_m2[g], n, a.eps);
        }
    }
    if (threadIdx.x < p.n_groups) {
        const int64_t at = int64_t(b) * a.groups + p.g0 + threadIdx.x;
        a.mean[at] = static_cast<float>(group_mean[threadIdx.x]);
        a.rstd[at] = rstd_of(group_m2[threadIdx.x], n, a.eps);
    }
    apply_forward<T, kSilu>(a, p, mean, rstd);
}

// Several splits.  partial[(b, split, group)] = {mean, sum of squared deviations}
template <class T>
__global__ void __launch_bounds__(kThreads) k_statistics(GroupNormArgs a, Shape s, double2 *partial) {
    __shared__ float sums[2][kThreads * 8];
    __shared__ double group_mean[kSlab], group_m2[kSlab];
    const int64_t part = blockIdx.x / s.n_slabs;
    const Part p = part_of(a, s, static_cast<int>(part / s.splits), static_cast<int>(part % s.splits),
                           blockIdx.x % s.n_slabs);
    statistics<T>(a, s, p, sums, group_mean, group_m2);
    if (threadIdx.x < p.n_groups)
        partial[part * a.groups + p.g0 + threadIdx.x] = make_double2(group_mean[threadIdx.x], group_m2[threadIdx.x]);
}

// One wave joins the splits of one (structure, group).
__global__ void __launch_bounds__(kThreads) k_join_statistics(GroupNormArgs a, Shape s, const double2 *partial) {
    const int64_t at = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (at >= int64_t(a.n_struct) * a.groups) return;
    const int b = static_cast<int>(at / a.groups), g = static_cast<int>(at % a.groups), lane = threadIdx.x & 63;
    const Span rows = span_of(a.ptr, b, a.rows);
    const int64_t len = rows.end - rows.begin;
    const double n = double(len) * s.cg;
    double mean = 0, m2 = 0;
    for (int i = lane; i < s.splits; i += 64) {
        const double k = double(len * (i + 1) / s.splits - len * i / s.splits) * s.cg;
        mean += k * partial[(int64_t(b) * s.splits + i) * a.groups + g].x;
    }
    mean = n > 0 ? wave_sum(mean) / n : 0;
    for (int i = lane; i < s.splits; i += 64) {
        const double k = double(len * (i + 1) / s.splits - len * i / s.splits) * s.cg;
        const double2 v = partial[(int64_t(b) * s.splits + i) * a.groups + g];
        if (k > 0) m2 += v.y + k * (v.x - mean) * (v.x - mean);
    }
    m2 = wave_sum(m2);
    if (lane == 0) {
        a.mean[at] = static_cast<float>(mean);
        a.rstd[at] = rstd_of(m2, n, a.eps);
    }
}

__device__ __forceinline__ void saved_statistics(const GroupNormArgs &a, const Shape &s, int b, const Part &p,
                                                 f32x8 *mean, f32x8 *rstd) {
    *mean = f32x8{};
    *rstd = f32x8{};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j < p.n) {
            const int64_t at = int64_t(b) * a.groups + (p.c + j) / s.cg;
            (*mean)[j] = a.mean[at];
            (*rstd)[j] = a.rstd[at];
        }
    }
}

template <class T, bool kSilu>
__global__ void __launch_bounds__(kThreads) k_apply(GroupNormArgs a, Shape s) {
    const int64_t part = blockIdx.x / s.n_slabs;
    const int b = static_cast<int>(part / s.splits);
    const Part p = part_of(a, s, b, static_cast<int>(part % s.splits), blockIdx.x % s.n_slabs);
    f32x8 mean, rstd;
    saved_statistics(a, s, b, p, &mean, &rstd);
    apply_forward<T, kSilu>(a, p, mean, rstd);
}

// ---- backward -----------------------------------------------------------------------

// xhat and dz of eight elements
template <class T, bool kSilu>
__device__ __forceinline__ void local_gradient(const GroupNormArgs &a, int64_t r, const Part &p, f32x8 mean, f32x8 rstd,
                                               f32x8 w, f32x8 bias, f32x8 *xhat, f32x8 *dz) {
    const f32x8 h = (fetch<T>(a.x, a.ld_x, r, p) - mean) * rstd;
    f32x8 g = fetch<T>(a.grad_out, a.ld_grad_out, r, p);
    if (kSilu) {
        const f32x8 z = h * w + bias;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float gate = sigmoid(z[j]);
            g[j] *= gate * (1.f + z[j] * (1.f - gate));
        }
    }
    *xhat = h;
    *dz = g;
}

// Sums of a part's dz and dz xhat by channel (to `column`, unless NULL: row `part` of two
// fp32 rows of C channels) and, weighted, by group of the slab (left in LDS).
template <class T, bool kSilu>
__device__ __forceinline__ void gradient_sums(const GroupNormArgs &a, const Shape &s, const Part &p, int64_t part,
                                              f32x8 mean, f32x8 rstd, f32x8 w, f32x8 bias, float *column,
                                              float (*sums)[kThreads * 8], double *group_dh, double *group_dhx) {
    f32x8 u = {}, v = {};
    if (p.n > 0) {
#pragma unroll 2
        for (int64_t r = p.begin + p.lane; r < p.end; r += p.lanes) {
            f32x8 xhat, dz;
            local_gradient<T, kSilu>(a, r, p, mean, rstd, w, bias, &xhat, &dz);
            u += dz;
            v += dz * xhat;
        }
    }
    channel_sums(u, v, p, s.cols, sums);
    if (column) {
        for (int c = threadIdx.x; c < p.width; c += kThreads) {
            column[part * 2 * a.channels + p.c0 + c] = sums[0][c];
            column[(part * 2 + 1) * a.channels + p.c0 + c] = sums[1][c];
        }
    }
    const int lane = threadIdx.x & 63;
    for (int g = threadIdx.x >> 6; g < p.n_groups; g += kThreads / 64) {
        double dh = 0, dhx = 0;
        for (int c = lane; c < s.cg; c += 64) {
            const double wc = a.weight ? a.weight[p.c0 + g * s.cg + c] : 1.f;
            dh += wc * sums[0][g * s.cg + c];
            dhx += wc * sums[1][g * s.cg + c];
        }
        dh = wave_sum(dh);
        dhx = wave_sum(dhx);
        if (lane == 0) {
            group_dh[g] = dh;
            group_dhx[g] = dhx;
        }
    }
    __syncthreads();
}

template <class T, bool kSilu>
__device__ __forceinline__ void apply_backward(const GroupNormArgs &a, const Part &p, f32x8 mean, f32x8 rstd, f32x8 w,
                                               f32x8 bias, f32x8 m1, f32x8 m2) {
    if (p.n <= 0) return;
#pragma unroll 2
    for (int64_t r = p.begin + p.lane; r < p.end; r += p.lanes) {
        f32x8 xhat, dz;
        local_gradient<T, kSilu>(a, r, p, mean, rstd, w, bias, &xhat, &dz);
        put<T>(a.grad_x, a.ld_grad_x, r, p, rstd * (dz * w - m1 - xhat * m2));
    }
}

template <class T, bool kSilu>
__global__ void __launch_bounds__(kThreads) k_backward(GroupNormArgs a, Shape s, float *column) {
    __shared__ float sums[2][kThreads * 8];
    __shared__ double group_dh[kSlab], group_dhx[kSlab];
    const int b = blockIdx.x / s.n_slabs;
    const Part p = part_of(a, s, b, 0, blockIdx.x % s.n_slabs);
    f32x8 mean, rstd;
    saved_statistics(a, s, b, p, &mean, &rstd);
    const f32x8 w = channel_values(a.weight, p, 1.f), bias = channel_values(a.bias, p, 0.f);
    gradient_sums<T, kSilu>(a, s, p, b, mean, rstd, w, bias, column, sums, group_dh, group_dhx);
    if (!a.grad_x) return;
    const double n = double(p.end - p.begin) * s.cg;
    f32x8 m1 = {}, m2 = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j < p.n && n > 0) {
            const int g = (p.c + j - p.c0) / s.cg;
            m1[j] = static_cast<float>(group_dh[g] / n);
            m2[j] = static_cast<float>(group_dhx[g] / n);
        }
    }
    apply_backward<T, kSilu>(a, p, mean, rstd, w, bias, m1, m2);
}

template <class T, bool kSilu>
__global__ void __launch_bounds__(kThreads) k_gradient_sums(GroupNormArgs a, Shape s, float *column, double2 *partial) {
    __shared__ float sums[2][kThreads * 8];
    __shared__ double group_dh[kSlab], group_dhx[kSlab];
    const int64_t part = blockIdx.x / s.n_slabs;
    const int b = static_cast<int>(part / s.splits);
    const Part p = part_of(a, s, b, static_cast<int>(part % s.splits), blockIdx.x % s.n_slabs);
    f32x8 mean, rstd;
    saved_statistics(a, s, b, p, &mean, &rstd);
    const f32x8 w = channel_values(a.weight, p, 1.f), bias = channel_values(a.bias, p, 0.f);
    gradient_sums<T, kSilu>(a, s, p, part, mean, rstd, w, bias, column, sums, group_dh, group_dhx);
    if (threadIdx.x < p.n_groups)
        partial[part * a.groups + p.g0 + threadIdx.x] = make_double2(group_dh[threadIdx.x], group_dhx[threadIdx.x]);
}

// The first `join_blocks` workgroups join the splits' group sums to means (one wave a
// (structure, group)); the others sum `column` over its rows, 16 channels a workgroup.
__global__ void __launch_bounds__(kThreads) k_join_gradients(GroupNormArgs a, Shape s, const double2 *partial,
                                                             float2 *joined, const float *column, int join_blocks) {
    if (static_cast<int>(blockIdx.x) < join_blocks) {
        const int64_t at = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
        if (at >= int64_t(a.n_struct) * a.groups) return;
        const int b = static_cast<int>(at / a.groups), g = static_cast<int>(at % a.groups), lane = threadIdx.x & 63;
        const Span rows = span_of(a.ptr, b, a.rows);
        const double n = double(rows.end - rows.begin) * s.cg;
        double u = 0, v = 0;
        for (int i = lane; i < s.splits; i += 64) {
            const double2 t = partial[(int64_t(b) * s.splits + i) * a.groups + g];
            u += t.x;
            v += t.y;
        }
        u = wave_sum(u);
        v = wave_sum(v);
        if (lane == 0) joined[at] = n > 0 ? make_float2(static_cast<float>(u / n), static_cast<float>(v / n))
                                          : make_float2(0.f, 0.f);
        return;
    }
    __shared__ double part[2][kThreads];
    const int c = (blockIdx.x - join_blocks) * 16 + (threadIdx.x & 15), lane = threadIdx.x >> 4;
    const int64_t n_parts = int64_t(a.n_struct) * s.splits;
    double u = 0, v = 0;
    if (c < a.channels) {
#pragma unroll 4
        for (int64_t r = lane; r < n_parts; r += kThreads / 16) {
            u += column[r * 2 * a.channels + c];
            v += column[(r * 2 + 1) * a.channels + c];
        }
    }
    part[0][threadIdx.x] = u;
    part[1][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x < 16 && c < a.channels) {
        for (int k = 1; k < kThreads / 16; ++k) {
            u += part[0][k * 16 + threadIdx.x];
            v += part[1][k * 16 + threadIdx.x];
        }
        if (a.grad_bias) a.grad_bias[c] = static_cast<float>(u);
        if (a.grad_weight) a.grad_weight[c] = static_cast<float>(v);
    }
}

template <class T, bool kSilu>
__global__ void __launch_bounds__(kThreads) k_apply_backward(GroupNormArgs a, Shape s, const float2 *joined) {
    const int64_t part = blockIdx.x / s.n_slabs;
    const int b = static_cast<int>(part / s.splits);
    const Part p = part_of(a, s, b, static_cast<int>(part % s.splits), blockIdx.x % s.n_slabs);
    f32x8 mean, rstd, m1 = {}, m2 = {};
    saved_statistics(a, s, b, p, &mean, &rstd);
    const f32x8 w = channel_values(a.weight, p, 1.f), bias = channel_values(a.bias, p, 0.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j < p.n) {
            const float2 t = joined[int64_t(b) * a.groups + (p.c + j) / s.cg];
            m1[j] = t.x;
            m2[j] = t.y;
        }
    }
    apply_backward<T, kSilu>(a, p, mean, rstd, w, bias, m1, m2);
}

constexpr size_t up(size_t v) { return (v + 255) / 256 * 256; }

// Workspace pieces: the splits' group sums, the joined means of the backward, the channel sums.
struct Pieces {
    size_t partial, joined, column, bytes;
};
Pieces pieces_of(const Shape &s, int32_t n_struct, int32_t channels, int32_t groups) {
    Pieces w;
    const size_t parts = static_cast<size_t>(n_struct) * s.splits;
    w.partial = 0;
    w.joined = w.partial + (s.splits > 1 ? up(parts * groups * sizeof(double2)) : 0);
    w.column = w.joined + (s.splits > 1 ? up(static_cast<size_t>(n_struct) * groups * sizeof(float2)) : 0);
    w.bytes = w.column + up(parts * channels * 2 * sizeof(float));
    return w;
}

template <class T, bool kSilu>
hipError_t forward(const GroupNormArgs &a, hipStream_t stream) {
    const Shape s = shape_of(a.rows, a.n_struct, a.channels, a.groups);
    const dim3 grid(static_cast<unsigned>(int64_t(a.n_struct) * s.splits * s.n_slabs)), threads(kThreads);
    if (s.splits == 1) {
        k_forward<T, kSilu><<<grid, threads, 0, stream>>>(a, s);
        return hipGetLastError();
    }
    double2 *partial = static_cast<double2 *>(a.workspace);
    k_statistics<T><<<grid, threads, 0, stream>>>(a, s, partial);
    const dim3 join(static_cast<unsigned>((int64_t(a.n_struct) * a.groups + 3) / 4));
    k_join_statistics<<<join, threads, 0, stream>>>(a, s, partial);
    k_apply<T, kSilu><<<grid, threads, 0, stream>>>(a, s);
    return hipGetLastError();
}

template <class T, bool kSilu>
hipError_t backward(const GroupNormArgs &a, hipStream_t stream) {
    const bool params = a.grad_weight || a.grad_bias;
    const int channel_blocks = params ? (a.channels + 15) / 16 : 0;
    const dim3 threads(kThreads);
    if (a.rows == 0 || a.n_struct == 0) {  // no parts: zeros
        if (params)
            k_join_gradients<<<dim3(channel_blocks), threads, 0, stream>>>(a, Shape{}, nullptr, nullptr, nullptr, 0);
        return hipGetLastError();
    }
    const Shape s = shape_of(a.rows, a.n_struct, a.channels, a.groups);
    const Pieces w = pieces_of(s, a.n_struct, a.channels, a.groups);
    char *ws = static_cast<char *>(a.workspace);
    double2 *partial = reinterpret_cast<double2 *>(ws + w.partial);
    float2 *joined = reinterpret_cast<float2 *>(ws + w.joined);
    float *column = params ? reinterpret_cast<float *>(ws + w.column) : nullptr;
    const dim3 grid(static_cast<unsigned>(int64_t(a.n_struct) * s.splits * s.n_slabs));
    if (s.splits == 1) {
        k_backward<T, kSilu><<<grid, threads, 0, stream>>>(a, s, column);
        if (params) k_join_gradients<<<dim3(channel_blocks), threads, 0, stream>>>(a, s, partial, joined, column, 0);
        return hipGetLastError();
    }
    k_gradient_sums<T, kSilu><<<grid, threads, 0, stream>>>(a, s, column, partial);
    const int join_blocks = a.grad_x ? static_cast<int>((int64_t(a.n_struct) * a.groups + 3) / 4) : 0;
    k_join_gradients<<<dim3(join_blocks + channel_blocks), threads, 0, stream>>>(a, s, partial, joined, column,
                                                                                join_blocks);
    if (a.grad_x) k_apply_backward<T, kSilu><<<grid, threads, 0, stream>>>(a, s, joined);
    return hipGetLastError();
}

template <class T>
hipError_t run(const GroupNormArgs &a, bool back, hipStream_t stream) {
    if (back) return a.silu ? backward<T, true>(a, stream) : backward<T, false>(a, stream);
    return a.silu ? forward<T, true>(a, stream) : forward<T, false>(a, stream);
}

hipError_t run(oeq_dtype dtype, const GroupNormArgs &a, bool back, hipStream_t stream) {
    switch (dtype) {
        case OEQ_F32: return run<float>(a, back, stream);
        case OEQ_F16: return run<f16>(a, back, stream);
        case OEQ_BF16: return run<bf16>(a, back, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

GroupNormBytes group_norm_workspace(int64_t rows, int32_t n_struct, int32_t channels, int32_t groups) {
    if (rows == 0 || n_struct == 0) return {0, 0};
    const Pieces w = pieces_of(shape_of(rows, n_struct, channels, groups), n_struct, channels, groups);
    return {w.joined, w.bytes};
}

int64_t group_norm_blocks(int64_t rows, int32_t n_struct, int32_t channels, int32_t groups) {
    const Shape s = shape_of(rows, n_struct, channels, groups);
    return int64_t(n_struct) * s.splits * s.n_slabs;
}

hipError_t group_norm_fwd(oeq_dtype dtype, const GroupNormArgs &a, hipStream_t stream) {
    return run(dtype, a, false, stream);
}
hipError_t group_norm_bwd(oeq_dtype dtype, const GroupNormArgs &a, hipStream_t stream) {
    return run(dtype, a, true, stream);
}

}  // namespace readout
}  // namespace oeq
