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
// Everything here is bound by memory.  A workgroup owns (part of a structure's rows, slab of
// whole groups, about 64 channels): lanes run along the channels in pieces of eight, so a row of
// the slab is one 128- or 256-byte access, and the sums over the rows are each thread's own until
// one reduction at the end.  Structures of few rows on average are one part each, whose workgroup
// computes the sums and then applies them (the second read comes from its cache), at the pace of the
// longest; others are cut into tiles of rows, whose partial sums go through the workspace to a joining
// kernel, and a third one applies them.  Tiles are as long in every structure, so there the longest one sets
// no pace.  No atomics: every result is bitwise repeatable.
//
// 280000 x 256 in 32 uneven structures, bf16, SiLU (143 MB an operand): statistics 39 us, output 51
// (5.6 TB/s), gradient sums 69 (4.1 TB/s, the vector unit three quarters busy), grad_x 79 (5.5 TB/s);
// 100003 x 128, fp32: 13.0 and 17.9 us.  A few molecules are one kernel of 6 us, its loads' latency.
//
// Sums are fp32 in a wave and fp64 from there on.  A thread sums squares about its own first row and moves
// to the mean of what it has after 1, 2, 4, ... steps; threads and parts are joined by their means and squared
// deviations (Chan, Golub and LeVeque, "Updating formulae and a pairwise algorithm for computing sample
// variances", 1982).  So the variance cancels neither against a large mean nor against an outlier, wherever
// it is: with 7937 rows in one part, the first one 100 deviations off, rstd is 1e-7 off, and was 1.2e-4
// off by sums about the part's first row, at the same time.
#include <type_traits>

#include "readout.hpp"
#include "readout_device.hpp"

namespace oeq {
namespace readout {

namespace {

constexpr int kThreads = 256;
constexpr int kSlab = 64;         // channels of a slab, where a group is not wider
constexpr int kWholeRows = 128;   // rows of a structure, on average, up to which it is one part
constexpr int kStep = 4;          // rows a thread has under way
constexpr int kJoinChannels = 8;  // channels of a workgroup that sums the weights' gradients

struct Shape {
    int cg;         // channels of a group
    int gps;        // groups of a slab
    int n_slabs;
    int cols;       // threads along a slab's channels (a power of two)
    int tile;       // rows of a part; 0: a structure is one part
    int64_t parts;
};

// One part a structure is two launches fewer, but goes at the longest structure's pace (SiLU, fp32, forward
// and backward of 128 channels): 64 structures of 78 rows take 6.6 and 10.5 us, the like of 187 rows 8.4 and
// 13.3, against 14.1 and 18.5 in tiles; 64 structures of which one has 7937 of 8000 rows take 81 and 170, and
// would take the same 14 and 19 in tiles.  The host knows the average alone, and up to it even batches are the
// usual ones.
// The tile fills the chip once or twice over (forward and backward, fp32, 128 channels; work is two for a row):
// 3000 rows take 11.5 and 13.8 us with tiles of 64 rows, 13.1 and 17.4 with 256; 48000 take 25.1 and 33.9
// with 128, 24.0 and 32.3 with 256, 28.6 and 40.7 with 64; 80000 take 31.3 and 42.5 with 256, 32.2 and 46.4
// with 512; 160000 take 49.0 and 73.6 with 256, 48.3 and 71.4 with 512.
Shape shape_of(int64_t rows, int32_t n_struct, int32_t channels, int32_t groups) {
    Shape s;
    s.cg = channels / groups;
    s.gps = s.cg >= kSlab ? 1 : kSlab / s.cg;
    if (s.gps > groups) s.gps = groups;
    s.n_slabs = (groups + s.gps - 1) / s.gps;
    s.gps = (groups + s.n_slabs - 1) / s.n_slabs;
    s.cols = 1;
    while (s.cols * 8 < s.gps * s.cg) s.cols *= 2;
    s.tile = 0;
    s.parts = n_struct;
    if (rows > int64_t(kWholeRows) * n_struct) {
        const int64_t work = rows * s.n_slabs;
        s.tile = work <= 64 * 256 ? 64 : work <= 128 * 512 ? 128 : work <= 256 * 768 ? 256 : 512;
        s.parts = tile_slots(rows, n_struct, 1, s.tile);
    }
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
// begin + lane, begin + lane + lanes, ..., `count` of them, of its part.
struct Part {
    int b;  // the structure
    int64_t begin, end;
    int c, n, lane, lanes, count, c0, width, g0, n_groups;
};

// kTiled: part `i` is a slot of the tiling, which may be past its structure's rows (no rows then).
template <bool kTiled>
__device__ __forceinline__ Part part_of(const GroupNormArgs &a, const Shape &s, int i, int slab) {
    Part p;
    if (kTiled) {
        const Owner w = find_structure(a.ptr, a.ptr, a.n_struct, 1, s.tile, i);
        const Span rows = span_of(w.ptr[0], w.ptr[1], a.rows);
        const int64_t at = rows.begin + (i - w.first) * s.tile;
        p.b = w.index;
        p.begin = at < rows.begin || at > rows.end ? rows.end : at;
        p.end = p.begin + s.tile < rows.end ? p.begin + s.tile : rows.end;
    } else {
        const Span rows = span_of(a.ptr, i, a.rows);
        p.b = i;
        p.begin = rows.begin;
        p.end = rows.end;
    }
    p.g0 = slab * s.gps;
    p.n_groups = a.groups - p.g0 < s.gps ? a.groups - p.g0 : s.gps;
    p.c0 = p.g0 * s.cg;
    p.width = p.n_groups * s.cg;
    const int col = threadIdx.x & (s.cols - 1);
    p.c = p.c0 + col * 8;
    p.n = p.width - col * 8 < 8 ? p.width - col * 8 : 8;
    p.lane = threadIdx.x / s.cols;
    p.lanes = kThreads / s.cols;
    p.count = p.n > 0 ? (static_cast<int>(p.end - p.begin) - p.lane + p.lanes - 1) / p.lanes : 0;
    return p;
}

// A thread's rows of one operand, kStep at a time.  kFull: every piece has all eight channels.
template <class T, bool kFull>
struct Walk {
    T *at;
    int64_t stride;
    int n;
    __device__ __forceinline__ Walk(const void *base, int64_t ld, const Part &p)
        : at(static_cast<T *>(const_cast<void *>(base)) + (p.begin + p.lane) * ld + p.c), stride(p.lanes * ld), n(p.n) {}
    // All loads of a step are issued together; in place of rows past the `left` ones the first is
    // read, and its value not used.
    __device__ __forceinline__ void load(vec8<T> (&v)[kStep], int left) const {
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
            const T *q = at + (i < left ? i * stride : 0);
            v[i] = kFull || n == 8 ? load8(q) : load_part(q, n);
        }
    }
    __device__ __forceinline__ void store(int i, f32x8 v) const {
        T *q = at + i * stride;
        const vec8<T> o = from_f32<T>(v);
        if (kFull || n == 8)
            store8(q, o);
        else
            store_part(q, o, n);
    }
    __device__ __forceinline__ void next() { at += kStep * stride; }
};

__device__ __forceinline__ f32x8 channel_values(const float *v, const Part &p, float without) {
    f32x8 o;
    if (v && p.n == 8) return load8(v + p.c);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = v && j < p.n ? v[p.c + j] : without;
    return o;
}

// f(j, group) for the thread's channels; channel c is the first of them, counted from the
// first channel of the first group.
template <class F>
__device__ __forceinline__ void each_group(const Part &p, const Shape &s, int c, F &&f) {
    if (p.n <= 0) return;
    int g = c / s.cg, in = c - g * s.cg;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j < p.n) f(j, g);
        if (++in == s.cg) {
            in = 0;
            ++g;
        }
    }
}

// Two sums per channel of all threads' rows: every thread leaves its own with those of the
// other row lanes of its wave, by set of waves that hold the same channels; channel_total
// adds the sets.
// For statistics they are not sums but the mean, from the part's first row on, and the squared deviations.
struct Sums {
    float v[2][kThreads * 8];
    float first[kThreads * 8], rows[kThreads / 64];  // statistics: the part's first row, the rows of each set
    int cols, sets;
    __device__ __forceinline__ double total(int which, int c) const {
        double t = v[which][c];
        for (int k = 1; k < sets; ++k) t += v[which][k * cols * 8 + c];
        return t;
    }
    // The mean and the squared deviations of channel c over all n rows.
    __device__ __forceinline__ double mean(int c, double n) const {
        double t = 0;
        for (int k = 0; k < sets; ++k) t += double(rows[k]) * v[0][k * cols * 8 + c];
        return t / n;
    }
    __device__ __forceinline__ double squares(int c, double mean) const {
        double t = 0;
        for (int k = 0; k < sets; ++k) {
            const double off = v[0][k * cols * 8 + c] - mean;
            t += v[1][k * cols * 8 + c] + double(rows[k]) * off * off;
        }
        return t;
    }
};
__device__ __forceinline__ void leave_in(Sums &sums, f32x8 u, f32x8 v, float rows, const Part &p, int cols) {
    const int per_set = cols > 64 ? cols / 64 : 1, wave = threadIdx.x >> 6;
    const int col = threadIdx.x & (cols - 1), set = wave / per_set;
    if (p.lane % (cols < 64 ? 64 / cols : 1) == 0 && p.n > 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sums.v[0][set * cols * 8 + col * 8 + j] = u[j];
            sums.v[1][set * cols * 8 + col * 8 + j] = v[j];
        }
        if (col == 0) sums.rows[set] = rows;
    }
    if (threadIdx.x == 0) {
        sums.cols = cols;
        sums.sets = kThreads / 64 / per_set;
    }
    __syncthreads();
}
__device__ __forceinline__ void channel_sums(f32x8 u, f32x8 v, const Part &p, int cols, Sums &sums) {
    for (int off = cols; off < 64; off <<= 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            u[j] += __shfl_xor(u[j], off);
            v[j] += __shfl_xor(v[j], off);
        }
    }
    leave_in(sums, u, v, 0.f, p, cols);
}
// The same of a thread's means and squared deviations over its p.count rows.
__device__ __forceinline__ void channel_moments(f32x8 mean, f32x8 squares, const Part &p, int cols, Sums &sums) {
    float n = static_cast<float>(p.count);
    for (int off = cols; off < 64; off <<= 1) {
        const float m = __shfl_xor(n, off), share = m > 0.f ? m * __builtin_amdgcn_rcpf(n + m) : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float apart = __shfl_xor(mean[j], off) - mean[j];
            squares[j] += __shfl_xor(squares[j], off) + apart * apart * (n * share);
            mean[j] += apart * share;
        }
        n += m;
    }
    leave_in(sums, mean, squares, n, p, cols);
}

// Groups of the slab, several a wave: `group` is -1 for lanes without one, `lane` the lane
// within the group's `lanes` (a power of two), which step through its channels.
struct GroupLanes {
    int lanes, lane, at;
    __device__ __forceinline__ explicit GroupLanes(int cg) {
        lanes = 1;
        while (lanes < cg && lanes < 64) lanes <<= 1;
        lane = threadIdx.x & (lanes - 1);
        at = threadIdx.x / lanes;
    }
    __device__ __forceinline__ int step() const { return kThreads / lanes; }
    __device__ __forceinline__ double sum(double v) const {
        for (int off = lanes >> 1; off > 0; off >>= 1) v += __shfl_xor(v, off);
        return v;
    }
};

__device__ __forceinline__ float rstd_of(double m2, double n, float eps) {
    if (!(n > 0)) return 0.f;
    const double var = m2 > 0 || !(m2 == m2) ? m2 / n : 0;  // rounding can leave a small negative sum
    // A Newton step; rsq(inf) is 0 already.  rsq takes what is below the normal numbers for zero (1e-40 is
    // an eps too), so small values go through it times 2^64.
    const double sum = var + double(eps);
    const bool small = sum < 0x1p-96;
    const float v = static_cast<float>(small ? sum * 0x1p64 : sum), r = __builtin_amdgcn_rsqf(v);
    return v < INFINITY ? r * fmaf(-0.5f * v * r, r, 1.5f) * (small ? 0x1p32f : 1.f) : r;
}

// Statistics of each group of the slab over the part's rows; emit(group of the slab, mean, sum
// of squared deviations) is called by one lane for each.  The part's first rows stay in `held`.
template <class T, bool kFull, class Emit>
__device__ __forceinline__ void statistics(const GroupNormArgs &a, const Shape &s, const Part &p, vec8<T> (&held)[kStep],
                                           Sums &sums, Emit &&emit) {
    const int64_t n = p.end - p.begin;
    f32x8 mean = {}, squares = {};
    if (p.count > 0) {
        Walk<T, kFull> x(a.x, a.ld_x, p);
        x.load(held, p.count);
        const T *first_row = static_cast<const T *>(a.x) + p.begin * a.ld_x + p.c;
        const f32x8 first = to_f32<T>(kFull || p.n == 8 ? load8(first_row) : load_part(first_row, p.n));
        f32x8 shift = to_f32<T>(held[0]), u = {}, v = {};  // sums of x - shift and its square
        const auto add = [&](const vec8<T>(&rows)[kStep], int left) {
#pragma unroll
            for (int i = 0; i < kStep; ++i) {
                if (i < left) {
                    const f32x8 d = to_f32<T>(rows[i]) - shift;
                    u += d;
                    v += d * d;
                }
            }
        };
        if (p.lane == 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) sums.first[p.c - p.c0 + j] = first[j];
        }
        add(held, p.count);
        int steps = 1;
        for (int left = p.count - kStep; left > 0; left -= kStep, ++steps) {
            vec8<T> rows[kStep];
            x.next();
            x.load(rows, left);
            if ((steps & (steps - 1)) == 0) {  // to the mean so far
                const float so_far = static_cast<float>(steps * kStep);
                const f32x8 to = shift + u * __builtin_amdgcn_rcpf(so_far), moved = to - shift;
                v -= moved * (2.f * u - so_far * moved);
                u -= so_far * moved;
                shift = to;
            }
            add(rows, left);
        }
        const f32x8 off = u * __builtin_amdgcn_rcpf(static_cast<float>(p.count));
        mean = (shift - first) + off;
        squares = v - u * off;
    }
    channel_moments(mean, squares, p, s.cols, sums);
    const GroupLanes gl(s.cg);
    for (int g = gl.at; g < (p.n_groups + gl.step() - 1) / gl.step() * gl.step(); g += gl.step()) {
        double mean = 0, m2 = 0;
        if (g < p.n_groups && n > 0) {
            const int c0 = g * s.cg;
            for (int c = gl.lane; c < s.cg; c += gl.lanes) mean += double(sums.first[c0 + c]) + sums.mean(c0 + c, double(n));
            mean = gl.sum(mean) / s.cg;
            for (int c = gl.lane; c < s.cg; c += gl.lanes) {
                const double of_channel = sums.mean(c0 + c, double(n));
                const double off = double(sums.first[c0 + c]) + of_channel - mean;
                m2 += sums.squares(c0 + c, of_channel) + double(n) * off * off;
            }
            m2 = gl.sum(m2);
        }
        if (gl.lane == 0 && g < p.n_groups) emit(g, mean, m2);
    }
}

// out of a part's rows; the first are in `held`.
template <class T, bool kFull, bool kSilu>
__device__ __forceinline__ void apply_forward(const GroupNormArgs &a, const Part &p, const vec8<T> (&held)[kStep],
                                              f32x8 mean, f32x8 w, f32x8 bias) {
    if (p.count <= 0) return;
    Walk<T, kFull> x(a.x, a.ld_x, p), out(a.out, a.ld_out, p);
    const auto apply = [&](const vec8<T>(&rows)[kStep], int left) {
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
            if (i < left) {
                f32x8 z = (to_f32<T>(rows[i]) - mean) * w + bias;
                if (kSilu) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[j] *= sigmoid(z[j]);
                }
                out.store(i, z);
            }
        }
    };
    apply(held, p.count);
    for (int left = p.count - kStep; left > 0; left -= kStep) {
        vec8<T> rows[kStep];
        x.next();
        out.next();
        x.load(rows, left);
        apply(rows, left);
    }
}

// One part a structure: statistics and output in one launch.
template <class T, bool kFull, bool kSilu>
__global__ void __launch_bounds__(kThreads) k_forward(GroupNormArgs a, Shape s) {
    __shared__ Sums sums;
    __shared__ float group_mean[kSlab], group_rstd[kSlab];
    const int b = blockIdx.x / s.n_slabs;
    const Part p = part_of<false>(a, s, b, blockIdx.x - b * s.n_slabs);
    f32x8 w = channel_values(a.weight, p, 1.f), bias = channel_values(a.bias, p, 0.f), mean = {};
    vec8<T> held[kStep];
    const double n = double(p.end - p.begin) * s.cg;
    statistics<T, kFull>(a, s, p, held, sums, [&](int g, double group, double m2) {
        const float rstd = rstd_of(m2, n, a.eps);
        group_mean[g] = static_cast<float>(group);
        group_rstd[g] = rstd;
        const int64_t at = int64_t(b) * a.groups + p.g0 + g;
        a.mean[at] = static_cast<float>(group);
        a.rstd[at] = rstd;
    });
    __syncthreads();
    each_group(p, s, p.c - p.c0, [&](int j, int g) {
        mean[j] = group_mean[g];
        w[j] *= group_rstd[g];
    });
    apply_forward<T, kFull, kSilu>(a, p, held, mean, w, bias);
}

// Tiles of structures.  partial[(part, group)] = {mean, sum of squared deviations}
template <class T, bool kFull>
__global__ void __launch_bounds__(kThreads) k_statistics(GroupNormArgs a, Shape s, double2 *partial) {
    __shared__ Sums sums;
    const int part = blockIdx.x / s.n_slabs;
    const Part p = part_of<true>(a, s, part, blockIdx.x - part * s.n_slabs);
    vec8<T> held[kStep];
    statistics<T, kFull>(a, s, p, held, sums, [&](int g, double mean, double m2) {
        partial[int64_t(part) * a.groups + p.g0 + g] = make_double2(mean, m2);
    });
}

// The parts of structure b: `first` and the `count` from there on, all but the last of tile rows.
struct Parts {
    int64_t first, count, rows;
    __device__ __forceinline__ Parts(const GroupNormArgs &a, const Shape &s, int b) {
        const Span span = span_of(a.ptr, b, a.rows);
        first = int64_t(a.ptr[b]) / s.tile + b;
        rows = span.end - span.begin;
        count = (rows + s.tile - 1) / s.tile;
        if (first < 0 || first + count > s.parts) count = 0;  // a row pointer that is none
    }
    __device__ __forceinline__ double rows_of(const Shape &s, int64_t i) const {
        return double(i + 1 < count ? int64_t(s.tile) : rows - i * s.tile);
    }
};

// One wave joins the parts of one (structure, group).
__global__ void __launch_bounds__(kThreads) k_join_statistics(GroupNormArgs a, Shape s, const double2 *partial) {
    const int64_t at = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (at >= int64_t(a.n_struct) * a.groups) return;
    const int b = static_cast<int>(at / a.groups), g = static_cast<int>(at % a.groups), lane = threadIdx.x & 63;
    const Parts parts(a, s, b);
    const double2 *from = partial + parts.first * a.groups + g;
    const double n = double(parts.rows);
    constexpr int kHeld = 4;  // parts a lane keeps from the first walk for the second
    double2 v[kHeld];
    double mean = 0, m2 = 0;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) v[j] = lane + 64 * j < parts.count ? from[(lane + 64 * j) * a.groups] : make_double2(0, 0);
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        if (lane + 64 * j < parts.count) mean += parts.rows_of(s, lane + 64 * j) * v[j].x;
    }
    for (int64_t i = lane + 64 * kHeld; i < parts.count; i += 64) mean += parts.rows_of(s, i) * from[i * a.groups].x;
    mean = n > 0 ? wave_sum(mean) / n : 0;
    const auto add = [&](int64_t i, double2 part) {
        const double off = part.x - mean;
        m2 += part.y + parts.rows_of(s, i) * s.cg * off * off;
    };
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        if (lane + 64 * j < parts.count) add(lane + 64 * j, v[j]);
    }
    for (int64_t i = lane + 64 * kHeld; i < parts.count; i += 64) add(i, from[i * a.groups]);
    m2 = wave_sum(m2);
    if (lane == 0) {
        a.mean[at] = static_cast<float>(mean);
        a.rstd[at] = rstd_of(m2, n * s.cg, a.eps);
    }
}

__device__ __forceinline__ void saved_statistics(const GroupNormArgs &a, const Shape &s, const Part &p, f32x8 *mean,
                                                 f32x8 *rstd) {
    *mean = f32x8{};
    *rstd = f32x8{};
    each_group(p, s, p.c, [&](int j, int g) {
        const int64_t at = int64_t(p.b) * a.groups + g;
        (*mean)[j] = a.mean[at];
        (*rstd)[j] = a.rstd[at];
    });
}

// The second pass over the rows takes the parts in the other order: what the first read last is
// still in the last-level cache (bf16 training step of 280000 x 256, 143 MB an operand: 261 -> 248 us, 240 in tiles).
__device__ __forceinline__ int from_last() { return static_cast<int>(gridDim.x - 1 - blockIdx.x); }

template <class T, bool kFull, bool kSilu>
__global__ void __launch_bounds__(kThreads) k_apply(GroupNormArgs a, Shape s) {
    const int block = from_last(), part = block / s.n_slabs;
    const Part p = part_of<true>(a, s, part, block - part * s.n_slabs);
    f32x8 mean, rstd;
    vec8<T> held[kStep];
    if (p.count > 0) Walk<T, kFull>(a.x, a.ld_x, p).load(held, p.count);
    saved_statistics(a, s, p, &mean, &rstd);
    const f32x8 w = channel_values(a.weight, p, 1.f) * rstd, bias = channel_values(a.bias, p, 0.f);
    apply_forward<T, kFull, kSilu>(a, p, held, mean, w, bias);
}

// ---- backward -----------------------------------------------------------------------

// What a thread needs of its channels; z = (x - mean) scale + bias with scale = rstd w.
struct Channels {
    f32x8 mean, rstd, scale, bias;
    __device__ __forceinline__ Channels(const GroupNormArgs &a, const Shape &s, const Part &p) {
        saved_statistics(a, s, p, &mean, &rstd);
        scale = channel_values(a.weight, p, 1.f) * rstd;
        bias = channel_values(a.bias, p, 0.f);
    }
    // x - mean and dz of one row
    template <class T, bool kSilu>
    __device__ __forceinline__ void local(vec8<T> x, vec8<T> g, f32x8 *centred, f32x8 *dz) const {
        const f32x8 xc = to_f32<T>(x) - mean;
        f32x8 d = to_f32<T>(g);
        if (kSilu) {
            const f32x8 z = xc * scale + bias;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float gate = sigmoid(z[j]);
                d[j] *= fmaf(z[j] * gate, 1.f - gate, gate);
            }
        }
        *centred = xc;
        *dz = d;
    }
};

// Sums of a part's dz and dz xhat by channel (to `column`, unless NULL: row `part` of two
// fp32 rows of C channels) and, weighted, by group (to emit, as in statistics).  The part's
// first rows stay in hx and hg.
template <class T, bool kFull, bool kSilu, class Emit>
__device__ __forceinline__ void gradient_sums(const GroupNormArgs &a, const Shape &s, const Part &p, int64_t part,
                                              const Channels &ch, vec8<T> (&hx)[kStep], vec8<T> (&hg)[kStep],
                                              float *column, Sums &sums, Emit &&emit) {
    f32x8 u = {}, v = {};
    if (p.count > 0) {
        Walk<T, kFull> x(a.x, a.ld_x, p), g(a.grad_out, a.ld_grad_out, p);
        const auto add = [&](const vec8<T>(&rx)[kStep], const vec8<T>(&rg)[kStep], int left) {
#pragma unroll
            for (int i = 0; i < kStep; ++i) {
                if (i < left) {
                    f32x8 xc, dz;
                    ch.local<T, kSilu>(rx[i], rg[i], &xc, &dz);
                    u += dz;
                    v += dz * xc;
                }
            }
        };
        add(hx, hg, p.count);
        for (int left = p.count - kStep; left > 0; left -= kStep) {
            vec8<T> rx[kStep], rg[kStep];
            x.next();
            g.next();
            x.load(rx, left);
            g.load(rg, left);
            add(rx, rg, left);
        }
        v *= ch.rstd;
    }
    channel_sums(u, v, p, s.cols, sums);
    if (column) {
        for (int c = threadIdx.x; c < p.width; c += kThreads) {
            column[part * 2 * a.channels + p.c0 + c] = static_cast<float>(sums.total(0, c));
            column[(part * 2 + 1) * a.channels + p.c0 + c] = static_cast<float>(sums.total(1, c));
        }
    }
    const GroupLanes gl(s.cg);
    for (int g = gl.at; g < (p.n_groups + gl.step() - 1) / gl.step() * gl.step(); g += gl.step()) {
        double dh = 0, dhx = 0;
        if (g < p.n_groups) {
            for (int c = gl.lane; c < s.cg; c += gl.lanes) {
                const double wc = a.weight ? a.weight[p.c0 + g * s.cg + c] : 1.f;
                dh += wc * sums.total(0, g * s.cg + c);
                dhx += wc * sums.total(1, g * s.cg + c);
            }
            dh = gl.sum(dh);
            dhx = gl.sum(dhx);
        }
        if (gl.lane == 0 && g < p.n_groups) emit(g, dh, dhx);
    }
}

// grad_x = scale dz - rstd m1 - (x - mean) rstd^2 m2
template <class T, bool kFull, bool kSilu>
__device__ __forceinline__ void apply_backward(const GroupNormArgs &a, const Part &p, const Channels &ch,
                                               const vec8<T> (&hx)[kStep], const vec8<T> (&hg)[kStep], f32x8 m1, f32x8 m2) {
    if (p.count <= 0) return;
    Walk<T, kFull> x(a.x, a.ld_x, p), g(a.grad_out, a.ld_grad_out, p), out(a.grad_x, a.ld_grad_x, p);
    const f32x8 k1 = ch.rstd * m1, k2 = ch.rstd * (ch.rstd * m2);
    const auto apply = [&](const vec8<T>(&rx)[kStep], const vec8<T>(&rg)[kStep], int left) {
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
            if (i < left) {
                f32x8 xc, dz;
                ch.local<T, kSilu>(rx[i], rg[i], &xc, &dz);
                out.store(i, dz * ch.scale - k1 - xc * k2);
            }
        }
    };
    apply(hx, hg, p.count);
    for (int left = p.count - kStep; left > 0; left -= kStep) {
        vec8<T> rx[kStep], rg[kStep];
        x.next();
        g.next();
        out.next();
        x.load(rx, left);
        g.load(rg, left);
        apply(rx, rg, left);
    }
}

template <class T, bool kFull>
__device__ __forceinline__ void hold(const GroupNormArgs &a, const Part &p, vec8<T> (&hx)[kStep], vec8<T> (&hg)[kStep]) {
    if (p.count <= 0) return;
    Walk<T, kFull>(a.x, a.ld_x, p).load(hx, p.count);
    Walk<T, kFull>(a.grad_out, a.ld_grad_out, p).load(hg, p.count);
}

template <class T, bool kFull, bool kSilu>
__global__ void __launch_bounds__(kThreads) k_backward(GroupNormArgs a, Shape s, float *column) {
    __shared__ Sums sums;
    __shared__ float group_m1[kSlab], group_m2[kSlab];
    const int b = blockIdx.x / s.n_slabs;
    const Part p = part_of<false>(a, s, b, blockIdx.x - b * s.n_slabs);
    vec8<T> hx[kStep], hg[kStep];
    hold<T, kFull>(a, p, hx, hg);
    const Channels ch(a, s, p);
    const double n = double(p.end - p.begin) * s.cg;
    gradient_sums<T, kFull, kSilu>(a, s, p, b, ch, hx, hg, column, sums, [&](int g, double dh, double dhx) {
        group_m1[g] = n > 0 ? static_cast<float>(dh / n) : 0.f;
        group_m2[g] = n > 0 ? static_cast<float>(dhx / n) : 0.f;
    });
    if (!a.grad_x) return;
    __syncthreads();
    f32x8 m1 = {}, m2 = {};
    each_group(p, s, p.c - p.c0, [&](int j, int g) {
        m1[j] = group_m1[g];
        m2[j] = group_m2[g];
    });
    apply_backward<T, kFull, kSilu>(a, p, ch, hx, hg, m1, m2);
}

template <class T, bool kFull, bool kSilu>
__global__ void __launch_bounds__(kThreads) k_gradient_sums(GroupNormArgs a, Shape s, float *column, double2 *partial) {
    __shared__ Sums sums;
    const int part = blockIdx.x / s.n_slabs;
    const Part p = part_of<true>(a, s, part, blockIdx.x - part * s.n_slabs);
    vec8<T> hx[kStep], hg[kStep];
    hold<T, kFull>(a, p, hx, hg);
    const Channels ch(a, s, p);
    gradient_sums<T, kFull, kSilu>(a, s, p, part, ch, hx, hg, column, sums, [&](int g, double dh, double dhx) {
        partial[int64_t(part) * a.groups + p.g0 + g] = make_double2(dh, dhx);
    });
}

// The first `by_group` workgroups join the parts' group sums to means (one wave a
// (structure, group)); the others sum `column` over its rows, kJoinChannels a workgroup.
__global__ void __launch_bounds__(kThreads) k_join_gradients(GroupNormArgs a, Shape s, const double2 *partial,
                                                             float2 *joined, const float *column, int by_group) {
    if (static_cast<int>(blockIdx.x) < by_group) {
        const int64_t at = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
        if (at >= int64_t(a.n_struct) * a.groups) return;
        const int b = static_cast<int>(at / a.groups), g = static_cast<int>(at % a.groups), lane = threadIdx.x & 63;
        const Parts parts(a, s, b);
        const double n = double(parts.rows) * s.cg;
        double u = 0, v = 0;
        for (int64_t i = lane; i < parts.count; i += 64) {
            const double2 t = partial[(parts.first + i) * a.groups + g];
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
    constexpr int kLanes = kThreads / kJoinChannels, kAhead = 8;
    const int col = threadIdx.x % kJoinChannels, lane = threadIdx.x / kJoinChannels;
    const int c = (blockIdx.x - by_group) * kJoinChannels + col;
    const int n_parts = static_cast<int>(s.parts);
    double u = 0, v = 0;
    if (c < a.channels) {
        for (int r = lane; r < n_parts; r += kLanes * kAhead) {
            float x[kAhead], y[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int64_t at = r + i * kLanes < n_parts ? r + i * kLanes : r;
                x[i] = column[at * 2 * a.channels + c];
                y[i] = column[(at * 2 + 1) * a.channels + c];
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (r + i * kLanes < n_parts) {
                    u += x[i];
                    v += y[i];
                }
            }
        }
    }
    part[0][threadIdx.x] = u;
    part[1][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x < kJoinChannels && c < a.channels) {
        for (int k = 1; k < kLanes; ++k) {
            u += part[0][k * kJoinChannels + col];
            v += part[1][k * kJoinChannels + col];
        }
        if (a.grad_bias) a.grad_bias[c] = static_cast<float>(u);
        if (a.grad_weight) a.grad_weight[c] = static_cast<float>(v);
    }
}

template <class T, bool kFull, bool kSilu>
__global__ void __launch_bounds__(kThreads) k_apply_backward(GroupNormArgs a, Shape s, const float2 *joined) {
    const int block = from_last(), part = block / s.n_slabs;
    const Part p = part_of<true>(a, s, part, block - part * s.n_slabs);
    vec8<T> hx[kStep], hg[kStep];
    hold<T, kFull>(a, p, hx, hg);
    const Channels ch(a, s, p);
    f32x8 m1 = {}, m2 = {};
    each_group(p, s, p.c, [&](int j, int g) {
        const float2 t = joined[int64_t(p.b) * a.groups + g];
        m1[j] = t.x;
        m2[j] = t.y;
    });
    apply_backward<T, kFull, kSilu>(a, p, ch, hx, hg, m1, m2);
}

constexpr size_t up(size_t v) { return (v + 255) / 256 * 256; }

// Workspace pieces: the parts' group sums, the joined means of the backward, the channel sums.
struct Pieces {
    size_t partial, joined, column, bytes;
};
Pieces pieces_of(const Shape &s, int32_t n_struct, int32_t channels, int32_t groups) {
    Pieces w;
    const size_t parts = static_cast<size_t>(s.parts);
    w.partial = 0;
    w.joined = w.partial + (s.tile ? up(parts * groups * sizeof(double2)) : 0);
    w.column = w.joined + (s.tile ? up(static_cast<size_t>(n_struct) * groups * sizeof(float2)) : 0);
    w.bytes = w.column + up(parts * channels * 2 * sizeof(float));
    return w;
}

// Workgroups of the joining kernels: one wave a (structure, group), and kJoinChannels channels.
int64_t join_blocks(int32_t n_struct, int32_t groups) { return (int64_t(n_struct) * groups + 3) / 4; }
int64_t channel_blocks(int32_t channels) { return (int64_t(channels) + kJoinChannels - 1) / kJoinChannels; }

template <class T, bool kFull, bool kSilu>
hipError_t forward(const GroupNormArgs &a, hipStream_t stream) {
    const Shape s = shape_of(a.rows, a.n_struct, a.channels, a.groups);
    const dim3 grid(static_cast<unsigned>(s.parts * s.n_slabs)), threads(kThreads);
    if (!s.tile) {
        k_forward<T, kFull, kSilu><<<grid, threads, 0, stream>>>(a, s);
        return hipGetLastError();
    }
    double2 *partial = static_cast<double2 *>(a.workspace);
    k_statistics<T, kFull><<<grid, threads, 0, stream>>>(a, s, partial);
    const dim3 join(static_cast<unsigned>(join_blocks(a.n_struct, a.groups)));
    k_join_statistics<<<join, threads, 0, stream>>>(a, s, partial);
    k_apply<T, kFull, kSilu><<<grid, threads, 0, stream>>>(a, s);
    return hipGetLastError();
}

template <class T, bool kFull, bool kSilu>
hipError_t backward(const GroupNormArgs &a, hipStream_t stream) {
    const bool params = a.grad_weight || a.grad_bias;
    const int by_channel = params ? static_cast<int>(channel_blocks(a.channels)) : 0;
    const dim3 threads(kThreads);
    if (a.rows == 0 || a.n_struct == 0) {  // no parts: zeros
        if (params)
            k_join_gradients<<<dim3(by_channel), threads, 0, stream>>>(a, Shape{}, nullptr, nullptr, nullptr, 0);
        return hipGetLastError();
    }
    const Shape s = shape_of(a.rows, a.n_struct, a.channels, a.groups);
    const Pieces w = pieces_of(s, a.n_struct, a.channels, a.groups);
    char *ws = static_cast<char *>(a.workspace);
    double2 *partial = reinterpret_cast<double2 *>(ws + w.partial);
    float2 *joined = reinterpret_cast<float2 *>(ws + w.joined);
    float *column = params ? reinterpret_cast<float *>(ws + w.column) : nullptr;
    const dim3 grid(static_cast<unsigned>(s.parts * s.n_slabs));
    if (!s.tile) {
        k_backward<T, kFull, kSilu><<<grid, threads, 0, stream>>>(a, s, column);
        if (params) k_join_gradients<<<dim3(by_channel), threads, 0, stream>>>(a, s, partial, joined, column, 0);
        return hipGetLastError();
    }
    k_gradient_sums<T, kFull, kSilu><<<grid, threads, 0, stream>>>(a, s, column, partial);
    const int by_group = a.grad_x ? static_cast<int>(join_blocks(a.n_struct, a.groups)) : 0;
    k_join_gradients<<<dim3(by_group + by_channel), threads, 0, stream>>>(a, s, partial, joined, column, by_group);
    if (a.grad_x) k_apply_backward<T, kFull, kSilu><<<grid, threads, 0, stream>>>(a, s, joined);
    return hipGetLastError();
}

template <class T, bool kFull>
hipError_t run(const GroupNormArgs &a, bool back, hipStream_t stream) {
    if (back) return a.silu ? backward<T, kFull, true>(a, stream) : backward<T, kFull, false>(a, stream);
    return a.silu ? forward<T, kFull, true>(a, stream) : forward<T, kFull, false>(a, stream);
}

template <class T>
hipError_t run(const GroupNormArgs &a, bool back, hipStream_t stream) {
    // whether every slab's channels come in whole pieces of eight
    const int gps = a.n_struct && a.rows ? shape_of(a.rows, a.n_struct, a.channels, a.groups).gps : 1;
    const bool full = a.channels % 8 == 0 && gps * (a.channels / a.groups) % 8 == 0;
    return full ? run<T, true>(a, back, stream) : run<T, false>(a, back, stream);
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
    const int64_t main = s.parts * s.n_slabs;
    const int64_t join = (s.tile ? join_blocks(n_struct, groups) : 0) + channel_blocks(channels);
    return main > join ? main : join;
}

hipError_t group_norm_fwd(oeq_dtype dtype, const GroupNormArgs &a, hipStream_t stream) {
    return run(dtype, a, false, stream);
}
hipError_t group_norm_bwd(oeq_dtype dtype, const GroupNormArgs &a, hipStream_t stream) {
    return run(dtype, a, true, stream);
}

}  // namespace readout
}  // namespace oeq
