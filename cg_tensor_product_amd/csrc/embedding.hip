// Embedding lookup with scaling, and its gradient by sorted indices.
//   out[i] = scale table[index[i]]          grad_table[t] = scale sum_{i: index[i] = t} grad_out[i]
// An index outside the table gives a row of zeros and takes no gradient.
//
// The lookup is a copy of rows: a thread takes eight columns of one.
//
// The gradient's sums have no atomics.  (index, position) pairs are sorted by index with the positions of
// one index in increasing order (a stable radix sort), the sorted list is cut into chunks of equal
// length, and a few lanes walk each chunk, their columns in registers, and write a table row where
// its run of equal indices ends.  So neither a common index (thousands of uses of one species) nor
// many rare ones (a vocabulary) leave lanes idle.  A run that a cut divides leaves a partial sum a
// chunk, and a second kernel adds those in order.  Rows that no index names are zeroed by workgroups
// of the sorting launches, and tables of few rows need no sort (k_small).
//
// Bound by HBM where there is enough to move: the lookup writes 280000 rows of 256 columns, bf16, in 27.2 us (143 MB,
// 5.3 TB/s), k_small reads as much in 33.8 us (4.2 TB/s).  A vocabulary's gradient (16384 uses of 1024 columns, 32000
// rows, bf16: 100 MB, 19 us at that rate) takes 52 us in six launches: 5.9 and 8.7 us for each of two
// sorting passes, in which the 65 MB of the table are zeroed, 13.4 for the sums and 8.9 for the runs that cuts divide.
#include <algorithm>
#include <type_traits>

#include "readout.hpp"
#include "readout_device.hpp"

namespace oeq {
namespace readout {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kNone = ~0u;

template <class T>
__device__ __forceinline__ vec8<T> load_cols(const T *p, int n) {
    return n >= 8 ? load8(p) : load_part(p, n);
}
template <class T>
__device__ __forceinline__ void store_cols(T *p, vec8<T> v, int n) {
    if (n >= 8)
        store8(p, v);
    else
        store_part(p, v, n);
}

// The table row that index i names, or `none`.  A 64-bit index is read as two words and both widths take
// the same loads, without a branch: a value that comes by two ways is waited for where they meet,
// and no two loads of a thread would overlap.
__device__ __forceinline__ uint32_t index_at(const EmbeddingArgs &a, int64_t i, uint32_t none) {
    const uint32_t *at = static_cast<const uint32_t *>(a.index) + (i << a.wide);
    const uint32_t low = at[0], high = at[a.wide] & (a.wide ? ~0u : 0u);
    return (low < static_cast<uint32_t>(a.table_rows)) & (high == 0) ? low : none;
}

// The first n of eight (or kW) columns, 0 < n; the others are zero.  All loads are made, as above.
template <class Vec, class T>
__device__ __forceinline__ Vec load_first(const T *p, int n) {
    constexpr int kW = sizeof(Vec) / sizeof(T);
    Vec v;
#pragma unroll
    for (int k = 0; k < kW; ++k) {
        const T x = p[min(k, n - 1)];
        v[k] = k < n ? x : T(0.f);
    }
    return v;
}

// ---- lookup ---------------------------------------------------------------------------

template <class T, class Index>
__global__ void __launch_bounds__(kThreads) k_lookup(EmbeddingArgs a, uint32_t per_row) {
    const Index total = static_cast<Index>(a.rows) * per_row, step = Index(gridDim.x) * kThreads;
    for (Index i = Index(blockIdx.x) * kThreads + threadIdx.x; i < total; i += step) {
        const Index row = i / per_row;
        const int64_t col = int64_t(i - row * per_row) * 8;
        const int n = static_cast<int>(min(a.cols - col, int64_t(8)));
        const uint32_t t = index_at(a, static_cast<int64_t>(row), kNone);
        f32x8 v = {};
        if (t != kNone) v = to_f32<T>(load_cols(static_cast<const T *>(a.table) + t * a.ld_table + col, n)) * a.scale;
        store_cols(static_cast<T *>(a.out) + static_cast<int64_t>(row) * a.ld_out + col, from_f32<T>(v), n);
        if (total - i <= step) break;  // before i + step can wrap
    }
}

template <class T>
hipError_t lookup(const EmbeddingArgs &a, hipStream_t stream) {
    const int64_t per_row = (a.cols + 7) / 8, total = a.rows * per_row;
    const int64_t grid = std::min<int64_t>((total + kThreads - 1) / kThreads, 1 << 23);  // fewer than 2^32 threads
    const dim3 blocks(static_cast<unsigned>(grid)), threads(kThreads);
    if (total >> 32)
        k_lookup<T, uint64_t><<<blocks, threads, 0, stream>>>(a, static_cast<uint32_t>(per_row));
    else
        k_lookup<T, uint32_t><<<blocks, threads, 0, stream>>>(a, static_cast<uint32_t>(per_row));
    return hipGetLastError();
}

// Zeroing of table rows [begin, end) by `blocks` workgroups of kIn threads, of which this is number `block`.
template <class T, int kIn>
__device__ __forceinline__ void zero_rows(const EmbeddingArgs &a, int64_t begin, int64_t end, int64_t block, int64_t blocks) {
    const uint32_t per_row = static_cast<uint32_t>((a.cols + 7) / 8);
    const int64_t n = (end - begin) * per_row;
    for (int64_t i = block * kIn + threadIdx.x; i < n; i += blocks * kIn) {
        const int64_t row = n >> 32 ? i / per_row : static_cast<uint32_t>(i) / per_row, col = (i - row * per_row) * 8;
        store_cols(static_cast<T *>(a.grad_table) + (begin + row) * a.ld_grad_table + col, vec8<T>(T(0.f)),
                   static_cast<int>(min(a.cols - col, int64_t(8))));
    }
}

using f64x8 = vec8<double>;

// Columns col .. col + kW - 1 of table row t from their sums.
template <class T, int kW>
__device__ __forceinline__ void write_sums(const EmbeddingArgs &a, int64_t t, int64_t col, const double (&sum)[kW]) {
    T *to = static_cast<T *>(a.grad_table) + t * a.ld_grad_table + col;
#pragma unroll
    for (int j = 0; j < kW; ++j)
        if (col + j < a.cols) to[j] = static_cast<T>(static_cast<float>(sum[j] * a.scale));
}

// ---- gradient of a small table ----------------------------------------------------------

// A table whose rows fit LDS: a workgroup takes a strip of rows of grad_out in their order, without
// a sorted list, and adds each to a sum of its index in LDS.  A thread owns four columns, `groups` threads
// share a column with sums of their own, so no two add to the same place and the order is fixed.  With
// more than one strip a second kernel adds their sums.
constexpr int kSmallCols = 4;  // columns of a thread
struct Strips {
    int threads;        // of a workgroup
    int groups, lanes;  // lanes: threads of a row's columns; groups x lanes = threads
    int slices;         // how often the lanes cover the columns
    int64_t count, rows;  // strips; rows of one
    float *part;          // [strip][table row][column]
};

// The rows of a strip that a thread adds to its sums at `mine`.  kWhole: all its columns are there.  kShared: sixteen
// threads or more have a row, and each loads one of the next sixteen rows' indices for all of them (two more
// loads a row would be as many as the rows' own: 280000 x 256, bf16, 37 us, and 34 so).
template <class T, bool kWhole, bool kShared>
__device__ __forceinline__ void add_strip(const EmbeddingArgs &a, const Strips &s, int64_t strip, int group, int64_t col,
                                          f32x4 *mine) {
    using Vec = T __attribute__((ext_vector_type(kSmallCols)));
    constexpr int kAhead = 16;
    const int n = kWhole ? kSmallCols : static_cast<int>(a.cols - col);
    const T *from = static_cast<const T *>(a.grad_out) + col;
    const int64_t end = min(a.rows, (strip + 1) * s.rows);
    const int64_t begin = strip * s.rows + group, step = int64_t(kAhead) * s.groups;
    if (begin >= end) return;
    const int lane = threadIdx.x & 63, in_row = lane & (s.lanes - 1), row_lane = lane - in_row;
    Vec v[kAhead];
    uint32_t t[kShared ? 1 : kAhead];
    const auto fetch = [&](int64_t i) {
        if (kShared) t[0] = index_at(a, min(i + (in_row & (kAhead - 1)) * s.groups, end - 1), kNone);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int64_t row = min(i + j * s.groups, end - 1);
            if (!kShared) t[kShared ? 0 : j] = index_at(a, row, kNone);
            const T *p = from + row * a.ld_grad_out;
            if (kWhole)
                __builtin_memcpy(&v[j], p, sizeof(Vec));
            else
                v[j] = load_first<Vec>(p, n);
        }
    };
    fetch(begin);
    for (int64_t i = begin; i < end; i += step) {
        Vec now[kAhead];
        uint32_t at[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            now[j] = v[j];
            at[j] = kShared ? __shfl(t[0], row_lane + j) : t[kShared ? 0 : j];
        }
        fetch(min(i + step, end - 1));  // at the end, again the last
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (at[j] != kNone && i + j * s.groups < end) mine[at[j] * s.lanes] += __builtin_convertvector(now[j], f32x4);
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) k_small(EmbeddingArgs a, Strips s) {
    constexpr int kW = kSmallCols;
    using Sum = f32x4;
    extern __shared__ char lds[];
    Sum *sums = reinterpret_cast<Sum *>(lds);
    const int tid = threadIdx.x, lane = tid & (s.lanes - 1), group = tid / s.lanes;
    const int table = static_cast<int>(a.table_rows);
    const uint32_t strip = blockIdx.x / static_cast<uint32_t>(s.slices), slice = blockIdx.x - strip * s.slices;
    const int64_t col = (int64_t(slice) * s.lanes + lane) * kW;
    for (int i = tid; i < table * s.threads; i += s.threads) sums[i] = Sum(0.f);
    __syncthreads();
    Sum *mine = sums + group * table * s.lanes + lane;
    // indices are shared where every thread of a row has its columns
    if (s.lanes >= 16 && a.cols % kW == 0 && a.cols % (s.lanes * kW) == 0)
        add_strip<T, true, true>(a, s, strip, group, col, mine);
    else if (col + kW <= a.cols)
        add_strip<T, true, false>(a, s, strip, group, col, mine);
    else if (col < a.cols)
        add_strip<T, false, false>(a, s, strip, group, col, mine);
    __syncthreads();
    for (int i = tid; i < table * s.lanes; i += s.threads) {
        const int t = i / s.lanes;
        const int64_t at = (int64_t(slice) * s.lanes + i - t * s.lanes) * kW;
        double total[kW] = {};
        for (int g = 0; g < s.groups; ++g) {
#pragma unroll
            for (int k = 0; k < kW; ++k) total[k] += sums[g * table * s.lanes + i][k];
        }
        if (s.count == 1) {
            write_sums<T, kW>(a, t, at, total);
        } else {
#pragma unroll
            for (int k = 0; k < kW; ++k)
                if (at + k < a.cols) s.part[(int64_t(strip) * table + t) * a.cols + at + k] = static_cast<float>(total[k]);
        }
    }
}

// A workgroup has 16 sums of the table, 64 threads for each.
constexpr int kJoinThreads = 1024, kJoinSums = 16;
template <class T>
__global__ void __launch_bounds__(kJoinThreads) k_join_small(EmbeddingArgs a, Strips s) {
    constexpr int kShares = kJoinThreads / kJoinSums;
    __shared__ double sums[kShares][kJoinSums];
    const int64_t n = a.table_rows * a.cols, at = int64_t(blockIdx.x) * kJoinSums + threadIdx.x % kJoinSums;
    const int share = threadIdx.x / kJoinSums;
    double sum[1] = {};
    if (at < n) {
#pragma unroll 8
        for (int64_t i = share; i < s.count; i += kShares) sum[0] += s.part[i * n + at];
    }
    sums[share][threadIdx.x % kJoinSums] = sum[0];
    __syncthreads();
    if (share || at >= n) return;
    for (int i = 1; i < kShares; ++i) sum[0] += sums[i][threadIdx.x];
    const int64_t t = at / a.cols;
    write_sums<T, 1>(a, t, at - t * a.cols, sum);
}

// ---- sort -----------------------------------------------------------------------------

// A workgroup sorts tiles of pairs, kItems a thread: lane l of wave w has the pairs 64 (kItems w + j) + l
// (j = 0 .. kItems - 1), so a wave's pairs are consecutive and its ballots rank them in order.
// The ballots keep a compute unit busy, so tiles are small: sixteen pairs a thread, 16384 in one workgroup,
// took 45 us for two passes; over 16 workgroups the four kernels take 20.
constexpr int kItems = 4, kRadix = 256, kTile = kThreads * kItems, kWaves = kThreads / 64;
// Up to so many pairs one workgroup sorts by itself, all passes in one launch: 8 us for one pass, 11 for two.
constexpr int kOneThreads = 1024, kOneWaves = kOneThreads / 64, kMostOne = kOneThreads * kItems;
constexpr int kMostBlocks = 256;  // workgroups of a pass
struct Sort {
    int64_t rows;
    uint32_t *key[2], *pos[2];  // key and position; the last pass writes [0]
    uint32_t *count;            // [block][digit]
    int blocks, tiles;          // of a pass; tiles of a block
    int bits, passes;
    int64_t zero_begin, zero_end;  // table rows that the workgroups past the sorting ones zero
};

template <class T, int kIn>
__device__ __forceinline__ void zero_share(const EmbeddingArgs &a, const Sort &s) {
    zero_rows<T, kIn>(a, s.zero_begin, s.zero_end, int64_t(blockIdx.x) - s.blocks, int64_t(gridDim.x) - s.blocks);
}

// Lanes of the wave with the same digit (of `bits` bits); those that are not `in` have none.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, int bits, bool in) {
    uint64_t same = __ballot(in);
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot(digit >> b & 1);
        same &= (digit >> b & 1) ? set : ~set;
    }
    return same;
}
__device__ __forceinline__ int lanes_below(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi(uint32_t(mask >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(mask), 0));
}

// Ranks of a thread's kItems digits among those of its wave's, in the order of the pairs; leaves the
// wave's count of each digit in `counts` (which are zero before).
__device__ __forceinline__ void rank_in_wave(const uint32_t (&digit)[kItems], const bool (&in)[kItems], int bits,
                                             uint32_t *counts, uint32_t (&rank)[kItems]) {
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const uint64_t same = same_digit(digit[j], bits, in[j]);
        const int below = lanes_below(same);
        uint32_t before = 0;
        if (in[j]) before = counts[digit[j]];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (in[j] && below == 0) counts[digit[j]] = before + __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        rank[j] = before + below;
    }
}

// Exclusive sums of `n` counters, at most four a thread, in order and in place; `scratch` holds a word for
// each of the kIn waves.
template <int kIn>
__device__ __forceinline__ void exclusive_sums(uint32_t *v, int n, uint32_t *scratch) {
    const int tid = threadIdx.x, lane = tid & 63;
    uint32_t mine[4], sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        mine[j] = 4 * tid + j < n ? v[4 * tid + j] : 0;
        sum += mine[j];
    }
    uint32_t scan = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t up = __shfl_up(scan, off);
        if (lane >= off) scan += up;
    }
    if (lane == 63) scratch[tid >> 6] = scan;
    __syncthreads();
    uint32_t run = scan - sum;
#pragma unroll
    for (int w = 0; w < kIn; ++w) run += w < (tid >> 6) ? scratch[w] : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (4 * tid + j < n) v[4 * tid + j] = run;
        run += mine[j];
    }
    __syncthreads();
}

// The first bit of pass p: the keys' bits are shared out evenly, at most eight a pass.
__device__ __forceinline__ int pass_shift(const Sort &s, int p) { return s.bits * p / s.passes; }

// All passes by one workgroup, in LDS, over at most kMostOne pairs.
template <class T>
__global__ void __launch_bounds__(kOneThreads) k_sort_one(EmbeddingArgs a, Sort s) {
    if (blockIdx.x) return zero_share<T, kOneThreads>(a, s);
    __shared__ uint32_t keys[kMostOne], counts[kRadix * kOneWaves], scratch[kOneWaves];
    __shared__ uint16_t at[kMostOne];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = static_cast<int>(s.rows);
    if (n == 0) return;
    uint32_t key[kItems], pos[kItems], rank[kItems], digit[kItems];
    bool in[kItems];
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const int i = 64 * (kItems * wave + j) + lane;
        in[j] = i < n;
        pos[j] = i;
        key[j] = index_at(a, min(i, n - 1), static_cast<uint32_t>(a.table_rows));
    }
    for (int p = 0; p < s.passes; ++p) {
        const int shift = pass_shift(s, p), width = pass_shift(s, p + 1) - shift;
#pragma unroll
        for (int j = 0; j < kRadix * kOneWaves / kOneThreads; ++j) counts[j * kOneThreads + tid] = 0;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kItems; ++j) digit[j] = key[j] >> shift & ((1u << width) - 1);
        // counters [wave][digit] for the ranks, read as [digit][wave] by the sums
        rank_in_wave(digit, in, width, counts + wave * kRadix, rank);
        __syncthreads();
        uint32_t turned[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) turned[j] = counts[(4 * tid + j) % kOneWaves * kRadix + (4 * tid + j) / kOneWaves];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) counts[4 * tid + j] = turned[j];
        __syncthreads();
        exclusive_sums<kOneWaves>(counts, kRadix * kOneWaves, scratch);
        const bool last = p + 1 == s.passes;
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const uint32_t to = counts[digit[j] * kOneWaves + wave] + rank[j];
            if (in[j] && last) {
                s.key[0][to] = key[j];
                s.pos[0][to] = pos[j];
            } else if (in[j]) {
                keys[to] = key[j];
                at[to] = static_cast<uint16_t>(pos[j]);
            }
        }
        if (last) return;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int i = 64 * (kItems * wave + j) + lane;
            if (in[j]) key[j] = keys[i], pos[j] = at[i];
        }
    }
}

// Key i of a pass: of the index itself in the first, else of what the pass before wrote.
template <bool kFirst>
__device__ __forceinline__ uint32_t key_at(const EmbeddingArgs &a, const Sort &s, int pass, int64_t i) {
    return kFirst ? index_at(a, i, static_cast<uint32_t>(a.table_rows)) : s.key[(s.passes - pass) & 1][i];
}

// Counts of each workgroup's digits of a pass.
template <class T, bool kFirst>
__global__ void __launch_bounds__(kThreads) k_count(EmbeddingArgs a, Sort s, int pass) {
    if (static_cast<int>(blockIdx.x) >= s.blocks) return zero_share<T, kThreads>(a, s);
    __shared__ uint32_t counts[kRadix];
    const int tid = threadIdx.x, shift = pass_shift(s, pass), width = pass_shift(s, pass + 1) - shift;
    counts[tid] = 0;
    __syncthreads();
    const int64_t first = int64_t(blockIdx.x) * s.tiles * kTile, end = min(s.rows, first + int64_t(s.tiles) * kTile);
#pragma unroll 4
    for (int64_t i = first + tid; i < end; i += kThreads)
        atomicAdd(&counts[key_at<kFirst>(a, s, pass, i) >> shift & ((1u << width) - 1)], 1u);
    __syncthreads();
    s.count[blockIdx.x * kRadix + tid] = counts[tid];
}

// One pass: every pair to its place.  The place of a workgroup's first pair of a digit is the number of
// pairs of smaller digits and of those of the digit in the workgroups before it, from the counts.
template <class T, bool kFirst>
__global__ void __launch_bounds__(kThreads) k_place(EmbeddingArgs a, Sort s, int pass) {
    if (static_cast<int>(blockIdx.x) >= s.blocks) return zero_share<T, kThreads>(a, s);
    __shared__ uint32_t total[kRadix], mine[kRadix], counts[kWaves * kRadix], scratch[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int shift = pass_shift(s, pass), width = pass_shift(s, pass + 1) - shift;
    const uint32_t digits = 1u << width;
    const int to_buffer = (s.passes - 1 - pass) & 1;  // the last pass writes [0]
    const uint32_t *pos_in = s.pos[to_buffer ^ 1];
    uint32_t *key_out = s.key[to_buffer], *pos_out = s.pos[to_buffer];

    total[tid] = 0, mine[tid] = 0;
    __syncthreads();
    {
        // a digit by kThreads / digits threads, which share the workgroups
        const uint32_t digit = tid & (digits - 1);
        const int step = kThreads >> width;
        uint32_t all = 0, before = 0;
#pragma unroll 8
        for (int b = tid >> width; b < s.blocks; b += step) {
            const uint32_t c = s.count[b * kRadix + digit];
            all += c;
            before += b < static_cast<int>(blockIdx.x) ? c : 0;
        }
        atomicAdd(&total[digit], all);
        atomicAdd(&mine[digit], before);
    }
    __syncthreads();
    exclusive_sums<kWaves>(total, kRadix, scratch);
    mine[tid] += total[tid];

    for (int tile = 0; tile < s.tiles; ++tile) {
        const int64_t first = (int64_t(blockIdx.x) * s.tiles + tile) * kTile;
        if (first >= s.rows) break;
        uint32_t key[kItems], pos[kItems], rank[kItems], digit[kItems];
        bool in[kItems];
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int64_t i = first + 64 * (kItems * wave + j) + lane;
            in[j] = i < s.rows;
            key[j] = key_at<kFirst>(a, s, pass, min(i, s.rows - 1));
            pos[j] = kFirst ? static_cast<uint32_t>(i) : pos_in[min(i, s.rows - 1)];
            digit[j] = key[j] >> shift & (digits - 1);
        }
#pragma unroll
        for (int j = 0; j < kWaves * kRadix / kThreads; ++j) counts[j * kThreads + tid] = 0;
        __syncthreads();
        rank_in_wave(digit, in, width, counts + wave * kRadix, rank);
        __syncthreads();
        // thread = digit: where each wave's pairs of it begin, and the next tile's
        {
            uint32_t run = mine[tid];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const uint32_t c = counts[w * kRadix + tid];
                counts[w * kRadix + tid] = run;
                run += c;
            }
            mine[tid] = run;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            if (!in[j]) continue;
            const uint32_t to = counts[wave * kRadix + digit[j]] + rank[j];
            key_out[to] = key[j];
            pos_out[to] = pos[j];
        }
        __syncthreads();
    }
}

// ---- sums of sorted rows ------------------------------------------------------------------

struct Chunks {
    const uint32_t *key, *pos;
    float *part;  // [chunk][head, tail][column, a multiple of eight]
    int64_t rows;  // sorted pairs, those of no table row at the end
    int64_t count;
    int length;
    int lanes, slices;  // lanes of a row's columns, and how often they cover them
    int64_t blocks;
};

template <class T>
__device__ __forceinline__ void write_row(const EmbeddingArgs &a, uint32_t t, int64_t col, f64x8 sum, int n) {
    sum *= static_cast<double>(a.scale);
    store_cols(static_cast<T *>(a.grad_table) + int64_t(t) * a.ld_grad_table + col,
               from_f32<T>(__builtin_convertvector(sum, f32x8)), n);
}

// kWhole: all eight columns are there.
template <class T, bool kWhole>
__device__ __forceinline__ void walk_chunk(const EmbeddingArgs &a, const Chunks &c, int64_t chunk, int64_t col) {
    const int n = kWhole ? 8 : static_cast<int>(a.cols - col);
    const int64_t begin = chunk * c.length, end = min(c.rows, begin + c.length);
    const T *from = static_cast<const T *>(a.grad_out) + col;
    float *part = c.part + chunk * 2 * c.lanes * c.slices * 8 + col;

    constexpr int kAhead = 8;
    uint32_t key[kAhead], pos[kAhead];
    const auto fetch = [&](int64_t i) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int64_t at = min(i + j, end - 1);
            key[j] = c.key[at];
            pos[j] = c.pos[at];
        }
    };
    fetch(begin);
    const uint32_t before = c.key[begin ? begin - 1 : 0], after = c.key[min(end, c.rows - 1)];
    uint32_t run = key[0];
    bool head = begin > 0 && before == run;  // whether the run began in an earlier chunk
    f64x8 sum = {};
    for (int64_t i = begin; i < end && run < a.table_rows; i += kAhead) {
        uint32_t now[kAhead];
        vec8<T> v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            now[j] = key[j];
            const T *p = from + int64_t(pos[j]) * a.ld_grad_out;
            v[j] = kWhole ? load8(p) : load_first<vec8<T>>(p, n);
        }
        fetch(min(i + kAhead, end - 1));
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (i + j >= end) break;
            if (now[j] != run) {
                if (head)
                    store8(part, __builtin_convertvector(sum, f32x8));
                else
                    write_row<T>(a, run, col, sum, n);
                head = false;
                run = now[j];
                sum = f64x8{};
                if (run >= a.table_rows) break;
            }
            sum += __builtin_convertvector(v[j], f64x8);
        }
    }
    if (run >= a.table_rows) return;  // from here on the list holds pairs of no table row
    const bool on = end < c.rows && after == run;
    if (head)
        store8(part, __builtin_convertvector(sum, f32x8));
    else if (on)
        store8(part + c.lanes * c.slices * 8, __builtin_convertvector(sum, f32x8));
    else
        write_row<T>(a, run, col, sum, n);
}

template <class T>
__global__ void __launch_bounds__(kThreads) k_sums(EmbeddingArgs a, Chunks c) {
    const int64_t item = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / c.lanes, chunk = item / c.slices;
    const int64_t col = ((item - chunk * c.slices) * c.lanes + threadIdx.x % c.lanes) * 8;
    if (chunk >= c.count || col >= a.cols) return;
    if (col + 8 <= a.cols)
        walk_chunk<T, true>(a, c, chunk, col);
    else
        walk_chunk<T, false>(a, c, chunk, col);
}

// The last chunk that a run reaches, which begins in `chunk` and reaches the next: the wave's 64 lanes probe
// the chunks' first keys, near ones first.
__device__ __forceinline__ int64_t last_chunk(const Chunks &c, int64_t chunk, uint32_t run) {
    const int lane = threadIdx.x & 63;
    int64_t lo = chunk + 1, step = 1;  // lo: reached
    for (;;) {
        const int64_t i = lo + step * (lane + 1);
        const bool reached = i < c.count && c.key[i * c.length] == run;
        const int n = __popcll(__ballot(reached));
        lo += step * n;
        if (n == 64) {
            step *= 64;
        } else {
            if (step == 1) return lo;
            step /= 64;
        }
    }
}

// A workgroup for each chunk whose last run goes on in the next and kJoinCols columns (blockIdx.y): the sum of
// what the chunks hold of it.
constexpr int kJoinLanes = 32, kJoinCols = kJoinLanes * 8;
template <class T>
__global__ void __launch_bounds__(kThreads) k_join_runs(EmbeddingArgs a, Chunks c) {
    constexpr int kGroups = kThreads / kJoinLanes;
    __shared__ double sums[kGroups][kJoinCols];
    const int64_t chunk = blockIdx.x, begin = chunk * c.length, end = begin + c.length;  // not the last chunk
    const uint32_t before = c.key[begin ? begin - 1 : 0], run = c.key[end - 1], after = c.key[end];
    if (run >= a.table_rows || after != run) return;
    if (begin > 0 && before == run) return;  // it began before this chunk
    const int64_t last = last_chunk(c, chunk, run);
    const int lane = threadIdx.x % kJoinLanes, group = threadIdx.x / kJoinLanes;
    const int64_t row = int64_t(c.lanes) * c.slices * 8, col = int64_t(blockIdx.y) * kJoinCols + lane * 8;
    f64x8 sum = {};
    if (col < a.cols) {
        if (group == 0) sum = __builtin_convertvector(load8(c.part + (chunk * 2 + 1) * row + col), f64x8);
        for (int64_t i = chunk + 1 + group; i <= last; i += 8 * kGroups) {
            f32x8 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = load8(c.part + min(i + j * kGroups, last) * 2 * row + col);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i + j * kGroups <= last) sum += __builtin_convertvector(v[j], f64x8);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[group][lane * 8 + j] = sum[j];
    __syncthreads();
    if (group || col >= a.cols) return;
    for (int g = 1; g < kGroups; ++g) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += sums[g][lane * 8 + j];
    }
    write_row<T>(a, run, col, sum, static_cast<int>(min<int64_t>(a.cols - col, 8)));
}

// ---- launches -------------------------------------------------------------------------

constexpr size_t up(size_t v) { return (v + 255) / 256 * 256; }

// Whether the table is summed in LDS.  At 17 to 32 rows a workgroup has 128 threads of sums, and wide rows
// are better sorted (a replayed graph with the gradient, us, sorted and here; about 18 of it are the replay's):
// 10 rows, 280000 x 256 bf16: 88 and 43; 10, 5000 x 512: 26 and 19; 32, 280000 x 256: 73 and 70; 32, 5000 x 512:
// 26 and 39; 32, 5000 x 128 fp32: 25 and 19; 64, 5000 x 128: 25 and 29.
bool small_table(int64_t table_rows, int64_t cols) { return table_rows <= 16 || (table_rows <= 32 && cols <= 256); }

struct Plan {
    bool small;  // see small_table
    Strips strips;
    bool one;  // one workgroup sorts
    int bits, passes, blocks, tiles;
    Chunks chunks;
    size_t list, count, part, bytes;  // bytes of one list of keys or positions, of the counts and partial sums
};

Plan plan_of(int64_t table_rows, int64_t cols, int64_t rows) {
    Plan p{};
    p.small = small_table(table_rows, cols);
    if (p.small) {
        Strips &s = p.strips;
        s.threads = table_rows <= 16 ? kThreads : kThreads / 2;  // 64 KB of sums at most
        const int64_t pieces = std::max<int64_t>((cols + kSmallCols - 1) / kSmallCols, 1);
        for (s.lanes = 1; s.lanes < s.threads && s.lanes < pieces; s.lanes *= 2) {
        }
        s.groups = s.threads / s.lanes;
        s.slices = static_cast<int>((pieces + s.lanes - 1) / s.lanes);
        // two workgroups a compute unit (with four, 10 rows, 280000 x 256 bf16: 46 us for 38, their sums are written
        // and read), 16 rows a thread at least and 4096 at most (fp32 sums)
        const int64_t least = (rows + int64_t(s.groups) * 4096 - 1) / (int64_t(s.groups) * 4096);
        const int64_t most = (rows + s.groups * 16 - 1) / (s.groups * 16);
        s.count = std::max<int64_t>(1, std::max(least, std::min<int64_t>(most, std::max(1, 512 / s.slices))));
        s.rows = (rows + s.count - 1) / s.count;
        p.part = s.count > 1 ? up(static_cast<size_t>(s.count) * table_rows * cols * 4) : 0;
        p.bytes = p.part;
        return p;
    }
    for (p.bits = 1; p.bits < 32 && (table_rows >> p.bits); ++p.bits) {
    }
    p.passes = (p.bits + 7) / 8;
    p.one = rows <= kMostOne;
    const int64_t tiles = (rows + kTile - 1) / kTile;
    p.tiles = static_cast<int>((tiles + kMostBlocks - 1) / kMostBlocks);
    p.blocks = p.tiles ? static_cast<int>((tiles + p.tiles - 1) / p.tiles) : 0;
    Chunks &c = p.chunks;
    c.rows = rows;
    const int64_t pieces = std::max<int64_t>((cols + 7) / 8, 1);
    for (c.lanes = 1; c.lanes < 64 && c.lanes < pieces; c.lanes *= 2) {
    }
    c.slices = static_cast<int>((pieces + c.lanes - 1) / c.lanes);
    // chunks of at least 16 pairs, and no more of them than fill the chip a few times
    c.length = static_cast<int>(std::max<int64_t>(16, (rows + 8191) / 8192 + 7)) / 8 * 8;
    c.count = (rows + c.length - 1) / c.length;
    c.blocks = (c.count * c.slices * c.lanes + kThreads - 1) / kThreads;
    p.list = up(static_cast<size_t>(rows) * 4);
    p.count = !p.one ? up(static_cast<size_t>(p.blocks) * kRadix * 4) : 0;
    p.part = c.count > 1 ? up(static_cast<size_t>(c.count) * 2 * c.lanes * c.slices * 8 * 4) : 0;
    p.bytes = p.list * (p.one || p.passes == 1 ? 2 : 4) + p.count + p.part;
    return p;
}

template <class T>
hipError_t gradient(const EmbeddingArgs &a, hipStream_t stream) {
    Plan p = plan_of(a.table_rows, a.cols, a.rows);
    char *ws = static_cast<char *>(a.workspace);
    if (p.small) {
        p.strips.part = reinterpret_cast<float *>(ws);
        const unsigned bytes = static_cast<unsigned>(a.table_rows * p.strips.threads * kSmallCols * 4);
        const dim3 blocks(static_cast<unsigned>(p.strips.count * p.strips.slices));
        k_small<T><<<blocks, dim3(p.strips.threads), bytes, stream>>>(a, p.strips);
        const int64_t joins = (a.table_rows * a.cols + kJoinSums - 1) / kJoinSums;
        if (p.strips.count > 1)
            k_join_small<T><<<dim3(static_cast<unsigned>(joins)), dim3(kJoinThreads), 0, stream>>>(a, p.strips);
        return hipGetLastError();
    }
    const auto take = [&](size_t bytes) {
        char *at = ws;
        ws += bytes;
        return reinterpret_cast<uint32_t *>(at);
    };
    Sort s{};
    s.rows = a.rows, s.blocks = p.blocks, s.tiles = p.tiles, s.bits = p.bits, s.passes = p.passes;
    s.key[0] = take(p.list);
    s.pos[0] = take(p.list);
    if (!p.one && p.passes > 1) {
        s.key[1] = take(p.list);
        s.pos[1] = take(p.list);
    }
    s.count = take(p.count);
    Chunks &c = p.chunks;
    c.part = reinterpret_cast<float *>(take(p.part));
    c.key = s.key[0], c.pos = s.pos[0];
    // The sort waits for memory more than it uses it, so its launches zero the table between them; the
    // sums then write the rows that are used.
    using Zero = typename std::conditional<sizeof(T) == 4, float, f16>::type;  // of T's size
    const int turns = p.one ? 1 : 2 * s.passes;
    const int64_t zeros = (a.table_rows / turns + 1) * ((a.cols + 7) / 8);
    s.blocks = p.one ? 1 : s.blocks;
    const dim3 threads(p.one ? kOneThreads : kThreads);
    const dim3 grid(static_cast<unsigned>(s.blocks + std::min<int64_t>((zeros + 4 * threads.x - 1) / (4 * threads.x), 2048)));
    for (int turn = 0; turn < turns; ++turn) {
        s.zero_begin = a.table_rows * turn / turns;
        s.zero_end = a.table_rows * (turn + 1) / turns;
        const auto run = [&](auto first) {
            constexpr bool kFirst = decltype(first)::value;
            if (turn % 2 == 0)
                k_count<Zero, kFirst><<<grid, threads, 0, stream>>>(a, s, turn / 2);
            else
                k_place<Zero, kFirst><<<grid, threads, 0, stream>>>(a, s, turn / 2);
        };
        if (p.one)
            k_sort_one<Zero><<<grid, threads, 0, stream>>>(a, s);
        else if (turn < 2)
            run(std::true_type());
        else
            run(std::false_type());
    }
    if (c.count) k_sums<T><<<dim3(static_cast<unsigned>(c.blocks)), dim3(kThreads), 0, stream>>>(a, c);
    if (c.count > 1) k_join_runs<T><<<dim3(static_cast<unsigned>(c.count - 1), static_cast<unsigned>((a.cols + kJoinCols - 1) / kJoinCols)),
                         dim3(kThreads), 0, stream>>>(a, c);
    return hipGetLastError();
}

}  // namespace

size_t embedding_workspace(int64_t table_rows, int64_t cols, int64_t rows) { return plan_of(table_rows, cols, rows).bytes; }

int64_t embedding_blocks(int64_t table_rows, int64_t cols, int64_t rows) {
    const Plan p = plan_of(table_rows, cols, rows);
    const int64_t joins = p.small ? (table_rows * cols + kJoinSums - 1) / kJoinSums * (kJoinThreads / kThreads)
                                  : p.chunks.count * ((cols + kJoinCols - 1) / kJoinCols);
    return std::max({p.chunks.blocks, joins, p.strips.count * p.strips.slices});
}

hipError_t embedding_fwd(oeq_dtype dtype, const EmbeddingArgs &a, hipStream_t stream) {
    switch (dtype) {
        case OEQ_F32: return lookup<float>(a, stream);
        case OEQ_F16: return lookup<f16>(a, stream);
        case OEQ_BF16: return lookup<bf16>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

hipError_t embedding_bwd(oeq_dtype dtype, const EmbeddingArgs &a, hipStream_t stream) {
    switch (dtype) {
        case OEQ_F32: return gradient<float>(a, stream);
        case OEQ_F16: return gradient<f16>(a, stream);
        case OEQ_BF16: return gradient<bf16>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace readout
}  // namespace oeq
