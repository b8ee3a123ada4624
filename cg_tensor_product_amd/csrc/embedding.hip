// Embedding lookup with scaling, and its gradient by sorted indices.
//   out[i] = scale table[index[i]]          grad_table[t] = scale sum_{i: index[i] = t} grad_out[i]
// An index outside the table gives a row of zeros and takes no gradient.
//
// The lookup is a copy of rows: a thread takes eight columns of one.
//
// The gradient's sums have no atomics: (index, position) pairs are sorted by index with the positions of
// one index in increasing order (a stable radix sort), the sorted list is cut into chunks of equal
// length, and a few lanes walk each chunk, their columns in registers, and write a table row where
// its run of equal indices ends.  So neither a common index (tens of thousands of uses of one species)
// nor many rare ones (a vocabulary) leave lanes idle.  A run that a cut divides leaves a partial sum a
// chunk, and a second kernel adds those in order.  Rows that no index names are zeroed by further
// workgroups of the same launch, which look for their rows in the sorted list.
#include <algorithm>

#include "readout.hpp"
#include "readout_device.hpp"

namespace oeq {
namespace readout {

namespace {

constexpr int kThreads = 256;

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

// The table row that index i names, or `none`.
__device__ __forceinline__ int64_t index_at(const EmbeddingArgs &a, int64_t i, int64_t none) {
    const int64_t t = a.wide ? static_cast<const int64_t *>(a.index)[i] : static_cast<const int32_t *>(a.index)[i];
    return t >= 0 && t < a.table_rows ? t : none;
}

// ---- lookup ---------------------------------------------------------------------------

template <class T, class Index>
__global__ void __launch_bounds__(kThreads) k_lookup(EmbeddingArgs a, uint32_t per_row) {
    const Index total = static_cast<Index>(a.rows) * per_row, step = Index(gridDim.x) * kThreads;
    for (Index i = Index(blockIdx.x) * kThreads + threadIdx.x; i < total; i += step) {
        const Index row = i / per_row;
        const int64_t col = int64_t(i - row * per_row) * 8;
        const int n = static_cast<int>(min(a.cols - col, int64_t(8)));
        const int64_t t = index_at(a, static_cast<int64_t>(row), -1);
        f32x8 v = {};
        if (t >= 0) v = to_f32<T>(load_cols(static_cast<const T *>(a.table) + t * a.ld_table + col, n)) * a.scale;
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

// ---- sort -----------------------------------------------------------------------------

// A workgroup sorts tiles of kTile pairs, four a thread: thread t of wave w has the pairs
// 256 w + 64 j + lane (j = 0..3), so a wave's pairs are consecutive and its ballots rank them in order.
constexpr int kItems = 4, kTile = kThreads * kItems, kWaves = kThreads / 64, kRadix = 256;
constexpr int kMostBlocks = 256;  // workgroups of a pass
constexpr int kOneWaves = 16, kOneTile = 64 * kOneWaves * kItems;  // what one workgroup sorts by itself

struct Sort {
    int64_t rows;
    uint32_t *key[2], *pos[2];  // key and position; the last pass writes [0]
    uint32_t *count;            // [pass][block][digit]
    int blocks, tiles;          // of a pass; tiles of a block
    int passes;
};

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

// Exclusive sums of `n` <= 4 * threads counters in order, in place; every thread takes four.  Returns
// nothing; `scratch` holds a word a wave.
template <int kWavesIn>
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
    for (int w = 0; w < (tid >> 6); ++w) run += scratch[w];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (4 * tid + j < n) v[4 * tid + j] = run;
        run += mine[j];
    }
    __syncthreads();
}

// Bits of pass p of `passes` over keys of `bits` bits, shared out evenly.
__device__ __forceinline__ int pass_shift(int bits, int passes, int p) { return bits * p / passes; }

// All passes by one workgroup of kOneWaves waves, in LDS.
__global__ void __launch_bounds__(64 * kOneWaves) k_sort_one(EmbeddingArgs a, Sort s, int bits) {
    __shared__ uint32_t keys[kOneTile], counts[kRadix * kOneWaves], scratch[kOneWaves];
    __shared__ uint16_t at[kOneTile];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = static_cast<int>(s.rows);
    uint32_t key[kItems], pos[kItems], rank[kItems], digit[kItems];
    bool in[kItems];
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const int i = 64 * (kItems * wave + j) + lane;
        in[j] = i < n;
        pos[j] = i;
        key[j] = in[j] ? static_cast<uint32_t>(index_at(a, i, a.table_rows)) : 0;
    }
    for (int p = 0; p < s.passes; ++p) {
        const int shift = pass_shift(bits, s.passes, p), width = pass_shift(bits, s.passes, p + 1) - shift;
        for (int i = tid; i < kRadix * kOneWaves; i += 64 * kOneWaves) counts[i] = 0;
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
        __syncthreads();
        if (!last) {
#pragma unroll
            for (int j = 0; j < kItems; ++j) {
                const int i = 64 * (kItems * wave + j) + lane;
                if (in[j]) key[j] = keys[i], pos[j] = at[i];
            }
        }
    }
}

// The first pass's counts of each workgroup's digits; the later passes' are zeroed.
__global__ void __launch_bounds__(kThreads) k_count(EmbeddingArgs a, Sort s, int bits) {
    __shared__ uint32_t counts[kRadix];
    const int tid = threadIdx.x, width = pass_shift(bits, s.passes, 1);
    counts[tid] = 0;
    __syncthreads();
    const int64_t first = int64_t(blockIdx.x) * s.tiles * kTile, end = min(s.rows, first + int64_t(s.tiles) * kTile);
    for (int64_t i = first + tid; i < end; i += kThreads)
        atomicAdd(&counts[static_cast<uint32_t>(index_at(a, i, a.table_rows)) & ((1u << width) - 1)], 1u);
    __syncthreads();
    s.count[blockIdx.x * kRadix + tid] = counts[tid];
    for (int p = 1; p < s.passes; ++p) s.count[(int64_t(p) * s.blocks + blockIdx.x) * kRadix + tid] = 0;
}

// One pass: every pair to its place.  The place of a workgroup's first pair of a digit is the number of
// pairs of smaller digits and of those of the digit in the workgroups before it, from the counts.
// Each pair also counts for the next pass, in the workgroup that will have it (integer sums: exact in
// any order).
__global__ void __launch_bounds__(kThreads) k_place(EmbeddingArgs a, Sort s, int bits, int pass) {
    __shared__ uint32_t total[kRadix], mine[kRadix], counts[kWaves * kRadix], scratch[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int shift = pass_shift(bits, s.passes, pass), width = pass_shift(bits, s.passes, pass + 1) - shift;
    const int next = pass + 1 < s.passes ? pass_shift(bits, s.passes, pass + 1) : 0;
    const int next_width = next ? pass_shift(bits, s.passes, pass + 2) - next : 0;
    const bool from_index = pass == 0;
    // the last pass writes [0], each one before it the other buffer
    const int to_buffer = (s.passes - 1 - pass) & 1;
    const uint32_t *key_in = s.key[to_buffer ^ 1], *pos_in = s.pos[to_buffer ^ 1];
    uint32_t *key_out = s.key[to_buffer], *pos_out = s.pos[to_buffer];

    // 2^width digits by 256 >> width threads each, which share the workgroups
    total[tid] = 0;
    mine[tid] = 0;
    __syncthreads();
    const uint32_t *count = s.count + int64_t(pass) * s.blocks * kRadix;
    {
        const int digit = tid & ((1 << width) - 1), step = kThreads >> width;
        uint32_t all = 0, before = 0;
#pragma unroll 8
        for (int b = tid >> width; b < s.blocks; b += step) {
            const uint32_t c = count[b * kRadix + digit];
            all += c;
            before += b < static_cast<int>(blockIdx.x) ? c : 0;
        }
        atomicAdd(&total[digit], all);
        atomicAdd(&mine[digit], before);
    }
    __syncthreads();
    exclusive_sums<kWaves>(total, kRadix, scratch);
    mine[tid] += total[tid];
    __syncthreads();

    for (int tile = 0; tile < s.tiles; ++tile) {
        const int64_t first = (int64_t(blockIdx.x) * s.tiles + tile) * kTile;
        if (first >= s.rows) break;
        uint32_t key[kItems], pos[kItems], rank[kItems], digit[kItems];
        bool in[kItems];
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int64_t i = first + 64 * (kItems * wave + j) + lane;
            in[j] = i < s.rows;
            key[j] = 0, pos[j] = 0;
            if (in[j] && from_index) {
                key[j] = static_cast<uint32_t>(index_at(a, i, a.table_rows));
                pos[j] = static_cast<uint32_t>(i);
            } else if (in[j]) {
                key[j] = key_in[i];
                pos[j] = pos_in[i];
            }
            digit[j] = key[j] >> shift & ((1u << width) - 1);
        }
#pragma unroll
        for (int w = 0; w < kWaves; ++w) counts[w * kRadix + tid] = 0;
        __syncthreads();
        rank_in_wave(digit, in, width, counts + wave * kRadix, rank);
        __syncthreads();
        // thread = digit: where each wave's pairs of it begin, and the next tile's
        uint32_t run = mine[tid];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const uint32_t c = counts[w * kRadix + tid];
            counts[w * kRadix + tid] = run;
            run += c;
        }
        mine[tid] = run;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            if (!in[j]) continue;
            const uint32_t to = counts[wave * kRadix + digit[j]] + rank[j];
            key_out[to] = key[j];
            pos_out[to] = pos[j];
            if (next_width) {
                const uint32_t block = to / static_cast<uint32_t>(s.tiles * kTile);
                atomicAdd(&s.count[(int64_t(pass + 1) * s.blocks + block) * kRadix +
                                   (key[j] >> next & ((1u << next_width) - 1))],
                          1u);
            }
        }
        __syncthreads();
    }
}

// ---- sums -----------------------------------------------------------------------------

struct Chunks {
    const uint32_t *key, *pos;
    float *part;  // [chunk][head, tail][column, a multiple of eight]
    int64_t rows;  // sorted pairs, those of no table row at the end
    int64_t count;
    int length;
    int lanes, slices;  // lanes of a row's columns, and how often they cover them
    int64_t blocks;     // workgroups that sum; the others zero table rows
    int fill_rows;      // table rows of one of those
};

using f64x8 = vec8<double>;

template <class T>
__device__ __forceinline__ void write_row(const EmbeddingArgs &a, uint32_t t, int64_t col, f64x8 sum, int n) {
    sum *= static_cast<double>(a.scale);
    store_cols(static_cast<T *>(a.grad_table) + int64_t(t) * a.ld_grad_table + col,
               from_f32<T>(__builtin_convertvector(sum, f32x8)), n);
}

// The number of sorted keys below t.
__device__ __forceinline__ int64_t lower_bound(const uint32_t *key, int64_t n, uint32_t t) {
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (key[mid] < t)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

template <class T>
__device__ __forceinline__ void zero_absent(const EmbeddingArgs &a, const Chunks &c, int64_t first) {
    __shared__ uint32_t absent[kThreads / 32];
    const int n = static_cast<int>(min<int64_t>(c.fill_rows, a.table_rows - first));
    if (threadIdx.x < kThreads / 32) absent[threadIdx.x] = 0;
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < n) {
        const uint32_t t = static_cast<uint32_t>(first + threadIdx.x);
        const int64_t at = lower_bound(c.key, c.rows, t);
        if (at == c.rows || c.key[at] != t) atomicOr(&absent[threadIdx.x >> 5], 1u << (threadIdx.x & 31));
    }
    __syncthreads();
    const int per_row = static_cast<int>((a.cols + 7) / 8);
    for (int r = 0; r < n; ++r) {
        if (!(absent[r >> 5] >> (r & 31) & 1)) continue;
        T *row = static_cast<T *>(a.grad_table) + (first + r) * a.ld_grad_table;
        for (int i = threadIdx.x; i < per_row; i += kThreads)
            store_cols(row + 8 * int64_t(i), vec8<T>(T(0.f)), static_cast<int>(min<int64_t>(a.cols - 8 * int64_t(i), 8)));
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) k_sums(EmbeddingArgs a, Chunks c) {
    if (blockIdx.x >= c.blocks) return zero_absent<T>(a, c, (int64_t(blockIdx.x) - c.blocks) * c.fill_rows);
    const int64_t item = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / c.lanes, chunk = item / c.slices;
    const int64_t col = ((item - chunk * c.slices) * c.lanes + threadIdx.x % c.lanes) * 8;
    if (chunk >= c.count || col >= a.cols) return;
    const int n = static_cast<int>(min<int64_t>(a.cols - col, 8));
    const int64_t begin = chunk * c.length, end = min(c.rows, begin + c.length);
    const T *from = static_cast<const T *>(a.grad_out) + col;
    float *part = c.part + chunk * 2 * c.lanes * c.slices * 8 + col;

    uint32_t run = c.key[begin];
    bool head = begin > 0 && c.key[begin - 1] == run;  // whether the run began in an earlier chunk
    f64x8 sum = {};
    constexpr int kAhead = 8;
    for (int64_t i = begin; i < end && run < a.table_rows; i += kAhead) {
        uint32_t key[kAhead];
        vec8<T> v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int64_t at = min(i + j, end - 1);
            key[j] = i + j < end ? c.key[at] : run;
            v[j] = load_cols(from + int64_t(c.pos[at]) * a.ld_grad_out, n);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (i + j >= end) break;
            if (key[j] != run) {
                if (head)
                    store8(part, __builtin_convertvector(sum, f32x8));
                else
                    write_row<T>(a, run, col, sum, n);
                head = false;
                run = key[j];
                sum = f64x8{};
                if (run >= a.table_rows) break;
            }
            sum += __builtin_convertvector(v[j], f64x8);
        }
    }
    if (run >= a.table_rows) return;  // from here on the list holds pairs of no table row
    const bool on = end < c.rows && c.key[end] == run;
    if (head)
        store8(part, __builtin_convertvector(sum, f32x8));
    else if (on)
        store8(part + c.lanes * c.slices * 8, __builtin_convertvector(sum, f32x8));
    else
        write_row<T>(a, run, col, sum, n);
}

// A workgroup for each chunk whose last run goes on in the next: the sum of what the chunks hold of it.
template <class T>
__global__ void __launch_bounds__(kThreads) k_join_runs(EmbeddingArgs a, Chunks c) {
    constexpr int kLanes = 32, kGroups = kThreads / kLanes;
    __shared__ double sums[kGroups][kLanes * 8];
    const int64_t chunk = blockIdx.x, begin = chunk * c.length, end = begin + c.length;  // not the last chunk
    const uint32_t run = c.key[end - 1];
    if (run >= a.table_rows || c.key[end] != run) return;
    if (begin > 0 && c.key[begin - 1] == run) return;  // it began before this chunk
    const int64_t stop = lower_bound(c.key, c.rows, run + 1), last = (stop - 1) / c.length;
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const int64_t row = int64_t(c.lanes) * c.slices * 8;
    for (int64_t col0 = 0; col0 < a.cols; col0 += kLanes * 8) {
        const int64_t col = col0 + lane * 8;
        f64x8 sum = {};
        if (col < a.cols) {
            if (group == 0) sum = __builtin_convertvector(load8(c.part + (chunk * 2 + 1) * row + col), f64x8);
#pragma unroll 4
            for (int64_t i = chunk + 1 + group; i <= last; i += kGroups)
                sum += __builtin_convertvector(load8(c.part + i * 2 * row + col), f64x8);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[group][lane * 8 + j] = sum[j];
        __syncthreads();
        if (group == 0 && col < a.cols) {
            for (int g = 1; g < kGroups; ++g) {
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += sums[g][lane * 8 + j];
            }
            write_row<T>(a, run, col, sum, static_cast<int>(min<int64_t>(a.cols - col, 8)));
        }
        __syncthreads();
    }
}

// ---- launches -------------------------------------------------------------------------

constexpr size_t up(size_t v) { return (v + 255) / 256 * 256; }

struct Plan {
    bool one;  // one workgroup sorts
    int bits, passes, blocks, tiles;
    Chunks chunks;
    int64_t fill_blocks;
    size_t list, count, part, bytes;  // bytes of one list of keys or positions, of the counts and partial sums
};

Plan plan_of(int64_t table_rows, int64_t cols, int64_t rows) {
    Plan p{};
    for (p.bits = 1; p.bits < 32 && (table_rows >> p.bits); ++p.bits) {
    }
    p.passes = (p.bits + 7) / 8;
    p.one = rows <= kOneTile;
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
    c.fill_rows = static_cast<int>(std::min<int64_t>(kThreads, std::max<int64_t>(1, 32768 / (pieces * 16))));
    p.fill_blocks = (table_rows + c.fill_rows - 1) / c.fill_rows;
    p.list = up(static_cast<size_t>(rows) * 4);
    p.count = p.one ? 0 : up(static_cast<size_t>(p.passes) * p.blocks * kRadix * 4);
    p.part = c.count > 1 ? up(static_cast<size_t>(c.count) * 2 * c.lanes * c.slices * 8 * 4) : 0;
    p.bytes = p.list * (p.one || p.passes == 1 ? 2 : 4) + p.count + p.part;
    return p;
}

template <class T>
hipError_t gradient(const EmbeddingArgs &a, hipStream_t stream) {
    Plan p = plan_of(a.table_rows, a.cols, a.rows);
    char *ws = static_cast<char *>(a.workspace);
    const auto take = [&](size_t bytes) {
        char *at = ws;
        ws += bytes;
        return reinterpret_cast<uint32_t *>(at);
    };
    Sort s{};
    s.rows = a.rows, s.blocks = p.blocks, s.tiles = p.tiles, s.passes = p.passes;
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
    if (a.rows && p.one) {
        k_sort_one<<<dim3(1), dim3(64 * kOneWaves), 0, stream>>>(a, s, p.bits);
    } else if (a.rows) {
        const dim3 blocks(static_cast<unsigned>(p.blocks)), threads(kThreads);
        k_count<<<blocks, threads, 0, stream>>>(a, s, p.bits);
        for (int pass = 0; pass < p.passes; ++pass) k_place<<<blocks, threads, 0, stream>>>(a, s, p.bits, pass);
    }
    k_sums<T><<<dim3(static_cast<unsigned>(c.blocks + p.fill_blocks)), dim3(kThreads), 0, stream>>>(a, c);
    if (c.count > 1) k_join_runs<T><<<dim3(static_cast<unsigned>(c.count - 1)), dim3(kThreads), 0, stream>>>(a, c);
    return hipGetLastError();
}

}  // namespace

size_t embedding_workspace(int64_t table_rows, int64_t cols, int64_t rows) { return plan_of(table_rows, cols, rows).bytes; }

int64_t embedding_blocks(int64_t table_rows, int64_t cols, int64_t rows) {
    const Plan p = plan_of(table_rows, cols, rows);
    return p.chunks.blocks + p.fill_blocks;
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
