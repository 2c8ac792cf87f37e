// Device kernels at the vocabulary matrix (zdo_vocab.h) for gfx950: the
// embedding lookup, its gradient over sorted tokens, and what surrounds the
// cross entropy's products (vocab_gemm.hip).
#include <hip/hip_runtime.h>

#include "device.h"
#include "vocab.h"
#include "vocab_device.h"

#pragma clang fp contract(off)

namespace zdo {
namespace {

// P consecutive elements of a row, widened: those of a 16-byte access, or 1
// where a row has fewer.
template <int P>
struct Some {
    float v[P];
};

// kOnce: non-temporally, for what a launch reads or writes once.
template <bool kOnce, typename V>
__device__ __forceinline__ V load_as(const void *p) {
    if constexpr (kOnce)
        return __builtin_nontemporal_load(static_cast<const V *>(p));
    else
        return *static_cast<const V *>(p);
}

template <int P, bool kOnce = false>
__device__ __forceinline__ Some<P> load_some(const uint16_t *p) {
    if constexpr (P == 8) {
        const u32x4 x = load_as<kOnce, loose_u32x4>(p);
        return {{lo_f32(x.x), hi_f32(x.x), lo_f32(x.y), hi_f32(x.y), lo_f32(x.z), hi_f32(x.z), lo_f32(x.w),
                 hi_f32(x.w)}};
    } else if constexpr (P == 4) {
        const u32x2 x = load_as<kOnce, loose_u32x2>(p);
        return {{lo_f32(x.x), hi_f32(x.x), lo_f32(x.y), hi_f32(x.y)}};
    } else {
        return {{h_f32(*p)}};
    }
}
template <int P, bool kOnce = false>
__device__ __forceinline__ Some<P> load_some(const float *p) {
    Some<P> e;
    if constexpr (P == 1)
        e.v[0] = *p;
    else
        for (int i = 0; i < P; i += 4) {
            const f32x4 x = load_as<kOnce, loose_f32x4>(p + i);
            for (int k = 0; k < 4; ++k)
                e.v[i + k] = x[k];
        }
    return e;
}
template <bool kOnce, typename V, typename X>
__device__ __forceinline__ void store_as(void *p, const X &x) {
    if constexpr (kOnce)
        __builtin_nontemporal_store(V(x), static_cast<V *>(p));
    else
        *static_cast<V *>(p) = x;
}

template <bool kOnce = false, int P>
__device__ __forceinline__ void store_some(uint16_t *p, const Some<P> &e) {
    if constexpr (P == 8)
        store_as<kOnce, loose_u32x4>(p, u32x4{to_bf16x2(e.v[0], e.v[1]), to_bf16x2(e.v[2], e.v[3]),
                                              to_bf16x2(e.v[4], e.v[5]), to_bf16x2(e.v[6], e.v[7])});
    else if constexpr (P == 4)
        store_as<kOnce, loose_u32x2>(p, u32x2{to_bf16x2(e.v[0], e.v[1]), to_bf16x2(e.v[2], e.v[3])});
    else
        *p = uint16_t(to_bf16x2(e.v[0], 0.0f));
}
template <bool kOnce = false, int P>
__device__ __forceinline__ void store_some(float *p, const Some<P> &e) {
    if constexpr (P == 1)
        *p = e.v[0];
    else
        for (int i = 0; i < P; i += 4)
            store_as<kOnce, loose_f32x4>(p + i, f32x4{e.v[i], e.v[i + 1], e.v[i + 2], e.v[i + 3]});
}

template <int P>
__device__ __forceinline__ void add(Some<P> &e, const Some<P> &x) {
    for (int i = 0; i < P; ++i)
        e.v[i] += x.v[i];
}

// The P columns, from `at`, that a lane takes of a row of dim >= P elements:
// from c, or the row's last P for the lane whose own, from c, are fewer. The
// first `skip` of those are the lane's before it as well, which writes the
// same values.
template <int P>
struct Columns {
    int64_t at;
    int skip;
    bool any;
    __device__ __forceinline__ Columns(int64_t c, int64_t dim)
        : at(c < dim - P ? c : dim - P), skip(c < dim ? int(c - at) : 0), any(c < dim) {}
};

// ---- lookup ------------------------------------------------------------------------------
// A wave takes kLookupChunks chunks of 64 lanes' columns of a row, all its
// loads first; a lane writes 16 bytes at once (so in fp32 it takes 4 columns), and
// non-temporally. Bound by HBM: 16,384 rows of Llama-3-8B's 4,096, W not in a cache,
// to bf16 40.4 us (79 MB read, for tokens repeat, and 134 written: 5.3 TB/s; by
// ordinary stores and half the loads 49.4), to fp32 72 us (84 by ordinary stores, 106
// with two stores a lane); one token 2.3 us.
constexpr int kLookupChunks = 4;

template <typename T, int P>
__global__ __launch_bounds__(256) void lookup_kernel(LookupArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t c0 = int64_t(blockIdx.y) * (64 * P * kLookupChunks) + lane * P;
    for (int64_t i = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); i < a.n; i += int64_t(gridDim.x) * 4) {
        const int64_t token = a.tokens[i];
        T *out = static_cast<T *>(a.out) + i * a.stride;
        const bool named = token >= 0 && token < a.vocab;
        const uint16_t *row = a.w + (named ? token : 0) * a.dim;
        Some<P> e[kLookupChunks];
#pragma unroll
        for (int k = 0; k < kLookupChunks; ++k) {
            const Columns<P> c(c0 + k * 64 * P, a.dim);
            e[k] = named && c.any ? load_some<P>(row + c.at) : Some<P>{};
        }
#pragma unroll
        for (int k = 0; k < kLookupChunks; ++k) {
            const Columns<P> c(c0 + k * 64 * P, a.dim);
            if (named)
                for (float &v : e[k].v)
                    v = a.scale * v;
            if (c.any)
                store_some<true>(out + c.at, e[k]);
        }
    }
}

// ---- sorting positions by token ------------------------------------------------------------
// A key is a token's row, or vocab for a token that names none, which come
// last and are left out by whoever reads the sorted keys.
__device__ __forceinline__ uint32_t key_of(int64_t token, int64_t vocab) {
    return token >= 0 && token < vocab ? uint32_t(token) : uint32_t(vocab);
}

// Few positions: a position's place is the number of keys below its own, or
// equal and before it. A workgroup counts for 32 positions, a lane each, each
// half of its 16 waves over a 32nd of the keys, which all of them hold in LDS.
// Bound by the comparisons (two instructions each; a read of LDS serves 4 keys):
// 8,192 positions, 67 M of them, 12 us.
__global__ __launch_bounds__(1024) void rank_kernel(const int64_t *tokens, int64_t vocab, int n, uint32_t *key_out,
                                                   uint32_t *pos_out) {
    __shared__ __align__(16) uint32_t keys[kRankMax];
    __shared__ int below[32][33];
    const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
    const int padded = (n + 31) & ~31;
    {
        // all of a thread's loads, then its stores
        constexpr int kEach = kRankMax / 1024;
        uint32_t key[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int j = k * 1024 + threadIdx.x;
            key[k] = j < n ? key_of(tokens[j], vocab) : 0xffffffffu;
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            if (k * 1024 + int(threadIdx.x) < padded)
                keys[k * 1024 + threadIdx.x] = key[k];
    }
    __syncthreads();
    const int i0 = blockIdx.x * 32, i = i0 + lane;
    const uint32_t mine = keys[i];   // i < padded
    int count = 0;
    const int blocks = padded / 32, from = blocks * part / 32, to = blocks * (part + 1) / 32;
    for (int b = from; b < to; ++b) {
        if (b * 32 == i0) {
            for (int j = 0; j < 32; ++j)
                count += keys[i0 + j] < mine || (keys[i0 + j] == mine && j < lane);
            continue;
        }
        // equal keys count where they come before: k <= mine is k < mine + 1
        const uint32_t limit = mine + (b * 32 < i0 ? 1u : 0u);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            const u32x4 k = *reinterpret_cast<const u32x4 *>(&keys[b * 32 + j]);
            count += (k.x < limit) + (k.y < limit) + (k.z < limit) + (k.w < limit);
        }
    }
    below[part][lane] = count;
    __syncthreads();
    if (part == 0 && i < n) {
        int place = 0;
        for (int w = 0; w < 32; ++w)
            place += below[w][lane];
        key_out[place] = mine;
        pos_out[place] = uint32_t(i);
    }
}

// More positions: by digits from the lowest, each pass stable: counts a workgroup,
// their sums over the workgroups, moves. A workgroup takes `items` positions, each
// of its 4 waves a quarter of them in order. 131,072 positions in two passes 34 us
// (counting 9.5, sums 8.6, moves 16.3), bound by the latency of six short launches.
struct SortArgs {
    const int64_t *tokens;  // the first pass's keys
    int64_t vocab, n, blocks;
    const uint32_t *key, *pos;
    uint32_t *key_out, *pos_out;
    uint32_t *hist;  // [bin][workgroup]: counts, then the sum of those before; and each bin's total
    int items, shift, bits;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs &a, int64_t i) {
    return a.tokens ? key_of(a.tokens[i], a.vocab) : a.key[i];
}

__global__ __launch_bounds__(256) void sort_count_kernel(SortArgs a) {
    __shared__ uint32_t count[kSortBins];
    const int bins = 1 << a.bits;
    for (int64_t b = blockIdx.x; b < a.blocks; b += gridDim.x) {
        for (int d = threadIdx.x; d < bins; d += 256)
            count[d] = 0;
        __syncthreads();
        for (int j = threadIdx.x; j < a.items; j += 256) {
            const int64_t i = b * a.items + j;
            if (i < a.n)
                atomicAdd(&count[(sort_key(a, i) >> a.shift) & (bins - 1)], 1u);
        }
        __syncthreads();
        for (int d = threadIdx.x; d < bins; d += 256)
            a.hist[d * a.blocks + b] = count[d];
        __syncthreads();
    }
}

// Each digit's counts to the sum of those before (a wave a digit), and their
// total behind them all: hist[bins * blocks + digit].
__global__ __launch_bounds__(256) void sort_scan_kernel(SortArgs a) {
    const int lane = threadIdx.x & 63, digit = blockIdx.x * 4 + (threadIdx.x >> 6), bins = 1 << a.bits;
    if (digit >= bins)
        return;
    uint32_t *row = a.hist + digit * a.blocks, before = 0;
    for (int64_t i0 = 0; i0 < a.blocks; i0 += 128) {
        const int64_t i = i0 + lane * 2;
        const uint32_t x = i < a.blocks ? row[i] : 0u, y = i + 1 < a.blocks ? row[i + 1] : 0u;
        uint32_t upto = x + y;
        for (int s = 1; s < 64; s <<= 1) {
            const uint32_t other = __shfl_up(upto, s);
            if (lane >= s)
                upto += other;
        }
        const uint32_t at = before + upto - x - y;
        if (i < a.blocks)
            row[i] = at;
        if (i + 1 < a.blocks)
            row[i + 1] = at + x;
        before += __shfl(upto, 63);
    }
    if (lane == 0)
        a.hist[bins * a.blocks + digit] = before;
}

__global__ __launch_bounds__(256) void sort_move_kernel(SortArgs a) {
    __shared__ uint32_t next[4][kSortBins];
    __shared__ uint32_t start[kSortBins], wave_sum[4];  // of each digit: where its first goes
    const int bins = 1 << a.bits, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    {
        // digits 2t and 2t + 1
        const int d = threadIdx.x * 2;
        const uint32_t x = d < bins ? a.hist[bins * a.blocks + d] : 0u;
        const uint32_t y = d + 1 < bins ? a.hist[bins * a.blocks + d + 1] : 0u;
        uint32_t upto = x + y;
        for (int s = 1; s < 64; s <<= 1) {
            const uint32_t other = __shfl_up(upto, s);
            if (lane >= s)
                upto += other;
        }
        if (lane == 63)
            wave_sum[wave] = upto;
        __syncthreads();
        uint32_t at = upto - x - y;
        for (int w = 0; w < wave; ++w)
            at += wave_sum[w];
        start[d] = at;
        start[d + 1] = at + x;
    }
    // the loop's first barrier comes before start is read
    for (int64_t b = blockIdx.x; b < a.blocks; b += gridDim.x) {
        for (int d = threadIdx.x; d < 4 * bins; d += 256)
            next[d / bins][d % bins] = 0;
        __syncthreads();
        const int64_t i0 = b * a.items + wave * (a.items / 4);
        for (int j = lane; j < a.items / 4; j += 64)
            if (i0 + j < a.n)
                atomicAdd(&next[wave][(sort_key(a, i0 + j) >> a.shift) & (bins - 1)], 1u);
        __syncthreads();
        for (int d = threadIdx.x; d < bins; d += 256) {
            uint32_t at = start[d] + a.hist[d * a.blocks + b];
            for (int w = 0; w < 4; ++w) {
                const uint32_t c = next[w][d];
                next[w][d] = at;
                at += c;
            }
        }
        __syncthreads();
        for (int j = lane; j < a.items / 4; j += 64) {
            const int64_t i = i0 + j;
            const bool in = i < a.n;
            const uint32_t key = in ? sort_key(a, i) : 0u;
            const uint32_t digit = (key >> a.shift) & (bins - 1);
            uint64_t same = __ballot(in);
            for (int bit = 0; bit < a.bits; ++bit) {
                const uint64_t ones = __ballot((digit >> bit) & 1);
                same &= (digit >> bit) & 1 ? ones : ~ones;
            }
            if (in) {
                const int leader = __builtin_ctzll(same);
                uint32_t base = 0;
                if (lane == leader)
                    base = atomicAdd(&next[wave][digit], uint32_t(__popcll(same)));
                base = __shfl(base, leader);
                const uint32_t place = base + uint32_t(__popcll(same & ((uint64_t(1) << lane) - 1)));
                a.key_out[place] = key;
                a.pos_out[place] = a.tokens ? uint32_t(i) : a.pos[i];
            }
        }
        __syncthreads();
    }
}

// ---- sums of rows ----------------------------------------------------------------------------
// A run is the sorted positions of one token. A wave sums a chunk of
// consecutive positions at its lanes' columns, whatever runs they belong to, so that
// the work is even however often a token occurs. A run within the chunk is
// finished there; of a run that goes on in other chunks the chunk's part is
// left in fp32, and join_kernel adds the parts in order.
struct SumArgs {
    RowsArgs r;
    const uint32_t *key, *pos;  // sorted
    int32_t chunk;
    int64_t chunks;
    int32_t workgroups;  // that take chunks; those behind them clear rows
    float *part;  // [chunk][2][dim]: of a run from before, of one that starts here and goes on
};

template <bool kAdd, int P>
__device__ __forceinline__ void write_row(const RowsArgs &r, uint32_t row, const Columns<P> &c, Some<P> e) {
    uint16_t *out = r.g + int64_t(row) * r.dim + c.at;
    for (float &v : e.v)
        v = r.scale * v;
    if constexpr (kAdd) {
        if (c.skip == 0) {
            const Some<P> old = load_some<P>(out);
            for (int i = 0; i < P; ++i)
                e.v[i] = old.v[i] + e.v[i];
            store_some(out, e);
        } else {
            // another wave may be adding to the columns that are not this lane's own
            for (int i = 1; i < P; ++i)
                if (i >= c.skip)
                    store_some(out + i, Some<1>{{h_f32(out[i]) + e.v[i]}});
        }
    } else {
        store_some(out, e);
    }
}

// Few tokens, without a sort: a workgroup takes a position at its lanes' columns,
// looks for its token among all positions, 64 a ballot, leaves if one before it
// has the same, and else sums the rows of those that have it in their order, a
// quarter by each of its 4 waves. The workgroups behind the first `workgroups`
// clear the rows that no token names, 64 each, a row a wave. Bound by latency for
// small matrices (300 tokens, 2,003 rows of 250 columns 4.8 us), by clearing for
// large ones.
template <typename T, int P, bool kAdd>
__global__ __launch_bounds__(256) void few_kernel(RowsArgs r, int workgroups) {
    __shared__ uint16_t list[kFewTokens];
    __shared__ Some<P> red[3][64];
    __shared__ uint32_t is_named[64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Columns<P> c((int64_t(blockIdx.y) * 64 + lane) * P, r.dim);
    const T *x = static_cast<const T *>(r.x) + c.at;
    const int n = int(r.n);
    int64_t tokens[kFewTokens / 64];
#pragma unroll
    for (int k = 0; k < kFewTokens / 64; ++k)
        tokens[k] = k * 64 + lane < n ? r.tokens[k * 64 + lane] : -1;
    if (!kAdd && int(blockIdx.x) >= workgroups) {
        const int64_t rows = r.numel / r.dim, groups = (rows + 63) / 64;
        for (int64_t g = blockIdx.x - workgroups; g < groups; g += gridDim.x - workgroups) {
            if (threadIdx.x < 64)
                is_named[threadIdx.x] = 0;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kFewTokens / 64; ++k)
                if (tokens[k] >= g * 64 && tokens[k] < g * 64 + 64 && tokens[k] < r.vocab)
                    is_named[tokens[k] - g * 64] = 1;   // by whoever has it
            __syncthreads();
            for (int k = wave; k < 64 && g * 64 + k < rows; k += 4)
                if (!is_named[k] && c.any)
                    store_some(r.g + (g * 64 + k) * r.dim + c.at, Some<P>{});
            if (g == groups - 1 && blockIdx.y == 0)
                for (int64_t i = rows * r.dim + threadIdx.x; i < r.numel; i += 256)
                    r.g[i] = 0;
            __syncthreads();
        }
        return;
    }
    for (int i = blockIdx.x; i < n; i += workgroups) {
        const int64_t token = r.tokens[i];
        if (token < 0 || token >= r.vocab)
            continue;
        int total = 0;
        bool first = true;
#pragma unroll
        for (int k = 0; k < kFewTokens / 64; ++k) {
            const int j = k * 64 + lane;
            const bool same = tokens[k] == token;
            const uint64_t all = __ballot(same);
            first = first && !__any(same && j < i);
            if (same)
                list[total + __popcll(all & ((uint64_t(1) << lane) - 1))] = uint16_t(j);   // by each wave alike
            total += __popcll(all);
        }
        if (!first)
            continue;
        __syncthreads();
        const int to = total * (wave + 1) / 4;
        Some<P> e{};
        if (c.any) {
            int k = total * wave / 4;
            for (; k + 8 <= to; k += 8) {
                Some<P> v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    v[u] = load_some<P>(x + int64_t(list[k + u]) * r.stride);
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    add(e, v[u]);
            }
            for (; k < to; ++k)
                add(e, load_some<P>(x + int64_t(list[k]) * r.stride));
        }
        if (wave < 3)
            red[wave][lane] = e;
        __syncthreads();
        if (wave == 3 && c.any) {   // the last quarter is never empty
            Some<P> sum = red[0][lane];
            add(sum, red[1][lane]);
            add(sum, red[2][lane]);
            add(sum, e);
            write_row<kAdd>(r, uint32_t(token), c, sum);
        }
        __syncthreads();
    }
}

// The first of key[from, to) that is not below `limit`: all 64 lanes probe.
__device__ __forceinline__ int64_t first_not_below(const uint32_t *key, int64_t from, int64_t to, uint32_t limit) {
    const int lane = threadIdx.x & 63;
    while (from < to) {
        const int64_t step = (to - from + 63) / 64, probe = from + (lane + 1) * step - 1;
        const int below = __popcll(__ballot(probe < to && key[probe] < limit));
        from += below * step;
        to = to < from + step - 1 ? to : from + step - 1;
    }
    return to;
}

// Clears the rows of the parameter that no token names, those behind the
// vocabulary among them, 64 a workgroup: lane l looks for row l among the keys.
// Beside the sums, for both wait for memory in different ways (8,192 tokens of
// GPT-2 small 34.6 us, 37.2 with all rows cleared beside the sort; Llama-3-8B,
// bound by writing a gigabyte, 232 and 228; every 2004th row a workgroup, so that
// all write one region together, 249).
constexpr int kClearRows = 64;

template <int P>
__device__ __forceinline__ void clear_unnamed(const SumArgs &a, const Columns<P> &c) {
    const RowsArgs &r = a.r;
    const int64_t rows = r.numel / r.dim, groups = (rows + kClearRows - 1) / kClearRows;
    for (int64_t g = blockIdx.x - a.workgroups; g < groups; g += gridDim.x - a.workgroups) {
        const int64_t row0 = g * kClearRows, row = row0 + (threadIdx.x & 63);
        const int64_t behind = row0 + kClearRows < r.vocab ? row0 + kClearRows : r.vocab;
        int64_t lo = r.n, end = r.n;
        if (row0 < r.vocab) {
            lo = first_not_below(a.key, 0, r.n, uint32_t(row0));
            end = first_not_below(a.key, lo, r.n, uint32_t(behind));
        }
        for (int64_t hi = end; lo < hi;) {
            const int64_t mid = (lo + hi) / 2;
            if (a.key[mid] < uint32_t(row))
                lo = mid + 1;
            else
                hi = mid;
        }
        const bool named = lo < end && a.key[lo] == uint32_t(row);
        for (uint64_t left = __ballot(row < rows && !named); left; left &= left - 1)
            if (c.any)
                store_some(r.g + (row0 + __builtin_ctzll(left)) * r.dim + c.at, Some<P>{});
        if (g == groups - 1 && blockIdx.y == 0)
            for (int64_t i = rows * r.dim + threadIdx.x; i < r.numel; i += blockDim.x)
                r.g[i] = 0;
    }
}

// Bound by HBM: 131,072 fp32 rows of 1,024 columns in random order 102 us (507 MB
// read, 74 written: 5.7 TB/s); 8,192 rows of Llama-3-8B and clearing the rest 204 us
// (1.06 GB written, 64 MB read: 5.5 TB/s).
template <typename T, int P, bool kAdd, bool kOnce>
__global__ __launch_bounds__(256) void runs_kernel(SumArgs a) {
    const RowsArgs &r = a.r;
    const int lane = threadIdx.x & 63;
    const Columns<P> c((int64_t(blockIdx.y) * blockDim.x + threadIdx.x) * P, r.dim);
    const T *x = static_cast<const T *>(r.x) + c.at;
    const uint32_t none = uint32_t(r.vocab);
    if (!kAdd && int(blockIdx.x) >= a.workgroups) {
        clear_unnamed(a, c);
        return;
    }
    for (int64_t b = blockIdx.x; b < a.chunks; b += a.workgroups) {
        const int64_t i0 = b * a.chunk;
        const int in = r.n - i0 < a.chunk ? int(r.n - i0) : a.chunk;
        const uint32_t my_key = lane < in ? a.key[i0 + lane] : none, my_pos = lane < in ? a.pos[i0 + lane] : 0u;
        const uint32_t before = i0 > 0 ? a.key[i0 - 1] : none, after = i0 + in < r.n ? a.key[i0 + in] : none;
        const int named = __popcll(__ballot(my_key != none));   // those without a row come last
        Some<P> e{};
        bool from_before = false;
        for (int j0 = 0; j0 < named; j0 += 8) {
            Some<P> v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int j = j0 + k < named ? j0 + k : named - 1;
                v[k] = c.any ? load_some<P, kOnce>(x + int64_t(__builtin_amdgcn_readlane(my_pos, j)) * r.stride)
                             : Some<P>{};
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int j = j0 + k;
                if (j >= named)
                    break;
                const uint32_t key = __builtin_amdgcn_readlane(my_key, j);
                if (j == 0)
                    from_before = key == before;
                add(e, v[k]);
                const bool last = j == in - 1;
                if ((last ? after : uint32_t(__builtin_amdgcn_readlane(my_key, last ? j : j + 1))) == key && !last)
                    continue;
                const bool goes_on = last && after == key;
                if (c.any) {
                    if (from_before || goes_on)
                        store_some(a.part + (2 * b + !from_before) * r.dim + c.at, e);
                    else
                        write_row<kAdd>(r, key, c, e);
                }
                from_before = false;
                e = Some<P>{};
            }
        }
    }
}

// A run that starts in chunk b and goes on: its parts, a quarter by each of
// the workgroup's waves, then the four. Bound by the latency of the longest run's
// loads: 8,192 tokens of text, one of them 8% of all, 6 us for GPT-2 small.
template <int P, bool kAdd>
__global__ __launch_bounds__(256) void join_kernel(SumArgs a) {
    __shared__ Some<P> red[3][64];
    const RowsArgs &r = a.r;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Columns<P> c((int64_t(blockIdx.y) * 64 + lane) * P, r.dim);
    for (int64_t b = blockIdx.x; b + 1 < a.chunks; b += gridDim.x) {
        const int64_t next = (b + 1) * a.chunk;
        const uint32_t key = a.key[next - 1];
        const bool from_before = b > 0 && a.key[b * a.chunk] == key && a.key[b * a.chunk - 1] == key;
        if (key == uint32_t(r.vocab) || a.key[next] != key || from_before)
            continue;
        // chunks b + 1 .. b + whole are all this run's, and one more begins with it
        // unless the run ends with them
        int64_t whole = 0;
        for (;;) {
            const int64_t last = (b + 2 + whole + lane) * a.chunk - 1;
            const uint64_t other = ~__ballot(last < r.n && a.key[last] == key);
            if (other) {
                whole += __builtin_ctzll(other);
                break;
            }
            whole += 64;
        }
        const int64_t begin = (b + 1 + whole) * a.chunk;
        const int64_t parts = whole + (begin < r.n && a.key[begin] == key);   // of chunks b + 1, b + 2, ...
        Some<P> e{};
        if (c.any) {
            if (wave == 0)
                e = load_some<P, true>(a.part + (2 * b + 1) * r.dim + c.at);
            const float *part = a.part + 2 * (b + 1) * r.dim + c.at;
            const int64_t to = parts * (wave + 1) / 4;
            int64_t k = parts * wave / 4;
            for (; k + 8 <= to; k += 8) {
                Some<P> v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    v[u] = load_some<P, true>(part + 2 * (k + u) * r.dim);
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    add(e, v[u]);
            }
            for (; k < to; ++k)
                add(e, load_some<P, true>(part + 2 * k * r.dim));
        }
        if (wave > 0)
            red[wave - 1][lane] = e;
        __syncthreads();
        if (wave == 0 && c.any) {
            for (int w = 0; w < 3; ++w)
                add(e, red[w][lane]);
            write_row<kAdd>(r, key, c, e);
        }
        __syncthreads();
    }
}

// Few workgroups clear faster than many: 1 GB by 256 in 160 us, by 512 in 195, by
// 4096 in 232, non-temporally in 166 to 264.
__global__ __launch_bounds__(256) void zero_kernel(uint16_t *p, int64_t n) {
    const int64_t head = (16 - (reinterpret_cast<uintptr_t>(p) & 15)) % 16 / 2, from = head < n ? head : n;
    const int64_t chunks = (n - from) / 8, upto = from + chunks * 8;
    if (blockIdx.x == 0) {
        if (int64_t(threadIdx.x) < from)
            p[threadIdx.x] = 0;
        if (upto + threadIdx.x < n)
            p[upto + threadIdx.x] = 0;
    }
    u32x4 *q = reinterpret_cast<u32x4 *>(p + from);
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < chunks; i += int64_t(gridDim.x) * 256)
        q[i] = u32x4{0, 0, 0, 0};
}

// ---- around the cross entropy's products --------------------------------------------------------

// Rows of dim elements, one every `stride`, to `padded` rows of kdim, zeros behind
// the elements and the rows, and where targets (if given) names no row; `copies`
// times, one behind the other.
struct Pack {
    const uint16_t *from;
    int64_t stride, rows, padded;
    const int64_t *targets;
    uint16_t *to;
    int32_t copies, workgroups;
};

// Two packings in one launch (the second may be empty). Bound by HBM: 8,192 rows of
// 768 columns, read and written, 6.6 us.
__global__ __launch_bounds__(256) void pack_kernel(Pack one, Pack two, int64_t dim, int64_t kdim, int64_t vocab) {
    const bool second = int(blockIdx.x) >= one.workgroups;
    const Pack p = second ? two : one;
    const int64_t per = kdim / 8, first = blockIdx.x - (second ? one.workgroups : 0);
    for (int64_t i = first * 256 + threadIdx.x; i < p.padded * per; i += int64_t(p.workgroups) * 256) {
        const int64_t r = i / per, c = i % per * 8;
        const uint16_t *from = p.from + r * p.stride + c;
        bool keep = r < p.rows;
        if (keep && p.targets) {
            const int64_t target = p.targets[r];
            keep = target >= 0 && target < vocab;
        }
        u32x4 x = {0, 0, 0, 0};
        if (keep && c + 8 <= dim)
            x = *reinterpret_cast<const loose_u32x4 *>(from);
        else if (keep)
            for (int k = 0; k < 7; ++k)
                if (c + k < dim)
                    x[k >> 1] |= uint32_t(from[k]) << (k & 1) * 16;
        for (int copy = 0; copy < p.copies; ++copy)
            *reinterpret_cast<u32x4 *>(p.to + (copy * p.padded + r) * kdim + c) = x;
    }
}

// The softmax's statistics of all tiles to each token's loss and lse: kTokens of
// them a workgroup, 256 / kTokens threads each over the tiles in turn. Bound by
// latency for one token a workgroup (GPT-2 small 3.9 us), by reading the statistics
// for 16 (8,192 tokens 7 us, 12.9 MB).
template <int kTokens>
__global__ __launch_bounds__(256) void combine_kernel(CeArgs a, const float2 *part, int64_t tiles, const float *pick) {
    constexpr int kEach = 256 / kTokens;
    __shared__ float2 red[kEach][kTokens];
    const int token = threadIdx.x % kTokens, slice = threadIdx.x / kTokens;
    for (int64_t t0 = int64_t(blockIdx.x) * kTokens; t0 < a.n; t0 += int64_t(gridDim.x) * kTokens) {
        const int64_t t = t0 + token;
        float2 all = {-INFINITY, 0.0f};
        if (t < a.n)
            for (int64_t k = slice; k < tiles; k += 8 * kEach) {
                float2 x[8];   // loads first
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    x[u] = k + u * kEach < tiles ? part[(k + u * kEach) * a.n + t] : float2{-INFINITY, 0.0f};
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    all = join_softmax(all, x[u]);
            }
        red[slice][token] = all;
        __syncthreads();
        for (int half = kEach / 2; half > 0; half /= 2) {
            if (slice < half)
                red[slice][token] = join_softmax(red[slice][token], red[slice + half][token]);
            __syncthreads();
        }
        if (slice == 0 && t < a.n) {
            all = red[0][token];
            // not by way of lse, where the largest logit's last bit may be more than the
            // whole loss; with an infinite or NaN logit both ways give the same
            const float log_sum = logf(all.y);
            const int64_t target = a.targets[t];
            a.lse[t] = all.x + log_sum;
            a.loss[t] = target >= 0 && target < a.vocab ? (all.x - pick[t]) + log_sum : 0.0f;
        }
        __syncthreads();
    }
}

// The sum of `splits` rows' columns at p, `step` elements from each other, added in
// their order, 8 loads at a time.
template <int P>
__device__ __forceinline__ Some<P> sum_of(const float *p, int64_t splits, int64_t step) {
    Some<P> e{};
    int64_t s = 0;
    for (; s + 8 <= splits; s += 8) {
        Some<P> v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] = load_some<P, true>(p + (s + u) * step);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            add(e, v[u]);
    }
    for (; s < splits; ++s)
        add(e, load_some<P, true>(p + s * step));
    return e;
}

// The splits' sums of grad_hidden, added in their order, and the rest of the
// target's d times its row; rounded. So the largest term of most sums is exact.
// Bound by reading: 8,192 tokens of GPT-2 small, two splits, 13.5 us (50 MB of sums,
// 13 of rows of W).
template <typename T, int P>
__global__ __launch_bounds__(256) void hidden_kernel(CeArgs a, const float *sum, int64_t splits, int64_t kdim,
                                                    const float *rest) {
    const int64_t per = (a.dim + P - 1) / P;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < a.n * per; i += int64_t(gridDim.x) * 256) {
        const int64_t r = i / per;
        const Columns<P> c(i % per * P, a.dim);
        const int64_t target = a.targets[r];
        Some<P> e{};
        if (target >= 0 && target < a.vocab) {
            const Some<P> w = load_some<P>(a.w + target * a.dim + c.at);
            e = sum_of<P>(sum + r * kdim + c.at, splits, a.n * kdim);
            const float x = rest[r];
            for (int k = 0; k < P; ++k)
                e.v[k] += x * w.v[k];
        }
        store_some(static_cast<T *>(a.grad_hidden) + r * a.grad_hidden_stride + c.at, e);
    }
}

// The splits' sums of a piece of W's gradient, added in their order. Bound by
// reading them, from the caches they were just written through.
template <int P, bool kAdd>
__global__ __launch_bounds__(256) void row_sums_kernel(RowsArgs r, const float *sum, int64_t splits, int64_t rows,
                                                      int64_t kdim) {
    const int64_t per = (r.dim + P - 1) / P;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < rows * per; i += int64_t(gridDim.x) * 256) {
        const int64_t row = i / per;
        const Columns<P> c(i % per * P, r.dim);
        write_row<kAdd>(r, uint32_t(row), c, sum_of<P>(sum + row * kdim + c.at, splits, rows * kdim));
    }
}

unsigned grid_of(int64_t blocks) { return unsigned(std::min<int64_t>(blocks, std::min<int64_t>(kMaxGrid, 1 << 20))); }

// The packings that a product needs, in one launch if there are any.
void launch_pack(Pack one, Pack two, const CeArgs &a, const CeLayout &l, hipStream_t stream) {
    for (Pack *p : {&one, &two})
        p->workgroups = int32_t(grid_of(ceil_div(p->padded * l.kdim, 2048)));
    if (one.workgroups + two.workgroups > 0)
        pack_kernel<<<unsigned(one.workgroups + two.workgroups), 256, 0, stream>>>(one, two, a.dim, l.kdim, a.vocab);
}

// Few tokens and W not in place: its rows are read as they lie by
// thin_score_kernel rather than copied (16 tokens of Llama-3-8B, W off by an
// element: 485 us, 648 with the copy; 10,007 rows of 1,537: 33 and 38. In place
// the products are as fast: 184 and 182, GPT-2 small 23.5 and 21.8).
bool by_rows(const CeArgs &a) { return a.n <= kThinTokens && !a.in_place; }

// A piece of W as the products take it: in place, or the copy that `p` describes.
const uint16_t *piece_of(const CeArgs &a, const CeLayout &l, int64_t row0, int64_t rows, Pack &p) {
    p = Pack{};
    const uint16_t *from = a.w + row0 * a.dim;
    if (a.in_place)
        return from;
    uint16_t *w = reinterpret_cast<uint16_t *>(a.workspace + l.w);
    p = Pack{from, a.dim, rows, rows, nullptr, w, 1, 0};
    return w;
}

}  // namespace

hipError_t launch_zero(uint16_t *p, int64_t n, hipStream_t stream) {
    if (n > 0)
        zero_kernel<<<grid_of(std::min<int64_t>(256, ceil_div(n, 2048))), 256, 0, stream>>>(p, n);
    return hipGetLastError();
}

hipError_t launch_lookup(const LookupArgs &a, hipStream_t stream) {
    if (a.n == 0)
        return hipSuccess;
    const int P = a.dim < 8 ? 1 : a.f32 ? 4 : 8;
    const dim3 grid(grid_of(ceil_div(a.n, 4)), unsigned(ceil_div(a.dim, 64 * P * kLookupChunks)));
    auto go = [&](auto kernel) { kernel<<<grid, 256, 0, stream>>>(a); };
    if (a.f32)
        P == 1 ? go(lookup_kernel<float, 1>) : go(lookup_kernel<float, 4>);
    else
        P == 1 ? go(lookup_kernel<uint16_t, 1>) : go(lookup_kernel<uint16_t, 8>);
    return hipGetLastError();
}

// The sums of rows, P columns a lane.
template <typename T, int P, bool kAdd>
void launch_sums(SumArgs s, hipStream_t stream) {
    const int64_t waves = std::min<int64_t>(4, ceil_div(s.r.dim, 64 * P));
    s.workgroups = int32_t(grid_of(s.chunks));
    const unsigned clear = kAdd ? 0 : grid_of(ceil_div(s.r.numel / s.r.dim, kClearRows));
    const dim3 grid(unsigned(s.workgroups) + clear, unsigned(ceil_div(s.r.dim, 64 * P * waves)));
    // rows that the 256 MB Infinity Cache can hold are mostly still in it
    // (GPT-2 small's 12 MB: 8.2 us, 10.0 non-temporally); more are not (537 MB:
    // 121 us, 101 non-temporally)
    if (P > 1 && s.r.n * s.r.dim * int64_t(sizeof(T)) > int64_t(1) << 28)
        runs_kernel<T, P, kAdd, (P > 1)><<<grid, unsigned(64 * waves), 0, stream>>>(s);
    else
        runs_kernel<T, P, kAdd, false><<<grid, unsigned(64 * waves), 0, stream>>>(s);
    if (s.chunks > 1) {
        constexpr int J = P == 1 ? 1 : 4;   // of fp32
        join_kernel<J, kAdd><<<dim3(unsigned(s.workgroups), unsigned(ceil_div(s.r.dim, 64 * J))), 256, 0, stream>>>(s);
    }
}

hipError_t launch_rows(const RowsArgs &a, hipStream_t stream) {
    if (a.n == 0)
        return a.accumulate ? hipSuccess : launch_zero(a.g, a.numel, stream);
    auto one_of = [&](auto f32, auto bf16, auto f32_add, auto bf16_add) {
        return a.accumulate ? (a.f32 ? f32_add : bf16_add) : (a.f32 ? f32 : bf16);
    };
    if (a.n <= kFewTokens) {
        const int P = a.dim < 8 ? 1 : a.f32 ? 4 : 8, workgroups = int(grid_of(a.n));
        const dim3 grid(unsigned(workgroups) + (a.accumulate ? 0 : grid_of(ceil_div(a.numel / a.dim, 64))),
                        unsigned(ceil_div(a.dim, 64 * P)));
        if (P == 1)
            one_of(few_kernel<float, 1, false>, few_kernel<uint16_t, 1, false>, few_kernel<float, 1, true>,
                   few_kernel<uint16_t, 1, true>)<<<grid, 256, 0, stream>>>(a, workgroups);
        else
            one_of(few_kernel<float, 4, false>, few_kernel<uint16_t, 8, false>, few_kernel<float, 4, true>,
                   few_kernel<uint16_t, 8, true>)<<<grid, 256, 0, stream>>>(a, workgroups);
        return hipGetLastError();
    }
    const RowsLayout l = rows_layout(a.n, a.dim);
    char *ws = static_cast<char *>(a.workspace);
    auto u32 = [&](int64_t at) { return reinterpret_cast<uint32_t *>(ws + at); };
    int set = 0;
    if (a.n <= kRankMax) {
        rank_kernel<<<unsigned(ceil_div(a.n, 32)), 1024, 0, stream>>>(a.tokens, a.vocab, int(a.n), u32(l.key[0]),
                                                                     u32(l.pos[0]));
    } else {
        const int bits = 64 - __builtin_clzll(uint64_t(a.vocab)), passes = (bits + 8) / 9;
        const int digit = (bits + passes - 1) / passes;
        SortArgs p{};
        p.vocab = a.vocab;
        p.n = a.n;
        p.blocks = l.blocks;
        p.hist = u32(l.hist);
        p.items = l.items;
        p.bits = digit;
        for (int k = 0; k < passes; ++k) {
            p.tokens = k ? nullptr : a.tokens;
            set = k & 1;
            p.key = u32(l.key[set ^ 1]);
            p.pos = u32(l.pos[set ^ 1]);
            p.key_out = u32(l.key[set]);
            p.pos_out = u32(l.pos[set]);
            p.shift = k * digit;
            sort_count_kernel<<<grid_of(l.blocks), 256, 0, stream>>>(p);
            sort_scan_kernel<<<unsigned(ceil_div(int64_t(1) << digit, 4)), 256, 0, stream>>>(p);
            sort_move_kernel<<<grid_of(l.blocks), 256, 0, stream>>>(p);
        }
    }
    SumArgs s{};
    s.r = a;
    s.key = u32(l.key[set]);
    s.pos = u32(l.pos[set]);
    s.chunk = l.chunk;
    s.chunks = l.chunks;
    s.part = reinterpret_cast<float *>(ws + l.part);
    if (a.dim < 8)
        one_of(launch_sums<float, 1, false>, launch_sums<uint16_t, 1, false>, launch_sums<float, 1, true>,
               launch_sums<uint16_t, 1, true>)(s, stream);
    else
        one_of(launch_sums<float, 4, false>, launch_sums<uint16_t, 8, false>, launch_sums<float, 4, true>,
               launch_sums<uint16_t, 8, true>)(s, stream);
    return hipGetLastError();
}

hipError_t launch_ce(const CeArgs &a, hipStream_t stream) {
    if (a.n == 0)
        return hipSuccess;
    const CeLayout &l = a.layout;
    GemmArgs g{};
    g.b = a.hidden;
    g.ldb = a.n <= 1 ? a.dim : a.hidden_stride;
    g.n = a.n;
    g.splits = 1;
    g.targets = a.targets;
    g.vocab = a.vocab;
    g.part = reinterpret_cast<float2 *>(a.workspace + l.part);
    g.pick = reinterpret_cast<float *>(a.workspace + l.pick);
    int64_t tiles = 0;
    if (by_rows(a)) {
        g.a = a.w;
        g.lda = a.dim;
        g.m = a.vocab;
        g.k = a.dim;
        if (hipError_t e = launch_thin_score(g, stream); e != hipSuccess)
            return e;
        tiles = ceil_div(g.m, kThinRows);
    } else {
        Pack hidden{}, w;
        if (a.dim % kDepth || g.ldb % 8 || g.ldb > int64_t(1) << 21 || (reinterpret_cast<uintptr_t>(a.hidden) & 15)) {
            uint16_t *h = reinterpret_cast<uint16_t *>(a.workspace + l.hidden);
            hidden = Pack{a.hidden, a.hidden_stride, a.n, a.n, nullptr, h, 1, 0};
            g.b = h;
            g.ldb = l.kdim;
        }
        g.lda = l.kdim;   // dim where W is used in place
        g.k = l.kdim;
        // in place, W needs no pieces but for the tiles' numbers
        const int64_t rows = a.in_place ? std::max(l.piece, (int64_t(1) << 36) / l.npad / 256 * 256) : l.piece;
        for (g.row0 = 0; g.row0 < a.vocab; g.row0 += rows) {
            g.m = std::min(rows, a.vocab - g.row0);
            g.a = piece_of(a, l, g.row0, g.m, w);
            launch_pack(hidden, w, a, l, stream);
            hidden = Pack{};
            g.tile0 = tiles;
            if (hipError_t e = launch_gemm(kScore, g, stream); e != hipSuccess)
                return e;
            tiles += ceil_div(g.m, tile_rows(g.m, g.n));
        }
    }
    // few tokens: a workgroup each (GPT-2 small, whole calls: 32 tokens 23.0 us, 16 a
    // workgroup 24.7; 256 31.7 both ways; 8,192 622 and 596)
    if (a.n <= 256)
        combine_kernel<1><<<grid_of(a.n), 256, 0, stream>>>(a, g.part, tiles, g.pick);
    else
        combine_kernel<16><<<grid_of(ceil_div(a.n, 16)), 256, 0, stream>>>(a, g.part, tiles, g.pick);
    return hipGetLastError();
}

hipError_t launch_ce_grad(const CeArgs &a, hipStream_t stream) {
    if (a.grads && !a.accumulate) {
        const int64_t kept = a.n == 0 ? 0 : a.vocab * a.dim;
        if (hipError_t e = launch_zero(a.grads + kept, a.numel - kept, stream); e != hipSuccess)
            return e;
    }
    if (a.n == 0)
        return hipSuccess;
    const CeLayout &l = a.layout;
    auto u16 = [&](int64_t at) { return reinterpret_cast<uint16_t *>(a.workspace + at); };
    uint16_t *hidden = u16(l.hidden), *d = u16(l.d);
    float *sum = reinterpret_cast<float *>(a.workspace + l.sum);
    // hidden with zeros where no target is: whatever those rows hold, nothing of it is left
    Pack packed{a.hidden, a.hidden_stride, a.n, l.npad, a.targets, hidden, int32_t(a.grads ? l.parts : 1), 0}, piece;
    float *rest = reinterpret_cast<float *>(a.workspace + l.rest);
    for (int64_t row0 = 0; row0 < a.vocab; row0 += l.piece) {
        const int64_t rows = std::min(l.piece, a.vocab - row0);
        const uint16_t *w = piece_of(a, l, row0, rows, piece);
        launch_pack(packed, piece, a, l, stream);
        packed = Pack{};
        GemmArgs g{};
        g.a = w;
        g.b = hidden;
        g.lda = l.kdim;
        g.ldb = l.kdim;
        g.m = rows;
        g.n = a.n;
        g.k = l.kdim;
        g.splits = 1;
        g.targets = a.targets;
        g.row0 = row0;
        g.vocab = a.vocab;
        g.lse = a.lse;
        g.weight = a.grad_loss;
        g.d = d;
        g.low = a.grads && l.parts == 2 ? d + l.npad * l.vpad : nullptr;
        g.ldd = l.vpad;
        g.rest = rest;
        if (hipError_t e = launch_gemm(kDiff, g, stream); e != hipSuccess)
            return e;
        if (a.grad_hidden) {
            GemmArgs h{};
            h.a = w;
            h.b = d;
            h.lda = l.kdim;
            h.ldb = l.vpad;
            h.m = a.dim;
            h.n = a.n;
            h.k = rows;
            h.splits = int32_t(l.splits);
            h.sum = sum;
            h.lds = l.kdim;
            h.first = row0 == 0;
            if (hipError_t e = launch_gemm(kSum, h, stream); e != hipSuccess)
                return e;
        }
        if (a.grads) {
            GemmArgs r{};
            r.a = hidden;
            r.b = d;
            r.lda = l.kdim;
            r.ldb = l.vpad;
            r.m = a.dim;
            r.n = rows;
            r.k = l.parts * l.npad;
            r.splits = int32_t(l.row_splits);
            r.rows = a.grads + row0 * a.dim;
            r.accumulate = a.accumulate;
            r.sum = reinterpret_cast<float *>(a.workspace + l.row_sum);
            r.lds = l.kdim;
            r.first = 1;
            if (hipError_t e = launch_gemm(l.row_splits > 1 ? kParts : kRows, r, stream); e != hipSuccess)
                return e;
            if (l.row_splits > 1) {
                RowsArgs to{};
                to.g = r.rows;
                to.dim = a.dim;
                to.scale = 1.0f;
                auto go = [&](auto kernel) {
                    kernel<<<grid_of(ceil_div(rows * l.kdim, 2048)), 256, 0, stream>>>(to, r.sum, l.row_splits, rows,
                                                                                       l.kdim);
                };
                if (a.accumulate)
                    a.dim >= 8 ? go(row_sums_kernel<8, true>) : go(row_sums_kernel<1, true>);
                else
                    a.dim >= 8 ? go(row_sums_kernel<8, false>) : go(row_sums_kernel<1, false>);
            }
        }
    }
    if (a.grad_hidden) {
        const unsigned grid = grid_of(ceil_div(a.n * l.kdim, 2048));
        auto go = [&](auto kernel) { kernel<<<grid, 256, 0, stream>>>(a, sum, l.splits, l.kdim, rest); };
        if (a.f32)
            a.dim >= 8 ? go(hidden_kernel<float, 8>) : go(hidden_kernel<float, 1>);
        else
            a.dim >= 8 ? go(hidden_kernel<uint16_t, 8>) : go(hidden_kernel<uint16_t, 1>);
    }
    return hipGetLastError();
}

}  // namespace zdo
