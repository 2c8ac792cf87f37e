// Device kernels at the vocabulary matrix (zdo_vocab.h) for gfx950: the
// embedding lookup, its gradient over sorted tokens, and what surrounds the
// cross entropy's products (vocab_gemm.hip).
//
// Rows of the matrix start at any element, so 16-byte accesses are written
// for 2-byte alignment; gfx950 takes them in one instruction.
#include <hip/hip_runtime.h>

#include "device.h"
#include "vocab.h"

#pragma clang fp contract(off)

namespace zdo {
namespace {

struct __attribute__((packed, aligned(2))) Loose16 {
    u32x4 v;
};
struct __attribute__((packed, aligned(4))) LooseF4 {
    f32x4 v;
};

// 8 elements of a row, or the first `count` of them and zeros.
struct Eight {
    float v[8];
};

__device__ __forceinline__ Eight widen(u32x4 x) {
    return {{lo_f32(x.x), hi_f32(x.x), lo_f32(x.y), hi_f32(x.y), lo_f32(x.z), hi_f32(x.z), lo_f32(x.w), hi_f32(x.w)}};
}

__device__ __forceinline__ Eight read8(const uint16_t *p, int count) {
    if (count >= 8)
        return widen(reinterpret_cast<const Loose16 *>(p)->v);
    Eight e{};
    for (int i = 0; i < 7; ++i)
        if (i < count)
            e.v[i] = h_f32(p[i]);
    return e;
}

__device__ __forceinline__ Eight read8(const float *p, int count) {
    Eight e{};
    if (count >= 8) {
        const f32x4 a = reinterpret_cast<const LooseF4 *>(p)->v, b = reinterpret_cast<const LooseF4 *>(p + 4)->v;
        for (int i = 0; i < 4; ++i) {
            e.v[i] = a[i];
            e.v[4 + i] = b[i];
        }
        return e;
    }
    for (int i = 0; i < 7; ++i)
        if (i < count)
            e.v[i] = p[i];
    return e;
}

__device__ __forceinline__ void write8(uint16_t *p, const Eight &e, int count) {
    u32x4 x;
    for (int i = 0; i < 4; ++i)
        x[i] = to_bf16x2(e.v[2 * i], e.v[2 * i + 1]);
    if (count >= 8)
        reinterpret_cast<Loose16 *>(p)->v = x;
    else
        for (int i = 0; i < 7; ++i)
            if (i < count)
                p[i] = uint16_t(x[i >> 1] >> (i & 1) * 16);
}

__device__ __forceinline__ void write8(float *p, const Eight &e, int count) {
    if (count >= 8) {
        reinterpret_cast<LooseF4 *>(p)->v = f32x4{e.v[0], e.v[1], e.v[2], e.v[3]};
        reinterpret_cast<LooseF4 *>(p + 4)->v = f32x4{e.v[4], e.v[5], e.v[6], e.v[7]};
    } else {
        for (int i = 0; i < 7; ++i)
            if (i < count)
                p[i] = e.v[i];
    }
}

// How many of the 8 elements from column c a row of dim elements has.
__device__ __forceinline__ int columns_left(int64_t dim, int64_t c) {
    return dim - c >= 8 ? 8 : dim > c ? int(dim - c) : 0;
}

// ---- lookup ------------------------------------------------------------------------------
// A wave takes kLookupWide columns of a row, all its loads first.
constexpr int kLookupChunks = 4, kLookupWide = 512 * kLookupChunks;

template <typename T>
__global__ __launch_bounds__(256) void lookup_kernel(LookupArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t c0 = int64_t(blockIdx.y) * kLookupWide + lane * 8;
    for (int64_t i = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); i < a.n; i += int64_t(gridDim.x) * 4) {
        const int64_t token = a.tokens[i];
        T *out = static_cast<T *>(a.out) + i * a.stride;
        const bool named = token >= 0 && token < a.vocab;
        const uint16_t *row = a.w + (named ? token : 0) * a.dim;
        Eight e[kLookupChunks];
#pragma unroll
        for (int k = 0; k < kLookupChunks; ++k) {
            const int64_t c = c0 + k * 512;
            e[k] = named && c < a.dim ? read8(row + c, columns_left(a.dim, c)) : Eight{};
        }
#pragma unroll
        for (int k = 0; k < kLookupChunks; ++k) {
            const int64_t c = c0 + k * 512;
            if (c >= a.dim)
                break;
            if (named)
                for (float &v : e[k].v)
                    v = a.scale * v;
            write8(out + c, e[k], columns_left(a.dim, c));
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
// equal and before it. A workgroup counts for 64 positions, its 16 waves each
// over a sixteenth of the keys, which all of them hold in LDS.
__global__ __launch_bounds__(1024) void rank_kernel(const int64_t *tokens, int64_t vocab, int n, uint32_t *key_out,
                                                   uint32_t *pos_out) {
    __shared__ __align__(16) uint32_t keys[kRankMax];
    __shared__ int below[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int padded = (n + 63) & ~63;
    for (int j = threadIdx.x; j < padded; j += 1024)
        keys[j] = j < n ? key_of(tokens[j], vocab) : 0xffffffffu;
    __syncthreads();
    const int i0 = blockIdx.x * 64, i = i0 + lane;
    const uint32_t mine = keys[i];   // i < padded
    int count = 0;
    const int blocks = padded / 64, from = blocks * wave / 16, to = blocks * (wave + 1) / 16;
    for (int b = from; b < to; ++b) {
        if (b * 64 == i0) {
            for (int j = 0; j < 64; ++j)
                count += keys[i0 + j] < mine || (keys[i0 + j] == mine && j < lane);
            continue;
        }
        // equal keys count where they come before: k <= mine is k < mine + 1
        const uint32_t limit = mine + (b * 64 < i0 ? 1u : 0u);
#pragma unroll 4
        for (int j = 0; j < 64; j += 4) {
            const u32x4 k = *reinterpret_cast<const u32x4 *>(&keys[b * 64 + j]);
            count += (k.x < limit) + (k.y < limit) + (k.z < limit) + (k.w < limit);
        }
    }
    below[wave][lane] = count;
    __syncthreads();
    if (wave == 0 && i < n) {
        int place = 0;
        for (int w = 0; w < 16; ++w)
            place += below[w][lane];
        key_out[place] = mine;
        pos_out[place] = uint32_t(i);
    }
}

// More positions: by digits from the lowest, each pass stable. A workgroup
// takes kSortItems positions, each of its 4 waves a quarter of them in order.
struct SortArgs {
    const int64_t *tokens;  // the first pass's keys
    int64_t vocab, n, blocks;
    const uint32_t *key, *pos;
    uint32_t *key_out, *pos_out;
    uint32_t *hist;  // [bin][workgroup]: counts, then where a workgroup's first of that digit goes
    int shift, bits;
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
        for (int j = threadIdx.x; j < kSortItems; j += 256) {
            const int64_t i = b * kSortItems + j;
            if (i < a.n)
                atomicAdd(&count[(sort_key(a, i) >> a.shift) & (bins - 1)], 1u);
        }
        __syncthreads();
        for (int d = threadIdx.x; d < bins; d += 256)
            a.hist[d * a.blocks + b] = count[d];
        __syncthreads();
    }
}

// hist to the sum of all entries before each, by one workgroup.
__global__ __launch_bounds__(1024) void sort_scan_kernel(uint32_t *hist, int64_t entries) {
    __shared__ uint32_t wave_sum[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t before = 0;
    for (int64_t i0 = 0; i0 < entries; i0 += 4096) {
        const int64_t i = i0 + threadIdx.x * 4;
        uint32_t v[4], own = 0;
        for (int k = 0; k < 4; ++k) {
            v[k] = i + k < entries ? hist[i + k] : 0u;
            own += v[k];
        }
        uint32_t upto = own;
        for (int s = 1; s < 64; s <<= 1) {
            const uint32_t other = __shfl_up(upto, s);
            if (lane >= s)
                upto += other;
        }
        if (lane == 63)
            wave_sum[wave] = upto;
        __syncthreads();
        uint32_t at = before + upto - own, total = 0;
        for (int w = 0; w < 16; ++w) {
            if (w < wave)
                at += wave_sum[w];
            total += wave_sum[w];
        }
        for (int k = 0; k < 4; ++k) {
            if (i + k < entries)
                hist[i + k] = at;
            at += v[k];
        }
        before += total;
        __syncthreads();
    }
}

__global__ __launch_bounds__(256) void sort_move_kernel(SortArgs a) {
    __shared__ uint32_t next[4][kSortBins];
    const int bins = 1 << a.bits, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t b = blockIdx.x; b < a.blocks; b += gridDim.x) {
        for (int d = threadIdx.x; d < 4 * bins; d += 256)
            next[d / bins][d % bins] = 0;
        __syncthreads();
        const int64_t i0 = b * kSortItems + wave * (kSortItems / 4);
        for (int j = lane; j < kSortItems / 4; j += 64)
            if (i0 + j < a.n)
                atomicAdd(&next[wave][(sort_key(a, i0 + j) >> a.shift) & (bins - 1)], 1u);
        __syncthreads();
        for (int d = threadIdx.x; d < bins; d += 256) {
            uint32_t at = a.hist[d * a.blocks + b];
            for (int w = 0; w < 4; ++w) {
                const uint32_t c = next[w][d];
                next[w][d] = at;
                at += c;
            }
        }
        __syncthreads();
        for (int j = lane; j < kSortItems / 4; j += 64) {
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

// Adds the rows of positions pos[from, to) to e, in that order, loads ahead.
template <typename T>
__device__ __forceinline__ void add_rows(Eight &e, const T *x, int64_t stride, const uint32_t *pos, int64_t from,
                                         int64_t to, int count) {
    int64_t i = from;
    for (; i + 8 <= to; i += 8) {
        Eight r[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            r[k] = read8(x + int64_t(pos[i + k]) * stride, count);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            for (int c = 0; c < 8; ++c)
                e.v[c] += r[k].v[c];
    }
    for (; i < to; ++i) {
        const Eight r = read8(x + int64_t(pos[i]) * stride, count);
        for (int c = 0; c < 8; ++c)
            e.v[c] += r.v[c];
    }
}

struct SumArgs {
    RowsArgs r;
    const uint32_t *key, *pos;  // sorted
    float *partial;             // [chunk][dim]
    int64_t chunks;             // 0: no partial sums
};

// The sum of every chunk that is all one token's.
template <typename T>
__global__ __launch_bounds__(64) void run_chunk_kernel(SumArgs a) {
    const int64_t c = int64_t(blockIdx.y) * 512 + threadIdx.x * 8;
    const int count = columns_left(a.r.dim, c);
    for (int64_t b = blockIdx.x; b < a.chunks; b += gridDim.x) {
        const int64_t from = b * kRunChunk;
        const uint32_t key = a.key[from];
        if (key == uint32_t(a.r.vocab) || a.key[from + kRunChunk - 1] != key || count <= 0)
            continue;
        Eight e{};
        add_rows(e, static_cast<const T *>(a.r.x) + c, a.r.stride, a.pos, from, from + kRunChunk, count);
        write8(a.partial + b * a.r.dim + c, e, count);
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

// A wave takes kRowGroup rows of the matrix at 512 columns.
constexpr int kRowGroup = 16;

template <typename T>
__global__ __launch_bounds__(64) void rows_kernel(SumArgs a) {
    const RowsArgs &r = a.r;
    const int64_t c = int64_t(blockIdx.y) * 512 + threadIdx.x * 8;
    const int count = columns_left(r.dim, c);
    const int64_t groups = (r.vocab + kRowGroup - 1) / kRowGroup;
    const T *x = static_cast<const T *>(r.x) + c;
    for (int64_t b = blockIdx.x; b < groups; b += gridDim.x) {
        const int64_t row0 = b * kRowGroup;
        int64_t at = first_not_below(a.key, 0, r.n, uint32_t(row0));
        for (int64_t row = row0; row < row0 + kRowGroup && row < r.vocab; ++row) {
            // the row's positions [at, end)
            const int64_t look = at + (threadIdx.x & 63);
            const int named = __popcll(__ballot(look < r.n && a.key[look] == uint32_t(row)));
            const int64_t end = named < 64 ? at + named : first_not_below(a.key, at + 64, r.n, uint32_t(row) + 1);
            uint16_t *out = r.g + row * r.dim + c;
            if (count > 0 && (end > at || !r.accumulate)) {
                Eight e{};
                const int64_t b0 = (at + kRunChunk - 1) / kRunChunk, b1 = end / kRunChunk;
                if (a.chunks && b0 < b1) {
                    add_rows(e, x, r.stride, a.pos, at, b0 * kRunChunk, count);
                    for (int64_t k = b0; k < b1; ++k) {
                        const Eight p = read8(a.partial + k * r.dim + c, count);
                        for (int i = 0; i < 8; ++i)
                            e.v[i] += p.v[i];
                    }
                    add_rows(e, x, r.stride, a.pos, b1 * kRunChunk, end, count);
                } else {
                    add_rows(e, x, r.stride, a.pos, at, end, count);
                }
                if (end > at)
                    for (float &v : e.v)
                        v = r.scale * v;
                if (r.accumulate) {
                    const Eight old = read8(out, count);
                    for (int i = 0; i < 8; ++i)
                        e.v[i] = old.v[i] + e.v[i];
                }
                write8(out, e, count);
            }
            at = end;
        }
    }
}

__global__ __launch_bounds__(256) void zero_kernel(uint16_t *p, int64_t n) {
    const int64_t chunks = (n + 7) / 8;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < chunks; i += int64_t(gridDim.x) * 256)
        write8(p + i * 8, Eight{}, columns_left(n, i * 8));
}

// ---- around the cross entropy's products --------------------------------------------------------

// Rows of dim elements, one every `stride`, to rows of kdim, zeros behind.
__global__ __launch_bounds__(256) void pack_kernel(const uint16_t *from, int64_t stride, int64_t rows, int64_t dim,
                                                  int64_t kdim, uint16_t *to) {
    const int64_t per = kdim / 8;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < rows * per; i += int64_t(gridDim.x) * 256) {
        const int64_t r = i / per, c = i % per * 8;
        const int count = columns_left(dim, c);
        write8(to + r * kdim + c, count > 0 ? read8(from + r * stride + c, count) : Eight{}, 8);
    }
}

// The transpose: to[c][r] = from[r][c], zero for r in [rows, padded) and where
// targets (if given) names no row for r. 64 x 64 elements a workgroup.
__global__ __launch_bounds__(256) void transpose_kernel(const uint16_t *from, int64_t stride, int64_t rows,
                                                        int64_t dim, int64_t padded, const int64_t *targets,
                                                        int64_t vocab, uint16_t *to) {
    __shared__ uint16_t tile[64][66];
    const int64_t across = (dim + 63) / 64, tiles = across * (padded / 64);
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t r0 = t / across * 64, c0 = t % across * 64;
        const int r = threadIdx.x >> 2, part = (threadIdx.x & 3) * 16;
        bool keep = r0 + r < rows;
        if (keep && targets) {
            const int64_t target = targets[r0 + r];
            keep = target >= 0 && target < vocab;
        }
#pragma unroll
        for (int h = 0; h < 16; h += 8) {
            const int count = keep ? columns_left(dim, c0 + part + h) : 0;
            u32x4 x = {0, 0, 0, 0};
            const uint16_t *p = from + (r0 + r) * stride + c0 + part + h;
            if (count >= 8)
                x = reinterpret_cast<const Loose16 *>(p)->v;
            else
                for (int i = 0; i < 7; ++i)
                    if (i < count)
                        x[i >> 1] |= uint32_t(p[i]) << (i & 1) * 16;
            for (int i = 0; i < 8; ++i)
                tile[r][part + h + i] = uint16_t(x[i >> 1] >> (i & 1) * 16);
        }
        __syncthreads();
        const int64_t c = c0 + r;
        if (c < dim) {
#pragma unroll
            for (int h = 0; h < 16; h += 8) {
                u32x4 x;
                for (int i = 0; i < 4; ++i)
                    x[i] = uint32_t(tile[part + h + 2 * i][r]) | uint32_t(tile[part + h + 2 * i + 1][r]) << 16;
                *reinterpret_cast<u32x4 *>(to + c * padded + r0 + part + h) = x;
            }
        }
        __syncthreads();
    }
}

// The softmax's statistics of all tiles to each token's loss and lse: 16
// tokens a workgroup, 16 threads each over every 16th tile.
__global__ __launch_bounds__(256) void combine_kernel(CeArgs a, const float2 *part, int64_t tiles, const float *pick) {
    __shared__ float2 red[16][16];
    const int token = threadIdx.x & 15, slice = threadIdx.x >> 4;
    auto join = [](float2 x, float2 y) {
        const float top = fmaxf(x.x, y.x);
        return float2{top, x.y * (x.x == top ? 1.0f : __expf(x.x - top)) + y.y * (y.x == top ? 1.0f : __expf(y.x - top))};
    };
    for (int64_t t0 = int64_t(blockIdx.x) * 16; t0 < a.n; t0 += int64_t(gridDim.x) * 16) {
        const int64_t t = t0 + token;
        float2 all = {-INFINITY, 0.0f};
        if (t < a.n)
            for (int64_t k = slice; k < tiles; k += 16)
                all = join(all, part[k * a.n + t]);
        red[slice][token] = all;
        __syncthreads();
        if (slice == 0 && t < a.n) {
            for (int s = 1; s < 16; ++s)
                all = join(all, red[s][token]);
            const float lse = all.x + logf(all.y);
            const int64_t target = a.targets[t];
            a.lse[t] = lse;
            a.loss[t] = target >= 0 && target < a.vocab ? lse - pick[t] : 0.0f;
        }
        __syncthreads();
    }
}

// The splits' sums of grad_hidden, added in their order and rounded.
template <typename T>
__global__ __launch_bounds__(256) void hidden_kernel(CeArgs a, const float *sum, int64_t splits, int64_t kdim) {
    const int64_t per = kdim / 8;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < a.n * per; i += int64_t(gridDim.x) * 256) {
        const int64_t r = i / per, c = i % per * 8;
        const int count = columns_left(a.dim, c);
        if (count <= 0)
            continue;
        const int64_t target = a.targets[r];
        Eight e{};
        if (target >= 0 && target < a.vocab)
            for (int64_t s = 0; s < splits; ++s) {
                const Eight x = read8(sum + (s * a.n + r) * kdim + c, 8);
                for (int k = 0; k < 8; ++k)
                    e.v[k] += x.v[k];
            }
        write8(static_cast<T *>(a.grad_hidden) + r * a.grad_hidden_stride + c, e, count);
    }
}

unsigned grid_of(int64_t blocks) { return unsigned(std::min<int64_t>(blocks, std::min<int64_t>(kMaxGrid, 1 << 20))); }

// W and hidden as the products need them: in place where their rows are 16-byte
// aligned whole steps, else a copy.
struct Operands {
    bool direct;
    const uint16_t *hidden;
    int64_t lda, ldb;
};

Operands operands(const CeArgs &a, const CeLayout &l, hipStream_t stream) {
    Operands o{};
    auto aligned = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    o.direct = a.dim % kDepth == 0 && aligned(a.w) && aligned(a.hidden) &&
               (a.n <= 1 || (a.hidden_stride % 8 == 0 && a.hidden_stride <= int64_t(1) << 21));
    if (o.direct) {
        o.hidden = a.hidden;
        o.ldb = a.n <= 1 ? a.dim : a.hidden_stride;
    } else {
        uint16_t *h = reinterpret_cast<uint16_t *>(a.workspace + l.hidden);
        pack_kernel<<<grid_of(ceil_div(a.n * l.kdim, 2048)), 256, 0, stream>>>(a.hidden, a.hidden_stride, a.n, a.dim,
                                                                              l.kdim, h);
        o.hidden = h;
        o.ldb = l.kdim;
    }
    o.lda = l.kdim;   // dim where direct
    return o;
}

const uint16_t *piece_of(const CeArgs &a, const CeLayout &l, const Operands &o, int64_t row0, int64_t rows,
                         hipStream_t stream) {
    if (o.direct)
        return a.w + row0 * a.dim;
    uint16_t *w = reinterpret_cast<uint16_t *>(a.workspace + l.w);
    pack_kernel<<<grid_of(ceil_div(rows * l.kdim, 2048)), 256, 0, stream>>>(a.w + row0 * a.dim, a.dim, rows, a.dim,
                                                                           l.kdim, w);
    return w;
}

}  // namespace

hipError_t launch_zero(uint16_t *p, int64_t n, hipStream_t stream) {
    if (n > 0)
        zero_kernel<<<grid_of(ceil_div(n, 2048)), 256, 0, stream>>>(p, n);
    return hipGetLastError();
}

hipError_t launch_lookup(const LookupArgs &a, hipStream_t stream) {
    if (a.n == 0)
        return hipSuccess;
    const dim3 grid(grid_of(ceil_div(a.n, 4)), unsigned(ceil_div(a.dim, kLookupWide)));
    if (a.f32)
        lookup_kernel<float><<<grid, 256, 0, stream>>>(a);
    else
        lookup_kernel<uint16_t><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_rows(const RowsArgs &a, hipStream_t stream) {
    if (!a.accumulate)
        if (hipError_t e = launch_zero(a.g + a.vocab * a.dim, a.numel - a.vocab * a.dim, stream); e != hipSuccess)
            return e;
    if (a.n == 0)
        return a.accumulate ? hipSuccess : launch_zero(a.g, a.vocab * a.dim, stream);
    const RowsLayout l = rows_layout(a.n, a.dim);
    char *ws = static_cast<char *>(a.workspace);
    auto u32 = [&](int64_t at) { return reinterpret_cast<uint32_t *>(ws + at); };
    SumArgs s{};
    s.r = a;
    int set = 0;
    if (a.n <= kRankMax) {
        rank_kernel<<<unsigned(ceil_div(a.n, 64)), 1024, 0, stream>>>(a.tokens, a.vocab, int(a.n), u32(l.key[0]),
                                                                     u32(l.pos[0]));
    } else {
        const int bits = 64 - __builtin_clzll(uint64_t(a.vocab)), passes = (bits + 8) / 9;
        const int digit = (bits + passes - 1) / passes;
        SortArgs p{};
        p.vocab = a.vocab;
        p.n = a.n;
        p.blocks = l.blocks;
        p.hist = u32(l.hist);
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
            sort_scan_kernel<<<1, 1024, 0, stream>>>(p.hist, l.blocks << digit);
            sort_move_kernel<<<grid_of(l.blocks), 256, 0, stream>>>(p);
        }
    }
    s.key = u32(l.key[set]);
    s.pos = u32(l.pos[set]);
    s.partial = reinterpret_cast<float *>(ws + l.partial);
    s.chunks = l.chunks;
    const unsigned across = unsigned(ceil_div(a.dim, 512));
    if (s.chunks) {
        const dim3 grid(grid_of(s.chunks), across);
        if (a.f32)
            run_chunk_kernel<float><<<grid, 64, 0, stream>>>(s);
        else
            run_chunk_kernel<uint16_t><<<grid, 64, 0, stream>>>(s);
    }
    const dim3 grid(grid_of(ceil_div(a.vocab, kRowGroup)), across);
    if (a.f32)
        rows_kernel<float><<<grid, 64, 0, stream>>>(s);
    else
        rows_kernel<uint16_t><<<grid, 64, 0, stream>>>(s);
    return hipGetLastError();
}

hipError_t launch_ce(const CeArgs &a, hipStream_t stream) {
    if (a.n == 0)
        return hipSuccess;
    const CeLayout l = ce_layout(a.n, a.vocab, a.dim);
    const Operands o = operands(a, l, stream);
    GemmArgs g{};
    g.b = o.hidden;
    g.lda = o.lda;
    g.ldb = o.ldb;
    g.n = a.n;
    g.k = l.kdim;
    g.splits = 1;
    g.targets = a.targets;
    g.vocab = a.vocab;
    g.part = reinterpret_cast<float2 *>(a.workspace + l.part);
    g.pick = reinterpret_cast<float *>(a.workspace + l.pick);
    // in place, W needs no pieces but for the tiles' numbers
    const int64_t rows = o.direct ? std::max(l.piece, (int64_t(1) << 36) / l.npad / 256 * 256) : l.piece;
    for (g.row0 = 0; g.row0 < a.vocab; g.row0 += rows) {
        g.m = std::min(rows, a.vocab - g.row0);
        g.a = piece_of(a, l, o, g.row0, g.m, stream);
        if (hipError_t e = launch_gemm(kScore, g, stream); e != hipSuccess)
            return e;
        g.tile0 += ceil_div(g.m, tile_rows(g.m, g.n));
    }
    combine_kernel<<<grid_of(ceil_div(a.n, 16)), 256, 0, stream>>>(a, g.part, g.tile0, g.pick);
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
    const CeLayout l = ce_layout(a.n, a.vocab, a.dim);
    const Operands o = operands(a, l, stream);
    auto u16 = [&](int64_t at) { return reinterpret_cast<uint16_t *>(a.workspace + at); };
    uint16_t *hidden_t = u16(l.hidden_t), *w_t = u16(l.w_t), *d = u16(l.d), *dt = u16(l.d_t);
    float *sum = reinterpret_cast<float *>(a.workspace + l.sum);
    const int64_t across = ceil_div(a.dim, 64);
    if (a.grads)
        transpose_kernel<<<grid_of(across * (l.npad / 64)), 256, 0, stream>>>(
            a.hidden, a.hidden_stride, a.n, a.dim, l.npad, a.targets, a.vocab, hidden_t);
    for (int64_t row0 = 0; row0 < a.vocab; row0 += l.piece) {
        const int64_t rows = std::min(l.piece, a.vocab - row0), padded = round_up(rows, kDepth);
        GemmArgs g{};
        g.a = piece_of(a, l, o, row0, rows, stream);
        g.b = o.hidden;
        g.lda = o.lda;
        g.ldb = o.ldb;
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
        g.ldd = l.vpad;
        g.dt = dt;
        g.lddt = l.npad;
        if (hipError_t e = launch_gemm(kDiff, g, stream); e != hipSuccess)
            return e;
        if (a.grad_hidden) {
            transpose_kernel<<<grid_of(across * (padded / 64)), 256, 0, stream>>>(
                a.w + row0 * a.dim, a.dim, rows, a.dim, padded, nullptr, 0, w_t);
            GemmArgs h{};
            h.a = w_t;
            h.b = d;
            h.lda = padded;
            h.ldb = l.vpad;
            h.m = a.dim;
            h.n = a.n;
            h.k = padded;
            h.splits = int32_t(l.splits);
            h.sum = sum;
            h.lds = l.kdim;
            h.first = row0 == 0;
            if (hipError_t e = launch_gemm(kSum, h, stream); e != hipSuccess)
                return e;
        }
        if (a.grads) {
            GemmArgs r{};
            r.a = hidden_t;
            r.b = dt;
            r.lda = l.npad;
            r.ldb = l.npad;
            r.m = a.dim;
            r.n = rows;
            r.k = l.npad;
            r.splits = 1;
            r.rows = a.grads + row0 * a.dim;
            r.accumulate = a.accumulate;
            if (hipError_t e = launch_gemm(kRows, r, stream); e != hipSuccess)
                return e;
        }
    }
    if (a.grad_hidden) {
        const unsigned grid = grid_of(ceil_div(a.n * l.kdim, 2048));
        if (a.f32)
            hidden_kernel<float><<<grid, 256, 0, stream>>>(a, sum, l.splits, l.kdim);
        else
            hidden_kernel<uint16_t><<<grid, 256, 0, stream>>>(a, sum, l.splits, l.kdim);
    }
    return hipGetLastError();
}

}  // namespace zdo
