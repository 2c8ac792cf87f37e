// Device kernels of the MXFP4 contributions and parameters (zdo_mx.h) for
// gfx950: quantising, the reduction of D contributions and its squared norm,
// the fused Adam step on them, and the all-gather of quantised parameters.
//
// Like the bf16 kernels they are streams bound by HBM bandwidth. A storage
// tile (512 slots: 256 bytes of codes, 16 scales) lies at the same phase
// modulo 64 as its WORLD and LOCAL elements, so full chunks of 8 slots are
// 16-byte aligned in every buffer. Lane l takes the tile's slots [8l, 8l + 8)
// and a block of 32 is 4 lanes.
//
// gfx950 converts between fp32 and E2M1 pairs with the block's scale in one
// instruction (v_cvt_scalef32_pk_f32_fp4, v_cvt_scalef32_pk_fp4_f32), the
// scale given as an fp32 whose exponent field is the E8M0 byte. The tests
// hold them to the oracle over all 256 scales x 256 pairs, every bf16, and
// 2^20 random fp32 at ten scales: exact, subnormal results kept, scale 255
// gives NaN, rounding to nearest even and saturating at 6.
#include <hip/hip_runtime.h>

#include "device.h"
#include "mx.h"

#pragma clang fp contract(off)

namespace zdo {
namespace {

static_assert(kBlock == 64 && kTileElems == 512, "a tile is one wave of 8-slot chunks");

// ---- storage -------------------------------------------------------------------------------

// One tile of a range's storage.
struct MxTile {
    int64_t w, k;     // WORLD and LOCAL index of its slot 0 (k: the plan's rank only)
    int lo, hi, own;  // its slots [lo, hi) lie in the range, [lo, own) are parameter elements
    int64_t local, world;  // its number in LOCAL and in WORLD storage
};

__device__ __forceinline__ int clamp_slot(int64_t x) { return x < 0 ? 0 : x > kTileElems ? kTileElems : int(x); }

// Tile i of rank r's range of bucket b.
__device__ __forceinline__ MxTile tile_in(ro_ptr<MxBucket> b, int dp, int r, int i) {
    MxTile t;
    const int64_t rs = b->offset + r * b->shard;
    const int64_t origin = rs / kAnchor * kAnchor;
    t.w = origin + int64_t(i) * kTileElems;
    t.k = b->base + (t.w - rs);
    const int64_t re = rs + b->shard, oe = b->offset + b->numel;
    t.lo = clamp_slot(rs - t.w);
    t.hi = clamp_slot(re - t.w);
    t.own = clamp_slot((oe < re ? oe : re) - t.w);
    t.local = b->tile0 + i;
    t.world = dp * b->tile0 + int64_t(r) * b->tiles + i;
    return t;
}

// The bucket holding LOCAL tile or unit x: the one that holds the first of
// its group of kTileGroup, unless buckets start within the group; then by
// halving (about 19,000 buckets of 2,100 elements at D = 4: step 64 us, 74 by
// one bucket after the other; quantise with residual and back 264 and 308).
template <bool kUnits>
__device__ __forceinline__ ro_ptr<MxBucket> bucket_of(const MxWalk &wk, int64_t x) {
    const ro_ptr<MxBucket> all = ro(wk.buckets);
    const ro_ptr<uint32_t> g = ro(wk.group) + x / kTileGroup;
    uint32_t lo = g[0], hi = g[1];
    while (lo < hi) {
        const uint32_t mid = (lo + hi + 1) / 2;
        if ((kUnits ? all[mid].unit0 : all[mid].tile0) <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    return all + lo;
}

// The tile at launch index i of a walk over the rank's tiles.
__device__ __forceinline__ MxTile local_tile(const MxWalk &wk, int64_t i) {
    const int64_t x = wk.first + i;
    const ro_ptr<MxBucket> b = bucket_of<false>(wk, x);
    return tile_in(b, wk.dp, wk.rank, int(x - b->tile0));
}

// The walk index that launch slot i takes. With `by_xcd`, as in the bf16
// kernels' short launches, each of the 8 XCDs takes 8 consecutive tiles out of
// every 64: those 8 tiles' scales are one 128-byte line of every contribution,
// which 8 XCDs would each fetch into their own L2 otherwise (1.11 times the
// bytes that a step with 8 contributions needs).
// Launches of fewer tiles than kShortLaunch are short. The step at 4e7 slots:
// 8 contributions 197 us as a long launch, 201 as a short one, 3 contributions
// 189 and 193; at 2e7 slots 101.6 and 102.7, 99.3 and 96.5.
#ifndef ZDO_MX_LONG_TILES
#define ZDO_MX_LONG_TILES (int64_t(1) << 16)
#endif
constexpr int64_t kShortLaunch = ZDO_MX_LONG_TILES;
__device__ __forceinline__ int64_t launch_order(bool by_xcd, int64_t count, int64_t i) {
    if (!by_xcd || i >= count / 64 * 64)
        return i;
    const int64_t r = i % 64;
    return i - r + (r % 8) * 8 + r / 8;
}

// A unit of up to kMxUnit consecutive tiles of one range: its first tile's
// number within the range and how many there are.
struct MxUnit {
    ro_ptr<MxBucket> b;
    int rank, tile, ntiles;
};
template <bool kWorld>
__device__ __forceinline__ MxUnit unit_at(const MxWalk &wk, int64_t i) {
    const uint32_t x = uint32_t(wk.first + i);
    MxUnit u;
    u.b = bucket_of<true>(wk, kWorld ? x / uint32_t(wk.dp) : x);
    uint32_t rel = x - uint32_t(kWorld ? wk.dp * u.b->unit0 : u.b->unit0);
    u.rank = wk.rank;
    if constexpr (kWorld) {
        u.rank = int(rel / uint32_t(u.b->units));
        rel -= uint32_t(u.rank) * uint32_t(u.b->units);
    }
    u.tile = int(rel) * kMxUnit;
    u.ntiles = u.b->tiles - u.tile < kMxUnit ? u.b->tiles - u.tile : kMxUnit;
    return u;
}

// ---- the format --------------------------------------------------------------------------------

__device__ __forceinline__ float scale_f32(uint32_t byte) { return __uint_as_float(byte << 23); }

// The 8 values of a word of codes.
__device__ __forceinline__ void values_of(uint32_t codes, float scale, float x[8]) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 3);
    x[0] = a[0];
    x[1] = a[1];
    x[2] = b[0];
    x[3] = b[1];
    x[4] = c[0];
    x[5] = c[1];
    x[6] = d[0];
    x[7] = d[1];
}

__device__ __forceinline__ uint32_t max_bits(uint32_t a, uint32_t b) { return a > b ? a : b; }
// The largest over the 4 lanes of a quad: 1 and 2 lanes away.
__device__ __forceinline__ uint32_t max_quad(uint32_t x) {
    x = max_bits(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0xB1, 0xf, 0xf, true)));
    return max_bits(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0x4E, 0xf, 0xf, true)));
}

// A lane's 8 values to a word of codes, with the scale of its block (4
// lanes): the largest magnitude's bits over the block, by integer compare, so
// that Inf and NaN win; byte = max(0, exponent - 2). Every lane of the wave
// takes part.
__device__ __forceinline__ void round_block(const float x[8], uint32_t &codes, uint32_t &byte) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        top = max_bits(top, __float_as_uint(x[e]) & 0x7fffffffu);
    top = max_quad(top);
    const uint32_t ex = top >> 23;
    byte = ex == 255 ? 255 : ex > 2 ? ex - 2 : 0;
    const float s = scale_f32(byte);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], s, 3);
    codes = ex == 255 ? 0 : c;
}

// The lane's word of codes of tile t, and its block's scale.
__device__ __forceinline__ void ld_block(const uint8_t *codes, const uint8_t *scales, int64_t t, uint32_t &c,
                                         uint32_t &s) {
    c = __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(codes + t * (kTileElems / 2)) + threadIdx.x);
    s = scales[t * kMxTileBlocks + threadIdx.x / 4];
}
// The codes go out non-temporally (quantising 1e9 bf16 elements: 406 us, 482
// with plain stores; 1.2e8: 54 us both).
__device__ __forceinline__ void st_block(uint8_t *codes, uint8_t *scales, int64_t t, uint32_t c, uint32_t s) {
    __builtin_nontemporal_store(c, reinterpret_cast<uint32_t *>(codes + t * (kTileElems / 2)) + threadIdx.x);
    if (threadIdx.x % 4 == 0)
        scales[t * kMxTileBlocks + threadIdx.x / 4] = uint8_t(s);
}

// The same for a lane's quad, whose blocks are 8 lanes: 16 bits of codes.
__device__ __forceinline__ void round_quad(const float x[4], uint32_t &codes, uint32_t &byte) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        top = max_bits(top, __float_as_uint(x[e]) & 0x7fffffffu);
    top = max_quad(top);
    // the other quad of the 8 lanes: the mirror image within them
    top = max_bits(top, uint32_t(__builtin_amdgcn_mov_dpp(int(top), 0x141, 0xf, 0xf, true)));
    const uint32_t ex = top >> 23;
    byte = ex == 255 ? 255 : ex > 2 ? ex - 2 : 0;
    const float s = scale_f32(byte);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], s, 1);
    codes = ex == 255 ? 0 : c;
}
// Quad h of tile t: half words, which do better as plain stores (quantising
// 1.2e8 elements with a residual: 208 us, 222 non-temporally).
__device__ __forceinline__ void st_quad(uint8_t *codes, uint8_t *scales, int64_t t, int h, uint32_t c, uint32_t s) {
    reinterpret_cast<uint16_t *>(codes + t * (kTileElems / 2))[64 * h + threadIdx.x] = uint16_t(c);
    if (threadIdx.x % 8 == 0)
        scales[t * kMxTileBlocks + 8 * h + threadIdx.x / 8] = uint8_t(s);
}

// The sum of the contributions over the lane's 8 * kW slots of kW consecutive
// tiles from tile `at` (lane l: slots [8 kW l, 8 kW (l + 1)), which lie in one
// block), in the order given, from -0 (which adds to any first term
// exactly). kN > 0: that many contributions, all their loads in flight
// together; kN = 0: any number, in batches of 16 and what is left, each
// batch's loads in flight together (kMost = kFew: fewer than 4, for which fewer
// registers are enough and more waves fit). (A batch of the same code for any count up
// to 16, its loads behind uniform branches, took 1.9 times as long at 16
// contributions and 4 times at 32: the waits behind a branch are for every
// load.)
constexpr int kBatch = 16, kFew = 4;
template <int kW, int kCount>
__device__ __forceinline__ void add_batch(const MxInputs &in, int j, int64_t at, float acc[8 * kW]) {
    typedef unsigned int words __attribute__((ext_vector_type(kW)));
    words c[kCount];
    uint32_t s[kCount];
    const int lane = int(threadIdx.x);
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
        c[i] = __builtin_nontemporal_load(
            reinterpret_cast<const words *>(in.codes[j + i] + at * (kTileElems / 2)) + lane);
        s[i] = in.scales[j + i][at * kMxTileBlocks + lane * kW / 4];
    }
#pragma unroll
    for (int i = 0; i < kCount; ++i)
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            float x[8];
            values_of(c[i][w], scale_f32(s[i]), x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                acc[8 * w + e] = acc[8 * w + e] + x[e];
        }
}
template <int kW, int kN, int kMost = kBatch>
__device__ __forceinline__ void sum_blocks(const MxInputs &in, int64_t at, float acc[8 * kW]) {
#pragma unroll
    for (int e = 0; e < 8 * kW; ++e)
        acc[e] = -0.0f;
    if constexpr (kN > 0) {
        add_batch<kW, kN>(in, 0, at, acc);
        return;
    }
    int j = 0;
    if constexpr (kMost == kBatch) {
        for (; j + kBatch <= in.n; j += kBatch)
            add_batch<kW, kBatch>(in, j, at, acc);
        if (in.n & 8) {
            add_batch<kW, 8>(in, j, at, acc);
            j += 8;
        }
        switch (in.n & 7) {
        case 4: add_batch<kW, 4>(in, j, at, acc); return;
        case 5: add_batch<kW, 5>(in, j, at, acc); return;
        case 6: add_batch<kW, 6>(in, j, at, acc); return;
        case 7: add_batch<kW, 7>(in, j, at, acc); return;
        default: break;
        }
    }
    switch (in.n & 3) {
    case 1: add_batch<kW, 1>(in, j, at, acc); break;
    case 2: add_batch<kW, 2>(in, j, at, acc); break;
    case 3: add_batch<kW, 3>(in, j, at, acc); break;
    default: break;
    }
}
__device__ __forceinline__ int64_t stored_at(const MxInputs &in, const MxTile &t) { return in.world ? t.world : t.local; }

// The lane's slots of its chunk below `end` of tile slots [lo, end).
struct Slots {
    int lo, hi;
    __device__ __forceinline__ bool full() const { return lo == 0 && hi == kChunk; }
};
__device__ __forceinline__ Slots slots_of(int lo, int end) {
    const int c0 = int(threadIdx.x) * kChunk;
    Slots s;
    s.lo = lo - c0 < 0 ? 0 : lo - c0;
    s.hi = end - c0 > kChunk ? kChunk : end - c0;
    return s;
}

__device__ __forceinline__ void st_bf16(uint16_t *p, const float x[8], Slots s) {
    if (s.full()) {
        st16_out(p, u32x4{to_bf16x2(x[0], x[1]), to_bf16x2(x[2], x[3]), to_bf16x2(x[4], x[5]),
                          to_bf16x2(x[6], x[7])});
    } else {
#pragma unroll
        for (int e = 0; e < kChunk; ++e)
            if (e >= s.lo && e < s.hi)
                p[e] = uint16_t(to_bf16x2(x[e], 0.0f));
    }
}

// ---- kernels -------------------------------------------------------------------------------------

// One tile of the reduction, whole or not.
__device__ __forceinline__ void reduce_tile(const MxReduceArgs &a, const MxTile &t) {
    if (t.lo >= t.hi)
        return;
    float acc[8];
    sum_blocks<1, 0>(a.in, stored_at(a.in, t), acc);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        acc[e] = acc[e] * a.scale;
    st_bf16(a.out + (a.out_local ? t.k : t.w) + threadIdx.x * kChunk, acc, slots_of(t.lo, t.hi));
}

// Short launches: a tile a wave, for the most waves.
__global__ __launch_bounds__(kBlock) void mx_reduce_kernel(MxReduceArgs a) {
    for (int64_t i = blockIdx.x; i < a.walk.count; i += gridDim.x)
        reduce_tile(a, local_tile(a.walk, launch_order(a.walk.by_xcd, a.walk.count, i)));
}

// Long ones: a unit a wave, kW tiles at a time, so that a load instruction
// covers kW * 256 bytes of codes and kW * 16 scales; the rounded sums change
// lanes through LDS (16 bytes a chunk, xor-placed against bank conflicts), so
// that a store covers 1 KiB without a gap.
__device__ __forceinline__ int chunk_place(int c) { return (c & ~7) | ((c ^ (c >> 3)) & 7); }

template <int kW, int kMost>
__global__ __launch_bounds__(kBlock) __attribute__((amdgpu_waves_per_eu(1, kMost < kBatch ? 8 : 4)))
void mx_reduce_wide_kernel(MxReduceArgs a) {
    __shared__ u32x4 chunks[kBlock * kW];
    const int lane = int(threadIdx.x);
    for (int64_t i = blockIdx.x; i < a.walk.count; i += gridDim.x) {
        const MxUnit u = unit_at<false>(a.walk, i);
        int j = 0;
        for (; j + kW <= u.ntiles; j += kW) {
            const MxTile t = tile_in(u.b, a.walk.dp, u.rank, u.tile + j);
            if (t.lo != 0 || tile_in(u.b, a.walk.dp, u.rank, u.tile + j + kW - 1).hi != kTileElems)
                break;
            float acc[8 * kW];
            sum_blocks<kW, 0, kMost>(a.in, stored_at(a.in, t), acc);
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                u32x4 o;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[k] = to_bf16x2(acc[8 * w + 2 * k] * a.scale, acc[8 * w + 2 * k + 1] * a.scale);
                chunks[chunk_place(kW * lane + w)] = o;
            }
            __syncthreads();
            uint16_t *out = a.out + (a.out_local ? t.k : t.w);
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                const int c = kBlock * w + lane;
                st16_out(out + c * kChunk, chunks[chunk_place(c)]);
            }
            __syncthreads();
        }
        for (; j < u.ntiles; ++j)   // the ends of a range
            reduce_tile(a, tile_in(u.b, a.walk.dp, u.rank, u.tile + j));
    }
}

// The squares of a lane's slots, those of [lo, hi) only, into four running
// sums by the slot's number modulo 4, which keeps the chain of fp64 additions
// short. A square of an fp32 is exact in fp64, so the fused operation rounds
// as an addition of it does.
struct Squares {
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    template <int kSlots>
    __device__ __forceinline__ void add(const float acc[kSlots], float scale, int lo, int hi) {
#pragma unroll
        for (int e = 0; e < kSlots; ++e) {
            const double g = double(acc[e] * scale);
            if (e >= lo && e < hi)
                s[e % 4] = __builtin_fma(g, g, s[e % 4]);
        }
    }
    __device__ __forceinline__ double total() const { return (s[0] + s[1]) + (s[2] + s[3]); }
};
__device__ __forceinline__ void norm_tile(const MxNormArgs &a, const MxTile &t, Squares &s) {
    if (t.lo >= t.own)
        return;
    float acc[8];
    sum_blocks<1, 0>(a.in, stored_at(a.in, t), acc);
    const Slots own = slots_of(t.lo, t.own);
    s.add<8>(acc, a.scale, own.lo, own.hi);
}
// A wave's lanes added by a fixed butterfly.
__device__ __forceinline__ double lanes_total(double s) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        s = s + __shfl_xor(s, off, 64);
    return s;
}
__device__ __forceinline__ void put_partial(double *at, double s) {
    s = lanes_total(s);
    if (threadIdx.x == 0)
        *at = s;
}

// As the reductions, but with at most kMxNormWaves waves, each of which takes
// every kMxNormWaves-th tile or unit and adds its lanes once at the end. A wave a
// unit spent its time filling and in the butterfly: 3e8 slots of 1
// contribution 62 us instead of 119, of 3 92 instead of 138, 5e8 of 16 688
// instead of 694, GPT-2 small rank 20.8 instead of 21.9. With 16384, 8192 and
// 4096 waves, in turn in a later run: 62.9, 64.7 and 70.5 us, 92.0, 96.7 and
// 99.8, 671, 675 and 687, 20.7, 20.0 and 21.4; 1e8 of 4 52.1, 50.2 and 50.2.
// HBM bounds it from 8 contributions (8 of 3e8 213 us, 5.97 TB/s); with fewer,
// vector instructions: of 1 contribution 5.3 an element for half a byte, whose
// issue alone takes 60% of 63 us.
__global__ __launch_bounds__(kBlock) void mx_norm_kernel(MxNormArgs a) {
    Squares s;
    for (int64_t i = blockIdx.x; i < a.walk.count; i += gridDim.x)
        norm_tile(a, local_tile(a.walk, launch_order(a.walk.by_xcd, a.walk.count, i)), s);
    put_partial(a.partial + blockIdx.x, s.total());
}
// From kFew contributions by 2 tiles (4: 4 contributions of 1e8 slots 49.0 us
// instead of 50.2, 8 of 1e8 76.0 and 75.7, 12 of 8e7 90.9 and 88.0, 16 of 6e7
// 87.2 and 85.8, 32 of 4e7 113.6 and 110.9, 64 of 3e7 168.9 and 168.1).
template <int kW, int kMost>
__global__ __launch_bounds__(kBlock) __attribute__((amdgpu_waves_per_eu(1, kMost < kBatch ? 8 : 4)))
void mx_norm_wide_kernel(MxNormArgs a) {
    Squares s;
    for (int64_t i = blockIdx.x; i < a.walk.count; i += gridDim.x) {
        const MxUnit u = unit_at<false>(a.walk, i);
        int j = 0;
        for (; j + kW <= u.ntiles; j += kW) {
            const MxTile t = tile_in(u.b, a.walk.dp, u.rank, u.tile + j);
            if (t.lo != 0 || tile_in(u.b, a.walk.dp, u.rank, u.tile + j + kW - 1).own != kTileElems)
                break;
            float acc[8 * kW];
            sum_blocks<kW, 0, kMost>(a.in, stored_at(a.in, t), acc);
            s.add<8 * kW>(acc, a.scale, 0, 8 * kW);
        }
        for (; j < u.ntiles; ++j)
            norm_tile(a, tile_in(u.b, a.walk.dp, u.rank, u.tile + j), s);
    }
    put_partial(a.partial + blockIdx.x, s.total());
}

// The sums of a workgroup's waves (threadIdx.y), added in order by its first
// work-item.
template <int kWaves>
__device__ __forceinline__ void put_total(double s, double *out) {
    __shared__ double waves[kWaves];
    s = lanes_total(s);
    if (threadIdx.x == 0)
        waves[threadIdx.y] = s;
    __syncthreads();
    if (threadIdx.x == 0 && threadIdx.y == 0) {
        double t = waves[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w)
            t = t + waves[w];
        *out = t;
    }
}

// The norms' wave sums added by one workgroup: work-item t takes sums t, t +
// 1024, ..., all loads first.
constexpr int kSumWaves = 16, kSumItems = 64 * kSumWaves, kSumEach = int(kMxNormWaves / kSumItems);
__global__ __launch_bounds__(kSumItems) void mx_sum_kernel(const double *partial, int64_t n, double *out) {
    double x[kSumEach];
#pragma unroll
    for (int j = 0; j < kSumEach; ++j) {
        const int64_t i = int64_t(j) * kSumItems + threadIdx.y * 64 + threadIdx.x;
        x[j] = i < n ? partial[i] : 0.0;
    }
    double s = x[0];
#pragma unroll
    for (int j = 1; j < kSumEach; ++j)
        s = s + x[j];
    put_total<kSumWaves>(s, out);
}

// The norm of a few tiles in one launch instead of two: up to 64 tiles, and 512
// tiles times contributions (8 contributions of 16 tiles 6.9 us a call, 10.2
// in two launches, of 63 tiles both 10.1 but the step behind it 3 us sooner;
// 64 contributions of 32 tiles 19.1 and 10.2).
constexpr int64_t kNormAtOnceTiles = 64, kNormAtOnceWork = 512;
__global__ __launch_bounds__(kSumItems) void mx_norm_at_once_kernel(MxNormArgs a, double *out) {
    Squares s;
    for (int64_t i = threadIdx.y; i < a.walk.count; i += kSumWaves)
        norm_tile(a, local_tile(a.walk, i), s);
    put_total<kSumWaves>(s.total(), out);
}

// ---- the step --------------------------------------------------------------------------------
// The state is read and rewritten once and a training step finds it cold:
// its accesses are non-temporal (GPT-2 small rank, 187 MB of state, three
// states in turn: 80.3 us, with plain accesses 87.2; back to back on one
// state 79.1 and 77.7; Llama-3-8B rank 4973 and 5274 us).

// A tile that lies whole inside the rank's elements. The state goes by
// quads: lane l takes slots [4l, 4l + 4) and [256 + 4l, 256 + 4l + 4), so that
// every access of the wave covers 1 KiB without a gap (by 8 consecutive
// slots a lane, every second 16 bytes: 8.43 ms instead of 4.97 on the
// Llama-3-8B rank). The codes go by chunks of 8 slots (a word a lane; by quads,
// in half words, 5.02 ms), and the sums change lanes through 2 KiB of LDS.
template <int kN>
__device__ __forceinline__ void step_whole(const MxStepArgs &a, const MxTile &t, bool clip, float cf, f32x4 *sums) {
    const int lane = int(threadIdx.x);
    f32x4 pv[2], mv[2], vv[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t k = t.k + h * (kTileElems / 2) + 4 * lane;
        pv[h] = ld_state<true>(a.master + k);
        mv[h] = ld_state<true>(a.m + k);
        vv[h] = ld_state<true>(a.v + k);
    }
    float acc[8];
    sum_blocks<1, kN>(a.in, stored_at(a.in, t), acc);
    sums[2 * lane] = f32x4{acc[0], acc[1], acc[2], acc[3]};
    sums[2 * lane + 1] = f32x4{acc[4], acc[5], acc[6], acc[7]};
    __syncthreads();
    f32x4 g[2] = {sums[lane], sums[64 + lane]};
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t at = h * (kTileElems / 2) + 4 * lane, k = t.k + at;
        float p[4], m[4], v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            g[h][e] = g[h][e] * a.scale;
            if (clip)
                g[h][e] = g[h][e] * cf;
            p[e] = pv[h][e];
            m[e] = mv[h][e];
            v[e] = vv[h][e];
            adam(a.c, g[h][e], p[e], m[e], v[e]);
        }
        st_state<true>(a.master + k, f32x4{p[0], p[1], p[2], p[3]});
        st_state<true>(a.m + k, f32x4{m[0], m[1], m[2], m[3]});
        st_state<true>(a.v + k, f32x4{v[0], v[1], v[2], v[3]});
        if (a.main_grad)
            stf4_out(a.main_grad + k, g[h]);
        if (a.param)
            __builtin_nontemporal_store(u32x2{to_bf16x2(p[0], p[1]), to_bf16x2(p[2], p[3])},
                                        reinterpret_cast<u32x2 *>(a.param + (a.param_local ? t.k : t.w) + at));
        if (a.codes) {
            uint32_t c, s;
            round_quad(p, c, s);
            st_quad(a.codes, a.scales, a.mx_world ? t.world : t.local, h, c, s);
        }
    }
}

// Any other tile, by chunks.
__device__ __forceinline__ void step_edge(const MxStepArgs &a, const MxTile &t, bool clip, float cf) {
    const Slots own = slots_of(t.lo, t.own);
    const int64_t k = t.k + threadIdx.x * kChunk;
    float p[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        p[e] = 0.0f;
    if (t.lo < t.own) {
        float m[8], v[8], g[8];
        if (own.full()) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 pv = ld_state<true>(a.master + k + 4 * h), mv = ld_state<true>(a.m + k + 4 * h),
                            vv = ld_state<true>(a.v + k + 4 * h);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[4 * h + e] = pv[e];
                    m[4 * h + e] = mv[e];
                    v[4 * h + e] = vv[e];
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool in = e >= own.lo && e < own.hi;
                p[e] = in ? a.master[k + e] : 0.0f;
                m[e] = in ? a.m[k + e] : 0.0f;
                v[e] = in ? a.v[k + e] : 0.0f;
            }
        }
        sum_blocks<1, 0>(a.in, stored_at(a.in, t), g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            g[e] = g[e] * a.scale;
            if (clip)
                g[e] = g[e] * cf;
            if (e >= own.lo && e < own.hi)
                adam(a.c, g[e], p[e], m[e], v[e]);
        }
        if (own.full()) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                st_state<true>(a.master + k + 4 * h, f32x4{p[4 * h], p[4 * h + 1], p[4 * h + 2], p[4 * h + 3]});
                st_state<true>(a.m + k + 4 * h, f32x4{m[4 * h], m[4 * h + 1], m[4 * h + 2], m[4 * h + 3]});
                st_state<true>(a.v + k + 4 * h, f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]});
                if (a.main_grad)
                    stf4_out(a.main_grad + k + 4 * h, f32x4{g[4 * h], g[4 * h + 1], g[4 * h + 2], g[4 * h + 3]});
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e >= own.lo && e < own.hi) {
                    a.master[k + e] = p[e];
                    a.m[k + e] = m[e];
                    a.v[k + e] = v[e];
                    if (a.main_grad)
                        a.main_grad[k + e] = g[e];
                }
        }
        if (a.param)
            st_bf16(a.param + (a.param_local ? k : t.w + threadIdx.x * kChunk), p, own);
    }
    if (a.codes) {
        uint32_t c, s;
        round_block(p, c, s);
        st_block(a.codes, a.scales, a.mx_world ? t.world : t.local, c, s);
    }
}

// The occupancy bound tells the compiler how many registers a wave may have,
// and so how many of a tile's loads it puts in flight before the first wait:
// 4 waves a SIMD serve long launches of 8 and 16 contributions best (4778 and
// 2842 us; 4812 and 2926 with 5), 5 the short ones (GPT-2 small rank 78.9 us,
// 80.6 with 4, 82.9 with 6; fragmented 32.7, 34.1, 32.7) and other counts (3
// contributions of 3e8 1376 us, 1396 with 4; 12 of 1.5e8 790 and 799).
template <int kN, bool kShort>
__global__ __launch_bounds__(kBlock) __attribute__((amdgpu_waves_per_eu(1, kN > 0 && !kShort ? 4 : 5)))
void mx_step_kernel(MxStepArgs a) {
    __shared__ f32x4 sums[kTileElems / 4];
    const bool clip = a.coeff != nullptr;
    const float cf = clip ? *ro(a.coeff) : 1.0f;
    const int64_t iend = clip && cf != cf ? 0 : a.walk.count;   // NaN: found-inf, nothing changes
    for (int64_t i = blockIdx.x; i < iend; i += gridDim.x) {
        const MxTile t = local_tile(a.walk, launch_order(a.walk.by_xcd, a.walk.count, i));
        if (t.lo == 0 && t.own == kTileElems)
            step_whole<kN>(a, t, clip, cf, sums);
        else
            step_edge(a, t, clip, cf);
    }
}

// ---- rounding to MXFP4 ---------------------------------------------------------------------------

enum { kGrads, kGradsResidual, kMaster };   // what is rounded

// A tile that is not whole, by chunks.
template <int kSource>
__device__ __forceinline__ void quant_edge(const MxQuantArgs &a, const MxTile &t) {
    const Slots own = slots_of(t.lo, t.own);
    const int64_t at = (a.local ? t.k : t.w) + threadIdx.x * kChunk;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] = 0.0f;
        if (e >= own.lo && e < own.hi) {
            if constexpr (kSource == kMaster)
                x[e] = a.master[at + e];
            else
                x[e] = h_f32(a.grads[at + e]);
            if constexpr (kSource == kGradsResidual)
                x[e] = x[e] + a.residual[at + e];
        }
    }
    uint32_t c, s;
    round_block(x, c, s);
    st_block(a.codes, a.scales, a.world ? t.world : t.local, c, s);
    if (kSource == kGradsResidual && s != 255) {
        float y[8];
        values_of(c, scale_f32(s), y);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e >= own.lo && e < own.hi)
                a.residual[at + e] = x[e] - y[e];
    }
}

// A unit of whole tiles from t: bf16 by chunks, fp32 by quads (and the bf16
// beside it), so that every access covers a run without a gap; all loads
// first. The fp32 is non-temporal, like the step's state (1.2e8 elements with
// a residual 208 us, with plain accesses 257; the write-back of 1.25e8
// elements 93 and 109 us). Tile by tile it took 212 and 96 us.
template <int kSource>
__device__ __forceinline__ void quant_whole(const MxQuantArgs &a, const MxTile &t) {
    const int lane = int(threadIdx.x);
    constexpr int kRun = kMxUnit;
    const int64_t first = a.local ? t.k : t.w, to = a.world ? t.world : t.local;
    if constexpr (kSource == kGrads) {
        u32x4 r[kRun];
#pragma unroll
        for (int j = 0; j < kRun; ++j)
            r[j] = ld_rep(a.grads + first + j * kTileElems + lane * kChunk);
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            float x[8];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                x[2 * h] = lo_f32(r[j][h]);
                x[2 * h + 1] = hi_f32(r[j][h]);
            }
            uint32_t c, s;
            round_block(x, c, s);
            st_block(a.codes, a.scales, to + j, c, s);
        }
    } else {
        f32x4 f[2 * kRun];
        u32x2 r[2 * kRun];
#pragma unroll
        for (int q = 0; q < 2 * kRun; ++q) {
            const int64_t at = first + q * (kTileElems / 2) + 4 * lane;
            f[q] = ld_state<true>(kSource == kMaster ? a.master + at : a.residual + at);
            if constexpr (kSource == kGradsResidual)
                r[q] = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(a.grads + at));
        }
#pragma unroll
        for (int q = 0; q < 2 * kRun; ++q) {
            float x[4] = {f[q][0], f[q][1], f[q][2], f[q][3]};
            if constexpr (kSource == kGradsResidual) {
                x[0] = lo_f32(r[q][0]) + x[0];
                x[1] = hi_f32(r[q][0]) + x[1];
                x[2] = lo_f32(r[q][1]) + x[2];
                x[3] = hi_f32(r[q][1]) + x[3];
            }
            uint32_t c, s;
            round_quad(x, c, s);
            st_quad(a.codes, a.scales, to + q / 2, q % 2, c, s);
            if (kSource == kGradsResidual && s != 255) {
                const f32x2 y0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale_f32(s), 0);
                const f32x2 y1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale_f32(s), 1);
                st_state<true>(a.residual + first + q * (kTileElems / 2) + 4 * lane,
                               f32x4{x[0] - y0[0], x[1] - y0[1], x[2] - y1[0], x[3] - y1[1]});
            }
        }
    }
}

template <int kSource, bool kWorld>
__global__ __launch_bounds__(kBlock) void mx_quant_kernel(MxQuantArgs a) {
    for (int64_t i = blockIdx.x; i < a.walk.count; i += gridDim.x) {
        const MxUnit u = unit_at<kWorld>(a.walk, i);
        const MxTile t = tile_in(u.b, a.walk.dp, u.rank, u.tile);
        if (u.ntiles == kMxUnit && t.lo == 0 &&
            tile_in(u.b, a.walk.dp, u.rank, u.tile + kMxUnit - 1).own == kTileElems) {
            quant_whole<kSource>(a, t);
            continue;
        }
        for (int j = 0; j < u.ntiles; ++j)
            quant_edge<kSource>(a, tile_in(u.b, a.walk.dp, u.rank, u.tile + j));
    }
}

// ---- the gather ------------------------------------------------------------------------------------

__global__ __launch_bounds__(kBlock) void mx_gather_kernel(MxGatherArgs a) {
    for (int64_t i = blockIdx.x; i < a.walk.count; i += gridDim.x) {
        const MxUnit u = unit_at<true>(a.walk, i);
        const uint8_t *codes = a.in.codes[u.rank], *scales = a.in.scales[u.rank];
        const MxTile t = tile_in(u.b, a.walk.dp, u.rank, u.tile);
        const int64_t at = stored_at(a.in, t);
        uint32_t c[kMxUnit], s[kMxUnit];
        if (u.ntiles == kMxUnit && t.lo == 0 &&
            tile_in(u.b, a.walk.dp, u.rank, u.tile + kMxUnit - 1).hi == kTileElems) {
#pragma unroll
            for (int j = 0; j < kMxUnit; ++j)
                ld_block(codes, scales, at + j, c[j], s[j]);
#pragma unroll
            for (int j = 0; j < kMxUnit; ++j) {
                float x[8];
                values_of(c[j], scale_f32(s[j]), x);
                st_bf16(a.out + t.w + j * kTileElems + threadIdx.x * kChunk, x, {0, kChunk});
            }
        } else {
            for (int j = 0; j < u.ntiles; ++j) {
                const MxTile e = tile_in(u.b, a.walk.dp, u.rank, u.tile + j);
                ld_block(codes, scales, at + j, c[0], s[0]);
                float x[8];
                values_of(c[0], scale_f32(s[0]), x);
                st_bf16(a.out + e.w + threadIdx.x * kChunk, x, slots_of(e.lo, e.hi));
            }
        }
    }
}

// The form of a reduction of n contributions over `tiles` tiles. Measured,
// us, a tile a wave / 2 / 4 tiles at a time (waves per compute unit in
// brackets; 0: no cap):
//   2.5e8 to 1e9 slots: 8 contributions 1178 / 970 [0] / 985 [0];
//     16: 917 / 831 [10], 866 [0] / 836 [6]; 32: 885 / 797 [0] / 772 [6],
//     833 [0]; 64: 854 / 801 [0] / 756 [6]; 3e8 slots: 1: 240 / 158 [0] /
//     144 [0]; 3: 291 / 203 [0] / 189 [0]; 4: 293 / 191 [0] / 203 [0].
//   30 M slots: 8: 35.9 / 32.6 / 33.1; 32: 96.3 / 98.7 / 95.9.
//   15.5 M slots, 8: 19.5 / 20.1 / 20.3; 1e7 slots, 64: 60.2 / 68.4 / 66.2.
#ifndef ZDO_MX_WIDE_TILES
#define ZDO_MX_WIDE_TILES (int64_t(1) << 15)
#endif
struct ReduceForm {
    int tiles, waves;
};
ReduceForm reduce_form(int n, int64_t tiles) {
    if (tiles < ZDO_MX_WIDE_TILES)
        return {1, 0};
    if (n >= 32)
        return {4, 6};
    if (n <= 3)
        return {4, 0};
    return {2, n >= 16 ? 10 : 0};
}
// LDS to reserve beside the kernel's own.
unsigned reserve(int lds_per_cu, int waves, unsigned own) {
    const unsigned cap = lds_for_waves(lds_per_cu, waves);
    return cap > own ? cap - own : 0;
}

}  // namespace

hipError_t launch_mx_reduce(const MxReduceArgs &args, int lds_per_cu, hipStream_t stream) {
    MxReduceArgs a = args;
    const ReduceForm f = reduce_form(a.in.n, a.walk.count);
    if (f.tiles > 1)
        a.walk = args.units;
    else
        a.walk.by_xcd = 1;
    if (a.walk.count <= 0)
        return hipSuccess;
    const dim3 grid(grid_for(a.walk.count)), block(kBlock);
    const unsigned lds = reserve(lds_per_cu, f.waves, unsigned(f.tiles * kTileElems * sizeof(uint16_t)));
    if (f.tiles == 1)
        hipLaunchKernelGGL(mx_reduce_kernel, grid, block, 0, stream, a);
    else if (a.in.n < kFew)
        hipLaunchKernelGGL((mx_reduce_wide_kernel<4, kFew>), grid, block, lds, stream, a);
    else if (f.tiles == 2)
        hipLaunchKernelGGL((mx_reduce_wide_kernel<2, kBatch>), grid, block, lds, stream, a);
    else
        hipLaunchKernelGGL((mx_reduce_wide_kernel<4, kBatch>), grid, block, lds, stream, a);
    return hipGetLastError();
}

hipError_t launch_mx_norm(const MxNormArgs &args, double *norm_sq, hipStream_t stream) {
    MxNormArgs a = args;
    if (a.walk.count <= kNormAtOnceTiles && a.walk.count * a.in.n <= kNormAtOnceWork) {
        hipLaunchKernelGGL(mx_norm_at_once_kernel, dim3(1), dim3(64, kSumWaves), 0, stream, a, norm_sq);
        return hipGetLastError();
    }
    const ReduceForm f = reduce_form(a.in.n, a.walk.count);
    if (f.tiles > 1)
        a.walk = args.units;
    else
        a.walk.by_xcd = 1;
    const dim3 grid(grid_for(a.walk.count < kMxNormWaves ? a.walk.count : kMxNormWaves)), block(kBlock);
    if (f.tiles == 1)
        hipLaunchKernelGGL(mx_norm_kernel, grid, block, 0, stream, a);
    else if (a.in.n < kFew)
        hipLaunchKernelGGL((mx_norm_wide_kernel<4, kFew>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((mx_norm_wide_kernel<2, kBatch>), grid, block, 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(mx_sum_kernel, dim3(1), dim3(64, kSumWaves), 0, stream, a.partial, int64_t(grid.x), norm_sq);
    return hipGetLastError();
}

// Counts of contributions that have a kernel of their own: 8 and 16, the usual
// ones of a node and of two. Against the kernel for any count, long launches:
// 8 4960 us instead of 5063, 16 2906 instead of 3044. 2, 3, 4 and 12 would gain
// 2 to 3% (3e8 slots of 2 1321 instead of 1358, of 3 1362 and 1399, of 4 1393
// and 1432, 1.5e8 of 12 783 and 797; 8e6 of 4 40.2 and 42.8, but 2e6 of 4 12.3
// and 11.2) at two more kernels each and are left to the one for any count; 1,
// 24 and 32 would lose (1314 and 1308, 9e7 of 24 610 and 591, 2.5e8 of 32 1913
// and 1826).
// Waves that share a compute unit in the step. Long launches, Llama-3-8B
// shapes: 8 contributions with all loads in flight 4809 us at 9 waves (8:
// 4802, 10: 5227, 12: 5404, 6: 5901), 16 2871 us (8: 2875, 12: 2882); other
// counts 14 (3 contributions: 1331, at 12 1342 and at 16 1381; 32: 1828, 1826
// and 1838; 12: 812, 814 and 820). Short launches take 16 (GPT-2 small rank:
// the same from 10 up; fragmented, 16 contributions: 34.6 us, 36.3 at 10).
// Tiles go by XCD in short launches (GPT-2 small rank 80.3 us, 82.7 in
// dispatch order; 64 contributions of 1e7 elements 107.4 and 109.5) and from 8
// contributions in long ones, where the scales weigh enough (8: 4800 us, 4975
// in dispatch order; 12: 813 and 847; 16: 2887 and 3062; 32: 1819 and 1893; but
// 5: 716 and 718, 3: 1402 and 1381, 1: 1347 and 1311).
constexpr int kStepWavesFixed = 9, kStepWaves = 14, kStepWavesShort = 16;

hipError_t launch_mx_step(const MxStepArgs &args, int lds_per_cu, hipStream_t stream) {
    if (args.walk.count <= 0)
        return hipSuccess;
    MxStepArgs a = args;
    const bool is_short = a.walk.count < kShortLaunch;
    a.walk.by_xcd = is_short || a.in.n >= 8;
    const dim3 grid(grid_for(a.walk.count)), block(kBlock);
    const bool fixed = a.in.n == 8 || a.in.n == 16;
    const unsigned lds = reserve(lds_per_cu, is_short ? kStepWavesShort : fixed ? kStepWavesFixed : kStepWaves,
                                 kTileElems * sizeof(float));
    if (a.in.n == 8 && is_short)
        hipLaunchKernelGGL((mx_step_kernel<8, true>), grid, block, lds, stream, a);
    else if (a.in.n == 8)
        hipLaunchKernelGGL((mx_step_kernel<8, false>), grid, block, lds, stream, a);
    else if (a.in.n == 16 && is_short)
        hipLaunchKernelGGL((mx_step_kernel<16, true>), grid, block, lds, stream, a);
    else if (a.in.n == 16)
        hipLaunchKernelGGL((mx_step_kernel<16, false>), grid, block, lds, stream, a);
    else
        hipLaunchKernelGGL((mx_step_kernel<0, true>), grid, block, lds, stream, a);
    return hipGetLastError();
}

// No cap on the waves: 1.2e8 elements 54 us (62 at 16 waves per compute unit),
// 1e9 406 us (425 at 16), with a residual 208 us (206 at 12, 212 at 16).
hipError_t launch_mx_quant(const MxQuantArgs &a, hipStream_t stream) {
    if (a.walk.count <= 0)
        return hipSuccess;
    const dim3 grid(grid_for(a.walk.count)), block(kBlock);
    if (!a.grads)
        hipLaunchKernelGGL((mx_quant_kernel<kMaster, false>), grid, block, 0, stream, a);
    else if (a.residual && a.local)
        hipLaunchKernelGGL((mx_quant_kernel<kGradsResidual, false>), grid, block, 0, stream, a);
    else if (a.residual)
        hipLaunchKernelGGL((mx_quant_kernel<kGradsResidual, true>), grid, block, 0, stream, a);
    else if (a.local)
        hipLaunchKernelGGL((mx_quant_kernel<kGrads, false>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((mx_quant_kernel<kGrads, true>), grid, block, 0, stream, a);
    return hipGetLastError();
}

// 20 waves per compute unit: 1e9 elements 408 us, 404 at 16, 547 at 8, 442
// without a cap; 1.2e8 elements 52.6, 53.4, 70.4 and 54.9 us.
constexpr int kMxGatherWaves = 20;

hipError_t launch_mx_gather(const MxGatherArgs &a, int lds_per_cu, hipStream_t stream) {
    if (a.walk.count <= 0)
        return hipSuccess;
    hipLaunchKernelGGL(mx_gather_kernel, dim3(grid_for(a.walk.count)), dim3(kBlock),
                       lds_for_waves(lds_per_cu, kMxGatherWaves), stream, a);
    return hipGetLastError();
}

}  // namespace zdo
