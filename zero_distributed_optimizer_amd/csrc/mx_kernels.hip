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
// scale given as an fp32 whose exponent field is the E8M0 byte. Checked on
// the device over all 256 scales x 256 pairs, and over every bf16 and 2^20
// random fp32 values: exact, subnormal results kept, scale 255 gives NaN,
// rounding to nearest even and saturating at 6.
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
    int rank;
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
    t.rank = r;
    return t;
}

// The bucket holding LOCAL tile or unit x.
template <bool kUnits>
__device__ __forceinline__ ro_ptr<MxBucket> bucket_of(const MxWalk &wk, int64_t x) {
    const ro_ptr<MxBucket> all = ro(wk.buckets);
    int32_t b = int32_t(ro(wk.group)[x / kTileGroup]);
    while (b + 1 < wk.nbuckets && (kUnits ? all[b + 1].unit0 : all[b + 1].tile0) <= x)
        ++b;
    return all + b;
}

// The tile at launch index i of a walk over the rank's tiles.
__device__ __forceinline__ MxTile local_tile(const MxWalk &wk, int64_t i) {
    const int64_t x = wk.first + i;
    const ro_ptr<MxBucket> b = bucket_of<false>(wk, x);
    return tile_in(b, wk.dp, wk.rank, int(x - b->tile0));
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

// A lane's 8 values to a word of codes, with the scale of its block (4
// lanes): the largest magnitude's bits over the block, by integer compare, so
// that Inf and NaN win; byte = max(0, exponent - 2). Every lane of the wave
// takes part.
__device__ __forceinline__ void round_block(const float x[8], uint32_t &codes, uint32_t &byte) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t a = __float_as_uint(x[e]) & 0x7fffffffu;
        top = a > top ? a : top;
    }
    // lanes 1 and 2 away within the quad
    const uint32_t t1 = uint32_t(__builtin_amdgcn_mov_dpp(int(top), 0xB1, 0xf, 0xf, true));
    top = t1 > top ? t1 : top;
    const uint32_t t2 = uint32_t(__builtin_amdgcn_mov_dpp(int(top), 0x4E, 0xf, 0xf, true));
    top = t2 > top ? t2 : top;
    const uint32_t ex = top >> 23;
    byte = ex > 2 ? ex - 2 : 0;
    const float s = scale_f32(byte);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], s, 3);
    const bool bad = ex == 255;
    codes = bad ? 0 : c;
    byte = bad ? 255 : byte;
}

// The lane's word of codes of tile t, and its block's scale.
__device__ __forceinline__ void ld_block(const uint8_t *codes, const uint8_t *scales, int64_t t, uint32_t &c,
                                         uint32_t &s) {
    c = __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(codes + t * (kTileElems / 2)) + threadIdx.x);
    s = scales[t * kMxTileBlocks + threadIdx.x / 4];
}
__device__ __forceinline__ void st_block(uint8_t *codes, uint8_t *scales, int64_t t, uint32_t c, uint32_t s) {
    reinterpret_cast<uint32_t *>(codes + t * (kTileElems / 2))[threadIdx.x] = c;
    if (threadIdx.x % 4 == 0)
        scales[t * kMxTileBlocks + threadIdx.x / 4] = uint8_t(s);
}

// The sum of the contributions over the lane's 8 slots of tile t, in the
// order given, from -0 (which adds to any first term exactly). Batches of
// kBatch contributions have their loads in flight together.
constexpr int kBatch = 8;
template <int kCount>
__device__ __forceinline__ void add_batch(const MxInputs &in, int j, int64_t t, float acc[8]) {
    uint32_t c[kCount], s[kCount];
#pragma unroll
    for (int i = 0; i < kCount; ++i)
        ld_block(in.codes[j + i], in.scales[j + i], t, c[i], s[i]);
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
        float x[8];
        values_of(c[i], scale_f32(s[i]), x);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            acc[e] = acc[e] + x[e];
    }
}
__device__ __forceinline__ void sum_blocks(const MxInputs &in, const MxTile &t, float acc[8]) {
    const int64_t at = in.world ? t.world : t.local;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        acc[e] = -0.0f;
    int j = 0;
    for (; j + kBatch <= in.n; j += kBatch)
        add_batch<kBatch>(in, j, at, acc);
    if (in.n & 4) {
        add_batch<4>(in, j, at, acc);
        j += 4;
    }
    if (in.n & 2) {
        add_batch<2>(in, j, at, acc);
        j += 2;
    }
    if (in.n & 1)
        add_batch<1>(in, j, at, acc);
}

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

__global__ __launch_bounds__(kBlock) void mx_reduce_kernel(MxReduceArgs a) {
    for (int64_t i = blockIdx.x; i < a.walk.count; i += gridDim.x) {
        const MxTile t = local_tile(a.walk, i);
        if (t.lo >= t.hi)
            continue;
        float acc[8];
        sum_blocks(a.in, t, acc);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            acc[e] = acc[e] * a.scale;
        st_bf16(a.out + (a.out_local ? t.k : t.w) + threadIdx.x * kChunk, acc, slots_of(t.lo, t.hi));
    }
}

__global__ __launch_bounds__(kBlock) void mx_norm_kernel(MxNormArgs a) {
    for (int64_t i = blockIdx.x; i < a.walk.count; i += gridDim.x) {
        const MxTile t = local_tile(a.walk, i);
        double s = 0.0;
        if (t.lo < t.own) {
            float acc[8];
            sum_blocks(a.in, t, acc);
            const Slots own = slots_of(t.lo, t.own);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double g = double(acc[e] * a.scale);
                if (e >= own.lo && e < own.hi)
                    s = s + g * g;
            }
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1)
            s = s + __shfl_xor(s, off, 64);
        if (threadIdx.x == 0)
            a.partial[i] = s;
    }
}

template <bool kNT>
__global__ __launch_bounds__(kBlock) void mx_step_kernel(MxStepArgs a) {
    const bool clip = a.coeff != nullptr;
    const float cf = clip ? *ro(a.coeff) : 1.0f;
    const int64_t iend = clip && cf != cf ? 0 : a.walk.count;   // NaN: found-inf, nothing changes
    for (int64_t i = blockIdx.x; i < iend; i += gridDim.x) {
        const MxTile t = local_tile(a.walk, i);
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
                    const f32x4 pv = ld_state<kNT>(a.master + k + 4 * h), mv = ld_state<kNT>(a.m + k + 4 * h),
                                vv = ld_state<kNT>(a.v + k + 4 * h);
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
            sum_blocks(a.in, t, g);
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
                    st_state<kNT>(a.master + k + 4 * h, f32x4{p[4 * h], p[4 * h + 1], p[4 * h + 2], p[4 * h + 3]});
                    st_state<kNT>(a.m + k + 4 * h, f32x4{m[4 * h], m[4 * h + 1], m[4 * h + 2], m[4 * h + 3]});
                    st_state<kNT>(a.v + k + 4 * h, f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]});
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
}

// kMaster: the fp32 master; otherwise bf16 gradients, plus a residual if
// there is one.
template <bool kMaster, bool kWorld, bool kNT>
__global__ __launch_bounds__(kBlock) void mx_quant_kernel(MxQuantArgs a) {
    for (int64_t i = blockIdx.x; i < a.walk.count; i += gridDim.x) {
        const MxUnit u = unit_at<kWorld>(a.walk, i);
        for (int j = 0; j < u.ntiles; ++j) {
            const MxTile t = tile_in(u.b, a.walk.dp, u.rank, u.tile + j);
            const Slots own = slots_of(t.lo, t.own);
            const int64_t at = (a.local ? t.k : t.w) + threadIdx.x * kChunk;
            float x[8];
            if constexpr (kMaster) {
                if (own.full()) {
                    const f32x4 x0 = ld_state<kNT>(a.master + at), x1 = ld_state<kNT>(a.master + at + 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[e] = x0[e];
                        x[4 + e] = x1[e];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[e] = e >= own.lo && e < own.hi ? a.master[at + e] : 0.0f;
                }
            } else {
                if (own.full()) {
                    const u32x4 r = ld_rep(a.grads + at);
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        x[2 * h] = lo_f32(r[h]);
                        x[2 * h + 1] = hi_f32(r[h]);
                    }
                    if (a.residual) {
                        const f32x4 r0 = ldf4(a.residual + at), r1 = ldf4(a.residual + at + 4);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[e] = x[e] + r0[e];
                            x[4 + e] = x[4 + e] + r1[e];
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[e] = 0.0f;
                        if (e >= own.lo && e < own.hi) {
                            x[e] = h_f32(a.grads[at + e]);
                            if (a.residual)
                                x[e] = x[e] + a.residual[at + e];
                        }
                    }
                }
            }
            uint32_t c, s;
            round_block(x, c, s);
            st_block(a.codes, a.scales, a.world ? t.world : t.local, c, s);
            if (!kMaster && a.residual && s != 255) {
                float y[8];
                values_of(c, scale_f32(s), y);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[e] = x[e] - y[e];
                if (own.full()) {
                    stf4(a.residual + at, f32x4{y[0], y[1], y[2], y[3]});
                    stf4(a.residual + at + 4, f32x4{y[4], y[5], y[6], y[7]});
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e >= own.lo && e < own.hi)
                            a.residual[at + e] = y[e];
                }
            }
        }
    }
}

__global__ __launch_bounds__(kBlock) void mx_gather_kernel(MxGatherArgs a) {
    for (int64_t i = blockIdx.x; i < a.walk.count; i += gridDim.x) {
        const MxUnit u = unit_at<true>(a.walk, i);
        const uint8_t *codes = a.in.codes[u.rank], *scales = a.in.scales[u.rank];
        uint32_t c[kMxUnit], s[kMxUnit];
        const MxTile t0 = tile_in(u.b, a.walk.dp, u.rank, u.tile);
        const int64_t at = a.in.world ? t0.world : t0.local;
#pragma unroll
        for (int j = 0; j < kMxUnit; ++j)
            if (j < u.ntiles)
                ld_block(codes, scales, at + j, c[j], s[j]);
#pragma unroll
        for (int j = 0; j < kMxUnit; ++j)
            if (j < u.ntiles) {
                const MxTile t = tile_in(u.b, a.walk.dp, u.rank, u.tile + j);
                float x[8];
                values_of(c[j], scale_f32(s[j]), x);
                st_bf16(a.out + t.w + threadIdx.x * kChunk, x, slots_of(t.lo, t.hi));
            }
    }
}

}  // namespace

hipError_t launch_mx_reduce(const MxReduceArgs &a, int lds_per_cu, hipStream_t stream) {
    if (a.walk.count <= 0)
        return hipSuccess;
    hipLaunchKernelGGL(mx_reduce_kernel, dim3(grid_for(a.walk.count)), dim3(kBlock), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_mx_norm(const MxNormArgs &a, double *norm_sq, int lds_per_cu, hipStream_t stream) {
    if (a.walk.count > 0) {
        hipLaunchKernelGGL(mx_norm_kernel, dim3(grid_for(a.walk.count)), dim3(kBlock), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return launch_tile_sums(a.partial, a.walk.count, norm_sq, stream);
}

hipError_t launch_mx_step(const MxStepArgs &a, int lds_per_cu, hipStream_t stream) {
    if (a.walk.count <= 0)
        return hipSuccess;
    const dim3 grid(grid_for(a.walk.count)), block(kBlock);
    if (state_nontemporal(a.state_numel))
        hipLaunchKernelGGL(mx_step_kernel<true>, grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL(mx_step_kernel<false>, grid, block, 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_mx_quant(const MxQuantArgs &a, int lds_per_cu, hipStream_t stream) {
    if (a.walk.count <= 0)
        return hipSuccess;
    const dim3 grid(grid_for(a.walk.count)), block(kBlock);
    if (a.grads) {
        if (a.local)
            hipLaunchKernelGGL((mx_quant_kernel<false, false, false>), grid, block, 0, stream, a);
        else
            hipLaunchKernelGGL((mx_quant_kernel<false, true, false>), grid, block, 0, stream, a);
    } else if (state_nontemporal(a.state_numel)) {
        hipLaunchKernelGGL((mx_quant_kernel<true, false, true>), grid, block, 0, stream, a);
    } else {
        hipLaunchKernelGGL((mx_quant_kernel<true, false, false>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_mx_gather(const MxGatherArgs &a, int lds_per_cu, hipStream_t stream) {
    if (a.walk.count <= 0)
        return hipSuccess;
    hipLaunchKernelGGL(mx_gather_kernel, dim3(grid_for(a.walk.count)), dim3(kBlock), 0, stream, a);
    return hipGetLastError();
}

}  // namespace zdo
