// What the device files share: bf16 conversions, the cache policies of their
// loads and stores, Adam's arithmetic, and the launch geometry's helpers.
#pragma once

#include <hip/hip_runtime.h>

#include "kernels.h"

#pragma clang fp contract(off)

namespace zdo {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// ---- bf16 ----------------------------------------------------------------------
// A bf16 is the top half of an fp32: widening is a shift or a mask.
__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float h_f32(uint16_t h) { return __uint_as_float(uint32_t(h) << 16); }

// Two fp32 to their nearest bf16 (ties to even), packed a | b << 16: one
// v_cvt_pk_bf16_f32 on gfx950.
__device__ __forceinline__ uint32_t to_bf16x2(float a, float b) {
    f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// ---- memory ------------------------------------------------------------------------
// The replicas are read exactly once per launch: their loads carry the
// non-temporal hint, which keeps them from displacing the fp32 state in the
// caches (measured: +2% on a 42 GB step, +18% when the state fits the
// 256 MB Infinity Cache between steps). The write-only outputs (parameters,
// reduced gradient, main grad) are non-temporal stores too (Llama-3-8B-shaped
// step: 6.83 ms in every run against 6.83-7.48 ms with plain stores;
// Llama-3-70B-shaped reduce-scatter 7% faster). The fp32 state is read and
// then rewritten. While it is at most a few times the 256 MB Infinity
// Cache, plain loads and stores serve it best (GPT-2-shaped step, 187 MB of
// state, back to back: 97.5 us against 109.8 us with non-temporal state
// accesses). Beyond 1 GiB (see launch_step) the step loads and stores it
// non-temporally as well (Llama-3-8B-shaped step: 6.92-6.98 -> 6.75-6.77
// ms); non-temporal stores after plain loads of the same lines are far
// slower than either (3.4-3.6 TB/s).
__device__ __forceinline__ u32x4 ld_rep(const uint16_t *p) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
}
__device__ __forceinline__ f32x4 ldf4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }
__device__ __forceinline__ void st16_out(uint16_t *p, u32x4 v) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p));
}
__device__ __forceinline__ void stf4(float *p, f32x4 v) { *reinterpret_cast<f32x4 *>(p) = v; }
__device__ __forceinline__ void stf4_out(float *p, f32x4 v) {
    __builtin_nontemporal_store(v, reinterpret_cast<f32x4 *>(p));
}
template <bool kNT>
__device__ __forceinline__ f32x4 ld_state(const float *p) {
    if constexpr (kNT)
        return __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p));
    else
        return ldf4(p);
}
template <bool kNT>
__device__ __forceinline__ void st_state(float *p, f32x4 v) {
    if constexpr (kNT)
        __builtin_nontemporal_store(v, reinterpret_cast<f32x4 *>(p));
    else
        stf4(p, v);
}

// The plan's tables are read-only for the life of the plan: read through the
// constant address space, the compiler fetches them with scalar loads (one
// per wave, into scalar registers) instead of 64-lane vector loads of one
// address.
template <typename T>
using ro_ptr = const __attribute__((address_space(4))) T *;
template <typename T>
__device__ __forceinline__ ro_ptr<T> ro(const T *p) {
    return (ro_ptr<T>)(p);
}
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

// ---- Adam --------------------------------------------------------------------------------------
__device__ __forceinline__ void adam(const AdamConst &c, float g, float &p, float &m, float &v) {
    const float m1 = c.b1 * m;
    const float m2 = c.omb1 * g;
    const float mn = m1 + m2;
    const float gg = g * g;
    const float v1 = c.b2 * v;
    const float v2 = c.omb2 * gg;
    const float vn = v1 + v2;
    const float mh = mn / c.bc1;
    const float vh = vn / c.bc2;
    const float den = __builtin_sqrtf(vh) + c.eps;
    const float u = mh / den;
    const float wdp = c.wd * p;
    const float u2 = u + wdp;
    const float st = c.lr * u2;
    p = p - st;
    m = mn;
    v = vn;
}

// ---- launch geometry ------------------------------------------------------------------------
// Enough blocks to cover every tile once, up to a cap that keeps the grid's
// work-item count in range; larger launches loop over tiles (every kernel's
// tile loop steps by gridDim.x). A build with a small cap makes every
// launch take that loop.
#ifndef ZDO_MAX_GRID
#define ZDO_MAX_GRID (int64_t(1) << 24)
#endif
constexpr int64_t kMaxGrid = ZDO_MAX_GRID;
static_assert(kMaxGrid >= 1 && kMaxGrid <= (int64_t(1) << 24), "grid cap out of range");

inline unsigned grid_for(int64_t ntiles) {
    return unsigned(ntiles < kMaxGrid ? ntiles : kMaxGrid);
}

// LDS per workgroup that lets at most `waves` waves share a compute unit.
inline unsigned lds_for_waves(int lds_per_cu, int waves) {
    if (waves <= 0 || lds_per_cu <= 0)
        return 0;
    const int waves_per_group = kBlock / 64;
    int groups = waves / waves_per_group;
    if (groups < 4 / waves_per_group + (waves_per_group > 4))
        groups = 4 / waves_per_group + (waves_per_group > 4);
    return unsigned(lds_per_cu / groups) & ~127u;
}

}  // namespace
}  // namespace zdo
