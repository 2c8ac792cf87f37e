// What the vocabulary matrix's device files share: accesses of rows that start at
// any element, and the softmax's statistics.
#pragma once

#include <hip/hip_runtime.h>

#include "device.h"

#pragma clang fp contract(off)

namespace zdo {
namespace {

// 16 and 8 bytes at any address that is aligned to an element; gfx950 takes them in
// one instruction.
typedef u32x4 loose_u32x4 __attribute__((aligned(2)));
typedef u32x2 loose_u32x2 __attribute__((aligned(2)));
typedef f32x4 loose_f32x4 __attribute__((aligned(4)));

// What the exponentials of values up to `top` are taken relative to: `top`, or 0
// where that is infinite (the difference would be NaN: the sum is then 0 or
// infinite, as it should be).
__device__ __forceinline__ float base_of(float top) { return fabsf(top) < INFINITY ? top : 0.0f; }

// The largest value and the sum of exponentials relative to it (to base_of it) of
// two sets of values together. A set whose largest is -Inf adds nothing (or, of
// NaN only, NaN).
__device__ __forceinline__ float2 join_softmax(float2 x, float2 y) {
    const float top = fmaxf(x.x, y.x), base = base_of(top);
    const float fx = x.x == -INFINITY ? 0.0f : __expf(base_of(x.x) - base);
    const float fy = y.x == -INFINITY ? 0.0f : __expf(base_of(y.x) - base);
    return {top, x.y * fx + y.y * fy};
}

}  // namespace
}  // namespace zdo
