// Argument checks and host-side constants that the C-ABI's files share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "kernels.h"
#include "zdo_internal.h"

namespace zdo {

struct Span {
    uintptr_t lo, hi;
};

inline Span span_of(const void *p, int64_t elems, int64_t elem_bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + uintptr_t(elems) * uintptr_t(elem_bytes)};
}

inline bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi; }

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool aligned_to(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int fail(int code, const std::string &msg) {
    set_error(msg);
    return code;
}

// The plan must be device-ready, and on the current device.
inline int check_plan(const zdo_plan *plan, const char *fn) {
    if (!plan)
        return fail(ZDO_EINVAL, std::string(fn) + ": plan is NULL");
    if (!plan->d_table)
        return fail(ZDO_EHIP, std::string(fn) + ": the plan has no device table (no HIP device when it was built)");
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess)
        return fail(ZDO_EHIP, std::string(fn) + ": hipGetDevice failed");
    if (dev != plan->device)
        return fail(ZDO_EINVAL, std::string(fn) + ": the plan was built on device " + std::to_string(plan->device) +
                                    " but device " + std::to_string(dev) + " is current");
    return ZDO_OK;
}

inline int check_coords(int32_t c, const char *fn, const char *what) {
    if (c != ZDO_WORLD && c != ZDO_LOCAL)
        return fail(ZDO_EINVAL, std::string(fn) + ": " + what + " must be ZDO_WORLD or ZDO_LOCAL");
    return ZDO_OK;
}

inline int check_ptr(const void *p, const char *fn, const char *what) {
    if (!p)
        return fail(ZDO_EINVAL, std::string(fn) + ": " + what + " is NULL");
    if (!aligned16(p))
        return fail(ZDO_EALIGN, std::string(fn) + ": " + what + " is not 16-byte aligned");
    return ZDO_OK;
}

inline int64_t extent(const zdo_plan *p, int32_t coords) { return coords == ZDO_WORLD ? p->buffer_numel : p->shard_numel; }

inline int launch_result(hipError_t e, const char *fn) {
    if (e != hipSuccess)
        return fail(ZDO_EHIP, std::string(fn) + ": launch failed: " + hipGetErrorString(e));
    return ZDO_OK;
}

inline int check_buckets(const zdo_plan *plan, int32_t b0, int32_t b1, const char *fn) {
    if (b0 < 0 || b1 < b0 || b1 > int32_t(plan->buckets.size()))
        return fail(ZDO_EINVAL, std::string(fn) + ": need 0 <= bucket_begin <= bucket_end <= " +
                                    std::to_string(plan->buckets.size()));
    return ZDO_OK;
}

// Adam's hyper-parameters (abi.cpp): their checks, and the constants of one
// step.
int check_adam(const zdo_adam *hp, const char *fn);
AdamConst adam_const(const zdo_adam &hp);

}  // namespace zdo
