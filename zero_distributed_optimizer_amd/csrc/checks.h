// Argument checks and host-side constants that the C-ABI's files share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "kernels.h"
#include "zdo_internal.h"

namespace zdo {

// The bytes [lo, hi) of an array; of rows with gaps between them those `width` bytes
// that follow lo and every `step` bytes from it (step = 0: no gaps).
struct Span {
    uintptr_t lo, hi, step, width;
};

inline Span span_of(const void *p, int64_t elems, int64_t elem_bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + uintptr_t(elems) * uintptr_t(elem_bytes), 0, 0};
}

// n rows of dim elements, one every `stride` >= dim (of one row not looked at).
inline Span span_of_rows(const void *p, int64_t n, int64_t dim, int64_t stride, int64_t elem_bytes) {
    if (n <= 1)
        return span_of(p, n == 1 ? dim : 0, elem_bytes);
    Span s = span_of(p, (n - 1) * stride + dim, elem_bytes);
    if (stride > dim) {
        s.step = uintptr_t(stride * elem_bytes);
        s.width = uintptr_t(dim * elem_bytes);
    }
    return s;
}

// Whether two arrays share a byte. Rows may lie in the gaps of rows whose step is the
// same, and an array without gaps within one; with steps that differ, arrays whose
// extents meet count as sharing.
inline bool overlap(Span a, Span b) {
    if (!(a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi))
        return false;
    if (a.step == b.step ? a.step == 0 : a.step && b.step)
        return true;
    const uintptr_t step = a.step ? a.step : b.step;
    const uintptr_t wide_a = a.step ? a.width : a.hi - a.lo, wide_b = b.step ? b.width : b.hi - b.lo;
    if (wide_a > step || wide_b > step - wide_a)
        return true;
    // where b's rows begin, from a's
    const uintptr_t off = b.lo >= a.lo ? (b.lo - a.lo) % step : (step - (a.lo - b.lo) % step) % step;
    return off < wide_a || off > step - wide_b;
}

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

// A call's body: no exception leaves the C entry.
template <typename F>
int guarded(F body) {
    try {
        return body();
    } catch (...) {
        set_error("out of memory");   // short enough to need no allocation
        return ZDO_ENOMEM;
    }
}

// The buffers of one call: what it writes must not overlap anything else of
// it.
struct Buffers {
    static constexpr int kMaxReads = 2 * ZDO_MAX_REPLICAS + 2, kMaxWrites = 8;
    Span read[kMaxReads], write[kMaxWrites];
    const char *read_name[kMaxReads], *write_name[kMaxWrites];
    int nread = 0, nwrite = 0;

    void reads(Span s, const char *name) {
        read[nread] = s;
        read_name[nread++] = name;
    }
    void writes(Span s, const char *name) {
        write[nwrite] = s;
        write_name[nwrite++] = name;
    }
    int check(const char *fn) const {
        for (int i = 0; i < nwrite; ++i) {
            for (int k = i + 1; k < nwrite; ++k)
                if (overlap(write[i], write[k]))
                    return fail(ZDO_EALIAS, std::string(fn) + ": " + write_name[i] + " overlaps " + write_name[k]);
            for (int k = 0; k < nread; ++k)
                if (overlap(write[i], read[k]))
                    return fail(ZDO_EALIAS, std::string(fn) + ": " + write_name[i] + " overlaps " + read_name[k]);
        }
        return ZDO_OK;
    }
};

// Adam's hyper-parameters (abi.cpp): their checks, and the constants of one
// step.
int check_adam(const zdo_adam *hp, const char *fn);
AdamConst adam_const(const zdo_adam &hp);

}  // namespace zdo
