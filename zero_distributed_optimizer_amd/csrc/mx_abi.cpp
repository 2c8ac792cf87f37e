// The C-ABI of the MXFP4 calls: argument checks and launches. Declared and
// documented in include/zdo_mx.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>

#include "checks.h"
#include "mx.h"
#include "zdo_mx.h"

namespace zdo {
namespace {

int64_t mx_tiles(const zdo_plan *p, int32_t coords) { return p->mx_tiles * (coords == ZDO_WORLD ? p->dp_size : 1); }

int64_t mx_blocks(const zdo_plan *p, int32_t coords) { return mx_tiles(p, coords) * kMxTileBlocks; }

// The coordinates of a storage, and that its tiles can be numbered.
int check_storage(const zdo_plan *p, int32_t coords, const char *fn, const char *what) {
    if (int rc = check_coords(coords, fn, what))
        return rc;
    if (mx_tiles(p, coords) > kMxMaxTiles)
        return fail(ZDO_EINVAL, std::string(fn) + ": the plan's MXFP4 storage has " +
                                    std::to_string(mx_tiles(p, coords)) + " tiles, more than " +
                                    std::to_string(kMxMaxTiles));
    return ZDO_OK;
}

// n storages to be read.
int take_inputs(const zdo_plan *p, const uint8_t *const *codes, const uint8_t *const *scales, int32_t n,
                int32_t coords, const char *fn, MxInputs &in, Buffers &bufs) {
    if (n < 1 || n > ZDO_MAX_REPLICAS)
        return fail(ZDO_EINVAL, std::string(fn) + ": n must be in [1, " + std::to_string(ZDO_MAX_REPLICAS) + "]");
    if (int rc = check_storage(p, coords, fn, "coords"))
        return rc;
    if (!codes || !scales)
        return fail(ZDO_EINVAL, std::string(fn) + ": codes or scales list is NULL");
    for (int32_t j = 0; j < n; ++j) {
        if (int rc = check_ptr(codes[j], fn, "codes[j]"))
            return rc;
        if (int rc = check_ptr(scales[j], fn, "scales[j]"))
            return rc;
        in.codes[j] = codes[j];
        in.scales[j] = scales[j];
        bufs.reads(span_of(codes[j], mx_blocks(p, coords), kMxBlock / 2), "the codes");
        bufs.reads(span_of(scales[j], mx_blocks(p, coords), 1), "the scales");
    }
    in.n = n;
    in.world = coords == ZDO_WORLD;
    return ZDO_OK;
}

// A storage to be written.
int take_storage(const zdo_plan *p, uint8_t *codes, uint8_t *scales, int32_t coords, const char *fn, Buffers &bufs) {
    if (int rc = check_ptr(codes, fn, "codes"))
        return rc;
    if (int rc = check_ptr(scales, fn, "scales"))
        return rc;
    bufs.writes(span_of(codes, mx_blocks(p, coords), kMxBlock / 2), "the written codes");
    bufs.writes(span_of(scales, mx_blocks(p, coords), 1), "the written scales");
    return ZDO_OK;
}

// A walk over buckets [b0, b1): the rank's tiles, or units of the rank's
// ranges or of every rank's.
MxWalk walk_of(const zdo_plan *p, int32_t b0, int32_t b1, bool units, bool world) {
    auto start = [&](int32_t b) {
        const bool end = size_t(b) == p->mx_buckets.size();
        const int64_t x = units ? (end ? p->mx_units : p->mx_buckets[size_t(b)].unit0)
                                : (end ? p->mx_tiles : p->mx_buckets[size_t(b)].tile0);
        return x * (world ? p->dp_size : 1);
    };
    MxWalk w{};
    w.buckets = p->d_mx_buckets;
    w.group = units ? p->d_mx_unit_group : p->d_mx_tile_group;
    w.dp = p->dp_size;
    w.rank = p->rank;
    w.first = start(b0);
    w.count = start(b1) - w.first;
    return w;
}

int32_t nbuckets(const zdo_plan *p) { return int32_t(p->mx_buckets.size()); }

}  // namespace
}  // namespace zdo

using namespace zdo;

extern "C" {

int64_t zdo_plan_mx_blocks(const zdo_plan *p, int32_t coords) {
    if (!p || (coords != ZDO_WORLD && coords != ZDO_LOCAL))
        return -1;
    return mx_blocks(p, coords);
}

int zdo_plan_mx_buckets(const zdo_plan *p, zdo_mx_bucket *out, int32_t cap, int32_t *n) {
    return guarded([&] {
        if (!p || !n)
            return fail(ZDO_EINVAL, "zdo_plan_mx_buckets: plan or n is NULL");
        *n = nbuckets(p);
        if (out && cap >= *n)
            for (int32_t i = 0; i < *n; ++i) {
                const MxBucket &b = p->mx_buckets[size_t(i)];
                out[i] = {b.tile0 * kMxTileBlocks, mx_range_tiles(b.shard) * kMxTileBlocks};
            }
        return ZDO_OK;
    });
}

int64_t zdo_plan_norm_mxfp4_workspace_bytes(const zdo_plan *p) {
    if (!p)
        return -1;
    // one sum per wave, of at most one a tile
    return std::min(p->mx_tiles, kMxNormWaves) * int64_t(sizeof(double));
}

int quantize_grads_mxfp4(const zdo_plan *plan, int32_t bucket_begin, int32_t bucket_end, const uint16_t *grads,
                         int32_t coords, float *residual, uint8_t *codes, uint8_t *scales, void *stream) {
    return guarded([&] {
        const char *fn = "quantize_grads_mxfp4";
        if (int rc = check_plan(plan, fn))
            return rc;
        if (int rc = check_buckets(plan, bucket_begin, bucket_end, fn))
            return rc;
        if (int rc = check_storage(plan, coords, fn, "coords"))
            return rc;
        if (int rc = check_ptr(grads, fn, "grads"))
            return rc;
        Buffers bufs;
        bufs.reads(span_of(grads, extent(plan, coords), 2), "grads");
        if (residual) {
            if (int rc = check_ptr(residual, fn, "residual"))
                return rc;
            bufs.writes(span_of(residual, extent(plan, coords), 4), "residual");
        }
        if (int rc = take_storage(plan, codes, scales, coords, fn, bufs))
            return rc;
        if (int rc = bufs.check(fn))
            return rc;
        MxQuantArgs a{};
        a.walk = walk_of(plan, bucket_begin, bucket_end, true, coords == ZDO_WORLD);
        a.local = coords == ZDO_LOCAL;
        a.world = coords == ZDO_WORLD;
        a.grads = grads;
        a.residual = residual;
        a.codes = codes;
        a.scales = scales;
        return launch_result(launch_mx_quant(a, static_cast<hipStream_t>(stream)), fn);
    });
}

int reduce_scatter_local_mxfp4(const zdo_plan *plan, int32_t bucket_begin, int32_t bucket_end,
                               const uint8_t *const *codes, const uint8_t *const *scales, int32_t n, int32_t coords,
                               float scale, uint16_t *out, int32_t out_coords, void *stream) {
    return guarded([&] {
        const char *fn = "reduce_scatter_local_mxfp4";
        if (int rc = check_plan(plan, fn))
            return rc;
        if (int rc = check_buckets(plan, bucket_begin, bucket_end, fn))
            return rc;
        MxReduceArgs a{};
        Buffers bufs;
        if (int rc = take_inputs(plan, codes, scales, n, coords, fn, a.in, bufs))
            return rc;
        if (int rc = check_coords(out_coords, fn, "out_coords"))
            return rc;
        if (int rc = check_ptr(out, fn, "out"))
            return rc;
        bufs.writes(span_of(out, extent(plan, out_coords), 2), "out");
        if (int rc = bufs.check(fn))
            return rc;
        a.walk = walk_of(plan, bucket_begin, bucket_end, false, false);
        a.units = walk_of(plan, bucket_begin, bucket_end, true, false);
        a.out_local = out_coords == ZDO_LOCAL;
        a.scale = scale;
        a.out = out;
        return launch_result(launch_mx_reduce(a, plan->lds_per_cu, static_cast<hipStream_t>(stream)), fn);
    });
}

int grad_norm_sq_mxfp4(const zdo_plan *plan, const uint8_t *const *codes, const uint8_t *const *scales, int32_t n,
                       int32_t coords, float scale, void *workspace, double *norm_sq_out, void *stream) {
    return guarded([&] {
        const char *fn = "grad_norm_sq_mxfp4";
        if (int rc = check_plan(plan, fn))
            return rc;
        MxNormArgs a{};
        Buffers bufs;
        if (int rc = take_inputs(plan, codes, scales, n, coords, fn, a.in, bufs))
            return rc;
        if (int rc = check_ptr(workspace, fn, "workspace"))
            return rc;
        if (!norm_sq_out)
            return fail(ZDO_EINVAL, std::string(fn) + ": norm_sq_out is NULL");
        if (!aligned_to(norm_sq_out, 8))
            return fail(ZDO_EALIGN, std::string(fn) + ": norm_sq_out is not 8-byte aligned");
        bufs.writes(span_of(workspace, zdo_plan_norm_mxfp4_workspace_bytes(plan), 1), "workspace");
        bufs.writes(span_of(norm_sq_out, 1, 8), "norm_sq_out");
        if (int rc = bufs.check(fn))
            return rc;
        a.walk = walk_of(plan, 0, nbuckets(plan), false, false);
        a.units = walk_of(plan, 0, nbuckets(plan), true, false);
        a.scale = scale;
        a.partial = static_cast<double *>(workspace);
        return launch_result(launch_mx_norm(a, norm_sq_out, static_cast<hipStream_t>(stream)), fn);
    });
}

int sharded_adam_step_mxfp4(const zdo_plan *plan, int32_t bucket_begin, int32_t bucket_end,
                            const uint8_t *const *codes, const uint8_t *const *scales, int32_t n, int32_t coords,
                            float scale, float *master, float *exp_avg, float *exp_avg_sq, uint16_t *param_out,
                            int32_t param_coords, uint8_t *param_codes, uint8_t *param_scales,
                            int32_t param_mx_coords, const zdo_adam *hp, const float *grad_coeff,
                            float *main_grad_out, void *stream) {
    return guarded([&] {
        const char *fn = "sharded_adam_step_mxfp4";
        if (int rc = check_plan(plan, fn))
            return rc;
        if (int rc = check_buckets(plan, bucket_begin, bucket_end, fn))
            return rc;
        MxStepArgs a{};
        Buffers bufs;
        if (int rc = take_inputs(plan, codes, scales, n, coords, fn, a.in, bufs))
            return rc;
        if (int rc = check_adam(hp, fn))
            return rc;
        const int64_t L = plan->shard_numel;
        const struct {
            float *p;
            const char *name;
        } state[3] = {{master, "master"}, {exp_avg, "exp_avg"}, {exp_avg_sq, "exp_avg_sq"}};
        for (const auto &s : state) {
            if (int rc = check_ptr(s.p, fn, s.name))
                return rc;
            bufs.writes(span_of(s.p, L, 4), s.name);
        }
        if (param_out) {
            if (int rc = check_coords(param_coords, fn, "param_coords"))
                return rc;
            if (int rc = check_ptr(param_out, fn, "param_out"))
                return rc;
            bufs.writes(span_of(param_out, extent(plan, param_coords), 2), "param_out");
        }
        if ((param_codes != nullptr) != (param_scales != nullptr))
            return fail(ZDO_EINVAL, std::string(fn) + ": param_codes and param_scales go together");
        if (param_codes) {
            if (int rc = check_storage(plan, param_mx_coords, fn, "param_mx_coords"))
                return rc;
            if (int rc = take_storage(plan, param_codes, param_scales, param_mx_coords, fn, bufs))
                return rc;
        }
        if (main_grad_out) {
            if (int rc = check_ptr(main_grad_out, fn, "main_grad_out"))
                return rc;
            bufs.writes(span_of(main_grad_out, L, 4), "main_grad_out");
        }
        if (grad_coeff) {
            if (!aligned_to(grad_coeff, 4))
                return fail(ZDO_EALIGN, std::string(fn) + ": grad_coeff is not 4-byte aligned");
            bufs.reads(span_of(grad_coeff, 1, 4), "grad_coeff");
        }
        if (int rc = bufs.check(fn))
            return rc;
        a.walk = walk_of(plan, bucket_begin, bucket_end, false, false);
        a.param_local = param_coords == ZDO_LOCAL;
        a.mx_world = param_mx_coords == ZDO_WORLD;
        a.scale = scale;
        a.master = master;
        a.m = exp_avg;
        a.v = exp_avg_sq;
        a.param = param_out;
        a.codes = param_codes;
        a.scales = param_scales;
        a.main_grad = main_grad_out;
        a.coeff = grad_coeff;
        a.c = adam_const(*hp);
        return launch_result(launch_mx_step(a, plan->lds_per_cu, static_cast<hipStream_t>(stream)), fn);
    });
}

int writeback_params_mxfp4(const zdo_plan *plan, const float *master, uint8_t *codes, uint8_t *scales,
                           int32_t coords, void *stream) {
    return guarded([&] {
        const char *fn = "writeback_params_mxfp4";
        if (int rc = check_plan(plan, fn))
            return rc;
        if (int rc = check_storage(plan, coords, fn, "coords"))
            return rc;
        if (int rc = check_ptr(master, fn, "master"))
            return rc;
        Buffers bufs;
        bufs.reads(span_of(master, plan->shard_numel, 4), "master");
        if (int rc = take_storage(plan, codes, scales, coords, fn, bufs))
            return rc;
        if (int rc = bufs.check(fn))
            return rc;
        MxQuantArgs a{};
        a.walk = walk_of(plan, 0, nbuckets(plan), true, false);
        a.local = 1;
        a.world = coords == ZDO_WORLD;
        a.master = master;
        a.codes = codes;
        a.scales = scales;
        return launch_result(launch_mx_quant(a, static_cast<hipStream_t>(stream)), fn);
    });
}

int all_gather_params_mxfp4(const zdo_plan *plan, const uint8_t *const *codes, const uint8_t *const *scales,
                            int32_t n, int32_t coords, uint16_t *out, void *stream) {
    return guarded([&] {
        const char *fn = "all_gather_params_mxfp4";
        if (int rc = check_plan(plan, fn))
            return rc;
        if (n != plan->dp_size)
            return fail(ZDO_EINVAL, std::string(fn) + ": n must equal the DP size " + std::to_string(plan->dp_size));
        // the launch walks every rank's ranges
        if (int rc = check_storage(plan, ZDO_WORLD, fn, "coords"))
            return rc;
        MxGatherArgs a{};
        Buffers bufs;
        if (int rc = take_inputs(plan, codes, scales, n, coords, fn, a.in, bufs))
            return rc;
        if (int rc = check_ptr(out, fn, "out"))
            return rc;
        bufs.writes(span_of(out, plan->buffer_numel, 2), "out");
        if (int rc = bufs.check(fn))
            return rc;
        a.walk = walk_of(plan, 0, nbuckets(plan), true, true);
        a.out = out;
        return launch_result(launch_mx_gather(a, plan->lds_per_cu, static_cast<hipStream_t>(stream)), fn);
    });
}

}  // extern "C"
