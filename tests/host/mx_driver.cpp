// Host-only exercise of the MXFP4 calls' argument checks and of the plan's
// MXFP4 storage, for a build with AddressSanitizer and
// UndefinedBehaviorSanitizer on the host code (tests/test_mx_host.py). The
// current device is answered here and the plans are given a stand-in for
// their device table, so that the checks behind the plan's own are reached;
// the launchers are stand-ins that record what they were asked for. No device
// is used, and no pointer that is passed is ever followed.
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>
#include "kernels.h"
#include "mx.h"
#include "zdo_mx.h"

extern "C" hipError_t hipGetDevice(int *d) {
    *d = 0;
    return hipSuccess;
}

namespace zdo {
static long launches = 0;
static MxWalk last;
hipError_t launch_reduce(const ReduceArgs &, int, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_step(const StepArgs &, int, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_writeback(const WritebackArgs &, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_copy(void *, const void *, int64_t, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_norm(const NormArgs &, double *, int, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_clip(const double *, int32_t, float, float *, double *, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_gather(const GatherArgs &, int, hipStream_t) { return hipErrorNoDevice; }
hipError_t no_alloc_scratch(void **out) { *out = nullptr; return hipErrorNoDevice; }
hipError_t launch_probe(const ProbeArgs &, int, int, hipStream_t) { return hipErrorNoDevice; }
static hipError_t seen(const MxWalk &w) { ++launches; last = w; return hipSuccess; }
hipError_t launch_mx_reduce(const MxReduceArgs &a, int, hipStream_t) { return seen(a.walk); }
hipError_t launch_mx_norm(const MxNormArgs &a, double *, hipStream_t) { return seen(a.walk); }
hipError_t launch_mx_step(const MxStepArgs &a, int, hipStream_t) { return seen(a.walk); }
hipError_t launch_mx_quant(const MxQuantArgs &a, hipStream_t) { return seen(a.walk); }
hipError_t launch_mx_gather(const MxGatherArgs &a, int, hipStream_t) { return seen(a.walk); }
}  // namespace zdo

#define WANT(code, call)                                                                     \
    do {                                                                                     \
        const int got_ = (call);                                                             \
        if (got_ != (code)) {                                                                \
            std::printf("line %d: %s gave %d, not %d (%s)\n", __LINE__, #call, got_, (code), \
                        zdo_last_error());                                                   \
            return 1;                                                                        \
        }                                                                                    \
    } while (0)

// Addresses that overlap only where a test means them to.
template <typename T>
T *at(uint64_t slot, uint64_t byte = 0) {
    return reinterpret_cast<T *>((slot << 44) + byte + (1u << 20));
}

static zdo_plan *make(const std::vector<int64_t> &sizes, int64_t bucket, int32_t D, int32_t rank) {
    zdo_plan *p = nullptr;
    if (build_range_map(sizes.data(), int32_t(sizes.size()), bucket, D, rank, &p) != ZDO_OK)
        return nullptr;
    p->d_table = &zdo::launches;   // a stand-in: taken back before the plan is destroyed
    p->device = 0;
    return p;
}
static void drop(zdo_plan *p) {
    p->d_table = nullptr;
    zdo_plan_destroy(p);
}

static int storage_of_random_plans() {
    std::mt19937_64 rng(11);
    for (int trial = 0; trial < 2000; ++trial) {
        std::vector<int64_t> sizes(1 + rng() % 30);
        for (auto &x : sizes) x = 1 + int64_t(rng() % (rng() % 2 ? 40 : 6000));
        const int32_t D = 1 + int32_t(rng() % 64), rank = int32_t(rng() % D);
        zdo_plan *p = make(sizes, 1 + int64_t(rng() % 20000), D, rank);
        if (!p) return 1;
        int32_t nb = 0;
        WANT(ZDO_OK, zdo_plan_mx_buckets(p, nullptr, 0, &nb));
        std::vector<zdo_mx_bucket> mb(nb);
        WANT(ZDO_OK, zdo_plan_mx_buckets(p, mb.data(), nb, &nb));
        std::vector<zdo_bucket> b(nb);
        WANT(ZDO_OK, zdo_plan_buckets(p, b.data(), nb, &nb));
        int64_t sum = 0, units = 0;
        for (int32_t i = 0; i < nb; ++i) {
            const int64_t T = (b[i].shard_numel + 574) / 512;
            if (mb[i].block0 != sum || mb[i].blocks != 16 * T) return 2;
            // the tiles reach from the start's multiple of 64 past the range's end, for every rank
            for (int32_t r = 0; r < D; ++r) {
                const int64_t rs = b[i].offset + r * b[i].shard_numel;
                if (rs / 64 * 64 + 512 * T < rs + b[i].shard_numel) return 3;
            }
            if (p->mx_buckets[i].units != (T + 3) / 4 || p->mx_buckets[i].unit0 != units) return 4;
            sum += 16 * T;
            units += (T + 3) / 4;
        }
        if (zdo_plan_mx_blocks(p, ZDO_LOCAL) != sum || zdo_plan_mx_blocks(p, ZDO_WORLD) != sum * D) return 5;
        if (p->mx_units != units) return 6;
        // a call over a bucket range walks those buckets' units
        const int32_t b0 = int32_t(rng() % (nb + 1)), b1 = b0 + int32_t(rng() % (nb - b0 + 1));
        WANT(ZDO_OK, quantize_grads_mxfp4(p, b0, b1, at<uint16_t>(1), ZDO_WORLD, nullptr, at<uint8_t>(2), at<uint8_t>(3), nullptr));
        int64_t first = 0, count = 0;
        for (int32_t i = 0; i < b1; ++i) (i < b0 ? first : count) += D * int64_t(p->mx_buckets[i].units);
        if (zdo::last.first != first || zdo::last.count != count) return 7;
        drop(p);
    }
    return 0;
}

static int refusals() {
    zdo_plan *p = make({100, 28, 5000}, 64, 2, 1);
    if (!p) return 1;
    const int32_t nb = int32_t(p->buckets.size());
    const int64_t blocks = zdo_plan_mx_blocks(p, ZDO_WORLD);
    const uint8_t *codes[65], *scales[65];
    for (int j = 0; j < 65; ++j) {
        codes[j] = at<uint8_t>(100 + j);
        scales[j] = at<uint8_t>(200 + j);
    }
    zdo_adam hp{1e-3f, 0.9f, 0.999f, 1e-8f, 0.0f, 0, 1};
    uint16_t *g = at<uint16_t>(1), *out = at<uint16_t>(2);
    uint8_t *c = at<uint8_t>(3), *s = at<uint8_t>(4);
    float *P = at<float>(5), *M = at<float>(6), *V = at<float>(7), *R = at<float>(8), *K = at<float>(9);
    void *ws = at<char>(10);
    double *ns = at<double>(11);
    const long before = zdo::launches;

    // quantize
    WANT(ZDO_EINVAL, quantize_grads_mxfp4(nullptr, 0, nb, g, 0, R, c, s, nullptr));
    WANT(ZDO_EINVAL, quantize_grads_mxfp4(p, -1, nb, g, 0, R, c, s, nullptr));
    WANT(ZDO_EINVAL, quantize_grads_mxfp4(p, 0, nb + 1, g, 0, R, c, s, nullptr));
    WANT(ZDO_EINVAL, quantize_grads_mxfp4(p, 2, 1, g, 0, R, c, s, nullptr));
    WANT(ZDO_EINVAL, quantize_grads_mxfp4(p, 0, nb, g, 2, R, c, s, nullptr));
    WANT(ZDO_EINVAL, quantize_grads_mxfp4(p, 0, nb, nullptr, 0, R, c, s, nullptr));
    WANT(ZDO_EINVAL, quantize_grads_mxfp4(p, 0, nb, g, 0, R, nullptr, s, nullptr));
    WANT(ZDO_EINVAL, quantize_grads_mxfp4(p, 0, nb, g, 0, R, c, nullptr, nullptr));
    WANT(ZDO_EALIGN, quantize_grads_mxfp4(p, 0, nb, g + 1, 0, R, c, s, nullptr));
    WANT(ZDO_EALIGN, quantize_grads_mxfp4(p, 0, nb, g, 0, R + 1, c, s, nullptr));
    WANT(ZDO_EALIGN, quantize_grads_mxfp4(p, 0, nb, g, 0, R, c + 8, s, nullptr));
    WANT(ZDO_EALIGN, quantize_grads_mxfp4(p, 0, nb, g, 0, R, c, s + 1, nullptr));
    WANT(ZDO_EALIAS, quantize_grads_mxfp4(p, 0, nb, g, 0, R, reinterpret_cast<uint8_t *>(g) + 16, s, nullptr));
    WANT(ZDO_EALIAS, quantize_grads_mxfp4(p, 0, nb, g, 0, reinterpret_cast<float *>(g), c, s, nullptr));
    WANT(ZDO_EALIAS, quantize_grads_mxfp4(p, 0, nb, g, 0, R, c, c + 16 * blocks - 16, nullptr));
    // reduce
    WANT(ZDO_EINVAL, reduce_scatter_local_mxfp4(nullptr, 0, nb, codes, scales, 2, 0, 1.0f, out, 0, nullptr));
    WANT(ZDO_EINVAL, reduce_scatter_local_mxfp4(p, 0, nb + 1, codes, scales, 2, 0, 1.0f, out, 0, nullptr));
    WANT(ZDO_EINVAL, reduce_scatter_local_mxfp4(p, 0, nb, codes, scales, 0, 0, 1.0f, out, 0, nullptr));
    WANT(ZDO_EINVAL, reduce_scatter_local_mxfp4(p, 0, nb, codes, scales, 65, 0, 1.0f, out, 0, nullptr));
    WANT(ZDO_EINVAL, reduce_scatter_local_mxfp4(p, 0, nb, nullptr, scales, 2, 0, 1.0f, out, 0, nullptr));
    WANT(ZDO_EINVAL, reduce_scatter_local_mxfp4(p, 0, nb, codes, nullptr, 2, 0, 1.0f, out, 0, nullptr));
    WANT(ZDO_EINVAL, reduce_scatter_local_mxfp4(p, 0, nb, codes, scales, 2, 3, 1.0f, out, 0, nullptr));
    WANT(ZDO_EINVAL, reduce_scatter_local_mxfp4(p, 0, nb, codes, scales, 2, 0, 1.0f, out, 3, nullptr));
    WANT(ZDO_EINVAL, reduce_scatter_local_mxfp4(p, 0, nb, codes, scales, 2, 0, 1.0f, nullptr, 0, nullptr));
    WANT(ZDO_EALIGN, reduce_scatter_local_mxfp4(p, 0, nb, codes, scales, 2, 0, 1.0f, out + 4, 0, nullptr));
    const uint8_t *odd[2] = {codes[0], codes[1] + 4}, *none[2] = {codes[0], nullptr};
    WANT(ZDO_EALIGN, reduce_scatter_local_mxfp4(p, 0, nb, odd, scales, 2, 0, 1.0f, out, 0, nullptr));
    WANT(ZDO_EALIGN, reduce_scatter_local_mxfp4(p, 0, nb, codes, odd, 2, 0, 1.0f, out, 0, nullptr));
    WANT(ZDO_EINVAL, reduce_scatter_local_mxfp4(p, 0, nb, none, scales, 2, 0, 1.0f, out, 0, nullptr));
    WANT(ZDO_EINVAL, reduce_scatter_local_mxfp4(p, 0, nb, codes, none, 2, 0, 1.0f, out, 0, nullptr));
    WANT(ZDO_EALIAS, reduce_scatter_local_mxfp4(p, 0, nb, codes, scales, 2, 0, 1.0f,
                                                reinterpret_cast<uint16_t *>(const_cast<uint8_t *>(scales[1])), 0, nullptr));
    // norm
    WANT(ZDO_EINVAL, grad_norm_sq_mxfp4(nullptr, codes, scales, 2, 0, 1.0f, ws, ns, nullptr));
    WANT(ZDO_EINVAL, grad_norm_sq_mxfp4(p, codes, scales, 0, 0, 1.0f, ws, ns, nullptr));
    WANT(ZDO_EINVAL, grad_norm_sq_mxfp4(p, codes, scales, 2, 0, 1.0f, nullptr, ns, nullptr));
    WANT(ZDO_EINVAL, grad_norm_sq_mxfp4(p, codes, scales, 2, 0, 1.0f, ws, nullptr, nullptr));
    WANT(ZDO_EALIGN, grad_norm_sq_mxfp4(p, codes, scales, 2, 0, 1.0f, static_cast<char *>(ws) + 8, ns, nullptr));
    WANT(ZDO_EALIGN, grad_norm_sq_mxfp4(p, codes, scales, 2, 0, 1.0f, ws,
                                        reinterpret_cast<double *>(reinterpret_cast<char *>(ns) + 4), nullptr));
    WANT(ZDO_EALIAS, grad_norm_sq_mxfp4(p, codes, scales, 2, 0, 1.0f, ws, static_cast<double *>(ws) + 1, nullptr));
    WANT(ZDO_EALIAS, grad_norm_sq_mxfp4(p, codes, scales, 2, 0, 1.0f, const_cast<uint8_t *>(codes[1]), ns, nullptr));
    // step
#define STEP(n, pm, po, pc, cc, cs, cx, h, k, mg) \
    sharded_adam_step_mxfp4(p, 0, nb, codes, scales, n, 0, 1.0f, pm, M, V, po, pc, cc, cs, cx, h, k, mg, nullptr)
    WANT(ZDO_EINVAL, sharded_adam_step_mxfp4(nullptr, 0, nb, codes, scales, 2, 0, 1.0f, P, M, V, out, 0, c, s, 1, &hp, K, R, nullptr));
    WANT(ZDO_EINVAL, sharded_adam_step_mxfp4(p, 1, 0, codes, scales, 2, 0, 1.0f, P, M, V, out, 0, c, s, 1, &hp, K, R, nullptr));
    WANT(ZDO_EINVAL, STEP(0, P, out, 0, c, s, 1, &hp, K, R));
    WANT(ZDO_EINVAL, STEP(2, nullptr, out, 0, c, s, 1, &hp, K, R));
    WANT(ZDO_EINVAL, STEP(2, P, out, 5, c, s, 1, &hp, K, R));
    WANT(ZDO_EINVAL, STEP(2, P, out, 0, c, nullptr, 1, &hp, K, R));
    WANT(ZDO_EINVAL, STEP(2, P, out, 0, nullptr, s, 1, &hp, K, R));
    WANT(ZDO_EINVAL, STEP(2, P, out, 0, c, s, 2, &hp, K, R));
    WANT(ZDO_EINVAL, STEP(2, P, out, 0, c, s, 1, nullptr, K, R));
    zdo_adam bad = hp;
    bad.step = 0;
    WANT(ZDO_EINVAL, STEP(2, P, out, 0, c, s, 1, &bad, K, R));
    bad = hp;
    bad.beta2 = 1.0f;
    WANT(ZDO_EINVAL, STEP(2, P, out, 0, c, s, 1, &bad, K, R));
    bad = hp;
    bad.reserved = 1;
    WANT(ZDO_EINVAL, STEP(2, P, out, 0, c, s, 1, &bad, K, R));
    WANT(ZDO_EALIGN, STEP(2, P + 1, out, 0, c, s, 1, &hp, K, R));
    WANT(ZDO_EALIGN, STEP(2, P, out + 1, 0, c, s, 1, &hp, K, R));
    WANT(ZDO_EALIGN, STEP(2, P, out, 0, c + 1, s, 1, &hp, K, R));
    WANT(ZDO_EALIGN, STEP(2, P, out, 0, c, s, 1, &hp, reinterpret_cast<float *>(reinterpret_cast<char *>(K) + 2), R));
    WANT(ZDO_EALIGN, STEP(2, P, out, 0, c, s, 1, &hp, K, R + 2));
    WANT(ZDO_EALIAS, STEP(2, M, out, 0, c, s, 1, &hp, K, R));
    WANT(ZDO_EALIAS, STEP(2, P, reinterpret_cast<uint16_t *>(V), 0, c, s, 1, &hp, K, R));
    WANT(ZDO_EALIAS, STEP(2, P, out, 0, const_cast<uint8_t *>(codes[0]), s, 1, &hp, K, R));
    WANT(ZDO_EALIAS, STEP(2, P, out, 0, c, c + 16, 1, &hp, K, R));
    WANT(ZDO_EALIAS, STEP(2, P, out, 0, c, s, 1, &hp, M + 1, R));
    WANT(ZDO_EALIAS, STEP(2, P, out, 0, c, s, 1, &hp, K, P));
    // write-back and gather
    WANT(ZDO_EINVAL, writeback_params_mxfp4(nullptr, P, c, s, 1, nullptr));
    WANT(ZDO_EINVAL, writeback_params_mxfp4(p, P, c, s, 4, nullptr));
    WANT(ZDO_EINVAL, writeback_params_mxfp4(p, nullptr, c, s, 1, nullptr));
    WANT(ZDO_EINVAL, writeback_params_mxfp4(p, P, c, nullptr, 1, nullptr));
    WANT(ZDO_EALIGN, writeback_params_mxfp4(p, P, c, s + 4, 1, nullptr));
    WANT(ZDO_EALIAS, writeback_params_mxfp4(p, P, reinterpret_cast<uint8_t *>(P), s, 1, nullptr));
    WANT(ZDO_EINVAL, all_gather_params_mxfp4(nullptr, codes, scales, 2, 1, out, nullptr));
    WANT(ZDO_EINVAL, all_gather_params_mxfp4(p, codes, scales, 3, 1, out, nullptr));
    WANT(ZDO_EINVAL, all_gather_params_mxfp4(p, codes, scales, 2, 7, out, nullptr));
    WANT(ZDO_EINVAL, all_gather_params_mxfp4(p, none, scales, 2, 1, out, nullptr));
    WANT(ZDO_EINVAL, all_gather_params_mxfp4(p, codes, scales, 2, 1, nullptr, nullptr));
    WANT(ZDO_EALIAS, all_gather_params_mxfp4(p, codes, scales, 2, 1,
                                             reinterpret_cast<uint16_t *>(const_cast<uint8_t *>(codes[1])), nullptr));
    if (zdo::launches != before) return 2;   // nothing was launched by a refused call

    // and the calls that are right
    WANT(ZDO_OK, quantize_grads_mxfp4(p, 0, nb, g, ZDO_WORLD, R, c, s, nullptr));
    WANT(ZDO_OK, reduce_scatter_local_mxfp4(p, 0, 0, codes, scales, 64, ZDO_LOCAL, 1.0f, out, ZDO_WORLD, nullptr));
    if (zdo::last.count != 0) return 3;
    WANT(ZDO_OK, grad_norm_sq_mxfp4(p, codes, scales, 1, ZDO_WORLD, 1.0f, ws, ns, nullptr));
    WANT(ZDO_OK, STEP(64, P, out, 0, c, s, 1, &hp, K, R));
    WANT(ZDO_OK, STEP(2, P, nullptr, 9, nullptr, nullptr, 9, &hp, nullptr, nullptr));
    WANT(ZDO_OK, writeback_params_mxfp4(p, P, c, s, ZDO_WORLD, nullptr));
    const uint8_t *same[2] = {codes[0], codes[0]}, *same_s[2] = {scales[0], scales[0]};
    WANT(ZDO_OK, all_gather_params_mxfp4(p, same, same_s, 2, ZDO_WORLD, out, nullptr));
    if (zdo::launches != before + 7) return 4;
    drop(p);

    // a plan on another device, one without a table, and one too large to number
    p = make({64}, 64, 2, 0);
    p->device = 1;
    WANT(ZDO_EINVAL, quantize_grads_mxfp4(p, 0, 1, g, 0, R, c, s, nullptr));
    p->device = 0;
    drop(p);
    p = make({64}, 64, 2, 0);
    p->d_table = nullptr;
    WANT(ZDO_EHIP, writeback_params_mxfp4(p, P, c, s, 1, nullptr));
    WANT(ZDO_EHIP, all_gather_params_mxfp4(p, codes, scales, 2, 1, out, nullptr));
    zdo_plan_destroy(p);
    p = make({int64_t(1) << 40}, 64, 4, 0);   // 2^31 tiles in WORLD storage, 2^29 in LOCAL
    WANT(ZDO_EINVAL, quantize_grads_mxfp4(p, 0, 1, g, ZDO_WORLD, nullptr, c, s, nullptr));
    WANT(ZDO_EINVAL, all_gather_params_mxfp4(p, codes, scales, 4, ZDO_LOCAL, out, nullptr));
    WANT(ZDO_OK, quantize_grads_mxfp4(p, 0, 1, g, ZDO_LOCAL, nullptr, c, s, nullptr));
    drop(p);
    p = make({int64_t(1) << 55, int64_t(1) << 54}, 64, 1, 0);
    if (zdo_plan_mx_blocks(p, ZDO_LOCAL) <= 0) return 5;
    WANT(ZDO_EINVAL, quantize_grads_mxfp4(p, 0, 1, g, ZDO_LOCAL, nullptr, c, s, nullptr));
    drop(p);
    if (zdo_plan_mx_blocks(nullptr, 0) != -1 || zdo_plan_norm_mxfp4_workspace_bytes(nullptr) != -1) return 6;
    WANT(ZDO_EINVAL, zdo_plan_mx_buckets(nullptr, nullptr, 0, nullptr));
    return 0;
}

int main() {
    if (int rc = storage_of_random_plans()) {
        std::printf("storage: %d\n", rc);
        return 1;
    }
    if (int rc = refusals()) {
        std::printf("refusals: %d\n", rc);
        return 1;
    }
    std::printf("ok: storage of 2000 plans, refusals of the MXFP4 calls\n");
    return 0;
}
