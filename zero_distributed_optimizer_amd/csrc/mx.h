// Launch arguments and launchers of the MXFP4 kernels (mx_kernels.hip).
#pragma once

#include "kernels.h"

namespace zdo {

// A walk over MXFP4 storage: tiles or units (see MxBucket) of the rank's
// ranges (LOCAL order) or of every rank's (WORLD order), [first, first +
// count).
struct MxWalk {
    const MxBucket *buckets;
    const uint32_t *group;  // the bucket of every kTileGroup-th LOCAL tile or unit, then the last bucket
    int32_t dp, rank;
    int32_t by_xcd;         // 8 consecutive tiles to an XCD (the launchers set it)
    int64_t first, count;
};

// MXFP4 storages that a kernel reads.
struct MxInputs {
    const uint8_t *codes[ZDO_MAX_REPLICAS];
    const uint8_t *scales[ZDO_MAX_REPLICAS];
    int32_t n;
    int32_t world;  // storage order: WORLD (1) or LOCAL (0)
};

struct MxReduceArgs {
    MxWalk walk, units;  // the same buckets' LOCAL tiles and units
    MxInputs in;
    int32_t out_local;
    float scale;
    uint16_t *out;
};

// Most waves of a squared norm, each of which leaves one sum.
constexpr int64_t kMxNormWaves = 16384;

struct MxNormArgs {
    MxWalk walk, units;  // LOCAL tiles, and units
    MxInputs in;
    float scale;
    double *partial;  // one per wave
};

struct MxStepArgs {
    MxWalk walk;  // LOCAL tiles
    MxInputs in;
    int32_t param_local, mx_world;
    float scale;
    float *master, *m, *v;
    uint16_t *param;        // may be NULL
    uint8_t *codes, *scales;  // may be NULL (both)
    float *main_grad;       // may be NULL
    const float *coeff;     // may be NULL
    AdamConst c;
};

// bf16 gradients or the fp32 master to MXFP4.
struct MxQuantArgs {
    MxWalk walk;  // units, LOCAL or WORLD
    int32_t local;   // source indexed by LOCAL position
    int32_t world;   // storage order
    const uint16_t *grads;  // or NULL:
    const float *master;
    float *residual;  // with grads; may be NULL
    uint8_t *codes, *scales;
};

struct MxGatherArgs {
    MxWalk walk;  // WORLD units
    MxInputs in;
    uint16_t *out;
};

hipError_t launch_mx_reduce(const MxReduceArgs &a, int lds_per_cu, hipStream_t stream);
hipError_t launch_mx_norm(const MxNormArgs &a, double *norm_sq, hipStream_t stream);
hipError_t launch_mx_step(const MxStepArgs &a, int lds_per_cu, hipStream_t stream);
hipError_t launch_mx_quant(const MxQuantArgs &a, hipStream_t stream);
hipError_t launch_mx_gather(const MxGatherArgs &a, int lds_per_cu, hipStream_t stream);

}  // namespace zdo
