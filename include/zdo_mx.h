/*
 * zdo_mx.h — the sharded step's traffic between ranks in 4 bits: gradient
 * contributions and updated parameters in the microscaled format MXFP4, on
 * AMD Instinct MI355X (gfx950). The calls stand beside those of zdo.h and
 * share its plan, coordinates, streams, error codes and conventions (its
 * first comment); every call here only enqueues work, allocates nothing and
 * may be captured into a HIP graph.
 *
 * Format (OCP Microscaling Formats v1.0, MXFP4): a block of 32 elements
 * shares one scale byte e (E8M0: 2^(e - 127), 255 = NaN); an element is a
 * 4-bit code, its top bit the sign, the others an E2M1 magnitude
 * (0, 0.5, 1, 1.5, 2, 3, 4, 6). A slot's value is magnitude * 2^(e - 127) in
 * fp32. Two codes a byte, the even slot in the low half: 16 bytes a block.
 *
 * Storage follows the flat buffer's ranges. Let S = padded_numel / D be the
 * length of every rank's range of a bucket. A range is stored as
 * T = floor((S + 574) / 512) tiles of 16 blocks: slot i of the range's
 * storage is WORLD element o + i, o the range's first WORLD element rounded
 * down to a multiple of 64. LOCAL storage holds the rank's ranges bucket
 * after bucket (16 * sum T blocks, the same for every rank); WORLD storage
 * holds, bucket after bucket, the D ranges in rank order. So a bucket's
 * storage splits into D equal parts, one a rank, as the bucket does, and no
 * block is shared by two ranges. Slots that are no parameter element of
 * their range (before it, its padding, behind it) are written as zero
 * (code 0), and blocks without any as scale 0; the calls that read storage
 * use the slots of the range, its padding included, and no others.
 *
 * A storage is two device arrays, both 16-byte aligned: codes (16 bytes a
 * block) and scales (1 byte a block), for zdo_plan_mx_blocks(plan, coords)
 * blocks. Plans of more than 2^30 tiles in a storage that a call uses are
 * refused with ZDO_EINVAL; all_gather_params_mxfp4, which walks every rank's
 * ranges, refuses those of more than 2^30 in WORLD storage (D times the LOCAL
 * ones), whatever its coordinates.
 *
 * Rounding to MXFP4, per block: A = max |x| over its slots;
 * e = max(0, X - 2), X the biased fp32 exponent of A (0 for subnormals), so
 * that A / 2^(e - 127) < 8; a code is the E2M1 nearest to x / 2^(e - 127),
 * ties to the even code, magnitudes above 6 to 6, the sign kept. A block
 * with an Inf or a NaN gets scale 255 and codes 0: it reads as NaN.
 */
#ifndef ZDO_MX_H
#define ZDO_MX_H

#include <stdint.h>

#include "zdo.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Where a bucket lies in storage: blocks [block0, block0 + blocks) of LOCAL
 * storage, and in WORLD storage, for rank r's range, the `blocks` blocks from
 * D * block0 + r * blocks. */
typedef struct {
    int64_t block0, blocks;
} zdo_mx_bucket;

/* Blocks of the plan's storage in LOCAL or WORLD coordinates; -1 for a NULL
 * plan or other coordinates. */
int64_t zdo_plan_mx_blocks(const zdo_plan *plan, int32_t coords);

/* Two-call query as zdo_plan_buckets. */
int zdo_plan_mx_buckets(const zdo_plan *plan, zdo_mx_bucket *out, int32_t cap, int32_t *n);

/* Workspace bytes grad_norm_sq_mxfp4 needs: 8 per LOCAL tile, 128 KiB at
 * most. */
int64_t zdo_plan_norm_mxfp4_workspace_bytes(const zdo_plan *plan);

/* A gradient buffer to MXFP4, for the buckets [bucket_begin, bucket_end): the
 * contribution that a rank sends. grads: bf16, N elements (coords ZDO_WORLD:
 * every rank's range of those buckets is quantised) or L (ZDO_LOCAL: the
 * plan's rank's ranges). codes, scales: storage in the same coordinates; all
 * blocks of those buckets are written.
 * residual: NULL, or fp32 with as many elements as grads: x = grad +
 * residual (one fp32 addition) is quantised, and the residual becomes
 * x - value, the part that the 4 bits did not carry, to be sent with the
 * next step (exact in fp32: nothing is lost between them). A block whose x
 * holds an Inf or a NaN leaves its residual as it was. Only parameter
 * elements are read or rewritten. A contribution whose step is skipped is not
 * sent again: only its residual is carried over. Outputs must not overlap each
 * other or the grads. */
int quantize_grads_mxfp4(const zdo_plan *plan, int32_t bucket_begin, int32_t bucket_end, const uint16_t *grads,
                         int32_t coords, float *residual, uint8_t *codes, uint8_t *scales, void *stream);

/* reduce_scatter_local of contributions in MXFP4, for the buckets
 * [bucket_begin, bucket_end): per slot of the rank's ranges, padding
 * included, out = bf16(scale * (x_0 + x_1 + ... )), x_j the contributions'
 * values, added in fp32 in the order given. (The bf16 call rounds each
 * scaled term; here the contributions stay as they were sent, and the fp32
 * sum is scaled once.) codes, scales: host arrays of n (1..ZDO_MAX_REPLICAS)
 * device pointers, storage in `coords`. out: bf16, N (out_coords ZDO_WORLD)
 * or L (ZDO_LOCAL) elements; only the ranges are written; it must not
 * overlap the contributions. One contribution with scale 1 gives its
 * values. */
int reduce_scatter_local_mxfp4(const zdo_plan *plan, int32_t bucket_begin, int32_t bucket_end,
                               const uint8_t *const *codes, const uint8_t *const *scales, int32_t n, int32_t coords,
                               float scale, uint16_t *out, int32_t out_coords, void *stream);

/* The squared norm of the gradient that sharded_adam_step_mxfp4 steps with:
 * sum of g^2 over the rank's owned parameter elements, g = scale * (x_0 + x_1
 * + ...) in fp32 as above, squares (exact) and sums in fp64, in a fixed order
 * that depends on the plan and n only, so that equal inputs give equal bits:
 * each wave of the launch adds its tiles' squares into `workspace`, then the
 * waves' sums are added.
 * workspace: zdo_plan_norm_mxfp4_workspace_bytes(plan) bytes, 16-byte
 * aligned, this call's alone until it completes. norm_sq_out: device double.
 * A rank that owns nothing gets 0. A block with scale 255 makes it NaN, and
 * clip_coefficient then asks for the step to be skipped. */
int grad_norm_sq_mxfp4(const zdo_plan *plan, const uint8_t *const *codes, const uint8_t *const *scales, int32_t n,
                       int32_t coords, float scale, void *workspace, double *norm_sq_out, void *stream);

/* sharded_adam_step on contributions in MXFP4, for the buckets [bucket_begin,
 * bucket_end): main grad g = scale * (x_0 + x_1 + ...), in fp32 and not
 * rounded to bf16 in between; times *grad_coeff if grad_coeff (a device
 * float, as in sharded_adam_step_clipped: NaN changes nothing) is not NULL;
 * Adam on the owned elements as zdo.h states it; the updated parameters to
 * any of
 *   param_out: bf16, N (param_coords ZDO_WORLD) or L (ZDO_LOCAL) elements,
 *   param_codes and param_scales (both or neither): the fp32 parameters
 *     rounded to MXFP4, storage in param_mx_coords, all blocks of the rank's
 *     ranges of those buckets written.
 * main_grad_out: NULL or fp32, L elements. The other arguments and rules as
 * sharded_adam_step; no output may overlap another or an input.
 * A skipped step leaves param_codes and param_scales as they were, and what
 * they hold is gathered all the same: a storage is given its first contents by
 * writeback_params_mxfp4, before any step (zeroed memory would be gathered as
 * parameters of zero if the first step is skipped). */
int sharded_adam_step_mxfp4(const zdo_plan *plan, int32_t bucket_begin, int32_t bucket_end,
                            const uint8_t *const *codes, const uint8_t *const *scales, int32_t n, int32_t coords,
                            float scale, float *master, float *exp_avg, float *exp_avg_sq, uint16_t *param_out,
                            int32_t param_coords, uint8_t *param_codes, uint8_t *param_scales,
                            int32_t param_mx_coords, const zdo_adam *hp, const float *grad_coeff,
                            float *main_grad_out, void *stream);

/* The rank's fp32 master shard rounded to MXFP4: codes, scales: storage in
 * `coords`; every block of the rank's ranges is written, no other. */
int writeback_params_mxfp4(const zdo_plan *plan, const float *master, uint8_t *codes, uint8_t *scales,
                           int32_t coords, void *stream);

/* all_gather_params of parameters in MXFP4: rank j's range of every padded
 * bucket, padding included, from codes[j] and scales[j] (n == D host
 * pointers each; storage in `coords`: ZDO_WORLD, each rank having written
 * its own ranges, or ZDO_LOCAL, rank j's own storage) as bf16 into out (N
 * elements), which must not overlap them. Their values are bf16 numbers, so
 * nothing is rounded (a value whose size passes the largest finite one,
 * which no call here writes, becomes Inf). The same storage may be given for
 * several ranks: D times one WORLD storage gives all its values. */
int all_gather_params_mxfp4(const zdo_plan *plan, const uint8_t *const *codes, const uint8_t *const *scales,
                            int32_t n, int32_t coords, uint16_t *out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ZDO_MX_H */
