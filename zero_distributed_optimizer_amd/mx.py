"""The MXFP4 calls of include/zdo_mx.h: gradient contributions and updated
parameters in 4 bits. As in the package's other calls, the functions only
marshal arguments; every step of the work runs in the library's kernels.

A storage is a pair (codes, scales) of uint8 device tensors, 16 bytes and 1
byte for each of plan.mx_blocks(coords) blocks; mx_empty makes one.

    mx, mine = mx_empty(plan, WORLD), mx_empty(plan, LOCAL)
    writeback_params_mxfp4(plan, master, mine, LOCAL)   # once: a skipped step leaves it as it is
    # every step:
    quantize_grads_mxfp4(plan, grads, WORLD, mx, residual=residual)
    # the ranks exchange their storages' ranges; then the owner of a range:
    sharded_adam_step_mxfp4(plan, contributions, LOCAL, scale, master, exp_avg, exp_avg_sq,
                            param_mx=mine, lr=..., beta1=..., ..., step=t)
    all_gather_params_mxfp4(plan, storages_of_all_ranks, LOCAL, param_buffer)
"""

from __future__ import annotations

import ctypes

import numpy as np

from . import (EINVAL, LOCAL, WORLD, Adam, Plan, ZdoError, _bucket_list, _check, _dev_ptr, _stream, _torch,
               adam_hparams, require_library)

MX_BUCKET_DTYPE = np.dtype([("block0", "<i8"), ("blocks", "<i8")])
BLOCK = 32                # elements that share a scale
CODE_BYTES = BLOCK // 2   # a block's codes
NO_BUCKETS = ((0, 0),)    # an empty range, for the library's checks

# Every symbol include/zdo_mx.h declares.
MX_EXPORTS = ("zdo_plan_mx_blocks", "zdo_plan_mx_buckets", "zdo_plan_norm_mxfp4_workspace_bytes",
              "quantize_grads_mxfp4", "reduce_scatter_local_mxfp4", "grad_norm_sq_mxfp4",
              "sharded_adam_step_mxfp4", "writeback_params_mxfp4", "all_gather_params_mxfp4")


def declare(L: ctypes.CDLL) -> None:
    """Argument types of the library's MXFP4 calls."""
    i32, f32, vp = ctypes.c_int32, ctypes.c_float, ctypes.c_void_p
    L.zdo_plan_mx_blocks.argtypes = [vp, i32]
    L.zdo_plan_mx_blocks.restype = ctypes.c_int64
    L.zdo_plan_norm_mxfp4_workspace_bytes.argtypes = [vp]
    L.zdo_plan_norm_mxfp4_workspace_bytes.restype = ctypes.c_int64
    L.zdo_plan_mx_buckets.argtypes = [vp, vp, i32, ctypes.POINTER(i32)]
    L.quantize_grads_mxfp4.argtypes = [vp, i32, i32, vp, i32, vp, vp, vp, vp]
    L.reduce_scatter_local_mxfp4.argtypes = [vp, i32, i32, vp, vp, i32, i32, f32, vp, i32, vp]
    L.grad_norm_sq_mxfp4.argtypes = [vp, vp, vp, i32, i32, f32, vp, vp, vp]
    L.sharded_adam_step_mxfp4.argtypes = [vp, i32, i32, vp, vp, i32, i32, f32, vp, vp, vp, vp, i32, vp, vp, i32,
                                          ctypes.POINTER(Adam), vp, vp, vp]
    L.writeback_params_mxfp4.argtypes = [vp, vp, vp, vp, i32, vp]
    L.all_gather_params_mxfp4.argtypes = [vp, vp, vp, i32, i32, vp, vp]
    for f in ("zdo_plan_mx_buckets", "quantize_grads_mxfp4", "reduce_scatter_local_mxfp4", "grad_norm_sq_mxfp4",
              "sharded_adam_step_mxfp4", "writeback_params_mxfp4", "all_gather_params_mxfp4"):
        getattr(L, f).restype = ctypes.c_int


def mx_empty(plan: Plan, coords: int, device=None):
    """A zeroed storage for the plan: (codes [blocks, 16], scales [blocks])."""
    torch, n = _torch(), plan.mx_blocks(coords)
    device = "cuda" if device is None else device
    return (torch.zeros((n, CODE_BYTES), dtype=torch.uint8, device=device),
            torch.zeros(n, dtype=torch.uint8, device=device))


class MxBuffers:
    """Storages (the D contributions, or the ranks' parameters) checked and
    marshalled once, for calls repeated on the same tensors: pass it wherever
    a call takes a list of storages. It holds references to the tensors,
    which must keep their memory (no resize) while it is in use."""

    def __init__(self, storages, what: str = "storages"):
        self.storages = tuple((c, s) for c, s in storages)
        n = len(self.storages)
        self.codes, self.scales = (ctypes.c_void_p * n)(), (ctypes.c_void_p * n)()
        self.blocks, self.device = (1 << 62 if n else 0), None
        before = (None, None)
        for j, (c, s) in enumerate(self.storages):
            if c is before[0] and s is before[1]:   # the same storage again, as the gather may be given it
                self.codes[j], self.scales[j] = self.codes[j - 1], self.scales[j - 1]
                continue
            before = (c, s)
            self.codes[j] = _dev_ptr(c, f"{what}[{j}] codes", "bytes", None)
            self.scales[j] = _dev_ptr(s, f"{what}[{j}] scales", "bytes", None)
            self.blocks = min(self.blocks, c.numel() // CODE_BYTES, s.numel())
            for t in (c, s):
                if self.device is not None and t.get_device() != self.device:
                    raise ValueError(f"{what}[{j}]: on {t.device}, others on device {self.device}")
                self.device = t.get_device()

    def __len__(self) -> int:
        return len(self.storages)

    def __iter__(self):
        return iter(self.storages)

    def __getitem__(self, j):
        return self.storages[j]


class _Call:
    """Checks and marshals one call's tensors, which all live on the current
    device (the plan's, as the library checks)."""

    __slots__ = ("plan", "device")

    def __init__(self, plan: Plan):
        self.plan, self.device = plan, None

    def on(self, device: int, what: str) -> None:
        if self.device is None:
            self.device = _torch().cuda.current_device()
        if device != self.device:
            raise ValueError(f"{what}: on device {device}, but device {self.device} is current")

    def ptr(self, t, what: str, kind: str, numel: int) -> int:
        p = _dev_ptr(t, what, kind, numel)
        if t.get_device() != self.device:
            self.on(t.get_device(), what)
        return p

    def opt(self, t, what: str, kind: str, numel: int):
        return None if t is None else self.ptr(t, what, kind, numel)

    def inputs(self, storages, what: str, coords: int) -> MxBuffers:
        mx = storages if isinstance(storages, MxBuffers) else MxBuffers(storages, what)
        if len(mx.storages):
            need = self.plan.mx_blocks(coords)
            if mx.blocks < need:
                raise ValueError(f"{what}: needs at least {need} blocks per storage, has {mx.blocks}")
            self.on(mx.device, what)
        return mx

    def storage(self, mx, what: str, coords: int):
        if mx is None or len(mx) != 2:
            raise TypeError(f"{what}: expected a storage, a pair (codes, scales)")
        n = self.plan.mx_blocks(coords)
        return (self.ptr(mx[0], f"{what} codes", "bytes", CODE_BYTES * n),
                self.ptr(mx[1], f"{what} scales", "bytes", n))

    def stream(self, stream) -> int:
        if stream is not None:
            self.on(stream.device.index, "stream")
        return _stream(stream, self.device)

    def buckets(self, buckets):
        """The bucket ranges to launch: all buckets, one (begin, end), or a list
        of disjoint pairs, sorted and merged where they touch."""
        if buckets is None:
            return ((0, self.plan.num_buckets),)
        if _bucket_list(buckets) is None:
            return ((int(buckets[0]), int(buckets[1])),)
        runs = []
        for b, e in sorted((int(b), int(e)) for b, e in buckets):
            if not 0 <= b <= e <= self.plan.num_buckets:
                raise ZdoError(EINVAL, f"bucket range ({b}, {e}): need 0 <= begin <= end <= {self.plan.num_buckets}")
            if b == e:
                continue
            if runs and b < runs[-1][1]:
                raise ZdoError(EINVAL, f"bucket ranges {runs[-1]} and ({b}, {e}) overlap")
            if runs and b == runs[-1][1]:
                runs[-1] = (runs[-1][0], e)
            else:
                runs.append((b, e))
        return runs


def quantize_grads_mxfp4(plan: Plan, grads, coords: int, out, residual=None, buckets=None, stream=None) -> None:
    """The bf16 gradient buffer to MXFP4, into the storage `out` (both in
    `coords`). residual: a float32 tensor as long as grads, added first and
    left holding what the 4 bits did not carry. buckets=(begin, end), or a
    list of disjoint such pairs: those buckets only, one launch for each run
    of them that touch."""
    call, n = _Call(plan), plan.extent(coords)
    g = call.ptr(grads, "grads", "bf16", n)
    r = call.opt(residual, "residual", "f32", n)
    c, s = call.storage(out, "out", coords)
    st, L = call.stream(stream), require_library()
    for b0, b1 in call.buckets(buckets) or NO_BUCKETS:
        _check(L.quantize_grads_mxfp4(plan.handle, b0, b1, g, coords, r, c, s, st))


def reduce_scatter_local_mxfp4(plan: Plan, contributions, coords: int, scale: float, out, out_coords: int,
                               stream=None, buckets=None) -> None:
    """reduce_scatter_local of contributions in MXFP4 (storages in `coords`):
    bf16(scale * sum) over the rank's ranges. One contribution and scale 1
    give its values. buckets: as quantize_grads_mxfp4."""
    call = _Call(plan)
    mx = call.inputs(contributions, "contributions", coords)
    o = call.ptr(out, "out", "bf16", plan.extent(out_coords))
    st, L = call.stream(stream), require_library()
    for b0, b1 in call.buckets(buckets) or NO_BUCKETS:
        _check(L.reduce_scatter_local_mxfp4(plan.handle, b0, b1, mx.codes, mx.scales, len(mx), coords, scale, o,
                                            out_coords, st))


def grad_norm_sq_mxfp4(plan: Plan, contributions, coords: int, scale: float, workspace, norm_sq_out,
                       stream=None) -> None:
    """The rank's squared norm of the gradient that sharded_adam_step_mxfp4
    steps with, into norm_sq_out (one-element float64 device tensor);
    workspace: uint8 device tensor of plan.norm_mxfp4_workspace_bytes."""
    call = _Call(plan)
    mx = call.inputs(contributions, "contributions", coords)
    ws = call.ptr(workspace, "workspace", "bytes", plan.norm_mxfp4_workspace_bytes)
    ns = call.ptr(norm_sq_out, "norm_sq_out", "f64", 1)
    _check(require_library().grad_norm_sq_mxfp4(plan.handle, mx.codes, mx.scales, len(mx), coords, scale, ws, ns,
                                                call.stream(stream)))


def sharded_adam_step_mxfp4(plan: Plan, contributions, coords: int, scale: float, master, exp_avg, exp_avg_sq,
                            param_out=None, param_coords: int = WORLD, *, param_mx=None,
                            param_mx_coords: int = LOCAL, lr: float, beta1: float, beta2: float, eps: float,
                            weight_decay: float, step: int, grad_coeff=None, main_grad_out=None, stream=None,
                            buckets=None) -> None:
    """sharded_adam_step on contributions in MXFP4 (storages in `coords`). The
    updated parameters go to param_out (bf16) and, rounded to MXFP4, to the
    storage param_mx. grad_coeff: a one-element float32 device tensor that
    multiplies the main grad (NaN skips the step, and leaves param_out and
    param_mx as they were: writeback_params_mxfp4 gives param_mx its first
    contents). buckets: as quantize_grads_mxfp4."""
    call, L = _Call(plan), plan.shard_numel
    mx = call.inputs(contributions, "contributions", coords)
    m = call.ptr(master, "master", "f32", L)
    a = call.ptr(exp_avg, "exp_avg", "f32", L)
    v = call.ptr(exp_avg_sq, "exp_avg_sq", "f32", L)
    p = call.opt(param_out, "param_out", "bf16", plan.extent(param_coords))
    pc, ps = (None, None) if param_mx is None else call.storage(param_mx, "param_mx", param_mx_coords)
    gc = call.opt(grad_coeff, "grad_coeff", "f32", 1)
    mg = call.opt(main_grad_out, "main_grad_out", "f32", L)
    hp = adam_hparams(lr, beta1, beta2, eps, weight_decay, step)
    st, L = call.stream(stream), require_library()
    for b0, b1 in call.buckets(buckets) or NO_BUCKETS:
        _check(L.sharded_adam_step_mxfp4(plan.handle, b0, b1, mx.codes, mx.scales, len(mx), coords, scale, m, a, v, p,
                                         param_coords, pc, ps, param_mx_coords, ctypes.byref(hp), gc, mg, st))


def writeback_params_mxfp4(plan: Plan, master, out, coords: int, stream=None) -> None:
    """The rank's float32 master shard rounded to MXFP4, into its ranges of
    the storage `out` (in `coords`)."""
    call = _Call(plan)
    m = call.ptr(master, "master", "f32", plan.shard_numel)
    c, s = call.storage(out, "out", coords)
    _check(require_library().writeback_params_mxfp4(plan.handle, m, c, s, coords, call.stream(stream)))


def all_gather_params_mxfp4(plan: Plan, params, coords: int, out, stream=None) -> None:
    """Rank j's range of every padded bucket from the storage params[j] (D
    storages in `coords`), as bf16 into out (N elements)."""
    call = _Call(plan)
    mx = call.inputs(params, "params", coords)
    o = call.ptr(out, "out", "bf16", plan.buffer_numel)
    _check(require_library().all_gather_params_mxfp4(plan.handle, mx.codes, mx.scales, len(mx), coords, o,
                                                     call.stream(stream)))
