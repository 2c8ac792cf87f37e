"""The calls of include/zdo_vocab.h: the embedding lookup and the softmax cross
entropy on the vocabulary matrix where it lies in the parameter buffer, and
their gradients into the contribution that the rank sends. As in the package's
other calls, the functions only marshal arguments; every step of the work runs
in the library's kernels.

    ws = torch.empty(max(embedding_grad_workspace_bytes(n, dim),
                         linear_cross_entropy_workspace_bytes(n, vocab, dim)), dtype=torch.uint8, device="cuda")
    embedding_lookup(plan, 0, vocab, params, tokens, x)            # x: [n, dim]
    # ... the model's layers: hidden [n, dim] ...
    linear_cross_entropy(plan, head, vocab, params, hidden, targets, loss, lse, ws)
    linear_cross_entropy_grad(plan, head, vocab, params, hidden, targets, lse, grad_loss, grad_hidden, grads, ws)
    # ... the layers' backward pass: grad_x [n, dim] ...
    embedding_grad(plan, 0, vocab, tokens, grad_x, grads, ws, accumulate=tied)

With a tied matrix (head == 0) the last call adds to what the loss's gradient
wrote. Activations are bf16 or float32 tensors [n, dim], rows consecutive in
memory and at any distance from each other; tokens and targets int64 [n], a
number outside [0, vocab) naming no row.
"""

from __future__ import annotations

import ctypes

from . import Plan, _check, _torch, require_library
from .mx import _Call

BF16, F32 = 0, 1

# Every symbol include/zdo_vocab.h declares.
VOCAB_EXPORTS = ("embedding_lookup", "zdo_embedding_grad_workspace_bytes", "embedding_grad",
                 "zdo_linear_cross_entropy_workspace_bytes", "linear_cross_entropy", "linear_cross_entropy_grad")


def declare(L: ctypes.CDLL) -> None:
    """Argument types of the library's vocabulary calls."""
    i32, i64, f32, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
    matrix = [vp, i32, i64, i64]
    L.embedding_lookup.argtypes = [*matrix, vp, vp, i64, f32, vp, i32, i64, vp]
    L.embedding_grad.argtypes = [*matrix, vp, i64, vp, i32, i64, f32, i32, vp, vp, vp]
    L.linear_cross_entropy.argtypes = [*matrix, vp, vp, i64, vp, i64, vp, vp, vp, vp]
    L.linear_cross_entropy_grad.argtypes = [*matrix, vp, vp, i64, vp, i64, vp, vp, vp, i32, i64, i32, vp, vp, vp]
    for f in ("embedding_lookup", "embedding_grad", "linear_cross_entropy", "linear_cross_entropy_grad"):
        getattr(L, f).restype = ctypes.c_int
    L.zdo_embedding_grad_workspace_bytes.argtypes = [i64, i64]
    L.zdo_linear_cross_entropy_workspace_bytes.argtypes = [i64, i64, i64]
    for f in ("zdo_embedding_grad_workspace_bytes", "zdo_linear_cross_entropy_workspace_bytes"):
        getattr(L, f).restype = i64


def _bytes(n: int, what: str) -> int:
    if n < 0:
        raise ValueError(f"{what}: sizes out of range")
    return n


def embedding_grad_workspace_bytes(n: int, dim: int) -> int:
    """Bytes of the workspace that embedding_grad needs for n tokens."""
    return _bytes(int(require_library().zdo_embedding_grad_workspace_bytes(n, dim)), "embedding_grad_workspace_bytes")


def linear_cross_entropy_workspace_bytes(n: int, vocab: int, dim: int) -> int:
    """Bytes of the workspace that linear_cross_entropy and its gradient need
    for n tokens."""
    return _bytes(int(require_library().zdo_linear_cross_entropy_workspace_bytes(n, vocab, dim)),
                  "linear_cross_entropy_workspace_bytes")


class _VocabCall(_Call):
    """One call's checks; its activations share n and dim, which `rows` of the
    first of them sets."""

    __slots__ = ("n", "dim")

    def __init__(self, plan: Plan):
        super().__init__(plan)
        self.n = self.dim = None

    def rows(self, t, what: str, types=None):
        """A [n, dim] tensor of activations: (pointer, type, stride)."""
        torch = _torch()
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what}: expected a torch tensor")
        if not t.is_cuda:
            raise ValueError(f"{what}: must be a device (cuda) tensor")
        if t.dtype is torch.bfloat16:
            kind = BF16
        elif t.dtype is torch.float32 and types is None:
            kind = F32
        else:
            raise TypeError(f"{what}: dtype {t.dtype} is not bfloat16" + (" or float32" if types is None else ""))
        if t.dim() != 2:
            raise ValueError(f"{what}: expected 2 dimensions, has {t.dim()}")
        n, dim = t.shape
        if self.n is None:
            self.n, self.dim = n, dim
        elif (n, dim) != (self.n, self.dim):
            raise ValueError(f"{what}: shape {(n, dim)}, others {(self.n, self.dim)}")
        stride = t.stride(0)
        if dim > 1 and t.stride(1) != 1:
            raise ValueError(f"{what}: a row's elements must be consecutive")
        if n > 1 and stride < dim:
            raise ValueError(f"{what}: rows overlap (stride {stride}, {dim} elements)")
        if t.get_device() != self.device:
            self.on(t.get_device(), what)
        return t.data_ptr(), kind, stride

    def tokens(self, t, what: str, dtype: str):
        """One element a token: int64 or float32."""
        torch = _torch()
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what}: expected a torch tensor")
        if t.dtype is not getattr(torch, dtype):
            raise TypeError(f"{what}: dtype {t.dtype} is not {dtype}")
        if t.dim() != 1 or t.shape[0] != self.n:
            raise ValueError(f"{what}: expected {self.n} elements in one dimension, has shape {tuple(t.shape)}")
        if not t.is_cuda:
            raise ValueError(f"{what}: must be a device (cuda) tensor")
        if not t.is_contiguous():
            raise ValueError(f"{what}: must be contiguous")
        if t.get_device() != self.device:
            self.on(t.get_device(), what)
        return t.data_ptr()

    def workspace(self, t, need: int):
        if need < 0:
            return None   # the library says which size is out of range
        return self.ptr(t, "workspace", "bytes", need)


def embedding_lookup(plan: Plan, param_index: int, vocab: int, params, tokens, out, scale: float = 1.0,
                     stream=None) -> None:
    """out[i] = scale * W[tokens[i]], W the first `vocab` rows of parameter
    param_index in the bf16 buffer params (N elements); a token outside [0,
    vocab) gives zeros. out: bfloat16 or float32 [n, dim]."""
    call = _VocabCall(plan)
    o, kind, stride = call.rows(out, "out")
    p = call.ptr(params, "params", "bf16", plan.buffer_numel)
    t = call.tokens(tokens, "tokens", "int64")
    _check(require_library().embedding_lookup(plan.handle, param_index, vocab, call.dim, p, t, call.n, scale, o, kind,
                                              stride, call.stream(stream)))


def embedding_grad(plan: Plan, param_index: int, vocab: int, tokens, grad_out, grads, workspace, scale: float = 1.0,
                   accumulate: bool = False, stream=None) -> None:
    """The lookup's gradient, scale * (the sum of grad_out's rows by token),
    into parameter param_index of the bf16 buffer grads (N elements): over
    what it holds, zero for rows that no token names, or with accumulate added
    to it. workspace: uint8, embedding_grad_workspace_bytes(n, dim)."""
    call, L = _VocabCall(plan), require_library()
    x, kind, stride = call.rows(grad_out, "grad_out")
    t = call.tokens(tokens, "tokens", "int64")
    g = call.ptr(grads, "grads", "bf16", plan.buffer_numel)
    ws = call.workspace(workspace, L.zdo_embedding_grad_workspace_bytes(call.n, call.dim))
    _check(L.embedding_grad(plan.handle, param_index, vocab, call.dim, t, call.n, x, kind, stride, scale,
                            bool(accumulate), g, ws, call.stream(stream)))


def linear_cross_entropy(plan: Plan, param_index: int, vocab: int, params, hidden, targets, loss, lse, workspace,
                         stream=None) -> None:
    """Softmax cross entropy of the logits hidden W^T, which are not kept:
    lse[i] their log-sum-exp, loss[i] = lse[i] - logit[targets[i]], 0 where
    the target is outside [0, vocab). hidden: bfloat16 [n, dim]; loss, lse:
    float32 [n]; workspace: uint8,
    linear_cross_entropy_workspace_bytes(n, vocab, dim)."""
    call, L = _VocabCall(plan), require_library()
    h, _, stride = call.rows(hidden, "hidden", "bf16")
    p = call.ptr(params, "params", "bf16", plan.buffer_numel)
    t = call.tokens(targets, "targets", "int64")
    lo, ls = call.tokens(loss, "loss", "float32"), call.tokens(lse, "lse", "float32")
    ws = call.workspace(workspace, L.zdo_linear_cross_entropy_workspace_bytes(call.n, vocab, call.dim))
    _check(L.linear_cross_entropy(plan.handle, param_index, vocab, call.dim, p, h, stride, t, call.n, lo, ls, ws,
                                  call.stream(stream)))


def linear_cross_entropy_grad(plan: Plan, param_index: int, vocab: int, params, hidden, targets, lse, grad_loss,
                              grad_hidden, grads, workspace, accumulate: bool = False, stream=None) -> None:
    """The gradients of sum(grad_loss * loss), given linear_cross_entropy's
    lse: by hidden into grad_hidden (bfloat16 or float32 [n, dim], or None),
    by W into parameter param_index of the bf16 buffer grads (N elements, or
    None), over what it holds or with accumulate added to it. workspace: as
    linear_cross_entropy's."""
    call, L = _VocabCall(plan), require_library()
    h, _, stride = call.rows(hidden, "hidden", "bf16")
    p = call.ptr(params, "params", "bf16", plan.buffer_numel)
    t = call.tokens(targets, "targets", "int64")
    ls, w = call.tokens(lse, "lse", "float32"), call.tokens(grad_loss, "grad_loss", "float32")
    gh, kind, gh_stride = (None, BF16, 0) if grad_hidden is None else call.rows(grad_hidden, "grad_hidden")
    g = call.opt(grads, "grads", "bf16", plan.buffer_numel)
    ws = call.workspace(workspace, L.zdo_linear_cross_entropy_workspace_bytes(call.n, vocab, call.dim))
    _check(L.linear_cross_entropy_grad(plan.handle, param_index, vocab, call.dim, p, h, stride, t, call.n, ls, w, gh,
                                       kind, gh_stride, bool(accumulate), g, ws, call.stream(stream)))
