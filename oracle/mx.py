"""CPU oracle of the MXFP4 contributions and parameters: the format, its
storage and the calls on it, written from the definitions with numpy.

TEST INFRASTRUCTURE; see oracle/__init__.py.

Format (OCP Microscaling Formats v1.0): blocks of 32 share an E8M0 scale, the
elements are E2M1. Storage: per bucket and rank, T = (S + 574) // 512 tiles of
16 blocks from the range's first WORLD element rounded down to 64, bucket
after bucket; WORLD storage holds the D ranges of a bucket in rank order,
LOCAL storage one rank's.

The sums and Adam take the dtype to compute in: float32 repeats the fixed
order and roundings bit for bit, float64 is the plain value.
"""

from __future__ import annotations

import numpy as np

from . import layout as L
from . import numerics as N

WORLD, LOCAL = 0, 1
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ---- the format -------------------------------------------------------------------------

def decode(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """codes [B, 16], scales [B] -> values [B, 32] (float64, exact)."""
    nib = np.empty((codes.shape[0], 32), np.uint8)
    nib[:, 0::2] = codes & 15
    nib[:, 1::2] = codes >> 4
    v = MAGNITUDES[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    unit = np.ldexp(1.0, scales.astype(np.int64) - 127)
    return v * np.where(scales == 255, np.nan, unit)[:, None]


def encode(x: np.ndarray):
    """Values [B, 32] (float32 or float64) -> codes [B, 16], scales [B]: the
    nearest of the eight magnitudes, found by trying all of them; of two that
    are equally near the one with the even code."""
    with np.errstate(invalid="ignore"):     # NaN bits of any kind
        x = np.asarray(x, np.float64)
    top = np.abs(x).max(axis=1, initial=0.0)
    bad = ~np.isfinite(top)
    _, e = np.frexp(np.where(bad, 1.0, top))        # top = m * 2^e, 0.5 <= m < 1
    byte = np.where(top == 0, 0, np.maximum(e - 1 - 2 + 127, 0))
    y = np.abs(x) * np.ldexp(1.0, 127 - byte)[:, None]
    y = np.where(bad[:, None], 0.0, y)
    best = np.zeros(x.shape, np.uint8)
    dist = np.abs(y - MAGNITUDES[0])
    for c in range(1, 8):
        d = np.abs(y - MAGNITUDES[c])
        best = np.where((d < dist) | ((d == dist) & (c % 2 == 0)), c, best).astype(np.uint8)
        dist = np.minimum(d, dist)
    code = np.where(bad[:, None], 0, best + 8 * np.signbit(x)).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), np.where(bad, 255, byte).astype(np.uint8)


# ---- storage ------------------------------------------------------------------------------

def tiles(shard: int) -> int:
    return (shard + 574) // 512


def storage_blocks(layout: L.Layout, coords: int) -> int:
    n = sum(16 * tiles(b.shard_numel(layout.dp_size)) for b in layout.buckets)
    return n * layout.dp_size if coords == WORLD else n


def ranges(layout: L.Layout, rank: int):
    """The rank's ranges: (world Range, parameter end, LOCAL start, phase,
    block slices in WORLD and LOCAL storage)."""
    D, bases, out, at = layout.dp_size, L.shard_bases(layout, rank)[0], [], 0
    for b, base in zip(layout.buckets, bases):
        nb = 16 * tiles(b.shard_numel(D))
        r = L.rank_range(b, D, rank)
        own = max(r.start, min(r.end, b.offset + b.numel))
        w = D * at + rank * nb
        out.append((r, own, base, r.start % 64, slice(w, w + nb), slice(at, at + nb)))
        at += nb
    return out


def _values(storage, coords, rng):
    codes, scales = storage
    s = rng[4] if coords == WORLD else rng[5]
    return decode(codes[s], scales[s]).reshape(-1)[rng[3]:rng[3] + rng[0].size]


def _put(storage, coords, rng, x):
    """Rounds x (the range's parameter elements) into its blocks; all of the
    range's other slots are zero."""
    s = rng[4] if coords == WORLD else rng[5]
    flat = np.zeros(32 * (s.stop - s.start), x.dtype)
    flat[rng[3]:rng[3] + x.size] = x
    storage[0][s], storage[1][s] = encode(flat.reshape(-1, 32))


def empty(layout: L.Layout, coords: int, fill: int = 0):
    n = storage_blocks(layout, coords)
    return np.full((n, 16), fill, np.uint8), np.full(n, fill, np.uint8)


def _keep(buckets, b):
    return buckets is None or buckets[0] <= b < buckets[1]


# ---- the calls --------------------------------------------------------------------------------

def quantize(layout: L.Layout, rank: int, grads: np.ndarray, coords: int, storage, residual=None, buckets=None):
    """grads: uint16 bf16 bits; storage and residual (float32) in place."""
    g = (grads.astype(np.uint32) << 16).view(np.float32)
    for r in range(layout.dp_size) if coords == WORLD else [rank]:
        for b, rng in enumerate(ranges(layout, r)):
            if not _keep(buckets, b):
                continue
            at = slice(rng[0].start, rng[1]) if coords == WORLD else slice(rng[2], rng[2] + rng[1] - rng[0].start)
            x = g[at]
            if residual is not None:
                with np.errstate(invalid="ignore", over="ignore"):
                    x = x + residual[at]        # float32
            _put(storage, coords, rng, x)
            if residual is not None:
                y = _values(storage, coords, rng)[:x.size]
                with np.errstate(invalid="ignore"):
                    residual[at] = np.where(np.isnan(y), residual[at], x - y.astype(np.float32))


def total(layout, rank, storages, coords, b, dtype):
    rng = ranges(layout, rank)[b]
    with np.errstate(over="ignore", invalid="ignore"):
        acc = _values(storages[0], coords, rng).astype(dtype)
        for s in storages[1:]:
            acc = acc + _values(s, coords, rng).astype(dtype)
    return acc


def reduce_scatter(layout, rank, storages, coords, scale, out, out_coords, buckets=None):
    """out: uint16 bf16 bits."""
    for b, rng in enumerate(ranges(layout, rank)):
        if not _keep(buckets, b):
            continue
        with np.errstate(over="ignore", invalid="ignore"):
            v = total(layout, rank, storages, coords, b, np.float32) * np.float32(scale)
        s = rng[0].start if out_coords == WORLD else rng[2]
        out[s:s + v.size] = N.narrow(v)


def owned_grad(layout, rank, storages, coords, scale, b, dtype):
    rng = ranges(layout, rank)[b]
    with np.errstate(over="ignore", invalid="ignore"):
        return total(layout, rank, storages, coords, b, dtype)[:rng[1] - rng[0].start] * dtype(np.float32(scale))


def norm_sq(layout, rank, storages, coords, scale) -> float:
    t = 0.0
    for b in range(len(layout.buckets)):
        g = owned_grad(layout, rank, storages, coords, scale, b, np.float32).astype(np.float64)
        t = t + float(np.sum(g * g))
    return t


def adam(hp, g, p, m, v, dtype):
    """hp: oracle.numerics.hp_array; returns the new p, m, v."""
    lr, b1, b2, eps, wd, bc1, bc2 = (dtype(x) for x in hp)
    one = np.float32(1)
    omb1, omb2 = dtype(one - np.float32(hp[1])), dtype(one - np.float32(hp[2]))
    p, m, v, g = (np.asarray(x).astype(dtype) for x in (p, m, v, g))
    with np.errstate(all="ignore"):
        mn = b1 * m + omb1 * g
        vn = b2 * v + omb2 * (g * g)
        u = (mn / bc1) / (np.sqrt(vn / bc2) + eps)
        return p - lr * (u + wd * p), mn, vn


def step(layout, rank, storages, coords, scale, master, m, v, hp, param_out=None, param_coords=WORLD,
         param_mx=None, param_mx_coords=LOCAL, coeff=None, main_grad=None, buckets=None, dtype=np.float32):
    """In place on master, m, v (float32, or float64 with that dtype) and the outputs."""
    if coeff is not None and np.isnan(coeff):
        return
    for b, rng in enumerate(ranges(layout, rank)):
        if not _keep(buckets, b):
            continue
        g = owned_grad(layout, rank, storages, coords, scale, b, dtype)
        if coeff is not None:
            with np.errstate(invalid="ignore"):
                g = g * dtype(coeff)
        k = slice(rng[2], rng[2] + g.size)
        master[k], m[k], v[k] = adam(hp, g, master[k], m[k], v[k], dtype)
        if main_grad is not None:
            main_grad[k] = g
        if param_out is not None:
            s = rng[0].start if param_coords == WORLD else rng[2]
            param_out[s:s + g.size] = N.narrow(master[k].astype(np.float32))
        if param_mx is not None:
            _put(param_mx, param_mx_coords, rng, master[k])


def writeback(layout, rank, master, storage, coords):
    for rng in ranges(layout, rank):
        _put(storage, coords, rng, master[rng[2]:rng[2] + rng[1] - rng[0].start])


def all_gather(layout, storages, coords, out):
    """out: uint16 bf16 bits."""
    for j, s in enumerate(storages):
        for rng in ranges(layout, j):
            with np.errstate(over="ignore", invalid="ignore"):
                out[rng[0].start:rng[0].end] = N.narrow(_values(s, coords, rng).astype(np.float32))
