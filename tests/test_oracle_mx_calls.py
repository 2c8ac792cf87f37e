"""Pins of the MXFP4 oracle's calls (oracle/mx.py): the reduction, its squared
norm, the step with its options and the write-back, each against a reference
that goes element by element from the bucket table, with exact fractions for
values and roundings to the format. Then the mistakes that these pins must
notice, planted in a copy of the oracle."""

import os
import types
from fractions import Fraction

import numpy as np
import pytest

import oracle.layout as OL
import oracle.mx
import oracle.mx as MX
import oracle.numerics as ON

SOURCE = open(os.path.join(os.path.dirname(oracle.mx.__file__), "mx.py")).read()
WORLD, LOCAL = 0, 1
SENTINEL = 0x1234
MAGS = [Fraction(x) for x in ("0", "1/2", "1", "3/2", "2", "3", "4", "6")]
LAYOUTS = [([70, 9, 130], 80, 2), ([200], 200, 3), ([5, 3], 4, 4), ([64, 33, 31, 100], 64, 1)]


class Element:
    """One slot of a rank's range: its bucket, WORLD and LOCAL index, block in
    WORLD and LOCAL storage, place in the block, and whether it is a
    parameter element."""

    def __init__(self, b, w, k, world, local, i, own):
        self.b, self.w, self.k, self.block, self.i, self.own = b, w, k, (world, local), i, own


def elements(lay, rank):
    """Every slot of the rank's ranges, in order."""
    D, tile, end, out = lay.dp_size, 0, 0, []
    for b in lay.buckets:
        S = b.padded_numel // D
        T = (S + 574) // 512
        rs = b.offset + rank * S
        base = end
        while base % 64 != rs % 64:
            base += 1
        for w in range(rs, rs + S):
            at = w - rs // 64 * 64
            out.append(Element(b.index, w, base + w - rs, 16 * (D * tile + rank * T) + at // 32,
                               16 * tile + at // 32, at % 32, w < b.offset + b.numel))
        tile, end = tile + T, base + S
    return out


def value(storage, coords, e):
    """The slot's value, which an fp64 holds; the sign of a zero is kept."""
    codes, scales = storage
    blk = e.block[coords]
    if scales[blk] == 255:
        return float("nan")
    byte = int(codes[blk, e.i // 2])
    code = byte >> 4 if e.i % 2 else byte & 15
    size = float(MAGS[code & 7] * Fraction(2) ** (int(scales[blk]) - 127))
    return -size if code >> 3 else size


def grad(stores, coords, e, scale):
    """fp32 sum in the order given, times the scale."""
    acc = np.float32(value(stores[0], coords, e))
    for s in stores[1:]:
        acc = np.float32(acc + np.float32(value(s, coords, e)))
    return np.float32(acc * np.float32(scale))


def rounded(xs):
    """Up to 32 finite values that share a block to the format, as Fractions."""
    top = max(abs(x) for x in xs)
    e = -127
    while top >= Fraction(2) ** (e + 3):
        e += 1
    out = []
    for x in xs:
        y = abs(x) / Fraction(2) ** e
        near = min(abs(y - m) for m in MAGS)
        best = [c for c, m in enumerate(MAGS) if abs(y - m) == near]
        c = best[0] if len(best) == 1 or best[0] % 2 == 0 else best[1]
        out.append((1 if x >= 0 else -1) * MAGS[c] * Fraction(2) ** e)
    return out


def check_written(lay, rank, storage, coords, master, buckets, fill):
    """The storage holds the rounded master in the rank's blocks of those
    buckets, zero in their other slots, and `fill` everywhere else."""
    blocks, touched = {}, np.zeros(storage[1].size, bool)
    for e in elements(lay, rank):
        if buckets is None or buckets[0] <= e.b < buckets[1]:
            blocks.setdefault(e.block[coords], []).append(e)
    D, tile = lay.dp_size, 0
    for b in lay.buckets:
        T = (b.padded_numel // D + 574) // 512
        if buckets is None or buckets[0] <= b.index < buckets[1]:
            at = 16 * (D * tile + rank * T) if coords == WORLD else 16 * tile
            touched[at:at + 16 * T] = True
        tile += T
    for blk, es in blocks.items():
        own = [e for e in es if e.own]
        want = rounded([Fraction(float(master[e.k])) for e in own]) if own else []
        want = dict(zip((e.i for e in own), want))
        for i in range(32):
            e = Element(0, 0, 0, blk, blk, i, True)
            assert value(storage, coords, e) == want.get(i, 0), (blk, i)
    for blk in range(storage[1].size):
        if not touched[blk]:
            assert (storage[0][blk] == fill).all() and storage[1][blk] == fill
        elif blk not in blocks:
            assert not storage[0][blk].any() and storage[1][blk] == 0


def random_stores(rng, lay, coords, n, lo=118, hi=134):
    nb = MX.storage_blocks(lay, coords)
    return [(rng.integers(0, 256, (nb, 16), dtype=np.uint8), rng.integers(lo, hi, nb).astype(np.uint8))
            for _ in range(n)]


def some_buckets(lay):
    nb = len(lay.buckets)
    return [None, (0, 1), (nb - 1, nb), (nb, nb)]


@pytest.mark.parametrize("sizes, bucket, D", LAYOUTS)
def test_reduce(sizes, bucket, D):
    lay = OL.build_layout(sizes, bucket, D)
    rng = np.random.default_rng(D)
    for r in range(D):
        for coords in (WORLD, LOCAL):
            stores = random_stores(rng, lay, coords, 3)
            stores[1][1][::7] = 255
            for oc, scale, buckets in zip((WORLD, LOCAL, WORLD, LOCAL), (0.3, 1.0, 0.0625, 0.7), some_buckets(lay)):
                size = lay.buffer_numel if oc == WORLD else OL.shard_numel(lay, r)
                got, want = (np.full(size, SENTINEL, np.uint16) for _ in range(2))
                MX.reduce_scatter(lay, r, stores, coords, scale, got, oc, buckets)
                for e in elements(lay, r):
                    if buckets is None or buckets[0] <= e.b < buckets[1]:
                        want[e.w if oc == WORLD else e.k] = ON.narrow(np.array([grad(stores, coords, e, scale)]))[0]
                nan = (want & 0x7FFF) > 0x7F80
                assert np.array_equal(nan, (got & 0x7FFF) > 0x7F80) and np.array_equal(got[~nan], want[~nan])


@pytest.mark.parametrize("sizes, bucket, D", LAYOUTS)
def test_norm(sizes, bucket, D):
    """Against the exact sum of squares; every square is exact in fp64 and the
    fewer than 2^10 additions each round by 2^-53 at most, relatively."""
    lay = OL.build_layout(sizes, bucket, D)
    rng = np.random.default_rng(D)
    for r in range(D):
        for coords, scale in ((WORLD, 0.3), (LOCAL, 1.0)):
            stores = random_stores(rng, lay, coords, 3)
            want = sum((Fraction(float(grad(stores, coords, e, scale))) ** 2 for e in elements(lay, r) if e.own),
                       Fraction(0))
            got = Fraction(float(MX.norm_sq(lay, r, stores, coords, scale)))
            assert abs(got - want) <= want * Fraction(1, 1 << 43)
            own = [e for e in elements(lay, r) if e.own]
            if own:
                for s in stores:
                    s[1][own[-1].block[coords]] = 255
                assert np.isnan(MX.norm_sq(lay, r, stores, coords, scale))


@pytest.mark.parametrize("sizes, bucket, D", LAYOUTS)
def test_the_order_of_the_sum(sizes, bucket, D):
    """Scales far enough apart that every order of the sum has its own roundings."""
    lay = OL.build_layout(sizes, bucket, D)
    rng = np.random.default_rng(D)
    for r in range(D):
        stores = random_stores(rng, lay, LOCAL, 5, 100, 150)
        for b in range(len(lay.buckets)):
            want = [grad(stores, LOCAL, e, 0.3) for e in elements(lay, r) if e.b == b and e.own]
            got = MX.owned_grad(lay, r, stores, LOCAL, 0.3, b, np.float32)
            assert np.array_equal(got.view(np.uint32), np.array(want, np.float32).view(np.uint32))


def adam(hp, g, p, m, v):
    """One element in fp32, one operation after the other."""
    f = np.float32
    lr, b1, b2, eps, wd, bc1, bc2 = (f(x) for x in hp)
    m1 = f(f(b1 * m) + f(f(f(1) - b1) * g))
    v1 = f(f(b2 * v) + f(f(f(1) - b2) * f(g * g)))
    u = f(f(m1 / bc1) / f(f(np.sqrt(f(v1 / bc2))) + eps))
    return f(p - f(lr * f(u + f(wd * p)))), m1, v1


@pytest.mark.parametrize("sizes, bucket, D", LAYOUTS)
def test_step(sizes, bucket, D):
    """With and without a coefficient, the main grad, parameters in both
    formats and coordinates, all buckets and some."""
    lay = OL.build_layout(sizes, bucket, D)
    rng = np.random.default_rng(D)
    hp = ON.hp_array(dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1), 3)
    for r in range(D):
        Ln = OL.shard_numel(lay, r)
        st = [rng.standard_normal(Ln).astype(np.float32), (rng.standard_normal(Ln) * 1e-2).astype(np.float32),
              (rng.random(Ln) * 1e-3).astype(np.float32)]
        for i, buckets in enumerate(some_buckets(lay)):
            for coeff in (None, np.float32(0.37), np.float32(np.nan)):
                coords, pc, mc = (i % 2, (i + 1) % 2, i // 2)
                stores = random_stores(rng, lay, coords, 3)
                got, want = [x.copy() for x in st], [x.copy() for x in st]
                par, wpar = (np.full(lay.buffer_numel if pc == WORLD else Ln, SENTINEL, np.uint16) for _ in range(2))
                mg, wmg = (np.full(Ln, -7, np.float32) for _ in range(2))
                mx = MX.empty(lay, mc, 0xA7)
                MX.step(lay, r, stores, coords, 0.3, *got, hp, par, pc, mx, mc, coeff, mg, buckets)
                skip = coeff is not None and np.isnan(coeff)
                for e in [] if skip else elements(lay, r):
                    if not e.own or not (buckets is None or buckets[0] <= e.b < buckets[1]):
                        continue
                    g = grad(stores, coords, e, 0.3)
                    if coeff is not None:
                        g = np.float32(g * coeff)
                    for x, y in zip(want, adam(hp, g, *(x[e.k] for x in st))):
                        x[e.k] = y
                    wmg[e.k] = g
                    wpar[e.w if pc == WORLD else e.k] = ON.narrow(np.array([want[0][e.k]]))[0]
                for x, y in zip((*got, mg), (*want, wmg)):
                    assert np.array_equal(x.view(np.uint32), y.view(np.uint32))
                assert np.array_equal(par, wpar)
                check_written(lay, r, mx, mc, want[0], (0, 0) if skip else buckets, 0xA7)
                # no outputs but the state
                bare = [x.copy() for x in st]
                MX.step(lay, r, stores, coords, 0.3, *bare, hp, coeff=coeff, buckets=buckets)
                assert all(np.array_equal(x, y) for x, y in zip(bare, got))


@pytest.mark.parametrize("sizes, bucket, D", LAYOUTS)
def test_writeback(sizes, bucket, D):
    lay = OL.build_layout(sizes, bucket, D)
    rng = np.random.default_rng(D)
    for r in range(D):
        master = np.ldexp(rng.standard_normal(OL.shard_numel(lay, r)), rng.integers(-20, 20)).astype(np.float32)
        for coords in (WORLD, LOCAL):
            mx = MX.empty(lay, coords, 0xA7)
            MX.writeback(lay, r, master, mx, coords)
            check_written(lay, r, mx, coords, master, None, 0xA7)


# ---- planted mistakes -----------------------------------------------------------------------

MUTANTS = {
    "norm of g": ("np.sum(g * g)", "np.sum(g)"),
    "norm of the last bucket": ("t = t + float(np.sum", "t = float(np.sum"),
    "norm counts the padding": ("dtype)[:rng[1] - rng[0].start] * dtype", "dtype) * dtype"),
    "divided by the coefficient": ("g = g * dtype(coeff)", "g = g / dtype(coeff)"),
    "NaN coefficient does not skip": ("if coeff is not None and np.isnan(coeff):", "if False:"),
    "main grad doubled": ("main_grad[k] = g", "main_grad[k] = 2 * g"),
    "main grad not written": ("main_grad[k] = g", "pass"),
    "MXFP4 parameters not written": ("_put(param_mx, param_mx_coords, rng, master[k])", "pass"),
    "MXFP4 parameters in the other coordinates": ("_put(param_mx, param_mx_coords, rng",
                                                  "_put(param_mx, 1 - param_mx_coords, rng"),
    "MXFP4 parameters before the step": (
        "        master[k], m[k], v[k] = adam(hp, g, master[k], m[k], v[k], dtype)\n",
        "        was = master[k].copy()\n        master[k], m[k], v[k] = adam(hp, g, master[k], m[k], v[k], dtype)\n"
        "        if param_mx is not None:\n            _put(param_mx, param_mx_coords, rng, was)\n"
        "        param_mx = None\n"),
    "bf16 parameters in the other coordinates": ("s = rng[0].start if param_coords == WORLD else rng[2]",
                                                 "s = rng[0].start if param_coords != WORLD else rng[2]"),
    "step ignores the buckets": (
        "        if not _keep(buckets, b):\n            continue\n        g = owned_grad",
        "        g = owned_grad"),
    "reduce without the scale": ("np.float32) * np.float32(scale)\n        s = ", "np.float32)\n        s = "),
    "reduce ignores out_coords": ("s = rng[0].start if out_coords == WORLD else rng[2]", "s = rng[0].start"),
    "reduce ignores the buckets": (
        "        if not _keep(buckets, b):\n            continue\n        with np.errstate(over=\"ignore\", invalid",
        "        with np.errstate(over=\"ignore\", invalid"),
    "reduce by WORLD storage only": ("s = rng[4] if coords == WORLD else rng[5]\n    return decode",
                                     "s = rng[4]\n    return decode"),
    "the last bucket of a range counted": ("buckets[0] <= b < buckets[1]", "buckets[0] <= b <= buckets[1]"),
    "write-back doubled": ("_put(storage, coords, rng, master[", "_put(storage, coords, rng, 2 * master["),
    "write-back of the padding": ("master[rng[2]:rng[2] + rng[1] - rng[0].start])",
                                  "master[rng[2]:rng[2] + rng[0].size])"),
    "write-back from WORLD places": ("master[rng[2]:rng[2] + rng[1] - rng[0].start])",
                                     "master[rng[0].start:rng[1]])"),
    "the sum in 64 bits": ("acc = acc + _values(s, coords, rng).astype(dtype)",
                           "acc = (acc + _values(s, coords, rng)).astype(np.float64)"),
    "the sum from the last": ("for s in storages[1:]:\n            acc = acc + ",
                              "for s in storages[:0:-1]:\n            acc = acc + "),
}


def pins():
    for pin in (test_reduce, test_norm, test_the_order_of_the_sum, test_step, test_writeback):
        for case in LAYOUTS:
            yield lambda: pin(*case)


def failing(source, monkeypatch):
    """Whether some pin fails on this source."""
    mod = types.ModuleType("oracle.mx")
    mod.__package__ = "oracle"
    exec(compile(source, "mx.py", "exec"), mod.__dict__)
    monkeypatch.setitem(globals(), "MX", mod)
    with np.errstate(all="ignore"):
        for pin in pins():
            try:
                pin()
            except Exception:
                return True
    return False


def test_the_oracle_as_it_is_passes(monkeypatch):
    assert not failing(SOURCE, monkeypatch)


@pytest.mark.parametrize("name", MUTANTS)
def test_a_mistake_is_noticed(name, monkeypatch):
    old, new = MUTANTS[name]
    assert SOURCE.count(old) == 1, name
    assert failing(SOURCE.replace(old, new), monkeypatch), name
