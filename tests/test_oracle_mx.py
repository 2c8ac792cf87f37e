"""Pins of the MXFP4 oracle (oracle/mx.py): the format against the OCP
definition's own tables and exact fractions, the storage against an
element-by-element owner scan, and the composition against the bf16 oracle
where the two must agree."""

import random
from fractions import Fraction

import numpy as np
import pytest

import oracle.layout as OL
import oracle.mx as MX
import oracle.numerics as ON
import oracle.step as OS
import workloads as W


def test_decode_table():
    """E2M1: sign, exponent bias 1, one mantissa bit; E8M0: 2^(e - 127)."""
    for code in range(16):
        s, e, m = code >> 3, (code >> 1) & 3, code & 1
        mag = Fraction(m, 2) if e == 0 else (1 + Fraction(m, 2)) * Fraction(2) ** (e - 1)
        for byte in (0, 1, 126, 127, 128, 254):
            v = MX.decode(np.full((1, 16), code | code << 4, np.uint8), np.array([byte], np.uint8))
            want = (-1) ** s * mag * Fraction(2) ** (byte - 127)
            assert all(Fraction(float(x)) == want for x in v[0])
    assert np.isnan(MX.decode(np.zeros((1, 16), np.uint8), np.array([255], np.uint8))).all()
    # the even element sits in the low half
    v = MX.decode(np.full((1, 16), 0x21, np.uint8), np.array([127], np.uint8))[0]
    assert v[0::2].tolist() == [0.5] * 16 and v[1::2].tolist() == [1.0] * 16


@pytest.mark.parametrize("top", [7.9, 6.0, 5.0, 4.0])
def test_encode_rounds_to_nearest_even_and_saturates(top):
    """One block with its largest magnitude in [4, 8): scale 2^0. Every 1/64
    below it, in exact fractions."""
    grid = [Fraction(i, 64) for i in range(int(top * 64) + 1)]
    for i in range(0, len(grid), 31):
        xs = grid[i:i + 31]
        block = np.zeros(32)
        block[:len(xs)] = [float(x) for x in xs]
        block[31] = top
        codes, scales = MX.encode(block[None])
        assert scales[0] == 127
        got = MX.decode(codes, scales)[0]
        mags = [Fraction(x) for x in MX.MAGNITUDES]
        for x, g in zip(xs, got):
            near = min(abs(x - m) for m in mags)
            best = [c for c, m in enumerate(mags) if abs(x - m) == near]
            want = next(c for c in best if len(best) == 1 or c % 2 == 0)
            assert Fraction(float(g)) == mags[want]
        assert got[31] == {7.9: 6.0, 6.0: 6.0, 5.0: 4.0, 4.0: 4.0}[top]


def test_encode_scale_and_specials():
    x = np.zeros((8, 32), np.float32)
    x[1, 3] = -0.0
    x[2, 0] = np.float32(2.0**-149)         # the smallest subnormal
    x[3, 5] = np.float32(2.0**-125)         # exponent field 2: scale byte 0
    x[4, 5] = np.float32(2.0**-124)         # exponent field 3: scale byte 1
    x[5, 1] = np.finfo(np.float32).max
    x[6, 1] = np.inf
    x[7, 1] = np.nan
    codes, scales = MX.encode(x)
    assert scales.tolist() == [0, 0, 0, 0, 1, 252, 255, 255]
    v = MX.decode(codes, scales)
    assert not v[0].any() and np.signbit(v[1, 3]) and not v[2].any()
    assert v[3, 5] == 2.0**-125 and v[4, 5] == 2.0**-124 and v[5, 1] == 6 * 2.0**125
    assert np.isnan(v[6]).all() and np.isnan(v[7]).all() and not codes[6:].any()
    rng = np.random.default_rng(3)
    y = np.ldexp(rng.standard_normal((4000, 32)), rng.integers(-140, 120, (4000, 1))).astype(np.float32)
    top = np.abs(y).max(axis=1)
    _, s = MX.encode(y)
    assert np.array_equal(s, np.maximum((top.view(np.uint32) >> 23).astype(int) - 2, 0))
    assert (top.astype(np.float64) < 8 * np.ldexp(1.0, s.astype(int) - 127)).all()


def _layout(seed):
    pr = random.Random(seed)
    sizes = [pr.choice([1, 2, 31, 32, 33, 511, 512, 513, pr.randint(1, 3000)]) for _ in range(pr.randint(1, 12))]
    return pr, OL.build_layout(sizes, pr.randint(1, max(2, sum(sizes) // pr.choice([1, 2, 4]))),
                               pr.choice([1, 2, 3, 5, 8, 64]))


@pytest.mark.parametrize("seed", range(25))
def test_storage_holds_every_element_once(seed):
    """Writes each parameter element's WORLD index (small integers, each in a
    block of its own scale) through the storage formula, element by element
    from the bucket table, and reads the ranges back."""
    _, lay = _layout(seed)
    D = lay.dp_size
    at, seen = 0, set()
    for b in lay.buckets:
        S = b.padded_numel // D
        T = (S + 574) // 512
        for r in range(D):
            rs = b.offset + r * S
            origin = rs // 64 * 64
            for w in range(rs, rs + S):
                block = D * at + r * 16 * T + (w - origin) // 32
                assert D * at + r * 16 * T <= block < D * at + (r + 1) * 16 * T
                slot = (block, (w - origin) % 32)
                assert slot not in seen
                seen.add(slot)
        at += 16 * T
    assert D * at == MX.storage_blocks(lay, MX.WORLD) and at == MX.storage_blocks(lay, MX.LOCAL)
    for r in range(D):
        for (rng, own, base, phase, ws, ls), b in zip(MX.ranges(lay, r), lay.buckets):
            assert phase == rng.start % 64 == base % 64
            assert own - rng.start == sum(p.gbuf_world.size for p in OL.rank_pieces(lay, r)
                                          if p.bucket_index == b.index)


@pytest.mark.parametrize("seed", range(6))
def test_local_storage_is_the_ranks_part_of_world_storage(seed):
    pr, lay = _layout(100 + seed)
    rng = np.random.default_rng(seed)
    g = ON.narrow(rng.standard_normal(lay.buffer_numel).astype(np.float32))
    whole = MX.empty(lay, MX.WORLD)
    MX.quantize(lay, 0, g, MX.WORLD, whole)
    for r in range(lay.dp_size):
        mine = MX.empty(lay, MX.LOCAL)
        MX.quantize(lay, r, OS.local_slices(lay, r, g), MX.LOCAL, mine)
        for x in MX.ranges(lay, r):
            assert np.array_equal(whole[0][x[4]], mine[0][x[5]]) and np.array_equal(whole[1][x[4]], mine[1][x[5]])


@pytest.mark.parametrize("seed", range(4))
def test_step_equals_the_bf16_step_on_values_that_both_hold(seed):
    """Contributions whose elements are +-2^k times a block's scale survive
    both formats and sum exactly: with a power-of-two scale factor the MXFP4
    step equals the bf16 oracle's, padding and all ranks included."""
    pr, lay = _layout(200 + seed)
    D, N = lay.dp_size, lay.buffer_numel
    rng = np.random.default_rng(seed)
    vals = rng.choice([0.0, 0.5, -0.5, 1.0, -1.0, 2.0, -2.0, 4.0], (D, N)).astype(np.float32)
    vals[:, ::16] = 4.0    # every block's scale is 2^0
    reps = [ON.narrow(x) for x in vals]
    stores = []
    for g in reps:
        s = MX.empty(lay, MX.WORLD)
        MX.quantize(lay, 0, g, MX.WORLD, s)
        stores.append(s)
    hp = ON.hp_array(W.get("tiny").hp, 3)
    for r in range(D):
        Ln = OL.shard_numel(lay, r)
        st = [(rng.standard_normal(Ln) * 0.02).astype(np.float32), (rng.standard_normal(Ln) * 1e-3).astype(np.float32),
              (rng.random(Ln) * 1e-6).astype(np.float32)]
        a, b = [x.copy() for x in st], [x.copy() for x in st]
        pa, pb = np.full(N, 7, np.uint16), np.full(N, 7, np.uint16)
        OS.rank_step(lay, r, reps, OS.WORLD, 0.0625, *a, hp, pa, OS.WORLD)
        MX.step(lay, r, stores, MX.WORLD, 0.0625, *b, hp, pb, MX.WORLD)
        for x, y in zip(a, b):
            assert np.array_equal(x.view(np.uint32), y.view(np.uint32))
        assert np.array_equal(pa, pb)


def test_residual_carries_what_the_codes_did_not():
    """x = value + residual exactly, so over several steps the values sent and
    the residual left add up to the gradients given, as long as the fp32
    additions are exact (integers here)."""
    lay = OL.build_layout([700, 33], 800, 3)
    rng = np.random.default_rng(0)
    res = np.zeros(lay.buffer_numel, np.float32)
    sent, given = np.zeros(lay.buffer_numel), np.zeros(lay.buffer_numel)
    inside = np.zeros(lay.buffer_numel, bool)
    for b in lay.buckets:
        inside[b.offset:b.offset + b.numel] = True
    for _ in range(6):
        x = rng.integers(-100, 101, lay.buffer_numel).astype(np.float32)
        s = MX.empty(lay, MX.WORLD)
        MX.quantize(lay, 0, ON.narrow(x), MX.WORLD, s, res)
        out = np.zeros(lay.buffer_numel, np.uint16)
        MX.all_gather(lay, [s] * 3, MX.WORLD, out)
        sent += (out.astype(np.uint32) << 16).view(np.float32)
        given += x
    assert np.array_equal((sent + res)[inside], given[inside])
    assert not res[~inside].any()
