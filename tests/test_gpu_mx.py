"""The MXFP4 calls (include/zdo_mx.h) on the GPU against the oracle
(oracle/mx.py). Storage, bf16 outputs and the fp32 state are compared bit for
bit with the fixed-order fp32 oracle (NaN by NaN-ness), with sentinels
wherever a call must not write; the same outputs are held to the 64-bit
definition within bounds derived from the roundings (see `bounds`)."""

import random

import numpy as np
import pytest
import torch

import oracle.layout as OL
import oracle.mx as MX
import oracle.numerics as ON
import oracle.step as OS
import workloads as W
import zero_distributed_optimizer_amd as Z
from zero_distributed_optimizer_amd import build as ZB
from test_gpu_clip import assert_norm
from test_gpu_parity import (DEV, SENTINEL, assert_bf16, assert_f32, bf16_host, free, host_f32, host_u16, hp_kwargs,
                             to_dev)

pytestmark = pytest.mark.gpu

FILL = 0xA7   # storage bytes that no call may touch
EDGES = [1, 2, 7, 31, 32, 33, 63, 64, 65, 511, 512, 513, 1025, 2047, 2048, 2049, 6000, 20011]


def layout_of(seed, dps=(1, 2, 3, 4, 5, 7, 8, 16, 33, 64)):
    pr = random.Random(seed)
    sizes = [pr.choice(EDGES + [pr.randint(1, 9000)]) for _ in range(pr.randint(1, 14))]
    D = pr.choice(dps)
    return pr, sizes, pr.randint(1, max(2, sum(sizes) // pr.choice([1, 2, 5]))), D


def dev_mx(s):
    return tuple(torch.from_numpy(x.copy()).to(DEV) for x in s)


def host_mx(s):
    return tuple(x.cpu().numpy() for x in s)


def assert_mx(got, want, what):
    for g, w, n in zip(host_mx(got), want, ("codes", "scales")):
        bad = np.flatnonzero(g.reshape(-1) != w.reshape(-1))
        assert bad.size == 0, f"{what}: {bad.size} {n} differ, first at {bad[:5]}"


def random_mx(rng, lay, coords, lo=110, hi=130):
    """A storage of any codes in every slot, whatever lies in its padding."""
    n = MX.storage_blocks(lay, coords)
    return rng.integers(0, 256, (n, 16), dtype=np.uint8), rng.integers(lo, hi, n).astype(np.uint8)


def state_of(rng, n):
    return [(rng.standard_normal(n) * 0.02).astype(np.float32), (rng.standard_normal(n) * 1e-3).astype(np.float32),
            ((rng.standard_normal(n) * 1e-3) ** 2 + 1e-12).astype(np.float32)]


@pytest.fixture(params=["library", "long forms"])
def either(gpu, request):
    """The library, and the build that takes the forms for long launches at
    any length, with 64 workgroups at most."""
    if request.param == "library":
        yield gpu
        return
    with Z.use_library(ZB.GRID_LOOP_LIB):
        yield gpu
        free()


# ---- quantising ------------------------------------------------------------------------------

def check_quantize(gpu, sizes, bucket, D, r, coords, g, res=None, buckets=None):
    lay = OL.build_layout(sizes, bucket, D)
    plan = gpu.build_range_map(sizes, bucket, D, r)
    want, want_res = MX.empty(lay, coords, FILL), None if res is None else res.copy()
    MX.quantize(lay, r, g, coords, want, want_res, buckets)
    got = dev_mx(MX.empty(lay, coords, FILL))
    d_res = None if res is None else to_dev(res)
    gpu.quantize_grads_mxfp4(plan, to_dev(g), coords, got, residual=d_res, buckets=buckets)
    assert_mx(got, want, f"D={D} r={r} coords={coords}")
    if res is not None:
        assert np.array_equal(host_f32(d_res).view(np.uint32), want_res.view(np.uint32)), "residual"
    return got


@pytest.mark.parametrize("coords", [0, 1])
@pytest.mark.parametrize("seed", range(12))
def test_quantize_random_layouts(gpu, seed, coords):
    pr, sizes, bucket, D = layout_of(seed)
    rng = np.random.default_rng(seed)
    lay = OL.build_layout(sizes, bucket, D)
    r, N, nb = pr.randrange(D), lay.buffer_numel, len(lay.buckets)
    n = N if coords == gpu.WORLD else OL.shard_numel(lay, r)
    # magnitudes of every size, padding and gaps full of NaN
    x = np.ldexp(rng.standard_normal(n), rng.integers(-140, 100, n)).astype(np.float32)
    g = ON.narrow(np.where(rng.random(n) < 0.1, 0.0, x if seed % 2 else rng.standard_normal(n)).astype(np.float32))
    keep = np.zeros(N, bool)
    for b in lay.buckets:
        keep[b.offset:b.offset + b.numel] = True
    if coords == gpu.LOCAL:
        keep = OS.local_slices(lay, r, keep)
    g = np.where(keep, g, 0x7FC0).astype(np.uint16)
    res = (rng.standard_normal(n) * 0.2).astype(np.float32) if pr.random() < 0.6 else None
    check_quantize(gpu, sizes, bucket, D, r, coords, g, res)
    b0 = pr.randrange(nb)
    check_quantize(gpu, sizes, bucket, D, r, coords, g, res, (b0, pr.randint(b0, nb)))
    free()


def test_quantize_every_bf16_at_every_phase(gpu):
    """Every bf16 pattern, sorted by magnitude so that a block's scale fits
    its members, with single Inf and NaN; ranges that start at odd phases."""
    order = np.argsort(np.arange(1 << 16) & 0x7FFF, kind="stable").astype(np.uint16)
    for D, pre in ((1, 0), (3, 5), (7, 64)):
        n = (1 << 16) + pre
        g = np.concatenate([np.zeros(pre, np.uint16), order])
        g = np.concatenate([g, np.zeros(-(-n // D) * D - n, np.uint16)])
        check_quantize(gpu, [n], n, D, 0, gpu.WORLD, g)
        rng = np.random.default_rng(D)
        res = np.ldexp(rng.standard_normal(g.size), rng.integers(-100, 60, g.size)).astype(np.float32)
        check_quantize(gpu, [n], n, D, 0, gpu.WORLD, g, res)
    free()


@pytest.mark.parametrize("D", [1, 3])
@pytest.mark.parametrize("coords", [0, 1])
def test_quantize_whole_units(either, D, coords):
    """Ranges of many whole units beside their cut ends, with Inf and NaN in
    some blocks, with and without a residual."""
    gpu, rng = either, np.random.default_rng(D)
    sizes, bucket = [50_000, 33, 70_001, 8192, 4096, 2048], 60_000
    lay = OL.build_layout(sizes, bucket, D)
    n = lay.buffer_numel if coords == gpu.WORLD else OL.shard_numel(lay, D - 1)
    g = bf16_host(rng, n)
    g[rng.integers(0, n, 20)] = 0x7F80
    g[rng.integers(0, n, 20)] = 0xFFC1
    check_quantize(gpu, sizes, bucket, D, D - 1, coords, g)
    check_quantize(gpu, sizes, bucket, D, D - 1, coords, g, (rng.standard_normal(n) * 1e-3).astype(np.float32))
    free()


@pytest.mark.parametrize("coords", [0, 1])
def test_parameters_of_whole_units(either, coords):
    gpu, rng = either, np.random.default_rng(7)
    sizes, bucket, D = [50_000, 33, 70_001, 8192], 60_000, 3
    lay = OL.build_layout(sizes, bucket, D)
    want, got = [], []
    for r in range(D):
        plan = gpu.build_range_map(sizes, bucket, D, r)
        m = (rng.standard_normal(plan.shard_numel) * 0.02).astype(np.float32)
        m[rng.integers(0, m.size, 5)] = np.inf
        want.append(MX.empty(lay, coords, FILL))
        got.append(dev_mx(want[-1]))
        MX.writeback(lay, r, m, want[-1], coords)
        gpu.writeback_params_mxfp4(plan, to_dev(m), got[-1], coords)
        assert_mx(got[-1], want[-1], f"write-back r={r}")
    out = torch.full((lay.buffer_numel,), SENTINEL, dtype=torch.int16, device=DEV)
    ref = np.full(lay.buffer_numel, SENTINEL, np.uint16)
    gpu.all_gather_params_mxfp4(plan, got, coords, out)
    MX.all_gather(lay, want, coords, ref)
    assert_bf16(host_u16(out), ref, "gather")
    free()


def test_residual_of_a_block_that_is_not_finite_stays(gpu):
    n = 1000
    rng = np.random.default_rng(0)
    g = bf16_host(rng, n, 1.0)
    g[100], g[300], g[301] = 0x7F80, 0x7FC1, 0xFF80
    res = rng.standard_normal(n).astype(np.float32)
    res[600] = np.inf
    check_quantize(gpu, [n], n, 1, 0, gpu.WORLD, g, res)
    free()


def test_residual_feeds_back_exactly(gpu):
    """values + residual == gradient + the residual before, in fp32."""
    sizes, bucket, D = [5000, 77, 30000], 9000, 4
    lay = OL.build_layout(sizes, bucket, D)
    plan = gpu.build_range_map(sizes, bucket, D, 0)
    rng = np.random.default_rng(4)
    N = plan.buffer_numel
    mx, out = gpu.mx_empty(plan, gpu.WORLD), torch.zeros(N, dtype=torch.bfloat16, device=DEV)
    res = torch.zeros(N, device=DEV)
    inside = torch.zeros(N, dtype=torch.bool, device=DEV)
    for b in lay.buckets:
        inside[b.offset:b.offset + b.numel] = True
    for _ in range(4):
        g = to_dev(bf16_host(rng, N)).view(torch.bfloat16)
        x = g.float() + res
        gpu.quantize_grads_mxfp4(plan, g, gpu.WORLD, mx, residual=res)
        gpu.all_gather_params_mxfp4(plan, [mx] * D, gpu.WORLD, out)
        assert torch.equal((out.float() + res)[inside], x[inside]) and not res[~inside].any()
    free()


# ---- reducing ---------------------------------------------------------------------------------

def sources(gpu, rng, lay, r, D, coords, **kw):
    """D contributions in `coords` and the rank's parts of them as they are."""
    stores = [random_mx(rng, lay, coords, **kw) for _ in range(D)]
    return stores, [dev_mx(s) for s in stores]


@pytest.mark.parametrize("seed", range(14))
def test_reduce_random_layouts(either, seed):
    gpu = either
    pr, sizes, bucket, D = layout_of(300 + seed)
    rng = np.random.default_rng(seed)
    lay = OL.build_layout(sizes, bucket, D)
    N, nb = lay.buffer_numel, len(lay.buckets)
    n = pr.choice([D, D, 1, pr.randint(1, 64)])
    for r in sorted({0, D - 1, pr.randrange(D)}):
        plan = gpu.build_range_map(sizes, bucket, D, r)
        for coords in (gpu.WORLD, gpu.LOCAL):
            stores, dev = sources(gpu, rng, lay, r, n, coords)
            scale = pr.choice([1.0, 1.0 / n, 0.3])
            for oc in (gpu.WORLD, gpu.LOCAL):
                b0 = pr.randrange(nb)
                for buckets in (None, (b0, pr.randint(b0, nb))):
                    size = max(8, N if oc == gpu.WORLD else plan.shard_numel)
                    out = torch.full((size,), SENTINEL, dtype=torch.int16, device=DEV)
                    want = np.full(size, SENTINEL, np.uint16)
                    gpu.reduce_scatter_local_mxfp4(plan, dev, coords, scale, out, oc, buckets=buckets)
                    MX.reduce_scatter(lay, r, stores, coords, scale, want, oc, buckets)
                    assert_bf16(host_u16(out), want, f"n={n} r={r} in={coords} out={oc} {buckets}")
    free()


@pytest.mark.parametrize("n", range(1, 20))
def test_reduce_every_small_count(either, n):
    """Every number of contributions around the kernels' batches, at scales
    far enough apart that the order of the sum shows."""
    gpu = either
    rng = np.random.default_rng(n)
    lay = OL.build_layout([2500], 2500, 1)
    plan = gpu.build_range_map([2500], 2500, 1, 0)
    stores, dev = sources(gpu, rng, lay, 0, n, gpu.LOCAL, lo=100, hi=140)
    out, want = torch.zeros(2500, dtype=torch.int16, device=DEV), np.zeros(2500, np.uint16)
    gpu.reduce_scatter_local_mxfp4(plan, gpu.MxBuffers(dev), gpu.LOCAL, 1.0 / n, out, gpu.LOCAL)
    MX.reduce_scatter(lay, 0, stores, gpu.LOCAL, 1.0 / n, want, gpu.LOCAL)
    assert_bf16(host_u16(out), want, f"n={n}")


def test_values_of_every_code_and_scale(either):
    """One contribution, scale 1: all 256 scales x 16 codes, in bf16; scale 255
    is NaN, 2^127 times 2 and more overflows, 2^-127 times 0.5 is subnormal."""
    gpu = either
    n = 256 * 32
    lay = OL.build_layout([n], n, 1)
    plan = gpu.build_range_map([n], n, 1, 0)
    s = MX.empty(lay, gpu.LOCAL)
    s[0][:256] = np.tile(np.array([x | ((x + 1) & 15) << 4 for x in range(0, 16)], np.uint8), (256, 1))
    s[1][:256] = np.arange(256)
    for D in (1, 2):
        out, want = torch.zeros(n, dtype=torch.int16, device=DEV), np.zeros(n, np.uint16)
        gpu.reduce_scatter_local_mxfp4(plan, [dev_mx(s)] * D, gpu.LOCAL, 1.0, out, gpu.LOCAL)
        MX.reduce_scatter(lay, 0, [s] * D, gpu.LOCAL, 1.0, want, gpu.LOCAL)
        assert_bf16(host_u16(out), want, f"D={D}")
    out = torch.zeros(n, dtype=torch.int16, device=DEV)
    gpu.all_gather_params_mxfp4(plan, [dev_mx(s)], gpu.LOCAL, out)
    MX.all_gather(lay, [s], gpu.LOCAL, want)
    assert_bf16(host_u16(out), want, "gather")


def test_every_pair_of_codes_and_scale(either):
    """All 256 bytes of codes at all 256 scales: their values in fp32 (the
    step's main grad) and in bf16 (the gather)."""
    gpu = either
    n = 256 * 512
    lay = OL.build_layout([n], n, 1)
    plan = gpu.build_range_map([n], n, 1, 0)
    s = MX.empty(lay, gpu.LOCAL)
    s[0][:4096] = np.tile(np.arange(256, dtype=np.uint8), 256).reshape(4096, 16)
    s[1][:4096] = np.repeat(np.arange(256), 16)
    with np.errstate(over="ignore"):
        want = MX.decode(s[0][:4096], s[1][:4096]).reshape(-1).astype(np.float32)
    st = [torch.ones(n, device=DEV) for _ in range(3)]
    g, out = torch.zeros(n, device=DEV), torch.zeros(n, dtype=torch.int16, device=DEV)
    gpu.sharded_adam_step_mxfp4(plan, [dev_mx(s)], gpu.LOCAL, 1.0, *st, main_grad_out=g,
                                **hp_kwargs(W.get("tiny").hp, 1))
    gpu.all_gather_params_mxfp4(plan, [dev_mx(s)], gpu.LOCAL, out)
    assert_f32(host_f32(g), want, "fp32")
    assert np.array_equal(np.signbit(host_f32(g))[~np.isnan(want)], np.signbit(want)[~np.isnan(want)])
    assert_bf16(host_u16(out), ON.narrow(want), "bf16")


@pytest.mark.parametrize("top", ["any", 0, 1, 3, 40, 100, 127, 150, 200, 254])
def test_rounding_of_random_fp32(gpu, top):
    """2^20 fp32 of random bits, by themselves and below one element of a
    block that sets its scale from exponent field `top` (0: its subnormals),
    beside every border between two codes and its neighbours, both signs."""
    n = 1 << 20
    rng = np.random.default_rng(5)
    x = rng.integers(0, 1 << 32, n, dtype=np.uint32).view(np.float32)
    if top != "any":
        y = np.abs(x)
        unit = np.float32(np.ldexp(1.0, max(top, 1) - 127 - 2))   # the block's largest lies in [4, 8) of it
        with np.errstate(invalid="ignore"):
            x = np.where((y < 8 * unit.astype(np.float64)) & np.isfinite(x), x, rng.uniform(-6, 6, n) * unit)
        x = x.astype(np.float32)
        if top == 0:
            x = np.where(np.abs(x) < np.float32(2.0**-126), x, np.float32(0)).astype(np.float32)
        t = np.array([0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.5], np.float64) * unit
        t = t[(t >= 2.0**-149) & (t < (2.0**-126 if top == 0 else np.inf))].astype(np.float32)
        near = np.concatenate([t, np.nextafter(t, np.float32(0)), np.nextafter(t, np.float32(np.inf))])
        if top == 0:
            near = near[near < np.float32(2.0**-126)]
        near = np.concatenate([near, -near])
        at = rng.permutation(n // 32)[:near.size]
        x[32 * at + 1 + rng.integers(0, 31, near.size)] = near
        x[::32] = np.float32(2.0**-127) if top == 0 else 4 * unit
    lay = OL.build_layout([n], n, 1)
    plan = gpu.build_range_map([n], n, 1, 0)
    want, got = MX.empty(lay, MX.LOCAL), gpu.mx_empty(plan, gpu.LOCAL)
    MX.writeback(lay, 0, x, want, MX.LOCAL)
    gpu.writeback_params_mxfp4(plan, to_dev(x), got, gpu.LOCAL)
    assert_mx(got, want, f"top {top}")


@pytest.mark.parametrize("n", [1, 2, 3, 8, 13, 16, 32, 45])
def test_long_reductions(gpu, n):
    """20 M slots in ragged buckets: the forms for long launches, reduction and
    norm, at a fresh order of three storages."""
    sizes, bucket, D = [7_000_001, 65, 4_999_999, 33, 8_000_011], 6_000_000, 1
    lay = OL.build_layout(sizes, bucket, D)
    plan = gpu.build_range_map(sizes, bucket, D, 0)
    gen = torch.Generator(device=DEV).manual_seed(n)
    blocks, L = plan.mx_blocks(gpu.LOCAL), plan.shard_numel
    three = [(torch.randint(0, 256, (blocks, 16), dtype=torch.uint8, device=DEV, generator=gen),
              torch.randint(112, 128, (blocks,), dtype=torch.uint8, device=DEV, generator=gen)) for _ in range(3)]
    order = [(j * j + j // 3) % 3 for j in range(n)]
    out = torch.full((L,), SENTINEL, dtype=torch.int16, device=DEV)
    gpu.reduce_scatter_local_mxfp4(plan, [three[j] for j in order], gpu.LOCAL, 0.3, out, gpu.LOCAL)
    ws = torch.empty(plan.norm_mxfp4_workspace_bytes, dtype=torch.uint8, device=DEV)
    ns = torch.zeros(1, dtype=torch.float64, device=DEV)
    gpu.grad_norm_sq_mxfp4(plan, [three[j] for j in order], gpu.LOCAL, 0.3, ws, ns)
    host, got, total = [host_mx(s) for s in three], host_u16(out), 0.0
    for b, rng in enumerate(MX.ranges(lay, 0)):
        v = [MX._values(s, MX.LOCAL, rng).astype(np.float32) for s in host]
        acc = v[order[0]]
        for j in order[1:]:
            acc = acc + v[j]
        acc = acc * np.float32(0.3)
        s = slice(rng[2], rng[2] + acc.size)
        assert_bf16(got[s], ON.narrow(acc), f"bucket {b}")
        got[s] = SENTINEL
        own = acc[:rng[1] - rng[0].start].astype(np.float64)
        total += float(np.sum(own * own))
    assert (got == SENTINEL).all()
    assert_norm(float(ns), total, plan.owned_numel, "norm")
    free()


@pytest.mark.parametrize("n", [1, 3, 8, 64])
@pytest.mark.parametrize("size", [1, 3000, 32_000, 40_000, 300_000])
def test_norm_of_few_and_many_tiles(either, size, n):
    """On both sides of the lengths at which the norm's form changes; the
    squares of a rank's ranges beside padding and cut tiles."""
    gpu, rng = either, np.random.default_rng(size + n)
    lay = OL.build_layout([size, 77], size, 2)
    for r in range(2):
        plan = gpu.build_range_map([size, 77], size, 2, r)
        store = random_mx(rng, lay, gpu.LOCAL)
        dev = dev_mx(store)
        ws = torch.full((max(16, plan.norm_mxfp4_workspace_bytes),), FILL, dtype=torch.uint8, device=DEV)
        ns = torch.full((1,), -1.0, dtype=torch.float64, device=DEV)
        gpu.grad_norm_sq_mxfp4(plan, [dev] * n, gpu.LOCAL, 0.3, ws, ns)
        assert_norm(float(ns), MX.norm_sq(lay, r, [store] * n, gpu.LOCAL, 0.3), plan.owned_numel, f"r={r}")


@pytest.mark.parametrize("n, tiles", [(1, 63), (1, 64), (1, 65), (8, 63), (8, 64), (8, 65), (9, 56), (9, 57),
                                      (64, 8), (64, 9)])
def test_norm_at_the_change_of_its_form(either, n, tiles):
    """One launch up to 64 tiles and 512 tiles times contributions, two above."""
    gpu, rng = either, np.random.default_rng(64 * n + tiles)
    size = 512 * tiles - 100
    lay = OL.build_layout([size], size, 1)
    plan = gpu.build_range_map([size], size, 1, 0)
    assert plan.mx_blocks(gpu.LOCAL) == 16 * tiles
    store = [random_mx(rng, lay, gpu.LOCAL) for _ in range(2)]
    dev, order = [dev_mx(s) for s in store], [j % 2 for j in range(n)]
    ws = torch.full((max(16, plan.norm_mxfp4_workspace_bytes),), FILL, dtype=torch.uint8, device=DEV)
    ns = torch.full((1,), -1.0, dtype=torch.float64, device=DEV)
    gpu.grad_norm_sq_mxfp4(plan, [dev[j] for j in order], gpu.LOCAL, 0.3, ws, ns)
    assert_norm(float(ns), MX.norm_sq(lay, 0, [store[j] for j in order], gpu.LOCAL, 0.3), size, f"{tiles} tiles")


@pytest.mark.parametrize("n, size", [(1, 10_000_003), (5, 8_388_609), (1, 35_000_003), (8, 34_000_001)])
def test_norm_of_more_tiles_than_waves(gpu, n, size):
    """A tile a wave beyond 16384 tiles, and units beyond 16384 of them: waves
    that take several, every one of whose sums is added, in a workspace of
    the stated size and nothing behind it."""
    plan = gpu.build_range_map([size], size, 1, 0)
    assert plan.norm_mxfp4_workspace_bytes == 8 * 16384
    gen = torch.Generator(device=DEV).manual_seed(n)
    blocks = plan.mx_blocks(gpu.LOCAL)
    two = [(torch.randint(0, 256, (blocks, 16), dtype=torch.uint8, device=DEV, generator=gen),
            torch.randint(112, 128, (blocks,), dtype=torch.uint8, device=DEV, generator=gen)) for _ in range(2)]
    order = [j % 2 for j in range(n)]
    buf = torch.full((8 * 16384 + 4096,), FILL, dtype=torch.uint8, device=DEV)
    ns = torch.full((1,), -1.0, dtype=torch.float64, device=DEV)
    for _ in range(2):
        gpu.grad_norm_sq_mxfp4(plan, [two[j] for j in order], gpu.LOCAL, 0.3, buf[:8 * 16384], ns)
        assert bool((buf[8 * 16384:] == FILL).all())
    v = [MX.decode(*host_mx(s)).reshape(-1)[:size].astype(np.float32) for s in two]
    acc = v[order[0]]
    for j in order[1:]:
        acc = acc + v[j]
    own = (acc * np.float32(0.3)).astype(np.float64)
    assert_norm(float(ns), float(np.sum(own * own)), size, f"n={n}")
    # the last slot alone, and one behind it that is no parameter element
    for c, s in two:
        s.fill_(0)
        c.fill_(0)
    at = (size - 1) // 32
    two[0][0][at, (size - 1) % 32 // 2] = 0x77
    two[0][1][at] = 127
    gpu.grad_norm_sq_mxfp4(plan, [two[j] for j in order], gpu.LOCAL, 1.0, buf[:8 * 16384], ns)
    assert size % 2 == 1 and float(ns) == (6.0 * order.count(0)) ** 2
    free()


@pytest.mark.parametrize("seed", range(6))
def test_norm(either, seed):
    gpu = either
    pr, sizes, bucket, D = layout_of(500 + seed)
    rng = np.random.default_rng(seed)
    lay = OL.build_layout(sizes, bucket, D)
    for r in sorted({0, D - 1}):
        plan = gpu.build_range_map(sizes, bucket, D, r)
        coords = pr.choice([gpu.WORLD, gpu.LOCAL])
        stores, dev = sources(gpu, rng, lay, r, D, coords)
        ws = torch.full((plan.norm_mxfp4_workspace_bytes,), FILL, dtype=torch.uint8, device=DEV)
        got = []
        for _ in range(2):
            ns = torch.full((1,), -1.0, dtype=torch.float64, device=DEV)
            gpu.grad_norm_sq_mxfp4(plan, dev, coords, 1.0 / D, ws, ns)
            got.append(float(ns))
        assert got[0] == got[1]
        assert_norm(got[0], MX.norm_sq(lay, r, stores, coords, 1.0 / D), plan.owned_numel, f"r={r}")
        if plan.owned_numel:
            # one block of scale 255 over an owned element
            rng_ = next(x for x in MX.ranges(lay, r) if x[1] > x[0].start)
            at = (rng_[4] if coords == gpu.WORLD else rng_[5]).start + rng_[3] // 32
            dev[0][1][at] = 255
            gpu.grad_norm_sq_mxfp4(plan, dev, coords, 1.0 / D, ws, ns)
            assert np.isnan(float(ns))
    free()


# ---- the step ------------------------------------------------------------------------------------

def check_step(gpu, sizes, bucket, D, r, stores, dev, coords, scale, hp, t, state, pc=None, mc=None, coeff=None,
               mg=False, buckets=None):
    lay = OL.build_layout(sizes, bucket, D)
    plan = gpu.build_range_map(sizes, bucket, D, r)
    N, Ln = plan.buffer_numel, plan.shard_numel
    st = [to_dev(x) for x in state]
    want = [x.copy() for x in state]
    size = max(8, N if pc == gpu.WORLD else Ln)
    par = None if pc is None else torch.full((size,), SENTINEL, dtype=torch.int16, device=DEV)
    wpar = None if pc is None else np.full(size, SENTINEL, np.uint16)
    mx = None if mc is None else dev_mx(MX.empty(lay, mc, FILL))
    wmx = None if mc is None else MX.empty(lay, mc, FILL)
    g = torch.full((max(8, Ln),), -7.0, device=DEV) if mg else None
    wg = np.full(max(8, Ln), -7.0, np.float32) if mg else None
    cf = None if coeff is None else torch.tensor([coeff], dtype=torch.float32, device=DEV)
    gpu.sharded_adam_step_mxfp4(plan, dev, coords, scale, *st, par, gpu.WORLD if pc is None else pc, param_mx=mx,
                                param_mx_coords=gpu.LOCAL if mc is None else mc, grad_coeff=cf, main_grad_out=g,
                                buckets=buckets, **hp_kwargs(hp, t))
    MX.step(lay, r, stores, coords, scale, *want, ON.hp_array(hp, t), wpar, pc, wmx, mc,
            None if coeff is None else np.float32(coeff), wg, buckets)
    for a, b, n in zip(st, want, ("master", "exp_avg", "exp_avg_sq")):
        assert_f32(host_f32(a), b, f"{n} r={r}")
    if par is not None:
        assert_bf16(host_u16(par), wpar, "parameters")
    if mx is not None:
        assert_mx(mx, wmx, "MXFP4 parameters")
    if mg:
        assert_f32(host_f32(g), wg, "main grad")
    return st, want


@pytest.mark.parametrize("seed", range(20))
def test_step_random_layouts(gpu, seed):
    pr, sizes, bucket, D = layout_of(700 + seed)
    rng = np.random.default_rng(seed)
    lay = OL.build_layout(sizes, bucket, D)
    nb = len(lay.buckets)
    hp = dict(lr=1e-3, beta1=0.9, beta2=pr.choice([0.999, 0.95]), eps=1e-8, weight_decay=pr.choice([0.0, 0.1]))
    n = pr.choice([D, D, 1, pr.randint(1, 64)])
    for r in sorted({0, D - 1, pr.randrange(D)}):
        coords = pr.choice([gpu.WORLD, gpu.LOCAL])
        stores, dev = sources(gpu, rng, lay, r, n, coords)
        b0 = pr.randrange(nb)
        check_step(gpu, sizes, bucket, D, r, stores, dev, coords, pr.choice([1.0 / n, 0.3]), hp, pr.choice([1, 7, 900]),
                   state_of(rng, OL.shard_numel(lay, r)), pc=pr.choice([None, gpu.WORLD, gpu.LOCAL]),
                   mc=pr.choice([None, gpu.WORLD, gpu.LOCAL]), coeff=pr.choice([None, 0.37, 1.0]), mg=pr.random() < 0.5,
                   buckets=pr.choice([None, (b0, pr.randint(b0, nb))]))
    free()


@pytest.mark.parametrize("n", [*range(1, 20), 24, 31, 32, 33, 48, 63, 64])
def test_step_every_small_count(either, n):
    """Every number of contributions around the kernels' fixed counts and
    batches, over ranges of whole tiles beside their cut ends, at scales far
    enough apart that the order of the sum shows; every place of the
    parameters, with and without a coefficient and the main grad."""
    gpu = either
    sizes, bucket, D, r = [9000, 33, 2049], 7000, 2, 1
    lay = OL.build_layout(sizes, bucket, D)
    rng = np.random.default_rng(n)
    st = state_of(rng, OL.shard_numel(lay, r))
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)
    stores = {c: sources(gpu, rng, lay, r, n, c, lo=100, hi=140) for c in (gpu.WORLD, gpu.LOCAL)}
    k = 0
    for pc in (None, gpu.WORLD, gpu.LOCAL):
        for mc in (None, gpu.WORLD, gpu.LOCAL):
            for coeff in (None, 0.37):
                k += 1
                coords = (gpu.WORLD, gpu.LOCAL)[k % 2]
                check_step(gpu, sizes, bucket, D, r, *stores[coords], coords, 1.0 / n, hp, 5, st, pc=pc, mc=mc,
                           coeff=coeff, mg=k % 3 == 0)


def test_the_order_of_the_sum_shows():
    """The contributions of the test above, summed in any other order, or in
    parts, differ from the stated order."""
    lay = OL.build_layout([9000, 33, 2049], 7000, 2)
    for n in (7, 8, 9, 15, 16, 17):
        rng = np.random.default_rng(n)
        stores = [random_mx(rng, lay, MX.LOCAL, lo=100, hi=140) for _ in range(n)]
        v = [MX._values(s, MX.LOCAL, MX.ranges(lay, 1)[0]).astype(np.float32) for s in stores]

        def total(x):
            acc = x[0]
            for y in x[1:]:
                acc = acc + y
            return acc
        want = total(v)
        swapped = v[:n // 2 - 1] + [v[n // 2], v[n // 2 - 1]] + v[n // 2 + 1:]
        for other in (total(v[::-1]), total(swapped), total(v[:n // 2]) + total(v[n // 2:]),
                      total([total(v[0::2]), total(v[1::2])]), total(v[:-1])):
            assert (other != want).any()


@pytest.fixture()
def long_forms(gpu):
    """The build that takes the forms for long launches at any length."""
    with Z.use_library(ZB.GRID_LOOP_LIB):
        yield gpu
        free()


@pytest.mark.parametrize("seed", range(20))
def test_step_random_layouts_in_the_long_forms(long_forms, seed):
    """Random layouts through the step's kernels for long launches: 8 and 16
    contributions have kernels of their own there, other counts one."""
    gpu = long_forms
    pr, sizes, bucket, D = layout_of(1100 + seed)
    sizes = sizes + [pr.randint(3000, 9000)]   # whole tiles in some range
    rng = np.random.default_rng(seed)
    lay = OL.build_layout(sizes, bucket, D)
    nb = len(lay.buckets)
    hp = dict(lr=1e-3, beta1=0.9, beta2=pr.choice([0.999, 0.95]), eps=1e-8, weight_decay=pr.choice([0.0, 0.1]))
    n = (8, 16, 8, 16, pr.randint(1, 64))[seed % 5]
    for r in sorted({0, D - 1, pr.randrange(D)}):
        coords = pr.choice([gpu.WORLD, gpu.LOCAL])
        stores, dev = sources(gpu, rng, lay, r, n, coords, lo=100, hi=140)
        b0 = pr.randrange(nb)
        check_step(gpu, sizes, bucket, D, r, stores, dev, coords, pr.choice([1.0 / n, 0.3]), hp, pr.choice([1, 7, 900]),
                   state_of(rng, OL.shard_numel(lay, r)), pc=pr.choice([None, gpu.WORLD, gpu.LOCAL]),
                   mc=pr.choice([None, gpu.WORLD, gpu.LOCAL]), coeff=pr.choice([None, 0.37, 1.0]), mg=pr.random() < 0.5,
                   buckets=pr.choice([None, (b0, pr.randint(b0, nb))]))


@pytest.mark.parametrize("n", [2, 8, 16])
def test_step_specials_in_the_long_forms(long_forms, n):
    """Any scale byte, 255 among them, and a NaN coefficient, which skips the step."""
    gpu = long_forms
    sizes, bucket, D = [6000, 9], 7000, 2
    lay = OL.build_layout(sizes, bucket, D)
    rng = np.random.default_rng(n)
    hp = W.get("tiny").hp
    stores = [random_mx(rng, lay, gpu.LOCAL, 0, 256) for _ in range(n)]
    dev = [dev_mx(s) for s in stores]
    for r in range(D):
        st = state_of(rng, OL.shard_numel(lay, r))
        k = OL.shard_bases(lay, r)[0][0]
        st[0][k + 700], st[0][k + 1400] = np.inf, np.nan
        check_step(gpu, sizes, bucket, D, r, stores, dev, gpu.LOCAL, 0.5, hp, 2, st, pc=gpu.WORLD, mc=gpu.WORLD, mg=True)
        got, _ = check_step(gpu, sizes, bucket, D, r, stores, dev, gpu.LOCAL, 0.5, hp, 2, st, pc=gpu.LOCAL,
                            mc=gpu.LOCAL, coeff=float("nan"), mg=True)
        for a, b in zip(got, st):
            assert np.array_equal(host_f32(a).view(np.uint32), b.view(np.uint32))


def test_long_steps(gpu):
    """35 M slots in ragged buckets, above the length from which the library
    itself takes the step's forms for long launches; every slot compared."""
    sizes, bucket, D = [9_000_001, 65, 8_999_999, 33, 17_000_011], 10_000_000, 1
    lay = OL.build_layout(sizes, bucket, D)
    plan = gpu.build_range_map(sizes, bucket, D, 0)
    assert plan.mx_blocks(gpu.LOCAL) // 16 > 1 << 16
    rng, hp, Ln = np.random.default_rng(9), W.get("gpt2_small").hp, plan.shard_numel
    host = [random_mx(rng, lay, gpu.LOCAL, lo=108, hi=124) for _ in range(3)]
    dev = [dev_mx(s) for s in host]
    state = state_of(rng, Ln)
    ranges = MX.ranges(lay, 0)
    values = [[MX._values(s, MX.LOCAL, x)[:x[1] - x[0].start].astype(np.float32) for s in host] for x in ranges]
    for n in (3, 8, 16):
        order = [(j * j + j // 3) % 3 for j in range(n)]
        st = [to_dev(x) for x in state]
        par = torch.full((Ln,), SENTINEL, dtype=torch.int16, device=DEV)
        mx = dev_mx(MX.empty(lay, MX.LOCAL, FILL))
        gpu.sharded_adam_step_mxfp4(plan, [dev[j] for j in order], gpu.LOCAL, 0.3, *st, par, gpu.LOCAL, param_mx=mx,
                                    **hp_kwargs(hp, 5))
        got, got_par, got_mx = [host_f32(x) for x in st], host_u16(par), host_mx(mx)
        want_mx, rest = MX.empty(lay, MX.LOCAL, FILL), np.ones(Ln, bool)
        for b, (x, v) in enumerate(zip(ranges, values)):
            acc = v[order[0]]
            for j in order[1:]:
                acc = acc + v[j]
            k = slice(x[2], x[2] + acc.size)
            want = MX.adam(ON.hp_array(hp, 5), acc * np.float32(0.3), *(s[k] for s in state), np.float32)
            for g, w, name in zip(got, want, ("master", "exp_avg", "exp_avg_sq")):
                assert_f32(g[k], w, f"n={n} bucket {b} {name}")
            assert_bf16(got_par[k], ON.narrow(want[0]), f"n={n} bucket {b} parameters")
            MX._put(want_mx, MX.LOCAL, x, want[0])
            rest[k] = False
        assert_mx(mx, want_mx, f"n={n} MXFP4 parameters")
        assert (got_par[rest] == SENTINEL).all()
        for g, s in zip(got, state):
            assert np.array_equal(g[rest].view(np.uint32), s[rest].view(np.uint32))
    free()


def test_step_beyond_32_bits(gpu):
    """8 contributions to 1.1e9 slots (state offsets past 2^32 bytes), the
    last two of three buckets: their heads, middles and tails against the
    oracle, the first bucket as it was."""
    sizes, bucket, D, n = [400_000_007, 400_000_065, 300_004_099], 400_000_000, 1, 8
    lay = OL.build_layout(sizes, bucket, D)
    plan = gpu.build_range_map(sizes, bucket, D, 0)
    Ln, hp = plan.shard_numel, W.get("llama3_8b").hp
    assert 4 * Ln > 1 << 32 and len(lay.buckets) == 3
    gen = torch.Generator(device=DEV).manual_seed(3)
    blocks = plan.mx_blocks(gpu.LOCAL)
    dev = [(torch.randint(0, 256, (blocks, 16), dtype=torch.uint8, device=DEV, generator=gen),
            torch.randint(108, 124, (blocks,), dtype=torch.uint8, device=DEV, generator=gen)) for _ in range(3)]
    order = [(j * j + j // 3) % 3 for j in range(n)]
    st = [torch.randn(Ln, device=DEV, generator=gen) * 0.02, torch.randn(Ln, device=DEV, generator=gen) * 1e-3]
    st.append((torch.randn(Ln, device=DEV, generator=gen) * 1e-3).square_())
    before = [x.clone() for x in st]
    par = torch.full((Ln,), SENTINEL, dtype=torch.int16, device=DEV)
    gpu.sharded_adam_step_mxfp4(plan, [dev[j] for j in order], gpu.LOCAL, 0.25, *st, par, gpu.LOCAL, buckets=(1, 3),
                                **hp_kwargs(hp, 5))
    ranges = MX.ranges(lay, 0)
    head = ranges[1][2]
    for a, b in zip(st, before):
        assert torch.equal(a[:head], b[:head])
    assert bool((par[:head] == SENTINEL).all())
    for x in ranges[1:]:
        size, phase, blk = x[1] - x[0].start, x[3], x[5]
        for lo in (0, size // 2, size - 5000):
            # the blocks over elements [lo, lo + 5000) of the bucket
            b0, b1 = (phase + lo) // 32, (phase + lo + 5000 + 31) // 32
            at = slice(phase + lo - 32 * b0, phase + lo - 32 * b0 + 5000)
            part = slice(blk.start + b0, blk.start + b1)
            v = [MX.decode(c[part].cpu().numpy(), s[part].cpu().numpy()).reshape(-1)[at].astype(np.float32)
                 for c, s in dev]
            acc = v[order[0]]
            for j in order[1:]:
                acc = acc + v[j]
            k = slice(x[2] + lo, x[2] + lo + 5000)
            want = MX.adam(ON.hp_array(hp, 5), acc * np.float32(0.25), *(host_f32(s[k]) for s in before), np.float32)
            for g, w, name in zip(st, want, ("master", "exp_avg", "exp_avg_sq")):
                assert_f32(host_f32(g[k]), w, f"{name} from {lo}")
            assert_bf16(host_u16(par[k]), ON.narrow(want[0]), f"parameters from {lo}")
    free()


def test_step_specials(gpu):
    """Scale 255, sums that overflow, subnormal values, a NaN coefficient that
    skips the step, an Inf master in the MXFP4 output."""
    sizes, bucket, D = [3000, 9], 4000, 2
    lay = OL.build_layout(sizes, bucket, D)
    rng = np.random.default_rng(2)
    hp = W.get("tiny").hp
    stores = [random_mx(rng, lay, gpu.LOCAL, 0, 256) for _ in range(D)]
    dev = [dev_mx(s) for s in stores]
    for r in range(D):
        st = state_of(rng, OL.shard_numel(lay, r))
        k = OL.shard_bases(lay, r)[0][0]
        st[0][k + 40], st[0][k + 100] = np.inf, np.nan
        check_step(gpu, sizes, bucket, D, r, stores, dev, gpu.LOCAL, 0.5, hp, 2, st, pc=gpu.WORLD, mc=gpu.WORLD, mg=True)
        got, _ = check_step(gpu, sizes, bucket, D, r, stores, dev, gpu.LOCAL, 0.5, hp, 2, st, pc=gpu.LOCAL,
                            mc=gpu.LOCAL, coeff=float("nan"), mg=True)
        for a, b in zip(got, st):
            assert np.array_equal(host_f32(a).view(np.uint32), b.view(np.uint32))
    free()


def test_rank_with_only_padding(gpu):
    rng = np.random.default_rng(3)
    sizes, bucket, D = [3, 2], 100, 4
    lay = OL.build_layout(sizes, bucket, D)
    stores, dev = sources(gpu, rng, lay, 3, D, gpu.WORLD)
    st = [np.full(72, 1.5, np.float32) for _ in range(3)]
    check_step(gpu, sizes, bucket, D, 3, stores, dev, gpu.WORLD, 0.25, W.get("tiny").hp, 1, st, pc=gpu.WORLD,
               mc=gpu.WORLD)
    plan = gpu.build_range_map(sizes, bucket, D, 3)
    assert plan.owned_numel == 0
    ws = torch.empty(plan.norm_mxfp4_workspace_bytes, dtype=torch.uint8, device=DEV)
    ns = torch.full((1,), -1.0, dtype=torch.float64, device=DEV)
    gpu.grad_norm_sq_mxfp4(plan, dev, gpu.WORLD, 0.25, ws, ns)
    assert float(ns) == 0.0


def test_per_bucket_calls_equal_the_whole(gpu):
    pr, sizes, bucket, D = layout_of(41, dps=(4,))
    sizes, bucket = sizes + [9000, 77, 5000, 1400, 1500, 1600, 2000, 3000], 1500
    lay = OL.build_layout(sizes, bucket, D)
    rng = np.random.default_rng(1)
    plan = gpu.build_range_map(sizes, bucket, D, 2)
    stores, dev = sources(gpu, rng, lay, 2, D, gpu.WORLD)
    st0 = state_of(rng, plan.shard_numel)
    res = []
    nb = len(lay.buckets)
    assert nb >= 4
    for parts in ([None], [(b, b + 1) for b in reversed(range(nb))],
                  [[(b, b + 1) for b in range(k, nb, 3)] for k in (1, 0, 2)] + [[], [(2, 2)]]):
        st, mx = [to_dev(x) for x in st0], gpu.mx_empty(plan, gpu.LOCAL)
        for b in parts:
            gpu.sharded_adam_step_mxfp4(plan, dev, gpu.WORLD, 0.25, *st, param_mx=mx, buckets=b,
                                        **hp_kwargs(W.get("tiny").hp, 4))
        # the step's MXFP4 parameters are the write-back's of the new master
        wb = gpu.mx_empty(plan, gpu.LOCAL)
        gpu.writeback_params_mxfp4(plan, st[0], wb, gpu.LOCAL)
        assert torch.equal(wb[0], mx[0]) and torch.equal(wb[1], mx[1])
        res.append(st + list(mx))
    for other in res[1:]:
        assert all(torch.equal(a, b) for a, b in zip(res[0], other))
    free()


@pytest.mark.parametrize("coords", [0, 1])
def test_bucket_lists_of_quantize_and_reduce(gpu, coords):
    """Lists of buckets in any order, those that touch and those that do not,
    against the oracle bucket by bucket; what no list names stays."""
    sizes, bucket, D, r = [5000, 77, 9000, 1400, 1500, 1600, 2000, 3000], 1500, 4, 2
    lay = OL.build_layout(sizes, bucket, D)
    plan = gpu.build_range_map(sizes, bucket, D, r)
    rng, nb = np.random.default_rng(8), plan.num_buckets
    n = lay.buffer_numel if coords == gpu.WORLD else plan.shard_numel
    g, res0 = bf16_host(rng, n), (rng.standard_normal(n) * 1e-3).astype(np.float32)
    stores, dev = sources(gpu, rng, lay, r, 3, coords)
    assert nb >= 6
    for lists in ([(4, 6), (0, 1), (1, 2)], [(nb - 1, nb), (2, 2), (1, 3)], [(0, nb)], []):
        want, want_res, got, res = MX.empty(lay, coords, FILL), res0.copy(), dev_mx(MX.empty(lay, coords, FILL)), to_dev(res0)
        wout, out = np.full(n, SENTINEL, np.uint16), torch.full((n,), SENTINEL, dtype=torch.int16, device=DEV)
        for b in lists:
            MX.quantize(lay, r, g, coords, want, want_res, b)
            MX.reduce_scatter(lay, r, stores, coords, 0.3, wout, coords, b)
        gpu.quantize_grads_mxfp4(plan, to_dev(g), coords, got, residual=res, buckets=lists)
        gpu.reduce_scatter_local_mxfp4(plan, dev, coords, 0.3, out, coords, buckets=lists)
        assert_mx(got, want, f"{lists}")
        assert np.array_equal(host_f32(res).view(np.uint32), want_res.view(np.uint32))
        assert_bf16(host_u16(out), wout, f"{lists}")
    free()


# ---- parameters ------------------------------------------------------------------------------------

@pytest.mark.parametrize("coords", [0, 1])
@pytest.mark.parametrize("seed", range(8))
def test_writeback_and_gather_random_layouts(gpu, seed, coords):
    """Every rank's write-back into its own storage (or, in WORLD coordinates,
    one after another into one), then the gather: both against the oracle."""
    pr, sizes, bucket, D = layout_of(900 + seed)
    rng = np.random.default_rng(seed)
    lay = OL.build_layout(sizes, bucket, D)
    N = lay.buffer_numel
    one = coords == gpu.WORLD and seed % 2 == 0
    want, got = [], []
    for r in range(D):
        plan = gpu.build_range_map(sizes, bucket, D, r)
        m = (rng.standard_normal(plan.shard_numel) * 0.02).astype(np.float32)
        if not (one and r):
            want.append(MX.empty(lay, coords, FILL))
            got.append(dev_mx(want[-1]))
        MX.writeback(lay, r, m, want[-1], coords)
        gpu.writeback_params_mxfp4(plan, to_dev(m), got[-1], coords)
        assert_mx(got[-1], want[-1], f"write-back r={r}")
    if one:
        want, got = want * D, got * D
    out = torch.full((N + 8,), SENTINEL, dtype=torch.int16, device=DEV)
    ref = np.full(N + 8, SENTINEL, np.uint16)
    gpu.all_gather_params_mxfp4(plan, got, coords, out)
    MX.all_gather(lay, want, coords, ref)
    assert_bf16(host_u16(out), ref, "gather")
    assert (host_u16(out)[:N] != SENTINEL).all()
    free()


# ---- against 64 bits ----------------------------------------------------------------------------------

def bounds(lay, r, stores, coords, scale, hp, st, b):
    """How far fp32 in the stated order may be from exact values, per owned
    element of bucket b; u = 2^-24 is half a step of fp32, c its state in 64
    bits. Each first-order bound is doubled once for the higher orders.

    sum and scale: each of n - 1 additions and the product is off by at most u
      relative to its result, which is at most S = |scale| sum |x_j|:
      dg <= n u S.
    m' = b1 m + o1 g: two products and a sum: dm <= u (2 |b1 m| + 2 |o1 g|) + o1 dg.
    v' = b2 v + o2 g^2: one more product: dv <= u (2 b2 v + 3 o2 g^2) + 2 o2 |g| dg.
    step: mh = m'/bc1, den = sqrt(v'/bc2) + eps, w = mh/den + wd p,
      p' = p - lr w. den is off by (dv / v' + 4 u) den at most, in all
      d(mh/den) <= dm/(bc1 den) + |mh/den| (dv/v' + 6 u), and the products and
      sums behind it add 3 u (|mh/den| + |wd p|), lr of it, and u |p'|."""
    u = 2.0**-24
    lr, b1, b2, eps, wd, bc1, bc2 = (float(x) for x in hp)
    o1, o2 = float(np.float32(1) - np.float32(hp[1])), float(np.float32(1) - np.float32(hp[2]))
    rng = MX.ranges(lay, r)[b]
    n = rng[1] - rng[0].start
    g = MX.owned_grad(lay, r, stores, coords, scale, b, np.float64)
    S = abs(float(np.float32(scale))) * sum(np.abs(MX._values(s, coords, rng)[:n]) for s in stores)
    dg = len(stores) * u * S
    k = slice(rng[2], rng[2] + n)
    p, m, v = (x[k].astype(np.float64) for x in st)
    m1, v1 = b1 * m + o1 * g, b2 * v + o2 * g * g
    dm = u * (2 * np.abs(b1 * m) + 2 * np.abs(o1 * g)) + o1 * dg
    dv = u * (2 * b2 * v + 3 * o2 * g * g) + 2 * o2 * np.abs(g) * dg
    den = np.sqrt(v1 / bc2) + eps
    q = (m1 / bc1) / den
    dq = dm / (bc1 * den) + np.abs(q) * (dv / v1 + 6 * u)
    p1 = p - lr * (q + wd * p)
    dp = lr * (dq + 3 * u * (np.abs(q) + np.abs(wd * p))) + u * np.abs(p1)
    return k, (p1, m1, v1), (2 * dp, 2 * dm, 2 * dv), g, 2 * dg


@pytest.mark.parametrize("n", [1, 3, 8, 64])
def test_against_64_bits(gpu, n):
    sizes, bucket, D = [9000, 33, 2049, 511], 7000, 4
    lay = OL.build_layout(sizes, bucket, D)
    rng = np.random.default_rng(n)
    hp = ON.hp_array(W.get("gpt2_small").hp, 5)
    tiny = 2.0**-126
    for r in range(D):
        plan = gpu.build_range_map(sizes, bucket, D, r)
        stores, dev = sources(gpu, rng, lay, r, n, gpu.LOCAL, lo=108, hi=118)
        st0 = state_of(rng, plan.shard_numel)
        st = [to_dev(x) for x in st0]
        out = torch.zeros(plan.shard_numel, dtype=torch.bfloat16, device=DEV)
        mg = torch.zeros(plan.shard_numel, device=DEV)
        gpu.reduce_scatter_local_mxfp4(plan, dev, gpu.LOCAL, 0.3, out, gpu.LOCAL)
        gpu.sharded_adam_step_mxfp4(plan, dev, gpu.LOCAL, 0.3, *st, main_grad_out=mg,
                                    **hp_kwargs(W.get("gpt2_small").hp, 5))
        for b in range(len(lay.buckets)):
            k, want, bound, g, dg = bounds(lay, r, stores, gpu.LOCAL, 0.3, hp, st0, b)
            for x, w, e in zip(st, want, bound):
                assert (np.abs(host_f32(x)[k].astype(np.float64) - w) <= e + tiny).all()
            assert (np.abs(host_f32(mg)[k].astype(np.float64) - g) <= dg + tiny).all()
            # one more rounding, to bf16
            red = out.float().cpu().numpy()[k].astype(np.float64)
            assert (np.abs(red - g) <= dg + 2.0**-8 * (np.abs(g) + dg) + tiny).all()
    free()


@pytest.mark.parametrize("sigma", [1e-30, 1e-3, 1.0, 1e30])
def test_quantize_against_64_bits(gpu, sigma):
    """Of a block whose largest magnitude A lies in [4, 8) 2^E, a value x
    moves by at most half the step around it: 2^E/4 for |x| < 2 2^E, 2^E/2
    below 4 2^E, 2^E below 6 2^E, and to 6 2^E above."""
    n = 100_003
    plan = gpu.build_range_map([n], n, 1, 0)
    x = W.normal_bf16(n, sigma, 5, DEV)
    mx, out = gpu.mx_empty(plan, gpu.LOCAL), torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    gpu.quantize_grads_mxfp4(plan, x, gpu.LOCAL, mx)
    gpu.reduce_scatter_local_mxfp4(plan, [mx], gpu.LOCAL, 1.0, out, gpu.LOCAL)
    h = np.zeros((n + 31) // 32 * 32)
    h[:n] = x.double().cpu().numpy()
    q = np.zeros_like(h)
    q[:n] = out.double().cpu().numpy()
    h, q = h.reshape(-1, 32), q.reshape(-1, 32)
    unit = np.ldexp(1.0, np.frexp(np.abs(h).max(axis=1, keepdims=True))[1] - 3)
    y = np.abs(h) / unit
    half = np.where(y < 2, 0.25, np.where(y < 4, 0.5, np.where(y <= 6, 1.0, y - 6)))
    assert (np.abs(q - h) <= half * unit).all()
    free()


# ---- together ------------------------------------------------------------------------------------------

class Loop:
    """D ranks on one device: quantise with residual, exchange, clip by the
    global norm, step, gather; on the GPU and in the oracle."""

    def __init__(self, gpu, sizes, bucket, D, seed=0):
        self.gpu, self.D, self.lay = gpu, D, OL.build_layout(sizes, bucket, D)
        self.N = self.lay.buffer_numel
        self.plans = [gpu.build_range_map(sizes, bucket, D, r) for r in range(D)]
        rng = np.random.default_rng(seed)
        self.state0 = [state_of(rng, p.shard_numel) for p in self.plans]
        self.grads = [bf16_host(rng, self.N, 1e-2) for _ in range(D)]
        self.hp = W.get("tiny").hp

    def device(self):
        gpu, D = self.gpu, self.D
        return dict(grads=[to_dev(g) for g in self.grads], res=[torch.zeros(self.N, device=DEV) for _ in range(D)],
                    con=[gpu.mx_empty(self.plans[0], gpu.WORLD) for _ in range(D)],
                    st=[[to_dev(x) for x in s] for s in self.state0],
                    ws=[torch.empty(p.norm_mxfp4_workspace_bytes, dtype=torch.uint8, device=DEV) for p in self.plans],
                    parts=torch.zeros(D, dtype=torch.float64, device=DEV), coeff=torch.zeros(1, device=DEV),
                    par=[gpu.mx_empty(p, gpu.LOCAL) for p in self.plans],
                    out=torch.full((self.N,), SENTINEL, dtype=torch.int16, device=DEV))

    def run(self, d, t, max_norm):
        gpu, D = self.gpu, self.D
        for j in range(D):
            gpu.quantize_grads_mxfp4(self.plans[j], d["grads"][j], gpu.WORLD, d["con"][j], residual=d["res"][j])
        for r in range(D):
            gpu.grad_norm_sq_mxfp4(self.plans[r], d["con"], gpu.WORLD, 1.0 / D, d["ws"][r], d["parts"][r:r + 1])
        gpu.clip_coefficient(d["parts"], max_norm, d["coeff"])
        for r in range(D):
            gpu.sharded_adam_step_mxfp4(self.plans[r], d["con"], gpu.WORLD, 1.0 / D, *d["st"][r],
                                        param_mx=d["par"][r], grad_coeff=d["coeff"], **hp_kwargs(self.hp, t))
        gpu.all_gather_params_mxfp4(self.plans[0], d["par"], gpu.LOCAL, d["out"])

    def oracle(self):
        return dict(res=[np.zeros(self.N, np.float32) for _ in range(self.D)],
                    con=[MX.empty(self.lay, MX.WORLD) for _ in range(self.D)],
                    st=[[x.copy() for x in s] for s in self.state0],
                    par=[MX.empty(self.lay, MX.LOCAL) for _ in range(self.D)], out=np.zeros(self.N, np.uint16))

    def run_oracle(self, o, t, coeff):
        D = self.D
        for j in range(D):
            MX.quantize(self.lay, j, self.grads[j], MX.WORLD, o["con"][j], o["res"][j])
        parts = [MX.norm_sq(self.lay, r, o["con"], MX.WORLD, 1.0 / D) for r in range(D)]
        for r in range(D):
            MX.step(self.lay, r, o["con"], MX.WORLD, 1.0 / D, *o["st"][r], ON.hp_array(self.hp, t),
                    param_mx=o["par"][r], param_mx_coords=MX.LOCAL, coeff=coeff)
        MX.all_gather(self.lay, o["par"], MX.LOCAL, o["out"])
        return parts


def test_whole_loop(gpu):
    loop = Loop(gpu, [5000, 17, 1, 30000, 2049, 999, 64], 12000, 4)
    d, o = loop.device(), loop.oracle()
    for t in (1, 2, 3):
        loop.run(d, t, 0.05)
        coeff = np.float32(float(d["coeff"]))
        parts = loop.run_oracle(o, t, coeff)
        assert 0 < coeff < 1
        for r in range(loop.D):
            assert_norm(float(d["parts"][r]), parts[r], loop.plans[r].owned_numel, f"norm {r}")
            assert_mx(d["con"][r], o["con"][r], f"contribution {r}")
            assert_mx(d["par"][r], o["par"][r], f"parameters {r}")
            assert np.array_equal(host_f32(d["res"][r]).view(np.uint32), o["res"][r].view(np.uint32))
            for a, b in zip(d["st"][r], o["st"][r]):
                assert_f32(host_f32(a), b, f"state {r}")
        assert_bf16(host_u16(d["out"]), o["out"], f"gathered, step {t}")
    free()


def test_overflow_skips_the_step(gpu):
    """An Inf in one rank's gradients: scale 255, a NaN norm, a NaN
    coefficient, and no rank's state or parameters change."""
    loop = Loop(gpu, [5000, 17, 3000], 4000, 4)
    d = loop.device()
    loop.run(d, 1, 1.0)
    d["grads"][2][1234] = 0x7F80
    before = [x.clone() for s in d["st"] for x in s] + [x.clone() for p in d["par"] for x in p] + [d["out"].clone()]
    loop.run(d, 2, 1.0)
    assert torch.isnan(d["coeff"]).all()
    after = [x for s in d["st"] for x in s] + [x for p in d["par"] for x in p] + [d["out"]]
    assert all(torch.equal(a, b) for a, b in zip(before, after))
    assert all(torch.isfinite(x).all() for x in d["res"])
    free()


def test_overflow_in_the_first_step(gpu):
    """The documented order: the parameters' storage is written once before
    the first step, which is skipped; the gather then gives the parameters as
    they are, and no zeros."""
    loop = Loop(gpu, [5000, 17, 3000], 4000, 4)
    d, o = loop.device(), loop.oracle()
    for r in range(loop.D):
        gpu.writeback_params_mxfp4(loop.plans[r], d["st"][r][0], d["par"][r], gpu.LOCAL)
        MX.writeback(loop.lay, r, loop.state0[r][0], o["par"][r], MX.LOCAL)
    MX.all_gather(loop.lay, o["par"], MX.LOCAL, o["out"])
    d["grads"][1][77] = 0x7F80
    loop.run(d, 1, 1.0)
    assert torch.isnan(d["coeff"]).all() and np.count_nonzero(o["out"] & 0x7FFF) > 7000
    assert_bf16(host_u16(d["out"]), o["out"], "gathered")
    for r in range(loop.D):
        for a, b in zip(d["st"][r], loop.state0[r]):
            assert np.array_equal(host_f32(a).view(np.uint32), b.view(np.uint32))
    free()


def test_two_graphs_replay_as_the_eager_loop(gpu):
    """Two captured loops with buffers of their own, replayed in turn with
    eager work between; every replay equals the eager loop."""
    loop = Loop(gpu, [5000, 17, 1, 30000, 2049, 999, 64], 12000, 4)
    sets = [loop.device() for _ in range(3)]
    graphs = []
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for d in sets[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            with torch.cuda.graph(g, stream=stream):
                loop.run(d, 3, 0.05)
        graphs.append(g)
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    for replay in range(4):
        loop.run(sets[2], 3, 0.05)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        torch.randn(1 << 20, device=DEV).mul_(2.0)
        for d in sets[:2]:
            for k in ("st", "res", "con", "par"):
                for a, b in zip(d[k], sets[2][k]):
                    for x, y in zip(a, b) if k != "res" else [(a, b)]:
                        assert torch.equal(x, y), (replay, k)
            assert torch.equal(d["out"], sets[2]["out"]) and torch.equal(d["parts"], sets[2]["parts"])
    del graphs
    free()


def test_calls_on_another_stream(gpu):
    """The `stream` argument and torch's current stream, two loops at once."""
    loop = Loop(gpu, [50000, 17, 20000], 30000, 4)
    ref, a, b = loop.device(), loop.device(), loop.device()
    loop.run(ref, 2, 0.05)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        loop.run(a, 2, 0.05)
    with torch.cuda.stream(s2):
        loop.run(b, 2, 0.05)
    out = torch.empty(loop.N, dtype=torch.int16, device=DEV)
    s1.wait_stream(torch.cuda.current_stream())
    gpu.all_gather_params_mxfp4(loop.plans[1], a["par"], gpu.LOCAL, out, stream=s1)
    torch.cuda.synchronize()
    for d in (a["out"], b["out"], out):
        assert torch.equal(d, ref["out"])
    for x, y in zip(a["st"] + b["st"], ref["st"] * 2):
        assert all(torch.equal(p, q) for p, q in zip(x, y))
    free()


def test_two_threads(gpu):
    """Two host threads, each with a stream and buffers of its own, on one set
    of plans."""
    import threading
    loop = Loop(gpu, [50000, 17, 20000], 30000, 4)
    ref, sets, errors = loop.device(), [loop.device() for _ in range(2)], []
    for t in range(1, 9):
        loop.run(ref, t, 0.05)
    torch.cuda.synchronize()

    def work(d):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for t in range(1, 9):
                    loop.run(d, t, 0.05)
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(d,)) for d in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for d in sets:
        assert torch.equal(d["out"], ref["out"])
        for x, y in zip(d["st"], ref["st"]):
            assert all(torch.equal(p, q) for p, q in zip(x, y))
    free()


# ---- beyond the first grid, and beyond 32 bits ------------------------------------------------------------

def test_loops_beyond_the_grid(gpu):
    """Every MXFP4 kernel through the build whose launches are capped at 64
    workgroups: the whole loop, against the library's."""
    sizes, bucket, D = [300000, 17, 123456, 2049], 200000, 4
    loop = Loop(gpu, sizes, bucket, D)
    ref = loop.device()
    loop.run(ref, 2, 0.05)
    torch.cuda.synchronize()
    with Z.use_library(ZB.GRID_LOOP_LIB):
        small = Loop(gpu, sizes, bucket, D)
        d = small.device()
        small.run(d, 2, 0.05)
        wb, red = gpu.mx_empty(small.plans[1], gpu.LOCAL), torch.zeros(small.N, dtype=torch.int16, device=DEV)
        gpu.writeback_params_mxfp4(small.plans[1], d["st"][1][0], wb, gpu.LOCAL)
        gpu.reduce_scatter_local_mxfp4(small.plans[1], d["con"], gpu.WORLD, 0.25, red, gpu.WORLD)
        torch.cuda.synchronize()
        for p in small.plans:
            p.destroy()
    assert torch.equal(wb[0], d["par"][1][0]) and torch.equal(wb[1], d["par"][1][1])
    want = np.zeros(loop.N, np.uint16)
    MX.reduce_scatter(loop.lay, 1, [host_mx(c) for c in ref["con"]], MX.WORLD, 0.25, want, MX.WORLD)
    assert_bf16(host_u16(red), want, "reduce-scatter")
    assert torch.equal(d["coeff"], ref["coeff"])   # else the steps below differ
    for k in ("st", "con", "par"):
        for a, b in zip(d[k], ref[k]):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), k
    assert torch.equal(d["out"], ref["out"])
    for r in range(D):   # the waves of the two builds, and so the order of their sums, differ
        assert_norm(float(d["parts"][r]), float(ref["parts"][r]), loop.plans[r].owned_numel, f"norm {r}")
    free()


def test_buffers_beyond_32_bits(gpu):
    """The Llama-3-8B layout in WORLD coordinates: 8.03e9 elements (4.3 GB of
    codes, byte offsets past 2^32). The ranges of the first and the last
    buckets of several ranks are compared with the oracle."""
    w = W.get("llama3_8b")
    lay = OL.build_layout(w.param_numel, w.bucket_numel, w.dp_size)
    plan = gpu.build_range_map(w.param_numel, w.bucket_numel, w.dp_size, 7)
    N, D, nb = plan.buffer_numel, w.dp_size, len(lay.buckets)
    assert N > 1 << 32
    g = W.normal_bf16(N, w.grad_sigma, 77, DEV)
    mx = gpu.mx_empty(plan, gpu.WORLD)
    gpu.quantize_grads_mxfp4(plan, g, gpu.WORLD, mx)
    out = torch.full((N,), SENTINEL, dtype=torch.int16, device=DEV)
    gpu.all_gather_params_mxfp4(plan, [mx] * D, gpu.WORLD, out)
    red = torch.full((N,), SENTINEL, dtype=torch.int16, device=DEV)
    gpu.reduce_scatter_local_mxfp4(plan, [mx] * 2, gpu.WORLD, 0.5, red, gpu.WORLD, buckets=(nb - 2, nb))
    for r in (0, 6, 7):
        ranges = MX.ranges(lay, r)
        for b in (0, nb // 2, nb - 1):
            rng, own, _, phase, blocks, _ = ranges[b]
            x = np.zeros(32 * (blocks.stop - blocks.start), np.float32)
            x[phase:phase + own - rng.start] = g[rng.start:own].float().cpu().numpy()
            want = MX.encode(x.reshape(-1, 32))
            assert_mx([t[blocks] for t in mx], want, f"r={r} bucket {b}")
            vals = MX.decode(*want).reshape(-1)[phase:phase + rng.size].astype(np.float32)
            assert_bf16(host_u16(out[rng.start:rng.end]), ON.narrow(vals), f"gather r={r} bucket {b}")
            if r == 7 and b == nb - 1:
                assert_bf16(host_u16(red[rng.start:rng.end]), ON.narrow(vals), "reduce")
                assert (host_u16(red[rng.start - 8:rng.start]) == SENTINEL).all()
    free()


# ---- refusals ------------------------------------------------------------------------------------------------

def test_refusals(gpu):
    plan = gpu.build_range_map([1000, 28], 600, 2, 1)
    g = torch.zeros(plan.buffer_numel, dtype=torch.bfloat16, device=DEV)
    f = [torch.zeros(plan.shard_numel, device=DEV) for _ in range(3)]
    hp = hp_kwargs(W.get("tiny").hp, 1)
    world, local = gpu.mx_empty(plan, gpu.WORLD), gpu.mx_empty(plan, gpu.LOCAL)
    with pytest.raises(ValueError, match="blocks"):
        gpu.reduce_scatter_local_mxfp4(plan, [local, local], gpu.WORLD, 1.0, g, gpu.WORLD)
    with pytest.raises(ValueError, match="elements"):
        gpu.quantize_grads_mxfp4(plan, g, gpu.WORLD, local)
    with pytest.raises(ValueError, match="elements"):
        gpu.quantize_grads_mxfp4(plan, g[:8], gpu.WORLD, world)
    with pytest.raises(TypeError):
        gpu.quantize_grads_mxfp4(plan, g.float(), gpu.WORLD, world)
    for missing in (None, (world[0],), (world[0], None)):
        with pytest.raises(TypeError):
            gpu.quantize_grads_mxfp4(plan, g, gpu.WORLD, missing)
    with pytest.raises(TypeError):
        gpu.quantize_grads_mxfp4(plan, None, gpu.WORLD, world)
    with pytest.raises(TypeError):
        gpu.sharded_adam_step_mxfp4(plan, [local], gpu.LOCAL, 1.0, f[0], None, f[2], **hp)
    with pytest.raises(ValueError, match="contiguous"):
        gpu.MxBuffers([(world[0].t(), world[1])])
    with pytest.raises(ValueError, match="device"):
        gpu.quantize_grads_mxfp4(plan, g, gpu.WORLD, (world[0].cpu(), world[1]))
    for call, code in (
            (lambda: gpu.reduce_scatter_local_mxfp4(plan, [], gpu.LOCAL, 1.0, g, gpu.WORLD), gpu.EINVAL),
            (lambda: gpu.reduce_scatter_local_mxfp4(plan, [local] * 65, gpu.LOCAL, 1.0, g, gpu.WORLD), gpu.EINVAL),
            (lambda: gpu.quantize_grads_mxfp4(plan, g, gpu.WORLD, world, buckets=(1, 0)), gpu.EINVAL),
            (lambda: gpu.quantize_grads_mxfp4(plan, g, gpu.WORLD, world, buckets=(0, 99)), gpu.EINVAL),
            (lambda: gpu.all_gather_params_mxfp4(plan, [world], gpu.WORLD, g), gpu.EINVAL),
            (lambda: gpu.writeback_params_mxfp4(plan, f[0], (local[0], local[0].view(-1)[16:]), gpu.LOCAL),
             gpu.EALIAS),
            (lambda: gpu.sharded_adam_step_mxfp4(plan, [local], gpu.LOCAL, 1.0, f[0], f[0], f[2], **hp), gpu.EALIAS),
            (lambda: gpu.sharded_adam_step_mxfp4(plan, [local], gpu.LOCAL, 1.0, *f, param_mx=local, **hp),
             gpu.EALIAS),
            (lambda: gpu.sharded_adam_step_mxfp4(plan, [local], gpu.LOCAL, 1.0, *f, **dict(hp, step=0)), gpu.EINVAL)):
        with pytest.raises(gpu.ZdoError) as e:
            call()
        assert e.value.code == code
    torch.cuda.synchronize()


@pytest.mark.parametrize("buckets", [[], [(1, 1)], (1, 1)])
def test_refusals_without_buckets(gpu, buckets):
    """Arguments are checked also where no bucket is asked for, as the bf16
    calls do; a right call then changes nothing."""
    plan = gpu.build_range_map([1000, 28], 600, 2, 1)
    g = torch.full((plan.buffer_numel,), SENTINEL, dtype=torch.int16, device=DEV)
    f = [torch.full((plan.shard_numel,), 1.5, device=DEV) for _ in range(3)]
    hp = hp_kwargs(W.get("tiny").hp, 1)
    local = gpu.mx_empty(plan, gpu.LOCAL)
    for step, given, coords in ((gpu.sharded_adam_step_mxfp4, local, gpu.LOCAL), (gpu.sharded_adam_step, g, gpu.WORLD)):
        for bad, code in ((dict(hp, step=0), gpu.EINVAL), (dict(hp, beta1=1.0), gpu.EINVAL)):
            with pytest.raises(gpu.ZdoError) as e:
                step(plan, [given], coords, 1.0, *f, buckets=buckets, **bad)
            assert e.value.code == code
        with pytest.raises(gpu.ZdoError) as e:
            step(plan, [given], coords, 1.0, f[0], f[0], f[2], buckets=buckets, **hp)
        assert e.value.code == gpu.EALIAS
        with pytest.raises(gpu.ZdoError) as e:
            step(plan, [given] * 65, coords, 1.0, *f, buckets=buckets, **hp)
        assert e.value.code == gpu.EINVAL
    with pytest.raises(gpu.ZdoError) as e:
        gpu.reduce_scatter_local_mxfp4(plan, [], gpu.LOCAL, 1.0, g, gpu.WORLD, buckets=buckets)
    assert e.value.code == gpu.EINVAL
    world = gpu.mx_empty(plan, gpu.WORLD)
    gpu.quantize_grads_mxfp4(plan, g, gpu.WORLD, world, buckets=buckets)
    gpu.reduce_scatter_local_mxfp4(plan, [local], gpu.LOCAL, 1.0, g, gpu.WORLD, buckets=buckets)
    gpu.sharded_adam_step_mxfp4(plan, [local], gpu.LOCAL, 1.0, *f, g, gpu.WORLD, buckets=buckets, **hp)
    torch.cuda.synchronize()
    assert bool((g == SENTINEL).all()) and not world[0].any() and all(bool((x == 1.5).all()) for x in f)
