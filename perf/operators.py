"""The microscaled 4-bit (MXFP4) operators of the sharded optimizer step, as
cases to be measured and compared.

A contribution, or a rank's updated parameters, held in 4 bits: blocks of 32
consecutive elements share one power-of-two scale (E8M0, one byte, bias 127,
255 = NaN); each element is an E2M1 number (sign, two exponent bits, one
mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte, the even element in
the low half. Storage follows the optimizer's layout: rank r's range of bucket
b has T_b = (S_b + 574) // 512 tiles of 16 blocks, starting at the range's
first WORLD element rounded down to 64; slots of those blocks outside the
range's parameter elements hold zero. LOCAL storage holds one rank's tiles,
bucket after bucket; WORLD storage holds, bucket after bucket, every rank's.

Operators (`op` of a case):
  quantize  a bf16 gradient buffer (plus a residual kept from the last step,
            if the case has one) to MXFP4, and its values back in bf16
  reduce    the D contributions' values added in fp32 in rank order, times
            `scale`, rounded to bf16, over the rank's ranges
  step      the same sum as the fp32 main grad (times the clipping
            coefficient, where the case clips by the global norm), Adam on the
            rank's fp32 shard, and the updated parameters in bf16 or in MXFP4
  params    the rank's fp32 master shard to MXFP4, and the all-gather of the D
            ranks' MXFP4 parameters into a whole bf16 buffer
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=7)
MAX_NORM = 1.0


# ---- cases ------------------------------------------------------------------------------

def listed():
    # model: a parameter list of that shape; else `numel` elements in `params`
    # tensors of uneven sizes. coords: where the gradients or contributions
    # live (world: whole buffers; local: one rank's slices, as a rank receives
    # them from its peers).
    return [
        # a smoke-sized step: nothing but latency
        dict(name="step, 1000 elements", op="step", model="", numel=1000, params=6, bucket=1000, dp=4, rank=1,
             coords="world", clip=False, to="bf16"),
        # the everyday step of a small model on one 8-GPU node
        dict(name="step, GPT-2 small rank", op="step", model="gpt2_small", numel=124439808, params=148,
             bucket=40000000, dp=8, rank=1, coords="local", clip=False, to="bf16"),
        # many small tensors in many buckets, clipped by the global norm
        dict(name="step, fragmented, clipped", op="step", model="", numel=77000003, params=20064, bucket=4000000,
             dp=16, rank=3, coords="world", clip=True, to="bf16"),
        # the widest reduction, off every alignment, parameters leaving in 4 bits
        dict(name="step, 64 ranks, to MXFP4", op="step", model="", numel=640000321, params=331, bucket=90000000,
             dp=64, rank=63, coords="local", clip=True, to="mxfp4"),
        # a billion elements a rank
        dict(name="step, Llama-3-8B rank", op="step", model="llama3_8b", numel=8030261248, params=291,
             bucket=100000000, dp=8, rank=1, coords="local", clip=False, to="bf16"),
        # a small odd bucket as soon as its gradients are ready
        dict(name="reduce, one odd bucket", op="reduce", model="", numel=100003, params=5, bucket=100003, dp=3,
             rank=2, coords="world"),
        # 32 ranks' contributions to one rank's quarter of a billion elements
        dict(name="reduce, Llama-3-8B, 32 ranks", op="reduce", model="llama3_8b", numel=8030261248, params=291,
             bucket=200000000, dp=32, rank=5, coords="local"),
        # a whole contribution with the error of the last step fed back
        dict(name="quantize, GPT-2 small, residual", op="quantize", model="gpt2_small", numel=124439808, params=148,
             bucket=40000000, dp=8, rank=0, coords="world", residual=True),
        # a billion-element contribution, ragged, as it is
        dict(name="quantize, 1e9 elements", op="quantize", model="", numel=1000000007, params=900, bucket=100000000,
             dp=16, rank=0, coords="world", residual=False),
        # the smallest gather
        dict(name="params, 20001 elements", op="params", model="", numel=20001, params=9, bucket=8000, dp=4, rank=2,
             coords="world"),
        # every step of a small model
        dict(name="params, GPT-2 small", op="params", model="gpt2_small", numel=124439808, params=148,
             bucket=40000000, dp=8, rank=7, coords="local"),
        # a billion parameters gathered
        dict(name="params, 1e9 elements", op="params", model="", numel=1000000007, params=900, bucket=100000000,
             dp=8, rank=3, coords="local"),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["step", "step", "reduce", "quantize", "params"])
    dp = rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 24, 32, 48, 64])
    if op in ("step", "reduce"):
        coords = rng.choice(["local", "local", "world"])
        # per rank up to 2e8 elements; a world case holds every rank's ranges
        # of every contribution, so its whole buffer stays below 1e8
        shard = log(400, 2e8 if coords == "local" else 1e8 / dp)
        numel = shard * dp + rng.randrange(dp)
        if shard * dp > 4_000_000_000:
            numel = 4_000_000_000 // dp * dp + rng.randrange(dp)
    else:
        coords = rng.choice(["local", "world"])
        numel = log(2000, 8e8)
    params = min(log(1, 3000), max(1, numel // 8))
    case = dict(op=op, model="", numel=numel, params=params, bucket=max(1, numel // rng.choice([1, 2, 5, 11, 30])),
                dp=dp, rank=rng.randrange(dp), coords=coords)
    if op == "step":
        case.update(clip=rng.random() < 0.4, to=rng.choice(["bf16", "bf16", "mxfp4"]))
    if op == "quantize":
        case.update(residual=rng.random() < 0.5)
    return case


# ---- the optimizer's layout: buckets, ranges, blocks -----------------------------------------

def sizes_of(case):
    if case["model"] == "gpt2_small":
        h, sizes = 768, [50257 * 768, 1024 * 768]
        for _ in range(12):
            sizes += [h, h, 3 * h * h, 3 * h, h * h, h, h, h, 4 * h * h, 4 * h, 4 * h * h, h]
        return sizes + [h, h]
    if case["model"] == "llama3_8b":
        h, kv, f, sizes = 4096, 1024, 14336, [128256 * 4096]
        for _ in range(32):
            sizes += [h, h * h, h * kv, h * kv, h * h, h, h * f, h * f, f * h]
        return sizes + [h, 128256 * h]
    # uneven sizes that add up to numel, each at least 1
    n, k = case["numel"], case["params"]
    w = np.exp(np.random.Generator(np.random.PCG64(1000003 * k + n % 999983)).normal(0.0, 1.5, k))
    cut = np.floor(np.cumsum(w) / w.sum() * (n - k)).astype(np.int64)
    cut[-1] = n - k
    return [int(x) + 1 for x in np.diff(np.concatenate([[0], cut]))]


class Layout:
    """Buckets as (offset, numel, range length S, tiles T, first LOCAL tile),
    and the LOCAL base of the rank's range of each."""

    def __init__(self, case):
        self.dp, self.rank, self.sizes = case["dp"], case["rank"], sizes_of(case)
        self.buckets, self.base = [], []
        off = fill = tile = end = 0
        for i, n in enumerate(self.sizes):
            fill += n
            if fill >= case["bucket"] or i == len(self.sizes) - 1:
                s = -(-fill // self.dp)
                t = (s + 574) // 512
                rs = off + self.rank * s
                self.base.append(end + (rs - end) % 64)
                end = self.base[-1] + s
                self.buckets.append((off, fill, s, t, tile))
                off, tile, fill = off + s * self.dp, tile + t, 0
        self.N, self.L, self.tiles = off, end, tile
        self.owned = sum(max(0, min(o + n - (o + self.rank * s), s)) for o, n, s, _, _ in self.buckets)
        # buffers end on a whole block row
        self.rows_w = max((o + (self.dp - 1) * s) // 64 * 2 + 16 * t for o, _, s, t, _ in self.buckets)
        self.rows_l = max(b // 64 * 2 + 16 * t for b, (_, _, _, t, _) in zip(self.base, self.buckets))

    def blocks(self, coords):
        return 16 * self.tiles * (self.dp if coords == "world" else 1)

    def rows(self, coords):
        return self.rows_w if coords == "world" else self.rows_l

    def table(self, space, every):
        """For each block of the rank's ranges, or of every rank's: the 32-slot
        row of the buffer it lies in (space: the buffer's coordinates), its
        slots [lo, hi) that are parameter elements and [lo, end) that are of
        the range, its block in WORLD and in LOCAL storage, and its rank."""
        cols = [[] for _ in range(7)]
        for (o, n, s, t, t0), base in zip(self.buckets, self.base):
            for r in range(self.dp) if every else [self.rank]:
                rs = o + r * s
                i = np.arange(16 * t, dtype=np.int64)
                first = rs // 64 * 64 + 32 * i
                row = (rs // 64 * 2 if space == "world" else base // 64 * 2) + i
                for c, v in zip(cols, (row, rs - first, min(rs + s, o + n) - first, rs + s - first,
                                       16 * (self.dp * t0 + r * t) + i, 16 * t0 + i, np.full_like(i, r))):
                    c.append(v)
        row, lo, hi, end, world, local, rank = (torch.from_numpy(np.concatenate(c)).to(DEV) for c in cols)
        small = [x.clamp(0, 32).to(torch.int32) for x in (lo, hi, end)]
        return dict(row=row, lo=small[0], hi=small[1], end=small[2], world=world, local=local, rank=rank)


def inside(t, end="hi"):
    i = torch.arange(32, dtype=torch.int32, device=DEV)
    return (i >= t["lo"][:, None]) & (i < t[end][:, None])


# ---- the plain form ------------------------------------------------------------------------

def encode(x):
    """Blocks [B, 32] of fp32 to codes [B, 16], scales [B] and the values they
    stand for."""
    top = x.abs().amax(dim=1)
    byte = ((top.view(torch.int32) >> 23) - 2).clamp(min=0)
    bad = ~torch.isfinite(top)
    y = x.abs() * ((254 - byte) << 23).view(torch.float32)[:, None]
    code = (y > 0.25).to(torch.uint8)
    # one up for each border passed; a tie goes to the even code
    code += (y >= 0.75)
    code += (y > 1.25)
    code += (y >= 1.75)
    code += (y > 2.5)
    code += (y >= 3.5)
    code += (y > 5.0)
    code += torch.signbit(x).to(torch.uint8) * 8
    code = torch.where(bad[:, None], torch.zeros_like(code), code)
    byte = torch.where(bad, torch.full_like(byte, 255), byte).to(torch.uint8)
    pair = code.view(-1, 16, 2)
    return pair[..., 0] | (pair[..., 1] << 4), byte


def decode(codes, scales):
    """Codes [..., 16] and scales [...] to fp32 values [..., 32]."""
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                       device=DEV)
    code = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    e = scales.to(torch.int32)
    # 2^-127 is a subnormal of fp32
    factor = torch.where(e == 0, torch.full_like(e, 0x00400000), e << 23).view(torch.float32)
    factor = torch.where(e == 255, torch.full_like(factor, math.nan), factor)
    return lut[code.to(torch.int32)] * factor[..., None]


def total(state):
    """The contributions' sum over the rank's blocks, [B, 32] in fp32: at most
    2^28 values are decoded at a time."""
    codes, scales, t = state["codes"], state["scales"], state["table"]
    if state["coords"] == "world":
        codes, scales = codes[:, t["world"]], scales[:, t["world"]]
    d, b = codes.shape[:2]
    per = max(1, 2**28 // (32 * b))
    acc = decode(codes[:per], scales[:per, :b]).sum(dim=0)
    for j in range(per, d, per):
        acc = acc + decode(codes[j:j + per], scales[j:j + per, :b]).sum(dim=0)
    return acc


def placed(rows, t, values, keep):
    """Block values to buffer order (rows of 32 slots); slots outside the mask are 0."""
    return torch.zeros(rows, 32, device=DEV).index_add_(0, t["row"], torch.where(keep, values, 0.0))


def plain(state):
    case, t, op = state["case"], state["table"], state["case"]["op"]
    if op == "quantize":
        mask = inside(t)
        x = state["grad"].view(-1, 32)[t["row"]].float()
        if state["residual"] is not None:
            x = x + state["residual"].view(-1, 32)[t["row"]]
        x = torch.where(mask, x, 0.0)
        codes, scales = encode(x)
        state["mx"][0].copy_(codes)
        state["mx"][1].copy_(scales)
        value = decode(codes, scales)
        out = {"values": placed(state["rows"], t, value, mask).to(torch.bfloat16).view(-1)}
        if state["residual"] is not None:
            # the residual of what is no parameter element stays; so does that of a block that is not finite
            r = state["residual"].view(-1, 32)
            live = placed(state["rows"], t, 1.0, mask & (scales != 255)[:, None])
            r.copy_(torch.where(live > 0, placed(state["rows"], t, x - value, mask), r))
            out["residual"] = state["residual"]
        return out
    if op == "reduce":
        v = total(state) * state["scale"]
        return placed(state["rows"], t, v, inside(t, "end")).to(torch.bfloat16).view(-1)
    if op == "step":
        mask, g = inside(t), total(state) * state["scale"]
        if case["clip"]:
            sq = torch.where(mask, g, 0.0).double().square().sum()
            state["parts"][case["rank"]] = sq
            norm = state["parts"].sum().sqrt()
            coeff = torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)
            g = g * coeff.float()
        rows = state["rows"]
        live = placed(rows, t, 1.0, mask).view(-1) > 0
        g = placed(rows, t, g, mask).view(-1)
        p, m, v, k = state["master"], state["m"], state["v"], state["const"]
        mn = k["b1"] * m + k["omb1"] * g
        vn = k["b2"] * v + k["omb2"] * (g * g)
        u = (mn / k["bc1"]) / ((vn / k["bc2"]).sqrt() + k["eps"])
        pn = p - k["lr"] * (u + k["wd"] * p)
        for old, new in ((p, pn), (m, mn), (v, vn)):
            old.copy_(torch.where(live, new, old))
        out = {"master": p, "m": m, "v": v}
        if case["clip"]:
            out["norm"] = norm.view(1)
        if case["to"] == "mxfp4":
            codes, scales = encode(torch.where(mask, p.view(-1, 32)[t["row"]], 0.0))
            state["mx"][0].copy_(codes)
            state["mx"][1].copy_(scales)
            out["params"] = placed(rows, t, decode(codes, scales), mask).to(torch.bfloat16).view(-1)
        else:
            out["params"] = torch.where(live, p, 0.0).to(torch.bfloat16)
        return out
    # params
    mine = state["mine"]
    codes, scales = encode(torch.where(inside(mine), state["master"].view(-1, 32)[mine["row"]], 0.0))
    at = mine["world"] if state["coords"] == "world" else mine["local"]
    state["codes"][case["rank"]].index_copy_(0, at, codes)
    state["scales"][case["rank"]].index_copy_(0, at, scales)
    block = t["world"] if state["coords"] == "world" else t["local"]
    value = decode(state["codes"][t["rank"], block], state["scales"][t["rank"], block])
    return placed(state["rows"], t, value, inside(t, "end")).to(torch.bfloat16).view(-1)


# ---- inputs --------------------------------------------------------------------------------

def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device=DEV)


def _spread(b, gen):
    """One standard deviation a block of 32, near its neighbours' (a tensor's
    gradients share their order of magnitude), and 1 block in 20 at zero, as
    rows of an embedding that no token touched."""
    group = torch.exp(0.8 * torch.randn(b // 64 + 1, generator=gen, device=DEV)).repeat_interleave(64)[:b]
    return 1e-3 * group * (torch.rand(b, generator=gen, device=DEV) >= 0.05)


def prepare(case, seed):
    lay, coords, op = Layout(case), case["coords"], case["op"]
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + case["numel"] % 104729)
    s = dict(case=case, coords=coords, rows=lay.rows(coords), scale=1.0 / case["dp"])
    nb = lay.blocks(coords)
    pad = (nb + 15) // 16 * 16
    if op == "quantize":
        s["table"] = lay.table(coords, every=coords == "world")
        spread = _spread(s["rows"], gen)
        s["grad"] = (_normal((s["rows"], 32), gen) * spread[:, None]).to(torch.bfloat16).view(-1)
        s["residual"] = None
        if case["residual"]:
            s["residual"] = (_normal((s["rows"], 32), gen) * (0.1 * spread)[:, None]).view(-1)
        s["mx"] = (torch.zeros(nb, 16, dtype=torch.uint8, device=DEV), torch.zeros(nb, dtype=torch.uint8, device=DEV))
        s["out"] = torch.zeros(32 * s["rows"], dtype=torch.bfloat16, device=DEV)
    else:
        # D buffers in MXFP4: contributions, or the ranks' parameters
        s["codes"] = torch.zeros(case["dp"], nb, 16, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.zeros(case["dp"], pad, dtype=torch.uint8, device=DEV)
        here = lay.table("local", every=False)
        t = lay.table("world", every=True) if coords == "world" or op == "params" else here
        mask = inside(t) if coords == "world" else inside(here)
        spread = _spread(nb, gen)[:, None]
        for j in range(case["dp"]):
            if op == "params":
                x = 0.02 * _normal((nb, 32), gen)
            else:
                x = (_normal((nb, 32), gen) * spread).to(torch.bfloat16).float()
            # other ranks' ranges end at other places: their own slots are all kept here
            x = x if op == "params" and coords == "local" and j != case["rank"] else torch.where(mask, x, 0.0)
            s["codes"][j], s["scales"][j, :nb] = encode(x)
        del mask, spread, x
        if op == "params":
            s["mine"], s["table"], s["rows"] = here, t, lay.rows("world")
        else:
            s["table"] = here if op == "step" or coords == "local" else lay.table("world", every=False)
            s["rows"] = lay.rows("local") if op == "step" else s["rows"]
        n_l, n_out = 32 * lay.rows("local"), 32 * s["rows"]
        if op in ("step", "params"):
            s["master"] = 0.02 * _normal(n_l, gen)
        if op == "step":
            s["m"], s["v"] = 1e-4 * _normal(n_l, gen), (3e-4 * _normal(n_l, gen)).square_()
            f = np.float32
            const = dict(lr=f(HP["lr"]), b1=f(HP["beta1"]), b2=f(HP["beta2"]), omb1=f(1) - f(HP["beta1"]),
                         omb2=f(1) - f(HP["beta2"]), eps=f(HP["eps"]), wd=f(HP["weight_decay"]),
                         bc1=f(1.0 - math.prod([float(f(HP["beta1"]))] * HP["step"])),
                         bc2=f(1.0 - math.prod([float(f(HP["beta2"]))] * HP["step"])))
            s["const"] = {k: torch.tensor(float(v), device=DEV) for k, v in const.items()}
            # the other ranks' squared norms
            s["parts"] = lay.owned * 1e-6 / case["dp"] * (
                1 + torch.rand(case["dp"], generator=gen, device=DEV, dtype=torch.float64))
            s["mx"] = (torch.zeros(lay.blocks("local"), 16, dtype=torch.uint8, device=DEV),
                       torch.zeros(lay.blocks("local"), dtype=torch.uint8, device=DEV))
        s["out"] = torch.zeros(n_out, dtype=torch.bfloat16, device=DEV)
    if own:
        import zero_distributed_optimizer_amd as zdo
        s["plan"] = zdo.build_range_map(lay.sizes, case["bucket"], case["dp"], case["rank"])
        if op != "quantize":
            s["list"] = zdo.MxBuffers([(c, x[:nb]) for c, x in zip(s["codes"], s["scales"])])
        if op == "step":
            s["workspace"] = torch.empty(s["plan"].norm_mxfp4_workspace_bytes, dtype=torch.uint8, device=DEV)
            s["coeff"] = torch.empty(1, device=DEV)
            s["norm"] = torch.empty(1, dtype=torch.float64, device=DEV)
    return s


def run(state):
    if not own:
        return plain(state)
    import zero_distributed_optimizer_amd as zdo
    case, plan = state["case"], state["plan"]
    where = zdo.WORLD if state["coords"] == "world" else zdo.LOCAL
    if case["op"] == "quantize":
        mx, out = state["mx"], state["out"]
        zdo.quantize_grads_mxfp4(plan, state["grad"], where, mx, residual=state["residual"])
        if where == zdo.WORLD:
            zdo.all_gather_params_mxfp4(plan, [mx] * case["dp"], zdo.WORLD, out)
        else:
            zdo.reduce_scatter_local_mxfp4(plan, [mx], zdo.LOCAL, 1.0, out, zdo.LOCAL)
        return {"values": out} if state["residual"] is None else {"values": out, "residual": state["residual"]}
    if case["op"] == "reduce":
        zdo.reduce_scatter_local_mxfp4(plan, state["list"], where, state["scale"], state["out"], where)
        return state["out"]
    if case["op"] == "step":
        r, to_mx, out = case["rank"], case["to"] == "mxfp4", state["out"]
        coeff = None
        if case["clip"]:
            zdo.grad_norm_sq_mxfp4(plan, state["list"], where, state["scale"], state["workspace"],
                                   state["parts"][r:r + 1])
            zdo.clip_coefficient(state["parts"], MAX_NORM, state["coeff"], state["norm"])
            coeff = state["coeff"]
        zdo.sharded_adam_step_mxfp4(plan, state["list"], where, state["scale"], state["master"], state["m"],
                                    state["v"], None if to_mx else out, zdo.LOCAL,
                                    param_mx=state["mx"] if to_mx else None, param_mx_coords=zdo.LOCAL,
                                    grad_coeff=coeff, **HP)
        if to_mx:
            zdo.reduce_scatter_local_mxfp4(plan, [state["mx"]], zdo.LOCAL, 1.0, out, zdo.LOCAL)
        res = {"master": state["master"], "m": state["m"], "v": state["v"], "params": out}
        return dict(res, norm=state["norm"]) if case["clip"] else res
    zdo.writeback_params_mxfp4(plan, state["master"], state["list"][case["rank"]], where)
    zdo.all_gather_params_mxfp4(plan, state["list"], where, state["out"])
    return state["out"]


def work(case):
    lay = Layout(case)
    d, e, mx = case["dp"], lay.owned, 17.0 / 32.0
    n = sum(lay.sizes)
    if case["op"] == "quantize":
        k = n if case["coords"] == "world" else e
        b = k * (2 + mx + (8 if case["residual"] else 0)) + k * (mx + 2)
        return {"bytes": b, "flops": 4 * k}
    if case["op"] == "reduce":
        return {"bytes": e * (d * mx + 2), "flops": 2 * d * e}
    if case["op"] == "step":
        b = e * (d * mx + 24 + (2 if case["to"] == "bf16" else 2 * mx + 2))
        return {"bytes": b, "flops": e * (2 * d + 16)}
    return {"bytes": e * (4 + mx) + n * (mx + 2), "flops": 2 * n}


# ---- the definition in 64 bits ----------------------------------------------------------------

def _power64(e):
    """2^e in fp64, by its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round64(x):
    """Blocks [B, 32] in fp64 to the values that MXFP4 keeps of them."""
    top = x.abs().amax(dim=1, keepdim=True)
    fine = torch.isfinite(top)
    e = (torch.frexp(torch.where(fine, top, torch.ones_like(top))).exponent - 3).clamp(-127, 127)
    e = torch.where(top == 0, torch.full_like(e, -127), e)
    unit = _power64(e)
    y = x.abs() / unit
    step = 0.5 + 0.5 * (y >= 2) + 1.0 * (y >= 4)
    q = (torch.round(y / step) * step).clamp(max=6.0)
    return torch.where(fine, torch.sign(x) * q * unit, torch.full_like(x, math.nan))


def _value64(codes, scales):
    c = torch.stack([codes % 16, codes // 16], dim=-1).flatten(-2).double()
    sign, c = 1 - 2 * (c >= 8).double(), c % 8
    e, m = torch.div(c, 2, rounding_mode="floor"), c % 2
    q = torch.where(e == 0, m / 2, (1 + m / 2) * _power64(e - 1))
    unit = _power64(scales.to(torch.int64) - 127)
    return sign * q * torch.where(scales == 255, torch.full_like(unit, math.nan), unit)[..., None]


def exact(case, seed):
    if case["numel"] // (1 if case["coords"] == "world" else case["dp"]) * case["dp"] > 3e10:
        return None
    s, lay, op = prepare(case, seed), Layout(case), case["op"]
    r, world = case["rank"], case["coords"] == "world"

    def pieces(j, b):
        """Bucket b, rank j: parameter elements [rs, own) and range end in
        WORLD, the LOCAL slot of rs, and storage blocks in both coordinates."""
        o, n, size, t, t0 = lay.buckets[b]
        rs = o + j * size
        return (rs, max(rs, min(rs + size, o + n)), rs + size, lay.base[b],
                slice(16 * (lay.dp * t0 + j * t), 16 * (lay.dp * t0 + (j + 1) * t)), slice(16 * t0, 16 * (t0 + t)))

    def summed(b):
        rs, own_end, end, base, wb, lb = pieces(r, b)
        at, g = wb if world else lb, 0.0
        for j in range(lay.dp):
            g = g + _value64(s["codes"][j, at], s["scales"][j, at])
        a = rs % 64
        return g.view(-1)[a:a + end - rs] / case["dp"]

    def rounded(x, rs):
        """A run of fp64 values that begins at WORLD index rs, as MXFP4 keeps it."""
        a = rs % 64
        y = torch.zeros((a + x.numel() + 31) // 32 * 32, dtype=torch.float64, device=DEV)
        y[a:a + x.numel()] = x
        return _round64(y.view(-1, 32)).view(-1)[a:a + x.numel()]

    out = torch.zeros_like(s["out"], dtype=torch.float64)
    if op == "quantize":
        res = None if s["residual"] is None else s["residual"].double()
        for b in range(len(lay.buckets)):
            for j in range(lay.dp) if world else [r]:
                rs, own_end, _, base, _, _ = pieces(j, b)
                k = slice(rs, own_end) if world else slice(base, base + own_end - rs)
                x = s["grad"][k].double()
                if res is not None:
                    x = x + res[k]
                out[k] = rounded(x, rs)
                if res is not None:
                    res[k] = x - out[k]
        return {"values": out} if res is None else {"values": out, "residual": res}
    if op == "reduce":
        for b in range(len(lay.buckets)):
            rs, _, end, base, _, _ = pieces(r, b)
            out[slice(rs, end) if world else slice(base, base + end - rs)] = summed(b)
        return out
    if op == "step":
        parts, grads = s["parts"].clone(), []
        for b in range(len(lay.buckets)):
            rs, own_end, _, _, _, _ = pieces(r, b)
            grads.append(summed(b)[:own_end - rs])
        coeff = 1.0
        if case["clip"]:
            parts[r] = sum(g.square().sum() for g in grads)
            norm = parts.sum().sqrt()
            coeff = torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)
        k = {n: v.double() for n, v in s["const"].items()}
        p, m, v = (s[n].double() for n in ("master", "m", "v"))
        for b, g in enumerate(grads):
            rs, own_end, _, base, _, _ = pieces(r, b)
            at = slice(base, base + own_end - rs)
            g = g * coeff
            m[at] = k["b1"] * m[at] + k["omb1"] * g
            v[at] = k["b2"] * v[at] + k["omb2"] * g.square()
            u = (m[at] / k["bc1"]) / (torch.sqrt(v[at] / k["bc2"]) + k["eps"])
            p[at] = p[at] - k["lr"] * (u + k["wd"] * p[at])
            out[at] = rounded(p[at], rs) if case["to"] == "mxfp4" else p[at]
        res = {"master": p, "m": m, "v": v, "params": out}
        return dict(res, norm=norm.view(1)) if case["clip"] else res
    for b in range(len(lay.buckets)):
        for j in range(lay.dp):
            rs, own_end, end, base, wb, lb = pieces(j, b)
            at, a = wb if world else lb, rs % 64
            out[rs:end] = _value64(s["codes"][j, at], s["scales"][j, at]).view(-1)[a:a + end - rs]
            if j == r:
                out[own_end:end] = 0.0
                out[rs:own_end] = rounded(s["master"][base:base + own_end - rs].double(), rs)
    return out
