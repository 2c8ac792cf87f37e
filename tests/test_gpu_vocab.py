"""GPU tests of the calls at the vocabulary matrix (include/zdo_vocab.h) against
their formulas in 64 bits. Every tolerance is the sum of the roundings that the
call makes, derived where it is formed:

  - a rounding to bf16 is off by at most U16 = 2^-8 of the value, one to fp32 by
    U32 = 2^-24;
  - a sum of k terms in fp32, in whatever order, by at most k * U32 * (the sum
    of the terms' sizes); the matrix instructions' inner additions need not
    round to nearest, so a product's sum counts 2 * U32 a term;
  - exp(x) by at most 2^-22 + |x| 2^-23 relative (the product with log2(e) is
    rounded, so the exponent is off by |x| U32 or less, and the instruction by
    one unit in the last place).
"""

import numpy as np
import pytest
import torch

import zero_distributed_optimizer_amd as Z
from zero_distributed_optimizer_amd import build as ZB

pytestmark = pytest.mark.gpu

DEV = "cuda"
U16, U32 = 2.0 ** -8, 2.0 ** -24
TINY = 2.0 ** -120   # far below every bound; covers results that underflow
BF = torch.bfloat16


def plan_for(before, rows, dim, dp=4, rank=1):
    """A plan whose matrix follows `before` elements (0: is the first parameter)."""
    sizes = ([before] if before else []) + [rows * dim, 37]
    plan = Z.build_range_map(sizes, sum(sizes), dp, rank)
    return plan, (1 if before else 0), slice(before, before + rows * dim)


def rand(*shape, seed, scale=1.0, dtype=BF):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def tokens_for(n, vocab, kind, seed):
    """uniform, zipf (1/k), one (all the same), ends (first and last row and
    out of range), none (all out of range)."""
    rng = np.random.Generator(np.random.PCG64(seed))
    if kind == "uniform":
        t = rng.integers(0, vocab, n)
    elif kind == "zipf":
        t = np.minimum(np.exp(rng.random(n) * np.log(vocab + 1)).astype(np.int64) - 1, vocab - 1)
        t[rng.random(n) < 0.1] = -100
    elif kind == "one":
        t = np.full(n, vocab // 2)
    elif kind == "ends":
        t = rng.choice([0, vocab - 1, vocab, -1, 2 ** 31 + 1, -2 ** 62, 2 ** 62, 2 ** 32], n)
    else:
        t = rng.choice([-100, vocab, 2 ** 32, 2 ** 32 + 1], n)
    return torch.from_numpy(t.astype(np.int64)).to(DEV)


def strided(n, dim, how, dtype):
    """[n, dim] rows: contiguous, every second row slot and 3 columns wider,
    or one element off the alignment."""
    if how == "contiguous":
        return torch.empty(n, dim, dtype=dtype, device=DEV)
    if how == "wide":
        return torch.full((n, 2 * (dim + 3)), 7.0, dtype=dtype, device=DEV)[:, :dim]
    return torch.full((n * dim + 1,), 7.0, dtype=dtype, device=DEV)[1:].view(n, dim)


def bits(t):
    return t.view({2: torch.int16, 4: torch.int32}[t.element_size()])


def assert_within(got, want, bound, what):
    got, want = got.double(), want.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - bound
    worst = over.max().item() if over.numel() else 0.0
    assert worst <= 0, f"{what}: {int((over > 0).sum())} values beyond their bound, by up to {worst}"


# ---- lookup ------------------------------------------------------------------------------

@pytest.mark.parametrize("n,vocab,dim,before,pad,kind,scale,dtype,how", [
    (1, 7, 1, 0, 0, "uniform", 1.0, BF, "contiguous"),
    (1, 50, 8, 3, 0, "ends", 2.5, torch.float32, "off"),
    (65, 50, 7, 5, 2, "zipf", 1.0, BF, "wide"),
    (300, 1003, 64, 0, 5, "ends", 8.0, BF, "contiguous"),
    (129, 40, 513, 1, 0, "zipf", 22.6, torch.float32, "wide"),
    (33, 40, 2049, 1, 0, "uniform", 1 / 3, BF, "off"),
    (17, 40, 4096, 4096, 1, "ends", 1.0, BF, "contiguous"),
    (5, 3, 8200, 2, 0, "uniform", 64.0, torch.float32, "contiguous"),
    (40, 9, 100, 0, 0, "none", 1.0, BF, "wide"),
])
def test_lookup_is_exact(gpu, n, vocab, dim, before, pad, kind, scale, dtype, how):
    plan, param, at = plan_for(before, vocab + pad, dim)
    params = rand(plan.buffer_numel, seed=1)
    params[at][vocab * dim:] = float("nan")   # rows behind the vocabulary
    tokens = tokens_for(n, vocab, kind, 3)
    out = strided(n, dim, how, dtype)
    base = out._base if out._base is not None else out
    before_bits = bits(base).clone()
    Z.embedding_lookup(plan, param, vocab, params, tokens, out, scale=scale)
    named = (tokens >= 0) & (tokens < vocab)
    w = params[at].view(-1, dim)[torch.where(named, tokens, 0)].float()
    want = torch.where(named[:, None], w * torch.tensor(scale, dtype=torch.float32, device=DEV), 0.0).to(dtype)
    assert torch.equal(bits(out), bits(want))
    # nothing else of the buffer was written
    out.copy_(torch.zeros_like(out))
    ref = before_bits.clone()
    torch.as_strided(ref, out.shape, out.stride(), out.storage_offset()).copy_(bits(torch.zeros_like(out)))
    assert torch.equal(bits(base), ref)


# ---- the lookup's gradient --------------------------------------------------------------------

def rows_reference(tokens, x, scale, rows, vocab):
    """(sum, sum of sizes, number of terms) by row, in 64 bits."""
    named = (tokens >= 0) & (tokens < vocab)
    idx = tokens[named].cpu()
    x = x[named].double().cpu() * np.float32(scale).item()
    total = torch.zeros(rows, x.shape[1], dtype=torch.float64).index_add_(0, idx, x)
    size = torch.zeros(rows, x.shape[1], dtype=torch.float64).index_add_(0, idx, x.abs())
    count = torch.bincount(idx, minlength=rows).double()[:, None]
    return total.to(DEV), size.to(DEV), count.to(DEV)


ROWS_CASES = [
    # n, vocab, dim, before, pad, kind, scale, type, rows' layout
    (1, 7, 1, 0, 0, "uniform", 1.0, BF, "contiguous"),
    (2, 5, 3, 1, 1, "one", 3.0, torch.float32, "off"),
    (64, 5, 9, 1, 0, "one", 1.0, BF, "wide"),
    (65, 33, 17, 0, 3, "zipf", 0.5, BF, "off"),
    (128, 16, 520, 7, 0, "one", 1.0, torch.float32, "contiguous"),
    (500, 100, 100, 0, 28, "zipf", 10.0, BF, "wide"),
    (1000, 3, 64, 64, 0, "uniform", 1.0, BF, "contiguous"),
    (1025, 1000, 33, 0, 1, "ends", 1.0, BF, "contiguous"),
    (4097, 2003, 250, 77, 1, "zipf", 1.0, BF, "contiguous"),
    (8192, 17, 40, 0, 0, "zipf", 1.0, torch.float32, "contiguous"),
    (8193, 17, 40, 0, 0, "zipf", 1.0, BF, "contiguous"),
    (8193, 300, 24, 5, 0, "one", 1.0, BF, "contiguous"),
    (20000, 511, 16, 0, 0, "uniform", 2.0, BF, "wide"),
    (20000, 512, 16, 0, 0, "uniform", 2.0, BF, "contiguous"),
    (50001, 128256, 8, 8, 0, "zipf", 1.0, BF, "contiguous"),
    (30000, 300000, 5, 8, 0, "uniform", 1.0, torch.float32, "off"),
    (9000, 50, 12, 0, 2, "none", 1.0, BF, "contiguous"),
    (70, 50, 12, 0, 2, "none", 1.0, BF, "contiguous"),
]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,vocab,dim,before,pad,kind,scale,dtype,how", ROWS_CASES)
def test_embedding_grad(gpu, n, vocab, dim, before, pad, kind, scale, dtype, how, accumulate):
    rows = vocab + pad
    plan, param, at = plan_for(before, rows, dim)
    tokens = tokens_for(n, vocab, kind, 5)
    x = strided(n, dim, how, dtype)
    x.copy_(rand(n, dim, seed=7, dtype=dtype))
    x[(tokens < 0) | (tokens >= vocab)] = float("nan")   # rows that name nothing are not read into any sum
    old = rand(plan.buffer_numel, seed=9)
    grads = old.clone()
    ws = torch.full((Z.embedding_grad_workspace_bytes(n, dim),), 255, dtype=torch.uint8, device=DEV)
    Z.embedding_grad(plan, param, vocab, tokens, x, grads, ws, scale=scale, accumulate=accumulate)
    total, size, count = rows_reference(tokens, x, scale, rows, vocab)
    want = total + old[at].view(rows, dim).double() * accumulate
    size = size + old[at].view(rows, dim).double().abs() * accumulate
    # count additions, the product with the scale, the addition to what was there; then bf16
    bound = U16 * want.abs() + (1 + U16) * (count + 2) * U32 * size + TINY
    got = grads[at].view(rows, dim)
    assert_within(got, want, bound, "grads")
    empty = (count == 0)[:, 0]
    if accumulate:
        assert torch.equal(bits(got[empty]), bits(old[at].view(rows, dim)[empty]))
    else:
        assert not got[empty].any()
    outside = torch.ones(plan.buffer_numel, dtype=torch.bool, device=DEV)
    outside[at] = False
    assert torch.equal(bits(grads[outside]), bits(old[outside]))
    again = old.clone()
    ws.random_(0, 255)
    Z.embedding_grad(plan, param, vocab, tokens, x, again, ws, scale=scale, accumulate=accumulate)
    assert torch.equal(bits(again), bits(grads))


# ---- cross entropy ----------------------------------------------------------------------------

class Reference:
    """The loss, lse and gradients in 64 bits, and how far the calls may be off."""

    def __init__(self, w, h, targets, weight, vocab, lse_given=None):
        w, h, weight = w[:vocab].double(), h.double(), weight.double()
        n, dim = h.shape
        named = (targets >= 0) & (targets < vocab)
        z = h @ w.t()
        size = h.abs() @ w.abs().t()
        at = torch.where(named, targets, 0)[:, None]
        self.lse = torch.logsumexp(z, 1)
        pick = z.gather(1, at)[:, 0]
        self.loss = torch.where(named, self.lse - pick, 0.0)
        # a logit: dim products, exact, added
        dz = dim * 2 * U32 * size + TINY
        p = torch.exp(z - self.lse[:, None])
        x = z.amax(1, keepdim=True) - z
        # the sum of exponentials: each moves with its logit and by exp's own
        # error; tiles join by more exponentials of at most the same x (twice);
        # and at most 64 + vocab / 128 additions of positive terms follow each
        # other; then the logarithm (2 units) and its addition to the maximum
        rel = (p * (dz + 3 * (4 * U32 + x * 2 * U32))).sum(1) + (64 + vocab / 128) * U32
        log_s = self.lse - z.amax(1)
        self.d_lse = (dz * p).sum(1) + dz.amax(1) * U32 + rel * 1.01 + 4 * U32 * log_s.abs() + \
            2 * U32 * (self.lse.abs() + z.amax(1).abs()) + TINY
        self.d_loss = torch.where(named, self.d_lse + dz.gather(1, at)[:, 0] + U32 * self.loss.abs() + TINY, 0.0)
        # d: exp of a difference that is off by the logit's and lse's errors and
        # its rounding; minus one, times the weight (a rounding each); to bf16
        hot = torch.zeros_like(p).scatter_(1, at, 1.0) * named[:, None]
        weight = torch.where(named, weight, 0.0)[:, None]
        d = (p - hot) * weight
        off = dz + self.d_lse[:, None] + U32 * (z.abs() + self.lse.abs()[:, None])
        dp = p * (torch.expm1(off) + 4 * U32 + (self.lse[:, None] - z).abs() * 2 * U32)
        dd = weight.abs() * (dp + 2 * U32 * (p + hot))
        dd = dd + U16 * (d.abs() + dd) + TINY
        self.grad_hidden, self.grad_w = d @ w, d.t() @ h
        size_d = d.abs() + dd
        # the products' sums (over the vocabulary also in splits and pieces), rounded at the end
        self.d_hidden = dd @ w.abs() + (vocab + 64) * 2 * U32 * (size_d @ w.abs()) + TINY
        hn = torch.where(named[:, None], h, 0.0)
        self.grad_w = d.t() @ hn
        self.d_w = dd.t() @ hn.abs() + (n + 64) * 2 * U32 * (size_d.t() @ hn.abs()) + TINY


CE_CASES = [
    # n, vocab, dim, before, pad, targets, layout of hidden and grad_hidden
    (1, 1, 1, 0, 0, "uniform", "contiguous"),
    (1, 2, 64, 0, 0, "uniform", "contiguous"),
    (1, 300, 64, 0, 0, "none", "contiguous"),
    (2, 129, 63, 0, 1, "ends", "off"),
    (3, 1000, 65, 1, 0, "uniform", "wide"),
    (16, 257, 128, 0, 0, "zipf", "contiguous"),
    (17, 511, 128, 8, 3, "zipf", "wide"),
    (64, 128, 64, 64, 0, "uniform", "contiguous"),
    (100, 1003, 251, 13, 2, "zipf", "contiguous"),
    (129, 513, 192, 0, 0, "zipf", "off"),
    (301, 2000, 100, 7, 0, "ends", "wide"),
    (520, 3001, 320, 0, 0, "zipf", "contiguous"),
    (1000, 300, 64, 0, 0, "none", "contiguous"),
    (2049, 513, 64, 0, 0, "zipf", "contiguous"),
    (40, 20011, 72, 3, 0, "zipf", "contiguous"),
]


def ce_inputs(n, vocab, dim, before, pad, kind, how, seed=11):
    plan, param, at = plan_for(before, vocab + pad, dim)
    params = rand(plan.buffer_numel, seed=seed, scale=0.3)
    w = params[at].view(-1, dim)
    targets = tokens_for(n, vocab, kind, seed + 1)
    h = strided(n, dim, how, BF)
    named = (targets >= 0) & (targets < vocab)
    # about half of the tokens lean to their target, logits up to about +-10
    lean = rand(n, 1, seed=seed + 2, scale=1.0, dtype=torch.float32).clamp(0, 3)
    h.copy_(rand(n, dim, seed=seed + 3, scale=8 / max(1.0, dim ** 0.5), dtype=torch.float32)
            + lean * w[torch.where(named, targets, 0)].float())
    w[vocab:] = float("nan")
    weight = rand(n, seed=seed + 4, scale=0.1, dtype=torch.float32)
    return plan, param, at, params, w, targets, h, weight


def ce_workspace(n, vocab, dim):
    return torch.full((Z.linear_cross_entropy_workspace_bytes(n, vocab, dim),), 255, dtype=torch.uint8, device=DEV)


def check_ce(n, vocab, dim, before, pad, kind, how, accumulate=False, dtype=BF, parts="both"):
    plan, param, at, params, w, targets, h, weight = ce_inputs(n, vocab, dim, before, pad, kind, how)
    ref = Reference(w, h, targets, weight, vocab)
    ws = ce_workspace(n, vocab, dim)
    loss, lse = (torch.full((n,), 7.0, device=DEV) for _ in range(2))
    Z.linear_cross_entropy(plan, param, vocab, params, h, targets, loss, lse, ws)
    assert_within(lse, ref.lse, ref.d_lse, "lse")
    assert_within(loss, ref.loss, ref.d_loss, "loss")
    named = (targets >= 0) & (targets < vocab)
    # what tokens without a target hold reaches nothing
    h[~named] = float("nan")
    lse[~named] = float("nan")
    weight[~named] = float("nan")
    old = rand(plan.buffer_numel, seed=17)
    ws.fill_(255)
    grads = old.clone() if parts != "hidden" else None
    gh = strided(n, dim, how, dtype) if parts != "rows" else None
    Z.linear_cross_entropy_grad(plan, param, vocab, params, h, targets, lse, weight, gh, grads, ws,
                                accumulate=accumulate)
    if gh is not None:
        rounding = U16 if dtype == BF else U32
        assert_within(gh, ref.grad_hidden, rounding * ref.grad_hidden.abs() + (1 + rounding) * ref.d_hidden,
                      "grad_hidden")
        assert not gh[~named].any()
    if grads is not None:
        rows = vocab + pad
        want, bound = (torch.zeros(rows, dim, dtype=torch.float64, device=DEV) for _ in range(2))
        want[:vocab], bound[:vocab] = ref.grad_w, ref.d_w
        before_sum = old[at].view(rows, dim).double() * accumulate
        bound = bound + U32 * (before_sum.abs() + want.abs()) * accumulate
        want = want + before_sum
        assert_within(grads[at].view(rows, dim), want, U16 * want.abs() + (1 + U16) * bound, "grads")
        if not accumulate:
            assert not grads[at].view(rows, dim)[vocab:].any()
        else:
            assert torch.equal(bits(grads[at].view(rows, dim)[vocab:]), bits(old[at].view(rows, dim)[vocab:]))
        outside = torch.ones(plan.buffer_numel, dtype=torch.bool, device=DEV)
        outside[at] = False
        assert torch.equal(bits(grads[outside]), bits(old[outside]))
    # again on a dirty workspace: the same bits
    ws.random_(0, 255)
    loss2, lse2 = torch.empty_like(loss), torch.empty_like(lse)
    h2 = h.clone()
    h2[~named] = 0.0
    Z.linear_cross_entropy(plan, param, vocab, params, h2, targets, loss2, lse2, ws)
    assert torch.equal(bits(loss2), bits(loss)) and torch.equal(bits(lse2[named]), bits(lse[named]))
    ws.random_(0, 255)
    again = old.clone() if grads is not None else None
    gh2 = torch.empty(n, dim, dtype=dtype, device=DEV) if gh is not None else None
    Z.linear_cross_entropy_grad(plan, param, vocab, params, h2, targets, lse, weight, gh2, again, ws,
                                accumulate=accumulate)
    if gh is not None:
        assert torch.equal(bits(gh2), bits(gh))
    if grads is not None:
        assert torch.equal(bits(again), bits(grads))


@pytest.mark.parametrize("n,vocab,dim,before,pad,kind,how", CE_CASES)
def test_cross_entropy(gpu, n, vocab, dim, before, pad, kind, how):
    check_ce(n, vocab, dim, before, pad, kind, how)


@pytest.mark.parametrize("case", [4, 7, 8, 10, 11])
@pytest.mark.parametrize("accumulate,dtype,parts", [(True, BF, "both"), (False, torch.float32, "hidden"),
                                                   (True, BF, "rows"), (True, torch.float32, "both")])
def test_cross_entropy_options(gpu, case, accumulate, dtype, parts):
    check_ce(*CE_CASES[case], accumulate=accumulate, dtype=dtype, parts=parts)
