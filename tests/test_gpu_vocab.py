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
    # where the forms change: few tokens to sorted ones, and the chunks of positions
    (512, 60, 72, 0, 0, "zipf", 1.0, BF, "contiguous"),
    (513, 60, 72, 0, 0, "zipf", 1.0, BF, "contiguous"),
    (512, 9, 5, 1, 3, "one", 1.0, BF, "contiguous"),
    (513, 9, 5, 1, 3, "one", 1.0, torch.float32, "contiguous"),
    (16384, 200, 12, 0, 70, "zipf", 1.0, BF, "contiguous"),
    (32769, 200, 9, 3, 0, "zipf", 1.0, torch.float32, "contiguous"),
    (65536, 200, 8, 8, 0, "zipf", 1.0, BF, "contiguous"),
    (70000, 4, 513, 8, 0, "uniform", 1.0, torch.float32, "contiguous"),
    # an odd number of columns over several waves, ends shared by two of them
    (600, 40, 2051, 3, 1, "zipf", 1.0, BF, "contiguous"),
    (600, 40, 1029, 3, 1, "zipf", 1.0, torch.float32, "wide"),
    # beyond 256 MB of rows
    (140000, 1000, 1000, 0, 0, "zipf", 1.0, BF, "contiguous"),
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
    # where the forms change: rows as they lie, two parts of d, tile sizes, pieces, splits
    (32, 700, 100, 1, 0, "zipf", "contiguous"),
    (33, 700, 100, 1, 0, "zipf", "contiguous"),
    (15, 700, 7, 1, 0, "zipf", "contiguous"),
    (31, 64, 4, 0, 1, "uniform", "off"),
    (20, 131, 129, 5, 0, "zipf", "wide"),
    (128, 1000, 64, 0, 0, "zipf", "contiguous"),
    (129, 1000, 64, 0, 0, "zipf", "contiguous"),
    (1, 40000, 128, 0, 0, "uniform", "contiguous"),
    (3500, 5000, 192, 0, 7, "zipf", "contiguous"),
    (4100, 20000, 64, 64, 0, "zipf", "contiguous"),
    (9000, 16500, 64, 0, 0, "zipf", "contiguous"),
    (260, 30000, 576, 0, 0, "zipf", "contiguous"),
    (700, 300, 1000, 9, 0, "zipf", "off"),
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


# W's gradient is a few tiles, and its sum over the tokens is split
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,vocab,dim,before,pad,kind,how", [
    (4097, 300, 192, 0, 0, "zipf", "contiguous"),
    (3001, 515, 65, 3, 2, "ends", "off"),
    (2500, 1, 3, 0, 1, "uniform", "contiguous"),
    (2049, 129, 1000, 8, 0, "zipf", "wide"),
    (20000, 40, 7, 1, 0, "uniform", "off"),
])
def test_cross_entropy_of_few_rows(gpu, n, vocab, dim, before, pad, kind, how, accumulate):
    check_ce(n, vocab, dim, before, pad, kind, how, accumulate=accumulate)


@pytest.mark.parametrize("case", [4, 7, 8, 10, 11])
@pytest.mark.parametrize("accumulate,dtype,parts", [(True, BF, "both"), (False, torch.float32, "hidden"),
                                                   (True, BF, "rows"), (True, torch.float32, "both")])
def test_cross_entropy_options(gpu, case, accumulate, dtype, parts):
    check_ce(*CE_CASES[case], accumulate=accumulate, dtype=dtype, parts=parts)


def test_cross_entropy_of_large_logits(gpu):
    """Logits of several thousands: one row has all the weight."""
    n, vocab, dim = 70, 600, 128
    plan, param, at = plan_for(0, vocab, dim)
    params = rand(plan.buffer_numel, seed=1, scale=10.0)
    h = rand(n, dim, seed=2, scale=30.0)
    targets = tokens_for(n, vocab, "zipf", 3)
    weight = rand(n, seed=4, dtype=torch.float32)
    ref = Reference(params[at].view(-1, dim), h, targets, weight, vocab)
    assert ref.lse.max() > 4000
    loss, lse = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    ws = ce_workspace(n, vocab, dim)
    Z.linear_cross_entropy(plan, param, vocab, params, h, targets, loss, lse, ws)
    assert_within(lse, ref.lse, ref.d_lse, "lse")
    assert_within(loss, ref.loss, ref.d_loss, "loss")
    gh, grads = torch.empty(n, dim, device=DEV), torch.zeros_like(params)
    Z.linear_cross_entropy_grad(plan, param, vocab, params, h, targets, lse, weight, gh, grads, ws)
    assert_within(gh, ref.grad_hidden, U32 * ref.grad_hidden.abs() + (1 + U32) * ref.d_hidden, "grad_hidden")
    assert_within(grads[at].view(-1, dim), ref.grad_w, U16 * ref.grad_w.abs() + (1 + U16) * ref.d_w, "grads")


@pytest.mark.parametrize("n,dim", [(300, 64), (20, 60)])
def test_a_poisoned_token_stays_alone(gpu, n, dim):
    """Inf and NaN in one token's hidden state reach its own loss, and no
    other token's loss or grad_hidden."""
    vocab = 500
    plan, param, at, params, w, targets, h, weight = ce_inputs(n, vocab, dim, 0, 0, "uniform", "contiguous")
    loss, lse, gh = torch.empty(n, device=DEV), torch.empty(n, device=DEV), torch.empty(n, dim, dtype=BF, device=DEV)
    ws = ce_workspace(n, vocab, dim)
    Z.linear_cross_entropy(plan, param, vocab, params, h, targets, loss, lse, ws)
    Z.linear_cross_entropy_grad(plan, param, vocab, params, h, targets, lse, weight, gh, None, ws)
    for value in (float("inf"), float("nan")):
        bad = h.clone()
        bad[7, 3] = value
        loss2, lse2, gh2 = torch.empty_like(loss), torch.empty_like(lse), torch.empty_like(gh)
        Z.linear_cross_entropy(plan, param, vocab, params, bad, targets, loss2, lse2, ws)
        Z.linear_cross_entropy_grad(plan, param, vocab, params, bad, targets, lse2, weight, gh2, None, ws)
        assert not torch.isfinite(loss2[7])
        others = torch.arange(n, device=DEV) != 7
        for a, b in ((loss, loss2), (lse, lse2), (gh, gh2)):
            assert torch.equal(bits(a[others]), bits(b[others]))


def test_no_tokens(gpu):
    """n = 0: gradients of no tokens, and nothing else."""
    vocab, dim = 40, 12
    plan, param, at = plan_for(5, vocab + 1, dim)
    old = rand(plan.buffer_numel, seed=1)
    none, rows = torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, dim, dtype=BF, device=DEV)
    f = torch.empty(0, device=DEV)
    ws = torch.empty(max(Z.embedding_grad_workspace_bytes(0, dim), Z.linear_cross_entropy_workspace_bytes(0, vocab, dim)),
                     dtype=torch.uint8, device=DEV)
    Z.embedding_lookup(plan, param, vocab, old, none, rows)
    Z.linear_cross_entropy(plan, param, vocab, old, rows, none, f, f.clone(), ws)
    for call in (lambda g, add: Z.embedding_grad(plan, param, vocab, none, rows, g, ws, accumulate=add),
                 lambda g, add: Z.linear_cross_entropy_grad(plan, param, vocab, old, rows, none, f, f.clone(),
                                                            torch.empty_like(rows), g, ws, accumulate=add)):
        g = old.clone()
        call(g, True)
        assert torch.equal(bits(g), bits(old))
        call(g, False)
        assert not g[at].any()
        g[at] = old[at]
        assert torch.equal(bits(g), bits(old))


# ---- the largest sizes ---------------------------------------------------------------------------

@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,dim,dtype", [((1 << 20) + 9, 3, BF), (1 << 20, 3, torch.float32), (513, 1 << 20, BF), (20, 1 << 20, BF)])
def test_many_tokens_and_columns_of_rows(gpu, n, dim, dtype, accumulate):
    test_embedding_grad(gpu, n, 40, dim, 1, 1, "zipf", 1.0, dtype, "contiguous", accumulate)


def test_lookup_of_the_longest_rows(gpu):
    test_lookup_is_exact(gpu, 3, 5, 1 << 20, 1, 0, "ends", 1.0, BF, "off")
    test_lookup_is_exact(gpu, 3, 5, (1 << 20) - 1, 0, 0, "ends", 1.0, torch.float32, "contiguous")


def test_cross_entropy_of_the_most_tokens(gpu):
    check_ce(1 << 22, 17, 8, 0, 1, "uniform", "contiguous")


@pytest.mark.parametrize("dim,before", [(1 << 20, 0), ((1 << 20) - 1, 1)])
@pytest.mark.parametrize("n", [3, 40])
def test_cross_entropy_of_the_longest_rows(gpu, n, dim, before):
    """Rows of -1, 0 and 1 against rows of those over 512: every sum that a logit
    is made of is a multiple of 1/512 below 2^11, so logits are exact."""
    vocab = 3
    plan, param, at = plan_for(before, vocab, dim)
    gen = torch.Generator(device=DEV).manual_seed(n)
    params = torch.randint(-1, 2, (plan.buffer_numel,), generator=gen, device=DEV).to(BF)
    h = (torch.randint(-1, 2, (n, dim), generator=gen, device=DEV) / 512).to(BF)
    w, targets = params[at].view(vocab, dim).double(), tokens_for(n, vocab, "uniform", 3)
    weight = rand(n, seed=4, dtype=torch.float32)
    z = h.double() @ w.t()
    lse, named = torch.logsumexp(z, 1), (targets >= 0) & (targets < vocab)
    hot = torch.nn.functional.one_hot(torch.where(named, targets, 0), vocab) * named[:, None]
    loss_got, lse_got = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    gh, grads = torch.empty(n, dim, dtype=torch.float32, device=DEV), torch.zeros_like(params)
    ws = ce_workspace(n, vocab, dim)
    Z.linear_cross_entropy(plan, param, vocab, params, h, targets, loss_got, lse_got, ws)
    Z.linear_cross_entropy_grad(plan, param, vocab, params, h, targets, lse_got, weight, gh, grads, ws)
    # exponentials of differences up to x, each within (4 + 2x) units and joined
    # three times, 67 additions of positive terms, a logarithm (4 units) and
    # its addition: (12 + 6x + 67 + 4 + 2 + 2 |lse|) 2^-24 < 2^-17 (1 + x)
    x = 2 * z.abs().amax(1) + 2
    off = 2.0 ** -17 * (1 + x)
    assert_within(lse_got, lse, off, "lse")
    assert_within(loss_got, torch.where(named, lse - (z * hot).sum(1), 0.0), 2 * off, "loss")
    weight = torch.where(named, weight.double(), 0.0)[:, None]
    p = torch.exp(z - lse[:, None])
    d = (p - hot) * weight
    # p moves with lse, and has an exponential's error; one, the weight: a rounding each; bf16
    dd = weight.abs() * (p * 3 * off[:, None] + 2 * U32 * (p + hot))
    dd = dd + U16 * (d.abs() + dd) + TINY
    size = d.abs() + dd
    want, bound = d @ w, dd @ w.abs() + 8 * U32 * (size @ w.abs())
    assert_within(gh, want, U32 * want.abs() + (1 + U32) * bound, "grad_hidden")
    hn = torch.where(named[:, None], h.double(), 0.0)
    want, bound = d.t() @ hn, dd.t() @ hn.abs() + (n + 8) * 2 * U32 * (size.t() @ hn.abs()) + TINY
    assert_within(grads[at].view(vocab, dim), want, U16 * want.abs() + (1 + U16) * bound, "grads")


# ---- the test build: 64 workgroups walk every launch ----------------------------------------------

@pytest.mark.parametrize("n,vocab,dim,kind", [(3000, 5000, 40, "zipf"), (20000, 700, 24, "zipf"), (400, 9000, 1300, "zipf"),
                                              (100, 9000, 70, "uniform"), (70000, 300, 8, "one")])
def test_embedding_by_64_workgroups(gpu, n, vocab, dim, kind):
    sizes = [vocab * dim + 13]
    tokens, x, params = tokens_for(n, vocab, kind, 1), rand(n, dim, seed=2), rand(sizes[0] + 3, seed=3)
    outs = []
    for lib in (Z.LIB_PATH, ZB.GRID_LOOP_LIB):
        with Z.use_library(lib):
            plan = Z.build_range_map(sizes, sizes[0], 4, 1)
            out, grads = torch.empty(n, dim, dtype=torch.float32, device=DEV), torch.full_like(params, 7.0)
            added = params.clone()
            ws = torch.empty(Z.embedding_grad_workspace_bytes(n, dim), dtype=torch.uint8, device=DEV)
            Z.embedding_lookup(plan, 0, vocab, params, tokens, out)
            Z.embedding_grad(plan, 0, vocab, tokens, x, grads, ws)
            Z.embedding_grad(plan, 0, vocab, tokens, x, added, ws, accumulate=True)
            torch.cuda.synchronize()
            plan.destroy()
        outs.append((out, grads[:sizes[0]], added))
    for a, b in zip(*outs):
        assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("n,vocab,dim,off", [(3000, 20000, 64, 0), (600, 20000, 100, 1), (16, 9000, 72, 1), (16, 9000, 64, 0),
                                             (5000, 1300, 136, 0)])
def test_cross_entropy_by_64_workgroups(gpu, n, vocab, dim, off):
    sizes = ([off] if off else []) + [vocab * dim]
    total = sum(sizes) + 3
    params, h, targets = rand(total, seed=1, scale=0.2), rand(n, dim, seed=2), tokens_for(n, vocab, "zipf", 3)
    weight = rand(n, seed=4, dtype=torch.float32)
    outs = []
    for lib in (Z.LIB_PATH, ZB.GRID_LOOP_LIB):
        with Z.use_library(lib):
            plan = Z.build_range_map(sizes, sum(sizes), 4, 1)
            param = 1 if off else 0
            loss, lse = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
            gh, grads = torch.empty(n, dim, device=DEV), torch.zeros(total, dtype=BF, device=DEV)
            ws = ce_workspace(n, vocab, dim)
            Z.linear_cross_entropy(plan, param, vocab, params, h, targets, loss, lse, ws)
            Z.linear_cross_entropy_grad(plan, param, vocab, params, h, targets, lse, weight, gh, grads, ws)
            torch.cuda.synchronize()
            plan.destroy()
        outs.append((loss, lse, gh, grads))
    for a, b in zip(*outs):
        assert torch.equal(bits(a), bits(b))


# ---- beyond 32 bits -------------------------------------------------------------------------------

def test_a_matrix_behind_four_billion_elements(gpu):
    """The matrix starts at element 2^32 + 24 and, in another plan, is itself
    longer than 2^32 elements; the same rows give the same results as at 0."""
    vocab, dim, n = 300, 64, 700
    before = 2 ** 32 + 24
    plan, param, at = plan_for(before, vocab, dim, dp=8)
    params = torch.zeros(plan.buffer_numel, dtype=BF, device=DEV)
    w = rand(vocab * dim, seed=1, scale=0.3)
    params[at] = w
    near, near_param, near_at = plan_for(0, vocab, dim, dp=8)
    tokens, h = tokens_for(n, vocab, "zipf", 2), rand(n, dim, seed=3)
    weight = rand(n, seed=4, dtype=torch.float32)
    got = []
    grads_far = torch.zeros_like(params)
    for p, i, buffer, grads in ((near, near_param, torch.nn.functional.pad(w, (0, near.buffer_numel - vocab * dim)),
                                 torch.zeros(near.buffer_numel, dtype=BF, device=DEV)), (plan, param, params, grads_far)):
        out, loss, lse, gh = (torch.empty(n, dim, device=DEV), torch.empty(n, device=DEV), torch.empty(n, device=DEV),
                              torch.empty(n, dim, device=DEV))
        ws = torch.empty(max(Z.embedding_grad_workspace_bytes(n, dim),
                             Z.linear_cross_entropy_workspace_bytes(n, vocab, dim)), dtype=torch.uint8, device=DEV)
        Z.embedding_lookup(p, i, vocab, buffer, tokens, out)
        Z.linear_cross_entropy(p, i, vocab, buffer, h, tokens, loss, lse, ws)
        Z.linear_cross_entropy_grad(p, i, vocab, buffer, h, tokens, lse, weight, gh, grads, ws)
        Z.embedding_grad(p, i, vocab, tokens, h, grads, ws, accumulate=True)
        got.append((out, loss, lse, gh, grads[near_at if p is near else at].clone()))
        if p is plan:
            grads[at] = 0
            assert not grads.any()
    for a, b in zip(*got):
        assert torch.equal(bits(a), bits(b))


def test_a_matrix_of_more_than_four_billion_elements(gpu):
    vocab, dim, n = 530000, 8192, 600   # 4.3e9 elements
    plan, param, at = plan_for(0, vocab, dim, dp=8)
    params = torch.empty(plan.buffer_numel, dtype=BF, device=DEV)
    tokens = torch.cat([torch.tensor([vocab - 1, 0, 524288, 524287, vocab, -1], device=DEV),
                        tokens_for(n - 6, vocab, "uniform", 1)])
    named = (tokens >= 0) & (tokens < vocab)
    rows = tokens[named].unique()
    params.view(-1)[:vocab * dim].view(vocab, dim)[rows] = rand(len(rows), dim, seed=2)
    out = torch.empty(n, dim, dtype=BF, device=DEV)
    Z.embedding_lookup(plan, param, vocab, params, tokens, out)
    want = params[:vocab * dim].view(vocab, dim)[torch.where(named, tokens, 0)]
    assert torch.equal(bits(out), bits(torch.where(named[:, None], want, torch.zeros_like(want))))
    del out, want
    params.fill_(1.0)
    x = rand(n, dim, seed=3)
    ws = torch.empty(Z.embedding_grad_workspace_bytes(n, dim), dtype=torch.uint8, device=DEV)
    Z.embedding_grad(plan, param, vocab, tokens, x, params, ws)
    total = torch.zeros(len(rows), dim, dtype=torch.float64, device=DEV)
    size = torch.zeros_like(total)
    place = torch.searchsorted(rows, tokens[named])
    total.index_add_(0, place, x[named].double())
    size.index_add_(0, place, x[named].double().abs())
    m = params[:vocab * dim].view(vocab, dim)
    assert_within(m[rows], total, U16 * total.abs() + (1 + U16) * (n + 2) * U32 * size + TINY, "grads")
    m[rows] = 0
    assert not m.any()
    assert (params[vocab * dim:] == 1.0).all()


# ---- gradients against differences ------------------------------------------------------------------

@pytest.mark.parametrize("n,dim,before", [(200, 64, 0), (60, 40, 3)])
def test_gradients_against_differences(gpu, n, dim, before):
    """Central differences of sum(weight * loss) along the signs of the formula's
    gradient (so that the terms add up), at points that bf16 holds exactly. Along
    it the logits move at rates r, and the third
    derivative of a log-sum-exp is at most (max r - min r)^3, so the difference
    quotient is off by at most step^2 / 6 times that, and by the losses' own
    errors over the step."""
    vocab, step = 300, 2.0 ** -4
    plan, param, at = plan_for(before, vocab, dim)
    g = torch.Generator(device=DEV).manual_seed(5)
    grid = lambda *shape: torch.randint(-24, 25, shape, generator=g, device=DEV).double() / 64   # noqa: E731
    h, w = grid(n, dim) * 4, grid(vocab, dim) / 4
    targets = tokens_for(n, vocab, "zipf", 6)
    weight = rand(n, seed=7, dtype=torch.float32)
    ws = ce_workspace(n, vocab, dim)

    def total(h, w):
        params = torch.zeros(plan.buffer_numel, dtype=BF, device=DEV)
        params[at] = w.reshape(-1).to(BF)
        hb = h.to(BF)
        assert torch.equal(hb.double(), h) and torch.equal(params[at].double().view(vocab, dim), w)
        loss, lse = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
        Z.linear_cross_entropy(plan, param, vocab, params, hb, targets, loss, lse, ws)
        ref = Reference(params[at].view(vocab, dim), hb, targets, weight, vocab)
        return (weight.double() * loss.double()).sum(), (weight.double().abs() * ref.d_loss).sum(), (params, hb, lse, ref)

    _, _, (params, hb, lse, ref) = total(h, w)
    dh, dw = ref.grad_hidden.sign(), ref.grad_w.sign() / 16
    gh, grads = torch.empty(n, dim, device=DEV), torch.zeros_like(params)
    Z.linear_cross_entropy_grad(plan, param, vocab, params, hb, targets, lse, weight, gh, grads, ws)
    along = lambda rates: ((rates.amax(1) - rates.amin(1)) ** 3 * weight.double().abs()).sum()   # noqa: E731
    for direction, got, rates, bound in (
            ((dh, 0.0), (gh.double() * dh).sum(), dh @ w.t(),
             ((ref.d_hidden * (1 + U32) + U32 * ref.grad_hidden.abs()) * dh.abs()).sum()),
            ((0.0, dw), (grads[at].double().view(vocab, dim) * dw).sum(), h @ dw.t(),
             ((ref.d_w * (1 + U16) + U16 * ref.grad_w.abs()) * dw.abs()).sum())):
        up, up_off, _ = total(h + step * direction[0], w + step * direction[1])
        down, down_off, _ = total(h - step * direction[0], w - step * direction[1])
        difference = (up - down) / (2 * step)
        allowed = along(rates) * step ** 2 / 6 + (up_off + down_off) / (2 * step) + bound
        assert (difference - got).abs() <= allowed
        assert allowed < 0.2 * got.abs(), "the test says something"


def test_the_embedding_gradient_is_the_lookups_adjoint(gpu):
    """sum(lookup(V) * g) = sum(V * gradient(g)) for any V and g."""
    n, vocab, dim = 3000, 700, 72
    plan, param, at = plan_for(0, vocab, dim)
    v, g, tokens = rand(plan.buffer_numel, seed=1), rand(n, dim, seed=2, dtype=torch.float32), tokens_for(n, vocab, "zipf", 3)
    out, grads = torch.empty(n, dim, device=DEV), torch.zeros_like(v)
    Z.embedding_lookup(plan, param, vocab, v, tokens, out, scale=3.0)
    ws = torch.empty(Z.embedding_grad_workspace_bytes(n, dim), dtype=torch.uint8, device=DEV)
    Z.embedding_grad(plan, param, vocab, tokens, g, grads, ws, scale=3.0)
    left = (out.double() * g.double()).sum()
    right = (v[at].double() * grads[at].double()).sum()
    total, size, count = rows_reference(tokens, g, 3.0, vocab, vocab)
    bound = U16 * total.abs() + (1 + U16) * (count + 2) * U32 * size
    allowed = (bound * v[at].double().abs().view(vocab, dim)).sum() + U32 * (out.double() * g.double()).abs().sum()
    assert (left - right).abs() <= allowed


# ---- as they are used -----------------------------------------------------------------------------------

def test_a_training_loop_of_two_ranks(gpu):
    """Three steps of a tied model without layers (hidden = lookup): each rank's
    lookup, loss and gradients into its contribution, the sharded steps, the
    all-gather. Every loss and contribution is held to its formula on the
    parameters of that step, and every step to the oracle bit for bit."""
    import oracle.layout as OL
    import oracle.numerics as ON
    import oracle.step as OS
    vocab, dim, n, D = 211, 72, 160, 2
    sizes = [17, vocab * dim, 40]
    lay = OL.build_layout(sizes, sum(sizes), D)
    plans = [Z.build_range_map(sizes, sum(sizes), D, r) for r in range(D)]
    N, at = plans[0].buffer_numel, slice(17, 17 + vocab * dim)
    hp = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.01)
    start = np.zeros(N, np.float32)
    start[:sum(sizes)] = rand(sum(sizes), seed=1, scale=0.1).float().cpu().numpy()
    params = torch.from_numpy(start.copy()).to(DEV).to(BF)
    state = [[torch.from_numpy(OS.gather_shard(lay, r, start)).to(DEV)] +
             [torch.zeros(plans[r].shard_numel, device=DEV) for _ in range(2)] for r in range(D)]
    ws = torch.empty(max(Z.embedding_grad_workspace_bytes(n, dim), Z.linear_cross_entropy_workspace_bytes(n, vocab, dim)),
                     dtype=torch.uint8, device=DEV)
    for t in range(1, 4):
        contributions = []
        for r in range(D):
            tokens, targets = tokens_for(n, vocab, "zipf", 10 * t + r), tokens_for(n, vocab, "zipf", 100 * t + r)
            grads = torch.zeros(N, dtype=BF, device=DEV)
            x, gx = torch.empty(n, dim, dtype=BF, device=DEV), torch.empty(n, dim, dtype=BF, device=DEV)
            loss, lse = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
            weight = torch.full((n,), 1.0 / n, device=DEV)
            Z.embedding_lookup(plans[r], 1, vocab, params, tokens, x, scale=8.0)
            Z.linear_cross_entropy(plans[r], 1, vocab, params, x, targets, loss, lse, ws)
            Z.linear_cross_entropy_grad(plans[r], 1, vocab, params, x, targets, lse, weight, gx, grads, ws)
            first = grads[at].clone()
            Z.embedding_grad(plans[r], 1, vocab, tokens, gx, grads, ws, scale=8.0, accumulate=True)
            w = params[at].view(vocab, dim)
            ref = Reference(w, x, targets, weight, vocab)
            assert_within(loss, ref.loss, ref.d_loss, "loss")
            assert_within(first.view(vocab, dim), ref.grad_w, U16 * ref.grad_w.abs() + (1 + U16) * ref.d_w, "grads")
            total, size, count = rows_reference(tokens, gx, 8.0, vocab, vocab)
            want = first.double().view(vocab, dim) + total
            assert_within(grads[at].view(vocab, dim), want,
                          U16 * want.abs() + (1 + U16) * (count + 2) * U32 * (size + first.double().view(vocab, dim).abs())
                          + TINY, "grads with the lookup's")
            contributions.append(grads)
        host = [c.view(torch.int16).cpu().numpy().view(np.uint16) for c in contributions]
        outs = [params.clone() for _ in range(D)]
        for r in range(D):
            want = [x.cpu().numpy().copy() for x in state[r]]
            buffer = outs[r].view(torch.int16).cpu().numpy().view(np.uint16).copy()
            Z.sharded_adam_step(plans[r], contributions, Z.WORLD, 0.5, *state[r], outs[r], Z.WORLD, step=t, **hp)
            OS.rank_step(lay, r, host, OS.WORLD, 0.5, *want, ON.hp_array(hp, t), buffer, OS.WORLD)
            for a, b in zip(state[r], want):
                assert np.array_equal(a.cpu().numpy().view(np.uint32), b.view(np.uint32))
            assert np.array_equal(outs[r].view(torch.int16).cpu().numpy().view(np.uint16), buffer)
        Z.all_gather_params(plans[0], outs, params)


def step_of(n, vocab, dim, seed):
    """The four calls on inputs of their own, as a function of nothing, with what
    they write."""
    plan, param, at, params, w, targets, h, weight = ce_inputs(n, vocab, dim, 8, 0, "zipf", "contiguous", seed)
    out = dict(x=torch.zeros(n, dim, device=DEV), loss=torch.zeros(n, device=DEV), lse=torch.zeros(n, device=DEV),
               gh=torch.zeros(n, dim, dtype=BF, device=DEV), grads=torch.zeros(plan.buffer_numel, dtype=BF, device=DEV))
    ws = torch.full((max(Z.embedding_grad_workspace_bytes(n, dim),
                         Z.linear_cross_entropy_workspace_bytes(n, vocab, dim)),), 255, dtype=torch.uint8, device=DEV)

    def run():
        Z.embedding_lookup(plan, param, vocab, params, targets, out["x"], scale=2.0)
        Z.linear_cross_entropy(plan, param, vocab, params, h, targets, out["loss"], out["lse"], ws)
        Z.linear_cross_entropy_grad(plan, param, vocab, params, h, targets, out["lse"], weight, out["gh"], out["grads"],
                                    ws)
        Z.embedding_grad(plan, param, vocab, targets, out["gh"], out["grads"], ws, scale=2.0, accumulate=True)
    return run, out, (plan, params, h, targets, weight, ws)


@pytest.mark.parametrize("sizes", [((700, 900, 64), (9000, 300, 40)), ((16, 500, 30), (300, 2000, 128))])
def test_two_graphs_replayed_in_turn(gpu, sizes):
    steps = [step_of(*s, seed=20 + i) for i, s in enumerate(sizes)]
    want, graphs = [], []
    for run, out, _ in steps:
        run()
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in out.items()})
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graphs.append(graph)
    for turn in range(4):
        for i in (turn % 2, 1 - turn % 2):
            for v in steps[i][1].values():
                v.fill_(float("nan"))
            noise = torch.randn(1 << 20, device=DEV).sum()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.isfinite(noise)
            for k, v in steps[i][1].items():
                got, ref = (v, want[i][k]) if k != "grads" else (v[8:8 + sizes[i][1] * sizes[i][2]],
                                                                want[i][k][8:8 + sizes[i][1] * sizes[i][2]])
                assert torch.equal(bits(got), bits(ref)), k
    # other inputs in the same tensors: the graph reads them anew
    run, out, (plan, params, h, targets, weight, ws) = steps[0]
    targets.copy_(targets.flip(0))
    h.mul_(0.5)
    graphs[0].replay()
    torch.cuda.synchronize()
    got = {k: v.clone() for k, v in out.items()}
    run()
    torch.cuda.synchronize()
    for k, v in out.items():
        assert torch.equal(bits(v), bits(got[k])), k


def test_two_streams_at_once(gpu):
    steps = [step_of(2000, 3000, 192, seed=40), step_of(9000, 2000, 64, seed=41)]
    want = []
    for run, out, _ in steps:
        run()
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in out.items()})
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        for v in (v for _, out, _ in steps for k, v in out.items() if k != "grads"):
            v.fill_(7.0)
        torch.cuda.synchronize()
        for (run, _, _), stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                run()
        torch.cuda.synchronize()
        for (_, out, _), ref in zip(steps, want):
            for k, v in out.items():
                assert torch.equal(bits(v), bits(ref[k])), k


def test_the_stream_argument(gpu):
    """A call is made on the stream that it is given, whatever is current."""
    n, vocab, dim = 500, 300, 64
    plan, param, at = plan_for(0, vocab, dim)
    params, tokens = rand(plan.buffer_numel, seed=1), tokens_for(n, vocab, "uniform", 2)
    out, want = torch.zeros(n, dim, dtype=BF, device=DEV), torch.zeros(n, dim, dtype=BF, device=DEV)
    Z.embedding_lookup(plan, param, vocab, params, tokens, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        Z.embedding_lookup(plan, param, vocab, params, tokens, out, stream=side)
    assert not out.any()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(out), bits(want))


# ---- refusals ---------------------------------------------------------------------------------------------

def test_refusals(gpu):
    n, vocab, dim = 10, 30, 16
    plan, param, at = plan_for(8, vocab, dim)
    params, grads = rand(plan.buffer_numel, seed=1), torch.zeros(plan.buffer_numel, dtype=BF, device=DEV)
    tokens = tokens_for(n, vocab, "uniform", 2)
    h, x = rand(n, dim, seed=3), rand(n, dim, seed=4)
    f = lambda: torch.zeros(n, device=DEV)   # noqa: E731
    loss, lse, weight = f(), f(), f()
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    before = [t.clone() for t in (params, grads, h, x, loss, lse)]

    def refused(error, what, call):
        with pytest.raises(error, match=what):
            call()

    def code(code, call):
        with pytest.raises(Z.ZdoError) as e:
            call()
        assert e.value.code == code, e.value

    look = lambda **k: Z.embedding_lookup(**{**dict(plan=plan, param_index=param, vocab=vocab, params=params,   # noqa: E731
                                                    tokens=tokens, out=x), **k})
    grad = lambda **k: Z.embedding_grad(**{**dict(plan=plan, param_index=param, vocab=vocab, tokens=tokens,   # noqa: E731
                                                  grad_out=x, grads=grads, workspace=ws), **k})
    ce = lambda **k: Z.linear_cross_entropy(**{**dict(plan=plan, param_index=param, vocab=vocab, params=params,   # noqa: E731
                                                      hidden=h, targets=tokens, loss=loss, lse=lse, workspace=ws), **k})
    ceg = lambda **k: Z.linear_cross_entropy_grad(**{**dict(   # noqa: E731
        plan=plan, param_index=param, vocab=vocab, params=params, hidden=h, targets=tokens, lse=lse, grad_loss=weight,
        grad_hidden=x, grads=grads, workspace=ws), **k})

    for call in (look, grad, ce, ceg):
        code(Z.EINVAL, lambda: call(param_index=3))
        code(Z.EINVAL, lambda: call(param_index=-1))
        code(Z.EINVAL, lambda: call(vocab=0))
        code(Z.EINVAL, lambda: call(vocab=vocab + 1))     # more than the parameter holds
        code(Z.EINVAL, lambda: call(param_index=0))       # the parameter of 8 elements
        tok = "tokens" if call in (look, grad) else "targets"
        refused(TypeError, "int64", lambda: call(**{tok: tokens.int()}))
        refused(ValueError, "10 elements", lambda: call(**{tok: tokens[:9]}))
        refused(ValueError, "contiguous", lambda: call(**{tok: torch.zeros(2 * n, dtype=torch.int64, device=DEV)[::2]}))
        refused(ValueError, "device", lambda: call(**{tok: tokens.cpu()}))
    for call in (look, ce, ceg):
        refused(ValueError, "at least", lambda: call(params=params[:-1]))
        refused(TypeError, "bf16", lambda: call(params=params.float()))
    for call in (grad, ceg):
        refused(ValueError, "at least", lambda: call(grads=grads[:-1]))
        refused(ValueError, "at least", lambda: call(workspace=ws[:100]))
        code(Z.EALIAS, lambda: call(grads=ws[:2 * plan.buffer_numel].view(BF)))
        code(Z.EALIGN, lambda: call(workspace=ws[1:]))
    refused(TypeError, "bfloat16", lambda: ce(hidden=h.float()))
    refused(TypeError, "bfloat16 or float32", lambda: look(out=x.half()))
    refused(ValueError, "dimensions", lambda: look(out=x[None]))
    refused(ValueError, "consecutive", lambda: look(out=torch.empty(dim, n, dtype=BF, device=DEV).t()))
    refused(ValueError, "overlap", lambda: grad(grad_out=x[0].expand(n, dim)))
    refused(ValueError, "shape", lambda: ceg(grad_hidden=x[:, :8]))
    refused(ValueError, "shape", lambda: ceg(grad_hidden=x[:9]))
    refused(TypeError, "float32", lambda: ce(loss=loss.double()))
    refused(TypeError, "tensor", lambda: ceg(hidden=None))
    code(Z.EALIAS, lambda: ce(lse=loss))
    code(Z.EALIAS, lambda: ceg(grads=params))
    code(Z.EALIAS, lambda: ceg(grad_hidden=h))
    code(Z.EALIAS, lambda: look(out=params[8:8 + n * dim].view(n, dim)))
    code(Z.EINVAL, lambda: ceg(grad_hidden=None, grads=None))
    with pytest.raises(ValueError):
        Z.embedding_grad_workspace_bytes(-1, 4)
    with pytest.raises(ValueError):
        Z.linear_cross_entropy_workspace_bytes(2 ** 22 + 1, 4, 4)
    torch.cuda.synchronize()
    for a, b in zip(before, (params, grads, h, x, loss, lse)):
        assert torch.equal(bits(a), bits(b))
