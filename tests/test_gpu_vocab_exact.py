"""GPU tests of the calls at the vocabulary matrix on inputs whose results are
known to a few units of fp32, or to the last bit: what a bound that adds up the
roundings of general inputs would hide."""

import numpy as np
import pytest
import torch
from test_gpu_vocab import (BF, DEV, TINY, U32, Reference, assert_within, bits, ce_inputs, ce_workspace, plan_for,
                            rand, step_of, tokens_for)

import zero_distributed_optimizer_amd as Z

pytestmark = pytest.mark.gpu


# ---- small losses of large logits ---------------------------------------------------------

@pytest.mark.parametrize("n,vocab,dim,before", [(20, 300, 64, 0), (20, 300, 60, 3), (256, 300, 64, 0), (300, 1003, 64, 8),
                                                (2049, 513, 64, 0)])
def test_small_losses_of_large_logits(gpu, n, vocab, dim, before):
    """The target's logit is 4096 and all others g below it, all exact, so that
    loss = log(1 + (vocab - 1) exp(-g)) whatever the logits' size. Of that sum s the
    exponentials are off by (4 + 2g) units (with their joins by no more than three
    times that), the additions by 64 + vocab / 128 units of s; the logarithm by 2
    units of itself and 1 / s of what s is off; with the last addition by 2 more.
    Where the logarithm is rounded together with the largest logit, its error is up
    to 2^-12 alone."""
    plan, param, at = plan_for(before, vocab, dim)
    params = torch.zeros(plan.buffer_numel, dtype=BF, device=DEV)
    w = params[at].view(vocab, dim)
    gap = (torch.arange(n, device=DEV) % 20 + 1).double()
    targets = (torch.arange(n, device=DEV) * 7 + 3) % 5          # rows 0 to 4
    # columns 0 to 4: which row is the target; 5: the gap; 6: what all rows share
    w[:5, :5] = torch.eye(5, device=DEV).to(BF)
    w[:, 5], w[:, 6] = -1.0, 64.0
    h = torch.zeros(n, dim, dtype=BF, device=DEV)
    h[torch.arange(n, device=DEV), targets] = gap.to(BF)
    h[:, 5], h[:, 6] = gap.to(BF), 64.0
    z = h.double() @ w.double().t()
    assert torch.equal(z.amax(1), torch.full((n,), 4096.0, dtype=torch.float64, device=DEV))
    want = torch.log1p((vocab - 1) * torch.exp(-gap))
    off = ((4 + 2 * gap) * 3 + 64 + vocab / 128 + 4) * U32 * (1 + want)
    loss, lse = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    Z.linear_cross_entropy(plan, param, vocab, params, h, targets, loss, lse, ce_workspace(n, vocab, dim))
    assert_within(loss, want, off, "loss")
    assert (loss >= 0).all()
    assert_within(lse, 4096 + want, off + 2.0 ** -12, "lse")
    # by way of lse in fp32 it would be beyond the bound
    assert (((4096 + want).float().double() - 4096 - want).abs() > off).any()


# ---- no tokens -----------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_the_gradient_by_hidden_of_no_tokens(gpu, dtype):
    """An empty grad_hidden and no grads: nothing to do, and no error."""
    vocab, dim = 40, 12
    plan, param, at = plan_for(5, vocab, dim)
    params = torch.ones(plan.buffer_numel, dtype=BF, device=DEV)
    rows, f = torch.empty(0, dim, dtype=BF, device=DEV), torch.empty(0, device=DEV)
    Z.linear_cross_entropy_grad(plan, param, vocab, params, rows, torch.empty(0, dtype=torch.int64, device=DEV), f,
                                f.clone(), torch.empty(0, dim, dtype=dtype, device=DEV), None, ce_workspace(0, vocab, dim))
    torch.cuda.synchronize()
    assert (params == 1).all()


# ---- arrays between one another's rows ---------------------------------------------------------

@pytest.mark.parametrize("n,vocab,dim,before,room", [(70, 300, 64, 0, 0), (300, 1003, 128, 8, 0), (20, 200, 60, 3, 4),
                                                     (700, 500, 251, 1, 1), (2049, 513, 64, 0, 8)])
def test_rows_between_rows(gpu, n, vocab, dim, before, room):
    """hidden and grad_hidden as the two halves of one buffer's columns, the
    tokens' x and its gradient too: the same bits as in buffers of their own, and
    nothing else of the buffers is written."""
    plan, param, at, params, w, targets, h, weight = ce_inputs(n, vocab, dim, before, 0, "zipf", "contiguous")
    ws = torch.empty(max(Z.embedding_grad_workspace_bytes(n, dim), Z.linear_cross_entropy_workspace_bytes(n, vocab, dim)),
                     dtype=torch.uint8, device=DEV)
    wide = torch.full((n, 2 * (dim + room)), 7.0, dtype=BF, device=DEV)
    left, right = wide[:, :dim], wide[:, dim + room:2 * dim + room]
    results = []
    for hidden, gh in ((h, torch.zeros_like(h)), (left, right), (right, left)):
        wide.fill_(7.0)
        hidden.copy_(h)
        loss, lse = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
        grads = torch.zeros_like(params)
        Z.linear_cross_entropy(plan, param, vocab, params, hidden, targets, loss, lse, ws)
        Z.linear_cross_entropy_grad(plan, param, vocab, params, hidden, targets, lse, weight, gh, grads, ws)
        Z.embedding_grad(plan, param, vocab, targets, gh, grads, ws, accumulate=True)
        results.append((loss, lse, gh.clone(), grads))
        if gh._base is not None:
            assert torch.equal(bits(hidden), bits(h))
            Z.embedding_lookup(plan, param, vocab, params, targets, hidden)   # over hidden, beside its gradient
            assert torch.equal(bits(gh), bits(results[-1][2]))
            hidden.fill_(7.0)
            gh.fill_(7.0)
            assert (wide == 7.0).all()
    for other in results[1:]:
        for a, b in zip(results[0], other):
            assert torch.equal(bits(a), bits(b))


# ---- sums that are whole numbers ------------------------------------------------------------------

# n, vocab, dim, elements before W, and the form that the sizes get: pieces of the
# vocabulary (a copy of W's rows each, or W in place) and the last one's rows, then
# the tile and the splits of grad_hidden's sum and of W's gradient
# (tests/test_vocab_forms_host.py holds the forms to the library's rules)
WHOLE_CASES = [
    (8403, 500, 1000, 3, "1 copied, last 500; sum 256/1, rows 128/6"),
    (300, 8403, 1000, 3, "1 copied, last 8403; sum 128/9, rows 256/1"),
    (513, 9687, 2601, 1, "1 copied, last 9687; sum 128/4, rows 256/1"),
    (8403, 8403, 1000, 3, "1 copied, last 8403; sum 256/3, rows 256/3"),
    (8403, 8403, 1024, 0, "1 in place, last 8403; sum 256/3, rows 256/3"),
    (16001, 17001, 1000, 3, "3 copied, last 5225; sum 256/1, rows 256/2"),
    (16001, 25001, 1024, 8, "5 in place, last 4521; sum 256/1, rows 256/3"),
    (20001, 16500, 63, 1, "3 copied, last 5236; sum 128/3, rows 128/9"),
    (100, 1100003, 64, 0, "3 in place, last 366307; sum 128/474, rows 128/1"),
    (200, 17001, 16383, 1, "3 copied, last 5225; sum 128/2, rows 256/1"),
    (4096, 33000, 2048, 0, "3 in place, last 10984; sum 256/2, rows 128/1"),
    # the most tokens
    (1 << 22, 40, 24, 8, "1 copied, last 40; sum 128/1, rows 128/474"),
    ((1 << 22) - 1, 17, 8, 0, "1 copied, last 17; sum 128/1, rows 128/474"),
]


def whole_inputs(n, vocab, dim, before):
    """Logits of 0 and -256: columns of one kind hold a -16 for a token, by its
    class, and a 16 for the rows that its class is against. Of the others, one half
    is a token's alone (-1, 0, 1) and one W's alone (-3 to 3)."""
    gen = torch.Generator(device=DEV).manual_seed(n + 31 * vocab + dim)
    draw = lambda lo, hi, *shape: torch.randint(lo, hi + 1, shape, generator=gen, device=DEV)   # noqa: E731
    plan, param, at = plan_for(before, vocab, dim)
    columns = torch.randperm(dim, generator=gen, device=DEV)
    classes = min(8, dim // 4)
    hidden_only, w_only = columns[classes:classes + dim // 3], columns[classes + dim // 3:]
    kind, against = draw(0, classes - 1, n), draw(0, 1, vocab, classes)
    h = torch.zeros(n, dim, dtype=BF, device=DEV)
    h[torch.arange(n, device=DEV), columns[kind]] = -16.0
    h[:, hidden_only] = draw(-1, 1, n, len(hidden_only)).to(BF)
    params = torch.zeros(plan.buffer_numel, dtype=BF, device=DEV)
    w = params[at].view(vocab, dim)
    w[:, columns[:classes]] = 16.0 * against.to(BF)
    w[:, w_only] = draw(-3, 3, vocab, len(w_only)).to(BF)
    targets = draw(0, vocab - 1, n)
    targets[draw(0, 15, n) == 0] = -100
    weight = draw(1, 3 if n < 1 << 20 else 1, n).float()
    return plan, param, at, params, w, h, kind, 1 - against, targets, weight


@pytest.mark.parametrize("accumulate,dtype", [(False, BF), (True, torch.float32)])
@pytest.mark.parametrize("n,vocab,dim,before,form", WHOLE_CASES)
def test_sums_of_whole_numbers(gpu, n, vocab, dim, before, form, accumulate, dtype):
    """With lse = 0, exponentials are 1 and 0 and d, its products and all their
    sums (below 2^24, or multiples of 16 below 2^28) are whole numbers that fp32
    holds: gradients are exact but for the last rounding. Where W's gradient is
    added, what is there takes the sum away but for what its rounding to bf16 left,
    so that one token or row too few or too many shows in the last digit."""
    plan, param, at, params, w, h, kind, p, targets, weight = whole_inputs(n, vocab, dim, before)
    named = targets >= 0
    ws = ce_workspace(n, vocab, dim)
    loss, lse = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    Z.linear_cross_entropy(plan, param, vocab, params, h, targets, loss, lse, ws)
    count = p.sum(0).double()
    assert (count > 0).all()
    want, target = count.log()[kind], torch.where(named, targets, 0)
    pick = -256.0 * (1 - p[target, kind]).double()
    # a sum that is exact, its logarithm (2 units), and the additions to 0 and 256
    assert_within(lse, want, 4 * U32 * want + TINY, "lse")
    assert_within(loss, torch.where(named, want - pick, 0.0), 4 * U32 * (want + 256), "loss")

    # sums over the vocabulary, by class; sums over the tokens, by class and by target
    over_rows = p.double().t() @ w.double()
    want_hidden = torch.where(named[:, None], weight.double()[:, None] * (over_rows[kind] - w[target].double()), 0.0)
    by_class = torch.zeros(p.shape[1], dim, dtype=torch.float64, device=DEV)
    by_target = torch.zeros(vocab, dim, dtype=torch.float64, device=DEV)
    for i in range(0, n, 1 << 20):
        k = torch.arange(i, min(n, i + (1 << 20)), device=DEV)[named[i:i + (1 << 20)]]
        x = weight[k].double()[:, None] * h[k].double()
        by_class.index_add_(0, kind[k], x)
        by_target.index_add_(0, targets[k], x)
    want_rows = p.double() @ by_class - by_target
    h[~named], weight[~named] = float("nan"), float("nan")
    old = -want_rows.to(BF) if accumulate else torch.full_like(w, 7.0)
    grads = torch.full_like(params, 5.0)
    grads[at] = old.view(-1)
    gh = torch.empty(n, dim, dtype=dtype, device=DEV)
    ws.fill_(255)
    Z.linear_cross_entropy_grad(plan, param, vocab, params, h, targets, torch.zeros_like(lse), weight, gh, grads, ws,
                                accumulate=accumulate)
    assert torch.equal(gh, want_hidden.to(dtype))
    got = grads[at].view(vocab, dim)
    assert torch.equal(got, ((want_rows + old.double()) if accumulate else want_rows).to(BF))
    if accumulate:
        assert (got.abs() <= 2.0 ** -8 * want_rows.abs()).all()
    grads[at] = 5.0
    assert (grads == 5.0).all()


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,vocab,dim,before,kind,dtype", [
    ((1 << 20) + 9, 40, 3, 1, "zipf", BF),
    (1 << 20, 40, 3, 1, "one", torch.float32),
    ((1 << 22) + 1, 1000, 8, 0, "zipf", BF),
    ((1 << 22) + 1, 2, 9, 3, "uniform", torch.float32),
    (300000, 7, 1030, 8, "zipf", torch.float32),
    (8192, 3, 2051, 3, "one", BF),
    (512, 3, 72, 0, "one", BF),
])
def test_embedding_grad_of_whole_numbers(gpu, n, vocab, dim, before, kind, dtype, accumulate):
    """Rows of -1, 0 and 1: every sum is exact, as in the test above."""
    plan, param, at = plan_for(before, vocab, dim)
    gen = torch.Generator(device=DEV).manual_seed(n)
    x = torch.randint(-1, 2, (n, dim), generator=gen, device=DEV).to(dtype)
    tokens = tokens_for(n, vocab, kind, 5)
    named = (tokens >= 0) & (tokens < vocab)
    want = torch.zeros(vocab, dim, dtype=torch.float64, device=DEV)
    for i in range(0, n, 1 << 20):
        k = slice(i, i + (1 << 20))
        want.index_add_(0, torch.where(named[k], tokens[k], 0), torch.where(named[k, None], x[k].double(), 0.0) * 2.0)
    x[~named] = float("nan")
    old = -want.to(BF) if accumulate else torch.full((vocab, dim), 7.0, dtype=BF, device=DEV)
    grads = torch.full((plan.buffer_numel,), 5.0, dtype=BF, device=DEV)
    grads[at] = old.view(-1)
    ws = torch.full((Z.embedding_grad_workspace_bytes(n, dim),), 255, dtype=torch.uint8, device=DEV)
    Z.embedding_grad(plan, param, vocab, tokens, x, grads, ws, scale=2.0, accumulate=accumulate)
    got = grads[at].view(vocab, dim)
    assert torch.equal(got, ((want + old.double()) if accumulate else want).to(BF))
    grads[at] = 5.0
    assert (grads == 5.0).all()


# ---- what d's rounding leaves ------------------------------------------------------------------------

def bf16_of(x):
    return x.to(BF).double()


@pytest.mark.parametrize("n,vocab,dim,before", [(1, 7, 9, 0), (33, 700, 100, 1), (100, 700, 64, 0), (129, 300, 64, 8),
                                                (300, 1003, 251, 13), (2100, 5001, 65, 3), (9000, 9000, 192, 0),
                                                (20001, 16500, 63, 1)])
def test_the_rest_of_the_targets_d(gpu, n, vocab, dim, before):
    """With hidden = 0 and lse = 300 every exponential is 0, d has the target's
    -weight alone, and grad_hidden is -weight * W[target]: of d's bf16 part an exact
    product, of the rest a product and an addition in fp32. Without the rest it would
    be off by up to 2^-8 of itself."""
    plan, param, at = plan_for(before, vocab, dim)
    params = rand(plan.buffer_numel, seed=1)
    w = params[at].view(vocab, dim)
    h, targets = torch.zeros(n, dim, dtype=BF, device=DEV), tokens_for(n, vocab, "zipf", 2)
    weight = rand(n, seed=3, dtype=torch.float32)
    gh = torch.empty(n, dim, device=DEV)
    for grads in (None, torch.zeros_like(params)):
        gh.fill_(7.0)
        Z.linear_cross_entropy_grad(plan, param, vocab, params, h, targets, torch.full((n,), 300.0, device=DEV), weight,
                                    gh, grads, ce_workspace(n, vocab, dim))
        named = ((targets >= 0) & (targets < vocab))[:, None]
        rows = w[torch.where(named[:, 0], targets, 0)].double()
        want = torch.where(named, -weight.double()[:, None] * rows, 0.0)
        assert_within(gh, want, 2 * U32 * want.abs(), "grad_hidden")
        coarse = torch.where(named, -bf16_of(weight)[:, None] * rows, 0.0)
        assert ((coarse - want).abs() > 2 * U32 * want.abs())[named[:, 0]].float().mean() > 0.9 or n == 1


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,vocab,dim,before", [(2, 5, 8, 0), (50, 60, 60, 3), (64, 300, 64, 0), (127, 64, 128, 8),
                                                (128, 700, 251, 1), (128, 1100003, 64, 0)])
def test_ds_two_parts_for_few_tokens(gpu, n, vocab, dim, before, accumulate):
    """As above, and tokens in pairs with the same target and hidden state (whole
    numbers), of weights a and -b in [1, 2) with 16 digits: two bf16 parts hold them,
    and the row's sum (b - a) * hidden is exact. By one part each, a and b are off by
    up to 2^-8, as much as their difference may be."""
    plan, param, at = plan_for(before, vocab, dim)
    gen = torch.Generator(device=DEV).manual_seed(n + vocab)
    params = torch.zeros(plan.buffer_numel, dtype=BF, device=DEV)
    pairs = n // 2
    pair = torch.randperm(vocab, generator=gen, device=DEV)[:pairs]
    order = torch.randperm(n, generator=gen, device=DEV)   # an odd one names nothing
    targets = torch.cat([pair, pair, pair.new_full((n - 2 * pairs,), -1)])[order]
    row_h = torch.randint(-7, 8, (pairs, dim), generator=gen, device=DEV).double()
    h = torch.cat([row_h, row_h, row_h.new_full((n - 2 * pairs, dim), float("nan"))])[order].to(BF)
    a, b = (1 + torch.randint(0, 1 << 15, (2, pairs), generator=gen, device=DEV).double() / (1 << 15)).unbind(0)
    weight = torch.cat([a, -b, a.new_full((n - 2 * pairs,), float("nan"))])[order].float()

    def total(x, y):
        rows = torch.zeros(vocab, dim, dtype=torch.float64, device=DEV)
        rows[pair] = (y - x)[:, None] * row_h
        return rows

    want = total(a, b)
    old = -want.to(BF) if accumulate else torch.full((vocab, dim), 7.0, dtype=BF, device=DEV)
    grads = torch.full_like(params, 5.0)
    grads[at] = old.view(-1)
    for gh in (None, torch.empty(n, dim, dtype=BF, device=DEV)):
        out = grads.clone()
        Z.linear_cross_entropy_grad(plan, param, vocab, params, h, targets, torch.full((n,), 300.0, device=DEV), weight,
                                    gh, out, ce_workspace(n, vocab, dim), accumulate=accumulate)
        result = ((want + old.double()) if accumulate else want).to(BF)
        assert torch.equal(out[at].view(vocab, dim), result)
    coarse = total(bf16_of(a), bf16_of(b)).to(BF)
    assert (coarse != want.to(BF))[pair].float().mean() > 0.5


# ---- two streams ------------------------------------------------------------------------------------------

def test_two_streams_write_all_of_w_gradient(gpu):
    """Two steps at once on two streams, W's gradient (and every other output)
    filled with NaN before each round: what a call left unwritten shows."""
    sizes = [(2000, 3000, 192), (9000, 2000, 64)]
    steps = [step_of(*s, seed=40 + i) for i, s in enumerate(sizes)]
    slices = [slice(8, 8 + vocab * dim) for _, vocab, dim in sizes]
    want = []
    for run, out, _ in steps:
        run()
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in out.items()})
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(4):
        for (_, out, _), at in zip(steps, slices):
            for k, v in out.items():
                (v[at] if k == "grads" else v).fill_(float("nan"))
        torch.cuda.synchronize()
        for (run, _, _), stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                run()
        torch.cuda.synchronize()
        for (_, out, _), ref in zip(steps, want):
            for k, v in out.items():
                assert torch.equal(bits(v), bits(ref[k])), k


# ---- rows far from each other, and a workspace of 16-byte alignment --------------------------------------

@pytest.mark.parametrize("n,vocab,dim,before,stride", [(3, 300, 64, 0, 1 << 30), (3, 300, 60, 3, (1 << 30) - 1),
                                                       (300, 700, 64, 8, 1 << 21), (300, 700, 64, 8, (1 << 21) + 8),
                                                       (520, 700, 70, 0, 1 << 22)])
def test_rows_far_apart(gpu, n, vocab, dim, before, stride):
    """Activations' rows at strides up to the largest, some of them beyond 2^32
    bytes: the same bits as from rows that follow each other."""
    plan, param, at, params, w, targets, h, weight = ce_inputs(n, vocab, dim, before, 0, "zipf", "contiguous")
    need = max(Z.embedding_grad_workspace_bytes(n, dim), Z.linear_cross_entropy_workspace_bytes(n, vocab, dim))
    far = [torch.zeros((n - 1) * stride + dim, dtype=BF, device=DEV).as_strided((n, dim), (stride, 1)) for _ in range(2)]
    results = []
    for hidden, gh, off in ((h, torch.empty_like(h), 0), (*far, 16)):
        ws = torch.full((need + off,), 255, dtype=torch.uint8, device=DEV)[off:]
        hidden.copy_(h)
        loss, lse, grads = torch.empty(n, device=DEV), torch.empty(n, device=DEV), torch.zeros_like(params)
        Z.linear_cross_entropy(plan, param, vocab, params, hidden, targets, loss, lse, ws)
        Z.linear_cross_entropy_grad(plan, param, vocab, params, hidden, targets, lse, weight, gh, grads, ws)
        gx = gh.clone()
        Z.embedding_grad(plan, param, vocab, targets, gh, grads, ws, accumulate=True)
        Z.embedding_lookup(plan, param, vocab, params, targets, gh, scale=3.0)
        results.append((loss, lse, gx.contiguous(), grads, gh.contiguous()))
    for a, b in zip(*results):
        assert torch.equal(bits(a), bits(b))


# ---- every bf16 number, and Inf and NaN in a token's gradient --------------------------------------------

@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("scale", [1.0, 0.5, 2.0 ** -9, 3.0, 2.0 ** 127, -1.0, 0.0, float("inf")])
def test_lookup_of_every_bf16_number(gpu, scale, dtype):
    """Subnormal numbers, zeros of both signs, infinities and NaN among them: one
    fp32 product, rounded once."""
    vocab, dim = 512, 128
    plan, param, at = plan_for(8, vocab, dim)
    params = torch.zeros(plan.buffer_numel, dtype=BF, device=DEV)
    params[at] = torch.arange(-(1 << 15), 1 << 15, device=DEV).to(torch.int16).view(BF)
    tokens = torch.randperm(vocab, device=DEV)
    out = torch.empty(vocab, dim, dtype=dtype, device=DEV)
    Z.embedding_lookup(plan, param, vocab, params, tokens, out, scale=scale)
    # on the host, where no product or rounding takes subnormal numbers for zero
    w = params[at].view(vocab, dim).cpu()[tokens.cpu()].float().numpy()
    with np.errstate(all="ignore"):
        want = torch.from_numpy(w * np.float32(scale)).to(dtype)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(out.cpu()), nan)
    assert torch.equal(bits(out.cpu())[~nan], bits(want)[~nan])


@pytest.mark.parametrize("n", [40, 600, 9000])
def test_a_poisoned_gradient_stays_in_its_row(gpu, n):
    """Inf and NaN in one token's grad_out reach the elements of its token's row
    that they stand at, and nothing else."""
    vocab, dim = 300, 72
    plan, param, at = plan_for(3, vocab, dim)
    x, tokens = rand(n, dim, seed=1), tokens_for(n, vocab, "zipf", 2)
    tokens[5] = 7
    ws = torch.empty(Z.embedding_grad_workspace_bytes(n, dim), dtype=torch.uint8, device=DEV)
    results = []
    for poison in (False, True):
        if poison:
            x[5, 3], x[5, 64], x[5, 71] = float("inf"), float("nan"), float("-inf")
        grads = torch.ones(plan.buffer_numel, dtype=BF, device=DEV)
        Z.embedding_grad(plan, param, vocab, tokens, x, grads, ws, accumulate=True)
        results.append(grads)
    row = results[1][at].view(vocab, dim)[7]
    assert row[3] == float("inf") and torch.isnan(row[64]) and row[71] == float("-inf")
    row[[3, 64, 71]] = results[0][at].view(vocab, dim)[7, [3, 64, 71]]
    assert torch.equal(bits(results[1]), bits(results[0]))


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("n,vocab,dim,before,row", [(100, 300, 64, 0, 5), (100, 300, 64, 0, 299), (600, 301, 72, 3, 300),
                                                    (9000, 9000, 192, 0, 8999)])
def test_a_poisoned_row_of_w_stays_in_its_column(gpu, n, vocab, dim, before, row, value):
    """An infinite logit of minus infinity has no weight: losses of other targets
    stay as they are without that row, and grad_hidden is not finite in the column
    only where the infinity stands (0 times it), as the formula has it. A NaN reaches
    every token's loss."""
    plan, param, at, params, w, targets, h, weight = ce_inputs(n, vocab, dim, before, 0, "uniform", "contiguous")
    h[:, 3] = -1.0
    w[row, 3] = value
    loss, lse = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    gh, grads = torch.empty(n, dim, device=DEV), torch.zeros_like(params)
    ws = ce_workspace(n, vocab, dim)
    Z.linear_cross_entropy(plan, param, vocab, params, h, targets, loss, lse, ws)
    if value != value:
        assert torch.isnan(loss).all() and torch.isnan(lse).all()
        return
    hits = targets == row
    assert torch.isfinite(lse).all() and torch.isfinite(loss[~hits]).all() and (loss[hits] == value).all()
    # the row adds an exact 0
    ref = Reference(torch.cat([w[:row], w[row + 1:]]), h, torch.zeros_like(targets), weight, vocab - 1)
    assert_within(lse, ref.lse, ref.d_lse, "lse")
    Z.linear_cross_entropy_grad(plan, param, vocab, params, h, targets, lse, weight, gh, grads, ws)
    assert not torch.isfinite(gh[:, 3]).any()
    others = torch.arange(dim, device=DEV) != 3
    assert torch.isfinite(gh[:, others]).all() and torch.isfinite(grads.float()).all()
