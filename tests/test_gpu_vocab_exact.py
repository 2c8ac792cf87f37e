"""GPU tests of the calls at the vocabulary matrix on inputs whose results are
known to a few units of fp32, or to the last bit: what a bound that adds up the
roundings of general inputs would hide."""

import pytest
import torch
from test_gpu_vocab import BF, DEV, U32, assert_within, bits, ce_inputs, ce_workspace, plan_for

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
