"""The operators at a language model's two vocabulary ends, as cases to be
measured and compared.

The vocabulary matrix W (a row of `dim` numbers for each of `vocab` tokens) is
one parameter of the optimizer's flat buffers: its bf16 rows are read from the
parameter buffer that the all-gather leaves, and its gradient is written into
the bf16 contribution that the rank sends. It starts wherever the parameters
before it end (`before` elements), and may hold more rows than the vocabulary
has (`pad`), which get a gradient of zero.

Operators (`op` of a case):
  lookup   out_i = scale * W[token_i], zero for a token outside the vocabulary
  rows     W's gradient of that lookup: for each row the sum of scale *
           grad_out_i over the tokens that named it, in bf16 over the whole
           parameter
  score    the softmax cross entropy of logits hidden W^T at a target, a
           token, loss_i = lse_i - logit_i[target_i], and lse_i; a target
           outside the vocabulary has loss 0
  train    score, and the gradients of sum_i grad_loss_i * loss_i by hidden
           and by W; where the case is tied, W's gradient of its lookup (of
           `tokens`, scaled by `scale`) is added to the same rows
"""

from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"


# ---- cases ------------------------------------------------------------------------------

def listed():
    return [
        # one sequence being continued: nothing but latency
        dict(name="lookup, one token, GPT-2 small", op="lookup", n=1, vocab=50257, dim=768, pad=0, before=0,
             scale=1.0, to="bf16"),
        # a microbatch of a model with a scaled embedding and an fp32 residual stream, off every alignment
        dict(name="lookup, odd rows, scaled, fp32", op="lookup", n=5001, vocab=10007, dim=1537, pad=3, before=1001,
             scale=39.2, to="f32"),
        # a long microbatch of a large model
        dict(name="lookup, Llama-3-8B, 16384 tokens", op="lookup", n=16384, vocab=128256, dim=4096, pad=0, before=0,
             scale=1.0, to="bf16"),
        # the smallest model's microbatch
        dict(name="rows, 300 tokens", op="rows", n=300, vocab=2003, dim=250, pad=1, before=77, scale=1.0, to="bf16"),
        # the everyday microbatch of a small model, its vocabulary padded to a multiple of 128
        dict(name="rows, GPT-2 small, 8192 tokens", op="rows", n=8192, vocab=50257, dim=768, pad=47, before=0,
             scale=1.0, to="bf16"),
        # many tokens and few rows: long runs of the same token; fp32 residual stream
        dict(name="rows, 131072 tokens, fp32", op="rows", n=131072, vocab=32000, dim=1024, pad=0, before=4096,
             scale=32.0, to="f32"),
        # a large model's microbatch: a gigabyte of gradient
        dict(name="rows, Llama-3-8B, 8192 tokens", op="rows", n=8192, vocab=128256, dim=4096, pad=0, before=0,
             scale=1.0, to="bf16"),
        # the last tokens of a few sequences
        dict(name="score, 5 tokens, GPT-2 small", op="score", n=5, vocab=50257, dim=768, pad=0, before=0),
        # an evaluation batch
        dict(name="score, Llama-3-8B, 4096 tokens", op="score", n=4096, vocab=128256, dim=4096, pad=0, before=4096),
        # a small model of odd sizes
        dict(name="train, 301 tokens, odd", op="train", n=301, vocab=1003, dim=251, pad=2, before=13, tied=False,
             scale=1.0),
        # the whole step at the tied matrix of a small model
        dict(name="train, GPT-2 small, tied, 8192 tokens", op="train", n=8192, vocab=50257, dim=768, pad=0, before=0,
             tied=True, scale=1.0),
        # the untied head of a large model: it follows the final norm
        dict(name="train, Llama-3-8B, 4096 tokens", op="train", n=4096, vocab=128256, dim=4096, pad=0, before=4096,
             tied=False, scale=1.0),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["lookup", "rows", "score", "train", "train"])
    vocab = log(100, 131072)
    dim = 64 * log(1, 128) if rng.random() < 0.6 else log(16, 8192)
    before = rng.choice([0, dim, dim, rng.randrange(1, 5000)])
    case = dict(op=op, vocab=vocab, dim=dim, pad=rng.choice([0, 0, -vocab % 128, rng.randrange(40)]), before=before)
    if op in ("lookup", "rows"):
        # up to 2^29 numbers of input or output, and of the matrix
        case["vocab"] = vocab = min(vocab, (1 << 29) // dim)
        return dict(case, n=min(log(1, 262144), (1 << 28) // dim), scale=rng.choice([1.0, dim ** 0.5]),
                    to=rng.choice(["bf16", "bf16", "f32"]))
    n = max(1, min(log(1, 16384), int(4096 * 4096 * 128256 / (dim * vocab))))
    if op == "train":
        case.update(tied=rng.random() < 0.4, scale=rng.choice([1.0, dim ** 0.5]))
    return dict(case, n=n)


def work(case):
    n, v, d, rows = case["n"], case["vocab"], case["dim"], case["vocab"] + case["pad"]
    wide = 4 if case.get("to") == "f32" else 2
    if case["op"] == "lookup":
        # the tokens, the distinct rows that they name (about this many of those drawn below), the output
        return {"bytes": 8 * n + 2 * d * min(n, v) + wide * n * d, "flops": n * d}
    if case["op"] == "rows":
        return {"bytes": 8 * n + wide * n * d + 2 * rows * d, "flops": n * d}
    score = 2 * d * (v + n) + 8 * n + 8 * n
    if case["op"] == "score":
        return {"bytes": score, "flops": 2 * n * v * d}
    more = 4 * n + 2 * n * d + 2 * rows * d + (8 * n + 2 * n * d if case["tied"] else 0)
    return {"bytes": score + more, "flops": 6 * n * v * d}


# ---- inputs --------------------------------------------------------------------------------

def _tokens(n, vocab, gen):
    """Token numbers as text has them: the k-th commonest about as often as 1/k,
    and 1 in 16 outside the vocabulary (padding, masked targets)."""
    u = torch.rand(n, generator=gen, device=DEV, dtype=torch.float64)
    t = torch.exp(u * math.log(vocab + 1)).floor().long().sub(1).clamp(0, vocab - 1)
    out = torch.rand(n, generator=gen, device=DEV) < 1 / 16
    return torch.where(out & (torch.arange(n, device=DEV) > 0), -100, t)


def prepare(case, seed):
    n, v, d, op = case["n"], case["vocab"], case["dim"], case["op"]
    rows, before = v + case["pad"], case["before"]
    sizes = ([before] if before else []) + [rows * d, 1024]
    param = 1 if before else 0
    at = slice(before, before + rows * d)
    total = sum(sizes) + (-sum(sizes)) % 8
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + (n * 31 + v * 17 + d) % 104729)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)  # noqa: E731
    s = dict(case=case, param=param, at=at, rows=rows)
    dtype = torch.float32 if case.get("to") == "f32" else torch.bfloat16
    if op != "rows":
        # the parameter buffer, weights of a model's usual size
        s["params"] = torch.empty(total, dtype=torch.bfloat16, device=DEV)
        for i in range(0, total, 1 << 28):
            j = min(total, i + (1 << 28))
            s["params"][i:j] = normal(j - i) * 0.02
    if op != "lookup":
        s["grads"] = torch.zeros(total, dtype=torch.bfloat16, device=DEV)
    if op in ("lookup", "rows") or case.get("tied"):
        s["tokens"] = _tokens(n, v, gen)
    if op == "lookup":
        s["out"] = torch.empty(n, d, dtype=dtype, device=DEV)
    if op == "rows":
        s["grad_out"] = (normal(n, d) * 1e-3).to(dtype)
    if op in ("score", "train"):
        s["targets"] = _tokens(n, v, gen)
        # normalised hidden states that lean towards their target's row, some
        # not at all and some far: losses from the vocabulary's entropy to near 0
        w = s["params"][at].view(rows, d)[s["targets"].clamp(0)].float()
        lean = torch.rand(n, 1, generator=gen, device=DEV) * 12 / (0.02 * d ** 0.5)
        h = normal(n, d) + w / (0.02 * d ** 0.5) * lean.clamp(max=d ** 0.5)
        s["hidden"] = (h * torch.rsqrt(h.square().mean(1, keepdim=True))).to(torch.bfloat16)
        s["loss"], s["lse"] = (torch.empty(n, device=DEV) for _ in range(2))
    if op == "train":
        # a weight a token, as sequences of different lengths have it
        s["grad_loss"] = (0.5 + torch.rand(n, generator=gen, device=DEV)) / n
        s["grad_hidden"] = torch.empty(n, d, dtype=torch.bfloat16, device=DEV)
        if case["tied"]:
            s["grad_out"] = (normal(n, d) / n).to(torch.bfloat16)
    if own:
        import zero_distributed_optimizer_amd as zdo
        s["plan"] = zdo.build_range_map(sizes, total, 8, 1)
        need = 0
        if op == "rows" or case.get("tied"):
            need = zdo.embedding_grad_workspace_bytes(n, d)
        if op in ("score", "train"):
            need = max(need, zdo.linear_cross_entropy_workspace_bytes(n, v, d))
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return s


# ---- one pass ----------------------------------------------------------------------------------

def run(state):
    if not own:
        return plain(state)
    import zero_distributed_optimizer_amd as zdo
    case, plan, param = state["case"], state["plan"], state["param"]
    v, op, s = case["vocab"], case["op"], state
    if op == "lookup":
        zdo.embedding_lookup(plan, param, v, s["params"], s["tokens"], s["out"], scale=case["scale"])
        return s["out"]
    if op == "rows":
        zdo.embedding_grad(plan, param, v, s["tokens"], s["grad_out"], s["grads"], s["workspace"],
                           scale=case["scale"])
        return s["grads"][s["at"]]
    zdo.linear_cross_entropy(plan, param, v, s["params"], s["hidden"], s["targets"], s["loss"], s["lse"],
                             s["workspace"])
    if op == "score":
        return {"loss": s["loss"], "lse": s["lse"]}
    zdo.linear_cross_entropy_grad(plan, param, v, s["params"], s["hidden"], s["targets"], s["lse"], s["grad_loss"],
                                  s["grad_hidden"], s["grads"], s["workspace"])
    if case["tied"]:
        zdo.embedding_grad(plan, param, v, s["tokens"], s["grad_out"], s["grads"], s["workspace"],
                           scale=case["scale"], accumulate=True)
    return {"loss": s["loss"], "lse": s["lse"], "grad_hidden": s["grad_hidden"], "grads": s["grads"][s["at"]]}


def _row_sums(state, out):
    """out (fp32 rows) plus scale * the sums of grad_out's rows by token."""
    case, t = state["case"], state["tokens"]
    named = (t >= 0) & (t < case["vocab"])
    x = torch.where(named[:, None], state["grad_out"].float(), 0.0)
    return out.add_(torch.zeros_like(out).index_add_(0, torch.where(named, t, 0), x), alpha=case["scale"])


def plain(state):
    case = state["case"]
    n, v, d, op = case["n"], case["vocab"], case["dim"], case["op"]
    if op == "lookup":
        t = state["tokens"]
        named = (t >= 0) & (t < v)
        w = state["params"][state["at"]].view(-1, d)[torch.where(named, t, 0)].float()
        return torch.where(named[:, None], w * case["scale"], 0.0).to(state["out"].dtype)
    if op == "rows":
        out = torch.zeros(state["rows"], d, device=DEV)
        return _row_sums(state, out).to(torch.bfloat16).view(-1)
    w = state["params"][state["at"]].view(-1, d)[:v].float()
    h, t = state["hidden"].float(), state["targets"]
    named = (t >= 0) & (t < v)
    at = torch.where(named, t, 0)
    logits = h @ w.t()
    top = logits.amax(1)
    picked = logits.gather(1, at[:, None])[:, 0]
    p = logits.sub_(top[:, None]).exp_()
    total = p.sum(1)
    lse = top + total.log()
    loss = torch.where(named, lse - picked, 0.0)
    if op == "score":
        return {"loss": loss, "lse": lse}
    # softmax minus one at the target, weighted
    p.div_(total[:, None]).scatter_add_(1, at[:, None], torch.full((n, 1), -1.0, device=DEV))
    p.mul_(torch.where(named, state["grad_loss"], 0.0)[:, None])
    grad_hidden = (p @ w).to(torch.bfloat16)
    grads = torch.zeros(state["rows"], d, device=DEV)
    torch.mm(p.t(), h, out=grads[:v])
    if case["tied"]:
        _row_sums(state, grads)
    return {"loss": loss, "lse": lse, "grad_hidden": grad_hidden, "grads": grads.to(torch.bfloat16).view(-1)}


# ---- the definition in 64 bits -------------------------------------------------------------------

def exact(case, seed):
    """What run() returns for these inputs, from the definitions, in 64 bits:
    one-hot rows by equality, the logits in blocks of tokens, the softmax by
    its logarithm."""
    s = prepare(case, seed)
    n, v, d, rows = case["n"], case["vocab"], case["dim"], s["rows"]
    f64 = dict(dtype=torch.float64, device=DEV)

    def gathered(tokens, x):
        """Sum over i of x_i in row token_i: by runs of the sorted tokens."""
        keep = ((tokens >= 0) & (tokens < v)).nonzero()[:, 0]
        out = torch.zeros(rows, d, **f64)
        if not len(keep):
            return out
        order = keep[torch.sort(tokens[keep], stable=True).indices]
        names, count = torch.unique_consecutive(tokens[order], return_counts=True)
        end = count.cumsum(0)
        for c in range(0, d, 512):
            run = torch.cat([torch.zeros(1, min(512, d - c), **f64), x[order, c:c + 512].double().cumsum(0)])
            out[names, c:c + 512] = run[end] - run[end - count]
        return out

    if case["op"] == "lookup":
        w = torch.cat([s["params"][s["at"]].view(rows, d)[:v], torch.zeros(1, d, dtype=torch.bfloat16, device=DEV)])
        t = s["tokens"]
        return w[torch.where((t < 0) | (t >= v), v, t)].double() * case["scale"]
    if case["op"] == "rows":
        return (gathered(s["tokens"], s["grad_out"]) * case["scale"]).view(-1)
    w, h, t = s["params"][s["at"]].view(rows, d)[:v].double(), s["hidden"].double(), s["targets"]
    block = max(1, min(n, (1 << 28) // v))
    loss, lse, train = torch.zeros(n, **f64), torch.zeros(n, **f64), case["op"] == "train"
    grad_hidden, grads = torch.zeros(n if train else 0, d, **f64), torch.zeros(rows if train else 0, d, **f64)
    columns = torch.arange(v, device=DEV)
    for i in range(0, n, block):
        k = slice(i, min(n, i + block))
        hot = t[k, None] == columns
        logits = torch.mm(h[k], w.t())
        lse[k] = torch.logsumexp(logits, 1)
        named = hot.any(1)
        loss[k] = torch.where(named, lse[k] - (logits * hot).sum(1), 0.0)
        if train:
            weight = torch.where(named, s["grad_loss"][k].double(), 0.0)
            g = (torch.exp(logits - lse[k, None]) - hot.double()) * weight[:, None]
            grad_hidden[k] = torch.mm(g, w)
            grads[:v] += torch.mm(g.t(), h[k])
    if not train:
        return {"loss": loss, "lse": lse}
    if case["tied"]:
        grads += gathered(s["tokens"], s["grad_out"]) * case["scale"]
    return {"loss": loss, "lse": lse, "grad_hidden": grad_hidden, "grads": grads.view(-1)}
