"""The operators at the two ends of a language model's vocabulary matrix, as cases to be measured.

* the softmax cross entropy of the lm_head product, without keeping the logits: the loss alone (scoring), the
  gradient for a known log-sum-exp, and loss and gradient in one call (a training step);
* the embedding lookup with scaling, and its gradient by sorted tokens;
* both on one tied matrix.

The matrix is vocab-parallel: `tp` blocks of `shard` rows, block r holding the vocabulary's entries r*shard and on.
`vocab` is the real vocabulary (the rows past it are padding), a label of -100 leaves its row out, a token outside the
matrix (-1: padding) gives a row of zeros.
"""

import math

import torch

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False

own = False

IGNORE = -100
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------- the cases


def listed():
    return [
        # the log-probability of one given token per decode step, at the benchmark's head (TP = 8, V = 163840)
        head("score_token", "score", tp=8, shard=20480, hidden=7168, m=1),
        # 16 requests of 4 rows each (speculative tokens to be verified), a padded vocabulary of odd width
        head("score_batch", "score", tp=8, shard=20480, hidden=7168, m=64, vocab=163837),
        # scoring a prompt of 1000 tokens
        head("score_prompt", "score", tp=8, shard=20480, hidden=7168, m=1000),
        # the smallest training step: latency counts; few rows, some left out
        head("step_small", "step", tp=2, shard=2048, hidden=264, m=33, vocab=4091, dtype="fp16", left_out=0.2),
        # fine-tuning on answers alone: the prompt's rows, 40 %, are left out; odd rows and vocabulary
        head("step_answers", "step", tp=4, shard=8000, hidden=2048, m=2047, vocab=31999, left_out=0.4),
        # the largest: 4096 tokens on the benchmark's head
        head("step_large", "step", tp=8, shard=20480, hidden=7168, m=4096),
        # the second half of a step whose upstream gradient comes later: log-sum-exp kept, fp16, with the z-loss
        head("grad_later", "grad", tp=8, shard=4096, hidden=4096, m=777, dtype="fp16", left_out=0.1, scale=0.5,
             z_weight=1e-3),
        # one matrix at both ends of the model: the head's gradient and the embedding's in one buffer
        head("tied_step", "tied", tp=8, shard=4096, hidden=1024, m=8192, left_out=0.05),
        # the lookup of one decode step, and of a long prompt
        table("lookup_token", "lookup", tp=8, shard=20480, hidden=7168, n=4),
        table("lookup_prompt", "lookup", tp=8, shard=20480, hidden=7168, n=16383, left_out=0.02),
        # the gradient of a small table held in 32 bits, and of a long batch with frequent tokens
        table("scatter_small", "scatter", tp=2, shard=2048, hidden=264, n=129, dtype="fp32", left_out=0.1),
        table("scatter_large", "scatter", tp=8, shard=20480, hidden=2048, n=65536, left_out=0.02),
    ]


def head(name, op, *, tp, shard, hidden, m, vocab=0, dtype="bf16", left_out=0.0, scale=1.0, z_weight=0.0):
    case = {"op": op, "tp": tp, "shard": shard, "hidden": hidden, "m": m, "vocab": vocab or tp * shard, "dtype": dtype,
            "left_out": left_out, "scale": scale, "z_weight": z_weight}
    return {"name": name, **case} if name else case


def table(name, op, *, tp, shard, hidden, n, dtype="bf16", left_out=0.0, scale=None):
    case = {"op": op, "tp": tp, "shard": shard, "hidden": hidden, "m": n, "dtype": dtype, "left_out": left_out,
            "scale": math.sqrt(hidden) if scale is None else scale}
    return {"name": name, **case} if name else case


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["score", "score", "step", "step", "grad", "tied", "lookup", "scatter", "scatter"])
    tp = rng.choice([1, 2, 3, 4, 8])
    shard = 32 * max(1, _log(rng, 1024, 163840) // (32 * tp))
    hidden = 8 * max(8, _log(rng, 64, 7168) // 8)
    if op in ("lookup", "scatter"):
        return table("", op, tp=tp, shard=shard, hidden=hidden, n=_log(rng, 1, 65536),
                     dtype=rng.choice(["bf16", "fp16", "fp32"]), left_out=rng.choice([0.0, 0.1]),
                     scale=rng.choice([1.0, math.sqrt(hidden)]))
    m = _log(rng, 1, 256 if op == "score" and rng.random() < 0.5 else 4096)
    return head("", op, tp=tp, shard=shard, hidden=hidden, m=m, vocab=tp * shard - rng.choice([0, rng.randrange(1, 32)]),
                dtype=rng.choice(["bf16", "fp16"]), left_out=rng.choice([0.0, 0.0, 0.3]),
                scale=rng.choice([1.0, 0.5]), z_weight=rng.choice([0.0, 1e-3]))


def work(case):
    rows, hidden, m = case["tp"] * case["shard"], case["hidden"], case["m"]
    size = 4 if case["dtype"] == "fp32" else 2
    kept = m * (1.0 - case["left_out"])
    if case["op"] == "lookup":
        return {"bytes": kept * hidden * size + m * hidden * size + 8 * m, "flops": kept * hidden}
    if case["op"] == "scatter":  # the gradient is dense: every row of the matrix is written
        return {"bytes": kept * hidden * size + rows * hidden * size + 8 * m, "flops": kept * hidden}
    product = 2.0 * kept * case["vocab"] * hidden
    x, w = kept * hidden * 2, case["vocab"] * hidden * 2
    if case["op"] == "score":
        return {"bytes": x + w + 8 * m + 8 * m, "flops": product}
    # the logits, and the gradient's two products; the logits are not kept, so `grad` computes them again
    grads = m * hidden * 2 + rows * hidden * 2
    more = 8 * m + kept * hidden * 2 + kept * hidden if case["op"] == "tied" else 0
    return {"bytes": x + w + grads + 20 * m + more, "flops": 3.0 * product + (kept * hidden if more else 0)}


# ---------------------------------------------------------------------------------------------- inputs


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)
    rows, hidden, m = case["tp"] * case["shard"], case["hidden"], case["m"]
    dtype = TYPES[case["dtype"]]
    state = dict(case)
    if case["op"] != "scatter":
        w = torch.empty(rows, hidden, dtype=dtype, device=dev)
        for r in range(case["tp"]):
            block = torch.randn(case["shard"], hidden, generator=g, device=dev)
            w[r * case["shard"]:(r + 1) * case["shard"]] = block * 0.02
        state["w"] = w
    # frequencies as in text: the k-th most frequent entry is met about 1/k times as often as the first
    entries = case.get("vocab", rows)

    def frequent():
        rank = torch.exp(torch.rand(m, generator=g, device=dev, dtype=torch.float64) * math.log(entries)).long() - 1
        return (rank.clamp(0, entries - 1) * 7919 + 13) % entries

    left = torch.rand(m, generator=g, device=dev) < case["left_out"]
    if case["op"] in ("lookup", "scatter"):
        state["tokens"] = torch.where(left, -1, frequent())
        if case["op"] == "scatter":
            state["dy"] = (torch.randn(m, hidden, generator=g, device=dev) * 0.01).to(dtype)
        return state
    labels = frequent()
    # hidden states after a norm, that lean to their labels: probabilities from the uniform one's to nearly one
    lean = torch.rand(m, 1, generator=g, device=dev) * 1.2 * math.log(rows) / (case["scale"] * 0.02 ** 2 * hidden)
    x = torch.randn(m, hidden, generator=g, device=dev) + lean * state["w"][labels].float()
    state["x"] = x.to(dtype)
    state["labels"] = torch.where(left, IGNORE, labels)
    if case["op"] != "score":
        # the mean over the rows that count, and a weight of its own for each
        share = 0.5 + torch.rand(m, generator=g, device=dev)
        state["grad"] = share / max(1, m)
    if case["op"] == "grad":
        state["lse"] = _lse_of(state)
    if case["op"] == "tied":
        state["tokens"] = torch.where(left, -1, frequent())
        state["dy"] = (torch.randn(m, hidden, generator=g, device=dev) * 0.01 / m).to(dtype)
    return state


def _lse_of(state):
    """What the first half of the step kept: the rows' log-sum-exp, 0 where the row is left out."""
    lse = torch.logsumexp(_logits(state), dim=1)
    return torch.where(state["labels"] == IGNORE, 0.0, lse)


# ---------------------------------------------------------------------------------------------- one pass


def run(state):
    op = state["op"]
    if own:
        return _own(state)
    if op == "lookup":
        return _lookup(state)
    if op == "scatter":
        return _scatter(state).to(state["dy"].dtype)
    z = _logits(state)
    if op == "grad":
        return _gradient(state, z, state["lse"])
    top = z.amax(dim=1, keepdim=True)
    lse = (top + (z - top).exp().sum(dim=1, keepdim=True).log()).squeeze(1)
    counts = state["labels"] != IGNORE
    target = z.gather(1, state["labels"].clamp(min=0)[:, None]).squeeze(1)
    loss = torch.where(counts, lse - target + state["z_weight"] * lse * lse, 0.0)
    lse = torch.where(counts, lse, 0.0)
    if op == "score":
        return loss, lse
    return (loss, lse) + _gradient(state, z, lse)


def _logits(state):
    w = state["w"][:state["vocab"]].float()
    return state["scale"] * (state["x"].float() @ w.t())


def _gradient(state, z, lse):
    counts = (state["labels"] != IGNORE)[:, None]
    d = (z - lse[:, None]).exp() * (1.0 + 2.0 * state["z_weight"] * lse)[:, None]
    at = torch.arange(state["vocab"], device=d.device)
    d = d - (at[None, :] == state["labels"][:, None]).float()
    d = torch.where(counts, d * (state["scale"] * state["grad"])[:, None], 0.0)
    w, x = state["w"][:state["vocab"]].float(), torch.where(counts, state["x"].float(), 0.0)
    dw = torch.zeros(state["tp"] * state["shard"], state["hidden"], device=d.device)
    dw[:state["vocab"]] = d.t() @ x
    if state["op"] == "tied":
        dw += _scatter(state)
    return (d @ w).to(state["x"].dtype), dw.to(state["w"].dtype)


def _lookup(state):
    tokens = state["tokens"]
    rows = state["w"][tokens.clamp(min=0)].float() * state["scale"]
    return torch.where((tokens >= 0)[:, None], rows, 0.0).to(state["w"].dtype)


def _scatter(state):
    tokens, dy = state["tokens"], state["dy"].float()
    scale = math.sqrt(state["hidden"]) if state["op"] == "tied" else state["scale"]
    dy = torch.where((tokens >= 0)[:, None], dy * scale, 0.0)
    dw = torch.zeros(state["tp"] * state["shard"], state["hidden"], device=dy.device)
    return dw.index_add_(0, tokens.clamp(min=0), dy)


def _own(state):
    """The calls that a user makes."""
    from tp_vocab_logits_amd import embed, embed_grad, head_xent, head_xent_grad, head_xent_step

    op, tp, shard = state["op"], state["tp"], state["shard"]
    if op == "lookup":
        return embed(state["tokens"], state["w"], tp, shard, scale=state["scale"])
    if op == "scatter":
        return embed_grad(state["tokens"], state["dy"], tp, shard, scale=state["scale"])
    how = {"vocab": state["vocab"], "ignore": IGNORE, "scale": state["scale"], "z_weight": state["z_weight"]}
    x, w, labels = state["x"], state["w"], state["labels"]
    if op == "score":
        return head_xent(x, w, labels, tp, shard, **how)
    if op == "grad":
        return head_xent_grad(x, w, labels, state["lse"], state["grad"], tp, shard, **how)
    loss, lse, dx, dw = head_xent_step(x, w, labels, state["grad"], tp, shard, **how)
    if op == "tied":
        embed_grad(state["tokens"], state["dy"], tp, shard, scale=math.sqrt(state["hidden"]), dw=dw, accumulate=True)
    return loss, lse, dx, dw


# ---------------------------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lookup":
        out = torch.zeros(case["m"], case["hidden"], dtype=torch.float64, device=s["w"].device)
        real = s["tokens"] >= 0
        out[real] = s["w"][s["tokens"][real]].double() * case["scale"]
        return out
    rows = case["tp"] * case["shard"]
    if case["op"] == "scatter":
        real = s["tokens"] >= 0
        dw = torch.zeros(rows, case["hidden"], dtype=torch.float64, device=s["dy"].device)
        return dw.index_put_((s["tokens"][real],), s["dy"][real].double() * case["scale"], accumulate=True)
    kept = torch.nonzero(s["labels"] != IGNORE).squeeze(1)  # the rows that count, alone
    x, t = s["x"][kept].double(), s["labels"][kept]
    w = s["w"][:case["vocab"]].double()
    logp = torch.mm(x, w.t()).mul_(case["scale"])
    lse = torch.logsumexp(logp, dim=1) if case["op"] != "grad" else s["lse"][kept].double()
    logp.sub_(lse[:, None])
    dev = x.device

    def spread(values):
        full = torch.zeros((case["m"],) + tuple(values.shape[1:]), dtype=torch.float64, device=dev)
        return full.index_copy_(0, kept, values)

    here = torch.arange(kept.numel(), device=dev)
    head_out = (spread(-logp[here, t] + case["z_weight"] * lse ** 2), spread(lse))
    if case["op"] == "score":
        return head_out
    g = s["grad"][kept].double() * case["scale"]
    p = logp.exp_()
    p.mul_((1.0 + 2.0 * case["z_weight"] * lse)[:, None])
    p[here, t] -= 1.0
    p.mul_(g[:, None])
    dx = spread(torch.mm(p, w))
    dw = torch.zeros(rows, case["hidden"], dtype=torch.float64, device=dev)
    torch.mm(p.t(), x, out=dw[:case["vocab"]])
    if case["op"] == "grad":
        return dx, dw
    if case["op"] == "tied":
        real = s["tokens"] >= 0
        dw.index_put_((s["tokens"][real],), s["dy"][real].double() * math.sqrt(case["hidden"]), accumulate=True)
    return head_out + (dx, dw)
