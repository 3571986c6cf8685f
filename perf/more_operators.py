"""Serving many requests at the vocabulary matrix, and training their adapters, as cases to be measured.

* low-rank adapters of many requests beside the shared head: what each row's adapter adds to the product's shards, and
  its gradients;
* beam search's selection over beams and vocabulary;
* the reordering of the beams' states (token histories, caches) in place.

Logits are vocab-parallel: `tp` blocks `[m, shard]`, as the product leaves them, or gathered rows `[m, vocab]`.
"""

import math

import torch

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int64": torch.int64}


# ---------------------------------------------------------------------------------------------- the cases


def listed():
    return [
        # one token of one request with one of 8 adapters, at the benchmark's head (TP = 8, V = 163840)
        adapters("adapt_token", "adapt", tp=8, shard=20480, hidden=7168, m=1, n=8, rank=16),
        # a decode step of 64 requests over 32 adapters, some without one
        adapters("adapt_batch", "adapt", tp=8, shard=20480, hidden=7168, m=64, n=32, rank=16, left_out=0.15),
        # every position's logits of a few long sequences (training's forward pass, scoring): runs of one adapter
        adapters("adapt_sequences", "adapt", tp=8, shard=20480, hidden=7168, m=2047, n=4, rank=64, run=500),
        # the smallest training step: latency counts
        adapters("grad_small", "grad", tp=2, shard=2048, hidden=264, m=33, n=3, rank=8, dtype="fp16", run=8),
        # eight adapters trained at once on short answers, rows of others between them
        adapters("grad_answers", "grad", tp=4, shard=8000, hidden=2048, m=2047, n=8, rank=16, run=60, left_out=0.3),
        # the largest: 4096 rows at the benchmark's head, two adapters
        adapters("grad_large", "grad", tp=8, shard=20480, hidden=7168, m=4096, n=2, rank=64, run=1024),
        # one request of four beams on the gathered rows
        beams("select_one", requests=1, beams=4, keep=8, vocab=163840),
        # 64 requests of eight beams on the padded vocabulary's slice (rows of odd width), some beams finished
        beams("select_batch", requests=64, beams=8, keep=16, vocab=163837, finished=0.1, masked=0.05),
        # the product's shards without a gather, a smaller vocabulary, fp16
        beams("select_shards", requests=16, beams=5, keep=10, vocab=31999, tp=4, shard=8000, dtype="fp16", masked=0.02),
        # token histories of 16 requests
        states("reorder_tokens", requests=16, beams=4, count=1, outer=1, steps=2048, width=1, dtype="int64", lengths=0.5),
        # keys and values of eight layers, [row, head, position, channel], requests of different lengths
        states("reorder_cache", requests=16, beams=4, count=16, outer=8, steps=1024, width=128, lengths=0.9),
        # states without positions (a recurrence's, the last hidden ones), five beams
        states("reorder_hidden", requests=33, beams=5, count=6, outer=1, steps=1, width=7168, dtype="fp32", lengths=0.0),
    ]


def adapters(name, op, *, tp, shard, hidden, m, n, rank, dtype="bf16", run=1, left_out=0.0):
    """`run`: rows that follow one another with the same adapter (a request's tokens)."""
    case = {"op": op, "tp": tp, "shard": shard, "hidden": hidden, "m": m, "n": n, "rank": rank, "dtype": dtype,
            "run": run, "left_out": left_out}
    return {"name": name, **case} if name else case


def beams(name, *, requests, beams, keep, vocab, tp=0, shard=0, dtype="bf16", finished=0.0, masked=0.0, scale=1.0):
    """`tp` 0: gathered rows; otherwise blocks of `shard` columns. `masked`: share of the vocabulary that is banned."""
    case = {"op": "select", "requests": requests, "beams": beams, "keep": keep, "vocab": vocab, "tp": tp,
            "shard": shard, "dtype": dtype, "finished": finished, "masked": masked, "scale": scale}
    return {"name": name, **case} if name else case


def states(name, *, requests, beams, count, outer, steps, width, dtype="bf16", lengths=0.0):
    """`count` tensors `[requests * beams, outer, steps, width]`; `lengths`: the requests' lengths lie between that
    share of `steps` and all of them (0: the whole rows move)."""
    case = {"op": "reorder", "requests": requests, "beams": beams, "count": count, "outer": outer, "steps": steps,
            "width": width, "dtype": dtype, "lengths": lengths}
    return {"name": name, **case} if name else case


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["adapt", "adapt", "grad", "grad", "select", "select", "select", "reorder", "reorder"])
    if op in ("adapt", "grad"):
        tp = rng.choice([1, 2, 3, 4, 8])
        return adapters("", op, tp=tp, shard=8 * max(1, _log(rng, 1024, 163840) // (8 * tp)),
                        hidden=8 * max(8, _log(rng, 64, 7168) // 8),
                        m=_log(rng, 1, 128) if op == "adapt" and rng.random() < 0.5 else _log(rng, 16, 2048),
                        n=_log(rng, 1, 32), rank=8 * rng.choice([1, 2, 3, 4, 8]), dtype=rng.choice(["bf16", "fp16"]),
                        run=_log(rng, 1, 500), left_out=rng.choice([0.0, 0.0, 0.3]))
    if op == "select":
        count = _log(rng, 1, 16)
        tp = rng.choice([0, 0, 1, 2, 4, 8])
        vocab = _log(rng, 100, 163840)
        shard = 8 * -(-vocab // (8 * tp)) if tp else 0
        return beams("", requests=_log(rng, 1, 512 // count), beams=count, keep=rng.choice([count, 2 * count]),
                     vocab=vocab, tp=tp, shard=shard, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                     finished=rng.choice([0.0, 0.2]), masked=rng.choice([0.0, 0.1]), scale=rng.choice([1.0, 0.7]))
    count, steps = _log(rng, 2, 16), _log(rng, 1, 2048)
    width, many = rng.choice([1, 33, 64, 80, 128]), rng.choice([1, 2, 5, 16])
    most = max(1, 2 ** 30 // (count * steps * width * many))  # values in all
    return states("", requests=_log(rng, 1, min(64, most)), beams=count, count=many, outer=1, steps=steps, width=width,
                  dtype=rng.choice(["bf16", "fp32"]), lengths=rng.choice([0.0, 0.3]))


def _distinct(n, draws):
    return n * (1.0 - (1.0 - 1.0 / n) ** draws)


def work(case):
    if case["op"] == "select":
        live = case["requests"] * case["beams"] * (1.0 - case["finished"])
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": live * case["vocab"] * size + case["requests"] * (case["keep"] * 20 + case["beams"] * 5),
                "flops": 4.0 * live * case["vocab"]}
    if case["op"] == "reorder":
        lost = _lost(case)
        row = case["outer"] * case["steps"] * case["width"] * torch.empty(0, dtype=TYPES[case["dtype"]]).element_size()
        share = (1.0 + case["lengths"]) / 2 if case["lengths"] else 1.0
        moved = lost + _distinct(case["beams"] - lost, lost)
        return {"bytes": case["count"] * case["requests"] * moved * row * share + 8 * case["requests"] * case["beams"],
                "flops": 0}
    vocab, hidden, m, n, rank = case["tp"] * case["shard"], case["hidden"], case["m"], case["n"], case["rank"]
    kept = m * (1.0 - case["left_out"])
    used = _distinct(n, max(1.0, kept / case["run"]))
    pairs = used * rank * (hidden + vocab)
    if case["op"] == "adapt":
        return {"bytes": 4.0 * m * vocab + 2.0 * kept * hidden + 2.0 * pairs + 8 * m,
                "flops": 2.0 * kept * rank * (hidden + vocab)}
    return {"bytes": 2.0 * (kept * vocab + kept * hidden + pairs + m * hidden + n * rank * (hidden + vocab)) + 8 * m,
            "flops": 2.0 * kept * rank * (3 * hidden + 2 * vocab)}


def _lost(case):
    """Beams of a request whose slots take another one's state: about half of them, at least one survives."""
    return min(case["beams"] - 1, (case["beams"] + 1) // 2)


# ---------------------------------------------------------------------------------------------- inputs


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)
    state = dict(case)
    if case["op"] == "select":
        _prepare_select(case, state, g, dev)
    elif case["op"] == "reorder":
        _prepare_reorder(case, state, g, dev)
    else:
        _prepare_adapters(case, state, g, dev)
    return state


def _prepare_adapters(case, state, g, dev):
    tp, shard, hidden, m, n, rank = (case[k] for k in ("tp", "shard", "hidden", "m", "n", "rank"))
    dtype = TYPES[case["dtype"]]
    many = -(-m // case["run"])  # requests, one adapter (or none) each
    who = torch.randint(0, n, (many,), generator=g, device=dev)
    who = torch.where(torch.rand(many, generator=g, device=dev) < case["left_out"], -1, who)
    state["index"] = who.repeat_interleave(case["run"])[:m].contiguous()
    state["x"] = torch.randn(m, hidden, generator=g, device=dev).to(dtype)
    state["a"] = (torch.randn(n, rank, hidden, generator=g, device=dev) / math.sqrt(hidden)).to(dtype)
    state["b"] = (torch.randn(n, tp * shard, rank, generator=g, device=dev) * 0.05).to(dtype)
    state["scale"] = 1.0 + torch.rand(n, generator=g, device=dev)  # alpha / rank
    # logits, or what a loss that was scaled for the type sends back
    sigma = 2.0 if case["op"] == "adapt" else 1e-3
    y = torch.empty(tp, m, shard, dtype=dtype, device=dev)
    for r in range(tp):
        y[r] = torch.randn(m, shard, generator=g, device=dev) * sigma
    state["y"] = y
    if case["op"] == "adapt":
        state["out"] = torch.empty_like(y)


def _prepare_select(case, state, g, dev):
    requests, count, vocab, tp, shard = (case[k] for k in ("requests", "beams", "vocab", "tp", "shard"))
    m, dtype = requests * count, TYPES[case["dtype"]]
    shape = (tp, m, shard) if tp else (m, vocab)
    z = torch.empty(shape, dtype=dtype, device=dev)
    rows = z.view(-1, shape[-1])
    for at in range(0, rows.shape[0], 64):
        part = rows[at:at + 64]
        part.copy_(torch.randn(part.shape, generator=g, device=dev) * 3.0)
    # banned tokens: half of them at minus infinity, half at the type's lowest value
    banned = torch.rand(shape[-1], generator=g, device=dev)
    z[..., banned < case["masked"] / 2] = -math.inf
    z[..., (banned >= case["masked"] / 2) & (banned < case["masked"])] = torch.finfo(dtype).min
    state["logits"] = z
    scores = -10.0 * torch.rand(requests, count, generator=g, device=dev)
    # a request's first step: all beams are the same, so the first alone counts
    first = torch.rand(requests, 1, generator=g, device=dev) < 0.1
    later = torch.arange(count, device=dev)[None, :] > 0
    state["scores"] = torch.where(first & later, -math.inf, scores)
    state["finished"] = torch.rand(requests, count, generator=g, device=dev) < case["finished"]
    state["pad"] = 2


def _prepare_reorder(case, state, g, dev):
    requests, count, dtype = case["requests"], case["beams"], TYPES[case["dtype"]]
    shape = (requests * count, case["outer"], case["steps"], case["width"])
    if dtype == torch.int64:
        state["states"] = [torch.randint(0, 163840, shape, generator=g, device=dev) for _ in range(case["count"])]
    else:
        state["states"] = [torch.empty(shape, dtype=dtype, device=dev).normal_(generator=g)
                           for _ in range(case["count"])]
    # the survivors keep their slots; the slots of the others take copies of them
    order = torch.rand(requests, count, generator=g, device=dev).argsort(dim=1)
    left = count - _lost(case)
    pick = torch.randint(0, left, (requests, count), generator=g, device=dev)
    place = torch.arange(count, device=dev)[None, :]
    parents = torch.empty(requests, count, dtype=torch.int64, device=dev)
    parents.scatter_(1, order, order.gather(1, torch.where(place < left, place, pick)))
    state["parents"] = parents
    state["lengths"] = None
    if case["lengths"]:
        share = case["lengths"] + (1.0 - case["lengths"]) * torch.rand(requests, generator=g, device=dev)
        state["lengths"] = (share * case["steps"]).long()


# ---------------------------------------------------------------------------------------------- one pass


def run(state):
    if own:
        return _own(state)
    if state["op"] == "select":
        return _select(state)
    if state["op"] == "reorder":
        return _reorder(state)
    return _adapt(state) if state["op"] == "adapt" else _adapt_grad(state)


def _own(state):
    """The calls that a user makes."""
    from tp_vocab_logits_amd import adapt, adapt_grad, beam_reorder, beam_select

    op = state["op"]
    if op == "select":
        return beam_select(state["logits"], state["scores"], state["keep"], vocab=state["vocab"], scale=state["scale"],
                           finished=state["finished"], pad=state["pad"])
    if op == "reorder":
        beam_reorder(state["states"], state["parents"], lengths=state["lengths"], time_dim=2)
        return state["states"]
    args = (state["x"], state["a"], state["b"], state["index"], state["tp"], state["shard"])
    if op == "adapt":
        return adapt(state["y"], *args, scale=state["scale"], out=state["out"])
    return adapt_grad(state["y"], *args, scale=state["scale"])


def _flat(state):
    """All adapters as one of n * rank columns, of which a row has its own ones: [n*rank, H], [V, n*rank], and the rows'
    factors [m, n*rank], 0 at the others' columns."""
    n, rank = state["n"], state["rank"]
    a = state["a"].float().reshape(n * rank, -1)
    b = state["b"].float().permute(1, 0, 2).reshape(-1, n * rank)
    mine = state["index"][:, None] == torch.arange(n, device=a.device)[None, :]
    return a, b, (mine * state["scale"]).repeat_interleave(rank, dim=1)


def _adapt(state):
    a, b, factor = _flat(state)
    more = ((state["x"].float() @ a.t()) * factor) @ b.t()
    more = more.view(state["m"], state["tp"], state["shard"]).transpose(0, 1)
    return (state["y"].float() + more).to(state["y"].dtype)


def _adapt_grad(state):
    a, b, factor = _flat(state)
    n, rank, dtype = state["n"], state["rank"], state["x"].dtype
    dy = state["y"].float().transpose(0, 1).reshape(state["m"], -1)
    x = state["x"].float()
    g = (dy @ b) * factor
    db = dy.t() @ ((x @ a.t()) * factor)
    db = db.view(-1, n, rank).permute(1, 0, 2).contiguous()
    return (g @ a).to(dtype), (g.t() @ x).view(n, rank, -1).to(dtype), db.to(dtype)


def _select(state):
    requests, count, vocab, keep = (state[k] for k in ("requests", "beams", "vocab", "keep"))
    m, scores, finished = requests * count, state["scores"], state["finished"]
    z = state["logits"]
    if state["tp"]:
        z = z.transpose(0, 1).reshape(m, -1)[:, :vocab]
    z = z.float() + 0.0  # (one zero)
    # a row's best, the first of equal ones: the logit's bits in the order of its value, then the place from behind
    bits = z.view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32
    order = order | (0xFFFFFFFF - torch.arange(vocab, device=z.device))
    least = min(keep, vocab)
    token = 0xFFFFFFFF - (order.topk(least, dim=1).values & 0xFFFFFFFF)
    wide = z.double() * state["scale"]
    top = wide.amax(dim=1, keepdim=True)
    lse = top + (wide - top).exp().sum(dim=1, keepdim=True).log()
    value = scores.reshape(m, 1).double() + (wide.gather(1, token) - lse)
    # a finished beam stands for itself, with the padding token
    done = finished.reshape(m, 1)
    alone = torch.arange(least, device=z.device)[None, :] == 0
    value = torch.where(done, torch.where(alone, scores.reshape(m, 1).double(), -math.inf), value)
    token = torch.where(done, state["pad"], token)
    value = torch.where(scores.reshape(m, 1).isfinite(), value, -math.inf)
    # over the request's beams: by the value, equal ones by their place
    beam = torch.arange(m, device=z.device)[:, None] % count
    place, value = (beam * vocab + token).view(requests, -1), value.view(requests, -1)
    place, by = place.sort(dim=1, stable=True)
    value, by = value.gather(1, by).sort(dim=1, descending=True, stable=True)
    place = place.gather(1, by)
    short = max(0, keep - value.shape[1])
    value = torch.nn.functional.pad(value[:, :keep], (0, short), value=-math.inf)
    place = torch.nn.functional.pad(place[:, :keep], (0, short))
    none = value == -math.inf
    return value.float(), torch.where(none, -1, place // vocab), torch.where(none, -1, place % vocab)


def _reorder(state):
    requests, count, steps = state["requests"], state["beams"], state["steps"]
    dev = state["parents"].device
    source = (state["parents"] + count * torch.arange(requests, device=dev)[:, None]).reshape(-1)
    if state["lengths"] is None:
        state["states"] = [t.copy_(t[source]) for t in state["states"]]
        return state["states"]
    live = torch.arange(steps, device=dev)[None, :] < state["lengths"].repeat_interleave(count)[:, None]
    live = live[:, None, :, None]
    state["states"] = [t.copy_(torch.where(live, t[source], t)) for t in state["states"]]
    return state["states"]


# ---------------------------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "select":
        return _exact_select(case, s)
    if case["op"] == "reorder":
        return _exact_reorder(case, s)
    tp, shard, hidden, m, n, rank = (case[k] for k in ("tp", "shard", "hidden", "m", "n", "rank"))
    dev = s["x"].device
    if case["op"] == "adapt":
        out = s["y"].double()
        for i in range(n):
            rows = torch.nonzero(s["index"] == i).squeeze(1)
            u = torch.mm(s["x"][rows].double(), s["a"][i].double().t()) * s["scale"][i].double()
            for r in range(tp):
                out[r, rows] += torch.mm(u, s["b"][i, r * shard:(r + 1) * shard].double().t())
        return out
    dx = torch.zeros(m, hidden, dtype=torch.float64, device=dev)
    da = torch.zeros(n, rank, hidden, dtype=torch.float64, device=dev)
    db = torch.zeros(n, tp * shard, rank, dtype=torch.float64, device=dev)
    for i in range(n):
        rows = torch.nonzero(s["index"] == i).squeeze(1)
        x, a, factor = s["x"][rows].double(), s["a"][i].double(), s["scale"][i].double()
        u = torch.mm(x, a.t()) * factor
        g = torch.zeros(rows.numel(), rank, dtype=torch.float64, device=dev)
        for r in range(tp):
            dy = s["y"][r, rows].double()
            g += torch.mm(dy, s["b"][i, r * shard:(r + 1) * shard].double())
            db[i, r * shard:(r + 1) * shard] = torch.mm(dy.t(), u)
        g *= factor
        dx[rows] = torch.mm(g, a)
        da[i] = torch.mm(g.t(), x)
    return dx, da, db


def _exact_select(case, s):
    requests, count, vocab, keep = (case[k] for k in ("requests", "beams", "vocab", "keep"))
    out = torch.full((requests, keep), -math.inf, dtype=torch.float64)
    parents = torch.full((requests, keep), -1, dtype=torch.int64)
    tokens = parents.clone()
    scores, finished = s["scores"].double().cpu(), s["finished"].cpu()
    for b in range(requests):
        rows = s["logits"][..., b * count:(b + 1) * count, :]
        if case["tp"]:
            rows = torch.cat(list(rows), dim=1)[:, :vocab]
        logp = torch.log_softmax(rows.double() * case["scale"], dim=1)
        for k in range(count):
            if not math.isfinite(scores[b, k]):
                logp[k] = -math.inf
            elif finished[b, k]:
                logp[k] = -math.inf
                logp[k, s["pad"]] = scores[b, k]
            else:
                logp[k] += scores[b, k]
        best, place = logp.reshape(-1).sort(descending=True, stable=True)
        real = best[:keep].cpu() > -math.inf
        got = int(real.sum())
        out[b, :got] = best[:got].cpu()
        parents[b, :got] = place[:got].cpu() // vocab
        tokens[b, :got] = place[:got].cpu() % vocab
    return out, parents, tokens


def _exact_reorder(case, s):
    parents = s["parents"].cpu().tolist()
    lengths = s["lengths"].cpu().tolist() if s["lengths"] is not None else [case["steps"]] * case["requests"]
    out = []
    for t in s["states"]:
        new = t.clone()
        for b, (row, length) in enumerate(zip(parents, lengths)):
            for k, p in enumerate(row):
                new[b * case["beams"] + k, :, :length] = t[b * case["beams"] + p, :, :length]
        out.append(new.double() if new.is_floating_point() else new)
    return out
