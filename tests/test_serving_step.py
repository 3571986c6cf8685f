"""A decode step of beam search with adapters as a serving program runs it: the
lookup, the head's product, the rows' adapters, the gather, the choice of
continuations and the reordering of the beams' states, eager and captured."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import adapters as oa
from oracle import beams as ob
from tp_vocab_logits_amd import HeadGather, adapt, beam_reorder, beam_select, embed
from tp_vocab_logits_amd.head_gather import lmhead

DEV = "cuda:0"
TP, SHARD, VOCAB, HIDDEN, RANK = 2, 256, 509, 64, 8
REQUESTS, BEAMS, STEPS, EOS = 3, 4, 12, 7
ROWS = REQUESTS * BEAMS


class Search:
    """One batch of searches: weights, states, and the step."""

    def __init__(self):
        g = torch.Generator().manual_seed(3)
        rand = lambda *shape: torch.randn(*shape, generator=g)  # noqa: E731
        self.w = (rand(TP * SHARD, HIDDEN) * 0.3).bfloat16().to(DEV)
        self.a = (rand(3, RANK, HIDDEN) / 8).bfloat16().to(DEV)
        self.b = (rand(3, TP * SHARD, RANK) * 0.3).bfloat16().to(DEV)
        self.scale = torch.tensor([0.5, 1.0, 2.0], device=DEV)
        self.index = torch.tensor([0, -1, 2], device=DEV).repeat_interleave(BEAMS)  # one adapter (or none) a request
        self.gather = HeadGather(TP, SHARD, ROWS, DEV, vocab=VOCAB)
        self.gather.set_device_parity(True)
        self.tokens = torch.full((ROWS,), 1, device=DEV)
        self.scores = torch.full((REQUESTS, BEAMS), -torch.inf, device=DEV)
        self.scores[:, 0] = 0.0
        self.finished = torch.zeros(REQUESTS, BEAMS, dtype=torch.bool, device=DEV)
        self.lengths = torch.zeros(REQUESTS, dtype=torch.int64, device=DEV)
        self.history = torch.full((ROWS, STEPS), -1, device=DEV)
        self.cache = torch.zeros(ROWS, 2, STEPS, HIDDEN, device=DEV, dtype=torch.bfloat16)
        self.out = {}

    def step(self):
        h = embed(self.tokens, self.w, TP, SHARD)
        position = self.lengths.repeat_interleave(BEAMS)
        self.cache.scatter_(2, position.view(-1, 1, 1, 1).expand(-1, 2, 1, HIDDEN), h.view(-1, 1, 1, HIDDEN).expand(-1, 2, 1, HIDDEN))
        live = torch.arange(STEPS, device=DEV)[None, :] <= position[:, None]
        x = (self.cache[:, 0].float() * live[..., None]).sum(1).mul(0.5).bfloat16()  # a body of its own
        plain = lmhead(x, self.w, TP, SHARD)
        shards = adapt(plain, x, self.a, self.b, self.index, TP, SHARD, scale=self.scale)
        logits = self.gather(shards)
        scores, parents, tokens = beam_select(logits, self.scores, BEAMS, finished=self.finished, pad=EOS)
        also = beam_select(shards, self.scores, BEAMS, vocab=VOCAB, finished=self.finished, pad=EOS)
        self.out = {"x": x, "plain": plain, "shards": shards, "logits": logits, "before": self.scores.clone(),
                    "done": self.finished.clone(), "chosen": (scores, parents, tokens), "also": also}
        beam_reorder([self.cache[:, 0], self.cache[:, 1]], parents, self.lengths + 1, time_dim=1)
        beam_reorder(self.history, parents, self.lengths, time_dim=1)
        self.history.scatter_(1, position[:, None], tokens.view(-1, 1))
        self.finished.copy_(self.finished.gather(1, parents.clamp(min=0)) | (tokens == EOS))
        self.scores.copy_(scores)
        self.tokens.copy_(tokens.view(-1))
        self.lengths.add_(1)


def check(s: Search, texts, caches):
    """The last step against the oracles, from the step's own inputs; texts and caches are the host's copies."""
    o = {k: (tuple(t.cpu() for t in v) if isinstance(v, tuple) else v.cpu()) for k, v in s.out.items()}
    flat = lambda t: t.double().transpose(0, 1).reshape(ROWS, -1).numpy()  # noqa: E731
    want, bound = oa.adapt_bound(flat(o["plain"]), o["x"].double().numpy(), s.a.cpu().double().numpy(),
                                 s.b.cpu().double().numpy(), s.index.cpu().numpy(), s.scale.cpu().double().numpy(), "bf16")
    assert (np.abs(flat(o["shards"]) - want) <= bound).all()
    assert np.array_equal(o["logits"].double().numpy(), flat(o["shards"])[:, :VOCAB])
    logits = o["logits"].double().numpy().reshape(REQUESTS, BEAMS, VOCAB)
    scores, parents, tokens = ob.beam_select(logits, o["before"].double().numpy(), BEAMS, o["done"].numpy(), EOS)
    for got in (o["chosen"], o["also"]):
        assert np.array_equal(got[1].numpy(), parents) and np.array_equal(got[2].numpy(), tokens)
        np.testing.assert_allclose(got[0].numpy(), scores, rtol=2.0 ** -24, atol=1e-9)
    for q in range(REQUESTS):
        rows = [texts[q * BEAMS + max(0, p)] + [int(t)] for p, t in zip(parents[q], tokens[q])]
        texts[q * BEAMS:(q + 1) * BEAMS] = rows
    length = len(texts[0])
    assert s.history[:, :length].cpu().tolist() == texts and (s.history[:, length:] == -1).all()
    caches[:] = [list(c) for c in caches]
    for q in range(REQUESTS):
        old = [caches[q * BEAMS + k] for k in range(BEAMS)]
        for k, p in enumerate(parents[q]):
            caches[q * BEAMS + k] = list(old[max(0, p)])


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_search_with_adapters(captured):
    print(f"[gpu] search captured={captured}", flush=True)
    s = Search()
    texts, caches = [[] for _ in range(ROWS)], [[] for _ in range(ROWS)]
    graph = None
    for k in range(STEPS):
        entered = [[*c, int(t)] for c, t in zip(caches, s.tokens.tolist())]  # what this step's cache gets
        caches[:] = entered
        if graph is not None:
            graph.replay()
            torch.cuda.synchronize()
        else:
            s.step()
        check(s, texts, caches)
        # every row's cache is the rows of W of the tokens that it went through
        for r in range(ROWS):
            want = s.w[torch.tensor(caches[r], device=DEV)]
            assert torch.equal(s.cache[r, 0, :k + 1], want) and torch.equal(s.cache[r, 1, :k + 1], want)
        if captured and k == 1:
            # captured once the searches are under way; capturing runs nothing
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                s.step()
