"""The operators of a decode step together, as examples/beam_decode.py uses
them: beam search over a cache in pages gives the hypotheses and scores of a
plain beam search that keeps no cache and runs the whole model on every
hypothesis in 64 bits.

The seed is one whose choices are clear: in the plain search every total differs
from the next, and every router's second logit from the third, by more than 1e-2, against 32-bit sums of some hundred terms of order one (errors
of some 1e-5, added up over 12 steps)."""
import math
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

PROMPTS = [[5, 17, 80, 3, 41], [9], [60, 61, 62, 63, 64, 65, 66, 67, 68]]
BEAMS, STEPS, END, SEED = 3, 12, 7, 22


def norm(x):
    d = x - x.mean(-1, keepdim=True)
    return d / torch.sqrt(d.square().mean(-1, keepdim=True) + 1e-5)


def plain_logits(model, tokens, gaps):
    """Logits behind the last of tokens, everything from the start, in 64 bits."""
    H, KV, D, n = model.heads, model.kv_heads, model.dim, len(tokens)
    x = model.embedding.double().cpu()[tokens]
    mask = torch.full((n, n), -math.inf, dtype=torch.float64).triu(1)
    for w in model.layers:
        w = {k: v.double().cpu() for k, v in w.items()}
        q, k, v = (norm(x) @ w["qkv"].t()).view(n, -1, D).split([H, KV, KV], 1)
        k, v = (t.repeat_interleave(H // KV, 1) for t in (k, v))
        p = torch.softmax(torch.einsum("qhd,khd->hqk", q, k) * D ** -0.5 + mask, 2)
        x = x + torch.einsum("hqk,khd->qhd", p, v).reshape(n, -1) @ w["o"].t()
        h = norm(x)
        logits = h @ w["router"].t()
        top = torch.sort(logits, 1, descending=True)
        gaps.append(float((top.values[:, model.top_k - 1] - top.values[:, model.top_k]).min()))
        share = torch.softmax(logits, 1).gather(1, top.indices[:, : model.top_k])
        share = share / share.sum(1, keepdim=True)
        y = torch.zeros_like(x)
        for t in range(n):
            for s, e in zip(share[t], top.indices[t]):
                g, u = (w["gate_up"][e] @ h[t]).chunk(2)
                y[t] += s * (w["down"][e] @ (g * torch.sigmoid(g) * u))
        x = x + y
    return norm(x[-1]) @ model.head.double().cpu().t()


def plain_search(model):
    found, gaps = [], []
    for prompt in PROMPTS:
        beams = [([], 0.0, False)]
        for _ in range(STEPS):
            every = []
            for hyp, score, ended in beams:
                if ended:
                    every.append((score, hyp + [END], True))
                    continue
                logp = torch.log_softmax(plain_logits(model, prompt + hyp, gaps), 0)
                every += [(score + float(lp), hyp + [t], t == END) for t, lp in enumerate(logp)]
            every.sort(key=lambda e: -e[0])
            gaps += [a[0] - b[0] for a, b in zip(every[:BEAMS], every[1:BEAMS + 1])]
            beams = [(h, s, e) for s, h, e in every[:BEAMS]]
        found.append(beams)
    return found, min(gaps)


def decoder(device, seed=SEED):
    from beam_decode import Decoder

    return Decoder(seed=seed, device=device)


@pytest.mark.gpu
@pytest.mark.parametrize("page_size", [4, 1, 7])
def test_beam_search_over_pages_equals_the_plain_search(page_size):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from beam_decode import beam_search

    model = decoder("cuda")
    r = beam_search(model, PROMPTS, BEAMS, STEPS, END, page_size)
    want, gap = plain_search(model)
    assert gap > 1e-2
    for b, beams in enumerate(want):
        assert r["tokens"][b] == [h for h, _, _ in beams]
        assert all(abs(got - s) < 1e-3 for got, (_, s, _) in zip(r["scores"][b], beams))
    assert r["status"] == 0 and r["compacted"] < 1e-3


@pytest.mark.gpu
def test_the_example_runs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import beam_decode

    r = beam_decode.main()
    assert r["status"] == 0 and all(math.isfinite(s) for row in r["scores"] for s in row)
