"""A small decoder of MoE blocks that answers prompts by beam search, with the
library's operators of a decode step.

The prompts run through the model at once and their keys and values are written
into pages (moe_cache_write). Then, token by token: the best continuations of
each prompt's beams (moe_beam_select); the page table that goes on from them
(moe_cache_fork: beams that are dropped free their pages, beams that split share
theirs and copy the one that both would write, moe_cache_copy); and the model on
the new tokens, whose keys and values go into the cache as its attention reads
it (moe_attention_decode, moe_layer). Finally the pool is compacted.

    python examples/beam_decode.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import padded_permute_combine_gb300 as p  # noqa: E402


class Decoder:
    """x += attention(norm(x)); x += MoE(norm(x)) for each layer, logits = norm(x) head^T."""

    def __init__(self, layers=2, hidden=64, heads=4, kv_heads=2, dim=16, ffn=48, experts=4, top_k=2, vocab=97, seed=0,
                 device="cuda", dtype=torch.float32):
        g = torch.Generator().manual_seed(seed)
        new = lambda *s: (torch.randn(s, generator=g) * s[-1] ** -0.5).to(device, dtype)  # noqa: E731
        self.heads, self.kv_heads, self.dim, self.top_k = heads, kv_heads, dim, top_k
        self.embedding, self.head = new(vocab, hidden) * 8, new(vocab, hidden) * 2
        self.norm = torch.ones(hidden, device=device, dtype=dtype)
        self.layers = [{"qkv": new((heads + 2 * kv_heads) * dim, hidden) * 2, "o": new(hidden, heads * dim),
                        "router": new(experts, hidden) * 2, "gate_up": new(experts, 2 * ffn, hidden),
                        "down": new(experts, hidden, ffn)} for _ in range(layers)]

    def qkv(self, w, x):
        h, _, _ = p.moe_layer_norm_fwd(x, self.norm)
        return (h @ w["qkv"].t()).view(x.shape[0], -1, self.dim).split([self.heads, self.kv_heads, self.kv_heads], 1)

    def after(self, w, x, attended):
        x = x + attended.reshape(x.shape[0], -1) @ w["o"].t()
        h, _, _ = p.moe_layer_norm_fwd(x, self.norm)
        y, _, _ = p.moe_layer(h, w["router"], w["gate_up"], w["down"], self.top_k)
        return x + y

    def logits(self, x):
        return p.moe_layer_norm_fwd(x, self.norm)[0] @ self.head.t()

    def prefill(self, tokens, offsets, caches, table, lengths):
        """All prompts' tokens, one prompt after another; logits of each prompt's last one."""
        x = self.embedding[tokens]
        ends = offsets.tolist()
        for w, (kc, vc) in zip(self.layers, caches):
            q, k, v = self.qkv(w, x)
            p.moe_cache_write(k, v, kc, vc, table, offsets, lengths)
            parts = []
            for a, b in zip(ends, ends[1:]):
                one = [t[None, a:b].transpose(1, 2) for t in (q, k, v)]
                parts.append(torch.nn.functional.scaled_dot_product_attention(*one, is_causal=True, enable_gqa=True)[0].transpose(0, 1))
            x = self.after(w, x, torch.cat(parts))
        return self.logits(x[offsets[1:].long() - 1])

    def step(self, tokens, caches, table, lengths):
        """One new token of every row; lengths count it."""
        x = self.embedding[tokens]
        for w, (kc, vc) in zip(self.layers, caches):
            q, k, v = self.qkv(w, x)
            x = self.after(w, x, p.moe_attention_decode(q, kc, vc, table, lengths, k, v)[0])
        return self.logits(x)


@torch.no_grad()
def beam_search(model: Decoder, prompts: list[list[int]], beams: int, steps: int, end_token: int, page_size: int = 4,
                num_pages: int = 256) -> dict:
    dev = model.embedding.device
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    B, W = len(prompts), beams
    shape = (len(model.layers), 2, num_pages, page_size, model.kv_heads, model.dim)
    pool = torch.zeros(shape, device=dev, dtype=model.embedding.dtype)
    caches = [(layer[0], layer[1]) for layer in pool]
    pages = list(pool.flatten(0, 1).unbind(0))
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    # Empty rows with room for the prompts, then for every step: one table is wide enough for all.
    width = -(-(max(map(len, prompts)) + steps) // page_size) + 1
    counts = [len(t) for t in prompts]
    table, lengths = torch.full((B, width), -1, dtype=torch.int32, device=dev), i32([0] * B)
    table = p.moe_cache_fork(table, lengths, i32(list(range(B))), page_size, num_pages, max(counts), status=status).page_table
    lengths = i32(counts)
    offsets = i32([sum(counts[:i]) for i in range(B + 1)])
    first = model.prefill(torch.tensor(sum(prompts, []), device=dev), offsets, caches, table, lengths)
    # Every beam begins as its prompt's; only the first counts until they differ.
    table, lengths, _, _ = p.moe_cache_fork(table, lengths, i32([b for b in range(B) for _ in range(W)]), page_size, num_pages, 0)
    logits = first[:, None].expand(B, W, -1).contiguous()
    scores = torch.full((B, W), -torch.inf, device=dev)
    scores[:, 0] = 0.0
    ended = torch.zeros((B, W), dtype=torch.bool, device=dev)
    tokens = torch.zeros((B * W, 0), dtype=torch.int64, device=dev)
    for step in range(steps):
        scores, parents, chosen = p.moe_beam_select(logits, scores, W, ended, end_token)
        from_row = parents.flatten().long()
        tokens = torch.cat([tokens[from_row], chosen.flatten().long()[:, None]], 1)
        ended = ended.flatten()[from_row].view(B, W) | (chosen == end_token)
        if step == steps - 1:
            break
        table, lengths, src, dst = p.moe_cache_fork(table, lengths, parents.flatten(), page_size, num_pages, status=status)
        p.moe_cache_copy(pages, src, dst)
        lengths = lengths + 1
        fed = tokens[:, -1]
        logits = model.step(fed, caches, table, lengths).view(B, W, -1)
    moved = p.moe_cache_compact(table, lengths, page_size, num_pages)
    p.moe_cache_copy(pages, moved.src, moved.dst, moved.count)
    again = model.step(fed, caches, moved.page_table, lengths).view(B, W, -1) if steps > 1 else logits
    return {"tokens": tokens.view(B, W, -1).tolist(), "scores": scores.tolist(), "status": int(status),
            "moved": int(moved.count), "compacted": float((again - logits).abs().max())}


def main():
    r = beam_search(Decoder(seed=22), [[5, 17, 80, 3, 41], [9], [60, 61, 62, 63, 64, 65, 66, 67, 68]], 3, 12, 7)
    for b, (beams, scores) in enumerate(zip(r["tokens"], r["scores"])):
        for t, s in zip(beams, scores):
            print("prompt %d  %8.4f  %s" % (b, s, t))
    print("pages moved by the compaction:", r["moved"], "  the step repeated on the compacted pool differs by", r["compacted"])
    return r


if __name__ == "__main__":
    main()
