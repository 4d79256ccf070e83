"""What is measured of the operators of a decode step around the MoE layer:
attention of one new token over a paged key-value cache, the write of a
prompt's keys and values into it, the moves of its pages (beams that fork,
sequences that end, a pool that is compacted) and beam search's selection.

Each case runs in one of two forms on the same inputs: the plain form
(elementary torch operations, in 64 bits where the order of near totals
decides, otherwise in 32, rounded once at the end) or, with ``own`` set, the
calls that a user makes of the package.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _attend(name, seqs, mean, heads, kv_heads, dim, page, dtype, layout="tokens", window=0):
    """``seqs`` sequences whose lengths are spread around ``mean``; ``layout``: whether a page holds its tokens' heads
    one after another ("tokens") or its heads' tokens ("heads")."""
    return {"name": name, "op": "attend", "seqs": seqs, "mean": mean, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "dtype": dtype, "layout": layout, "window": window}


def _write(name, seqs, tokens, kv_heads, dim, page, dtype, layout="tokens"):
    return {"name": name, "op": "write", "seqs": seqs, "tokens": tokens, "kv_heads": kv_heads, "dim": dim, "page": page,
            "dtype": dtype, "layout": layout}


def _pages(name, op, requests, beams, mean, page, row, caches, dtype, room=1.3):
    """``requests`` of ``beams`` rows each around ``mean`` tokens long; a page holds ``page`` tokens of ``row`` elements
    in each of ``caches`` tensors; the pool has ``room`` times the pages in use."""
    return {"name": name, "op": op, "requests": requests, "beams": beams, "mean": mean, "page": page, "row": row,
            "caches": caches, "dtype": dtype, "room": room}


def _select(name, requests, beams, vocab, num_out, dtype, ended):
    return {"name": name, "op": "select", "requests": requests, "beams": beams, "vocab": vocab, "num_out": num_out,
            "dtype": dtype, "ended": ended}


def listed():
    return [
        # A single request, a short chat so far: latency alone.
        _attend("attend 1 sequence of 200", 1, 200, 32, 8, 128, 16, "bf16"),
        # A serving batch of the Mixtral-8x7B shape: 64 requests of 300 to 8000 tokens each.
        _attend("attend 64 ragged sequences", 64, 2500, 32, 8, 128, 16, "bf16"),
        # Two long documents on the Mixtral-8x22B heads: few rows, a long axis.
        _attend("attend 2 sequences of 131072", 2, 131072, 48, 8, 128, 64, "bf16", "heads"),
        # fp32 with an odd head size, pages that end inside any tile and a sliding window.
        _attend("attend 9 odd sequences fp32", 9, 3001, 12, 4, 72, 13, "fp32", "tokens", 1777),
        # The prompts of a batch, one after another, into their pages.
        _write("write 16 prompts", 16, 32768, 8, 128, 16, "bf16"),
        # A few odd pieces of prompts in fp32.
        _write("write 5 odd pieces fp32", 5, 777, 4, 72, 13, "fp32", "heads"),
        # One step of a few requests' beams on one layer: latency of the table's kernel and a few pages.
        _pages("fork 4 requests of 4 beams", "fork", 4, 4, 500, 16, 1024, 2, "bf16"),
        # One step of 64 requests' beams over eight layers' keys and values.
        _pages("fork 64 requests of 4 beams", "fork", 64, 4, 400, 16, 1024, 16, "bf16"),
        # A small pool, after half of it was freed.
        _pages("compact a small pool", "compact", 16, 1, 700, 16, 1024, 2, "bf16", 2.0),
        # A large pool of two layers, after half of it was freed.
        _pages("compact 2 layers", "compact", 128, 1, 1000, 16, 1024, 4, "bf16", 2.0),
        # Three requests of five beams over an odd vocabulary in fp32, some beams at their end.
        _select("select 3 requests of 5 beams", 3, 5, 50257, 10, "fp32", True),
        # A batch of 64 requests of 8 beams over the DeepSeek-V3 vocabulary.
        _select("select 64 requests of 8 beams", 64, 8, 129280, 16, "bf16", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "write", "fork", "compact", "select", "select"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    layout = rng.choice(["tokens", "tokens", "heads"])
    page = rng.choice([1, 8, 16, 16, 16, 32, 64, 128, rng.randint(2, 100)])
    if op == "attend":
        kv_heads, group = rng.choice([1, 2, 3, 4, 8, 8, 8, 16]), rng.choice([1, 2, 3, 4, 4, 6, 7, 8, 12, 16, 24])
        dim = rng.choice([64, 80, 96, 128, 128, 128, 192, 256, rng.randint(16, 256)])
        seqs = _log(rng, 1, 256)
        most = (1 << 27) // (seqs * kv_heads * dim * (2 if dtype == "fp32" else 1))
        mean = _log(rng, 1, max(2, min(131072, most)))
        window = rng.choice([0, 0, 0, rng.randint(1, 2 * mean)])
        return _attend("drawn", seqs, mean, kv_heads * group, kv_heads, dim, page, dtype, layout, window)
    if op == "write":
        kv_heads, dim = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128, 128, 256, rng.randint(16, 256)])
        tokens = _log(rng, 1, max(2, (1 << 25) // (kv_heads * dim * (2 if dtype == "fp32" else 1))))
        return _write("drawn", _log(rng, 1, 64), tokens, kv_heads, dim, page, dtype, layout)
    if op in ("fork", "compact"):
        page, row = rng.choice([8, 16, 16, 32, rng.randint(3, 64)]), rng.choice([128, 512, 1024, 576, rng.randint(1, 1100)])
        requests, beams = _log(rng, 1, 64), rng.choice([1, 2, 4, 5, 8])
        caches = rng.choice([1, 2, 2, 8, 16])
        while requests * beams * page * row * caches > 1 << 26:
            requests, caches = max(1, requests // 2), max(1, caches // 2)
        most = (1 << 28) // (requests * beams * row * caches)
        return _pages("drawn", op, requests, beams, _log(rng, 4, max(5, min(2000, most))), page, row, caches, dtype,
                      rng.uniform(1.2, 3.0))
    requests, beams = _log(rng, 1, 64), rng.randint(1, 12)
    vocab = rng.choice([32000, 50257, 65536, 129280, rng.randint(1000, 150000)])
    while requests * beams * vocab * (2 if dtype == "fp32" else 1) > 64 * 8 * 129280:
        requests = max(1, requests // 2)
    return _select("drawn", requests, beams, vocab, rng.randint(1, 2 * beams), dtype, rng.random() < 0.3)


def _spread(n, mean, factor=2.0):
    """n lengths between mean / factor and mean * factor, the same for every seed."""
    if n == 1:
        return [mean]
    return [max(1, int(mean * factor ** (2.0 * ((i * 0.61803398875 + 0.1) % 1.0) - 1.0))) for i in range(n)]


def _lengths(case):
    """The sequences' lengths: within a factor of five of the mean where there are many, equal where there are two, and
    one empty sequence among eight or more."""
    n = case["seqs"]
    got = _spread(n, case["mean"], 5.0 if n > 2 else 1.0)
    if n >= 8:
        got[n // 2] = 0
    return got


def _counts(case):
    """Tokens that a write brings of each sequence, one of them none where there are several, and what it has already."""
    n, total = case["seqs"], case["tokens"]
    share = _spread(n, 1000, 3.0)
    if n > 2:
        share[n // 2] = 0
    got = [total * s // sum(share) for s in share]
    got[0] += total - sum(got)
    return got, [(i * 37) % (3 * case["page"]) for i in range(n)]


def _beams(case):
    """Rows' lengths, page numbers (of a pool in order) and parents. The beams of a request have its prompt's full pages
    in common and their own from there on; a request in eight has ended, and its rows' parents are -1."""
    R, W, page = case["requests"], case["beams"], case["page"]
    lengths, rows, parents, used = [], [], [], 0
    for q, n in enumerate(_spread(R, case["mean"])):
        common = int(n * 0.8) // page if W > 1 else 0
        prompt = list(range(used, used + common))
        used += common
        for w in range(W):
            own_pages = -(-n // page) - common
            rows.append(prompt + list(range(used, used + own_pages)))
            used += own_pages
            lengths.append(n)
            parents.append(-1 if q % 8 == 5 else q * W + (w * (w + q % 3)) % W)
    return lengths, rows, parents, used


def _width(case):
    return -(-2 * case["mean"] // case["page"]) + 2


def _rand(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(scale)


def _table(gen, counts, pool, width):
    """A page table whose rows name counts[i] distinct pages of the pool, and -1 behind them."""
    ids = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device="cuda")
    n = torch.tensor(counts, device="cuda")
    held = torch.arange(width, device="cuda") < n[:, None]
    table[held] = ids[: sum(counts)]
    return table


def _cache(gen, case, pool):
    """Keys or values of the pool's pages, as [pages, page, kv_heads, dim] whatever the layout."""
    page, heads, dim = case["page"], case["kv_heads"], case["dim"]
    shape = (pool, page, heads, dim) if case["layout"] == "tokens" else (pool, heads, page, dim)
    t = _rand(gen, shape, DTYPES[case["dtype"]])
    return t if case["layout"] == "tokens" else t.transpose(1, 2)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if case["op"] == "attend":
        lengths = _lengths(case)
        counts = [-(-n // case["page"]) for n in lengths]
        pool = sum(counts) + 3
        s["host_lengths"], s["lengths"] = lengths, i32(lengths)
        s["page_table"] = _table(gen, counts, pool, max(counts) + 2)
        s["k_cache"], s["v_cache"] = _cache(gen, case, pool), _cache(gen, case, pool)
        # Queries whose scores have a deviation of about two: some keys matter more than others.
        s["q"] = _rand(gen, (case["seqs"], case["heads"], case["dim"]), torch.float32, 2.0).to(dt)
        s["k_new"] = _rand(gen, (case["seqs"], case["kv_heads"], case["dim"]), dt)
        s["v_new"] = _rand(gen, (case["seqs"], case["kv_heads"], case["dim"]), dt)
        return s
    if case["op"] == "write":
        counts, before = _counts(case)
        lengths = [a + b for a, b in zip(counts, before)]
        pages = [-(-n // case["page"]) for n in lengths]
        pool = sum(pages) + 3
        offsets = [sum(counts[:i]) for i in range(len(counts) + 1)]
        s["host"] = (counts, before, offsets)
        s["lengths"], s["offsets"] = i32(lengths), i32(offsets)
        s["page_table"] = _table(gen, pages, pool, max(pages) + 2)
        s["k_cache"], s["v_cache"] = _cache(gen, case, pool), _cache(gen, case, pool)
        s["k"] = _rand(gen, (case["tokens"], case["kv_heads"], case["dim"]), dt)
        s["v"] = _rand(gen, (case["tokens"], case["kv_heads"], case["dim"]), dt)
        return s
    if case["op"] in ("fork", "compact"):
        lengths, rows, parents, used = _beams(case)
        pool = int(used * case["room"]) + 4 + 2 * len(rows)
        ids = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32).cpu()
        table = torch.full((len(rows), _width(case)), -1, dtype=torch.int32)
        for r, row in enumerate(rows):
            table[r, : len(row)] = ids[torch.tensor(row, dtype=torch.int64)]
        s["num_pages"], s["page_table"], s["lengths"], s["parents"] = pool, table.cuda(), i32(lengths), i32(parents)
        # One tensor for all layers' keys and values, each a slice of it.
        s["pool"] = _rand(gen, (case["caches"], pool, case["page"], case["row"]), dt)
        s["caches"] = list(s["pool"].unbind(0))
        return s
    R, W, V = case["requests"], case["beams"], case["vocab"]
    s["logits"] = _rand(gen, (R, W, V), torch.float32, 2.5).to(dt)
    s["scores"] = _rand(gen, (R, W), torch.float32, 1.0).sub_(20.0)
    s["ended"] = (torch.rand((R, W), generator=gen, device="cuda") < 0.25) if case["ended"] else None
    s["end_token"] = 2
    return s


def _own(s):
    import padded_permute_combine_gb300 as p

    c = s["case"]
    if c["op"] == "attend":
        out, lse = p.moe_attention_decode(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lengths"], s["k_new"],
                                          s["v_new"], window=c["window"])
        return out, lse, s["k_cache"], s["v_cache"]
    if c["op"] == "write":
        p.moe_cache_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["offsets"], s["lengths"])
        return s["k_cache"], s["v_cache"]
    if c["op"] == "fork":
        table, lengths, src, dst = p.moe_cache_fork(s["page_table"], s["lengths"], s["parents"], c["page"], s["num_pages"])
        p.moe_cache_copy(s["caches"], src, dst)
        return table, lengths, src, dst, s["pool"]
    if c["op"] == "compact":
        table, src, dst, count = p.moe_cache_compact(s["page_table"], s["lengths"], c["page"], s["num_pages"])
        p.moe_cache_copy(s["caches"], src, dst, count)
        return table, src, dst, count, s["pool"]
    return p.moe_beam_select(s["logits"], s["scores"], c["num_out"], s["ended"], s["end_token"])


def _plain_attend(s):
    c = s["case"]
    q, page, heads, kv = s["q"].float(), c["page"], c["heads"], c["kv_heads"]
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, device=q.device)
    for b, n in enumerate(s["host_lengths"]):
        if n == 0:
            continue
        at = s["page_table"][b, (n - 1) // page].long()
        s["k_cache"][at, (n - 1) % page] = s["k_new"][b]
        s["v_cache"][at, (n - 1) % page] = s["v_new"][b]
        first = max(0, n - c["window"]) if c["window"] else 0
        ids = s["page_table"][b, first // page : -(-n // page)].long()
        skip = first - first // page * page
        k = s["k_cache"][ids].float().flatten(0, 1)[skip : skip + n - first].transpose(0, 1)  # [kv_heads, tokens, dim]
        v = s["v_cache"][ids].float().flatten(0, 1)[skip : skip + n - first].transpose(0, 1)
        x = torch.matmul(q[b].view(kv, heads // kv, -1), k.transpose(1, 2)) * c["dim"] ** -0.5
        m = x.amax(2, keepdim=True)
        e = torch.exp(x - m)
        z = e.sum(2, keepdim=True)
        out[b] = (torch.matmul(e, v) / z).view(heads, -1)
        lse[b] = (m + torch.log(z)).view(heads)
    return out.to(s["q"].dtype), lse, s["k_cache"], s["v_cache"]


def _plain_fork(s):
    c = s["case"]
    page, table, parents = c["page"], s["page_table"], s["parents"].long()
    R, P = parents.numel(), table.shape[1]
    row = torch.arange(R, device=table.device)
    length = torch.where(parents >= 0, s["lengths"][parents.clamp(min=0)], 0)
    held = (length + page - 1) // page
    col = torch.arange(P, device=table.device)
    got = torch.where(col < held[:, None], table[parents.clamp(min=0)], -1)
    used = torch.zeros(s["num_pages"], dtype=torch.bool, device=table.device)
    used[got[got >= 0].long()] = True
    # The last page of a row that is not full: the first row that holds it keeps it, the others copy it.
    partial = (length % page != 0) & (parents >= 0)
    last = got.gather(1, (held - 1).clamp(min=0)[:, None].long())[:, 0]
    same = (last[:, None] == last) & partial[:, None] & partial
    copies = partial & (torch.where(same, row, R).amin(1) < row)
    need = torch.where(parents >= 0, (length + 1 + page - 1) // page - held, 0) + copies
    start = torch.cumsum(need, 0) - need
    free = torch.nonzero(~used)[:, 0]
    first = held - copies.long()
    fresh = (col >= first[:, None]) & (col < (first + need)[:, None])
    rank = start[:, None] + col - first[:, None]
    got = torch.where(fresh, free[rank.clamp(0, free.numel() - 1)].to(torch.int32), got)
    dst = torch.where(copies, got.gather(1, (held - 1).clamp(min=0)[:, None].long())[:, 0], -1)
    src = torch.where(copies, last, -1)
    a, b = src[copies].long(), dst[copies].long()
    for t in s["caches"]:
        t[b] = t[a]
    return got, length.to(torch.int32), src, dst, s["pool"]


def _plain_compact(s):
    c, table, N = s["case"], s["page_table"], s["num_pages"]
    held = (s["lengths"] + c["page"] - 1) // c["page"]
    got = torch.where(torch.arange(table.shape[1], device=table.device) < held[:, None], table, -1)
    used = torch.zeros(N, dtype=torch.bool, device=table.device)
    used[got[got >= 0].long()] = True
    live = int(used.sum())
    a, b = torch.nonzero(used[live:])[:, 0] + live, torch.nonzero(~used[:live])[:, 0]
    now = torch.arange(N, device=table.device, dtype=torch.int32)
    now[a] = b.to(torch.int32)
    got = torch.where(got >= 0, now[got.clamp(min=0).long()], got)
    src, dst = (torch.full((N // 2,), -1, dtype=torch.int32, device=table.device) for _ in range(2))
    src[: a.numel()], dst[: a.numel()] = a.to(torch.int32), b.to(torch.int32)
    for t in s["caches"]:
        t[b] = t[a]
    return got, src, dst, torch.full((1,), a.numel(), dtype=torch.int32, device=table.device), s["pool"]


def _plain_select(s):
    c, V = s["case"], s["case"]["vocab"]
    x = s["logits"].double()
    m = x.amax(2, keepdim=True)
    total = s["scores"].double()[:, :, None] + (x - (m + torch.log(torch.exp(x - m).sum(2, keepdim=True))))
    if s["ended"] is not None:  # a beam at its end goes on with the end's token alone, at the score that it has
        total = total.masked_fill(s["ended"][:, :, None], -math.inf)
        total[:, :, s["end_token"]] = torch.where(s["ended"], s["scores"].double(), total[:, :, s["end_token"]])
    top = torch.sort(total.flatten(1), dim=1, descending=True, stable=True)
    score, at = top.values[:, : c["num_out"]], top.indices[:, : c["num_out"]]
    row = at // V + torch.arange(c["requests"], device=at.device)[:, None] * c["beams"]
    some = score > -math.inf  # fewer candidates than are asked for: -1 in the place of the others
    return score.float(), torch.where(some, row, -1).to(torch.int32), torch.where(some, at % V, -1).to(torch.int32)


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    if op == "attend":
        return _plain_attend(s)
    if op == "fork":
        return _plain_fork(s)
    if op == "compact":
        return _plain_compact(s)
    if op == "select":
        return _plain_select(s)
    page, (counts, before, offsets) = s["case"]["page"], s["host"]
    for b, n in enumerate(counts):
        if n:
            pos = torch.arange(before[b], before[b] + n, device="cuda")
            ids = s["page_table"][b][pos // page].long()
            s["k_cache"][ids, pos % page] = s["k"][offsets[b] : offsets[b] + n]
            s["v_cache"][ids, pos % page] = s["v"][offsets[b] : offsets[b] + n]
    return s["k_cache"], s["v_cache"]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "attend":
        seen = [min(n, case["window"]) if case["window"] else n for n in _lengths(case)]
        rows, table = 2 * case["seqs"] * case["heads"] * case["dim"], sum(-(-n // case["page"]) for n in seen)
        new = 4 * case["seqs"] * case["kv_heads"] * case["dim"]  # read, and written to the cache
        return {"bytes": e * (2 * sum(seen) * case["kv_heads"] * case["dim"] + rows + new) + 4 * (table + case["seqs"] * (1 + case["heads"])),
                "flops": 4 * sum(seen) * case["heads"] * case["dim"]}
    if case["op"] == "write":
        return {"bytes": 4 * e * case["tokens"] * case["kv_heads"] * case["dim"] + 8 * case["seqs"], "flops": 0}
    if case["op"] in ("fork", "compact"):
        lengths, rows, parents, used = _beams(case)
        P, R, N = _width(case), len(rows), int(used * case["room"]) + 4 + 2 * len(rows)
        size = e * case["page"] * case["row"] * case["caches"]
        if case["op"] == "fork":
            taken = sorted(p for p in parents if p >= 0 and lengths[p] % case["page"])
            moved = len(taken) - len(set(taken))  # every child of a row but the first copies its last page
            entries = sum(len(rows[p]) for p in set(parents) if p >= 0)
            return {"bytes": 2 * size * moved + 4 * (entries + R * P + 5 * R), "flops": 0}
        moved = used * (1 - used / N)  # holes among the first pages, the expected number
        return {"bytes": 2 * size * moved + 4 * (used + R * P + 2 * (N // 2) + R), "flops": 0}
    n = case["requests"] * case["beams"]
    return {"bytes": e * n * case["vocab"] + 4 * n + 12 * case["requests"] * case["num_out"], "flops": 4 * n * case["vocab"]}


def exact(case, seed):
    if case["op"] not in ("attend", "select"):
        return None  # pages and tables: nothing is computed that could be off
    s = prepare(case, seed)
    if case["op"] == "select":
        logp = torch.log_softmax(s["logits"].double(), 2)
        if s["ended"] is not None:
            at_end = torch.full_like(logp, -math.inf)
            at_end[:, :, s["end_token"]] = 0.0
            logp = torch.where(s["ended"][:, :, None], at_end, logp)
        total = (s["scores"].double()[:, :, None] + logp).flatten(1)
        return torch.topk(total, case["num_out"], dim=1).values, None, None
    n_heads, kv, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    group = n_heads // kv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((case["seqs"], n_heads), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        first = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            continue
        pos = torch.arange(first, n, device="cuda")
        at = s["page_table"][b][pos // page].long()
        for h in range(kv):
            k, v = s["k_cache"][at, pos % page, h].double(), s["v_cache"][at, pos % page, h].double()
            k[-1], v[-1] = s["k_new"][b, h].double(), s["v_new"][b, h].double()
            rows = slice(h * group, (h + 1) * group)
            x = s["q"][b, rows].double() @ k.t() / math.sqrt(dim)
            lse[b, rows] = torch.logsumexp(x, 1)
            out[b, rows] = torch.softmax(x, 1) @ v
    return out, lse, None, None
