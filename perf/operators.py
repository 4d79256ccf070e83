"""What is measured of the operators around the routing: a whole MoE layer for
a few tokens, the layer norm in front of it (forward and backward), and the
global norm and clipping of many gradients.

Each case runs in one of two forms on the same inputs: the plain form
(elementary torch operations in 32 bits, rounded once at the end) or, with
``own`` set, the calls that a user makes of the package.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _layer(name, tokens, hidden, ffn, experts, top_k, mode, dtype):
    return {"name": name, "op": "layer", "tokens": tokens, "hidden": hidden, "ffn": ffn, "experts": experts,
            "top_k": top_k, "mode": mode, "dtype": dtype}


def _norm(name, op, rows, hidden, dtype, wdtype):
    return {"name": name, "op": op, "rows": rows, "hidden": hidden, "dtype": dtype, "wdtype": wdtype}


def _grads(name, op, tensors, mean, dtype, align):
    return {"name": name, "op": op, "tensors": tensors, "mean": mean, "dtype": dtype, "align": align}


def listed():
    return [
        # One token of a small model: latency, a few microseconds of weights.
        _layer("layer 1 token small", 1, 1024, 2048, 8, 2, "softmax", "bf16"),
        # One token of the Mixtral-8x7B shape: the serving step of a single request.
        _layer("layer 1 token mixtral-8x7b", 1, 4096, 14336, 8, 2, "softmax", "bf16"),
        # A decode batch of 48 requests on the Mixtral-8x22B hidden size: every expert is hit by several tokens.
        _layer("layer 48 tokens mixtral-8x22b", 48, 6144, 16384, 8, 2, "softmax", "bf16"),
        # A decode batch of 32 requests on the DeepSeek-V3 shape (256 experts, 8 each, sigmoid): most experts, one token each.
        _layer("layer 32 tokens deepseek-v3", 32, 7168, 2048, 256, 8, "sigmoid", "bf16"),
        # Odd sizes in fp32: rows that no vector load divides.
        _layer("layer 5 tokens odd fp32", 5, 1001, 777, 12, 3, "softmax", "fp32"),
        # The norm of four decoded tokens: latency alone.
        _norm("norm fwd 4 rows", "norm_fwd", 4, 7168, "bf16", "bf16"),
        # The norm over the DeepSeek-V3-shaped training batch, forward and backward.
        _norm("norm fwd 8192 rows", "norm_fwd", 8192, 7168, "bf16", "fp32"),
        _norm("norm bwd 8192 rows", "norm_bwd", 8192, 7168, "bf16", "fp32"),
        # A ragged backward pass in fp32 with odd rows.
        _norm("norm bwd 1531 odd rows fp32", "norm_bwd", 1531, 1001, "fp32", "fp32"),
        # A model's many small tensors (norms, biases, routers) of odd sizes, packed with no gap.
        _grads("clip 160 small odd tensors", "clip", 160, 9001, "bf16", 1),
        # The gradients of 8 experts of 3 matrices of 4096 x 14336 each: the largest clipping.
        _grads("clip 24 expert matrices fp32", "clip", 24, 4096 * 14336, "fp32", 128),
        # 256 experts' matrices of one layer, shrunk to a rank's share: the norm alone.
        _grads("norm of 768 tensors bf16", "grad_norm", 768, 1 << 20, "bf16", 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer", "layer", "norm_fwd", "norm_bwd", "clip", "grad_norm"])
    if op == "layer":
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        experts = rng.choice([4, 8, 12, 16, 60, 64, 128, 256])
        top_k = rng.randint(1, min(8, experts))
        tokens = _log(rng, 1, 64 if dtype == "bf16" else 16)
        most = 2.5e9 if dtype == "bf16" else 2.5e8  # weights of one expert set, in elements
        hidden, ffn = _log(rng, 256, 7168), _log(rng, 256, 16384)
        while experts * 3 * hidden * ffn > most:
            hidden, ffn = max(256, int(hidden / 1.3)), max(256, int(ffn / 1.3))
            if hidden == 256 and ffn == 256:
                break
        if dtype == "bf16" and rng.random() < 0.75:  # most models' sizes are multiples of 64 or so
            hidden, ffn = max(256, hidden // 64 * 64), max(256, ffn // 64 * 64)
        return _layer("drawn", tokens, hidden, ffn, experts, top_k, rng.choice(["softmax", "sigmoid"]), dtype)
    if op in ("norm_fwd", "norm_bwd"):
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        hidden = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            hidden = max(64, hidden // 64 * 64)
        rows = _log(rng, 1, min(65536, max(2, (1 << 26) // hidden)))
        return _norm("drawn", op, rows, hidden, dtype, rng.choice(["fp32", "fp32", dtype]))
    tensors = _log(rng, 1, 1000)
    mean = _log(rng, 100, min(1 << 26, (1 << 30) // tensors))
    return _grads("drawn", op, tensors, mean, rng.choice(["bf16", "fp32"]), rng.choice([1, 128]))


def _rand(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(scale)


def _sizes(case):
    """Element counts of the tensors, spread over a factor of sixteen around the mean, the same for every seed."""
    n, mean = case["tensors"], case["mean"]
    if case["align"] > 1 and mean >= 1 << 20:
        return [mean] * n
    return [max(1, int(mean * 2.0 ** (4.0 * ((i * 0.61803398875) % 1.0) - 2.0) * 0.74)) for i in range(n)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "layer":
        T, H, F, E = case["tokens"], case["hidden"], case["ffn"], case["experts"]
        # Activations on a grid of 1/16 and router weights on one of 2^-10: every partial sum of a logit is then a
        # float32, so the logits, and the experts chosen by them, do not depend on the order of the sum.
        x = torch.round(_rand(gen, (T, H), torch.float32) * 16).clamp(-120, 120).div(16).to(dt)
        router = torch.round(_rand(gen, (E, H), torch.float32, 1.5 / math.sqrt(H)) * 1024).clamp(-250, 250).div(1024).to(dt)
        return {"case": case, "x": x, "router": router,
                "w_gate_up": _rand(gen, (E, 2 * F, H), dt, 1.0 / math.sqrt(H)),
                "w_down": _rand(gen, (E, H, F), dt, 1.0 / math.sqrt(F))}
    if case["op"] in ("norm_fwd", "norm_bwd"):
        M, H, wdt = case["rows"], case["hidden"], DTYPES[case["wdtype"]]
        # Activations of a residual stream: a mean and a scale of their own in each row.
        x = _rand(gen, (M, H), torch.float32)
        x = x.mul_(0.5 + _rand(gen, (M, 1), torch.float32).abs()).add_(_rand(gen, (M, 1), torch.float32, 0.5)).to(dt)
        s = {"case": case, "x": x, "eps": 1e-5, "weight": (1 + _rand(gen, (H,), torch.float32, 0.1)).to(wdt),
             "bias": _rand(gen, (H,), torch.float32, 0.1).to(wdt)}
        if case["op"] == "norm_bwd":
            xf = x.float()
            s["mean"] = xf.mean(1)
            s["rstd"] = ((xf - s["mean"][:, None]).square().mean(1) + s["eps"]).rsqrt()
            s["dy"] = _rand(gen, (M, H), dt)
        return s
    sizes, step = _sizes(case), case["align"]
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += -(-n // step) * step
    # Gradients lie one after another in a bucket, and clipped ones in another, as a training program keeps them.
    bucket = _rand(gen, (total,), dt, 0.02)
    grads = [bucket[a:a + n] for a, n in zip(starts, sizes)]
    s = {"case": case, "bucket": bucket, "grads": grads, "max_norm": 1.0}
    if case["op"] == "clip":
        s["out"] = torch.zeros_like(bucket)
        s["outs"] = [s["out"][a:a + n] for a, n in zip(starts, sizes)]
    if own:  # the handle that a training program makes once for its gradients
        import padded_permute_combine_gb300 as p

        s["set"] = p.moe_grad_set(grads, s.get("outs"))
    return s


def _own(s):
    import padded_permute_combine_gb300 as p

    c = s["case"]
    if c["op"] == "layer":
        return p.moe_layer(s["x"], s["router"], s["w_gate_up"], s["w_down"], c["top_k"], c["mode"])
    if c["op"] == "norm_fwd":
        return p.moe_layer_norm_fwd(s["x"], s["weight"], s["bias"], s["eps"])
    if c["op"] == "norm_bwd":
        return p.moe_layer_norm_bwd(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])
    if c["op"] == "clip":
        return p.moe_clip_grads(s["set"], s["max_norm"]), s["out"]
    return p.moe_grad_norm(s["set"])


def _plain_layer(s):
    c, x = s["case"], s["x"].float()
    K, F, E = c["top_k"], c["ffn"], c["experts"]
    logits = x @ s["router"].float().t()
    scores = torch.softmax(logits, 1) if c["mode"] == "softmax" else torch.sigmoid(logits)
    top = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :K]
    w = scores.gather(1, top)
    w = w / w.sum(1, keepdim=True)
    if 2 * x.shape[0] * K <= E:  # few choices: the chosen experts' matrices, one copy for each
        gu = torch.matmul(s["w_gate_up"][top].float(), x[:, None, :, None]).squeeze(-1)
        g, u = gu[..., :F], gu[..., F:]
        h = g / (1 + torch.exp(-g)) * u
        y = torch.matmul(s["w_down"][top].float(), h[..., None]).squeeze(-1)
        y = (w[..., None] * y).sum(1)
    else:  # every expert on every token, weighted by zero where it was not chosen
        gu = torch.matmul(x, s["w_gate_up"].float().transpose(1, 2))
        g, u = gu[..., :F], gu[..., F:]
        h = g / (1 + torch.exp(-g)) * u
        y = torch.matmul(h, s["w_down"].float().transpose(1, 2))
        share = torch.zeros_like(logits).scatter(1, top, w)
        y = (share.t()[:, :, None] * y).sum(0)
    return y.to(s["x"].dtype), top.to(torch.int32), w


def run(s):
    c = s["case"]
    if own:
        return _own(s)
    if c["op"] == "layer":
        return _plain_layer(s)
    if c["op"] == "norm_fwd":
        x = s["x"].float()
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = (d.square().mean(1) + s["eps"]).rsqrt()
        y = d * rstd[:, None] * s["weight"].float() + s["bias"].float()
        return y.to(s["x"].dtype), mean, rstd
    if c["op"] == "norm_bwd":
        dy, r = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * r
        wdy = dy * s["weight"].float()
        dx = r * (wdy - wdy.mean(1, keepdim=True) - xhat * (wdy * xhat).mean(1, keepdim=True))
        wdt = s["weight"].dtype
        return dx.to(s["x"].dtype), (dy * xhat).sum(0).to(wdt), dy.sum(0).to(wdt)
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    if c["op"] == "grad_norm":
        return norm
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    [o.copy_(g.float() * coef) for g, o in zip(s["grads"], s["outs"])]
    return norm, s["out"]


def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "layer":
        T, H, F, E, K = case["tokens"], case["hidden"], case["ffn"], case["experts"], case["top_k"]
        hit = E * (1 - (1 - K / E) ** T)  # experts that T tokens reach when each takes K of E
        return {"bytes": b * (hit * 3 * H * F + E * H + 2 * T * H) + 8 * T * K,
                "flops": 6 * T * K * H * F + 2 * T * E * H}
    if case["op"] == "norm_fwd":
        M, H, w = case["rows"], case["hidden"], 2 if case["wdtype"] == "bf16" else 4
        return {"bytes": 2 * b * M * H + 2 * w * H + 8 * M, "flops": 8 * M * H}
    if case["op"] == "norm_bwd":
        M, H, w = case["rows"], case["hidden"], 2 if case["wdtype"] == "bf16" else 4
        return {"bytes": 3 * b * M * H + 3 * w * H + 8 * M, "flops": 14 * M * H}
    n = sum(_sizes(case))
    if case["op"] == "grad_norm":
        return {"bytes": b * n + 4, "flops": 2 * n}
    return {"bytes": 2 * b * n + 4, "flops": 3 * n}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layer":
        K, F = case["top_k"], case["ffn"]
        x = s["x"].double()
        logits = x @ s["router"].double().t()
        top = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :K]
        chosen = logits.gather(1, top)
        # Normalised over the chosen experts, a softmax over all of them is one over these.
        w = torch.softmax(chosen, 1) if case["mode"] == "softmax" else torch.sigmoid(chosen)
        w = w / w.sum(1, keepdim=True)
        y = torch.zeros_like(x)
        for e in torch.unique(top).tolist():
            t, k = torch.nonzero(top == e, as_tuple=True)
            gu = x[t] @ s["w_gate_up"][e].double().t()
            h = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
            y.index_add_(0, t, w[t, k][:, None] * (h @ s["w_down"][e].double().t()))
        return y, None, w
    if case["op"] == "norm_fwd":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = 1 / torch.sqrt(var + s["eps"])
        return (x - mean[:, None]) * rstd[:, None] * s["weight"].double() + s["bias"].double(), mean, rstd
    if case["op"] == "norm_bwd":
        r = s["rstd"].double()[:, None]
        xhat = (s["x"].double() - s["mean"].double()[:, None]) * r
        dy = s["dy"].double()
        v = dy * s["weight"].double()
        H = case["hidden"]
        dx = (v - v.sum(1, keepdim=True) / H - xhat * ((v * xhat).sum(1, keepdim=True) / H)) * r
        return dx, (dy * xhat).sum(0), dy.sum(0)
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(g, dtype=torch.float64)) ** 2 for g in s["grads"]))
    at = torch.tensor(norm, dtype=torch.float64)
    if case["op"] == "grad_norm":
        return at
    out = torch.zeros_like(s["bucket"], dtype=torch.float64)
    starts = [(g.data_ptr() - s["bucket"].data_ptr()) // g.element_size() for g in s["grads"]]
    for a, g in zip(starts, s["grads"]):
        out[a:a + g.numel()] = g.double() * min(1.0, s["max_norm"] / (norm + 1e-6))
    return at, out
