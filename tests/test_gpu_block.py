"""The operators around the routing (include/moe_block.h) against plain
implementations in 64 bits: the whole MoE layer for a few tokens, the layer
norm forward and backward, the global gradient norm and clipping.

Tolerances follow from the arithmetic, not from runs: u = 2^-24 is fp32's unit
roundoff, a sum of N terms in any order is off by at most N_serial * u times
the sum of the terms' magnitudes (N_serial: the longest chain of additions),
and a bf16 output adds 2^-8 of its own magnitude (half an ulp is 2^-9)."""
import numpy as np
import pytest
import torch

import padded_permute_combine_gb300 as p
from padded_permute_combine_gb300 import autograd as ag
from padded_permute_combine_gb300 import _lib
from gpu_util import misaligned_like

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib_loaded():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    p.load()


def randn(shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DEV).to(dtype)


def type_round(ref, dtype):
    return 2.0 ** -8 * ref.abs() if dtype == BF else U * ref.abs()


def check(got, ref, tol, what):
    got = got.double()
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= tol)
    assert not bool(bad.any()), "%s: %d of %d off, worst %g of its tolerance" % (
        what, int(bad.sum()), bad.numel(), float(((got - ref).abs() / tol.clamp(min=1e-300)).nan_to_num(1e9).max()))


# ------------------------------------------------------------------ layer

def layer_inputs(T, H, F, E, dtype, seed):
    """x and the router on grids on which every partial sum of a logit is an
    fp32 number, so that the choice of experts has one right answer."""
    x = torch.round(randn((T, H), seed) * 16).clamp(-120, 120).div(16).to(dtype)
    router = torch.round(randn((E, H), seed + 1, scale=1.5 / H ** 0.5) * 1024).clamp(-250, 250).div(1024).to(dtype)
    return x, router, randn((E, 2 * F, H), seed + 2, dtype, H ** -0.5), randn((E, H, F), seed + 3, dtype, F ** -0.5)


def route_ref(x, router, K, mode, normalize):
    logits = x.double() @ router.double().t()
    scores = torch.softmax(logits, 1) if mode == "softmax" else torch.sigmoid(logits)
    top = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :K]
    w = scores.gather(1, top)
    return top, w / w.sum(1, keepdim=True) if normalize else w


def experts_ref(x, top, w, wgu, wd):
    """y and its tolerance. A sum of N terms runs over 32 lanes or more, so its
    chain is at most N/32 + 32 (doubled: products round too, and tensor cores
    may truncate instead of rounding); h keeps at least 16 significant bits."""
    T, H = x.shape
    F = wd.shape[2]
    steps = 4 * (max(H, F) // 32 + 32) * U
    y = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    tol = torch.zeros_like(y)
    xd = x.double()
    for t in range(T):
        for k in range(top.shape[1]):
            e = int(top[t, k])
            if e < 0 or e >= wgu.shape[0]:
                continue
            gu = wgu[e].double() @ xd[t]
            mag = wgu[e].double().abs() @ xd[t].abs()
            g, u = gu[:F], gu[F:]
            h = g * torch.sigmoid(g) * u
            # |d silu / dg| <= 1.1
            dh = steps * (1.1 * u.abs() * mag[:F] + (g * torch.sigmoid(g)).abs() * mag[F:]) + (2.0 ** -16 + 8 * U) * h.abs()
            y[t] += w[t, k] * (wd[e].double() @ h)
            tol[t] += w[t, k].abs() * (wd[e].double().abs() @ (dh + (steps + 8 * U) * h.abs()))
    return y, tol + type_round(y, x.dtype) + 1e-30


SHAPES = [(1, 64, 32, 4, 1), (1, 1024, 512, 8, 2), (3, 1001, 77, 5, 5), (8, 256, 136, 16, 4), (9, 264, 24, 7, 3),
          (17, 512, 264, 8, 2), (64, 136, 64, 4, 2), (70, 72, 40, 3, 2), (256, 64, 48, 8, 8), (33, 7, 5, 6, 2),
          (2, 1, 1, 1, 1), (5, 4096, 16, 64, 8), (31, 2048, 8, 60, 4), (1, 8, 4104, 300, 6), (130, 520, 72, 2, 1)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H,F,E,K", SHAPES)
def test_layer(T, H, F, E, K, dtype):
    for mode, norm in (("softmax", True), ("sigmoid", False)):
        x, router, wgu, wd = layer_inputs(T, H, F, E, dtype, T + H + F)
        y, te, w = p.moe_layer(x, router, wgu, wd, K, mode, norm)
        top, wref = route_ref(x, router, K, mode, norm)
        assert torch.equal(te.long(), top)
        check(w, wref, 1e-5 * (1 + wref.abs()), "weights")
        ref, tol = experts_ref(x, top, w.double(), wgu, wd)
        check(y, ref, tol, "y %s" % mode)


# Beyond 2^24 elements of the choices' matrices, where bf16 layers run on the tensor cores; H and F of every remainder
# by the blocks of 64, one, two and more SMs to a tile of y's columns, two tiles an SM, several passes over an expert.
LARGE = [(16, 1024, 1040, 8, 2), (1, 4096, 4104, 4, 1), (5, 1096, 1048, 16, 3), (70, 512, 264, 8, 2), (256, 136, 72, 8, 8),
         (256, 64, 136, 8, 8), (64, 264, 1000, 300, 4), (130, 2048, 72, 2, 1), (3, 12288, 520, 6, 1), (2, 20480, 1024, 4, 2),
         (40, 6144, 136, 5, 2), (256, 1024, 80, 8, 8), (23, 1400, 904, 12, 5), (8, 7168, 512, 32, 8),
         # rows off 16 bytes
         (16, 1025, 1041, 8, 2), (1, 4099, 4102, 4, 1), (5, 1097, 1049, 16, 3), (70, 513, 263, 8, 2), (256, 137, 73, 8, 8),
         (256, 65, 135, 8, 8), (64, 267, 1001, 300, 4), (130, 2046, 77, 2, 1), (3, 12289, 521, 6, 1), (2, 20481, 1023, 4, 2),
         (40, 6145, 137, 5, 2), (255, 1023, 81, 8, 8), (23, 1400, 903, 12, 5), (23, 1401, 904, 12, 5), (8, 7167, 513, 32, 8)]


@pytest.mark.parametrize("T,H,F,E,K", LARGE)
def test_large_layer(T, H, F, E, K):
    x, router, wgu, wd = layer_inputs(T, H, F, E, BF, T + H + F)
    y, te, w = p.moe_layer(x, router, wgu, wd, K)
    top, wref = route_ref(x, router, K, "softmax", True)
    assert torch.equal(te.long(), top)
    check(w, wref, 1e-5 * (1 + wref.abs()), "weights")
    ref, tol = experts_ref(x, top, w.double(), wgu, wd)
    check(y, ref, tol, "y")
    out, ws = torch.empty_like(y), p.block.layer_workspace(T, H, F, E, K, DEV).fill_(0xff)
    assert torch.equal(p.moe_experts(x, te, w, wgu, wd, out=out, workspace=ws), y)
    wide = torch.full((T, H + 8), float("nan"), dtype=BF, device=DEV)
    wide[:, :H] = x
    assert torch.equal(p.moe_experts(wide[:, :H], te, w, wgu, wd), y)


@pytest.mark.parametrize("T,H,F,K", [(40, 1032, 520, 3), (256, 264, 88, 8), (9, 5120, 1024, 2)])
def test_large_experts_one_expert_takes_all_and_empty_slots(T, H, F, K):
    E = 8
    x, _, wgu, wd = layer_inputs(T, H, F, E, BF, 5)
    w = randn((T, K), 6).abs()
    top = torch.full((T, K), 3, dtype=torch.int32, device=DEV)
    ref, tol = experts_ref(x, top, w.double(), wgu, wd)
    check(p.moe_experts(x, top, w, wgu, wd), ref, tol, "one expert")
    top = torch.randint(-1, E, (T, K), generator=torch.Generator().manual_seed(T), dtype=torch.int32).to(DEV)
    top[T // 2] = -1
    top[0, 0] = E + 7
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = p.moe_experts(x, top, w, wgu, wd, status=status)
    ref, tol = experts_ref(x, top, w.double(), wgu, wd)
    check(y, ref, tol, "empty slots")
    assert bool((y[T // 2] == 0).all()) and not bool(torch.signbit(y[T // 2].float()).any())
    assert int(status) == _lib.MOE_STATUS_BAD_EXPERT
    status.zero_()
    assert bool((p.moe_experts(x, torch.full_like(top, -1), w, wgu, wd, status=status) == 0).all())
    assert int(status) == 0


@pytest.mark.parametrize("T", [4, 24])
def test_large_layer_nan_and_infinity_stay_with_their_token(T):
    H, F, E = 2048, 1160, 6
    x, _, wgu, wd = layer_inputs(T, H, F, E, BF, 9)
    top = torch.tensor([[t % 3, 3 + t % 2] for t in range(T)], dtype=torch.int32, device=DEV)
    w = torch.full((T, 2), 0.5, device=DEV)
    wd[5] = float("nan")  # chosen by nobody
    wgu[5] = float("inf")
    clean = p.moe_experts(x, top, w, wgu, wd)
    assert bool(torch.isfinite(clean).all())
    wd[2, 100, :] = float("nan")  # one row of an expert of tokens 2, 5, ...
    hit = torch.tensor([t % 3 == 2 for t in range(T)], device=DEV)
    y = p.moe_experts(x, top, w, wgu, wd)
    rest = torch.arange(H, device=DEV) != 100
    assert torch.equal(y[:, rest], clean[:, rest]) and torch.equal(y[~hit], clean[~hit])
    assert bool(torch.isnan(y[hit, 100]).all())
    x2 = x.clone()
    x2[1, 0] = float("nan")
    y = p.moe_experts(x2, top, w, wgu, wd)
    keep = ~hit
    keep[1] = False
    assert torch.equal(y[keep], clean[keep]) and bool(torch.isnan(y[1]).all())


def test_large_layer_streams_graphs_and_repeats():
    T, H, F, E, K = 11, 1024, 1024, 8, 2
    x, router, wgu, wd = layer_inputs(T, H, F, E, BF, 12)
    y, te, w = p.moe_layer(x, router, wgu, wd, K)
    ref, tol = experts_ref(x, te, w.double(), wgu, wd)
    check(y, ref, tol, "y")
    for which in range(4):
        args = [x, router, wgu, wd]
        args[which] = misaligned_like(args[which])
        y2, te2, _ = p.moe_layer(*args, K)
        assert torch.equal(te2, te)
        check(y2, ref, tol, "misaligned %d" % which)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2 = p.moe_layer(x, router, wgu, wd, K)[0]
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y2, y)
    out, ws = torch.empty_like(y), p.block.layer_workspace(T, H, F, E, K, DEV)
    routing = (torch.empty_like(te), torch.empty_like(w))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):  # the same workspace in calls that follow one another
            p.moe_layer(x, router, wgu, wd, K, out=out, routing=routing, workspace=ws)
    for _ in range(2):
        out.fill_(float("nan"))
        ws.fill_(0xff)
        graph.replay()
        assert torch.equal(out, y) and torch.equal(routing[0], te)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,K", [(1, 1), (6, 2), (40, 3), (256, 8)])
def test_experts_one_expert_takes_all_and_empty_slots(T, K, dtype):
    H, F, E = 264, 88, 8
    x, _, wgu, wd = layer_inputs(T, H, F, E, dtype, 5)
    w = randn((T, K), 6).abs()
    top = torch.full((T, K), 3, dtype=torch.int32, device=DEV)  # every slot the same expert, repeats within a token
    ref, tol = experts_ref(x, top, w.double(), wgu, wd)
    check(p.moe_experts(x, top, w, wgu, wd), ref, tol, "one expert")
    top = torch.randint(-1, E, (T, K), generator=torch.Generator().manual_seed(T), dtype=torch.int32).to(DEV)
    top[T // 2] = -1  # a token without any expert
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = p.moe_experts(x, top, w, wgu, wd, status=status)
    ref, tol = experts_ref(x, top, w.double(), wgu, wd)
    check(y, ref, tol, "empty slots")
    assert bool((y[T // 2] == 0).all()) and not bool(torch.signbit(y[T // 2].float()).any())
    assert int(status) == 0
    y = p.moe_experts(x, torch.full_like(top, -1), w, wgu, wd)
    assert bool((y == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_experts_report_ids_out_of_range(dtype):
    x, _, wgu, wd = layer_inputs(4, 64, 32, 4, dtype, 8)
    top = torch.tensor([[0, 4], [1, 2], [-2, 3], [2 ** 30, 1]], dtype=torch.int32, device=DEV)
    w = torch.ones((4, 2), device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = p.moe_experts(x, top, w, wgu, wd, status=status)
    assert int(status) == _lib.MOE_STATUS_BAD_EXPERT
    ref, tol = experts_ref(x, top, w.double(), wgu, wd)  # skips them too
    check(y, ref, tol, "others")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [2, 12])
def test_nan_and_infinity_stay_with_their_token(T, dtype):
    H, F, E = 256, 72, 6
    x, _, wgu, wd = layer_inputs(T, H, F, E, dtype, 9)
    top = torch.tensor([[t % 3, 3 + t % 2] for t in range(T)], dtype=torch.int32, device=DEV)
    w = torch.full((T, 2), 0.5, device=DEV)
    wd[5] = float("nan")  # chosen by nobody
    wgu[5] = float("inf")
    clean = p.moe_experts(x, top, w, wgu, wd)
    assert bool(torch.isfinite(clean).all())
    wd[2, :, :] = float("nan")  # chosen by tokens 2, 5, ...
    hit = torch.tensor([t % 3 == 2 for t in range(T)], device=DEV)
    y = p.moe_experts(x, top, w, wgu, wd)
    assert torch.equal(y[~hit], clean[~hit])
    assert bool(torch.isnan(y[hit]).all())
    x2 = x.clone()
    x2[1, 0] = float("nan")
    y = p.moe_experts(x2, top, w, wgu, wd)
    keep = ~hit
    keep[1] = False
    assert torch.equal(y[keep], clean[keep]) and bool(torch.isnan(y[1]).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_layer_strides_alignment_streams_and_repeats(dtype):
    T, H, F, E, K = 11, 512, 256, 8, 2
    x, router, wgu, wd = layer_inputs(T, H, F, E, dtype, 12)
    y, te, w = p.moe_layer(x, router, wgu, wd, K)
    for pad in (8, 3):  # a slice of a wider tensor, on 16-byte boundaries and off them
        wide = torch.full((T, H + pad), float("nan"), dtype=dtype, device=DEV)
        wide[:, :H] = x
        y2, te2, w2 = p.moe_layer(wide[:, :H], router, wgu, wd, K)
        ref, tol = experts_ref(x, te, w.double(), wgu, wd)
        assert torch.equal(te2, te) and torch.equal(w2, w)
        check(y2, ref, tol, "stride H+%d" % pad)
    for which in range(4):
        args = [x, router, wgu, wd]
        args[which] = misaligned_like(args[which])
        y2, te2, _ = p.moe_layer(*args, K)
        assert torch.equal(te2, te)
        check(y2, ref, tol, "misaligned %d" % which)
    for _ in range(3):
        assert torch.equal(p.moe_layer(x, router, wgu, wd, K)[0], y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2 = p.moe_layer(x, router, wgu, wd, K)[0]
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y2, y)
    # into given buffers, from a CUDA graph
    out, ws = torch.empty_like(y), p.block.layer_workspace(T, H, F, E, K, DEV)
    routing = (torch.empty_like(te), torch.empty_like(w))
    run = lambda: p.moe_layer(x, router, wgu, wd, K, out=out, routing=routing, workspace=ws)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(2):
        out.fill_(float("nan"))
        ws.fill_(0xff)
        graph.replay()
        assert torch.equal(out, y) and torch.equal(routing[0], te)


def test_layer_equals_its_parts():
    """moe_layer is the gating and moe_experts of the library, and agrees with the path for many tokens."""
    T, H, F, E, K = 24, 256, 128, 8, 2
    x, router, wgu, wd = layer_inputs(T, H, F, E, BF, 14)
    y, te, w = p.moe_layer(x, router, wgu, wd, K)
    te2, w2 = p.moe_topk_gating(x.float() @ router.float().t(), K)
    assert torch.equal(te, te2)
    check(w, w2.double(), 1e-5 * (1 + w2.double()), "weights")
    assert torch.equal(p.moe_experts(x, te, w, wgu, wd), y)
    route = p.moe_route_build(te, E, 16)
    xe = p.moe_padded_gather(x, route.indices, route.bins, route.padded_bins, K, positions=route.positions)
    edge = [0] + route.padded_bins.tolist()
    ye = torch.zeros_like(xe, dtype=F32)
    for e in range(E):
        gu = xe[edge[e]:edge[e + 1]].float() @ wgu[e].float().t()
        ye[edge[e]:edge[e + 1]] = (torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]) @ wd[e].float().t()
    y2 = p.moe_padded_scatter(ye, route.indices, route.bin_ids, route.bins, route.padded_bins, w.reshape(-1), T, K,
                              positions=route.positions)
    ref, tol = experts_ref(x, te, w.double(), wgu, wd)
    check(y, ref, tol, "few")
    check(y2, ref, tol, "many")


def test_layer_refusals():
    x, router, wgu, wd = layer_inputs(4, 64, 32, 4, BF, 1)
    with pytest.raises(ValueError):
        p.moe_layer(x, router[:, :32].contiguous(), wgu, wd, 2)
    with pytest.raises(TypeError):
        p.moe_layer(x, router.float(), wgu, wd, 2)
    with pytest.raises(TypeError):
        p.moe_layer(x.half(), router.half(), wgu.half(), wd.half(), 2)
    with pytest.raises(ValueError):
        p.moe_layer(x, router, wgu, wd.transpose(1, 2), 2)
    with pytest.raises(ValueError):
        p.moe_layer(x.t().contiguous().t(), router, wgu, wd, 2)
    with pytest.raises(ValueError):
        p.moe_layer(x.cpu(), router, wgu, wd, 2)
    with pytest.raises(ValueError):
        p.moe_layer(x[:1].expand(4, 64), router, wgu, wd, 2)
    with pytest.raises(ValueError):
        p.moe_layer(x, router, wgu, wd, 2, mode="max")
    with pytest.raises(p.MoeError):
        p.moe_layer(x, router, wgu, wd, 5)
    big = torch.zeros((257, 64), dtype=BF, device=DEV)
    with pytest.raises(p.MoeError):
        p.moe_layer(big, router, wgu, wd, 1)
    with pytest.raises(p.MoeError):
        p.moe_layer(x, router, wgu, wd, 2, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    y, te, w = p.moe_layer(x[:0], router, wgu, wd, 2)
    assert y.shape == (0, 64) and te.shape == (0, 2)


# ------------------------------------------------------------- layer norm

def norm_ref(x, w, b, eps):
    x = x.double()
    var, mean = torch.var_mean(x, 1, correction=0)
    rstd = 1 / torch.sqrt(var + eps)
    xhat = (x - mean[:, None]) * rstd[:, None]
    y = xhat * (1 if w is None else w.double()) + (0 if b is None else b.double())
    return y, mean, rstd, xhat


# A row's sum runs over a warp or a CTA: at most 128 values in a thread, then 10 levels.
ROW = 160 * U

NORM_SHAPES = [(1, 1), (3, 7), (5, 64), (2, 1000), (7, 1001), (4, 1024), (33, 2048), (300, 96), (3, 4099), (9, 7168),
               (2, 8200), (1000, 256), (3, 16384), (2, 17001), (2, 40000), (700, 33)]


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("M,H", NORM_SHAPES)
def test_layer_norm(M, H, dtype, wdtype):
    x = (randn((M, H), M + H) * (0.5 + randn((M, 1), 2).abs()) + randn((M, 1), 3)).to(dtype)
    w, b = (1 + randn((H,), 4, scale=0.1)).to(wdtype), randn((H,), 5, wdtype)
    dy = randn((M, H), 6, dtype)
    y, mean, rstd = p.moe_layer_norm_fwd(x, w, b, 1e-5)
    ref, rmean, rrstd, xhat = norm_ref(x, w, b, 1e-5)
    mag = x.double().abs().mean(1)
    check(mean, rmean, ROW * mag + 1e-30, "mean")
    # The centred values carry the mean's error, which cancels in the sum to second order.
    rel = ROW + 4 * U * (1 + mag * rrstd)
    check(rstd, rrstd, rel * rrstd, "rstd")
    off = (ROW * mag * rrstd)[:, None] + (rel[:, None] + 8 * U) * xhat.abs() + 2 * U * mag[:, None] * rrstd[:, None]
    check(y, ref, off * w.double().abs() + 4 * U * (ref.abs() + b.double().abs()) + type_round(ref, dtype) + 1e-30, "y")

    dx, dw, db = p.moe_layer_norm_bwd(dy, x, w, mean, rstd)
    md, rd = mean.double()[:, None], rstd.double()[:, None]
    xh = (x.double() - md) * rd
    v = dy.double() * w.double()
    c0, c1 = v.mean(1, keepdim=True), (v * xh).mean(1, keepdim=True)
    ref = rd * (v - c0 - xh * c1)
    dxh = 4 * U * (x.double().abs() + md.abs()) * rd  # error of xhat
    tol = rd * (4 * U * v.abs() + ROW * v.abs().mean(1, keepdim=True) + dxh * c1.abs()
                + xh.abs() * (ROW * (v * xh).abs().mean(1, keepdim=True) + (v.abs() * dxh).mean(1, keepdim=True))
                + 8 * U * (v.abs() + c0.abs() + (xh * c1).abs()))
    check(dx, ref, tol + type_round(ref, dtype) + 1e-30, "dx")
    # A column's chain: a CTA's rows, then the parts.
    col = (M // 32 + 64) * U
    refw, refb = (dy.double() * xh).sum(0), dy.double().sum(0)
    check(dw, refw, col * (dy.double() * xh).abs().sum(0) + (dy.double().abs() * dxh).sum(0) + type_round(refw, wdtype) + 1e-30, "dw")
    check(db, refb, col * dy.double().abs().sum(0) + type_round(refb, wdtype) + 1e-30, "db")
    assert torch.equal(dw, p.moe_layer_norm_bwd(dy, x, w, mean, rstd)[1])


@pytest.mark.parametrize("H", [64, 1000, 1001, 9000])
def test_layer_norm_without_weight_bias_or_columns(H):
    x, dy = randn((6, H), 1), randn((6, H), 2)
    one, zero = torch.ones(H, device=DEV), torch.zeros(H, device=DEV)
    y, mean, rstd = p.moe_layer_norm_fwd(x)
    y1 = p.moe_layer_norm_fwd(x, one, zero)[0]
    assert torch.equal(y, y1)
    dx, dw, db = p.moe_layer_norm_bwd(dy, x, None, mean, rstd)
    dx1, dw1, db1 = p.moe_layer_norm_bwd(dy, x, one, mean, rstd)
    assert torch.equal(dx, dx1) and torch.equal(dw, dw1) and torch.equal(db, db1)
    dx2, dw2, db2 = p.moe_layer_norm_bwd(dy, x, one, mean, rstd, need_cols=False)
    assert torch.equal(dx, dx2) and dw2 is None and db2 is None
    b = randn((H,), 3)
    assert torch.equal(p.moe_layer_norm_fwd(x, one, b)[0], p.moe_layer_norm_fwd(x, None, b)[0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", [256, 1000, 7168, 515])
def test_layer_norm_strides_and_alignment(H, dtype):
    M = 13
    x, dy = randn((M, H), 1, dtype), randn((M, H), 2, dtype)
    w, b = randn((H,), 3), randn((H,), 4)
    y, mean, rstd = p.moe_layer_norm_fwd(x, w, b)
    ref, _, rrstd, xhat = norm_ref(x, w, b, 1e-5)
    mag = x.double().abs().mean(1)[:, None]
    tol = (3 * ROW * (mag * rrstd[:, None] + xhat.abs() + 1)) * w.double().abs() + 4 * U * (ref.abs() + b.double().abs()) + type_round(ref, dtype)
    dx, dw, db = p.moe_layer_norm_bwd(dy, x, w, mean, rstd)
    for pad in (8, 5):
        wide = torch.full((M, 2 * H + pad), float("nan"), dtype=dtype, device=DEV)
        wide[:, :H], wide[:, H + pad:] = x, dy
        xs, ds = wide[:, :H], wide[:, H + pad:]
        y2, mean2, rstd2 = p.moe_layer_norm_fwd(xs, w, b)
        check(y2, ref, tol, "stride %d" % pad)
        dx2, dw2, db2 = p.moe_layer_norm_bwd(ds, xs, w, mean, rstd)
        big = (dx.double().abs().max() + 1)
        check(dx2, dx.double(), 8 * ROW * big + 2 * type_round(dx.double(), dtype), "dx")
        check(dw2, dw.double(), 200 * U * (dy.double().abs() * xhat.abs()).sum(0) + 1e-6, "dw")
    check(p.moe_layer_norm_fwd(misaligned_like(x), misaligned_like(w), b)[0], ref, tol, "misaligned")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", [123, 125, 129, 247, 249, 250, 255, 257, 495, 497, 505, 993, 1985, 2047, 3969, 7935, 7937, 9001])
def test_layer_norm_unaligned_rows(H, dtype):
    """Rows off 16 bytes, with ends at and around a warp's 31 vectors; neighbours of every output stay untouched."""
    M = 5
    wide = randn((M, H + 3), H, dtype)
    x, dy = wide[:, 1:H + 1], randn((M, H + 1), H + 1, dtype)[:, 1:]
    w, b = 1 + randn((H + 1,), 3, scale=0.1)[1:], randn((H,), 4)
    guard = torch.full((2, M * H + 16), 7.0, dtype=dtype, device=DEV)
    y, dx = guard[0, 3:3 + M * H].view(M, H), guard[1, 5:5 + M * H].view(M, H)
    _, mean, rstd = p.moe_layer_norm_fwd(x, w, b, out=y)
    _, dw, db = p.moe_layer_norm_bwd(dy, x, w, mean, rstd, out=dx)
    assert bool((guard[0, :3] == 7).all()) and bool((guard[0, 3 + M * H:] == 7).all())
    assert bool((guard[1, :5] == 7).all()) and bool((guard[1, 5 + M * H:] == 7).all())
    ref, rmean, rrstd, xhat = norm_ref(x, w, b, 1e-5)
    mag = x.double().abs().mean(1)[:, None]
    check(mean, rmean, ROW * mag[:, 0], "mean")
    check(y, ref, 3 * ROW * (mag * rrstd[:, None] + xhat.abs() + 1) * w.double().abs() + 4 * U * (ref.abs() + b.double().abs())
          + type_round(ref, dtype), "y")
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    v = dy.double() * w.double()
    c0, c1 = v.mean(1, keepdim=True), (v * xh).mean(1, keepdim=True)
    ref = rstd.double()[:, None] * (v - c0 - xh * c1)
    size = rstd.double()[:, None] * (v.abs() + v.abs().mean(1, keepdim=True) + xh.abs() * (v * xh).abs().mean(1, keepdim=True))
    check(dx, ref, 3 * ROW * size + type_round(ref, dtype), "dx")
    check(dw, (dy.double() * xh).sum(0), 64 * U * (dy.double() * xh).abs().sum(0) + 16 * U * dy.double().abs().sum(0), "dw")
    check(db, dy.double().sum(0), 64 * U * dy.double().abs().sum(0), "db")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,H", [(1216, 257), (1217, 1001), (1301, 303), (2439, 511), (1300, 2047), (1223, 4095), (4001, 999),
                                 (331, 8196), (331, 9000), (310, 12800), (200, 12804)])
def test_layer_norm_many_packed_rows(M, H, dtype):
    """Rows without gaps, eight of which are a multiple of 16 bytes; the last few short of that, in place as well; and
    long rows, several to a CTA."""
    x, dy = randn((M, H), M + H, dtype), randn((M, H), M, dtype)
    w, b = 1 + randn((H,), 3, scale=0.1), randn((H,), 4)
    guard = torch.full((2, M * H + 32), 7.0, dtype=dtype, device=DEV)
    lo = 16 // x.element_size()
    y, dx = guard[0, lo:lo + M * H].view(M, H), guard.reshape(-1)[-M * H - lo:-lo].view(M, H)
    dx = dx if dx.data_ptr() % 16 == 0 else torch.empty_like(x)
    _, mean, rstd = p.moe_layer_norm_fwd(x, w, b, out=y)
    _, dw, db = p.moe_layer_norm_bwd(dy, x, w, mean, rstd, out=dx)
    assert bool((guard[0, :lo] == 7).all()) and bool((guard[0, lo + M * H:] == 7).all())
    ref, rmean, rrstd, xhat = norm_ref(x, w, b, 1e-5)
    mag = x.double().abs().mean(1)[:, None]
    check(mean, rmean, ROW * mag[:, 0], "mean")
    check(y, ref, 3 * ROW * (mag * rrstd[:, None] + xhat.abs() + 1) * w.double().abs() + 4 * U * (ref.abs() + b.double().abs())
          + type_round(ref, dtype), "y")
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    v = dy.double() * w.double()
    c0, c1 = v.mean(1, keepdim=True), (v * xh).mean(1, keepdim=True)
    ref = rstd.double()[:, None] * (v - c0 - xh * c1)
    size = rstd.double()[:, None] * (v.abs() + v.abs().mean(1, keepdim=True) + xh.abs() * (v * xh).abs().mean(1, keepdim=True))
    check(dx, ref, 3 * ROW * size + type_round(ref, dtype), "dx")
    check(dw, (dy.double() * xh).sum(0), 64 * U * (dy.double() * xh).abs().sum(0) + 16 * U * dy.double().abs().sum(0), "dw")
    check(db, dy.double().sum(0), 64 * U * dy.double().abs().sum(0), "db")
    again = p.moe_layer_norm_fwd(x, w, b, out=x)[0]
    assert torch.equal(again, y)


def test_layer_norm_special_rows():
    x = randn((6, 512), 1)
    clean = p.moe_layer_norm_fwd(x)[0]
    x[1] = 3.0  # no variance
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 1e30  # squares of centred values are zero, of the values beyond fp32
    y, mean, rstd = p.moe_layer_norm_fwd(x)
    assert bool((y[1] == 0).all()) and float(rstd[1]) == pytest.approx(1e-5 ** -0.5, rel=1e-6)
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3]).any())
    assert bool(torch.isfinite(y[4]).all())
    assert torch.equal(y[[0, 5]], clean[[0, 5]])
    y, mean, rstd = p.moe_layer_norm_fwd(x[:0])
    dx, dw, db = p.moe_layer_norm_bwd(x[:0], x[:0], torch.ones(512, device=DEV), mean, rstd)
    assert y.shape == (0, 512) and dx.shape == (0, 512) and bool((dw == 0).all()) and bool((db == 0).all())


def test_layer_norm_gradients_against_differences():
    """Autograd's gradients against central differences of the 64-bit formula."""
    M, H = 5, 24
    x = randn((M, H), 1).requires_grad_(True)
    w, b = randn((H,), 2).requires_grad_(True), randn((H,), 3).requires_grad_(True)
    dy = randn((M, H), 4)
    ag.layer_norm(x, w, b, 1e-3).backward(dy)

    def loss(x_, w_, b_):
        return float((norm_ref(x_, w_, b_, 1e-3)[0] * dy.double()).sum())

    args = [t.detach().double() for t in (x, w, b)]
    for i, t in enumerate((x, w, b)):
        flat = t.grad.double().reshape(-1)
        for j in range(flat.numel()):
            hi, lo = [a.clone() for a in args], [a.clone() for a in args]
            hi[i].view(-1)[j] += 1e-5
            lo[i].view(-1)[j] -= 1e-5
            d = (loss(*hi) - loss(*lo)) / 2e-5
            # differences are off by h^2 times third derivatives (below 1e3 here), gradients by fp32
            assert abs(float(flat[j]) - d) <= 1e-5 * (1 + abs(d)) + 1e-6, (i, j)


def test_layer_norm_autograd_shapes():
    x = randn((2, 3, 40), 1).requires_grad_(True)
    w = randn((40,), 2)
    y = ag.layer_norm(x, w)
    y.sum().backward()  # an expanded gradient
    y2 = torch.nn.functional.layer_norm(x.detach().double(), (40,), w.double())
    assert y.shape == (2, 3, 40) and float((y.detach().double() - y2).abs().max()) < 1e-5
    assert x.grad.shape == x.shape


def test_layer_norm_refusals():
    x = randn((4, 64), 1)
    mean = rstd = torch.zeros(4, device=DEV)
    with pytest.raises(ValueError):
        p.moe_layer_norm_fwd(x, torch.ones(63, device=DEV))
    with pytest.raises(TypeError):
        p.moe_layer_norm_fwd(x, torch.ones(64, device=DEV), torch.ones(64, device=DEV, dtype=BF))
    with pytest.raises(TypeError):
        p.moe_layer_norm_fwd(x.half())
    with pytest.raises(ValueError):
        p.moe_layer_norm_fwd(x.t())
    with pytest.raises(ValueError):
        p.moe_layer_norm_fwd(x[0])
    with pytest.raises(p.MoeError):
        p.moe_layer_norm_fwd(x, eps=-1.0)
    with pytest.raises(p.MoeError):
        p.moe_layer_norm_fwd(x[:, :0])
    with pytest.raises(TypeError):
        p.moe_layer_norm_bwd(x.to(BF), x, None, mean, rstd)
    with pytest.raises(ValueError):
        p.moe_layer_norm_bwd(x, x, None, mean[:3], rstd)
    with pytest.raises(p.MoeError):
        p.moe_layer_norm_bwd(x, x, None, mean, rstd, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


# --------------------------------------------------------- gradient norm

# A thread adds at most 64 squares in fp32, so the sum is off by 65 u, the norm by half of it.
NORM_REL = 34 * U


def norm64(grads):
    return float(torch.sqrt(sum(g.double().square().sum() for g in grads)))


@pytest.mark.parametrize("align", [1, 64])
@pytest.mark.parametrize("sizes,dtypes", [([1], [F32]), ([5, 1, 33, 70000], [F32, BF]), ([0, 3, 0], [BF]),
                                          (list(range(1, 300, 7)), [BF, F32]), ([32768 * 3 + 5, 17, 16385], [BF]),
                                          ([1 << 21, 100001], [F32])])
def test_grad_norm_and_clip(sizes, dtypes, align):
    grads, outs = [], []
    for i, n in enumerate(sizes):
        dt = dtypes[i % len(dtypes)]
        buf = torch.zeros(2, n + 3 * align + 4, dtype=dt, device=DEV)
        off = (i * 3 % 4) if align == 1 else align
        g = buf[0, off:off + n]
        g.copy_(randn((n,), i, dt))
        grads.append(g)
        # the output sometimes on another alignment than the gradient
        off2 = (off + i % 2) if align == 1 else align
        outs.append(buf[1, off2:off2 + n])
    ref = norm64(grads)
    got = p.moe_grad_norm(grads)
    assert abs(float(got) - ref) <= NORM_REL * ref
    for max_norm in (0.37, 1e9, 0.0):
        s = p.moe_grad_set(grads, outs)
        norm = p.moe_clip_grads(s, max_norm)
        assert float(norm) == float(got)
        c = min(1.0, max_norm / (ref + 1e-6))
        for g, o in zip(grads, outs):
            want = g.double() * c
            check(o, want, (NORM_REL + 4 * U) * want.abs() + type_round(want, g.dtype) * (c != 1), "clip %g" % max_norm)
    keep = [g.clone() for g in grads]
    p.moe_clip_grads(grads, 1e9)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    p.moe_clip_grads(grads, 0.37)  # in place
    c = min(1.0, 0.37 / (ref + 1e-6))
    for g, k in zip(grads, keep):
        check(g, k.double() * c, (NORM_REL + 4 * U) * k.double().abs() * c + type_round(k.double() * c, g.dtype), "in place")


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e15, 1e25, 3e37])
def test_grad_norm_beyond_the_range_of_squares(scale):
    grads = [randn((1000,), 1) * scale, randn((77,), 2), torch.zeros(5000, device=DEV)]
    for gs in (grads[:1], grads[:1] + grads[2:], grads):
        ref, got = norm64(gs), float(p.moe_grad_norm(gs))
        if ref > torch.finfo(F32).max:  # the norm itself has no fp32 value
            assert got == float("inf")
        else:
            assert abs(got - ref) <= NORM_REL * ref
    assert float(p.moe_grad_norm(grads[2:])) == 0.0


def test_grad_norm_special_values_and_guard_bytes():
    g = torch.full((3, 1000), 7.0, device=DEV)
    p.moe_clip_grads([g[1]], 1.0)
    assert bool((g[0] == 7).all()) and bool((g[2] == 7).all()) and float(g[1].norm()) == pytest.approx(1.0, rel=1e-5)
    g[1, 3] = float("inf")
    assert float(p.moe_grad_norm([g[1]])) == float("inf")
    out = torch.empty(1000, device=DEV)
    p.moe_clip_grads(p.moe_grad_set([g[1]], [out]), 1.0)
    assert bool(torch.isnan(out[3])) and bool((out[:3] == 0).all())
    g[1, 3] = float("nan")
    assert bool(torch.isnan(p.moe_clip_grads([g[1]], 1.0))) and bool(torch.isnan(g[1]).all())


def test_grad_norm_streams_graphs_and_repeats():
    grads = [randn((n,), n, BF) for n in (10, 70001, 3, 999999)]
    outs = [torch.empty_like(g) for g in grads]
    s = p.moe_grad_set(grads, outs)
    norm, ws = torch.empty(1, device=DEV), torch.empty_like(s.workspace)
    want = p.moe_clip_grads(s, 0.5).clone()
    keep = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p.moe_clip_grads(s, 0.5, norm, ws)
    torch.cuda.current_stream().wait_stream(side)
    assert float(norm) == float(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.moe_clip_grads(s, 0.5, norm, ws)
    for o in outs:
        o.fill_(float("nan"))
    norm.fill_(0)
    ws.fill_(0xff)
    graph.replay()
    assert float(norm) == float(want) and all(torch.equal(a, b) for a, b in zip(outs, keep))


def test_grad_set_refusals():
    g = randn((8,), 1)
    with pytest.raises(ValueError):
        p.moe_grad_set([])
    with pytest.raises(ValueError):
        p.moe_grad_set([g], [g, g])
    with pytest.raises(ValueError):
        p.moe_grad_set([g], [g[:4]])
    with pytest.raises(TypeError):
        p.moe_grad_set([g.half()])
    with pytest.raises(ValueError):
        p.moe_grad_set([g[::2]])
    with pytest.raises(ValueError):
        p.moe_grad_set([g.cpu()])
    with pytest.raises(p.MoeError):
        p.moe_clip_grads([g], -1.0)
    with pytest.raises(p.MoeError):
        p.moe_clip_grads([g], float("nan"))
    with pytest.raises(ValueError):
        p.moe_grad_norm([g], norm=torch.empty(2, device=DEV))
