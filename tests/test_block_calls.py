"""The native marshalling of the block operators' plain calls: it answers
None to every call that it does not take, and gives the step-by-step calls'
results for the ones that it takes."""
import pytest
import torch

import padded_permute_combine_gb300 as p
from padded_permute_combine_gb300 import _lib
from padded_permute_combine_gb300 import build as libbuild


@pytest.fixture(scope="module")
def calls():
    libbuild.build()
    return _lib.load_calls()


def test_what_is_not_plain_is_left_to_the_caller(calls):
    x, w, row = torch.zeros(2, 8), torch.zeros(8), torch.zeros(2)
    assert calls.layer_norm_fwd(x, w, w, 1e-5) is None  # not on a GPU
    assert calls.layer_norm_fwd(None, w, w, 1e-5) is None and calls.layer_norm_fwd(x, 3, w, 1e-5) is None
    assert calls.layer_norm_fwd(x, w, w) is None and calls.layer_norm_fwd(x, w, w, "a") is None
    assert calls.layer_norm_bwd(x, x, w, row, row, True) is None and calls.layer_norm_bwd(x, x, w, row, None, True) is None
    assert calls.layer(x, x, torch.zeros(2, 8, 8), torch.zeros(2, 8, 4), 1, 0, True) is None
    assert calls.layer(x, x, torch.zeros(2, 8, 8), torch.zeros(2, 8, 4), 1.0, 0, True) is None
    assert calls.experts(x, row.int()[:, None], row[:, None], torch.zeros(2, 8, 8), torch.zeros(2, 8, 4)) is None
    assert calls.grads(x, x, "a") is None and calls.grads() is None


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_plain_calls_equal_the_steps(dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g).cuda().to(dtype)  # noqa: E731
    x, w, b, dy = r(6, 264)[:, :256], r(256), r(256).float(), r(6, 256)
    for weight, bias in ((w, w), (None, None), (b, None), (None, b)):
        got = p.moe_layer_norm_fwd(x, weight, bias)
        steps = p.moe_layer_norm_fwd(x, weight, bias, out=torch.empty_like(dy))
        assert all(torch.equal(a, c) for a, c in zip(got, steps)) and got[0].dtype is dtype and got[0].shape == (6, 256)
        got = p.moe_layer_norm_bwd(dy, x, weight, *steps[1:])
        again = p.moe_layer_norm_bwd(dy, x, weight, *steps[1:], out=torch.empty_like(dy))
        assert all(torch.equal(a, c) and a.dtype is c.dtype for a, c in zip(got, again))
        alone = p.moe_layer_norm_bwd(dy, x, weight, *steps[1:], need_cols=False)
        assert torch.equal(alone[0], got[0]) and alone[1] is None and alone[2] is None
    router, gate_up, down = r(4, 256), r(4, 128, 256), r(4, 256, 64)
    for mode, norm in (("softmax", True), ("sigmoid", False)):
        y, te, wt = p.moe_layer(x, router, gate_up, down, 2, mode, norm)
        steps = p.moe_layer(x, router, gate_up, down, 2, mode, norm, out=torch.empty_like(dy))
        assert torch.equal(y, steps[0]) and torch.equal(te, steps[1]) and torch.equal(wt, steps[2])
        assert torch.equal(p.moe_experts(x, te, wt, gate_up, down), y)
        assert torch.equal(p.moe_experts(x, te, wt, gate_up, down, out=torch.empty_like(dy)), y)
    s = p.moe_grad_set([r(1000), r(33, 7)])
    norm = torch.empty((), device="cuda")
    assert torch.equal(p.moe_grad_norm(s), p.moe_grad_norm(s, norm=norm))
    before = [t.clone() for t in s.grads]
    got = p.moe_clip_grads(s, 1.0)
    after = [t.clone() for t in s.grads]
    for t, o in zip(s.grads, before):
        t.copy_(o)
    assert torch.equal(p.moe_clip_grads(s, 1, norm=norm), got)
    assert all(torch.equal(a, t) for a, t in zip(after, s.grads))
    # on another stream, and from a CUDA graph
    y = p.moe_layer_norm_fwd(x, w, w)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2 = p.moe_layer_norm_fwd(x, w, w)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, y2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3 = p.moe_layer_norm_fwd(x, w, w)[0]
    graph.replay()
    assert torch.equal(y, y3)
