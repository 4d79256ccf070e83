"""moe_beam_select against the definition in 64 bits. Scores are rounded once
(2^-24 relative) and come from log sums that are off by at most 2e-7 (32-bit
exponentials, 2^-22 each). Chosen beams and tokens must be the definition's
unless totals are closer than that; the inputs below keep them apart or equal."""
import math

import pytest
import torch

import padded_permute_combine_gb300 as p

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def totals(logits, scores, ended=None, end_token=-1):
    x = logits.double()
    t = scores.double()[:, :, None] + torch.log_softmax(x, 2)
    if ended is not None:
        t = torch.where(ended.bool()[:, :, None], torch.full_like(t, -math.inf), t)
        t[:, :, end_token] = torch.where(ended.bool(), scores.double(), t[:, :, end_token])
    bad = ~torch.isfinite(scores)[:, :, None] | torch.isnan(t)
    return torch.where(bad, torch.full_like(t, -math.inf), t)


def check(logits, scores, n, ended=None, end_token=-1, **kw):
    B, W, V = logits.shape
    got = p.moe_beam_select(logits, scores, n, ended, end_token, **kw)
    t = totals(logits, scores, ended, end_token).flatten(1)
    top = torch.sort(t, dim=1, descending=True, stable=True)
    k = min(n, W * V)
    score, at = top.values[:, :k], top.indices[:, :k]
    some = score > -math.inf
    rows = torch.where(some, at // V + torch.arange(B, device="cuda")[:, None] * W, -1)
    tokens = torch.where(some, at % V, -1)
    assert got[0].dtype == F32 and got[1].dtype == got[2].dtype == torch.int32
    assert torch.equal(got[0][:, :k] > -math.inf, some)
    assert bool(((got[0][:, :k].double() - score).abs()[some] <= 2e-7 + 2.0 ** -24 * score.abs()[some]).all())
    # The same choice, but where two totals of different beams are nearer than the log sums' error.
    flat = got[1][:, :k].long() % W * V + got[2][:, :k]
    alike = (got[1][:, :k] == rows) & (got[2][:, :k] == tokens)
    mine = torch.where(some, t.gather(1, flat.clamp(min=0)), score)
    assert bool((alike | ((mine - score).abs() <= 4e-7)).all())
    assert int((~alike).sum()) <= 2
    for b in range(B):  # no candidate twice
        real = flat[b][some[b]].tolist()
        assert len(set(real)) == len(real)
    assert bool((got[0][:, k:] == -math.inf).all()) and bool((got[1][:, k:] == -1).all()) and bool((got[2][:, k:] == -1).all())
    return got


def rand(*shape, dtype=F32, seed=0, scale=2.5):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).cuda().to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,W,V,n", [(1, 1, 1, 1), (1, 1, 1, 5), (2, 1, 31, 7), (1, 4, 32000, 8), (3, 5, 50257, 10), (2, 8, 511, 16),
                                     (2, 3, 513, 128), (70, 2, 1000, 4), (1, 64, 5000, 128), (4, 2, 129280, 1), (1, 64, 260000, 64)])
def test_shapes(dtype, B, W, V, n):
    check(rand(B, W, V, dtype=dtype, seed=V), rand(B, W, seed=1, scale=1.0) - 20, n)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ties_go_to_the_lowest(dtype):
    x = torch.zeros(2, 3, 5000, dtype=dtype, device="cuda")  # everything equal
    got = check(x, torch.zeros(2, 3, device="cuda"), 100)
    assert got[2][1].tolist() == list(range(100)) and bool((got[1][1] == 3).all())
    x[:, :, 4000:] = 1.0  # a thousand equal ones, behind
    got = check(x, torch.zeros(2, 3, device="cuda"), 128)
    assert got[2][0].tolist() == list(range(4000, 4128))
    x = (rand(2, 4, 30000) * 2).round().div(2).to(dtype)  # a few hundred values
    x[:, 1] = x[:, 0]  # a beam twice
    check(x, torch.zeros(2, 4, device="cuda"), 60)
    got = check(x[:, :2, :37].contiguous(), torch.zeros(2, 2, device="cuda"), 60)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sorted_logits(dtype):
    """The best all in one unit, in rising order: the worst case of the list of candidates."""
    x = torch.arange(20000, device="cuda").div(1000).to(dtype).repeat(2, 2, 1)
    s = torch.tensor([[0.0, -0.3], [-5.0, -9.0]], device="cuda")
    check(x, s, 128)
    check(x.flip(2).contiguous(), s, 128)
    check(x[:, :, :1000].contiguous(), s, 128)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_masks(dtype):
    x, s = rand(3, 4, 3000, dtype=dtype), rand(3, 4, seed=2, scale=1.0)
    x[:, :, ::2] = -math.inf            # tokens that are not allowed
    x[0, 1] = -math.inf                 # a beam without any
    x[1, :, :] = -math.inf
    x[1, 2, 77] = 0.5                   # a request with one candidate
    s[2, 0], s[2, 3] = -math.inf, math.nan  # beams that do not count
    x[0, 2, 5], x[2, 1, 7] = math.nan, math.inf  # nothing of these
    got = check(x, s, 12)
    assert got[2][1].tolist() == [77] + [-1] * 11 and got[0][1, 0] == s[1, 2]
    low = torch.finfo(dtype).min
    y = rand(1, 2, 1000, dtype=dtype)
    y[:, :, 500:] = low                 # masked by the type's lowest value: candidates all the same
    t = check(y[:, :, 495:].contiguous(), torch.zeros(1, 2, device="cuda"), 9)
    assert bool((t[2] < 5).all())
    check(torch.full((1, 1, 600), low, dtype=dtype, device="cuda"), torch.zeros(1, 1, device="cuda"), 3)
    all_dead = p.moe_beam_select(x, torch.full_like(s, -math.inf), 5)
    assert bool((all_dead[0] == -math.inf).all()) and bool((all_dead[1] == -1).all()) and bool((all_dead[2] == -1).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", [torch.bool, torch.uint8])
def test_ended(dtype, kind):
    x, s = rand(4, 3, 2000, dtype=dtype), rand(4, 3, seed=3, scale=1.0)
    ended = torch.tensor([[0, 0, 0], [1, 0, 0], [1, 1, 1], [0, 1, 0]], device="cuda").to(kind)
    x[2, 0] = math.nan  # what an ended beam's logits hold does not matter
    s[3, 1] = 50.0
    got = check(x, s, 6, ended, 2)
    assert got[1][3, 0] == 10 and got[2][3, 0] == 2 and got[0][3, 0] == 50.0
    assert bool((got[1][2, 3:] == -1).all())
    s[2] = -math.inf
    check(x, s, 6, ended, 1999)


def test_large_and_distant_values():
    for dtype in (BF16, F32):
        x = rand(2, 3, 4000, dtype=dtype, scale=1000.0)
        check(x, rand(2, 3, scale=100.0), 20)
        y = rand(1, 2, 4000, dtype=dtype)
        y[0, 0] += 1e6  # rows far apart whose totals are near each other
        check(y, torch.zeros(1, 2, device="cuda"), 20)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("off,pad", [(0, 8), (1, 0), (3, 5), (2, 2), (4, 4)])
def test_strides_and_alignment(dtype, off, pad):
    B, W, V = 3, 2, 4003
    wide = rand(B * W * (V + pad) + off, dtype=dtype)[off:].view(B, W, V + pad)
    x, s = wide[:, :, :V], rand(B, W, seed=4, scale=1.0)
    got = check(x, s, 9)
    # Rows off 16 bytes are summed in another order: both are within the log sums' error, not equal to the bit.
    one, packed = check(x[:, 1:], s[:, 1:].contiguous(), 9), check(x[:, 1:].contiguous(), s[:, 1:].contiguous(), 9)
    assert bool(((one[0] - packed[0]).abs() <= 4e-7 + 2.0 ** -23 * one[0].abs()).all())
    assert got[0].shape == (B, 9)


def test_outputs_streams_and_graphs():
    x, s = rand(3, 4, 9999, dtype=BF16), rand(3, 4, seed=5)
    want = check(x, s, 8)
    out = (torch.empty(3, 8, device="cuda"), *(torch.empty(3, 8, dtype=torch.int32, device="cuda") for _ in range(2)))
    ws = torch.full((p._lib.load().moe_beam_select_workspace_size(3, 4, 9999),), 255, dtype=torch.uint8, device="cuda")
    got = p.moe_beam_select(x, s, 8, out=out, workspace=ws)
    assert all(a is b for a, b in zip(got, out)) and all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = p.moe_beam_select(x, s, 8)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(other, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = p.moe_beam_select(x, s, 8)
    for seed in (6, 7):
        x.copy_(rand(3, 4, 9999, dtype=BF16, seed=seed))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(held, p.moe_beam_select(x, s, 8)))
    assert p.moe_beam_select(x[:0], s[:0], 8)[0].shape == (0, 8)
