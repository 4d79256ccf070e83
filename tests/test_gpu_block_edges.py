"""The operators around the routing where a fault was found by reading: each
test holds what went wrong, at sizes that reach it. References and tolerances
as in test_gpu_block.py."""
import pytest
import torch

import padded_permute_combine_gb300 as p
from padded_permute_combine_gb300 import _lib
from padded_permute_combine_gb300 import autograd as ag
from test_gpu_block import BF, DEV, F32, check, experts_ref, layer_inputs, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib_loaded():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    p.load()


# H from which on an SM has several tiles of y's columns (128 columns for each of 152 SMs, fewer where the sums of all
# tokens leave less memory), the last tile with fewer columns than the others.
@pytest.mark.parametrize("T,H,F,E,K", [(4, 24576, 96, 4, 2), (40, 24576, 96, 4, 2), (40, 38760, 72, 4, 2), (4, 24577, 97, 4, 2),
                                       (256, 10001, 65, 8, 8), (256, 14001, 65, 8, 8), (256, 24576, 64, 8, 8)])
def test_several_tiles_of_columns_an_sm(T, H, F, E, K):
    """The warps that add a tile's sums keep apart from one tile to the next, however far apart they run."""
    x, router, wgu, wd = layer_inputs(T, H, F, E, BF, T + H)
    y, te, w = p.moe_layer(x, router, wgu, wd, K)
    ref, tol = experts_ref(x, te, w.double(), wgu, wd)
    check(y, ref, tol, "y")
    for _ in range(20):
        assert torch.equal(p.moe_experts(x, te, w, wgu, wd), y)


@pytest.mark.parametrize("need_cols", [True, False])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int32, "fp32"])
def test_layer_norm_bwd_refuses_other_types_of_columns(dtype, need_cols):
    x, row = randn((4, 64), 1), torch.ones(4, device=DEV)
    with pytest.raises(TypeError):
        p.moe_layer_norm_bwd(x, x, None, row, row, weight_dtype=dtype, need_cols=need_cols)


@pytest.mark.parametrize("M,H", [(1, 1), (6, 1000), (40, 257)])
def test_layer_norm_bwd_types_of_columns_without_a_weight(M, H):
    """The type changes the last rounding alone."""
    x, dy = randn((M, H), 1, BF), randn((M, H), 2, BF)
    _, mean, rstd = p.moe_layer_norm_fwd(x)
    dx, dw, db = p.moe_layer_norm_bwd(dy, x, None, mean, rstd)
    for dtype in (F32, BF):
        got = p.moe_layer_norm_bwd(dy, x, None, mean, rstd, weight_dtype=dtype)
        assert got[1].dtype is got[2].dtype is dtype
        assert all(torch.equal(a, b.to(a.dtype)) for a, b in zip(got, (dx, dw, db)))


@pytest.fixture
def give_up():
    """Makes waits inside the kernels give up at once; restored at the end."""
    lib = _lib.load()
    yield lib.moe_test_block_waits
    torch.cuda.synchronize()
    lib.moe_test_block_waits(0)


# One SM, two and more to a tile of y's columns; rows on 16 bytes and off them.
@pytest.mark.parametrize("T,H,F,E,K", [(16, 1024, 1040, 8, 2), (8, 7168, 512, 32, 8), (3, 12288, 520, 6, 1),
                                       (16, 1025, 1041, 8, 2), (8, 7167, 513, 32, 8), (3, 12289, 521, 6, 1)])
@pytest.mark.parametrize("who", [1, 2, 4, 8, 15])
def test_layer_that_gives_up_leaves_nothing_behind(T, H, F, E, K, who, give_up):
    """Weights, tokens, products or sums that never come end the call with a
    status; what was on its way is waited for, and the next call is right."""
    x, router, wgu, wd = layer_inputs(T, H, F, E, BF, T + H)
    y, te, w = p.moe_layer(x, router, wgu, wd, K)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    give_up(who)
    p.moe_experts(x, te, w, wgu, wd, status=status)
    torch.cuda.synchronize()
    give_up(0)
    assert int(status) == _lib.MOE_STATUS_TIMEOUT
    status.zero_()
    for _ in range(3):
        assert torch.equal(p.moe_experts(x, te, w, wgu, wd, status=status), y)
    assert int(status) == 0


@pytest.mark.parametrize("T,H,F,E,K", [(16, 1024, 1040, 8, 2), (8, 7168, 512, 32, 8), (3, 12288, 520, 6, 1), (40, 24576, 96, 4, 2),
                                       (16, 1025, 1041, 8, 2), (8, 7167, 513, 32, 8), (3, 12289, 521, 6, 1)])
@pytest.mark.parametrize("who", [1, 2, 4, 8, 15])
def test_layer_that_gives_up_writes_nan(T, H, F, E, K, who, give_up):
    """No plausible number where sums did not come, whether or not the caller reads a status."""
    x, router, wgu, wd = layer_inputs(T, H, F, E, BF, T + H)
    y, te, w = p.moe_layer(x, router, wgu, wd, K)
    out, ws = torch.zeros_like(y), p.block.layer_workspace(T, H, F, E, K, DEV).zero_()
    give_up(who)
    p.moe_experts(x, te, w, wgu, wd, out=out, workspace=ws)
    plain = p.moe_experts(x, te, w, wgu, wd)
    torch.cuda.synchronize()
    give_up(0)
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(plain).all())
    assert torch.equal(p.moe_experts(x, te, w, wgu, wd, out=out, workspace=ws), y)


# Backward through rings of two and of four vectors a thread; rows off 16 bytes, eight at a time, forward and (the last:
# two arrays of eight such rows are too much for it) backward. What has no copies to wait for gives its ordinary results.
@pytest.mark.parametrize("M,H,dtype,copies", [(1300, 7168, BF, "b"), (3, 1000, BF, "b"), (701, 9000, BF, "b"), (700, 2048, F32, "b"),
                                              (300, 12800, F32, "b"), (1301, 1001, BF, "fb"), (2439, 303, F32, "fb"),
                                              (1223, 4095, BF, "f")])
def test_layer_norm_that_gives_up_writes_nan(M, H, dtype, copies, give_up):
    """Rows that never come leave no plausible number, neither in their own threads' columns nor in the others'; the copies
    on their way are waited for, and the next call is right."""
    x, dy, w = randn((M, H), 1, dtype), randn((M, H), 2, dtype), randn((H,), 3)
    fwd = p.moe_layer_norm_fwd(x, w, w)
    stats = fwd[1:]
    bwd = p.moe_layer_norm_bwd(dy, x, w, *stats)
    give_up(16)
    fwd2, bwd2 = p.moe_layer_norm_fwd(x, w, w), p.moe_layer_norm_bwd(dy, x, w, *stats)
    torch.cuda.synchronize()
    give_up(0)
    for which, got, ordinary in (("f", fwd2, fwd), ("b", bwd2, bwd)):
        if which in copies:
            assert all(bool(torch.isnan(t).all()) for t in got)
        else:
            assert all(torch.equal(a, b) for a, b in zip(got, ordinary))
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(p.moe_layer_norm_fwd(x, w, w), fwd))
        assert all(torch.equal(a, b) for a, b in zip(p.moe_layer_norm_bwd(dy, x, w, *stats), bwd))


def test_gradients_are_not_differentiated_in_silence():
    """A second derivative that the functions do not have is an error, not a missing term."""
    T, H, E, K = 6, 32, 4, 2
    x, w = randn((T, H), 1).requires_grad_(), randn((H,), 2).requires_grad_()
    probs = torch.softmax(randn((T, E), 3), 1).requires_grad_()
    chosen = torch.zeros(T, E, dtype=torch.bool, device=DEV).scatter(1, probs.topk(K).indices, True)
    weights, index = ag.routing_map_to_mok_inputs(probs, chosen, K)
    route = p.moe_route_build(index, E)
    xe = randn((E, T, H), 4).requires_grad_()
    share = weights.detach().requires_grad_()
    for out, leaf in ((ag.layer_norm(x, w), x), (ag.layer_norm(x, w), w), (weights, probs), (ag.permute(x, route, E, T, K), x),
                      (ag.combine(xe, share, route, T, K), xe), (ag.combine(xe, share, route, T, K), share)):
        (grad,) = torch.autograd.grad(out.square().sum(), leaf, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            grad.square().sum().backward()
