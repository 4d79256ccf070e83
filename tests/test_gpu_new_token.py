"""The new token that moe_attention_decode writes on its way, in every variant of
the kernels: the cache afterwards exactly, the output against 64 bits with the
tolerances of test_gpu_attention.py."""
import pytest
import torch

import padded_permute_combine_gb300 as p
from test_gpu_attention import check, make, rand

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def put(k, v, table, lengths, kn, vn):
    """The caches with the new tokens in their places."""
    page = k.shape[1]
    for t, new in ((k, kn), (v, vn)):
        t = t.clone()
        for b, n in enumerate(lengths):
            if n:
                t[table[b, (n - 1) // page].long(), (n - 1) % page] = new[b]
        yield t


def run(dtype, heads, kv, dim, page, heads_first=False, pad=0, window=0, off=0):
    lengths = [1, 0, 17, 16, 333, 1500, page, page + 1]
    k, v, table, dev = make(lengths, page, kv, dim, dtype, heads_first, pad=pad)
    B, rows = len(lengths), heads + 2 * kv
    qkv = rand(B, rows, dim + off, dtype=dtype, seed=5)[..., off:]  # slices of one projection, `off` elements off its alignment
    q, kn, vn = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    want = list(put(k, v, table, lengths, kn, vn))
    whole = [t.as_strided((t.numel() // dim * (dim + pad),), (1,), 0).clone() if pad else None for t in (k, v)]
    got = check(q, (k, v), table, dev, lengths, window=window, new=(kn, vn))
    for t, w in zip((k, v), want):
        assert torch.equal(torch.nan_to_num(t, 123.0), torch.nan_to_num(w, 123.0))
    for t, before in zip((k, v), whole):  # nothing between the rows
        if before is not None:
            now = t.as_strided((before.numel(),), (1,), 0)
            gap = torch.arange(now.numel(), device="cuda") % (dim + pad) >= dim
            assert torch.equal(now[gap], before[gap])
    again = p.moe_attention_decode(q, k, v, table, dev, window=window)  # the cache holds them now
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,kv", [(4, 2), (9, 1), (20, 1)])
@pytest.mark.parametrize("dim", [1, 2, 30, 33, 64, 66, 77, 96, 100, 126, 127, 128, 130, 150, 187, 192, 193, 198, 250, 251, 256])
def test_head_sizes(dtype, heads, kv, dim):
    """Rows on 16, 4 and 2 bytes, of one warp and of teams of two to four, up to 8 heads at a time, 16, and more."""
    run(dtype, heads, kv, dim, 16)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("dim,page,pad,off", [(128, 16, 8, 0), (100, 5, 2, 0), (100, 16, 28, 4), (64, 13, 1, 1), (250, 7, 6, 2), (192, 16, 64, 0), (256, 1, 1, 3)])
def test_padded_rows_and_odd_projections(dtype, heads_first, dim, page, pad, off):
    run(dtype, 6, 2, dim, page, heads_first, pad, off=off)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 77, 100, 128, 150, 250])
@pytest.mark.parametrize("window", [1, 2, 16, 100, 1499])
def test_windows(dtype, dim, window):
    run(dtype, 8, 2, dim, 16, window=window)
