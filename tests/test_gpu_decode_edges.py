"""The decode operators where their arguments end: tables that are full, numbers
that need more than 32 bits. What is compared is exact."""
import pytest
import torch

import padded_permute_combine_gb300 as p
from padded_permute_combine_gb300 import _lib

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(autouse=True)
def needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def rand(*shape, dtype=BF16, seed=1):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).cuda().to(dtype)


def ints(*v):
    return torch.tensor(v, dtype=I32, device="cuda")


def equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (BF16, 128), (BF16, 77), (BF16, 100), (BF16, 250), (F32, 64), (F32, 77), (F32, 200)])
@pytest.mark.parametrize("rows,window", [(1, 0), (3, 0), (3, 20), (40, 0)])
def test_a_new_token_beyond_the_table_is_left_out(dtype, dim, rows, window):
    """Rows whose table is full, their length one more: nothing is written, and what the table holds is looked at.
    With several rows, the second and third name the same last page, as after a fork without a column to grow into."""
    width, page = 3, 16
    table = torch.arange(rows * width, dtype=I32, device="cuda").view(rows, width)
    if rows > 2:
        table[2, width - 1] = table[1, width - 1]
    k, v = (rand(rows * width, page, 2, dim, dtype=dtype, seed=s) for s in (2, 3))
    q, kn, vn = (rand(rows, h, dim, dtype=dtype, seed=s) for h, s in ((6, 4), (2, 5), (2, 6)))
    full = torch.full((rows,), width * page, dtype=I32, device="cuda")
    want = p.moe_attention_decode(q, k, v, table, full, window=window)
    before, status = (k.clone(), v.clone()), ints(0)
    for more in (1, 1000):
        got = p.moe_attention_decode(q, k, v, table, full + more, kn, vn, window=window, status=status)
        assert int(status) == _lib.MOE_STATUS_BAD_INDEX
        assert equal((k, v), before) and equal(got, want)
        assert equal(p.moe_attention_decode(q, k, v, table, full + more, kn, vn, window=window), want) and equal((k, v), before)
    # The last place of a table is one all the same.
    own = table.clone()
    own[:, width - 1] = torch.arange(rows, device="cuda") * width + width - 1
    p.moe_attention_decode(q, k, v, own, full, kn, vn, window=window)
    assert torch.equal(k[own[:, -1].long(), page - 1], kn) and torch.equal(v[own[:, -1].long(), page - 1], vn)


def test_a_write_of_more_than_2_to_the_30_sequences():
    """Three tokens, of the sequences 5, 2^30 + 7 and the last one."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    n = (1 << 30) + 1000
    offsets, lengths, table = (torch.zeros(n + i, dtype=I32, device="cuda") for i in (1, 0, 0))
    table = table[:, None]
    for i, b in enumerate((5, (1 << 30) + 7, n - 1)):
        offsets[b + 1:], lengths[b], table[b, 0] = i + 1, i + 1, i  # to position i of page i
    k, v, new, status = rand(4, 4, 1, 8), rand(4, 4, 1, 8, seed=2), rand(3, 1, 8, seed=3), ints(0)
    want = k.clone(), v.clone()
    for i in range(3):
        want[0][i, i], want[1][i, i] = new[i], -new[i]
    p.moe_cache_write(new, -new, k, v, table, offsets, lengths, status=status)
    assert equal((k, v), want) and int(status) == 0


def test_a_selection_over_almost_2_to_the_31_rows():
    """A vocabulary of one token, so that totals are the scores: the best beam of each request."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    B, W = (1 << 25) - 1, 64
    logits = torch.zeros(B, W, 1, dtype=BF16, device="cuda")
    scores = torch.rand(B, W, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda")
    best, parents, tokens = p.moe_beam_select(logits, scores, 1)
    assert torch.equal(best[:, 0], scores.amax(1)) and bool((tokens == 0).all())
    assert torch.equal(parents[:, 0].long() // W, torch.arange(B, device="cuda"))
    assert torch.equal(scores.view(-1)[parents[:, 0].long()], best[:, 0])


def test_numbers_beyond_what_the_c_abi_takes_are_refused():
    """Not cut to their low bits: a window of 2^64 + 7 is none of 7 tokens."""
    table, lengths, parents = ints(0, 1, 2).view(1, 3), ints(40), ints(0, 0)
    q, k = rand(1, 4, 64), rand(4, 16, 2, 64)
    x, s = rand(1, 3, 100), torch.zeros(1, 3, device="cuda")
    for call, bits in ((lambda: p.moe_attention_decode(q, k, k, table, lengths, window=2 ** 64 + 7), 64),
                       (lambda: p.moe_cache_fork(table, lengths, parents, 16, 9, 2 ** 64 + 1), 64),
                       (lambda: p.moe_cache_fork(table, lengths, parents, 16, 2 ** 64 + 9), 64),
                       (lambda: p.moe_cache_compact(table, lengths, 16, 2 ** 64 + 9), 64),
                       (lambda: p.moe_beam_select(x, s, 2 ** 32 + 3), 32)):
        with pytest.raises(ValueError, match="%d bits" % bits):
            call()


@pytest.mark.parametrize("dim", [1, 2, 3])
def test_sizes_beyond_32_bits_are_refused(dim):
    """A cache's page size, kv heads or head size of 2^32 and some: their low bits alone would be a small cache."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    shape = [1, 1, 1, 1]
    shape[dim] = 2 ** 32 + 2
    k = torch.empty(shape, dtype=BF16, device="cuda")
    new = k[:, 0]
    for call in (lambda: p.moe_attention_decode(new, k, k, ints(0).view(1, 1), ints(1)),
                 lambda: p.moe_cache_write(new, new, k, k, ints(0).view(1, 1), ints(0, 1), ints(1))):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_beams_beyond_32_bits_are_refused():
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    x = torch.zeros(1, 2 ** 32 + 5, 1, dtype=BF16, device="cuda")
    with pytest.raises(ValueError, match="32 bits"):
        p.moe_beam_select(x, torch.zeros(1, 2 ** 32 + 5, device="cuda"), 2)


@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (BF16, 100), (BF16, 77), (F32, 64), (F32, 77)])
@pytest.mark.parametrize("length", [40, 5000])
def test_infinite_scores(dtype, dim, length):
    """+infinity among a head's scores: NaN. -infinity: no weight; nothing else: as without positions."""
    pages = -(-length // 16)
    k, v = rand(pages, 16, 2, dim, dtype=dtype, seed=2), rand(pages, 16, 2, dim, dtype=dtype, seed=3)
    q = rand(1, 6, dim, dtype=dtype, seed=4).abs() + 0.5  # positive: an infinite key has a score of its sign
    table, lengths = torch.arange(pages, dtype=I32, device="cuda")[None], ints(length)
    want = p.moe_attention_decode(q, k, v, table, lengths)
    k[1, 5, 0] = torch.inf
    out, lse = p.moe_attention_decode(q, k, v, table, lengths)
    assert bool(torch.isnan(out[0, :3]).all()) and bool(torch.isnan(lse[0, :3]).all())
    assert equal((out[0, 3:], lse[0, 3:]), (want[0][0, 3:], want[1][0, 3:]))
    k[:, :, 0] = -torch.inf
    out, lse = p.moe_attention_decode(q, k, v, table, lengths)
    assert bool((out[0, :3] == 0).all()) and bool((lse[0, :3] == -torch.inf).all())
    assert equal((out[0, 3:], lse[0, 3:]), (want[0][0, 3:], want[1][0, 3:]))
    k[0, 7, 0] = 0.25  # one score is a number: all weight
    out, lse = p.moe_attention_decode(q, k, v, table, lengths)
    assert torch.equal(out[0, :3], v[0, 7, 0].expand(3, dim)) and bool(torch.isfinite(lse).all())
