"""moe_attention_decode and moe_cache_write against plain arithmetic in 64 bits.

Tolerances, per element of an output y = sum_j p_j v_j with A = sum_j p_j |v_j|
over n positions: the rounding of y (half a step); a score is off by at most
ds = (D + 8) 2^-23 scale sum |q k| (each of D products and sums, cut or
rounded), which moves every p_j by at most 2 ds; the probabilities keep 16 bits
at least (2^-16) and sums of n terms lose n 2^-24. So
|err| <= half |y| + A (2 ds + 2^-16 + n 2^-24) in bf16, and 2^-21 in place of 2^-16
in fp32 (the exponential's own error)."""
import math

import pytest
import torch

import padded_permute_combine_gb300 as p
from padded_permute_combine_gb300 import _lib

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def make(lengths, page, kv, dim, dtype, heads_first=False, seed=0, spare=2, width=None, pad=0, nan=True):
    """Caches, table and lengths; what no position names holds NaN. ``pad``: elements between rows."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-n // page) for n in lengths]
    pool = sum(counts) + spare
    shape = (pool, kv, page, dim + pad) if heads_first else (pool, page, kv, dim + pad)
    caches = []
    for _ in range(2):
        t = torch.randn(shape, generator=g).cuda().to(dtype)
        caches.append((t.transpose(1, 2) if heads_first else t)[..., :dim])
    ids = torch.randperm(pool, generator=g).to(torch.int32)
    w = width or max(counts + [1]) + 1
    table = torch.full((len(lengths), w), -7, dtype=torch.int32)  # what lies behind a row's pages does not matter
    at = 0
    mask = torch.ones(pool, page, dtype=torch.bool)
    for b, c in enumerate(counts):
        table[b, :c] = ids[at:at + c]
        for j in range(c):
            mask[ids[at + j], : min(page, lengths[b] - j * page)] = False
        at += c
    if nan:
        for t in caches:
            t[mask.cuda()] = math.nan
    return *caches, table.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda")


def gathered(cache, table, b, first, n):
    page = cache.shape[1]
    pos = torch.arange(first, n, device="cuda")
    return cache[table[b][pos // page].long(), pos % page].double()  # [tokens, kv, dim]


def reference(q, k_cache, v_cache, table, lengths, window, scale, absent=()):
    """out, lse, and the tolerances of both (without out's own rounding)."""
    B, H, D = q.shape
    kv = k_cache.shape[2]
    out, lse, tol, ltol = (torch.zeros(s, dtype=torch.float64, device="cuda") for s in ((B, H, D), (B, H), (B, H, D), (B, H)))
    for b, n in enumerate(lengths):
        first = max(0, n - window) if window else 0
        keep = [j for j in range(first, n) if (b, j // k_cache.shape[1]) not in absent]
        if not keep:
            lse[b] = -math.inf
            continue
        at = torch.tensor(keep, device="cuda")
        ids, inside = table[b][at // k_cache.shape[1]].long(), at % k_cache.shape[1]
        k, v = (t[ids, inside].double().repeat_interleave(H // kv, 1).transpose(0, 1) for t in (k_cache, v_cache))
        x = torch.einsum("hd,hnd->hn", q[b].double(), k) * scale
        ds = (D + 8) * 2.0 ** -23 * abs(scale) * torch.einsum("hd,hnd->hn", q[b].double().abs(), k.abs()).amax(1)
        pr = torch.softmax(x, 1)
        out[b], lse[b] = torch.einsum("hn,hnd->hd", pr, v), torch.logsumexp(x, 1)
        base = 2.0 ** -21 if q.dtype == F32 else 2.0 ** -16
        part = 2 * ds + base + len(keep) * 2.0 ** -24
        tol[b] = torch.einsum("hn,hnd->hd", pr, v.abs()) * part[:, None]
        ltol[b] = part + 2.0 ** -22 * lse[b].abs()
    return out, lse, tol, ltol


def check(q, caches, table, lengths_dev, lengths, window=0, scale=None, new=None, absent=(), **kw):
    D = q.shape[2]
    s = D ** -0.5 if scale is None else scale
    out, lse = p.moe_attention_decode(q, *caches, table, lengths_dev, *(new or ()), scale=scale, window=window, **kw)
    want, wlse, tol, ltol = reference(q, *caches, table, lengths, window, s, absent)
    half = torch.finfo(q.dtype).eps / 2
    assert out.dtype == q.dtype and out.shape == q.shape and lse.dtype == F32
    err = (out.double() - want).abs()
    assert bool((err <= half * want.abs() + tol + 1e-30).all()), float((err / (half * want.abs() + tol + 1e-30)).max())
    empty = torch.isinf(wlse)
    assert torch.equal(torch.isinf(lse), empty) and bool((lse[empty] == -math.inf).all())
    assert bool(((lse.double() - wlse).abs()[~empty] <= ltol[~empty]).all())
    for t in (out, lse):
        assert bool((t[empty] == (0 if t is out else -math.inf)).all())
    return out, lse


def rand(*shape, dtype=BF16, seed=1, scale=1.5):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).cuda().to(dtype)


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,kv,dim,page", [
    (8, 8, 64, 16), (8, 2, 128, 16), (6, 1, 128, 1), (7, 1, 80, 13), (12, 2, 96, 32), (16, 1, 128, 64), (24, 2, 256, 16),
    (40, 2, 128, 8), (6, 2, 150, 16), (20, 1, 187, 9), (3, 3, 33, 5), (5, 5, 1, 4), (32, 4, 72, 7), (33, 1, 250, 100), (18, 2, 192, 16), (64, 1, 64, 16)])
def test_head_layouts(dtype, heads_first, heads, kv, dim, page):
    lengths = [1, 0, 37, 16, 15, 17, 300, 2]
    k, v, table, dev = make(lengths, page, kv, dim, dtype, heads_first)
    check(rand(len(lengths), heads, dim, dtype=dtype), (k, v), table, dev, lengths)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lengths", [[1], [0], [0, 0, 0], [5000], [4096, 1, 0, 9000], [3] * 700, [0] * 300 + [5] + [0] * 300 + [70],
                                     list(range(130)), [33000]])
def test_lengths(dtype, lengths):
    k, v, table, dev = make(lengths, 16, 2, 128, dtype, nan=len(lengths) < 100)
    check(rand(len(lengths), 8, 128, dtype=dtype), (k, v), table, dev, lengths)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window", [1, 15, 16, 100, 4096, 1 << 40])
def test_windows(dtype, window):
    lengths = [1, 0, 99, 100, 101, 5000, 64]
    k, v, table, dev = make(lengths, 16, 2, 64, dtype)
    check(rand(len(lengths), 4, 64, dtype=dtype), (k, v), table, dev, lengths, window=window)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,kv,dim,page", [(8, 2, 128, 16), (40, 2, 64, 3), (5, 1, 77, 16)])
def test_new_tokens_are_written_and_read(dtype, heads, kv, dim, page):
    lengths = [1, 0, 17, 16, 333, 4000]
    k, v, table, dev = make(lengths, page, kv, dim, dtype)
    qkv = rand(len(lengths), heads + 2 * kv, dim, dtype=dtype, seed=5)  # slices of one projection
    q, kn, vn = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    want = []
    for t, new in ((k, kn), (v, vn)):
        w = t.clone()
        for b, n in enumerate(lengths):
            if n:
                w[table[b, (n - 1) // page].long(), (n - 1) % page] = new[b]
        want.append(w)
    got = check(q, (k, v), table, dev, lengths, new=(kn, vn))
    for t, w in zip((k, v), want):
        assert torch.equal(torch.nan_to_num(t, 123.0), torch.nan_to_num(w, 123.0))
    again = p.moe_attention_decode(q, k, v, table, dev)  # the cache holds them now
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,pad", [(64, 1), (128, 8), (64, 4), (30, 2), (128, 128)])
def test_strides_and_alignment(dtype, dim, pad):
    lengths = [5, 100, 31]
    k, v, table, dev = make(lengths, 16, 2, dim, dtype, pad=pad)
    q = rand(3, 4, dim + pad, dtype=dtype)[..., pad:]
    wide = torch.full((3, table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    check(q, (k, v), wide[:, :table.shape[1]], dev, lengths)
    # one element off the allocation's start
    flat = [torch.empty(t.numel() + 1, dtype=dtype, device="cuda")[1:].view(t.shape) for t in (k, v)]
    for f, t in zip(flat, (k, v)):
        f.copy_(t)
    check(q, flat, table, dev, lengths)


def test_extreme_scores():
    lengths = [50, 200]
    for dtype in (BF16, F32):
        k, v, table, dev = make(lengths, 16, 1, 64, dtype)
        q = rand(2, 4, 64, dtype=dtype)
        check(q, (k, v), table, dev, lengths, scale=30.0)
        check(q, (k, v), table, dev, lengths, scale=-0.5)
        check(q, (k, v), table, dev, lengths, scale=0.0)
        big = torch.finfo(dtype).max
        ids = table[1].long()
        v[ids[0], 3] = big  # a value near the type's largest, among ordinary ones
        check(q, (k, v), table, dev, lengths)
        # An infinite score takes all weight or none, as the formula says: a NaN, or nothing of that key.
        v[ids[0], 3] = 1.0
        k[ids[0], 3] = -math.inf
        q2 = q.abs()
        out, lse = p.moe_attention_decode(q2, k, v, table, dev)
        v2, k2 = v.clone(), k.clone()
        k2[ids[0], 3] = 0
        pos = [j for j in range(200) if j != 3]
        kk, vv = (gathered(t, table, 1, 0, 200)[pos][:, 0] for t in (k2, v2))
        want = torch.softmax(q2[1].double() @ kk.t() / 8, 1) @ vv
        assert bool(((out[1].double() - want).abs() <= 2.0 ** -7 * (1 + want.abs())).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128, 77, 200])
@pytest.mark.parametrize("lengths", [[40, 200], [9000, 200]])
def test_nan_stays_with_its_row(dtype, dim, lengths):
    k, v, table, dev = make(lengths, 16, 2, dim, dtype)
    q = rand(2, 8, dim, dtype=dtype)
    want = p.moe_attention_decode(q, k, v, table, dev)
    k[table[0, 1].long(), 3, 0] = math.nan  # a key of the first sequence's first kv head
    out, lse = p.moe_attention_decode(q, k, v, table, dev)
    assert bool(torch.isnan(out[0, :4]).all()) and bool(torch.isnan(lse[0, :4]).all())
    assert torch.equal(out[0, 4:], want[0][0, 4:]) and torch.equal(lse[0, 4:], want[1][0, 4:])
    assert torch.equal(out[1], want[0][1]) and torch.equal(lse[1], want[1][1])


def test_bad_pages_and_lengths_are_flagged_and_left_out():
    lengths = [40, 64, 33]
    k, v, table, _ = make(lengths, 16, 2, 64, BF16)
    table[0, 1], table[2, 0] = k.shape[0], -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    q = rand(3, 4, 64)
    check(q, (k, v), table, dev, lengths, absent={(0, 1), (2, 0)}, status=status)
    assert int(status) == _lib.MOE_STATUS_BAD_INDEX
    status.zero_()
    odd = torch.tensor([-5, 10 ** 9, 33], dtype=torch.int32, device="cuda")
    width = table.shape[1]
    out, lse = p.moe_attention_decode(q, k, v, table, odd, status=status)
    assert int(status) == _lib.MOE_STATUS_BAD_INDEX and bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    full = torch.tensor([0, width * 16, 33], dtype=torch.int32, device="cuda")
    assert torch.equal(out, p.moe_attention_decode(q, k, v, table, full)[0])
    # all of a sequence's pages are bad: an empty row
    table[1] = -1
    out, lse = p.moe_attention_decode(q, k, v, table, dev)
    assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all())
    # a new token whose page is bad is left out, and nothing is written
    before = k.clone()
    kn = rand(3, 2, 64, seed=9)
    p.moe_attention_decode(q[1:2], k, v, table[1:2], dev[1:2], kn[1:2], kn[1:2])
    assert torch.equal(torch.nan_to_num(before, 99.0), torch.nan_to_num(k, 99.0))


def test_repeats_streams_graphs_and_outputs():
    lengths = [9000, 100, 0, 2000]
    k, v, table, dev = make(lengths, 16, 2, 128, BF16)
    q, kn = rand(4, 8, 128), rand(4, 2, 128, seed=3)
    out, lse = p.moe_attention_decode(q, k, v, table, dev, kn, kn)
    for _ in range(3):
        o2, l2 = p.moe_attention_decode(q, k, v, table, dev, kn, kn)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o3, _ = p.moe_attention_decode(q, k, v, table, dev)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, o3)
    ws = p.decode.attention_workspace(4, 8, 2, 128, "cuda:0")
    ws.fill_(255)  # its contents need no initialisation
    o4, l4 = torch.full_like(out, 7), torch.full_like(lse, 7)
    got = p.moe_attention_decode(q, k, v, table, dev, out=o4, lse=l4, workspace=ws)
    assert got[0] is o4 and got[1] is l4 and torch.equal(o4, out) and torch.equal(l4, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o5, l5 = p.moe_attention_decode(q, k, v, table, dev)
    graph.replay()
    assert torch.equal(o5, out)
    dev.copy_(torch.tensor([100, 9, 1, 1999]))  # other lengths in the same graph; sequence 2 has a page after all
    table[2, 0] = table[0, 500]
    graph.replay()
    want = p.moe_attention_decode(q, k, v, table, dev)
    assert torch.equal(o5, want[0]) and torch.equal(l5, want[1])


def test_offsets_beyond_32_bits():
    """A pool of 5 G elements: the page's number times its stride does not fit 32 bits, nor does it in bytes."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    pool, page, kv, dim = 1 << 17, 16, 16, 160
    k = torch.empty(pool, page, kv, dim, dtype=BF16, device="cuda")
    v = torch.empty_like(k)
    ids = torch.tensor([pool - 1, 0, pool // 2 + 7, pool - 3], device="cuda")
    for t in (k, v):
        t[ids] = torch.randn(4, page, kv, dim, device="cuda").to(BF16)
    table = ids.to(torch.int32)[None]
    dev = torch.tensor([60], dtype=torch.int32, device="cuda")
    check(rand(1, 32, dim), (k, v), table, dev, [60])
    kn = rand(5, kv, dim, seed=4)
    p.moe_cache_write(kn, kn, k, v, table, torch.tensor([0, 5], dtype=torch.int32, device="cuda"), dev)
    assert torch.equal(k[pool - 3, 7:12], kn) and torch.equal(v[pool - 3, 7:12], kn)


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kv,dim,page", [(2, 128, 16), (3, 33, 5), (1, 64, 1), (4, 6, 7), (2, 300, 16)])
def test_write(dtype, heads_first, kv, dim, page):
    counts, before = [5, 0, 1, 40, 0, 129], [0, 9, 16, 3, 0, 1000]
    lengths = [a + b for a, b in zip(counts, before)]
    k, v, table, dev = make(lengths, page, kv, dim, dtype, heads_first, nan=False)
    T = sum(counts)
    new = rand(T + 7, 2 * kv, dim, dtype=dtype)  # rows behind the last sequence are not written
    kn, vn = new[:, :kv], new[:, kv:]
    want = [k.clone(), v.clone()]
    offsets = [sum(counts[:i]) for i in range(7)]
    for b, n in enumerate(counts):
        for i in range(n):
            pos = before[b] + i
            for w, t in zip(want, (kn, vn)):
                w[table[b, pos // page].long(), pos % page] = t[offsets[b] + i]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p.moe_cache_write(kn, vn, k, v, table, torch.tensor(offsets, dtype=torch.int32, device="cuda"), dev, status=status)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and int(status) == 0


def test_write_of_many_sequences():
    counts = [(i * 7) % 4 for i in range(1500)]
    k, v, table, dev = make(counts, 2, 1, 16, F32, nan=False)
    kn = rand(sum(counts), 1, 16, dtype=F32)
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    p.moe_cache_write(kn, -kn, k, v, table, offsets, dev)
    for b in (0, 1, 700, 1499, 1498):
        n = counts[b]
        if n:
            assert torch.equal(gathered(k, table, b, 0, n), kn[int(offsets[b]):int(offsets[b]) + n].double())
            assert torch.equal(gathered(v, table, b, 0, n), -kn[int(offsets[b]):int(offsets[b]) + n].double())


def test_write_flags_bad_input():
    k, v, table, dev = make([20, 20], 16, 1, 32, F32, nan=False)
    kn = rand(10, 1, 32, dtype=F32)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    keep = k.clone()
    for offsets, lengths, bit in (((3, 5, 10), (20, 20), _lib.MOE_STATUS_BAD_BINS), ((0, 9, 4), (0, 0), _lib.MOE_STATUS_BAD_BINS | _lib.MOE_STATUS_BAD_INDEX),
                                  ((0, 5, 900), (5, 950), _lib.MOE_STATUS_BAD_BINS), ((0, 5, 10), (3, 10 ** 8), _lib.MOE_STATUS_BAD_INDEX)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        p.moe_cache_write(kn, kn, k, v, table, i32(*offsets), i32(*lengths), status=status)
        assert int(status) & bit and int(status) | bit == bit, (offsets, int(status))
    k.copy_(keep)
    table[1, 1] = 99
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p.moe_cache_write(kn, kn, k, v, table, i32(0, 0, 10), dev, status=status)
    assert int(status) == _lib.MOE_STATUS_BAD_INDEX
    keep[table[1, 0].long(), 10:16] = kn[:6]  # positions 10 .. 15 have their page, 16 .. 19 do not
    assert torch.equal(k, keep)
