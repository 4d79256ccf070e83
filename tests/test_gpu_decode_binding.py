"""The decode operators' binding on GPU tensors: what it refuses and with which
words, that the native marshalling and the step-by-step calls agree, and that a
failed native call is not made twice."""
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


def new(*s, dtype=BF16):
    return torch.randn(s, generator=torch.Generator().manual_seed(sum(s))).cuda().to(dtype)


def ints(*v):
    return torch.tensor(v, dtype=I32, device="cuda")


def good():
    table = ints(0, 1, 2, 3, 4, 5).view(2, 3)
    return dict(q=new(2, 4, 64), k_cache=new(7, 16, 2, 64), v_cache=new(7, 16, 2, 64), page_table=table, lengths=ints(40, 7),
                k_new=new(2, 2, 64), v_new=new(2, 2, 64))


def test_attention_refuses():
    assert p.moe_attention_decode(**good())[0].shape == (2, 4, 64)
    g = good()
    for change, error, words in (
            (dict(q=new(2, 4, 64, dtype=F32)), TypeError, "q must be"), (dict(q=new(2, 4, 32)), ValueError, "q must be"),
            (dict(q=new(2, 64)), ValueError, "3-D"), (dict(q=g["q"].cpu()), ValueError, "CUDA"),
            (dict(q=new(2, 4, 128)[..., ::2]), ValueError, "contiguous"),
            (dict(k_cache=g["k_cache"].half(), v_cache=g["v_cache"].half(), q=g["q"].half()), TypeError, "float32 or bfloat16"),
            (dict(v_cache=new(7, 16, 2, 32)), ValueError, "v_cache must be"), (dict(v_cache=new(7, 2, 16, 64).transpose(1, 2)), ValueError, "same strides"),
            (dict(k_cache=g["k_cache"][:, :1].expand(7, 16, 2, 64), v_cache=g["v_cache"][:, :1].expand(7, 16, 2, 64)), ValueError, "overlap"),
            (dict(page_table=g["page_table"].long()), TypeError, "page_table"), (dict(page_table=g["page_table"][:1]), ValueError, "lengths must be"),
            (dict(page_table=g["page_table"].t().contiguous().t()), ValueError, "contiguous"),
            (dict(page_table=g["page_table"][:1].expand(2, 3)), ValueError, "overlap"),
            (dict(lengths=ints(40, 7, 1)), ValueError, "lengths"), (dict(lengths=g["lengths"].cpu()), ValueError, "CUDA"),
            (dict(k_new=None), ValueError, "go together"), (dict(k_new=new(2, 4, 64)), ValueError, "k_new must be"),
            (dict(out=new(2, 4, 64, dtype=F32)), TypeError, "out"), (dict(lse=new(2, 4)), TypeError, "lse"),
            (dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda")), _lib.MoeError, "invalid argument"),
            (dict(status=torch.zeros(1, device="cuda")), TypeError, "status"), (dict(window=-1), _lib.MoeError, "invalid argument"),
            (dict(scale=float("nan")), _lib.MoeError, "invalid argument"),
            (dict(q=new(2, 3, 64)), _lib.MoeError, "invalid argument")):  # heads that kv heads do not divide
        with pytest.raises(error, match=words):
            p.moe_attention_decode(**(good() | change))
    wide = dict(q=new(2, 4, 257), k_cache=new(7, 16, 2, 257), v_cache=new(7, 16, 2, 257), k_new=None, v_new=None)
    with pytest.raises(_lib.MoeError, match="unsupported"):
        p.moe_attention_decode(**(good() | wide))


def test_the_others_refuse():
    g = good()
    k, offsets = new(5, 2, 64), ints(0, 3, 5)
    write = lambda **c: p.moe_cache_write(**(dict(k=k, v=k, k_cache=g["k_cache"], v_cache=g["v_cache"], page_table=g["page_table"],  # noqa: E731
                                                  offsets=offsets, lengths=g["lengths"]) | c))
    write()
    for c, e, w in ((dict(k=new(5, 1, 64)), ValueError, "k must be"), (dict(v=new(4, 2, 64)), ValueError, "v must be"),
                    (dict(offsets=ints(0, 5)), ValueError, "offsets"), (dict(offsets=offsets.long()), TypeError, "offsets")):
        with pytest.raises(e, match=w):
            write(**c)
    t, n, parents = g["page_table"], g["lengths"], ints(0, 1, 1)
    for call, e, w in ((lambda: p.moe_cache_fork(t, n, parents.long(), 16, 9), TypeError, "parents"),
                       (lambda: p.moe_cache_fork(t, n, parents[None], 16, 9), ValueError, "parents"),
                       (lambda: p.moe_cache_fork(t, n, parents, 0, 9), _lib.MoeError, "invalid"),
                       (lambda: p.moe_cache_fork(t, n, parents, 16, 9, -1), _lib.MoeError, "invalid"),
                       (lambda: p.moe_cache_fork(t, n, parents, 16, 9, width=2), _lib.MoeError, "invalid"),
                       (lambda: p.moe_cache_fork(t, n, parents, 2 ** 32 + 16, 9), ValueError, "32 bits"),
                       (lambda: p.moe_cache_fork(t, n, parents, 16, _lib.MOE_CACHE_MAX_PAGES + 1), _lib.MoeError, "unsupported"),
                       (lambda: p.moe_cache_compact(t, n[:1], 16, 9), ValueError, "lengths"),
                       (lambda: p.moe_cache_compact(t, n, -1, 9), _lib.MoeError, "invalid"),
                       (lambda: p.moe_cache_copy([g["k_cache"]], parents, n), ValueError, "dst"),
                       (lambda: p.moe_cache_copy([g["k_cache"], g["k_cache"][:6]], n, n), ValueError, "7 pages"),
                       (lambda: p.moe_cache_copy([g["k_cache"][:, ::2]], n, n), ValueError, "one block"),
                       (lambda: p.moe_cache_copy([g["k_cache"][:1].expand(7, 16, 2, 64)], n, n), ValueError, "overlap"),
                       (lambda: p.moe_cache_copy([g["k_cache"]], n, n, parents), ValueError, "count")):
        with pytest.raises(e, match=w):
            call()
    x, s = new(2, 3, 100), new(2, 3, dtype=F32)
    for call, e, w in ((lambda: p.moe_beam_select(x.half(), s, 2), TypeError, "float32 or bfloat16"), (lambda: p.moe_beam_select(x, s.bfloat16(), 2), TypeError, "scores"),
                       (lambda: p.moe_beam_select(x, s[:1], 2), ValueError, "scores"), (lambda: p.moe_beam_select(x, s, 0), _lib.MoeError, "invalid"),
                       (lambda: p.moe_beam_select(x, s, 129), _lib.MoeError, "unsupported"), (lambda: p.moe_beam_select(x.transpose(0, 1), s.t().contiguous(), 2), ValueError, "evenly"),
                       (lambda: p.moe_beam_select(x, s, 2, torch.zeros(2, 3, device="cuda"), 1), TypeError, "ended"),
                       (lambda: p.moe_beam_select(x, s, 2, torch.zeros(2, 3, device="cuda", dtype=torch.bool), 100), _lib.MoeError, "invalid"),
                       (lambda: p.moe_beam_select(x, s, 2, torch.zeros(2, 3, device="cuda", dtype=torch.bool), 2 ** 32), ValueError, "32 bits"),
                       (lambda: p.moe_beam_select(x[:, :1].expand(2, 3, 100), s, 2), ValueError, "evenly|overlap")):
        with pytest.raises(e, match=w):
            call()


def test_native_calls_equal_the_steps():
    g = good()
    status = ints(0)
    a, b = p.moe_attention_decode(**g), p.moe_attention_decode(**g, status=status)
    assert all(torch.equal(x, y) and x.dtype == y.dtype and x.shape == y.shape for x, y in zip(a, b))
    a, b = p.moe_attention_decode(**g, scale=0.3, window=9), p.moe_attention_decode(**g, scale=0.3, window=9, status=status)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    k, off = new(5, 2, 64), ints(0, 3, 5)
    caches = [(g["k_cache"].clone(), g["v_cache"].clone()) for _ in range(2)]
    p.moe_cache_write(k, -k, *caches[0], g["page_table"], off, g["lengths"])
    p.moe_cache_write(k, -k, *caches[1], g["page_table"], off, g["lengths"], status=status)
    assert all(torch.equal(x, y) for x, y in zip(*caches)) and not torch.equal(caches[0][0], g["k_cache"])
    parents = ints(1, 0, 1)
    for width in (None, 5):
        a = p.moe_cache_fork(g["page_table"], g["lengths"], parents, 16, 9, 2, width)
        b = p.moe_cache_fork(g["page_table"], g["lengths"], parents, 16, 9, 2, width, status=status)
        assert isinstance(a, p.CacheFork) and all(torch.equal(x, y) and x.shape == y.shape for x, y in zip(a, b))
    p.moe_cache_copy(list(caches[0]), a.src, a.dst)
    p.moe_cache_copy(list(caches[1]), a.src, a.dst, status=status)
    assert all(torch.equal(x, y) for x, y in zip(*caches))
    a, b = (p.moe_cache_compact(g["page_table"] + 1, g["lengths"], 16, 9, status=s) for s in (None, status))
    assert isinstance(a, p.CacheCompact) and all(torch.equal(x, y) for x, y in zip(a, b))
    x, s = new(2, 3, 100), new(2, 3, dtype=F32)
    ended = torch.tensor([[0, 1, 0], [0, 0, 0]], dtype=torch.bool, device="cuda")
    out = (torch.empty(2, 4, device="cuda"), torch.empty(2, 4, dtype=I32, device="cuda"), torch.empty(2, 4, dtype=I32, device="cuda"))
    a, b = p.moe_beam_select(x, s, 4, ended, 9), p.moe_beam_select(x, s, 4, ended, 9, out=out)
    assert all(torch.equal(u, v) for u, v in zip(a, b)) and int(status) == 0


def test_small_outputs_share_memory_without_overlap():
    a = p.moe_cache_fork(good()["page_table"], good()["lengths"], ints(0, 1, 1), 16, 9)
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * 4) for t in a)
    assert all(x[1] <= y[0] for x, y in zip(spans, spans[1:])) and all(t.data_ptr() % 16 == 0 for t in a)
    before = [t.clone() for t in a]
    a.lengths.add_(1)
    assert torch.equal(a.page_table, before[0]) and torch.equal(a.src, before[2]) and torch.equal(a.dst, before[3])


def test_empty_calls():
    g = good()
    out, lse = p.moe_attention_decode(g["q"][:0], g["k_cache"], g["v_cache"], g["page_table"][:0], g["lengths"][:0])
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    none = new(0, 16, 2, 64)  # a pool without pages
    out, lse = p.moe_attention_decode(g["q"], none, none, g["page_table"], ints(0, 0))
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())
    status = ints(0)
    out, lse = p.moe_attention_decode(g["q"], none, none, g["page_table"], g["lengths"], status=status)
    assert bool((out == 0).all()) and int(status) == _lib.MOE_STATUS_BAD_INDEX
    out, _ = p.moe_attention_decode(g["q"], g["k_cache"], g["v_cache"], g["page_table"][:, :0], ints(0, 0))
    assert bool((out == 0).all())
    p.moe_cache_write(new(0, 2, 64), new(0, 2, 64), g["k_cache"], g["v_cache"], g["page_table"], ints(0, 0, 0), g["lengths"])
    f = p.moe_cache_fork(g["page_table"], g["lengths"], ints(), 16, 9)
    assert f.page_table.shape == (0, 3)
    f = p.moe_cache_fork(g["page_table"][:0], g["lengths"][:0], ints(-1, -1), 16, 0)
    assert f.page_table.tolist() == [[-1] * 3] * 2 and f.lengths.tolist() == [0, 0]
    assert int(p.moe_cache_compact(g["page_table"][:0], g["lengths"][:0], 16, 0).count) == 0


def test_another_current_stream_and_no_synchronisation():
    """Calls are enqueued on the current stream alone, and return while work in front of them still runs."""
    g, parents, x, scores = good(), ints(0, 1, 1), new(2, 3, 100), torch.zeros(2, 3, device="cuda")

    def calls():
        out, _ = p.moe_attention_decode(**g)
        f = p.moe_cache_fork(g["page_table"], g["lengths"], parents, 16, 9)
        p.moe_cache_copy([g["k_cache"]], f.src, f.dst)
        return out, p.moe_beam_select(x, scores, 2)[0]

    want = calls()
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # 0.2 s of the GPU's clock
        got = calls()
        done.record()
    assert not done.query()
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_keys_and_values_in_one_tensor_and_other_orders(dtype):
    """[pages, 2, page_size, kv_heads, head_dim], and pages behind tokens: the same numbers give the same bits."""
    g = {n: t.to(dtype) if t.dtype == BF16 else t for n, t in good().items()}
    want = p.moe_attention_decode(**(g | {n: g[n].clone() for n in ("k_cache", "v_cache")}))
    both = torch.stack([g["k_cache"], g["v_cache"]], 1)
    got = p.moe_attention_decode(**(g | dict(k_cache=both[:, 0], v_cache=both[:, 1])))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for order in ((1, 0, 2, 3), (2, 1, 0, 3), (0, 2, 1, 3)):
        back = [order.index(i) for i in range(4)]
        k, v = (g[n].permute(order).contiguous().permute(back) for n in ("k_cache", "v_cache"))
        got = p.moe_attention_decode(**(g | dict(k_cache=k, v_cache=v)))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(k[0, 1, 0], g["k_cache"][0, 1, 0])
    flat = both.clone()
    p.moe_cache_write(g["k_new"], g["v_new"], flat[:, 0], flat[:, 1], g["page_table"], ints(0, 1, 2), g["lengths"])
    assert torch.equal(flat[2, 0, 7], g["k_new"][0]) and torch.equal(flat[2, 1, 7], g["v_new"][0])
    assert torch.equal(flat[3, 0, 6], g["k_new"][1]) and torch.equal(flat[3, 1, 6], g["v_new"][1])


def test_as_many_rows_as_there_may_be():
    R = _lib.MOE_CACHE_MAX_ROWS
    k, v = new(R, 2, 1, 16, dtype=F32), new(R + 1, 2, 1, 16, dtype=F32)[1:]
    table = torch.arange(R, dtype=I32, device="cuda")[:, None]
    lengths = (torch.arange(R, device="cuda") % 3).to(I32)
    q = new(R, 2, 16, dtype=F32)
    out, lse = p.moe_attention_decode(q, k, v, table, lengths)
    n = lengths.long()
    x = torch.einsum("rhd,rtd->rht", q.double(), k[:, :, 0].double()) / 4
    x = torch.where(torch.arange(2, device="cuda") < n[:, None, None], x, -torch.inf)
    want = torch.einsum("rht,rtd->rhd", torch.softmax(x, 2).nan_to_num(0), v[:, :, 0].double())
    assert bool(((out.double() - want).abs() <= 1e-5).all())  # two terms of order one: some 2^-20
    assert torch.equal(torch.isinf(lse), (n == 0)[:, None].expand(R, 2))


def test_inference_mode_and_concurrent_streams():
    with torch.inference_mode():
        g = good()
        out, lse = p.moe_attention_decode(**g)
        f = p.moe_cache_fork(g["page_table"], g["lengths"], ints(0, 1, 1), 16, 9)
        assert out.is_inference() and f.lengths.is_inference()
        f.lengths.add_(1)
    g = [good() | dict(q=new(2, 4, 64) * (1 + i), k_new=None, v_new=None) for i in range(4)]
    x, s = [new(2, 3, 4000 + 8 * i) for i in range(4)], torch.zeros(2, 3, device="cuda")
    want = [(*p.moe_attention_decode(**a), *p.moe_beam_select(b, s, 5)) for a, b in zip(g, x)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(20):  # four streams at the same time, each call with a workspace of its own
        got = []
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got.append((*p.moe_attention_decode(**g[i]), *p.moe_beam_select(x[i], s, 5)))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for u, w in zip(got, want) for a, b in zip(u, w))
