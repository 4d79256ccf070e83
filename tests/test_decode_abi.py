"""include/moe_decode.h on the CPU: every declared function is exported and
bound, bad arguments are refused on the host before any CUDA call, and the
binding words its own refusals."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import padded_permute_combine_gb300 as p
from padded_permute_combine_gb300 import _lib
from padded_permute_combine_gb300 import build as libbuild

FAKE = 1 << 20  # an aligned non-null address, never dereferenced: host checks fail first
OK, INVALID, UNSUPPORTED = _lib.MOE_OK, _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return _lib.load()


def test_header_exports_and_binding_agree(lib):
    declared = _lib.header_functions(_lib.DECODE_HEADER)
    assert len(declared) == len(set(declared)) and set(declared) == set(_lib.DECODE_SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    assert not [f for f in declared if f not in exported]
    assert all(hasattr(p, f) for f in declared if not f.endswith("_workspace_size"))


def test_header_is_plain_c_and_the_structs_agree(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    src = tmp_path / "host.c"
    sizes = [(n, ctypes.sizeof(t)) for n, t in (("moe_kv_cache", _lib.KvCache), ("moe_heads", _lib.Heads),
                                                ("moe_cache_pages", _lib.CachePages))]
    limits = [n for n in vars(_lib) if n.startswith(("MOE_ATTENTION_", "MOE_CACHE_", "MOE_BEAM_", "MOE_STATUS_NO"))]
    src.write_text('#include "moe_decode.h"\n' + "".join("_Static_assert(sizeof(%s) == %d, \"size\");\n" % s for s in sizes)
                   + "".join("_Static_assert(%s == %d, \"value\");\n" % (n, getattr(_lib, n)) for n in limits)
                   + "int main(void) { return 0; }\n")
    include = os.path.dirname(_lib.DECODE_HEADER)
    subprocess.run([gcc, "-std=c11", "-Wall", "-Werror", "-c", "-I", include, str(src), "-o", str(tmp_path / "host.o")],
                   check=True)


def cache(k=FAKE, v=FAKE, n=8, ps=16 * 2 * 64, ts=2 * 64, hs=64, dt=1, page=16, kv=2, dim=64):
    return ctypes.byref(_lib.KvCache(k, v, n, ps, ts, hs, dt, page, kv, dim))


def heads(data=FAKE, rs=8 * 64, hs=64):
    return ctypes.byref(_lib.Heads(data, rs, hs))


def test_attention_refusals(lib):
    size = lib.moe_attention_decode_workspace_size(3, 8, 2, 64)
    assert size > 0
    for bad in ((-1, 8, 2, 64), (3, 0, 2, 64), (3, 8, 0, 64), (3, 7, 2, 64), (3, 8, 2, 0), (3, 8, 2, 257), (4097, 8, 2, 64)):
        assert lib.moe_attention_decode_workspace_size(*bad) == 0

    def call(c=None, q=None, H=8, table=FAKE, ts=4, width=4, lens=FAKE, B=3, kn=None, vn=None, scale=0.1, window=0, out=FAKE,
             lse=FAKE, ws=FAKE, n=size, st=None):
        return lib.moe_attention_decode(c or cache(), q or heads(), H, table, ts, width, lens, B, kn, vn, scale, window, out, lse,
                                        ws, n, st, None)

    assert call(B=0) == OK
    for kw in (dict(B=-1), dict(H=0), dict(H=7), dict(ts=3), dict(width=-1), dict(window=-1), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(table=None), dict(lens=None), dict(out=None), dict(ws=None), dict(n=size - 1),
               dict(kn=heads()), dict(vn=heads()), dict(kn=heads(None), vn=heads()), dict(q=heads(None)), dict(q=heads(rs=-1)),
               dict(c=cache(k=None)), dict(c=cache(v=None)), dict(c=cache(n=-1)), dict(c=cache(ps=-1)), dict(c=cache(ts=-1)),
               dict(c=cache(hs=-1)), dict(c=cache(page=0)), dict(c=cache(kv=0)), dict(c=cache(dim=0))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(c=cache(dt=2)), dict(c=cache(dim=257)), dict(B=4097), dict(width=1 << 28, ts=1 << 28), dict(c=cache(k=FAKE + 1)),
               dict(c=cache(n=1 << 31)), dict(q=heads(FAKE + 1)), dict(out=FAKE + 1), dict(lse=FAKE + 2), dict(ws=FAKE + 8),
               dict(table=FAKE + 2), dict(lens=FAKE + 1), dict(st=FAKE + 2), dict(kn=heads(FAKE + 1), vn=heads()),
               dict(B=2000, width=1 << 20, ts=1 << 20, n=1 << 60)):
        assert call(**kw) == UNSUPPORTED, kw
    assert lib.moe_attention_decode(None, heads(), 8, FAKE, 4, 4, FAKE, 3, None, None, 0.1, 0, FAKE, FAKE, FAKE, size, None, None) == INVALID


def test_write_refusals(lib):
    def call(c=None, k=None, v=None, T=5, off=FAKE, table=FAKE, ts=4, width=4, lens=FAKE, B=3, st=None):
        return lib.moe_cache_write(c or cache(), k or heads(), v or heads(), T, off, table, ts, width, lens, B, st, None)

    assert call(T=0) == OK and call(B=0) == OK
    for kw in (dict(T=-1), dict(B=-1), dict(ts=3), dict(width=-1), dict(off=None), dict(table=None), dict(lens=None), dict(k=heads(None)),
               dict(v=heads(None)), dict(k=heads(rs=-1)), dict(c=cache(page=0)), dict(c=cache(k=None))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(c=cache(dt=5)), dict(T=1 << 31), dict(off=FAKE + 2), dict(k=heads(FAKE + 1)), dict(c=cache(dim=1 << 21)), dict(st=FAKE + 1)):
        assert call(**kw) == UNSUPPORTED, kw


def test_page_table_refusals(lib):
    def fork(table=FAKE, ts=4, width=4, lens=FAKE, B=3, par=FAKE, R=5, page=16, pool=100, grow=1, new=FAKE, nw=4, nl=FAKE, src=FAKE,
             dst=FAKE, st=None):
        return lib.moe_cache_fork(table, ts, width, lens, B, par, R, page, pool, grow, new, nw, nl, src, dst, st, None)

    assert fork(R=0) == OK
    for kw in (dict(R=-1), dict(B=-1), dict(ts=3), dict(page=0), dict(pool=-1), dict(grow=-1), dict(nw=3), dict(table=None), dict(lens=None),
               dict(par=None), dict(new=None), dict(nl=None), dict(src=None), dict(dst=None)):
        assert fork(**kw) == INVALID, kw
    for kw in (dict(R=4097), dict(B=4097), dict(pool=(1 << 22) + 1), dict(width=1 << 28, ts=1 << 28, nw=1 << 28), dict(par=FAKE + 2),
               dict(st=FAKE + 1), dict(grow=1 << 31), dict(new=FAKE + 1)):
        assert fork(**kw) == UNSUPPORTED, kw

    def compact(table=FAKE, ts=4, width=4, lens=FAKE, B=3, page=16, pool=100, new=FAKE, src=FAKE, dst=FAKE, count=FAKE, st=None):
        return lib.moe_cache_compact(table, ts, width, lens, B, page, pool, new, src, dst, count, st, None)

    for kw in (dict(B=-1), dict(ts=3), dict(page=0), dict(pool=-1), dict(table=None), dict(lens=None), dict(new=None), dict(src=None),
               dict(dst=None), dict(count=None)):
        assert compact(**kw) == INVALID, kw
    for kw in (dict(B=4097), dict(pool=(1 << 22) + 1), dict(src=FAKE + 1), dict(count=FAKE + 2)):
        assert compact(**kw) == UNSUPPORTED, kw


def test_copy_refusals(lib):
    def call(entries=((FAKE, 64, 64),), pool=10, src=FAKE, dst=FAKE, n=3, count=None, st=None, none=False):
        some = (_lib.CachePages * max(1, len(entries)))(*[_lib.CachePages(*e) for e in entries])
        return lib.moe_cache_copy(None if none else some, len(entries), pool, src, dst, n, count, st, None)

    assert call(n=0) == OK and call(pool=0) == OK and call(entries=((None, 0, 0),)) == OK and call(entries=()) == OK
    for kw in (dict(n=-1), dict(pool=-1), dict(src=None), dict(dst=None), dict(none=True), dict(entries=((None, 64, 64),)),
               dict(entries=((FAKE, 63, 64),)), dict(entries=((FAKE, 64, -1),))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(entries=((FAKE, 64, 64),) * 257), dict(pool=1 << 31), dict(src=FAKE + 1), dict(count=FAKE + 2), dict(st=FAKE + 2),
               dict(entries=((FAKE, 1 << 31, 1 << 31),))):
        assert call(**kw) == UNSUPPORTED, kw


def test_select_refusals(lib):
    size = lib.moe_beam_select_workspace_size(3, 4, 1000)
    assert size > 0
    for bad in ((-1, 4, 1000), (3, 0, 1000), (3, 4, 0), (3, 65, 1000), (3, 64, 512 * 512 + 1), (1 << 30, 4, 10)):
        assert lib.moe_beam_select_workspace_size(*bad) == 0

    def call(x=FAKE, dt=1, rs=1000, s=FAKE, ended=None, B=3, W=4, V=1000, n=8, end=-1, a=FAKE, b=FAKE, c=FAKE, ws=FAKE, size=size):
        return lib.moe_beam_select(x, dt, rs, s, ended, B, W, V, n, end, a, b, c, ws, size, None)

    assert call(B=0) == OK
    for kw in (dict(B=-1), dict(W=0), dict(V=0), dict(n=0), dict(rs=999), dict(ended=FAKE), dict(ended=FAKE, end=1000), dict(x=None),
               dict(s=None), dict(a=None), dict(b=None), dict(c=None), dict(ws=None), dict(size=size - 1)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(dt=2), dict(n=129), dict(W=65), dict(x=FAKE + 1), dict(s=FAKE + 2), dict(a=FAKE + 1), dict(ws=FAKE + 8)):
        assert call(**kw) == UNSUPPORTED, kw


def test_the_binding_refuses_tensors_that_are_not_on_a_gpu():
    x = torch.zeros(2, 4, 8)
    c, i = torch.zeros(3, 4, 2, 8), torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 3, dtype=torch.int32)
    for call in (lambda: p.moe_attention_decode(x, c, c, t, i), lambda: p.moe_cache_write(x, x, c, c, t, i, i),
                 lambda: p.moe_cache_fork(t, i, i, 4, 3), lambda: p.moe_cache_compact(t, i, 4, 3), lambda: p.moe_cache_copy([c], i, i),
                 lambda: p.moe_beam_select(x, x[:, :, 0], 2)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: p.moe_attention_decode(None, c, c, t, i), lambda: p.moe_cache_fork(3, i, i, 4, 3),
                 lambda: p.moe_beam_select([1], x, 2), lambda: p.moe_cache_copy([c], None, i)):
        with pytest.raises(TypeError):
            call()


def test_native_marshalling_leaves_the_rest_to_the_caller():
    libbuild.build()
    calls = _lib.load_calls()
    c, q, i, t = torch.zeros(3, 4, 2, 8), torch.zeros(2, 4, 8), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    assert calls.attention_decode(q, c, c, t, i, None, None, None, 0) is None  # not on a GPU
    assert calls.attention_decode(q, c, c, t, i, None, None, "a", 0) is None and calls.attention_decode(q) is None
    assert calls.attention_decode(q, None, c, t, i, None, None, None, 0) is None
    assert calls.cache_write(q, q, c, c, t, i, i) is None and calls.cache_write(1, 2, 3, 4, 5, 6, 7) is None
    assert calls.cache_fork(t, i, i, 4, 3, 1, None) is None and calls.cache_fork(t, i, i, 4, 3, 1, 2 ** 70) is None
    assert calls.cache_compact(t, i, 4, 3) is None and calls.cache_compact(t, i, 4.0, 3) is None
    assert calls.cache_copy([c], i, i, None) is None and calls.cache_copy((c,), i, i, None) is None and calls.cache_copy([], i, i, None) is None
    assert calls.beam_select(q, q[:, :, 0], 2, None, -1) is None and calls.beam_select(q, q[:, :, 0], 2 ** 70, None, -1) is None
