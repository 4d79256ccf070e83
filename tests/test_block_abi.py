"""include/moe_block.h on the CPU: every declared function is exported and
bound, bad arguments are refused on the host before any CUDA call, and the
gradient table (built on the host) covers each tensor exactly once."""
import ctypes
import os
import shutil
import subprocess

import pytest

from padded_permute_combine_gb300 import _lib
from padded_permute_combine_gb300 import build as libbuild

FAKE = 1 << 20  # an aligned non-null address, never dereferenced: host checks fail first
OK, INVALID, UNSUPPORTED = _lib.MOE_OK, _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return _lib.load()


def test_header_exports_and_binding_agree(lib):
    declared = _lib.header_functions(_lib.BLOCK_HEADER)
    assert len(declared) == len(set(declared)) and set(declared) == set(_lib.BLOCK_SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    assert not [f for f in declared if f not in exported]


def test_header_is_plain_c(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    src = tmp_path / "host.c"
    src.write_text('#include "moe_block.h"\nint main(void) { return sizeof(moe_grad_tensor) == sizeof(moe_grad_piece) ? 0 : 1; }\n')
    include = os.path.dirname(_lib.BLOCK_HEADER)
    subprocess.run([gcc, "-std=c11", "-Wall", "-Werror", "-c", "-I", include, str(src), "-o", str(tmp_path / "host.o")],
                   check=True)


def layer(lib, x=FAKE, dtype=1, stride=64, router=FAKE, gu=FAKE, dn=FAKE, T=4, H=64, F=32, E=8, K=2, mode=0, te=FAKE,
          w=FAKE, y=FAKE, ws=FAKE, size=1 << 30, status=None):
    return lib.moe_layer(x, dtype, stride, router, gu, dn, T, H, F, E, K, mode, 1, te, w, y, ws, size, status, None)


def test_layer_refusals(lib):
    assert lib.moe_layer_workspace_size(4, 64, 32, 8, 2) > 0
    for bad in ((-1, 64, 32, 8, 2), (4, 0, 32, 8, 2), (4, 64, 0, 8, 2), (4, 64, 32, 0, 1), (4, 64, 32, 8, 9),
                (4, 64, 32, 8, 0), (257, 64, 32, 8, 1), (256, 64, 32, 64, 9), (4, 64, 32, 1025, 2)):
        assert lib.moe_layer_workspace_size(*bad) == 0
    assert layer(lib, T=0) == OK
    for kw in (dict(T=-1), dict(H=0), dict(F=0), dict(E=0), dict(K=0), dict(K=9), dict(stride=63), dict(mode=2),
               dict(x=None), dict(router=None), dict(gu=None), dict(dn=None), dict(te=None), dict(w=None), dict(y=None),
               dict(ws=None), dict(size=100)):
        assert layer(lib, **kw) == INVALID, kw
    for kw in (dict(dtype=2), dict(T=257), dict(T=256, K=9, E=64), dict(E=1025), dict(x=FAKE + 1), dict(gu=FAKE + 1),
               dict(te=FAKE + 2), dict(w=FAKE + 2), dict(ws=FAKE + 8), dict(y=FAKE + 1), dict(status=FAKE + 2)):
        assert layer(lib, **kw) == UNSUPPORTED, kw
    ex = lambda **k: lib.moe_experts(*[dict(x=FAKE, dtype=0, stride=64, te=FAKE, w=FAKE, gu=FAKE, dn=FAKE, T=4, H=64,  # noqa: E731
                                            F=32, E=8, K=2, y=FAKE, ws=FAKE, size=1 << 30, st=None, s=None, **{})[n]
                                       if n not in k else k[n] for n in ("x", "dtype", "stride", "te", "w", "gu", "dn",
                                                                         "T", "H", "F", "E", "K", "y", "ws", "size",
                                                                         "st", "s")])
    assert ex(T=0) == OK
    assert ex(te=None) == INVALID and ex(w=None) == INVALID and ex(stride=8) == INVALID
    assert ex(dtype=7) == UNSUPPORTED and ex(x=FAKE + 2) == UNSUPPORTED


def test_layer_norm_refusals(lib):
    fwd = lambda x=FAKE, dt=0, st=64, w=None, b=None, wd=0, M=4, H=64, eps=1e-5, y=FAKE, m=None, r=None: (  # noqa: E731
        lib.moe_layer_norm_fwd(x, dt, st, w, b, wd, M, H, eps, y, m, r, None))
    assert fwd(M=0) == OK
    for kw in (dict(M=-1), dict(H=0), dict(st=63), dict(eps=-1.0), dict(eps=float("nan")), dict(x=None), dict(y=None)):
        assert fwd(**kw) == INVALID, kw
    for kw in (dict(dt=3), dict(wd=3), dict(x=FAKE + 2), dict(y=FAKE + 2), dict(w=FAKE + 2), dict(m=FAKE + 2)):
        assert fwd(**kw) == UNSUPPORTED, kw
    assert lib.moe_layer_norm_bwd_workspace_size(-1, 4) == 0 and lib.moe_layer_norm_bwd_workspace_size(4, 0) == 0
    size = lib.moe_layer_norm_bwd_workspace_size(4, 64)
    assert size >= 2 * 64 * 4
    bwd = lambda dy=FAKE, dst=64, x=FAKE, dt=0, st=64, w=None, wd=0, m=FAKE, r=FAKE, M=4, H=64, dx=FAKE, dw=FAKE, db=FAKE, ws=FAKE, n=size: (  # noqa: E731
        lib.moe_layer_norm_bwd(dy, dst, x, dt, st, w, wd, m, r, M, H, dx, dw, db, ws, n, None))
    assert bwd(M=0, dw=None, db=None, ws=None, n=0) == OK
    for kw in (dict(dst=1), dict(st=1), dict(dy=None), dict(m=None), dict(dx=None), dict(ws=None), dict(n=size - 1), dict(M=-1)):
        assert bwd(**kw) == INVALID, kw
    for kw in (dict(dt=9), dict(ws=FAKE + 4), dict(dw=FAKE + 1), dict(dy=FAKE + 1)):
        assert bwd(**kw) == UNSUPPORTED, kw


def table(lib, tensors):
    entries = (_lib.GradTensor * max(1, len(tensors)))(*[_lib.GradTensor(*t, 0) for t in tensors])
    n = lib.moe_grad_table_pieces(entries, len(tensors))
    assert n >= 0
    pieces = (_lib.GradTensor * max(1, n))()
    assert lib.moe_grad_table_fill(entries, len(tensors), pieces, n) == OK
    assert lib.moe_grad_table_fill(entries, len(tensors), pieces, n + 1) == INVALID
    return list(pieces)[:n]


@pytest.mark.parametrize("dtype,eb", [(0, 4), (1, 2)])
@pytest.mark.parametrize("off", [0, 1, 7, 15])
@pytest.mark.parametrize("numel", [0, 1, 16, 16383, 16384, 16385, 32768, 100003, (1 << 33) + 5])
def test_grad_table_covers_every_element_once(lib, numel, off, dtype, eb):
    if numel > 1 << 30 and off != 7:
        pytest.skip("one large offset is enough")
    grad, out = FAKE + off * eb, (FAKE << 22) + eb
    at = 0
    for p in table(lib, [(grad, out, numel, dtype)]):
        assert p.grad == grad + at * eb and p.out == out + at * eb and p.dtype == dtype
        assert 0 < p.numel <= 65536 // eb
        at += p.numel
        assert at == numel or (grad + at * eb) % 32 == 0  # later pieces start on 32 bytes
    assert at == numel


def test_grad_table_and_norm_refusals(lib):
    bad = [(None, None, 5, 0), (FAKE, None, -1, 0), (FAKE, None, 5, 2), (FAKE + 1, None, 5, 0), (FAKE, FAKE + 2, 5, 0)]
    for t in bad:
        e = (_lib.GradTensor * 1)(_lib.GradTensor(*t, 0))
        assert lib.moe_grad_table_pieces(e, 1) == -1
    assert lib.moe_grad_table_pieces(None, 1) == -1 and lib.moe_grad_table_pieces(None, 0) == 0
    assert table(lib, [(None, None, 0, 0)]) == []
    size = lib.moe_grad_norm_workspace_size()
    nan = ctypes.c_float(float("nan"))
    assert lib.moe_grad_norm(None, 3, FAKE, FAKE, size, None) == INVALID
    assert lib.moe_grad_norm(FAKE, -1, FAKE, FAKE, size, None) == INVALID
    assert lib.moe_grad_norm(FAKE, 3, None, FAKE, size, None) == INVALID
    assert lib.moe_grad_norm(FAKE, 3, FAKE, FAKE, size - 1, None) == INVALID
    assert lib.moe_grad_norm(FAKE, 3, FAKE, FAKE + 4, size, None) == UNSUPPORTED
    assert lib.moe_clip_grads(FAKE, 3, nan, FAKE, FAKE, size, None) == INVALID
    assert lib.moe_clip_grads(FAKE, 3, -1.0, FAKE, FAKE, size, None) == INVALID
