"""ctypes loader for libmoe_route.so and the raw C-ABI signatures.

Argument marshalling only: every computation runs in the CUDA library. The
loader fails loudly when the library has not been built; there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import re

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe_route.so")
CALLS_PATH = os.path.join(PKG, "_block_calls.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "moe_route.h")
BLOCK_HEADER = os.path.join(os.path.dirname(PKG), "include", "moe_block.h")
DECODE_HEADER = os.path.join(os.path.dirname(PKG), "include", "moe_decode.h")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA = 0, 1, 2, 3
MOE_F32, MOE_BF16 = 0, 1
MOE_STATUS_BAD_EXPERT, MOE_STATUS_BAD_INDEX, MOE_STATUS_BAD_BINS, MOE_STATUS_ROWS_MISMATCH = 1, 2, 4, 8
MOE_STATUS_TIMEOUT = 16
MOE_STATUS_NO_PAGES = 32
MOE_MAX_EXPERTS, MOE_MAX_TOP_K = 4096, 64
MOE_GATING_SOFTMAX, MOE_GATING_SIGMOID = 0, 1
MOE_GATING_MAX_EXPERTS = 1024
MOE_ATTENTION_MAX_DIM = 256
MOE_CACHE_MAX_ROWS, MOE_CACHE_MAX_PAGES, MOE_CACHE_MAX_CACHES = 4096, 1 << 22, 256
MOE_BEAM_MAX_BEAMS, MOE_BEAM_MAX_OUT, MOE_BEAM_MAX_UNITS = 64, 128, 1 << 15

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t

# name -> (restype, argtypes), in the order of include/moe_route.h
SIGNATURES = {
    "moe_error_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_version": (ctypes.c_int, []),
    "moe_route_build_workspace_size": (_SZ, [_I64, _I32]),
    "moe_route_build_gather_workspace_size": (_SZ, [_I64, _I32]),
    "moe_test_barrier_slack": (None, [ctypes.c_uint32]),
    "moe_route_build": (ctypes.c_int, [_P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P, _P]),
    "moe_route_build_noalloc": (ctypes.c_int, [_P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _P]),
    "moe_check_routing": (ctypes.c_int, [_P, _P, _P, _P, _P, _I64, _I32, _P, _P]),
    "moe_binned_gather": (ctypes.c_int, [_P, _I32, _P, _P, _P, _I64, _I64, _I32, _I32, _I32, _P, _P, _P]),
    "moe_padded_gather": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _I64, _I64, _I32, _I32, _P, _I64, _P, _P]),
    "moe_binned_gather_weighted": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _I64, _I64, _I32, _I32, _I32, _P, _P,
                                                  _P]),
    "moe_padded_gather_weighted": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _P, _I64, _I64, _I32, _I32, _P, _I64,
                                                  _P, _P]),
    "moe_route_build_binned_gather": (ctypes.c_int, [_P, _P, _I32, _I64, _I64, _I32, _I32, _I32, _I32, _P, _P, _P,
                                                     _P, _P, _P, _P, _SZ, _P, _P]),
    "moe_route_build_padded_gather": (ctypes.c_int, [_P, _P, _I32, _I64, _I64, _I32, _I32, _I32, _P, _P, _P, _P,
                                                     _P, _P, _I64, _P, _SZ, _P, _P]),
    "moe_scatter_workspace_size": (_SZ, [_I64]),
    "moe_binned_scatter": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _P, _I64, _I64, _I32, _I32, _I32, _P, _P, _SZ,
                                          _P, _P]),
    "moe_padded_scatter": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _P, _P, _I64, _I64, _I32, _I32, _I64, _P, _P,
                                          _SZ, _P, _P]),
    "moe_binned_wgrad": (ctypes.c_int, [_P, _P, _I32, _P, _P, _P, _I64, _I64, _I32, _I32, _I32, _P, _P, _P]),
    "moe_padded_wgrad": (ctypes.c_int, [_P, _P, _I32, _P, _P, _P, _P, _P, _I64, _I64, _I32, _I32, _I64, _P, _P,
                                        _P]),
    "moe_topk_gating": (ctypes.c_int, [_P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P]),
    "moe_routing_map_to_indices_fwd": (ctypes.c_int, [_P, _P, _I64, _I32, _I32, _P, _P, _P]),
    "moe_routing_map_to_indices_bwd": (ctypes.c_int, [_P, _P, _I64, _I32, _I32, _P, _P, _P]),
}

# The entry points of include/moe_block.h, in its order.
BLOCK_SIGNATURES = {
    "moe_layer_workspace_size": (_SZ, [_I64, _I64, _I64, _I32, _I32]),
    "moe_layer": (ctypes.c_int, [_P, _I32, _I64, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _I32, _I32, _P, _P, _P, _P,
                                 _SZ, _P, _P]),
    "moe_experts": (ctypes.c_int, [_P, _I32, _I64, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _P, _P, _SZ, _P, _P]),
    "moe_test_block_waits": (None, [ctypes.c_uint32]),
    "moe_layer_norm_fwd": (ctypes.c_int, [_P, _I32, _I64, _P, _P, _I32, _I64, _I64, ctypes.c_float, _P, _P, _P, _P]),
    "moe_layer_norm_bwd_workspace_size": (_SZ, [_I64, _I64]),
    "moe_layer_norm_bwd": (ctypes.c_int, [_P, _I64, _P, _I32, _I64, _P, _I32, _P, _P, _I64, _I64, _P, _P, _P, _P, _SZ,
                                          _P]),
    "moe_grad_table_pieces": (_I64, [_P, _I64]),
    "moe_grad_table_fill": (ctypes.c_int, [_P, _I64, _P, _I64]),
    "moe_grad_norm_workspace_size": (_SZ, []),
    "moe_grad_norm": (ctypes.c_int, [_P, _I64, _P, _P, _SZ, _P]),
    "moe_clip_grads": (ctypes.c_int, [_P, _I64, ctypes.c_float, _P, _P, _SZ, _P]),
}

# The entry points of include/moe_decode.h, in its order.
DECODE_SIGNATURES = {
    "moe_attention_decode_workspace_size": (_SZ, [_I64, _I32, _I32, _I32]),
    "moe_attention_decode": (ctypes.c_int, [_P, _P, _I32, _P, _I64, _I64, _P, _I64, _P, _P, ctypes.c_float, _I64, _P, _P,
                                            _P, _SZ, _P, _P]),
    "moe_cache_write": (ctypes.c_int, [_P, _P, _P, _I64, _P, _P, _I64, _I64, _P, _I64, _P, _P]),
    "moe_cache_fork": (ctypes.c_int, [_P, _I64, _I64, _P, _I64, _P, _I64, _I32, _I64, _I64, _P, _I64, _P, _P, _P, _P, _P]),
    "moe_cache_compact": (ctypes.c_int, [_P, _I64, _I64, _P, _I64, _I32, _I64, _P, _P, _P, _P, _P, _P]),
    "moe_cache_copy": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _I64, _P, _P, _P]),
    "moe_beam_select_workspace_size": (_SZ, [_I64, _I32, _I64]),
    "moe_beam_select": (ctypes.c_int, [_P, _I32, _I64, _P, _P, _I64, _I32, _I64, _I32, _I32, _P, _P, _P, _P, _SZ, _P]),
}


class KvCache(ctypes.Structure):
    """moe_kv_cache."""

    _fields_ = [("k", _P), ("v", _P), ("num_pages", _I64), ("page_stride", _I64), ("token_stride", _I64),
                ("head_stride", _I64), ("dtype", _I32), ("page_size", _I32), ("num_kv_heads", _I32), ("head_dim", _I32)]


class Heads(ctypes.Structure):
    """moe_heads."""

    _fields_ = [("data", _P), ("row_stride", _I64), ("head_stride", _I64)]


class CachePages(ctypes.Structure):
    """moe_cache_pages."""

    _fields_ = [("data", _P), ("page_stride", _I64), ("page_bytes", _I64)]


class GradTensor(ctypes.Structure):
    """moe_grad_tensor; moe_grad_piece has the same layout."""

    _fields_ = [("grad", _P), ("out", _P), ("numel", _I64), ("dtype", _I32), ("reserved", _I32)]


class MoeError(RuntimeError):
    """A C-ABI call returned a nonzero MOE_ERR_* code."""

    def __init__(self, fn: str, code: int, text: str):
        super().__init__("%s failed: %s (code %d)" % (fn, text, code))
        self.code = code


_lib = None


def header_functions(header: str = HEADER) -> list[str]:
    """Names of every function declared in include/moe_route.h (or another header)."""
    src = open(header).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return re.findall(r"\b(moe_\w+)\s*\(", src)


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the CUDA library once. Raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError("libmoe_route.so is not built (%s); run "
                           "`python -m padded_permute_combine_gb300.build` first" % p)
    lib = ctypes.CDLL(p)
    for name, (res, args) in (SIGNATURES | BLOCK_SIGNATURES | DECODE_SIGNATURES).items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


calls = None  # the module _block_calls, once loaded


def load_calls():
    """Load the native marshalling of the block operators once. Raises if it has not been built."""
    global calls
    if calls is None:
        if not os.path.exists(CALLS_PATH):
            raise RuntimeError("_block_calls.so is not built (%s); run "
                               "`python -m padded_permute_combine_gb300.build` first" % CALLS_PATH)
        import torch  # noqa: F401  (its libraries, which the module needs)

        load()
        spec = importlib.util.spec_from_file_location("_block_calls", CALLS_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        calls = module
    return calls


def call(name: str, *args) -> None:
    """Call a status-returning entry point and raise MoeError on failure."""
    lib = load()
    rc = getattr(lib, name)(*args)
    if rc != MOE_OK:
        raise MoeError(name, rc, lib.moe_error_string(rc).decode())
