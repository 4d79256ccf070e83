"""Python binding of include/moe_block.h: the operators around the routing in
an MoE block (same names, same semantics).

As in ops.py this is argument marshalling only. Rows (x, dy) may come with a
row stride, such as a slice of a wider tensor; everything else is contiguous.
The plain call (right arguments, outputs to be allocated) is marshalled by
csrc/block_calls.cpp; it answers None to any other, which is then taken step by
step here, with a message for what is wrong.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Sequence

import torch

from . import _lib
from .ops import _DTYPES, _act_dtype, _need

_MODES = {"softmax": _lib.MOE_GATING_SOFTMAX, "sigmoid": _lib.MOE_GATING_SIGMOID}


def _stream(device: torch.device) -> int:
    # torch.cuda.current_stream(device).cuda_stream without building the Stream object (2 us).
    return torch._C._cuda_getCurrentRawStream(device.index)


_SAME = contextlib.nullcontext()


def _on(device: torch.device):
    """Makes the tensors' device current for a C call, whose launches, SM
    counts and limits are those of the current device."""
    return _SAME if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _rows(t: torch.Tensor, name: str, dtype: torch.dtype | None = None, shape=None, device=None) -> int:
    """Checks a [rows, H] tensor whose rows are contiguous and returns its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError("%s must be %s, got %s" % (name, "2-D" if shape is None else list(shape), list(t.shape)))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.is_contiguous():
        return t.shape[1]
    stride = t.stride(0)
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s must have contiguous rows" % name)
    if t.shape[0] > 1 and stride < t.shape[1]:
        raise ValueError("%s must have rows that do not overlap" % name)
    return stride


def _take(t: torch.Tensor, shape: tuple, dtype: torch.dtype, name: str, device) -> int:
    """Checks a contiguous tensor and returns its address (one test of all at
    once: a few calls here are as long as a small kernel)."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        return t.data_ptr()
    _need(t, dtype, name, device)
    raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))


def _workspace(t: torch.Tensor | None, size: int, device) -> torch.Tensor:
    if t is None:
        return torch.empty(size, dtype=torch.uint8, device=device)
    return _need(t, torch.uint8, "workspace", device)


def _done(name: str, rc: int) -> None:
    if rc != _lib.MOE_OK:
        raise _lib.MoeError(name, rc, _lib.load().moe_error_string(rc).decode())


def _status(t: torch.Tensor | None, device) -> int | None:
    return None if t is None else _need(t, torch.int32, "status", device).data_ptr()


def _expert_weights(x, H, w_gate_up, w_down):
    """E, F and the addresses of the experts' matrices, which go with x."""
    if not isinstance(w_down, torch.Tensor) or w_down.dim() != 3 or w_down.shape[1] != H:
        _need(w_down, x.dtype, "w_down", x.device)
        raise ValueError("w_down must be [E, %d, F], got %s" % (H, list(w_down.shape)))
    E, _, F = w_down.shape
    down = _take(w_down, (E, H, F), x.dtype, "w_down", x.device)
    return E, F, _take(w_gate_up, (E, 2 * F, H), x.dtype, "w_gate_up", x.device), down


def layer_workspace(num_tokens: int, hidden: int, ffn: int, num_experts: int, top_k: int, device) -> torch.Tensor:
    """Workspace of moe_layer and moe_experts (one per stream that may run them at the same time)."""
    size = _lib.load().moe_layer_workspace_size(num_tokens, hidden, ffn, num_experts, top_k)
    return torch.empty(size, dtype=torch.uint8, device=device)


def moe_layer(x: torch.Tensor, router: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor, top_k: int,
              mode: str = "softmax", normalize: bool = True, out: torch.Tensor | None = None,
              routing: tuple[torch.Tensor, torch.Tensor] | None = None, workspace: torch.Tensor | None = None,
              status: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """A whole MoE layer for a few tokens (at most 256, and 2048 choices):
    x [T, H], router [E, H], w_gate_up [E, 2F, H], w_down [E, H, F] ->
    (y [T, H], top_expert [T, top_k] int32, weights [T, top_k] fp32). mode and
    normalize as for moe_topk_gating; ``routing``: the two tensors that take
    top_expert and weights."""
    if out is None and routing is None and workspace is None and status is None and mode in _MODES:
        done = (_lib.calls or _lib.load_calls()).layer(x, router, w_gate_up, w_down, top_k, _MODES[mode], bool(normalize))
        if done is not None:
            return done
    stride = _rows(x, "x")
    dt = _act_dtype(x, "x")
    dev = x.device
    T, H = x.shape
    E, F, gate_up, down = _expert_weights(x, H, w_gate_up, w_down)
    router_at = _take(router, (E, H), x.dtype, "router", dev)
    if mode not in _MODES:
        raise ValueError("mode must be softmax or sigmoid, got %r" % (mode,))
    if routing is None:
        te = torch.empty((T, top_k), dtype=torch.int32, device=dev)
        w = torch.empty((T, top_k), dtype=torch.float32, device=dev)
        te_at, w_at = te.data_ptr(), w.data_ptr()
    else:
        te, w = routing
        te_at = _take(te, (T, top_k), torch.int32, "top_expert", dev)
        w_at = _take(w, (T, top_k), torch.float32, "weights", dev)
    if out is None:
        out = torch.empty((T, H), dtype=x.dtype, device=dev)
    out_at = _take(out, (T, H), x.dtype, "out", dev)
    lib = _lib.load()
    ws = _workspace(workspace, lib.moe_layer_workspace_size(T, H, F, E, top_k), dev)
    with _on(dev):
        rc = lib.moe_layer(
            x.data_ptr(), dt, stride, router_at, gate_up, down, T, H, F, E, top_k, _MODES[mode], int(bool(normalize)),
            te_at, w_at, out_at, ws.data_ptr(), ws.numel(), _status(status, dev), _stream(dev))
    _done("moe_layer", rc)
    return out, te, w


def moe_experts(x: torch.Tensor, top_expert: torch.Tensor, weights: torch.Tensor, w_gate_up: torch.Tensor,
                w_down: torch.Tensor, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                status: torch.Tensor | None = None) -> torch.Tensor:
    """The gated experts and their weighted sum for a routing already made:
    x [T, H], top_expert [T, top_k] int32 (-1: no expert), weights [T, top_k]
    fp32 -> y [T, H]. Sizes as for moe_layer."""
    if out is None and workspace is None and status is None:
        done = (_lib.calls or _lib.load_calls()).experts(x, top_expert, weights, w_gate_up, w_down)
        if done is not None:
            return done[0]
    stride = _rows(x, "x")
    dt = _act_dtype(x, "x")
    dev = x.device
    T, H = x.shape
    E, F, gate_up, down = _expert_weights(x, H, w_gate_up, w_down)
    _need(top_expert, torch.int32, "top_expert", dev)
    if top_expert.dim() != 2 or top_expert.shape[0] != T:
        raise ValueError("top_expert must be [%d, top_k], got %s" % (T, list(top_expert.shape)))
    K = top_expert.shape[1]
    w_at = _take(weights, (T, K), torch.float32, "weights", dev)
    if out is None:
        out = torch.empty((T, H), dtype=x.dtype, device=dev)
    out_at = _take(out, (T, H), x.dtype, "out", dev)
    lib = _lib.load()
    ws = _workspace(workspace, lib.moe_layer_workspace_size(T, H, F, E, K), dev)
    with _on(dev):
        rc = lib.moe_experts(
            x.data_ptr(), dt, stride, top_expert.data_ptr(), w_at, gate_up, down, T, H, F, E, K, out_at, ws.data_ptr(),
            ws.numel(), _status(status, dev), _stream(dev))
    _done("moe_experts", rc)
    return out


def _affine(t, H, name, dev) -> tuple[int | None, int]:
    """Address and MOE_* dtype of weight or bias ([H], or None)."""
    if t is None:
        return None, _lib.MOE_F32
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    return _take(t, (H,), t.dtype, name, dev), _act_dtype(t, name)


def moe_layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                       eps: float = 1e-5, out: torch.Tensor | None = None,
                       stats: tuple[torch.Tensor, torch.Tensor] | None = None):
    """Layer norm of the rows of x [rows, H]: (y [rows, H], mean [rows] fp32,
    rstd [rows] fp32). ``stats``: the two tensors that take mean and rstd."""
    if out is None and stats is None:
        done = (_lib.calls or _lib.load_calls()).layer_norm_fwd(x, weight, bias, eps)
        if done is not None:
            return done
    stride = _rows(x, "x")
    dt = _act_dtype(x, "x")
    dev = x.device
    M, H = x.shape
    bias_at, wdt = _affine(bias, H, "bias", dev)
    if weight is not None or bias is None:
        weight_at, wdt = _affine(weight, H, "weight", dev)
        if bias is not None and weight.dtype is not bias.dtype:
            raise TypeError("weight and bias must have one dtype, got %s and %s" % (weight.dtype, bias.dtype))
    else:
        weight_at = None
    if out is None:
        out = torch.empty((M, H), dtype=x.dtype, device=dev)
        out_at = out.data_ptr()
    else:
        out_at = _take(out, (M, H), x.dtype, "out", dev)
    if stats is None:
        mean = torch.empty(M, dtype=torch.float32, device=dev)
        rstd = torch.empty(M, dtype=torch.float32, device=dev)
        mean_at, rstd_at = mean.data_ptr(), rstd.data_ptr()
    else:
        mean, rstd = stats
        mean_at = _take(mean, (M,), torch.float32, "mean", dev)
        rstd_at = _take(rstd, (M,), torch.float32, "rstd", dev)
    with _on(dev):
        rc = _lib.load().moe_layer_norm_fwd(
            x.data_ptr(), dt, stride, weight_at, bias_at, wdt, M, H, eps, out_at, mean_at, rstd_at, _stream(dev))
    _done("moe_layer_norm_fwd", rc)
    return out, mean, rstd


def moe_layer_norm_bwd(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor | None, mean: torch.Tensor,
                       rstd: torch.Tensor, weight_dtype: torch.dtype | None = None, need_cols: bool = True,
                       out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Gradients of moe_layer_norm_fwd: (dx [rows, H], dweight [H], dbias [H]).
    dweight and dbias have weight's dtype (``weight_dtype`` without a weight,
    fp32 by default), and are None with need_cols=False."""
    if out is None and workspace is None and (weight is not None or weight_dtype is None):
        done = (_lib.calls or _lib.load_calls()).layer_norm_bwd(dy, x, weight, mean, rstd, bool(need_cols))
        if done is not None:
            return done
    stride = _rows(x, "x")
    dt = _act_dtype(x, "x")
    dev = x.device
    M, H = x.shape
    dy_stride = _rows(dy, "dy", x.dtype, x.shape, dev)
    mean_at = _take(mean, (M,), torch.float32, "mean", dev)
    rstd_at = _take(rstd, (M,), torch.float32, "rstd", dev)
    weight_at, code = _affine(weight, H, "weight", dev)
    if weight is not None:
        weight_dtype = weight.dtype
    elif weight_dtype is None:
        weight_dtype = torch.float32
    elif weight_dtype in _DTYPES:
        code = _DTYPES[weight_dtype]
    else:  # the kernels write four bytes or two an element
        raise TypeError("weight_dtype must be float32 or bfloat16, got %s" % (weight_dtype,))
    if out is None:
        out = torch.empty((M, H), dtype=x.dtype, device=dev)
    out_at = _take(out, (M, H), x.dtype, "out", dev)
    lib = _lib.load()
    dw = db = dw_at = db_at = ws_at = None
    ws_bytes = 0
    if need_cols:
        dw = torch.empty(H, dtype=weight_dtype, device=dev)
        db = torch.empty(H, dtype=weight_dtype, device=dev)
        ws = _workspace(workspace, lib.moe_layer_norm_bwd_workspace_size(M, H), dev)
        dw_at, db_at, ws_at, ws_bytes = dw.data_ptr(), db.data_ptr(), ws.data_ptr(), ws.numel()
    with _on(dev):
        rc = lib.moe_layer_norm_bwd(
            dy.data_ptr(), dy_stride, x.data_ptr(), dt, stride, weight_at, code, mean_at, rstd_at, M, H, out_at, dw_at, db_at,
            ws_at, ws_bytes, _stream(dev))
    _done("moe_layer_norm_bwd", rc)
    return out, dw, db


class GradSet:
    """The gradients that one norm covers, as the device table that
    moe_grad_norm and moe_clip_grads read. Holds references to its tensors;
    they must stay where they are (a gradient that is allocated anew needs a
    new set). ``outs``: where clipping writes; the gradients themselves by
    default. A set has one workspace: calls with it on several streams that
    may run at the same time need workspaces of their own."""

    def __init__(self, grads: Sequence[torch.Tensor], outs: Sequence[torch.Tensor] | None = None):
        self.grads, self.outs = list(grads), None if outs is None else list(outs)
        if not self.grads:
            raise ValueError("a set needs at least one tensor")
        if self.outs is not None and len(self.outs) != len(self.grads):
            raise ValueError("%d gradients and %d outs" % (len(self.grads), len(self.outs)))
        dev = self.device = self.grads[0].device
        entries = (_lib.GradTensor * len(self.grads))()
        for i, g in enumerate(self.grads):
            _need(g, None, "grads[%d]" % i, dev)
            o = g if self.outs is None else self.outs[i]
            _take(o, g.shape, g.dtype, "outs[%d]" % i, dev)
            entries[i] = _lib.GradTensor(g.data_ptr() or None, o.data_ptr() or None, g.numel(), _act_dtype(g, "grads[%d]" % i), 0)
        lib = _lib.load()
        self.pieces = lib.moe_grad_table_pieces(entries, len(entries))
        if self.pieces < 0:
            raise ValueError("invalid gradient tensors")
        size = ctypes.sizeof(_lib.GradTensor)
        host = torch.empty(max(1, self.pieces) * size, dtype=torch.uint8)
        _lib.call("moe_grad_table_fill", entries, len(entries), host.data_ptr(), self.pieces)
        self.table = host.to(dev)
        self.workspace = torch.empty(lib.moe_grad_norm_workspace_size(), dtype=torch.uint8, device=dev)


def moe_grad_set(grads: Sequence[torch.Tensor], outs: Sequence[torch.Tensor] | None = None) -> GradSet:
    """The handle for moe_grad_norm and moe_clip_grads (fp32 and bf16 tensors may be mixed)."""
    return GradSet(grads, outs)


def _grad_args(grads, norm, workspace):
    s = grads if isinstance(grads, GradSet) else GradSet(grads)
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=s.device)
    elif _need(norm, torch.float32, "norm", s.device).numel() != 1:
        raise ValueError("norm must have one element, has %d" % norm.numel())
    return s, norm, s.workspace if workspace is None else _need(workspace, torch.uint8, "workspace", s.device)


def moe_grad_norm(grads: GradSet | Sequence[torch.Tensor], norm: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """2-norm over all elements of all gradients, fp32 on the device."""
    if norm is None and workspace is None and isinstance(grads, GradSet):
        done = (_lib.calls or _lib.load_calls()).grads(grads.table, grads.workspace, grads.pieces)
        if done is not None:
            return done[0]
    s, norm, ws = _grad_args(grads, norm, workspace)
    with _on(s.device):
        rc = _lib.load().moe_grad_norm(
            s.table.data_ptr(), s.pieces, norm.data_ptr(), ws.data_ptr(), ws.numel(), _stream(s.device))
    _done("moe_grad_norm", rc)
    return norm


def moe_clip_grads(grads: GradSet | Sequence[torch.Tensor], max_norm: float, norm: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)), into the
    set's outs or in place, and returns their norm before that."""
    if norm is None and workspace is None and isinstance(grads, GradSet):
        done = (_lib.calls or _lib.load_calls()).grads(grads.table, grads.workspace, grads.pieces, max_norm)
        if done is not None:
            return done[0]
    s, norm, ws = _grad_args(grads, norm, workspace)
    with _on(s.device):
        rc = _lib.load().moe_clip_grads(
            s.table.data_ptr(), s.pieces, max_norm, norm.data_ptr(), ws.data_ptr(), ws.numel(), _stream(s.device))
    _done("moe_clip_grads", rc)
    return norm
