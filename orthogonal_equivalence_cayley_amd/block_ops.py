"""The operators around a block's linears, through libpoetx: the residual's
addition with the root-mean-square norm (forward and backward, output in the
activations' dtype or as INT8 rows with scales), products with a weight that is
no longer trained (bias, activation, gating operand and residual in the
epilogue), and the clipping of all gradients by their global norm.

As for the layers, forward and backward are explicit calls (autograd records
nothing), torch provides memory and the current stream of the tensors' device,
and the arithmetic runs in the library's HIP kernels. Results and workspaces are
allocated by the call on that stream, so calls on several streams or captured
into several graphs share nothing. Matrices are [rows, columns] with contiguous
columns and any row stride.
"""
from __future__ import annotations

import ctypes
from array import array
from typing import NamedTuple, Optional, Sequence

import torch

from . import poetx as _px

_PX_DTYPE = {torch.float32: _px.POETX_FP32, torch.bfloat16: _px.POETX_BF16, torch.int8: _px.POETX_INT8}
_REAL = (torch.bfloat16, torch.float32)
_ACT = {name: i for i, name in enumerate(_px.ACTS)}
_LIB = _px.LIB


def _matrix(name: str, t: torch.Tensor, shape=None, dtype=None, device=None) -> int:
    """Checks a [rows, columns] argument; returns its row stride."""
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape or '[rows, columns]'}")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} is on {t.device}, expected {device or 'a GPU'}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: {t.dtype}, expected {dtype}")
    rows, cols = t.shape
    sr, sc = t.stride()
    if cols > 1 and sc != 1:
        raise ValueError(f"{name}: columns are not contiguous")
    return sr if rows > 1 else cols


def _vector(name: str, t: torch.Tensor, n: int, device) -> None:
    if t.dim() != 1 or t.shape[0] != n or t.dtype != torch.float32 or t.device != device or \
            not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous fp32 values on {device}")


def _call(fn, where: str, device: torch.device, *args) -> None:
    """fn(*args, stream) on the current stream of the tensors' device."""
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            st = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    else:
        st = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    if st != _px.POETX_OK:
        raise _px.PoetxError(st, where)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


class NormOut(NamedTuple):
    Y: torch.Tensor                  # normalised rows: X's dtype, or INT8
    H: torch.Tensor                  # X + residual (X itself without one)
    rstd: Optional[torch.Tensor]     # fp32 [T], with save
    scale: Optional[torch.Tensor]    # fp32 [T], with quantize


def add_rms_norm(X: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, quantize: bool = False, save: bool = False,
                 H: Optional[torch.Tensor] = None) -> NormOut:
    """h = X + residual (rounded to the dtype), y = h / sqrt(mean h^2 + eps) * weight.

    X, residual [T, dim] bf16 or fp32; weight fp32 [dim]. H: where h goes, X or
    residual itself for an update in place (default: a new tensor). quantize: y
    as INT8 rows, y = scale * Y. save: keep rstd for add_rms_norm_backward."""
    ld_x = _matrix("X", X)
    T, dim = X.shape
    dt, dev = X.dtype, X.device
    if dt not in _REAL:
        raise ValueError(f"X: {dt}, expected bfloat16 or float32")
    _vector("weight", weight, dim, dev)
    ld_r = ld_h = dim
    if residual is not None:
        ld_r = _matrix("residual", residual, (T, dim), dt, dev)
        if H is None:
            H = torch.empty(T, dim, dtype=dt, device=dev)
    if H is not None:
        ld_h = _matrix("H", H, (T, dim), dt, dev)
    Y = torch.empty(T, dim, dtype=torch.int8 if quantize else dt, device=dev)
    scale = torch.empty(T, dtype=torch.float32, device=dev) if quantize else None
    rstd = torch.empty(T, dtype=torch.float32, device=dev) if save else None
    d = _px.NormDesc(T, dim, _PX_DTYPE[dt], _px.POETX_INT8 if quantize else _PX_DTYPE[dt],
                     ld_x, ld_r, ld_h, dim, eps)
    _call(_LIB.poetx_add_rms_norm, "poetx_add_rms_norm", dev, d, X.data_ptr(), _ptr(residual),
          weight.data_ptr(), _ptr(H), Y.data_ptr(), _ptr(scale), _ptr(rstd))
    return NormOut(Y, X if H is None else H, rstd, scale)


def add_rms_norm_backward(G_Y: torch.Tensor, H: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                          G_H: Optional[torch.Tensor] = None, G_X: Optional[torch.Tensor] = None,
                          g_weight: Optional[torch.Tensor] = None):
    """(G_X, g_weight) from dL/dY and, with G_H, the gradient that reaches h
    through the residual stream. H and rstd are those of add_rms_norm; G_X is the
    gradient of X and of the residual alike, and may be G_Y or G_H itself.
    g_weight is fp32 [dim], overwritten."""
    ld_g = _matrix("G_Y", G_Y)
    T, dim = G_Y.shape
    dt, dev = G_Y.dtype, G_Y.device
    if dt not in _REAL:
        raise ValueError(f"G_Y: {dt}, expected bfloat16 or float32")
    ld_h = _matrix("H", H, (T, dim), dt, dev)
    _vector("weight", weight, dim, dev)
    _vector("rstd", rstd, T, dev)
    ld_gh = dim if G_H is None else _matrix("G_H", G_H, (T, dim), dt, dev)
    if G_X is None:
        G_X = torch.empty(T, dim, dtype=dt, device=dev)
    ld_gx = _matrix("G_X", G_X, (T, dim), dt, dev)
    if g_weight is None:
        g_weight = torch.empty(dim, dtype=torch.float32, device=dev)
    _vector("g_weight", g_weight, dim, dev)
    ws = torch.empty(_LIB.poetx_rms_norm_backward_workspace(T, dim), dtype=torch.uint8, device=dev)
    d = _px.NormBackwardDesc(T, dim, _PX_DTYPE[dt], ld_g, ld_gh, ld_h, ld_gx)
    _call(_LIB.poetx_rms_norm_backward, "poetx_rms_norm_backward", dev, d, G_Y.data_ptr(), _ptr(G_H),
          H.data_ptr(), weight.data_ptr(), rstd.data_ptr(), G_X.data_ptr(), g_weight.data_ptr(),
          ws.data_ptr(), ws.numel())
    return G_X, g_weight


def linear(X: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "none",
           mul: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
           x_scale: Optional[torch.Tensor] = None, w_scale: Optional[torch.Tensor] = None,
           out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """act(X W^T + bias) * mul + residual for a weight that is not trained.

    X [T, n], W [m, n] bf16, fp32, or INT8 rows with scales x_scale fp32 [T] and
    w_scale fp32 [m]. bias fp32 [m]; mul, residual [T, m] in the result's dtype.
    act: one of poetx.ACTS. The result is bf16 for INT8 operands and X's dtype
    otherwise, or out_dtype (fp32 always possible, bf16 unless X is fp32). out: a
    [T, m] tensor for it, mul or residual itself for an update in place."""
    ld_x, ld_w = _matrix("X", X), _matrix("W", W)
    T, n = X.shape
    m = W.shape[0]
    dt, dev = X.dtype, X.device
    if dt not in _PX_DTYPE:
        raise ValueError(f"X: {dt}, expected bfloat16, float32 or int8")
    if W.shape[1] != n or W.dtype != dt or W.device != dev:
        raise ValueError(f"W: {W.dtype} {tuple(W.shape)} on {W.device} for X: {dt} {tuple(X.shape)} on {dev}")
    if act not in _ACT:
        raise ValueError(f"act must be one of {_px.ACTS}")
    if dt == torch.int8:
        if x_scale is None or w_scale is None:
            raise ValueError("INT8 operands need x_scale and w_scale")
        _vector("x_scale", x_scale, T, dev)
        _vector("w_scale", w_scale, m, dev)
    elif x_scale is not None or w_scale is not None:
        raise ValueError("x_scale and w_scale are for INT8 operands")
    if bias is not None:
        _vector("bias", bias, m, dev)
    if out is None:
        out = torch.empty(T, m, dtype=out_dtype or (torch.bfloat16 if dt == torch.int8 else dt), device=dev)
        ld_y = m
    else:
        ld_y = _matrix("out", out, (T, m), out_dtype, dev)
    yt = out.dtype
    if yt not in _REAL or (dt == torch.float32 and yt != dt):
        raise ValueError(f"the result cannot be {yt} for {dt} operands")
    ld_m = m if mul is None else _matrix("mul", mul, (T, m), yt, dev)
    ld_r = m if residual is None else _matrix("residual", residual, (T, m), yt, dev)
    d = _px.LinearDesc(T, m, n, _PX_DTYPE[dt], _PX_DTYPE[yt], _ACT[act], ld_x, ld_w, ld_y, ld_m, ld_r)
    _call(_LIB.poetx_linear, "poetx_linear", dev, d, X.data_ptr(), W.data_ptr(), _ptr(x_scale),
          _ptr(w_scale), _ptr(bias), _ptr(mul), _ptr(residual), out.data_ptr())
    return out


class MergedLinear:
    """A layer whose weight is no longer trained: W [m, n] dense, or INT8 rows
    with w_scale, and an fp32 bias [m]. PoetxLayer.merged() makes one."""

    def __init__(self, W: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 w_scale: Optional[torch.Tensor] = None):
        if (W.dtype == torch.int8) != (w_scale is not None):
            raise ValueError("w_scale goes with an INT8 weight")
        self.W, self.bias, self.w_scale = W, bias, w_scale
        self.m, self.n = W.shape

    def forward(self, X: torch.Tensor, act: str = "none", mul: Optional[torch.Tensor] = None,
                residual: Optional[torch.Tensor] = None, x_scale: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None,
                out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
        """linear() with this weight: X in its dtype (INT8 weights: INT8 rows with
        x_scale, as add_rms_norm(quantize=True) gives them)."""
        return linear(X, self.W, self.bias, act, mul, residual, x_scale, self.w_scale, out, out_dtype)


def clip_grads(grads: Sequence[torch.Tensor], max_norm: float,
               out: Optional[Sequence[torch.Tensor]] = None) -> torch.Tensor:
    """The global 2-norm over all gradient tensors (fp32, one value, on the GPU)
    and their clipping by it: out[i] = grads[i] * min(1, max_norm / (norm + 1e-6)).

    grads: contiguous bf16 or fp32 tensors of one GPU. out: tensors of the same
    sizes and dtypes, grads itself for an update in place; None: the norm only."""
    grads = list(grads)
    if not grads:
        raise ValueError("no gradients")
    dev = grads[0].device
    if not grads[0].is_cuda:
        raise ValueError(f"gradients are on {dev}, expected a GPU")
    types = array("i")
    for g in grads:
        if g.dtype not in _REAL or g.device != dev or not g.is_contiguous():
            raise ValueError("gradients must be contiguous bf16 or fp32 tensors of one GPU")
        types.append(_PX_DTYPE[g.dtype])
    ptrs = array("Q", [g.data_ptr() for g in grads])
    ns = array("q", [g.numel() for g in grads])
    outs = None
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError(f"{len(out)} outputs for {len(grads)} gradients")
        for g, o in zip(grads, out):
            if o is not g and (o.dtype != g.dtype or o.device != dev or o.numel() != g.numel() or
                               not o.is_contiguous()):
                raise ValueError("an output differs from its gradient in size, dtype or device, or is "
                                 "not contiguous")
        outs = array("Q", [o.data_ptr() for o in out])
    norm = torch.empty((), dtype=torch.float32, device=dev)
    n = len(grads)
    ws = torch.empty(_LIB.poetx_clip_grads_workspace(n), dtype=torch.uint8, device=dev)
    addr = lambda a: None if a is None else a.buffer_info()[0]  # noqa: E731
    _call(_LIB.poetx_clip_grads, "poetx_clip_grads", dev, n, addr(ptrs), addr(ns), addr(types), addr(outs),
          max_norm, norm.data_ptr(), ws.data_ptr(), ws.numel())
    return norm
