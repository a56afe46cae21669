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

import operator
from array import array
from typing import NamedTuple, Optional, Sequence

import torch

from . import poetx as _px

_PX_DTYPE = {torch.float32: _px.POETX_FP32, torch.bfloat16: _px.POETX_BF16, torch.int8: _px.POETX_INT8}
_REAL = (torch.bfloat16, torch.float32)
_REAL_SET = frozenset(_REAL)
_ACT = {name: i for i, name in enumerate(_px.ACTS)}
_LIB = _px.LIB
_dtype_of = operator.attrgetter("dtype")
_raw_stream = torch._C._cuda_getCurrentRawStream   # of one GPU, without a Stream object around it


def _matrix(name: str, t: torch.Tensor, dev: int, shape=None, dtype=None) -> int:
    """Checks a [rows, columns] argument on GPU dev; returns its row stride."""
    size = t.shape
    if len(size) != 2 or (shape is not None and size != shape):
        raise ValueError(f"{name}: shape {tuple(size)}, expected {shape or '[rows, columns]'}")
    if dev < 0 or t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected {f'cuda:{dev}' if dev >= 0 else 'a GPU'}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: {t.dtype}, expected {dtype}")
    row, col = t.stride()
    if col != 1 and size[1] > 1:
        raise ValueError(f"{name}: columns are not contiguous")
    return row if size[0] > 1 else size[1]


def _vector(name: str, t: torch.Tensor, n: int, dev: int) -> int:
    if t.shape != (n,) or t.dtype != torch.float32 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous fp32 values on cuda:{dev}")
    return t.data_ptr()


def _call(fn, where: str, dev: int, *args) -> None:
    """fn(*args, stream) on the current stream of the tensors' GPU."""
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(dev))
    else:
        st = fn(*args, _raw_stream(dev))
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
    dev, dt = X.get_device(), X.dtype
    ld_x = _matrix("X", X, dev)
    shape = X.shape
    T, dim = shape
    if dt not in _REAL:
        raise ValueError(f"X: {dt}, expected bfloat16 or float32")
    w = _vector("weight", weight, dim, dev)
    ld_r = ld_h = dim
    if residual is not None:
        ld_r = _matrix("residual", residual, dev, shape, dt)
    if H is not None:
        ld_h = _matrix("H", H, dev, shape, dt)
    elif residual is not None:
        H = torch.empty_like(X, memory_format=torch.contiguous_format)
    code = _PX_DTYPE[dt]
    Y = torch.empty_like(X, dtype=torch.int8 if quantize else dt, memory_format=torch.contiguous_format)
    scale = torch.empty(T, dtype=torch.float32, device=X.device) if quantize else None
    rstd = torch.empty(T, dtype=torch.float32, device=X.device) if save else None
    d = _px.NormDesc(T, dim, code, _px.POETX_INT8 if quantize else code, ld_x, ld_r, ld_h, dim, eps)
    _call(_LIB.poetx_add_rms_norm, "poetx_add_rms_norm", dev, d, X.data_ptr(), _ptr(residual), w, _ptr(H),
          Y.data_ptr(), _ptr(scale), _ptr(rstd))
    return NormOut(Y, X if H is None else H, rstd, scale)


def add_rms_norm_backward(G_Y: torch.Tensor, H: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                          G_H: Optional[torch.Tensor] = None, G_X: Optional[torch.Tensor] = None,
                          g_weight: Optional[torch.Tensor] = None):
    """(G_X, g_weight) from dL/dY and, with G_H, the gradient that reaches h
    through the residual stream. H and rstd are those of add_rms_norm; G_X is the
    gradient of X and of the residual alike, and may be G_Y or G_H itself.
    g_weight is fp32 [dim], overwritten."""
    dev, dt = G_Y.get_device(), G_Y.dtype
    ld_g = _matrix("G_Y", G_Y, dev)
    shape = G_Y.shape
    T, dim = shape
    if dt not in _REAL:
        raise ValueError(f"G_Y: {dt}, expected bfloat16 or float32")
    ld_h = _matrix("H", H, dev, shape, dt)
    w, s = _vector("weight", weight, dim, dev), _vector("rstd", rstd, T, dev)
    ld_gh = dim if G_H is None else _matrix("G_H", G_H, dev, shape, dt)
    if G_X is None:
        G_X = torch.empty_like(G_Y, memory_format=torch.contiguous_format)
        ld_gx = dim
    else:
        ld_gx = _matrix("G_X", G_X, dev, shape, dt)
    if g_weight is None:
        g_weight = torch.empty(dim, dtype=torch.float32, device=G_Y.device)
    gw = _vector("g_weight", g_weight, dim, dev)
    n = _LIB.poetx_rms_norm_backward_workspace(T, dim)
    ws = torch.empty(n, dtype=torch.uint8, device=G_Y.device)
    d = _px.NormBackwardDesc(T, dim, _PX_DTYPE[dt], ld_g, ld_gh, ld_h, ld_gx)
    _call(_LIB.poetx_rms_norm_backward, "poetx_rms_norm_backward", dev, d, G_Y.data_ptr(), _ptr(G_H),
          H.data_ptr(), w, s, G_X.data_ptr(), gw, ws.data_ptr(), n)
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
    dev, dt = X.get_device(), X.dtype
    ld_x, ld_w = _matrix("X", X, dev), _matrix("W", W, dev, None, dt)
    T, n = X.shape
    m, k = W.shape
    if dt not in _PX_DTYPE:
        raise ValueError(f"X: {dt}, expected bfloat16, float32 or int8")
    if k != n:
        raise ValueError(f"W: {k} columns for {n} of X")
    if act not in _ACT:
        raise ValueError(f"act must be one of {_px.ACTS}")
    sx = sw = b = None
    if dt == torch.int8:
        if x_scale is None or w_scale is None:
            raise ValueError("INT8 operands need x_scale and w_scale")
        sx, sw = _vector("x_scale", x_scale, T, dev), _vector("w_scale", w_scale, m, dev)
    elif x_scale is not None or w_scale is not None:
        raise ValueError("x_scale and w_scale are for INT8 operands")
    if bias is not None:
        b = _vector("bias", bias, m, dev)
    shape = (T, m)
    if out is None:
        out = torch.empty(shape, dtype=out_dtype or (torch.bfloat16 if dt == torch.int8 else dt),
                          device=X.device)
        ld_y = m
    else:
        ld_y = _matrix("out", out, dev, shape, out_dtype)
    yt = out.dtype
    if yt not in _REAL or (dt == torch.float32 and yt != dt):
        raise ValueError(f"the result cannot be {yt} for {dt} operands")
    ld_m = m if mul is None else _matrix("mul", mul, dev, shape, yt)
    ld_r = m if residual is None else _matrix("residual", residual, dev, shape, yt)
    d = _px.LinearDesc(T, m, n, _PX_DTYPE[dt], _PX_DTYPE[yt], _ACT[act], ld_x, ld_w, ld_y, ld_m, ld_r)
    wsb = _LIB.poetx_linear_workspace(d) if T > 4 else 0
    ws = torch.empty(wsb, dtype=torch.uint8, device=X.device) if wsb else None
    _call(_LIB.poetx_linear, "poetx_linear", dev, d, X.data_ptr(), W.data_ptr(), sx, sw, b, _ptr(mul),
          _ptr(residual), out.data_ptr(), _ptr(ws), wsb)
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


def _facts(tensors, dev: int):
    """dtypes, element counts, addresses, and whether all are contiguous and on GPU dev."""
    T = torch.Tensor
    ok = all(map(T.is_contiguous, tensors)) and set(map(T.get_device, tensors)) == {dev}
    return (list(map(_dtype_of, tensors)), array("q", map(T.numel, tensors)),
            array("Q", map(T.data_ptr, tensors)), ok)


def clip_grads(grads: Sequence[torch.Tensor], max_norm: float,
               out: Optional[Sequence[torch.Tensor]] = None) -> torch.Tensor:
    """The global 2-norm over all gradient tensors (fp32, one value, on the GPU)
    and their clipping by it: out[i] = grads[i] * min(1, max_norm / (norm + 1e-6)).

    grads: contiguous bf16 or fp32 tensors of one GPU. out: tensors of the same
    sizes and dtypes, grads itself for an update in place; None: the norm only."""
    grads = list(grads)
    n = len(grads)
    if not n:
        raise ValueError("no gradients")
    first = grads[0]
    dev = first.get_device()
    if dev < 0:
        raise ValueError(f"gradients are on {first.device}, expected a GPU")
    # a step's gradients are hundreds of tensors: each question is one pass in C over all of them
    types, ns, ptrs, ok = _facts(grads, dev)
    if not ok or not _REAL_SET.issuperset(types):
        raise ValueError("gradients must be contiguous bf16 or fp32 tensors of one GPU")
    codes = array("i", map(_PX_DTYPE.__getitem__, types))
    outs = None
    if out is not None:
        out = list(out)
        if len(out) != n:
            raise ValueError(f"{len(out)} outputs for {n} gradients")
        if all(map(operator.is_, out, grads)):
            o_types, o_ns, outs = types, ns, ptrs
        else:
            o_types, o_ns, outs, ok = _facts(out, dev)
        if not ok or o_types != types or o_ns != ns:
            raise ValueError("an output differs from its gradient in size, dtype or device, or is not "
                             "contiguous")
    norm = torch.empty((), dtype=torch.float32, device=first.device)
    wsb = _LIB.poetx_clip_grads_workspace(n)
    ws = torch.empty(wsb, dtype=torch.uint8, device=first.device)
    _call(_LIB.poetx_clip_grads, "poetx_clip_grads", dev, n, ptrs.buffer_info()[0], ns.buffer_info()[0],
          codes.buffer_info()[0], None if outs is None else outs.buffer_info()[0], max_norm, norm.data_ptr(),
          ws.data_ptr(), wsb)
    return norm
