"""Layer norm over a voxel's channels, with an activation applied on the way.

The norm -> activation that stands before the convolutions of a residual block
(the lingbot-map README lists a layer norm; here the activation is fused into it),
its backward pass with the reduction of the weight's gradient, and a module over
SparseTensor.  All of it runs in libsubm3d.so.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from ._host import _ACTS, _DTYPES, _current_device, _device_of, _new, _no_tangents, \
    _on_side_stream, _same_device, _writable, _written

__all__ = ["layer_norm", "layer_norm_forward", "layer_norm_backward", "LayerNorm"]


def _rows(t: torch.Tensor, name: str):
    """t as rows of its last dimension: (tensor, row stride), a view where it can be.  (A
    single row is contiguous whatever torch gives as its stride.)"""
    shape = t.shape
    if not shape or shape[-1] == 0:
        raise ValueError(f"{name} must have at least one channel")
    c = shape[-1]
    if len(shape) == 2 and shape[0] > 1:
        row, col = t.stride()
        if col == 1 and row >= c:
            return t, row
    return t.contiguous(), c


def _affine(t, name: str, x_dtype, c: int, dev: int):
    """A weight or bias vector, checked and contiguous."""
    dtype = t.dtype
    if dtype is not torch.float32 and dtype is not x_dtype:
        raise ValueError(f"{name} must be float32 or {x_dtype}, got {dtype}")
    if t.dim() != 1 or t.numel() != c:
        raise ValueError(f"{name} must have shape [{c}]")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    return t if t.is_contiguous() else t.contiguous()


def _affine_code(weight, bias, x_dtype) -> int:
    if weight is None:
        return _DTYPES[x_dtype if bias is None else bias.dtype]
    if bias is not None and weight.dtype is not bias.dtype:
        raise ValueError("weight and bias must have one dtype")
    return _DTYPES[weight.dtype]


def _codes(dtype, act):
    try:
        return _DTYPES[dtype], _ACTS[act]
    except (KeyError, TypeError):
        if dtype not in _DTYPES:
            raise ValueError(f"unsupported dtype {dtype}") from None
        raise ValueError(f"unknown activation {act!r}") from None


def _norm(x, weight, bias, eps, act, out, stream, stats: bool):
    if out is not None:
        _writable(out)
    dev = x.get_device()
    if dev < 0 or dev != _current_device():
        with torch.cuda.device(_device_of(x, "x")):
            return _norm(x, weight, bias, eps, act, out, stream, stats)
    x_dtype = x.dtype
    dtype, act_code = _codes(x_dtype, act)
    rows, stride = _rows(x, "x")
    c = rows.shape[-1]
    n = x.numel() // c
    w = None if weight is None else _affine(weight, "weight", x_dtype, c, dev)
    b = None if bias is None else _affine(bias, "bias", x_dtype, c, dev)
    affine_dtype = _affine_code(w, b, x_dtype)
    if out is None:
        y = torch.empty_like(x) if x.is_contiguous() else \
            torch.empty_like(x, memory_format=torch.contiguous_format)
    else:
        _same_device(dev, "out", out)
        if out.shape != x.shape or out.dtype != x_dtype or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous {x_dtype} tensor of x's shape")
        y = out
    mean = rstd = None
    if stats:
        mean, rstd = y.new_empty((2, n), dtype=torch.float32).unbind()
    if stream is not None:
        _on_side_stream(stream, _new(rows, x), _new(w, weight), _new(b, bias), _new(y, out),
                        mean, rstd)
    _abi.subm3d_layer_norm(rows, n, c, stride, dtype, w, b, affine_dtype, eps, act_code, y, mean,
                           rstd, stream)
    if out is not None:
        _written(out)
    return y, mean, rstd


def layer_norm_forward(x: torch.Tensor, weight: torch.Tensor | None = None,
                       bias: torch.Tensor | None = None, eps: float = 1e-5,
                       act: str | None = None, out: torch.Tensor | None = None, stream=None):
    """(y, mean, rstd): layer_norm() and the row statistics (fp32 [rows]) that
    layer_norm_backward() takes.  Neither of these two is recorded by autograd."""
    return _norm(x, weight, bias, eps, act, out, stream, True)


def _stat(t, name: str, n: int, dev: int):
    if t.dtype is not torch.float32 or t.numel() != n:
        raise ValueError(f"{name} must be float32 with one value a row ({n})")
    if t.get_device() != dev:
        _same_device(dev, name, t)
    return t if t.is_contiguous() else t.contiguous()


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor,
                        rstd: torch.Tensor, weight: torch.Tensor | None = None,
                        bias: torch.Tensor | None = None, act: str | None = None,
                        wanted=(True, True, True), stream=None):
    """(dx, dweight, dbias) of layer_norm_forward(x, weight, bias, act=act).

    dy: the gradient of y, x's shape and dtype.  mean, rstd: as the forward
    returned them.  dx has x's dtype; dweight and dbias are fp32 [C] (the sum runs
    over all rows, in an order that does not change from call to call).  wanted:
    which of the three to compute; the others are None, and so are dweight without
    a weight and dbias without a bias.
    """
    dev = x.get_device()
    if dev < 0 or dev != _current_device():
        with torch.cuda.device(_device_of(x, "x")):
            return layer_norm_backward(dy, x, mean, rstd, weight, bias, act, wanted, stream)
    x_dtype, shape = x.dtype, x.shape
    dtype, act_code = _codes(x_dtype, act)
    if dy.shape != shape or dy.dtype is not x_dtype:
        raise ValueError("dy must have x's shape and dtype")
    if dy.get_device() != dev:
        _same_device(dev, "dy", dy)
    xr, x_stride = _rows(x, "x")
    dr, dy_stride = _rows(dy, "dy")
    c = shape[-1]
    n = x.numel() // c
    w = None if weight is None else _affine(weight, "weight", x_dtype, c, dev)
    b = None if bias is None else _affine(bias, "bias", x_dtype, c, dev)
    affine_dtype = _affine_code(w, b, x_dtype)
    mean_c, rstd_c = _stat(mean, "mean", n, dev), _stat(rstd, "rstd", n, dev)
    want_dx, want_dw, want_db = wanted
    dx = dw = db = ws = None
    if want_dx:
        dx = torch.empty_like(x, memory_format=torch.contiguous_format)
    if want_dw and w is not None:
        dw = mean_c.new_empty(c)
    if want_db and b is not None:
        db = mean_c.new_empty(c)
    ws_bytes = 0
    if dw is not None or db is not None:
        ws_bytes = _abi.subm3d_layer_norm_workspace_bytes(n, c)
        if ws_bytes:
            ws = mean_c.new_empty(ws_bytes // 4)
    if stream is not None:
        _on_side_stream(stream, dx, dw, db, ws, _new(xr, x), _new(dr, dy), _new(w, weight),
                        _new(b, bias), _new(mean_c, mean), _new(rstd_c, rstd))
    _abi.subm3d_layer_norm_backward(dr, dy_stride, xr, x_stride, n, c, dtype, mean_c, rstd_c, w,
                                    b, affine_dtype, act_code, dx, dw, db, ws, ws_bytes, stream)
    return dx, dw, db


class _LayerNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, act):
        y, mean, rstd = _norm(x, weight, bias, eps, act, None, None, True)
        ctx.save_for_backward(x, weight, bias, mean, rstd)
        ctx.act = act
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias, mean, rstd = ctx.saved_tensors
        dx, dw, db = layer_norm_backward(dy, x, mean, rstd, weight, bias, ctx.act,
                                         ctx.needs_input_grad[:3])
        if dw is not None:
            dw = dw.to(weight.dtype)
        if db is not None:
            db = db.to(bias.dtype)
        return dx, dw, db, None, None


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, eps: float = 1e-5, act: str | None = None,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = act((x - mean) / sqrt(var + eps) * weight + bias) over x's last dimension.

    x: [..., C] float32 or bfloat16 (rows of a matrix may be strided); weight, bias:
    optional [C], float32 or x's dtype.  act: None, "gelu" (exact erf form) or
    "silu".  fp32 arithmetic; y has x's dtype and is rounded once.  Differentiable
    in x, weight and bias (forward-mode tangents are refused); out (contiguous, may be
    x) and stream are for calls that autograd does not record.
    """
    _no_tangents(x, weight, bias)
    if torch.is_grad_enabled() and (x.requires_grad or
                                    (weight is not None and weight.requires_grad) or
                                    (bias is not None and bias.requires_grad)):
        if out is not None or stream is not None:
            raise ValueError("out and stream are not available where gradients are recorded")
        return _LayerNormFunction.apply(x, weight, bias, eps, act)
    return _norm(x, weight, bias, eps, act, out, stream, False)[0]


class LayerNorm(torch.nn.Module):
    """Layer norm over each voxel's channels, then `act` (None, "gelu", "silu").

    affine=True holds a weight (ones) and a bias (zeros) of `dtype`: float32, which
    serves float32 and bfloat16 features, or bfloat16 for bfloat16 features.
    Takes and returns a SparseTensor (or a tensor [..., C]).
    """

    def __init__(self, channels: int, eps: float = 1e-5, act: str | None = None,
                 affine: bool = True, dtype=torch.float32, device=None):
        super().__init__()
        self.channels = channels
        self.eps = eps
        self.act = act
        if affine:
            self.weight = torch.nn.Parameter(torch.ones(channels, dtype=dtype, device=device),
                                             requires_grad=False)
            self.bias = torch.nn.Parameter(torch.zeros(channels, dtype=dtype, device=device),
                                           requires_grad=False)
        else:
            self.weight = self.bias = None

    def forward(self, x):
        feats = x if isinstance(x, torch.Tensor) else x.feats
        if feats.shape[-1] != self.channels:
            raise ValueError(f"x must have {self.channels} channels")
        y = layer_norm(feats, self.weight, self.bias, self.eps, self.act)
        return y if isinstance(x, torch.Tensor) else x.replace(y)
