"""Rotary positions from voxel coordinates (or any positions with 1 to 4 axes).

The pages' flow models turn queries and keys by phases made from the sparse
coordinates (trellis_sparse_mrp_mlx commit log): each of the axes z, y, x has its
share of a head's channel pairs, and pairs that are left over keep their values.
It runs in libsubm3d.so.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from ._host import _DTYPES, _current_device, _device_of, _new, _no_tangents, _on_side_stream, \
    _same_device, _writable, _written

__all__ = ["rotary", "VoxelRotary"]


def _turn(x, positions, theta, axis_pairs, interleaved, inverse, out, stream):
    if out is not None:
        _writable(out)
    dev = x.get_device()
    if dev < 0 or dev != _current_device():
        with torch.cuda.device(_device_of(x, "x")):
            return _turn(x, positions, theta, axis_pairs, interleaved, inverse, out, stream)
    dtype, shape = x.dtype, x.shape
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    if len(shape) == 3:
        n, heads, d = shape
    elif len(shape) == 2:
        (n, d), heads = shape, 1
    else:
        raise ValueError("x must have shape [N, heads, head_dim] or [N, head_dim]")
    if d < 2 or d % 2:
        raise ValueError("head_dim must be even")
    pos_f32 = positions.dtype is torch.float32
    if not pos_f32 and positions.dtype is not torch.int32:
        raise ValueError(f"positions must be int32 or float32, got {positions.dtype}")
    p_shape = positions.shape
    if len(p_shape) != 2 or p_shape[0] != n or not 1 <= p_shape[1] <= 4:
        raise ValueError(f"positions must have shape [{n}, 1 to 4 axes]")
    axes = p_shape[1]
    if axis_pairs is None:
        axis_pairs = (d // 2 // axes,) * axes
    elif len(axis_pairs) != axes or min(axis_pairs) < 0 or sum(axis_pairs) > d // 2:
        raise ValueError(f"axis_pairs must give each of {axes} axes its pairs, {d // 2} at most")
    if positions.get_device() != dev:
        _same_device(dev, "positions", positions)
    x_in, pos_in = x, positions
    xs, ps = x.stride(), positions.stride()
    if xs[-1] != 1:
        if out is x:
            raise ValueError("x must have contiguous channels to be turned in place")
        x = x.contiguous()
        xs = x.stride()
    if ps[1] != 1:
        positions = positions.contiguous()
        ps = positions.stride()
    if out is None:
        y = torch.empty_like(x) if x.is_contiguous() else \
            torch.empty_like(x, memory_format=torch.contiguous_format)
        ys = (heads * d, d, 1)
    else:
        _same_device(dev, "out", out)
        if out.shape != shape or out.dtype != dtype or out.stride(-1) != 1:
            raise ValueError(f"out must be {dtype} of x's shape with contiguous channels")
        y, ys = out, out.stride()
    if stream is not None:
        _on_side_stream(stream, _new(x, x_in), _new(positions, pos_in), _new(y, out))
    x_head, y_head = (xs[1], ys[1]) if len(shape) == 3 else (0, d)
    _abi.subm3d_rotary(x, xs[0], x_head, n, heads, d, _DTYPES[dtype], positions, pos_f32, ps[0],
                       axis_pairs, theta, not interleaved, inverse, y, ys[0], y_head, stream)
    if out is not None:
        _written(out)
    return y


class _RotaryFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, positions, theta, axis_pairs, interleaved, inverse):
        ctx.save_for_backward(positions)
        ctx.how = theta, axis_pairs, interleaved
        ctx.inverse = inverse
        return _turn(x, positions, theta, axis_pairs, interleaved, inverse, None, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        dx = _turn(dy, *ctx.saved_tensors, *ctx.how, not ctx.inverse, None, None)
        return dx, None, None, None, None, None


def rotary(x: torch.Tensor, positions: torch.Tensor, theta: float = 10000.0, axis_pairs=None,
           interleaved: bool = True, inverse: bool = False, out: torch.Tensor | None = None,
           stream=None) -> torch.Tensor:
    """x's channel pairs turned by their row's position.

    x: [N, heads, head_dim] (or [N, head_dim]) float32 or bfloat16 with contiguous
    channels; rows and heads may be strided, so x may be the queries and keys of a
    packed projection.  positions: [N, axes] int32 or float32, 1 to 4 axes, e.g.
    coords[:, 1:] of a coordinate set.  axis_pairs: how many of the head_dim / 2
    pairs turn with each axis, in order (default: an equal share each); the rest is
    copied.  Pair j of an axis with n pairs turns by position * theta ** (-j / n).
    interleaved: pairs are (2p, 2p + 1), else (p, p + head_dim / 2).  inverse turns
    back.  out may be x (in place).  Differentiable in x, not in the positions, which
    may not require a gradient (forward-mode tangents are refused too); out and stream
    are for calls that autograd does not record.
    """
    _no_tangents(x, positions)
    if torch.is_grad_enabled() and (x.requires_grad or positions.requires_grad):
        if positions.requires_grad:
            raise ValueError("positions have no gradient: detach them")
        if out is not None or stream is not None:
            raise ValueError("out and stream are not available where gradients are recorded")
        return _RotaryFunction.apply(x, positions, theta, axis_pairs, interleaved, inverse)
    return _turn(x, positions, theta, axis_pairs, interleaved, inverse, out, stream)


class VoxelRotary(torch.nn.Module):
    """rotary() of a SparseTensor's features [N, heads * head_dim] by its own
    coordinates (z, y, x); the batch index does not turn."""

    def __init__(self, head_dim: int, theta: float = 10000.0, axis_pairs=None,
                 interleaved: bool = True):
        super().__init__()
        self.head_dim = head_dim
        self.theta = theta
        self.axis_pairs = axis_pairs
        self.interleaved = interleaved

    def forward(self, x):
        n, c = x.feats.shape
        if c % self.head_dim:
            raise ValueError(f"features must be whole heads of {self.head_dim} channels")
        heads = x.feats.reshape(n, c // self.head_dim, self.head_dim)
        y = rotary(heads, x.coords[:, 1:], self.theta, self.axis_pairs, self.interleaved)
        return x.replace(y.reshape(n, c))
