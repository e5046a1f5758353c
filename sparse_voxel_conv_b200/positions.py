"""Rotary positions from voxel coordinates (or any positions with 1 to 4 axes).

The pages' flow models turn queries and keys by phases made from the sparse
coordinates (rope_phases_from_coords, trellis_sparse_mrp_mlx commit log): each of
the axes z, y, x has its share of a head's channel pairs, and pairs that are left
over keep their values.  It runs in libsubm3d.so.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from ._host import _DTYPES, _new, _on_device, _on_side_stream, _same_device, _written

__all__ = ["rotary", "VoxelRotary"]


def _turn(x, positions, theta, axis_pairs, interleaved, inverse, out, stream):
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {x.dtype}")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    if x.dim() not in (2, 3):
        raise ValueError("x must have shape [N, heads, head_dim] or [N, head_dim]")
    n, d = x.shape[0], x.shape[-1]
    heads = x.shape[1] if x.dim() == 3 else 1
    if d < 2 or d % 2:
        raise ValueError("head_dim must be even")
    if positions.dtype not in (torch.int32, torch.float32):
        raise ValueError(f"positions must be int32 or float32, got {positions.dtype}")
    if positions.dim() != 2 or positions.shape[0] != n or not 1 <= positions.shape[1] <= 4:
        raise ValueError(f"positions must have shape [{n}, 1 to 4 axes]")
    axes = positions.shape[1]
    if axis_pairs is None:
        axis_pairs = (d // 2 // axes,) * axes
    elif len(axis_pairs) != axes or min(axis_pairs) < 0 or sum(axis_pairs) > d // 2:
        raise ValueError(f"axis_pairs must give each of {axes} axes its pairs, {d // 2} at most")
    dev = x.device
    _same_device(dev, positions=positions, out=out)
    given = (x, positions)
    if x.stride(-1) != 1:
        if out is x:
            raise ValueError("x must have contiguous channels to be turned in place")
        x = x.contiguous()
    if positions.stride(1) != 1:
        positions = positions.contiguous()
    with _on_device(dev):
        if out is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=dev)
        else:
            if out.shape != x.shape or out.dtype != x.dtype or out.stride(-1) != 1:
                raise ValueError(f"out must be {x.dtype} of x's shape with contiguous channels")
            y = out
        if stream is not None:
            _on_side_stream(stream, _new(x, given[0]), _new(positions, given[1]), _new(y, out))
        one = x.dim() == 2
        _abi.subm3d_rotary(x, x.stride(0), 0 if one else x.stride(1), n, heads, d,
                           _DTYPES[x.dtype], positions, positions.dtype == torch.float32,
                           positions.stride(0), axis_pairs, theta, not interleaved, inverse, y,
                           y.stride(0), d if one else y.stride(1), stream)
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
    back.  out may be x (in place).  Differentiable in x; out and stream are for
    calls that autograd does not record.
    """
    if torch.is_grad_enabled() and x.requires_grad:
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
        y = rotary(x.feats.view(n, c // self.head_dim, self.head_dim), x.coords[:, 1:], self.theta,
                   self.axis_pairs, self.interleaved)
        return x.replace(y.view(n, c))
