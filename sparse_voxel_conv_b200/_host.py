"""What the binding's modules share: type and activation codes, checks of a
tensor argument, and the rules for calls on another stream or device."""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

from . import _abi

_DTYPES = {torch.float32: _abi.SUBM3D_F32, torch.bfloat16: _abi.SUBM3D_BF16}
_ACTS = {None: _abi.SUBM3D_ACT_NONE, "none": _abi.SUBM3D_ACT_NONE, "gelu": _abi.SUBM3D_ACT_GELU,
         "silu": _abi.SUBM3D_ACT_SILU}


def _cuda_contig(t: torch.Tensor, name: str, dtype=None) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.contiguous()


def _new(t, orig):
    """t when this binding made it (an allocation or a contiguous copy), else None."""
    return None if t is orig else t


def _on_side_stream(stream, *made) -> None:
    """Before a call enqueued on `stream` when that is not torch's current stream.

    This binding allocates outputs and scratch, and makes contiguous copies, on
    the current stream; the caching allocator hands out memory that is free in
    that stream's order only.  So the side stream first waits for the work
    already queued on the current stream, and the tensors made here are
    recorded as in use by the side stream (their memory is not handed out again
    before its work has run).  `made`: only tensors created here (None skipped);
    the caller's own tensors are the caller's to manage."""
    if stream is None:
        return
    side = (stream if isinstance(stream, torch.cuda.Stream)
            else torch.cuda.ExternalStream(int(stream)))
    current = torch.cuda.current_stream()
    if side.cuda_stream == current.cuda_stream:
        return
    side.wait_stream(current)
    for t in made:
        if t is not None:
            t.record_stream(side)


def _device_of(t: torch.Tensor, name: str) -> int:
    """The CUDA device's index of a tensor argument."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _same_device(dev: int, name: str, t) -> None:
    if t is not None and t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")


# The current device's index (what torch.cuda.current_device() returns once CUDA is up,
# without its start-up checks): the library works on the current device, so a call on
# tensors of another one is made again with that device current.
_current_device = torch._C._cuda_getDevice


def _written(tensors) -> None:
    """Tells autograd that the library wrote these tensors in place, so that a
    backward pass that had saved one of them fails instead of using the new values."""
    torch.autograd.graph.increment_version(tensors)


def _no_tangents(*tensors) -> None:
    """Refuses forward-mode tangents: the library's calls would drop them."""
    if forward_ad._current_level < 0:
        return
    if any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise NotImplementedError("forward-mode derivatives are not implemented")


def _writable(out) -> None:
    """Refuses an `out` that autograd records: its gradient would go on as if the library had
    written nothing."""
    if out.requires_grad and torch.is_grad_enabled():
        raise ValueError("out is a recorded tensor (requires_grad): detach it or use no_grad()")
