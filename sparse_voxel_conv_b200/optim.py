"""AdamW over lists of tensors, with moments in 32 or in 8 bits.

What a training loop does with the gradients of backward_weight() and of the
autograd functions: one call of libsubm3d.so updates the weights and moments of all
tensors of one set of types, up to 400 of them in one launch.
"""
from __future__ import annotations

import torch

from . import _abi
from ._host import _DTYPES, _current_device, _device_of, _on_side_stream, _written

__all__ = ["adamw_step", "AdamW"]

_BLOCK = 32  # elements that share a scale of the 8-bit moments
_CODE, _SCALE = torch.float8_e4m3fn, torch.float8_e8m0fnu


def _each(name, tensors, dtype, dev: int, sizes):
    """The addresses of a list that runs along the parameters, after a check of their
    number, type, device, sizes and layout."""
    at = [t.data_ptr() for t in tensors
          if t.dtype is dtype and t.get_device() == dev and t.is_contiguous()]
    if len(at) == len(sizes) and [t.numel() for t in tensors] == sizes:
        return at
    if len(tensors) != len(sizes):
        raise ValueError(f"{name} must have one tensor for each of {len(sizes)} parameters")
    for i, (t, n) in enumerate(zip(tensors, sizes)):
        if t.dtype is not dtype:
            raise ValueError(f"{name}[{i}] must be {dtype}, got {t.dtype}")
        if t.get_device() != dev:
            raise ValueError(f"{name}[{i}] must be on cuda:{dev}, got {t.device}")
        if t.numel() != n:
            raise ValueError(f"{name}[{i}] has the wrong number of elements")
        if not t.is_contiguous():
            raise ValueError(f"{name}[{i}] must be contiguous")


def _scalar(t, name, dtype, dev: int):
    if t.numel() != 1 or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} as a tensor must be one {dtype} on cuda:{dev}")
    return t.data_ptr()


def adamw_step(params, grads, exp_avgs, exp_avg_sqs, step, lr=1e-3, betas=(0.9, 0.999),
               eps: float = 1e-8, weight_decay: float = 0.01, masters=None, exp_avg_scales=None,
               exp_avg_sq_scales=None, seed: int = 0, stream=None) -> None:
    """One AdamW step over lists of tensors, in place.

        m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
        p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)

    params: float32 or bfloat16, all of one dtype; grads: likewise (float32
    gradients of bfloat16 parameters are what backward_weight() gives).  masters:
    float32 copies that the step is taken on; params then receive their rounding.
    32-bit moments: exp_avgs (m) and exp_avg_sqs (v) float32.  8-bit moments:
    exp_avgs (m) and exp_avg_sqs (sqrt(v)) float8_e4m3fn, with exp_avg_scales and
    exp_avg_sq_scales, float8_e8m0fnu, one scale for each 32 elements; the value is
    code * scale, zero bytes are the zero state, and rounding is stochastic with
    random bits made from (seed, step, place in the list, element).
    step: t >= 1, an int or a CUDA int32 tensor of one element; lr: a float or a
    CUDA float32 tensor of one element (tensors: read when the work runs, for a
    captured graph).  All tensors contiguous and on one device.  A tensor that is
    written may not share memory with another one.
    """
    count = len(params)
    if count == 0:
        return
    dev = params[0].get_device()
    if dev < 0 or dev != _current_device():
        with torch.cuda.device(_device_of(params[0], "params")):
            return adamw_step(params, grads, exp_avgs, exp_avg_sqs, step, lr, betas, eps,
                              weight_decay, masters, exp_avg_scales, exp_avg_sq_scales, seed,
                              stream)
    if not len(grads) == len(exp_avgs) == count:
        raise ValueError(f"grads and exp_avgs must have one tensor for each of {count} parameters")
    p_type, g_type, s_type = params[0].dtype, grads[0].dtype, exp_avgs[0].dtype
    if p_type not in _DTYPES or g_type not in _DTYPES:
        raise ValueError(f"unsupported dtype {p_type} or {g_type}")
    bits8 = s_type is _CODE
    if not bits8 and s_type is not torch.float32:
        raise ValueError(f"moments must be float32 or {_CODE}, got {s_type}")
    sizes = [p.numel() for p in params]
    none = (0,) * count
    p_at = _each("params", params, p_type, dev, sizes)
    g_at = _each("grads", grads, g_type, dev, sizes)
    m_at = _each("exp_avgs", exp_avgs, s_type, dev, sizes)
    v_at = _each("exp_avg_sqs", exp_avg_sqs, s_type, dev, sizes)
    w_at = none if masters is None else _each("masters", masters, torch.float32, dev, sizes)
    ms_at = vs_at = none
    if bits8:
        if exp_avg_scales is None or exp_avg_sq_scales is None:
            raise ValueError("8-bit moments need exp_avg_scales and exp_avg_sq_scales")
        blocks = [(n + _BLOCK - 1) // _BLOCK for n in sizes]
        ms_at = _each("exp_avg_scales", exp_avg_scales, _SCALE, dev, blocks)
        vs_at = _each("exp_avg_sq_scales", exp_avg_sq_scales, _SCALE, dev, blocks)
    elif exp_avg_scales is not None or exp_avg_sq_scales is not None:
        raise ValueError("32-bit moments have no scales")
    step_at = lr_at = 0
    if isinstance(step, torch.Tensor):
        step, step_at = 0, _scalar(step, "step", torch.int32, dev)
    if isinstance(lr, torch.Tensor):
        lr, lr_at = 0.0, _scalar(lr, "lr", torch.float32, dev)
    if stream is not None:
        _on_side_stream(stream)
    _abi.subm3d_adamw(
        _abi.adamw_tensors(zip(p_at, g_at, m_at, v_at, ms_at, vs_at, w_at, sizes)), count,
        _abi.adamw_step(lr, betas[0], betas[1], eps, weight_decay, step, step_at, lr_at,
                        _DTYPES[p_type], _DTYPES[g_type], 8 if bits8 else 32, seed & 0xFFFFFFFF),
        stream)
    _written(params)
    if masters is not None:
        _written(masters)


class AdamW(torch.optim.Optimizer):
    """AdamW (decoupled weight decay) on adamw_step().

    state_bits: 32, or 8 for moments in about a byte each (see adamw_step).
    master_weights: keep float32 masters of bfloat16 parameters in the state;
    without them a bfloat16 weight loses every change below half its spacing.
    seed: of the 8-bit rounding; it is saved and loaded with the groups.  Parameters
    must be contiguous CUDA tensors.  In a captured graph call adamw_step() with a
    device step instead.
    """

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.01, state_bits: int = 32, master_weights: bool = False,
                 seed: int = 0):
        if state_bits not in (32, 8):
            raise ValueError("state_bits must be 32 or 8")
        if lr < 0 or eps < 0 or weight_decay < 0 or not all(0 <= b < 1 for b in betas):
            raise ValueError("lr, eps and weight_decay must not be negative, betas in [0, 1)")
        super().__init__(params, dict(lr=lr, betas=tuple(betas), eps=eps,
                                      weight_decay=weight_decay, state_bits=state_bits,
                                      master_weights=master_weights, seed=int(seed)))

    # The seed lies in the parameter groups, which a copy, a file and state_dict() hold: what
    # is loaded goes on with the saved stream of rounding bits.
    @property
    def seed(self) -> int:
        return self.param_groups[0]["seed"]

    @seed.setter
    def seed(self, seed: int) -> None:
        for at in (self.defaults, *self.param_groups):
            at["seed"] = int(seed)

    def __setstate__(self, state):
        super().__setstate__(state)
        for group in self.param_groups:     # saved before the groups held a seed
            group.setdefault("seed", self.defaults.get("seed", 0))
        self.defaults["seed"] = self.seed   # of groups that join later

    def _state_of(self, p, group):
        st = self.state[p]
        if not st:
            n = p.numel()
            st["step"] = 0
            if group["state_bits"] == 32:
                for k in ("exp_avg", "exp_avg_sq"):
                    st[k] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
            else:
                for k in ("exp_avg", "exp_avg_sq"):
                    st[k] = torch.zeros(p.shape, dtype=torch.uint8, device=p.device).view(_CODE)
                    st[k + "_scale"] = torch.zeros((n + _BLOCK - 1) // _BLOCK, dtype=torch.uint8,
                                                   device=p.device).view(_SCALE)
            if group["master_weights"] and p.dtype != torch.float32:
                st["master"] = p.detach().float()
        return st

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the step number would be frozen into the graph: capture "
                               "adamw_step() with a device step")
        call = 0
        for group in self.param_groups:
            sets = {}
            for p in group["params"]:
                if p.grad is None:
                    continue
                if p.grad.is_sparse:
                    raise ValueError("gradients must be dense")
                st = self._state_of(p, group)
                key = (p.device, p.dtype, p.grad.dtype, "master" in st, st["step"])
                sets.setdefault(key, []).append((p, st))
            for key, members in sets.items():
                params = [p for p, _ in members]
                states = [st for _, st in members]
                pick = lambda k: [st[k] for st in states]  # noqa: E731
                bits8 = group["state_bits"] == 8
                grads = [p.grad if p.grad.is_contiguous() else p.grad.contiguous()
                         for p in params]
                adamw_step(params, grads, pick("exp_avg"), pick("exp_avg_sq"),
                           key[-1] + 1, lr=group["lr"], betas=group["betas"], eps=group["eps"],
                           weight_decay=group["weight_decay"],
                           masters=pick("master") if key[3] else None,
                           exp_avg_scales=pick("exp_avg_scale") if bits8 else None,
                           exp_avg_sq_scales=pick("exp_avg_sq_scale") if bits8 else None,
                           seed=group["seed"] + 0x632BE5A7 * call)
                for st in states:
                    st["step"] += 1
                call += 1
        return loss

    def load_state_dict(self, state_dict):
        """As torch.optim.Optimizer, but the moments and masters keep their own types
        (the base class casts them to the parameter's)."""
        super().load_state_dict(state_dict)
        saved = [i for g in state_dict["param_groups"] for i in g["params"]]
        for i, p in zip(saved, (p for g in self.param_groups for p in g["params"])):
            for k, v in state_dict["state"].get(i, {}).items():
                if isinstance(v, torch.Tensor):
                    self.state[p][k] = v.detach().clone().to(p.device)
