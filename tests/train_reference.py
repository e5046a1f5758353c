"""The training operators in plain torch, 64 bits, and how far a kernel may be off.

u = 2^-24 is half a step of fp32.  A sum of k terms in any order of the kernels'
(a thread's share in turn, then a tree) is off by at most (depth) u sum |term|.
"""
import math

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def act(z, name):
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def act_slope(z, name):
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


class Norm:
    """Forward and backward of the layer norm in 64 bits, with error bounds.

    Bounds, per element.  The mean is off by depth u mean|x| (the sum's depth is a
    thread's share of the row plus the trees: C / 32 + 16 covers every kernel); so
    x - mean by that and u |x - mean|; the variance by (depth + 4) u of itself and
    the square of the mean's error (absolute: 0.5 rstd^2 of it goes into rstd,
    which matters where the row is constant and eps decides); xhat by
        e_x = rstd depth u mean|x| + |xhat| ((depth + 4) u / 2 + 6 u + ...).
    The activation has slope at most 1.13 and curvature at most 0.8, and is itself
    computed to 2.5 u |z| (the rational Phi) or (6 + 2 |z|) u |act| (SiLU)."""

    def __init__(self, x, weight, bias, eps, name):
        self.dtype = x.dtype
        self.name = name
        x = x.double().reshape(-1, x.shape[-1])
        c = x.shape[1]
        self.c = c
        self.w = torch.ones(c, dtype=torch.float64, device=x.device) if weight is None else weight.double()
        self.b = torch.zeros(c, dtype=torch.float64, device=x.device) if bias is None else bias.double()
        self.mean = x.mean(1, keepdim=True)
        var = (x - self.mean).square().mean(1, keepdim=True)
        self.rstd = 1 / (var + eps).sqrt()
        self.xhat = (x - self.mean) * self.rstd
        self.z = self.xhat * self.w + self.b
        self.y = act(self.z, name)
        depth = (c / 32 + 16) * U
        e_mean = depth * x.abs().mean(1, keepdim=True)
        self.e_mean = e_mean + U * self.mean.abs()
        # relative error of rstd: half the variance's, plus its own operations
        self.e_rstd = 0.5 * (depth + 4 * U) + 0.5 * (e_mean * self.rstd) ** 2 + 4 * U
        self.e_x = self.rstd * e_mean + self.xhat.abs() * (self.e_rstd + 3 * U)
        self.e_z = self.e_x * self.w.abs() + U * (self.z.abs() + (self.xhat * self.w).abs())

    def y_bound(self):
        own = {"gelu": 4 * U * self.z.abs(), "silu": (6 + 2 * self.z.abs()) * U * self.y.abs()}
        e = 1.13 * self.e_z + own.get(self.name, 0.0)
        return e + half_step(self.dtype) * (self.y.abs() + e)

    def backward(self, dy):
        """(dx, dw, db) and their bounds."""
        dy = dy.double().reshape(self.xhat.shape)
        n = dy.shape[0]
        s = act_slope(self.z, self.name)
        dz = dy * s
        dw, db = (dz * self.xhat).sum(0), dz.sum(0)
        g = dz * self.w
        gx = g * self.xhat
        dx = self.rstd * (g - g.mean(1, keepdim=True) - self.xhat * gx.mean(1, keepdim=True))
        e_dz = torch.zeros_like(dz)
        if self.name not in (None, "none"):
            e_dz = dy.abs() * (0.8 * self.e_z + (10 + 2 * self.z.abs()) * U * (1 + self.z.abs())) + U * dz.abs()
        rows = (n / 128 + 96) * U       # the longest chain of additions of a column sum
        e_dw = (e_dz * self.xhat.abs() + dz.abs() * self.e_x + 2 * U * (dz * self.xhat).abs()).sum(0) \
            + rows * (dz * self.xhat).abs().sum(0)
        e_db = e_dz.sum(0) + rows * dz.abs().sum(0)
        depth = (self.c / 32 + 16) * U
        e_g = e_dz * self.w.abs() + U * g.abs()
        e_gx = e_g * self.xhat.abs() + g.abs() * self.e_x + U * gx.abs()
        m1 = g.abs().mean(1, keepdim=True)
        m2 = gx.abs().mean(1, keepdim=True)
        e = e_g + e_g.mean(1, keepdim=True) + (depth + 2 * U) * m1 \
            + self.xhat.abs() * (e_gx.mean(1, keepdim=True) + (depth + 3 * U) * m2) + self.e_x * m2 \
            + 3 * U * (g.abs() + m1 + self.xhat.abs() * m2)
        e = self.rstd * (e + (g.abs() + m1 + self.xhat.abs() * m2) * (self.e_rstd + U))
        e_dx = e + half_step(self.dtype) * (dx.abs() + e)
        return (dx, dw, db), (e_dx, e_dw, e_db)


def rotary(x, pos, theta, axis_pairs, interleaved, inverse):
    """(y, bound).  The angle, in turns, is off by a few 2^-53 of itself (frequency,
    product) and 2^-26 (the rest in fp32); cos and sin by that times 2 pi and by two
    steps of their own; then two products and a sum."""
    n, h, d = x.shape
    half = d // 2
    angle = torch.zeros(n, half, dtype=torch.float64, device=x.device)
    at = 0
    for a, pairs in enumerate(axis_pairs):
        for j in range(pairs):
            angle[:, at + j] = pos[:, a].double() * theta ** (-j / pairs)
        at += pairs
    if inverse:
        angle = -angle
    xd = x.double()
    x0, x1 = (xd[..., 0::2], xd[..., 1::2]) if interleaved else (xd[..., :half], xd[..., half:])
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    y0, y1 = x0 * cos - x1 * sin, x0 * sin + x1 * cos
    e = (x0.abs() + x1.abs()) * (12 * U + angle.abs()[:, None] * 2.0 ** -47)
    put = (lambda p, q: torch.stack([p, q], -1).flatten(-2)) if interleaved else \
        (lambda p, q: torch.cat([p, q], -1))
    y, e = put(y0, y1), put(e, e)
    return y, e + half_step(x.dtype) * (y.abs() + e)


def adamw(p, g, m, v, t, lr, betas, eps, wd):
    """(p', m', v') in 64 bits."""
    b1, b2 = betas
    p, g, m, v = (q.double() for q in (p, g, m, v))
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = p * (1 - lr * wd) - lr / (1 - b1 ** t) * m / ((v / (1 - b2 ** t)).sqrt() + eps)
    return p, m, v


def check(got, want, bound, what=""):
    got = got.double().reshape(want.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - bound
    if (over > 0).any():
        i = int(over.argmax())
        raise AssertionError(f"{what}: {int((over > 0).sum())} of {over.numel()} beyond the bound; worst at {i}: "
                             f"{got.flatten()[i]!r} for {want.flatten()[i]!r} +- {bound.expand_as(want).flatten()[i]!r}")


def _stir(x):
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B1) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def random_bits(i, seed, step, place):
    """The 32 random bits of elements i (int64) of the tensor at `place` in the call."""
    k1 = _stir((seed + 0x9E3779B9 * step) & 0xFFFFFFFF)
    k2 = _stir((k1 + 0xBB67AE85 * (place + 1)) & 0xFFFFFFFF)
    x = ((i & 0xFFFFFFFF) + (i >> 32) * 0x3C6EF373 + k1) & 0xFFFFFFFF
    x = x ^ (x >> 16)
    x = ((x * 0x9E3779B1) & 0xFFFFFFFF) ^ k2
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def e4m3_blocks(x, low, root):
    """(code bytes, scale bytes) of x (fp32, whole blocks of 32 but the last) with the 16-bit
    random numbers `low`: the spacing's share in units of 2^-16, plus half a unit, added
    before the cut.  In 64 bits, where every step is exact."""
    n = x.numel()
    mag = x.double().abs()
    top = torch.nn.functional.pad(mag, (0, -n % 32)).view(-1, 32).amax(1)
    mant, e = torch.frexp(top)                      # top = mant 2^e, mant in [1/2, 1)
    k = torch.where(mant > 0.875, e - 8, e - 9)     # the smallest k with top <= 448 2^k = 0.875 2^(k + 9)
    k = torch.where(top > 0, k, -127).clamp(min=-127)
    y = mag * torch.exp2(-k.double()).repeat_interleave(32)[:n]
    gap = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6)))) / 8
    # fp32 words have 2^20 values between two codes: the cut sees x's share rounded to that
    share = torch.floor(y / gap * 2 ** 20)
    y = torch.floor((share + low.double() * 16 + 8) / 2 ** 20) * gap
    if root:
        y = torch.where(x > 0, y.clamp(min=2.0 ** -9), y)
    code = torch.where(x < 0, -y, y).float().to(torch.float8_e4m3fn).view(torch.uint8)
    return code, (k + 127).to(torch.uint8)
