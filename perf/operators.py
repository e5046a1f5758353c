"""The operators around the sparse convolution and the cases they are measured on.

Three families, each on voxel features [N, C] or on the weights that the
convolution's gradients update:

* layer norm with an activation applied on the way, forward and backward;
* rotary positions from voxel coordinates (three axes), forward and inverse
  (which is its gradient);
* one AdamW step over many tensors, with moments in 32 or in 8 bits.

`own` false: elementary torch operations in 32 bits (64 for the angles).
`own` true: the calls that a user makes of sparse_voxel_conv_b200.
"""
import math

import torch

own = False

BLOCK = 32          # values that share a scale of the 8-bit moments
E4M3_MAX = 448.0
M32 = 0xFFFFFFFF


# ------------------------------------------------------------------- cases ----

def listed():
    return [
        # one voxel's features at the headline width: the latency of a call
        dict(name="norm silu one voxel", op="norm", n=1, c=128, dtype="bf16", affine="fp32", act="silu"),
        # the residual block's norm -> SiLU on the headline set
        dict(name="norm silu headline", op="norm", n=329839, c=128, dtype="bf16", affine="fp32", act="silu"),
        # an odd width in fp32 with no activation: rows that are not 16-byte aligned
        dict(name="norm odd width fp32", op="norm", n=50021, c=203, dtype="fp32", affine="fp32", act="none"),
        # the 64^3 shell's training step in fp32, GELU
        dict(name="norm backward shell fp32", op="norm_bwd", n=14534, c=64, dtype="fp32", affine="fp32", act="gelu"),
        # the headline set's training step
        dict(name="norm backward headline", op="norm_bwd", n=329839, c=128, dtype="bf16", affine="fp32", act="silu"),
        # a wide row, as a transformer over a 64^3 structure has it
        dict(name="norm backward wide", op="norm_bwd", n=16384, c=1536, dtype="bf16", affine="same", act="none"),
        # one voxel's heads
        dict(name="rotary one voxel", op="rotary", n=1, heads=12, packed=12, d=128, dtype="bf16",
             interleaved=True, inverse=False, positions="int32", extent=64),
        # queries and keys inside a packed projection, 64 pairs of which 63 turn
        dict(name="rotary packed q and k", op="rotary", n=131072, heads=24, packed=36, d=128, dtype="bf16",
             interleaved=True, inverse=False, positions="int32", extent=256),
        # the gradient of an odd set in fp32, halves layout, far positions
        dict(name="rotary gradient fp32", op="rotary", n=33331, heads=5, packed=5, d=72, dtype="fp32",
             interleaved=False, inverse=True, positions="int32", extent=1000000),
        # a norm's weight and bias: the latency of a step
        dict(name="adamw one norm", op="adamw", sizes="128,128", param="fp32", grad="fp32", bits=32, master=False),
        # the decoder stack's four convolutions (64 -> 128 -> 128 -> 128 -> 64) in fp32
        dict(name="adamw decoder stack", op="adamw", sizes="221184,442368,442368,221184", param="fp32",
             grad="fp32", bits=32, master=False),
        # eight 512 -> 512 convolutions in bf16 with fp32 masters and 8-bit moments
        dict(name="adamw 8 bits large", op="adamw", sizes=",".join(["7077888"] * 8), param="bf16",
             grad="fp32", bits=8, master=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "rotary", "adamw"])
    if op in ("norm", "norm_bwd"):
        c = _log_int(rng, 8, 4096)
        if rng.random() < 0.5:
            c = max(8, c // 8 * 8)
        n = _log_int(rng, 1, max(1, min(400000, 42000000 // c)))
        return dict(op=op, n=n, c=c, dtype=rng.choice(["bf16", "fp32"]),
                    affine=rng.choice(["fp32", "same"]), act=rng.choice(["none", "gelu", "silu"]))
    if op == "rotary":
        heads = rng.randint(1, 24)
        d = 2 * rng.randint(3, 64) if rng.random() < 0.5 else 16 * rng.randint(1, 8)
        n = _log_int(rng, 1, max(1, min(131072, 400000000 // (heads * d))))
        return dict(op=op, n=n, heads=heads, packed=heads + rng.choice([0, 0, heads, 3]), d=d,
                    dtype=rng.choice(["bf16", "fp32"]), interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, positions=rng.choice(["int32", "int32", "fp32"]),
                    extent=rng.choice([64, 256, 1024, 1000000]))
    bits = rng.choice([32, 8])
    param = rng.choice(["fp32", "bf16"])
    sizes = [_log_int(rng, 1, 4000000) for _ in range(rng.randint(1, 8))]
    return dict(op=op, sizes=",".join(map(str, sizes)), param=param,
                grad=rng.choice(["fp32", "bf16"]) if param == "bf16" else "fp32", bits=bits,
                master=param == "bf16" and rng.random() < 0.7)


_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp32": 4}


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        e = _BYTES[case["dtype"]]
        nc = case["n"] * case["c"]
        w = 2 * case["c"] * (4 if case["affine"] == "fp32" else e)
        if op == "norm":
            return {"bytes": 2 * nc * e + w, "flops": 8 * nc}
        return {"bytes": 3 * nc * e + 8 * case["n"] + w + 8 * case["c"], "flops": 16 * nc}
    if op == "rotary":
        e = _BYTES[case["dtype"]]
        nhd = case["n"] * case["heads"] * case["d"]
        return {"bytes": 2 * nhd * e + 12 * case["n"], "flops": 3 * nhd}
    n = sum(int(s) for s in case["sizes"].split(","))
    each = _BYTES[case["grad"]]
    each += _BYTES[case["param"]] + 8 if case["master"] else 2 * _BYTES[case["param"]]
    each += 16 if case["bits"] == 32 else 4 + 4 / BLOCK
    return {"bytes": n * each, "flops": 15 * n}


# ------------------------------------------------------------------ inputs ----

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        dt = _DT[case["dtype"]]
        n, c = case["n"], case["c"]
        # features of a convolution's output: every channel with its own mean and spread
        x = (_normal(g, n, c) * (0.5 + torch.rand(c, device="cuda", generator=g)) + 0.5 * _normal(g, c)).to(dt)
        wt = torch.float32 if case["affine"] == "fp32" else dt
        st = dict(case=case, x=x, weight=(1 + 0.2 * _normal(g, c)).to(wt), bias=(0.2 * _normal(g, c)).to(wt),
                  act=None if case["act"] == "none" else case["act"], eps=1e-5)
        if op == "norm_bwd":
            st["dy"] = _normal(g, n, c).to(dt)
            # what the forward pass kept for the backward one: a row's mean and reciprocal deviation
            xf = x.float()
            mean = xf.mean(1)
            st["mean"] = mean
            st["rstd"] = torch.rsqrt((xf - mean[:, None]).square_().mean(1) + st["eps"])
        return st
    if op == "rotary":
        dt = _DT[case["dtype"]]
        n, h, d = case["n"], case["heads"], case["d"]
        whole = _normal(g, n, case["packed"], d).to(dt)
        if case["positions"] == "int32":
            coords = torch.randint(0, case["extent"], (n, 4), device="cuda", generator=g, dtype=torch.int32)
            pos = coords[:, 1:]     # (z, y, x) of a coordinate set's (b, z, y, x)
        else:
            pos = case["extent"] * torch.rand(n, 3, device="cuda", generator=g)
        return dict(case=case, x=whole[:, :h], pos=pos, theta=10000.0)
    return _prepare_adamw(case, g)


def _prepare_adamw(case, g):
    sizes = [int(s) for s in case["sizes"].split(",")]
    pt, gt = _DT[case["param"]], _DT[case["grad"]]
    st = dict(case=case, params=[], grads=[], masters=[] if case["master"] else None, m=[], v=[],
              m_scale=[] if case["bits"] == 8 else None, v_scale=[] if case["bits"] == 8 else None,
              step=100, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, seed=1234)
    for n in sizes:
        p = 0.02 * _normal(g, n)
        # the moments after some steps of gradients whose size differs between elements
        size = 1e-3 * torch.exp(_normal(g, n))
        st["grads"].append((size * _normal(g, n)).to(gt))
        m = 0.2 * size * _normal(g, n)
        v = size.square() * (0.5 + torch.rand(n, device="cuda", generator=g))
        st["params"].append(p.to(pt))
        if case["master"]:
            st["masters"].append(p)
        if case["bits"] == 32:
            st["m"].append(m)
            st["v"].append(v)
        else:
            none = torch.full((n,), 1 << 19, device="cuda", dtype=torch.int64)   # to the nearest
            for x, codes, scales in ((m, st["m"], st["m_scale"]), (v.sqrt(), st["v"], st["v_scale"])):
                q, s = _to_8_bits(x, none)
                codes.append(q)
                scales.append(s)
    return st


# -------------------------------------------------------------- plain form ----

def _act(z, act):
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _act_slope(z, act):
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return None


def _norm(st):
    x = st["x"].float()
    d = x - x.mean(1, keepdim=True)
    rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + st["eps"])
    return _act(d * rstd * st["weight"].float() + st["bias"].float(), st["act"]).to(st["x"].dtype)


def _norm_bwd(st):
    w = st["weight"].float()
    rstd = st["rstd"][:, None]
    xhat = (st["x"].float() - st["mean"][:, None]) * rstd
    dz = st["dy"].float()
    if st["act"] is not None:
        dz = dz * _act_slope(xhat * w + st["bias"].float(), st["act"])
    g = dz * w
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return dx.to(st["x"].dtype), (dz * xhat).sum(0), dz.sum(0)


def _angles(st):
    """[N, D / 2] in 64 bits: floor(D / 2 / axes) pairs an axis, zero for the pairs behind them."""
    pos = st["pos"].double()
    half = st["case"]["d"] // 2
    per = half // pos.shape[1]
    freq = st["theta"] ** (-torch.arange(per, device="cuda", dtype=torch.float64) / max(per, 1))
    a = (pos[:, :, None] * freq).reshape(pos.shape[0], -1)
    return torch.cat([a, a.new_zeros(a.shape[0], half - a.shape[1])], 1)


def _turn(x, cos, sin, interleaved):
    half = x.shape[-1] // 2
    x0, x1 = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    y0, y1 = x0 * cos - x1 * sin, x0 * sin + x1 * cos
    return torch.stack([y0, y1], -1).flatten(-2) if interleaved else torch.cat([y0, y1], -1)


def _rotary(st):
    a = _angles(st)
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    if st["case"]["inverse"]:
        sin = -sin
    return _turn(st["x"].float(), cos, sin, st["case"]["interleaved"]).to(st["x"].dtype)


def _stir(x):
    """A mix of 32-bit words, held in Python's or torch's 64-bit whole numbers."""
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B1) & M32
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & M32
    return x ^ (x >> 16)


def _bits(n, seed, step, index, device):
    """The 32 random bits of each of a tensor's n elements at this step."""
    k1 = _stir((seed + 0x9E3779B9 * step) & M32)
    k2 = _stir((k1 + 0xBB67AE85 * (index + 1)) & M32)
    i = torch.arange(n, device=device, dtype=torch.int64)
    x = ((i & M32) + (i >> 32) * 0x3C6EF373 + k1) & M32
    x = x ^ (x >> 16)
    x = ((x * 0x9E3779B1) & M32) ^ k2
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & M32
    return x ^ (x >> 16)


def _word(x):
    return x.view(torch.int32).to(torch.int64)


def _to_8_bits(x, add):
    """x (fp32) as e4m3 values and one power of two for each 32 of them; `add`: what is added
    to the 20 bits that go before they are cut off."""
    n = x.numel()
    mag = x.abs()
    top = torch.nn.functional.pad(mag, (0, -n % BLOCK)).view(-1, BLOCK).amax(1)
    scale = (((_word(top) + 0x1FFFFF) >> 23) - 8).clamp(min=0)          # biased exponent
    # 2^-k of the scale 2^k, k = scale - 127, then e4m3's exponents on fp32's subnormal ones
    inv = ((254 - scale) << 23).to(torch.int32).view(torch.float32).repeat_interleave(BLOCK)[:n]
    code = (_word(mag * inv * 2.0 ** -120) + add) >> 20
    code = torch.where(mag > 0, code, 0)
    code = code | torch.where(x < 0, 128, 0)
    return code.to(torch.uint8).view(torch.float8_e4m3fn), scale.to(torch.uint8).view(torch.float8_e8m0fnu)


def _from_8_bits(q, scale):
    return q.float() * scale.float().repeat_interleave(BLOCK)[: q.numel()]


def _adamw(st):
    case, (b1, b2) = st["case"], st["betas"]
    st["step"] += 1
    t = st["step"]
    step_size = st["lr"] / (1 - b1 ** t)
    for i, (p, g, qm, qv) in enumerate(zip(st["params"], st["grads"], st["m"], st["v"])):
        whole = st["masters"][i] if case["master"] else p
        g, w = g.float(), whole.float()
        if case["bits"] == 8:
            m, r = _from_8_bits(qm, st["m_scale"][i]), _from_8_bits(qv, st["v_scale"][i])
            v = r * r
        else:
            m, v = qm, qv
        m = m * b1 + g * (1 - b1)
        v = v * b2 + (g * g) * (1 - b2)
        r = v.sqrt()
        w = w * (1 - st["lr"] * st["weight_decay"]) - step_size * (m / (r / math.sqrt(1 - b2 ** t) + st["eps"]))
        whole.copy_(w)
        if case["master"]:
            p.copy_(w)
        if case["bits"] == 8:
            h = _bits(p.numel(), st["seed"], t, i, p.device)
            for x, low, q, s in ((m, h & 0xFFFF, qm, st["m_scale"][i]), (r, h >> 16, qv, st["v_scale"][i])):
                codes, scales = _to_8_bits(x, (low << 4) + 8)
                if q is qv:     # a positive second moment is not stored as none
                    codes = torch.where(r > 0, codes.view(torch.uint8).clamp(min=1),
                                        codes.view(torch.uint8)).view(torch.float8_e4m3fn)
                q.copy_(codes)
                s.copy_(scales)
        else:
            qm.copy_(m)
            qv.copy_(v)
    return _adamw_outputs(st)


def _adamw_outputs(st):
    return {k: st[k] for k in ("params", "masters", "m", "v", "m_scale", "v_scale") if st[k] is not None}


# --------------------------------------------------------- the framework's ----

def _run_own(st):
    import sparse_voxel_conv_b200 as S

    op = st["case"]["op"]
    if op == "norm":
        return S.layer_norm(st["x"], st["weight"], st["bias"], eps=st["eps"], act=st["act"])
    if op == "norm_bwd":
        return S.layer_norm_backward(st["dy"], st["x"], st["mean"], st["rstd"], st["weight"], st["bias"],
                                     act=st["act"])
    if op == "rotary":
        return S.rotary(st["x"], st["pos"], theta=st["theta"], interleaved=st["case"]["interleaved"],
                        inverse=st["case"]["inverse"])
    st["step"] += 1
    S.adamw_step(st["params"], st["grads"], st["m"], st["v"], st["step"], lr=st["lr"], betas=st["betas"],
                 eps=st["eps"], weight_decay=st["weight_decay"], masters=st["masters"],
                 exp_avg_scales=st["m_scale"], exp_avg_sq_scales=st["v_scale"], seed=st["seed"])
    return _adamw_outputs(st)


def run(st):
    if own:
        return _run_own(st)
    return {"norm": _norm, "norm_bwd": _norm_bwd, "rotary": _rotary, "adamw": _adamw}[st["case"]["op"]](st)


# ------------------------------------------------------------ in 64 bits ----

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        x, w, b = (st[k].double().requires_grad_(op == "norm_bwd") for k in ("x", "weight", "bias"))
        mean = x.sum(1, keepdim=True) / case["c"]
        var = ((x - mean) ** 2).sum(1, keepdim=True) / case["c"]
        z = (x - mean) / (var + st["eps"]) ** 0.5 * w + b
        if st["act"] == "gelu":
            y = z * (1 - 0.5 * torch.erfc(z / 2 ** 0.5))
        elif st["act"] == "silu":
            y = z / (1 + torch.exp(-z))
        else:
            y = z
        return y if op == "norm" else torch.autograd.grad(y, (x, w, b), st["dy"].double())
    if op == "rotary":
        x = st["x"].double()
        n, h, d = x.shape
        per = d // 2 // 3
        out = x.clone()
        pos = st["pos"].double()
        way = -1 if case["inverse"] else 1
        for axis in range(3):
            for j in range(per):
                pair = axis * per + j
                i0, i1 = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, pair + d // 2)
                z = torch.complex(x[:, :, i0], x[:, :, i1])
                turn = pos[:, axis] * math.exp(-math.log(st["theta"]) * j / per)
                z = z * torch.polar(torch.ones_like(turn), way * turn)[:, None]
                out[:, :, i0], out[:, :, i1] = z.real, z.imag
        return out
    return _exact_adamw(case, st)


def _exact_adamw(case, st):
    b1, b2 = st["betas"]
    t = st["step"] + 1
    out = {k: [] for k in ("params", "masters", "m", "v", "m_scale", "v_scale") if st[k] is not None}
    for i, p in enumerate(st["params"]):
        g = st["grads"][i].double()
        w = (st["masters"][i] if case["master"] else p).double()
        m, v = st["m"][i].double(), st["v"][i].double()
        if case["bits"] == 8:
            each = torch.arange(p.numel(), device=p.device) // BLOCK
            m = m * st["m_scale"][i].double()[each]
            v = (v * st["v_scale"][i].double()[each]) ** 2
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g ** 2
        w = w - st["lr"] * (st["weight_decay"] * w + m / (1 - b1 ** t) / ((v / (1 - b2 ** t)) ** 0.5 + st["eps"]))
        out["params"].append(w)
        if case["master"]:
            out["masters"].append(w)
        if case["bits"] == 32:
            out["m"].append(m)
            out["v"].append(v)
            continue
        h = _bits(p.numel(), st["seed"], t, i, p.device)
        for x, low, key in ((m, h & 0xFFFF, "m"), (v ** 0.5, h >> 16, "v")):
            top = torch.zeros(-(-p.numel() // BLOCK), device=p.device, dtype=torch.float64)
            top = top.scatter_reduce(0, each, x.abs(), "amax")
            scale = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)))      # 448 scale >= top
            y = x.abs() / scale[each]
            # the spacing of e4m3 where y lies: 2^-9 below 2^-6, an eighth of the power of two above
            gap = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6)))) / 8
            y = torch.floor(y / gap + (low.double() + 0.5) / 65536) * gap
            if key == "v":
                y = torch.where(x > 0, y.clamp(min=2.0 ** -9), y)
            out[key].append(torch.where(x < 0, -y, y))
            out[key + "_scale"].append(scale)
    return out
