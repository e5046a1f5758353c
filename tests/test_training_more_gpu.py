"""The training operators where their parts meet: a saved and resumed optimizer, a block
with and without recorded gradients, and calls at the edges of what the documents allow."""
import copy
import io

import pytest
import torch

import workloads as WL
from tests import train_reference as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def S():
    import sparse_voxel_conv_b200 as S
    return S


def _through_file(obj, **how):
    f = io.BytesIO()
    torch.save(obj, f)
    f.seek(0)
    return torch.load(f, weights_only=False, **how)


def test_resumed_optimizer_rounds_alike(S):
    """The 8-bit codes of the next step are the same bytes in a copy, in a file's optimizer and
    in one that was made without the seed and loaded the state (from host tensors too)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    sizes = [5000, 33]
    mk = lambda n, s: s * torch.randn(n, device="cuda", generator=g)  # noqa: E731
    start = [mk(n, 0.1).to(BF) for n in sizes]
    grads = [[mk(n, 1e-2).to(BF) for n in sizes] for _ in range(3)]
    how = dict(state_bits=8, master_weights=True)

    def steps(opt, which):
        for k in which:
            for p, q in zip(opt.param_groups[0]["params"], grads[k]):
                p.grad = q
            opt.step()

    def bytes_of(opt):
        out = []
        for p in opt.param_groups[0]["params"]:
            out += [p.detach()] + [opt.state[p][k] for k in sorted(opt.state[p]) if k != "step"]
        return [t.reshape(-1).view(torch.uint8).clone() for t in out]

    opt = S.AdamW([torch.nn.Parameter(t.clone()) for t in start], seed=77, **how)
    steps(opt, (0, 1))
    others = [copy.deepcopy(opt), _through_file(opt)]
    for where in ({}, dict(map_location="cpu")):
        saved = _through_file(opt.state_dict(), **where)
        new = S.AdamW([torch.nn.Parameter(p.detach().clone()) for p in opt.param_groups[0]["params"]], **how)
        new.load_state_dict(saved)
        others.append(new)
    plain = S.AdamW([torch.nn.Parameter(t.clone()) for t in start], seed=78, **how)
    steps(plain, (0, 1, 2))
    steps(opt, (2,))
    want = bytes_of(opt)
    for other in others:
        steps(other, (2,))
        assert all(torch.equal(p, q) for p, q in zip(bytes_of(other), want))
    assert not all(torch.equal(p, q) for p, q in zip(bytes_of(plain), want))    # the seed matters


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_of_a_single_row_of_a_wider_matrix(S, dtype):
    """One row is contiguous whatever its stride: it is normed in place, out of place and
    backwards like a row that lies alone, and nothing beside it is written."""
    c, wide = 64, 131
    buf = torch.randn(3, wide, device="cuda").to(dtype)
    w, b = torch.rand(c, device="cuda"), torch.rand(c, device="cuda")
    dy = torch.randn(1, wide, device="cuda").to(dtype)[:, :c]
    for x in (buf[:1, :c], buf[1:2, 2:c + 2], buf[2:, 64:64 + c]):
        assert x.stride(0) == wide and x.is_contiguous()
        ref = R.Norm(x, w, b, 1e-5, "silu")
        y, mean, rstd = S.layer_norm_forward(x, w, b, act="silu")
        R.check(y, ref.y, ref.y_bound(), "y")
        want, bounds = ref.backward(dy)
        for p, q, e in zip(S.layer_norm_backward(dy, x, mean, rstd, w, b, act="silu"), want, bounds):
            R.check(p, q, e, "gradient")
        around = buf.clone()
        assert S.layer_norm(x, w, b, act="silu", out=x) is x
        assert torch.equal(x, y)
        mine = torch.zeros_like(buf, dtype=torch.bool)
        torch.as_strided(mine, x.shape, x.stride(), x.storage_offset()).fill_(True)
        assert torch.equal(buf[~mine], around[~mine])


@pytest.mark.parametrize("dtype,c,key", [(BF, 64, "shell"), (BF, 32, "shell"), (F32, 24, "shell")])
def test_block_is_one_function(S, dtype, c, key):
    """SubMResBlock3d(norm=True) gives the same bits with and without recorded gradients, also
    for features that start between 16-byte borders; the skip's gradient is the output's."""
    wl = WL.make_workload(key)
    coords = torch.from_numpy(wl.coords).cuda()
    n = coords.shape[0]
    torch.manual_seed(3)
    block = S.SubMResBlock3d(c, dtype=dtype, device="cuda", norm=True)
    buf = torch.randn(n * c + 1, device="cuda").to(dtype)
    cache = {}
    for x in (buf[:-1].view(n, c), buf[1:].view(n, c), buf[:n // 2 * 2 * c].view(n // 2, 2 * c)[:, :c]):
        st = S.SparseTensor(coords[:x.shape[0]], x, wl.grid_dim, wl.batch, cache if x.shape[0] == n else None)
        with torch.no_grad():
            want = block(st).feats
        for p in block.parameters():
            p.requires_grad_(True)
        leaf = x.detach().requires_grad_(True)      # where x lies: the norm sums in the order of its borders
        y = block(st.replace(x)).feats
        assert y.requires_grad and torch.equal(y.detach(), want)
        y = block(st.replace(leaf)).feats
        assert torch.equal(y.detach(), want)
        dy = torch.randn_like(want)
        dx, = torch.autograd.grad(y, leaf, dy)
        # conv2's own output without the skip has the gradient dx - dy
        h = block.norm2(block.conv1(block.norm1(st.replace(leaf))))
        inner, = torch.autograd.grad(block.conv2(h).feats, leaf, dy)
        half = torch.finfo(dtype).eps / 2
        assert ((dx.double() - inner.double() - dy.double()).abs() <= half * dx.double().abs() * 1.01).all()
        for p in block.parameters():
            p.requires_grad_(False)


def _differences(forward, backward, x, dy, w, b, act):
    """[(name, difference quotient, <gradient, direction>, slack, the same product for gradients
    with a fault)] of f = <dy, y> in directions of x, w and b.

    forward(x, w, b) -> y and backward(x, w, b) -> (dx, dw, db) in fp32.  The quotient over
    +-h differs from the slope by the cubic term, told from the formula's own quotients at h
    and h / 2 in 64 bits (their difference is 3/4 of it), by what y's rounding puts into f, at
    most <|dy|, bound of y> on each side over 2 h, and by the gradient's own bound."""
    ref = R.Norm(x, w, b, 1e-5, act)
    (dx, dw, db), bounds = ref.backward(dy)
    dz = dy.double() * R.act_slope(ref.z, act)
    g = dz * ref.w
    mean0, mean1 = g.mean(1, keepdim=True), (g * ref.xhat).mean(1, keepdim=True)
    # directions that each of the gradient's terms reaches: along the rows' own shift and
    # scale (where y stands still and the two means have to cancel g), and any other
    r = torch.Generator(device="cpu")
    r.manual_seed(x.shape[1])
    v = torch.randn(x.shape, generator=r, dtype=torch.float64).to(x.device) + mean0.sign() + mean1.sign() * ref.xhat
    v = v + (ref.rstd * g).sign()
    faults = {
        "x": dict(nothing=0 * dx, sign=-dx, mean=dx + ref.rstd * mean0, slope=dx + ref.rstd * ref.xhat * mean1,
                  both=ref.rstd * g),
        "w": dict(nothing=0 * dw, sign=-dw, unnormed=(dz * x.double()).sum(0)),
        "b": dict(nothing=0 * db, sign=-db),
    }
    if act:     # the activation's slope forgotten
        faults["w"]["act"] = (dy.double() * ref.xhat).sum(0)
        faults["b"]["act"] = dy.double().sum(0)
    got = dict(zip("xwb", backward(x, w, b)))
    at = dict(x=x, w=w, b=b)
    out = []
    for name, bound in zip("xwb", bounds):
        d = v if name == "x" else dict(w=dw, b=db)[name].sign() * (0.5 + torch.rand(
            w.shape, generator=r, dtype=torch.float64).to(x.device))

        def quotient(h, kernel):
            """(quotient, its direction, the rounding's share); both sides are fp32 numbers."""
            sides = [{**at, name: (at[name].double() + s * h * d).float()} for s in (1, -1)]
            refs = [R.Norm(a["x"], a["w"], a["b"], 1e-5, act) for a in sides]
            ys = [forward(a["x"], a["w"], a["b"]).double() if kernel else n.y for a, n in zip(sides, refs)]
            f = [(dy.double() * y).sum().item() for y in ys]
            noise = sum((dy.double().abs() * n.y_bound()).sum().item() for n in refs)
            way = (sides[0][name].double() - sides[1][name].double()) / (2 * h)
            return (f[0] - f[1]) / (2 * h), way, noise / (2 * h)

        h = 2.0 ** -6
        num, way, noise = quotient(h, True)
        cubic = abs(quotient(h, False)[0] - quotient(h / 2, False)[0]) * 4 / 3
        slack = 2 * cubic + noise + (bound * way.abs()).sum().item()
        out.append((name, num, (got[name].double() * way).sum().item(), slack,
                    {k: (q * way).sum().item() for k, q in faults[name].items()}))
    return out


@pytest.mark.parametrize("n,c", [(64, 48), (64, 75), (24, 1536), (12, 8200)])
@pytest.mark.parametrize("act", [None, "gelu", "silu"])
def test_norm_gradient_against_differences(S, n, c, act):
    """fp32: the gradient is the slope that the forward's differences show, and a gradient with
    a term left out, a wrong sign or without the activation's slope is not."""
    g = torch.Generator(device="cpu")
    g.manual_seed(n + c + 1)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, dy, w, b = r(n, c) + 0.3 * r(c), r(n, c) + 0.3, 1 + 0.3 * r(c), 0.3 * r(c)
    x, dy, w, b = (t.cuda() for t in (x, dy, w, b))

    def backward(x, w, b):
        _, mean, rstd = S.layer_norm_forward(x, w, b, act=act)
        return S.layer_norm_backward(dy, x, mean, rstd, w, b, act=act)

    for name, num, ana, slack, faults in _differences(lambda *a: S.layer_norm(*a, act=act), backward, x, dy, w, b, act):
        assert abs(num - ana) <= slack, (name, num, ana, slack)
        for what, wrong in faults.items():
            assert abs(num - wrong) > 2 * slack, (name, what, num, wrong, slack)


def test_residual_alone_has_its_gradient(S):
    """A frozen convolution of features without a gradient hands the residual's on."""
    wl = WL.make_workload("shell")
    coords = torch.from_numpy(wl.coords).cuda()
    n, c = coords.shape[0], 32
    conv = S.SubMConv3d(c, c, device="cuda")
    st = S.SparseTensor(coords, torch.randn(n, c, device="cuda").to(BF), wl.grid_dim, wl.batch)
    residual = torch.randn(n, c, device="cuda").to(BF)
    want = conv(st, residual=residual).feats
    assert not want.requires_grad
    leaf = residual.clone().requires_grad_(True)
    y = conv(st, residual=leaf).feats
    dy = torch.randn_like(want)
    y.backward(dy)
    assert torch.equal(y.detach(), want) and torch.equal(leaf.grad, dy)
