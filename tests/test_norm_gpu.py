"""Layer norm, forward and backward, against the formulas in 64 bits."""
import pytest
import torch

from tests import train_reference as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def S():
    import sparse_voxel_conv_b200 as S
    return S


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _make(n, c, dtype, affine, seed, offset=0.3):
    g = _gen(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x = (r(n, c) * (0.5 + torch.rand(c, device="cuda", generator=g)) + offset * r(c)).to(dtype)
    dy = r(n, c).to(dtype)
    wt = {"fp32": F32, "same": dtype, None: None}[affine]
    w = b = None
    if wt is not None:
        w, b = (1 + 0.3 * r(c)).to(wt), (0.3 * r(c)).to(wt)
    return x, dy, w, b


def _both(S, x, dy, w, b, eps, act, what):
    ref = R.Norm(x, w, b, eps, act)
    y, mean, rstd = S.layer_norm_forward(x, w, b, eps=eps, act=act)
    assert y.dtype == x.dtype and y.shape == x.shape
    R.check(y, ref.y, ref.y_bound(), what + " y")
    R.check(mean, ref.mean[:, 0], ref.e_mean[:, 0], what + " mean")
    R.check(rstd, ref.rstd[:, 0], ref.rstd[:, 0] * (ref.e_rstd[:, 0] + R.U), what + " rstd")
    assert torch.equal(S.layer_norm(x, w, b, eps=eps, act=act), y)
    got = S.layer_norm_backward(dy, x, mean, rstd, w, b, act=act)
    want, bound = ref.backward(dy)
    assert (got[1] is None) == (w is None) and (got[2] is None) == (b is None)
    for k, name in enumerate(("dx", "dw", "db")):
        if got[k] is not None:
            assert got[k].dtype == (x.dtype if k == 0 else F32)
            R.check(got[k], want[k], bound[k], f"{what} {name}")
    again = S.layer_norm_backward(dy, x, mean, rstd, w, b, act=act)
    for p, q in zip(got, again):
        assert p is None or torch.equal(p, q), "the sums' order must not change"


# widths around every change of kernel: one channel, below and at a vector, a warp's
# and a block's share of a row, odd ones, and rows beyond a block's registers
WIDTHS = [1, 2, 3, 7, 8, 16, 24, 31, 32, 33, 64, 65, 96, 100, 128, 130, 200, 203, 256, 264, 320, 512, 520,
          640, 1000, 1024, 1032, 1536, 2048, 2056, 4096, 4104, 8192, 8200, 10001, 16384, 16392, 33000]


@pytest.mark.parametrize("c", WIDTHS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_every_width(S, c, dtype):
    act = [None, "gelu", "silu"][c % 3]
    affine = ["fp32", "same"][c // 3 % 2]
    for n in (1, 5, 67):
        x, dy, w, b = _make(n, c, dtype, affine, 10 * c + n)
        _both(S, x, dy, w, b, 1e-5, act, f"[{n}, {c}] {dtype} {act}")


@pytest.mark.parametrize("act", [None, "gelu", "silu"])
@pytest.mark.parametrize("affine", [None, "fp32", "same"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("c", [64, 75, 128, 1536])
def test_activations_and_affine(S, c, dtype, affine, act):
    x, dy, w, b = _make(300, c, dtype, affine, c)
    _both(S, x, dy, w, b, 1e-6, act, f"{c} {dtype} {affine} {act}")


@pytest.mark.parametrize("which", ["weight", "bias"])
def test_weight_or_bias_alone(S, which):
    x, dy, w, b = _make(130, 96, BF, "fp32", 3)
    w, b = (w, None) if which == "weight" else (None, b)
    _both(S, x, dy, w, b, 1e-5, "silu", which)


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 4095, 4097, 20011])
@pytest.mark.parametrize("c", [48, 128, 130])
def test_every_row_count(S, n, c):
    x, dy, w, b = _make(n, c, BF, "fp32", n)
    _both(S, x, dy, w, b, 1e-5, "gelu", f"n {n}")


def test_long_sums(S):
    x, dy, w, b = _make(400_003, 64, BF, "fp32", 5)
    _both(S, x, dy, w, b, 1e-5, "silu", "long")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("c", [64, 72, 77, 1536])
def test_far_mean_and_constant_rows(S, c, dtype):
    """A mean far above the spread, rows with no spread at all, and both in one batch."""
    x, dy, w, b = _make(40, c, dtype, "fp32", 9)
    x = (x.float() * 0.05 + 20).to(dtype)
    x[::4] = 3.0
    x[1::8] = 0.0
    _both(S, x, dy, w, b, 1e-3, "silu", f"far {c} {dtype}")


@pytest.mark.parametrize("c", [64, 96, 128, 99, 1536])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_strided_rows(S, c, dtype):
    """A slice of a wider matrix, at an aligned and at an odd offset, gives the bits of
    a contiguous copy; what lies beside it is not touched."""
    x, dy, w, b = _make(257, c, dtype, "fp32", 4)
    y0, mean, rstd = S.layer_norm_forward(x, w, b, act="silu")
    g0 = S.layer_norm_backward(dy, x, mean, rstd, w, b, act="silu")
    for off, pad in ((0, 8), (16, 32), (1, 2)):
        wide_x = torch.full((257, c + off + pad), float("nan"), dtype=dtype, device="cuda")
        wide_y = wide_x.clone()
        xs, ds = wide_x[:, off:off + c], wide_y[:, off:off + c]
        xs.copy_(x)
        ds.copy_(dy)
        ref = R.Norm(x, w, b, 1e-5, "silu")
        y, m, r = S.layer_norm_forward(xs, w, b, act="silu")
        R.check(y, ref.y, ref.y_bound(), "strided")
        want, bound = ref.backward(dy)
        for p, q, e in zip(S.layer_norm_backward(ds, xs, m, r, w, b, act="silu"), want, bound):
            R.check(p, q, e, "strided gradient")
        # dy alone strided, x contiguous
        for p, q, e in zip(S.layer_norm_backward(ds, x, mean, rstd, w, b, act="silu"), want, bound):
            R.check(p, q, e, "strided dy")
    assert torch.isfinite(y0).all() and all(torch.isfinite(t).all() for t in g0)


@pytest.mark.parametrize("n,c", [(60_001, 7), (60_001, 65), (30_005, 75), (30_003, 203), (20_002, 250), (20_009, 505),
                                 (20_001, 509), (9_001, 1001), (9_006, 1018), (5_003, 1030), (3_001, 2047), (2_999, 2049),
                                 (1_501, 4095), (1_203, 4097)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_between_borders(S, n, c, dtype):
    """Widths that are no multiple of 16 bytes, with more rows than there are teams, so that
    each team has several: contiguous, in a wider matrix whose rows lie alike against the
    borders, and in one whose rows do not."""
    act = [None, "gelu", "silu"][n % 3]
    x, dy, w, b = _make(n, c, dtype, "fp32", c)
    _both(S, x, dy, w, b, 1e-5, act, f"[{n}, {c}] {dtype} {act}")
    ref = R.Norm(x, w, b, 1e-5, act)
    want, bound = ref.backward(dy)
    for pad in (8, 3):
        wide_x = torch.full((n, c + pad), float("nan"), dtype=dtype, device="cuda")
        wide_y = wide_x.clone()
        xs, ds = wide_x[:, :c], wide_y[:, :c]
        xs.copy_(x)
        ds.copy_(dy)
        y, mean, rstd = S.layer_norm_forward(xs, w, b, act=act)
        R.check(y, ref.y, ref.y_bound(), f"{pad} y")
        for p, q, e in zip(S.layer_norm_backward(ds, xs, mean, rstd, w, b, act=act), want, bound):
            R.check(p, q, e, f"{pad} gradient")
        for p, q, e in zip(S.layer_norm_backward(dy, xs, mean, rstd, w, b, act=act), want, bound):
            R.check(p, q, e, f"{pad} gradient, dy contiguous")


@pytest.mark.parametrize("n,c", [(9_500, 520), (20_001, 768), (9_471, 1024), (9_472, 1024), (9_473, 1000), (7_103, 1032),
                                 (7_104, 1032), (15_000, 1536), (30_011, 1480), (8_000, 1544)])
@pytest.mark.parametrize("affine", [None, "fp32", "same"])
def test_long_rows_without_activation(S, n, c, affine):
    """Around the change from several warps to one warp a row, in rows and in channels."""
    x, dy, w, b = _make(n, c, BF, affine, c)
    _both(S, x, dy, w, b, 1e-5, None, f"[{n}, {c}] {affine}")
    ref = R.Norm(x, w, b, 1e-5, None)
    want, bound = ref.backward(dy)
    wide = torch.full((n, 2 * c + 16), float("nan"), dtype=BF, device="cuda")
    xs, ds = wide[:, :c], wide[:, c + 8:2 * c + 8]
    xs.copy_(x)
    ds.copy_(dy)
    _, mean, rstd = S.layer_norm_forward(xs, w, b)
    full = S.layer_norm_backward(ds, xs, mean, rstd, w, b)
    for p, q, e in zip(full, want, bound):
        if p is not None:
            R.check(p, q, e, "strided")
    only = S.layer_norm_backward(ds, xs, mean, rstd, w, b, wanted=(True, False, False))
    assert torch.equal(only[0], full[0])
    rest = S.layer_norm_backward(ds, xs, mean, rstd, w, b, wanted=(False, True, True))
    for p, q in zip(rest[1:], full[1:]):
        assert p is None or torch.equal(p, q)


def test_rows_do_not_meet_between_borders(S):
    """A row of NaN shares its 16-byte parts with its neighbours and not its values."""
    for dtype in (BF, F32):
        for c in (7, 65, 203, 1001):
            x, dy, w, b = _make(20_000, c, dtype, "fp32", 16)
            y0, m0, r0 = S.layer_norm_forward(x, w, b, act="silu")
            d0 = S.layer_norm_backward(dy, x, m0, r0, w, b, act="silu")[0]
            bad, bad_dy = x.clone(), dy.clone()
            bad[::7], bad_dy[::7] = float("nan"), float("inf")
            y, mean, rstd = S.layer_norm_forward(bad, w, b, act="silu")
            dx = S.layer_norm_backward(bad_dy, bad, mean, rstd, w, b, act="silu")[0]
            keep = torch.arange(20_000, device="cuda") % 7 != 0
            assert torch.equal(y[keep], y0[keep]) and torch.equal(dx[keep], d0[keep])
            assert torch.isnan(y[::7]).all() and torch.isnan(dx[::7]).all()


def test_rows_do_not_meet(S):
    """A row with a NaN or an infinity spoils itself (and the column sums), no other row."""
    for c in (64, 77, 1536):
        x, dy, w, b = _make(70, c, BF, "fp32", 6)
        clean = S.layer_norm(x, w, b, act="gelu")
        bad = x.clone()
        bad[13, 5] = float("nan")
        bad[40, 0] = float("inf")
        y, mean, rstd = S.layer_norm_forward(bad, w, b, act="gelu")
        keep = torch.ones(70, dtype=torch.bool, device="cuda")
        keep[13] = keep[40] = False
        assert torch.equal(y[keep], clean[keep])
        assert torch.isnan(y[13]).all() and torch.isnan(y[40]).any()
        _, m0, r0 = S.layer_norm_forward(x, w, b)
        dx0, _, _ = S.layer_norm_backward(dy, x, m0, r0, w, b, act="gelu")
        dx, dw, db = S.layer_norm_backward(dy, bad, mean, rstd, w, b, act="gelu")
        assert torch.equal(dx[keep], dx0[keep]) and torch.isnan(dx[13]).all()
        assert torch.isnan(dw).all()


@pytest.mark.parametrize("c", [8, 75, 128, 2048])
def test_no_rows(S, c):
    x = torch.empty(0, c, device="cuda", dtype=BF)
    w, b = torch.ones(c, device="cuda"), torch.zeros(c, device="cuda")
    y, mean, rstd = S.layer_norm_forward(x, w, b, act="silu")
    assert y.shape == (0, c) and mean.numel() == rstd.numel() == 0
    dx, dw, db = S.layer_norm_backward(x, x, mean, rstd, w, b, act="silu")
    assert dx.shape == (0, c) and not dw.any() and not db.any()


def test_in_place_and_out(S):
    for c in (64, 75, 1536):
        x, _, w, b = _make(1000, c, BF, "fp32", 8)
        want = S.layer_norm(x, w, b, act="silu")
        out = torch.full_like(x, float("nan"))
        assert S.layer_norm(x, w, b, act="silu", out=out) is out
        assert torch.equal(out, want)
        S.layer_norm(x, w, b, act="silu", out=x)
        assert torch.equal(x, want)


def test_wanted_parts(S):
    x, dy, w, b = _make(500, 128, BF, "fp32", 11)
    _, mean, rstd = S.layer_norm_forward(x, w, b)
    full = S.layer_norm_backward(dy, x, mean, rstd, w, b)
    for k in range(8):
        wanted = tuple(bool(k >> i & 1) for i in range(3))
        got = S.layer_norm_backward(dy, x, mean, rstd, w, b, wanted=wanted)
        for ask, p, q in zip(wanted, got, full):
            assert torch.equal(p, q) if ask else p is None


def test_shapes_of_more_dimensions(S):
    x, dy, w, b = _make(60, 96, F32, "fp32", 12)
    y = S.layer_norm(x, w, b)
    assert torch.equal(S.layer_norm(x.view(3, 4, 5, 96), w, b), y.view(3, 4, 5, 96))
    assert torch.equal(S.layer_norm(x[7], w, b), y[7])
    t = x.view(6, 10, 96).transpose(0, 1)
    assert torch.equal(S.layer_norm(t, w, b), y.view(6, 10, 96).transpose(0, 1))


@pytest.mark.parametrize("act", [None, "gelu", "silu"])
def test_gradient_against_differences(S, act):
    """<dy, y(x + h v) - y(x - h v)> / 2h against <dx, v>, fp32.  With h = 2^-6 the cubic
    term is below h^2 sum |dy| |v|^3 of an O(1) third derivative; y's own rounding adds
    its bound over h."""
    x, dy, w, b = _make(64, 48, F32, "fp32", 13)
    v = torch.randn(64, 48, device="cuda", generator=_gen(1))
    _, mean, rstd = S.layer_norm_forward(x, w, b, act=act)
    dx, dw, db = S.layer_norm_backward(dy, x, mean, rstd, w, b, act=act)
    h = 2.0 ** -6

    def f(x, w, b):
        return (S.layer_norm(x, w, b, act=act).double() * dy.double()).sum().item()

    vw, vb = v[0], v[1]
    slack = h * h * 20 * dy.abs().sum().item() + 64 * R.U / h * dy.abs().sum().item()
    for name, num, ana in (
            ("x", f(x + h * v, w, b) - f(x - h * v, w, b), (dx * v).double().sum().item()),
            ("w", f(x, w + h * vw, b) - f(x, w - h * vw, b), (dw * vw).double().sum().item()),
            ("b", f(x, w, b + h * vb) - f(x, w, b - h * vb), (db * vb).double().sum().item())):
        assert abs(num / (2 * h) - ana) <= slack, (name, num / (2 * h), ana, slack)


def test_autograd(S):
    x, dy, w, b = _make(200, 128, BF, "same", 14)
    leaves = [t.clone().requires_grad_(True) for t in (x, w, b)]
    y = S.layer_norm(*leaves, act="gelu")
    y.backward(dy)
    _, mean, rstd = S.layer_norm_forward(x, w, b, act="gelu")
    want = S.layer_norm_backward(dy, x, mean, rstd, w, b, act="gelu")
    assert torch.equal(leaves[0].grad, want[0])
    assert torch.equal(leaves[1].grad, want[1].to(BF)) and torch.equal(leaves[2].grad, want[2].to(BF))
    # a gradient broadcast from one value (stride 0)
    leaves[0].grad = None
    S.layer_norm(*leaves).float().sum().backward()
    only_x = x.clone().requires_grad_(True)
    S.layer_norm(only_x).backward(dy)
    assert only_x.grad.shape == x.shape
    # a saved input that the library then overwrites must fail the backward pass
    keep = x.clone().requires_grad_(True)
    twice = keep * 1
    z = S.layer_norm(twice, w, b)
    with torch.no_grad():
        S.layer_norm(twice, w, b, out=twice)
    with pytest.raises(RuntimeError, match="inplace"):
        z.backward(dy)


def test_module_and_stream(S):
    norm = S.LayerNorm(64, act="silu", device="cuda")
    norm.weight.copy_(torch.rand(64))
    x, dy, _, _ = _make(5000, 64, BF, None, 15)
    st = S.SparseTensor(torch.zeros(5000, 4, dtype=torch.int32, device="cuda"), x, 8)
    want = S.layer_norm(x, norm.weight, norm.bias, act="silu")
    assert torch.equal(norm(st).feats, want) and torch.equal(norm(x), want)
    assert norm(st).cache is st.cache
    side = torch.cuda.Stream()
    torch.cuda._sleep(2_000_000)
    xs = x * 1  # still queued on the current stream when the side stream is handed over
    y, mean, rstd = S.layer_norm_forward(xs.t().contiguous().t(), norm.weight, norm.bias, act="silu", stream=side)
    g = S.layer_norm_backward(dy, xs, mean, rstd, norm.weight, norm.bias, act="silu", stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    _, m0, r0 = S.layer_norm_forward(x, norm.weight, norm.bias, act="silu")
    for p, q in zip(g, S.layer_norm_backward(dy, x, m0, r0, norm.weight, norm.bias, act="silu")):
        assert torch.equal(p, q)


def test_refusals(S):
    x = torch.zeros(4, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    m = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError, match="unsupported dtype"):
        S.layer_norm(x.half())
    with pytest.raises(ValueError, match="activation"):
        S.layer_norm(x, act="relu")
    with pytest.raises(ValueError, match="weight must have shape"):
        S.layer_norm(x, w[:8])
    with pytest.raises(ValueError, match="float32 or"):
        S.layer_norm(x, w.bfloat16())
    with pytest.raises(ValueError, match="one dtype"):
        S.layer_norm(x.bfloat16(), w, w.bfloat16())
    with pytest.raises(ValueError, match="out must be"):
        S.layer_norm(x, out=x.t())
    with pytest.raises(ValueError, match="weight must be on"):
        S.layer_norm(x, w.cpu())
    with pytest.raises(S.Subm3dError):
        S.layer_norm(x, eps=-1.0)
    with pytest.raises(S.Subm3dError):
        S.layer_norm(x, eps=float("nan"))
    buf = torch.zeros(5, 16, device="cuda")
    with pytest.raises(S.Subm3dError):
        S.layer_norm(buf[:4], out=buf[1:])
    with pytest.raises(ValueError, match="dy must have"):
        S.layer_norm_backward(x[:2], x, m, m)
    with pytest.raises(ValueError, match="one value a row"):
        S.layer_norm_backward(x, x, m[:3], m)
    with pytest.raises(ValueError, match="recorded"):
        S.layer_norm(x.clone().requires_grad_(True), out=torch.empty_like(x))
