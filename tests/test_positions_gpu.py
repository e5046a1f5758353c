"""Rotary positions against the formula in 64 bits."""
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


def _case(n, h, d, dtype, axes, extent, seed, f32=False):
    g = _gen(seed)
    x = torch.randn(n, h, d, device="cuda", generator=g).to(dtype)
    if f32:
        pos = extent * (2 * torch.rand(n, axes, device="cuda", generator=g) - 1)
    else:
        pos = torch.randint(-extent, extent, (n, axes), device="cuda", generator=g, dtype=torch.int32)
    return x, pos


def _default(d, axes):
    return (d // 2 // axes,) * axes


@pytest.mark.parametrize("d", [2, 4, 6, 8, 12, 16, 18, 30, 32, 36, 48, 62, 64, 66, 72, 80, 96, 100, 126, 128, 136,
                               160, 256, 258, 512])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [True, False])
def test_every_head_size(S, d, dtype, interleaved):
    for n, h in ((1, 1), (3, 2), (50, 7)):
        x, pos = _case(n, h, d, dtype, 3, 300, d + n)
        for inverse in (False, True):
            y = S.rotary(x, pos, interleaved=interleaved, inverse=inverse)
            want, e = R.rotary(x, pos, 10000.0, _default(d, 3), interleaved, inverse)
            R.check(y, want, e, f"{n} {h} {d} {dtype} {interleaved} {inverse}")


@pytest.mark.parametrize("axes,pairs", [(1, None), (1, (5,)), (2, None), (2, (0, 32)), (2, (20, 3)), (3, (1, 2, 3)),
                                        (3, (0, 0, 0)), (4, None), (4, (9, 0, 1, 22))])
@pytest.mark.parametrize("interleaved", [True, False])
def test_axes(S, axes, pairs, interleaved):
    x, pos = _case(77, 3, 64, F32, axes, 1000, axes)
    y = S.rotary(x, pos, theta=500.0, axis_pairs=pairs, interleaved=interleaved)
    want, e = R.rotary(x, pos, 500.0, pairs or _default(64, axes), interleaved, False)
    R.check(y, want, e)
    if pairs == (0, 0, 0):
        assert torch.equal(y, x)


@pytest.mark.parametrize("f32", [False, True])
def test_far_positions(S, f32):
    """int32's whole range, and positions that fp32 angles would lose."""
    x, pos = _case(4000, 2, 96, F32, 3, 2 ** 31 - 1, 1, f32)
    if not f32:
        pos[0], pos[1] = 2 ** 31 - 1, -2 ** 31
    y = S.rotary(x, pos)
    want, e = R.rotary(x, pos, 10000.0, _default(96, 3), True, False)
    R.check(y, want, e)


@pytest.mark.parametrize("n", [1, 2, 31, 1000, 40_001])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_packed_and_in_place(S, n, dtype):
    """Queries and keys inside a packed projection, turned where they lie; the values
    beside them stay."""
    g = _gen(n)
    whole = torch.randn(n, 9, 64, device="cuda", generator=g).to(dtype)
    coords = torch.randint(0, 64, (n, 4), device="cuda", generator=g, dtype=torch.int32)
    for interleaved in (True, False):
        qk = whole[:, :6]
        want, e = R.rotary(qk, coords[:, 1:], 10000.0, _default(64, 3), interleaved, False)
        y = S.rotary(qk, coords[:, 1:], interleaved=interleaved)
        R.check(y, want, e)
        buf = whole.clone()
        got = S.rotary(buf[:, :6], coords[:, 1:], interleaved=interleaved, out=buf[:, :6])
        assert torch.equal(got, y) and torch.equal(buf[:, :6], y) and torch.equal(buf[:, 6:], whole[:, 6:])


@pytest.mark.parametrize("d", [64, 66, 72])
def test_layouts_of_memory(S, d):
    """Heads before rows, rows apart by an odd number of elements, odd starts, one row's
    values for all rows: the bits of a contiguous copy."""
    for dtype in (BF, F32):
        x, pos = _case(33, 4, d, dtype, 3, 100, d)
        want = S.rotary(x, pos)
        hn = x.transpose(0, 1).contiguous().transpose(0, 1)
        assert torch.equal(S.rotary(hn, pos), want)
        out = torch.empty_like(x.transpose(0, 1).contiguous()).transpose(0, 1)
        S.rotary(x, pos, out=out)
        assert torch.equal(out, want)
        flat = torch.zeros(33 * (4 * d + 5) + 1, device="cuda", dtype=dtype)
        odd = torch.as_strided(flat, (33, 4, d), (4 * d + 5, d, 1), 1)
        odd.copy_(x)
        assert torch.equal(S.rotary(odd, pos), want)
        last = x.permute(2, 0, 1).contiguous().permute(1, 2, 0)
        assert torch.equal(S.rotary(last, pos), want)
        one = x[:1].expand(33, 4, d)
        assert torch.equal(S.rotary(one, pos), S.rotary(one.contiguous(), pos))
        posx = pos.t().contiguous().t()
        assert torch.equal(S.rotary(x, posx), want)
        assert torch.equal(S.rotary(x[:, 0], pos), want[:, 0])


@pytest.mark.parametrize("d", [64, 72, 68, 70])
@pytest.mark.parametrize("start", [0, 1, 2, 4, 8])
def test_every_alignment(S, d, start):
    """Vectors that start on 2, 4, 8 or 16 bytes, in x, in the output or in both: the bits of
    aligned ones, and nothing beside them is written."""
    for dtype in (BF, F32):
        for interleaved in (True, False):
            x, pos = _case(61, 9, d, dtype, 3, 100, d)
            want = S.rotary(x, pos, interleaved=interleaved)
            size = 61 * 9 * d
            src = torch.full((size + 16,), float("nan"), device="cuda", dtype=dtype)
            dst = torch.full((size + 16,), 5.0, device="cuda", dtype=dtype)
            xs, ys = (b[start:start + size].view(61, 9, d) for b in (src, dst))
            xs.copy_(x)
            S.rotary(x, pos, interleaved=interleaved, out=ys)
            assert torch.equal(ys, want) and (dst[:start] == 5).all() and (dst[start + size:] == 5).all()
            assert torch.equal(S.rotary(xs, pos, interleaved=interleaved), want)
            S.rotary(xs, pos, interleaved=interleaved, out=xs)
            assert torch.equal(xs, want)


def test_round_trip_and_empty(S):
    x, pos = _case(500, 3, 60, F32, 3, 10 ** 6, 3)
    back = S.rotary(S.rotary(x, pos), pos, inverse=True)
    # two turns, each off by 12 u (|x0| + |x1|) and a half step
    assert ((back - x).abs().max() <= 32 * R.U * 2 * x.abs().max())
    assert S.rotary(x[:0], pos[:0]).shape == (0, 3, 60)
    assert S.rotary(x[:, :0], pos).shape == (500, 0, 60)


def test_special_values(S):
    """A NaN or an infinity stays in its pair; pairs that no axis turns are copied as they are."""
    x, pos = _case(9, 2, 64, F32, 3, 50, 4)
    clean = S.rotary(x, pos)
    x[4, 1, 10] = float("nan")
    x[5, 0, 63] = float("inf")      # pair 31 of 32: behind the three axes' ten pairs each
    y = S.rotary(x, pos)
    same = torch.ones_like(x, dtype=torch.bool)
    same[4, 1, 10:12] = False
    same[5, 0, 62:64] = False
    assert torch.equal(y[same], clean[same])
    assert torch.isnan(y[4, 1, 10:12]).all()
    assert torch.equal(y[5, 0, 62:64], x[5, 0, 62:64])


def test_autograd_and_module(S):
    x, pos = _case(40, 2, 48, F32, 3, 64, 5)
    dy = torch.randn_like(x)
    leaf = x.clone().requires_grad_(True)
    S.rotary(leaf, pos, interleaved=False).backward(dy)
    assert torch.equal(leaf.grad, S.rotary(dy, pos, interleaved=False, inverse=True))
    # a turn is linear: <dy, turn(v)> = <dx, v>
    v = torch.randn_like(x)
    lhs = (dy.double() * S.rotary(v, pos, interleaved=False).double()).sum()
    rhs = (leaf.grad.double() * v.double()).sum()
    assert abs(lhs - rhs) <= 64 * R.U * (dy.abs().double() * v.abs().double()).sum() * 2 + 1e-4
    coords = torch.cat([torch.arange(40, device="cuda", dtype=torch.int32)[:, None], pos], 1)
    st = S.SparseTensor(coords, x.reshape(40, 96), 64, 40)
    y = S.VoxelRotary(48, interleaved=False)(st)
    assert torch.equal(y.feats, S.rotary(x, pos, interleaved=False).reshape(40, 96))
    leaf.grad = None
    S.rotary(leaf, pos).sum().backward()    # a broadcast gradient
    assert torch.equal(leaf.grad, S.rotary(torch.ones_like(x), pos, inverse=True))


def test_stream(S):
    x, pos = _case(3000, 4, 64, BF, 3, 64, 6)
    want = S.rotary(x, pos)
    side = torch.cuda.Stream()
    torch.cuda._sleep(2_000_000)
    xs = x * 1
    y = S.rotary(xs, pos, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)


def test_refusals(S):
    x, pos = _case(4, 2, 8, F32, 3, 8, 7)
    with pytest.raises(ValueError, match="unsupported dtype"):
        S.rotary(x.half(), pos)
    with pytest.raises(ValueError, match="even"):
        S.rotary(x[:, :, :7], pos)
    with pytest.raises(ValueError, match="int32 or float32"):
        S.rotary(x, pos.long())
    with pytest.raises(ValueError, match="shape"):
        S.rotary(x, pos[:3])
    with pytest.raises(ValueError, match="axis_pairs"):
        S.rotary(x, pos, axis_pairs=(2, 2, 1))
    with pytest.raises(ValueError, match="axis_pairs"):
        S.rotary(x, pos, axis_pairs=(4,))
    with pytest.raises(ValueError, match="positions must be on"):
        S.rotary(x, pos.cpu())
    with pytest.raises(S.Subm3dError):
        S.rotary(x, pos, theta=0.0)
    with pytest.raises(S.Subm3dError):
        S.rotary(x, pos, theta=float("nan"))
    with pytest.raises(S.Subm3dError):
        S.rotary(torch.zeros(2, 1, 514, device="cuda"), pos[:2])
    buf = torch.zeros(5, 2, 8, device="cuda")
    with pytest.raises(S.Subm3dError):
        S.rotary(buf[:4], pos, out=buf[1:])
    with pytest.raises(S.Subm3dError):      # rows of out that are one another
        S.rotary(x, pos, out=torch.zeros(1, 2, 8, device="cuda").expand(4, 2, 8))
    with pytest.raises(ValueError, match="recorded"):
        S.rotary(x.requires_grad_(True), pos, out=torch.empty_like(x))
