"""Offsets beyond 2^32 elements: the last rows (elements) of a large call equal a small
call on them alone.  Each test holds up to 60 GB."""
import pytest
import torch

from tests import train_reference as R

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def S():
    import sparse_voxel_conv_b200 as S
    yield S
    torch.cuda.empty_cache()


@pytest.fixture(autouse=True)
def _room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 70 << 30:
        pytest.skip("needs 70 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def test_norm(S):
    n, c, tail = (1 << 25) + 5, 130, 1000       # 4.36e9 elements, 4-byte aligned rows
    x = torch.zeros(n, c, device="cuda", dtype=BF)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x[-tail:] = torch.randn(tail, c, device="cuda", generator=g).to(BF)
    x[:tail] = torch.randn(tail, c, device="cuda", generator=g).to(BF)
    w, b = torch.rand(c, device="cuda", generator=g), torch.rand(c, device="cuda", generator=g)
    y, mean, rstd = S.layer_norm_forward(x, w, b, act="silu")
    for rows in (slice(0, tail), slice(n - tail, n)):
        want, m, r = S.layer_norm_forward(x[rows], w, b, act="silu")
        assert torch.equal(y[rows], want) and torch.equal(mean[rows], m) and torch.equal(rstd[rows], r)
    mid = S.layer_norm(x[:1] * 0, w, b, act="silu")
    assert torch.equal(y[n // 2], mid[0])
    dx, dw, db = S.layer_norm_backward(x, x, mean, rstd, w, b, act="silu")
    del y
    want = None
    for rows in (slice(0, tail), slice(n - tail, n)):
        part = S.layer_norm_backward(x[rows], x[rows], mean[rows], rstd[rows], w, b, act="silu")
        assert torch.equal(dx[rows], part[0])
        sums = [p.double() for p in part[1:]]
        want = sums if want is None else [p + q for p, q in zip(want, sums)]
    # all rows between are zeros in dy; two sums of 1,000 terms, joined in another order
    for got, ref in zip((dw, db), want):
        R.check(got, ref, 1e-5 * (ref.abs() + ref.square().mean().sqrt()))


def test_rotary(S):
    n, h, d, tail = (1 << 24) + 3, 4, 66, 500   # 4.43e9 elements
    x = torch.zeros(n, h, d, device="cuda", dtype=BF)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x[-tail:] = torch.randn(tail, h, d, device="cuda", generator=g).to(BF)
    pos = torch.randint(0, 1000, (n, 3), device="cuda", generator=g, dtype=torch.int32)
    want = S.rotary(x[-tail:].clone(), pos[-tail:])
    assert torch.equal(S.rotary(x, pos)[-tail:], want)
    S.rotary(x, pos, out=x)
    assert torch.equal(x[-tail:], want) and not x[:1000].any()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(S, bits):
    n, tail = (1 << 32) + 4099, 4099            # the tail's indices begin at 2^32
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    p = torch.zeros(n, device="cuda", dtype=BF)
    grad = torch.zeros(n, device="cuda", dtype=BF)
    grad[-tail:] = torch.randn(tail, device="cuda", generator=g).to(BF)
    if bits == 32:
        m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        more = {}
    else:
        code = lambda k, t: torch.zeros(k, device="cuda", dtype=torch.uint8).view(t)  # noqa: E731
        m, v = code(n, torch.float8_e4m3fn), code(n, torch.float8_e4m3fn)
        ms, vs = (code((n + 31) // 32, torch.float8_e8m0fnu) for _ in range(2))
        more = dict(exp_avg_scales=[ms], exp_avg_sq_scales=[vs], seed=5)
    S.adamw_step([p], [grad], [m], [v], 1, lr=0.5, weight_decay=0.0, **more)
    f = grad[-tail:].float()
    assert not p[:100_000].any() and not p[n // 2:n // 2 + 100_000].any()
    # the first step moves a weight by lr m / (1 - b1) / (sqrt(v / (1 - b2)) + eps) = +- lr
    R.check(p[-tail:], torch.where(f == 0, 0.0, -0.5 * f.double().sign()), torch.full_like(f.double(), 0.5 * 2.0 ** -8))
    m1, v1 = f * (1 - 0.9), (f * f) * (1 - 0.999)
    if bits == 32:
        assert torch.equal(m[-tail:], m1) and torch.equal(v[-tail:], v1)
        return
    low = R.random_bits(torch.arange(1 << 32, n, device="cuda"), 5, 1, 0)
    want, scale = R.e4m3_blocks(m1, low & 0xFFFF, False)
    assert torch.equal(ms[-scale.numel():].view(torch.uint8), scale)
    got = m[-tail:].view(torch.uint8)
    assert ((got == want) | ((got & 127) + (want & 127) == 0)).all()
    want, scale = R.e4m3_blocks(v1.sqrt(), low >> 16, True)
    assert torch.equal(v[-tail:].view(torch.uint8), want)
