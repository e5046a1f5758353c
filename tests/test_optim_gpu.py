"""The AdamW step against its formula: moments bit for bit in elementary fp32
operations, weights in 64 bits, 8-bit moments by their rounding rule."""
import math

import pytest
import torch

from tests import train_reference as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
HYPER = dict(lr=2e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.05)


@pytest.fixture(scope="module")
def S():
    import sparse_voxel_conv_b200 as S
    return S


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _zero8(n):
    nb = (n + 31) // 32
    z = lambda k, t: torch.zeros(k, dtype=torch.uint8, device="cuda").view(t)  # noqa: E731
    return z(n, E4M3), z(n, E4M3), z(nb, E8M0), z(nb, E8M0)


class Set:
    """Parameters, gradients and zero moments of several tensors."""

    def __init__(self, sizes, ptype, gtype, bits, master, seed):
        g = _gen(seed)
        self.g, self.gtype, self.bits = g, gtype, bits
        w = [0.02 * torch.randn(n, device="cuda", generator=g) for n in sizes]
        self.params = [t.to(ptype) for t in w]
        self.masters = [t.clone() for t in w] if master else None
        if bits == 32:
            self.m = [torch.zeros_like(t) for t in w]
            self.v = [torch.zeros_like(t) for t in w]
            self.ms = self.vs = None
        else:
            self.m, self.v, self.ms, self.vs = map(list, zip(*[_zero8(n) for n in sizes]))
        self.new_grads()

    def new_grads(self):
        self.grads = [(1e-3 * torch.exp(torch.randn(p.numel(), device="cuda", generator=self.g))
                       * torch.randn(p.numel(), device="cuda", generator=self.g)).to(self.gtype)
                      for p in self.params]

    def step(self, S, t, seed=7, **over):
        S.adamw_step(self.params, self.grads, self.m, self.v, t, masters=self.masters, exp_avg_scales=self.ms,
                     exp_avg_sq_scales=self.vs, seed=seed, **{**HYPER, **over})

    def values(self, i):
        """(m, sqrt(v)) as fp32."""
        if self.bits == 32:
            return self.m[i].clone(), self.v[i].clone()
        return _value(self.m[i], self.ms[i]), _value(self.v[i], self.vs[i])

    def weights(self):
        return [t.clone() for t in (self.masters or self.params)]


def _value(code, scale):
    return code.float() * scale.float().repeat_interleave(32)[:code.numel()]


def _moments_fp32(m, v, g, betas):
    """m', v': every product and sum rounded by itself."""
    b1, b2 = betas
    g = g.float()
    return m * b1 + g * (1 - b1), v * b2 + (g * g) * (1 - b2)


def _check_weights(before, g, m, v, t, got, hyper, what):
    """p' in 64 bits from the moments before the step.  The update is made of some ten
    roundings (moments 3, root 1, quotient, two products): 16 u of it; the weight's own
    product and sum: 3 u |p|.  The update is taken as large as |b1 m| + |(1 - b1) g| makes
    it: where these two cancel, m' = b1 m + (1 - b1) g keeps the roundings of its terms,
    u (|b1 m| + |(1 - b1) g|), which are many u of m' itself."""
    of = lambda m, g: R.adamw(before, g, m, v, t, hyper["lr"], hyper["betas"], hyper["eps"],  # noqa: E731
                              hyper["weight_decay"])[0]
    want = of(m, g)
    update = (of(m.abs(), g.abs()) - before.double() * (1 - hyper["lr"] * hyper["weight_decay"])).abs()
    e = 16 * R.U * update + 3 * R.U * before.double().abs()
    if got.dtype == BF:
        e = e + R.half_step(BF) * (want.abs() + e)
    R.check(got, want, e, what)


SIZES = [1, 2, 3, 7, 31, 32, 33, 255, 257, 1000, 2047, 2048, 2049, 4096, 8191, 65_537]


@pytest.mark.parametrize("ptype,gtype,master", [(F32, F32, False), (F32, BF, False), (BF, BF, False), (BF, F32, False),
                                                (BF, BF, True), (BF, F32, True), (F32, F32, True)])
@pytest.mark.parametrize("bits", [32, 8])
def test_three_steps(S, ptype, gtype, master, bits):
    st = Set(SIZES, ptype, gtype, bits, master, 1)
    for t in (1, 2, 3):
        before = st.weights()
        old = [st.values(i) for i in range(len(SIZES))]
        st.new_grads()
        st.step(S, t)
        for i, n in enumerate(SIZES):
            m, v = old[i] if bits == 32 else (old[i][0], old[i][1] * old[i][1])
            g = st.grads[i].float()
            m1, v1 = _moments_fp32(m, v, st.grads[i], HYPER["betas"])
            got = (st.masters or st.params)[i]
            _check_weights(before[i], g, m, v, t, got, HYPER, f"n {n} t {t}")
            if master:
                assert torch.equal(st.params[i], st.masters[i].to(ptype))
            new = st.values(i)
            if bits == 32:
                assert torch.equal(new[0], m1) and torch.equal(new[1], v1), f"moments of {n} at {t}"
            else:
                _check_8_bits(m1, st.m[i], st.ms[i], False)
                _check_8_bits(v1.sqrt(), st.v[i], st.vs[i], True)


def _check_8_bits(x, code, scale, positive):
    """The scale is the smallest power of two with max <= 448 scale; the value is one of the
    two codes around x (x itself where it is one); a positive x does not become zero."""
    n = x.numel()
    s = scale.float()
    pad = torch.nn.functional.pad(x.abs().double(), (0, -n % 32)).view(-1, 32).amax(1)
    assert (pad <= 448 * s.double()).all()
    small = s.double() / 2
    assert ((pad > 448 * small) | (scale.view(torch.uint8) == 0)).all()
    s = s.double().repeat_interleave(32)[:n]
    y = x.double() / s
    gap = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))) / 8
    got = code.float().double()
    low, high = torch.floor(y / gap) * gap, torch.ceil(y / gap) * gap
    ok = (got == low) | (got == high)
    if positive:
        assert (got[x > 0] > 0).all() and (got >= 0).all()
        ok |= (x > 0) & (got == 2.0 ** -9) & (y < 2.0 ** -9)
    assert ok.all()


@pytest.mark.parametrize("n", [1, 31, 32, 33, 2047, 2049, 100_003])
def test_codes_bit_for_bit(S, n):
    """The stored codes and scales are the documented rounding of the moments, with the
    documented random bits; gradients over many powers of two, so that codes of every
    size, subnormal ones among them, occur."""
    st = Set([5, n], F32, F32, 8, False, 20)
    for t in (1, 2, 70_000):
        g = [torch.randn(k, device="cuda", generator=st.g) * torch.exp2(
            torch.randint(-20, 3, (k,), device="cuda", generator=st.g).float()) for k in (5, n)]
        st.grads = g
        old = [st.values(i) for i in range(2)]
        st.step(S, t, seed=99)
        for i, k in enumerate((5, n)):
            m, v = _moments_fp32(old[i][0], old[i][1] * old[i][1], g[i], HYPER["betas"])
            bits = R.random_bits(torch.arange(k, device="cuda"), 99, t, i)
            for x, low, code, scale, root in ((m, bits & 0xFFFF, st.m[i], st.ms[i], False),
                                              (v.sqrt(), bits >> 16, st.v[i], st.vs[i], True)):
                want, want_scale = R.e4m3_blocks(x, low, root)
                assert torch.equal(scale.view(torch.uint8), want_scale)
                got = code.view(torch.uint8)
                # (the sign of a zero that a negative moment was rounded to is free)
                same = (got == want) | ((got & 127) + (want & 127) == 0)
                assert same.all(), (n, t, int((~same).sum()))


def test_rounding_has_no_bias(S):
    """Over 400 seeds the mean of each stored moment is its value: within 5.5 standard
    deviations of a step's fair split for each of 4,096 elements (a fixed set of seeds:
    the test has one outcome), and 2^-17 of a step for the 16-bit random number."""
    n, runs = 4096, 400
    st = Set([n], F32, F32, 8, False, 3)
    g = st.grads[0].clone()
    sums = [torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(2)]
    for k in range(runs):
        st.m, st.v, st.ms, st.vs = ([q] for q in _zero8(n))
        S.adamw_step(st.params, [g], st.m, st.v, 1, exp_avg_scales=st.ms, exp_avg_sq_scales=st.vs, seed=k, **HYPER)
        for s, v in zip(sums, st.values(0)):
            s += v.double()
    m1, v1 = _moments_fp32(torch.zeros_like(g), torch.zeros_like(g), g, HYPER["betas"])
    for s, x, scale in zip(sums, (m1, v1.sqrt()), (st.ms[0], st.vs[0])):
        x = x.double()
        sc = scale.float().double().repeat_interleave(32)
        y = x.abs() / sc
        gap = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6)))) / 8
        f = y / gap - torch.floor(y / gap)
        sigma = (f * (1 - f) / runs).sqrt() * gap * sc
        off = (s / runs - x).abs()
        ok = off <= 5.5 * sigma + 2.0 ** -16 * gap * sc + 1e-6 * x.abs()
        assert (ok | (y < 2.0 ** -9)).all()
        # and together: the errors do not add up in one direction
        z = ((s / runs - x) / (sigma + 1e-30))[(f > 0.01) & (f < 0.99) & (y > 2.0 ** -9)]
        assert abs(z.mean().item()) < 5 / math.sqrt(z.numel())


def test_seeds_and_places(S):
    """The same call gives the same bits; another seed, step or place in the list others."""
    def go(seed, t, order=(0, 1)):
        st = Set([4096, 4096], F32, F32, 8, False, 4)
        st.grads[1] = st.grads[0].clone()
        st.step(S, t, seed=seed)
        return [st.m[i].view(torch.uint8).clone() for i in order]

    a = go(1, 5)
    assert all(torch.equal(p, q) for p, q in zip(a, go(1, 5)))
    assert not torch.equal(a[0], a[1])
    assert not torch.equal(a[0], go(2, 5)[0])
    share = (a[0] != go(1, 6)[0]).float().mean().item()
    assert 0.2 < share < 0.6      # two fair roundings differ in 2 f (1 - f), a third on average


def test_many_steps_follow_a_moment(S):
    """v in 8 bits follows a gradient that shrinks a thousandfold (0.1 % a step is far below
    the spacing: to the nearest it would stand still)."""
    st = Set([8192], F32, F32, 8, False, 5)
    t = 0
    for size in (1.0, 1e-3):
        for _ in range(3000 if size < 1 else 50):
            t += 1
            st.grads = [torch.full((8192,), size, device="cuda")]
            st.step(S, t, seed=0, lr=0.0)
    want = 0.0
    for k in range(1, t + 1):
        want = 0.999 * want + 0.001 * (1.0 if k <= 50 else 1e-6)
    got = st.values(0)[1].double().square().mean().item()
    # squares of an unbiased root lie above by its variance: each step adds at most a
    # hundredth of a 1/64 (p (1 - p) gap^2 with p <= 0.0005 * 16), kept for 1000 steps
    assert 0.9 * want < got < 1.3 * want


def test_zero_and_tiny_moments(S):
    """Zero gradients on the zero state change nothing but the decay; a lone tiny element
    beside a large one keeps a positive root; a block of zeros stays zero."""
    for bits in (32, 8):
        st = Set([96], F32, F32, bits, False, 6)
        before = st.weights()[0]
        st.grads = [torch.zeros(96, device="cuda")]
        st.step(S, 1)
        R.check(st.params[0], before.double() * (1 - 1e-4), 2 * R.U * before.double().abs())
        assert not any(t.any() for t in st.values(0))
    g = torch.zeros(96, device="cuda")
    g[0], g[1], g[40] = 1e4, 1e-18, 1e-30
    st.grads = [g]
    st.step(S, 1)
    m, r = st.values(0)
    assert r[0] > 0 and r[1] > 0 and not r[2:32].any() and not r[64:].any()
    assert torch.isfinite(st.params[0]).all()
    for t in range(2, 30):      # gradients that stop: the root must still hold the division
        st.grads = [torch.zeros(96, device="cuda")]
        st.step(S, t, lr=1e-3)
    assert torch.isfinite(st.params[0]).all() and (st.params[0] - before).abs().max() < 0.5


def test_infinite_and_nan_gradients(S):
    """32 bits: the element alone; 8 bits: its block of 32, whose scale becomes NaN."""
    for bad in (float("nan"), float("inf")):
        for bits in (32, 8):
            st = Set([100], F32, F32, bits, False, 7)
            st.step(S, 1)
            st.new_grads()
            st.grads[0][37] = bad
            st.step(S, 2)
            st.new_grads()
            st.step(S, 3)
            nan = torch.isnan(st.params[0])
            where = torch.zeros(100, dtype=torch.bool, device="cuda")
            if bits == 32:
                where[37] = True
            else:
                where[32:64] = True
            assert torch.equal(nan, where)


def test_unaligned_and_views(S):
    """Tensors that begin between 16-byte borders and lie in one buffer give the bits of
    separate ones, and what lies between them stays."""
    for bits, ptype, master in ((32, F32, False), (8, F32, False), (8, BF, True), (32, BF, False)):
        sizes = [1000, 333, 4097]
        a, b = (Set(sizes, ptype, BF if ptype == BF else F32, bits, master, 8) for _ in range(2))

        def moved(ts, off):
            if ts is None:
                return None, None
            total = sum(t.numel() + off for t in ts) + off
            raw = torch.full((total,), 77, dtype=torch.uint8, device="cuda") if ts[0].element_size() == 1 else \
                torch.full((total,), 77.0, dtype=ts[0].dtype, device="cuda")
            views, at, mask = [], off, torch.ones(total, dtype=torch.bool, device="cuda")
            for t in ts:
                v = raw[at:at + t.numel()]
                v = v.view(t.dtype)
                v.view(torch.uint8).copy_(t.view(torch.uint8)) if t.element_size() == 1 else v.copy_(t)
                mask[at:at + t.numel()] = False
                views.append(v)
                at += t.numel() + off
            return views, (raw, mask)

        kept = []
        for name, off in (("params", 1), ("grads", 3), ("m", 1), ("v", 5), ("ms", 3), ("vs", 1), ("masters", 1)):
            views, raw = moved(getattr(b, name), off)
            setattr(b, name, views)
            kept.append(raw)
        for t in (1, 2):
            a.step(S, t)
            b.step(S, t)
        for name in ("params", "m", "v", "ms", "vs", "masters"):
            for p, q in zip(getattr(a, name) or [], getattr(b, name) or []):
                same = torch.equal(p.view(torch.uint8), q.view(torch.uint8)) if p.element_size() == 1 else torch.equal(p, q)
                assert same, (name, bits)
        for raw in kept:
            if raw is not None:
                assert (raw[0][raw[1]] == 77).all()


def test_many_tensors(S):
    """More tensors than one launch takes, empty ones among them, give what each alone gives
    (32-bit moments: the place in the list does not matter)."""
    for count in (25, 60, 1000):
        sizes = [(i * 37) % 300 if i % 11 else 0 for i in range(count)]
        a, b = (Set(sizes, F32, F32, 32, False, 9) for _ in range(2))
        a.step(S, 3)
        for i in range(count):
            S.adamw_step([b.params[i]], [b.grads[i]], [b.m[i]], [b.v[i]], 3, **HYPER)
        assert all(torch.equal(p, q) for p, q in zip(a.params, b.params))
        assert all(torch.equal(p, q) for p, q in zip(a.v, b.v))


def test_places_across_launches(S):
    """8 bits: a tensor's random bits come from its place in the call, in whichever launch it
    lies and whatever empty tensors lie before it."""
    sizes = [64] * 500
    sizes[3] = sizes[470] = 0
    st = Set(sizes, F32, F32, 8, False, 10)
    same = torch.randn(64, device="cuda", generator=_gen(1))
    st.grads = [same[:n].clone() for n in sizes]
    st.step(S, 1)
    codes = torch.stack([st.m[i].view(torch.uint8) for i in range(500) if sizes[i]])
    assert torch.unique(codes, dim=0).shape[0] > 490
    first = Set(sizes[:460], F32, F32, 8, False, 10)
    first.grads = [same[:n].clone() for n in sizes[:460]]
    first.step(S, 1)
    for i in (0, 2, 4, 439, 440, 441, 459):
        assert torch.equal(first.m[i].view(torch.uint8), st.m[i].view(torch.uint8)), i


def test_device_step_and_rate(S):
    for bits in (32, 8):
        a, b = (Set([5000, 77], F32, F32, bits, False, 11) for _ in range(2))
        t = torch.zeros(1, dtype=torch.int32, device="cuda")
        rate = torch.tensor([2e-3], device="cuda")
        for k in (1, 2, 3):
            a.step(S, k, lr=rate.double().item())
            t += 1
            b.step(S, t, lr=rate)
        for i in range(2):
            assert all(torch.equal(p, q) for p, q in zip(a.values(i), b.values(i)))
            # the rate's factors are rounded from 64 bits on both sides, by other functions
            R.check(b.params[i], a.params[i].double(), 3 * 4 * R.U * (a.params[i].double().abs() + 2e-2))


def test_optimizer(S):
    """The class against the function; parameter groups, a parameter without a gradient,
    a state that is saved and loaded."""
    for bits, ptype, master in ((32, F32, False), (8, BF, True), (32, BF, True), (8, F32, False)):
        g = _gen(12)
        shapes = [(64, 3, 3, 3, 16), (64,), (7, 5), (33,)]
        ps = [torch.nn.Parameter((0.1 * torch.randn(s, device="cuda", generator=g)).to(ptype)) for s in shapes]
        groups = [dict(params=ps[:2]), dict(params=ps[2:], lr=5e-4, weight_decay=0.0)]
        opt = S.AdamW(groups, lr=1e-3, state_bits=bits, master_weights=master, seed=5)
        ref = [p.detach().double() for p in ps]
        mom = [(torch.zeros_like(r), torch.zeros_like(r)) for r in ref]
        for t in (1, 2, 3):
            for p in ps:
                p.grad = (0.01 * torch.randn(p.shape, device="cuda", generator=g)).to(ptype)
            if t == 1:
                ps[3].grad = None
            grads = [p.grad for p in ps]
            opt.step()
            if t == 2:
                again = S.AdamW([dict(params=ps[:2]), dict(params=ps[2:], lr=1.0)], state_bits=bits,
                                master_weights=master, seed=5)
                again.load_state_dict(opt.state_dict())
                for p in ps:
                    for k, v in opt.state[p].items():
                        w = again.state[p][k]
                        if isinstance(v, torch.Tensor):
                            assert w.dtype == v.dtype and w.data_ptr() != v.data_ptr()
                            bytes_of = lambda q: q.reshape(-1).view(torch.uint8)  # noqa: E731
                            assert torch.equal(bytes_of(v), bytes_of(w))
                        else:
                            assert v == w
                assert again.param_groups[1]["lr"] == 5e-4
                opt = again
            if bits == 32 and (ptype == F32 or master):
                for i, p in enumerate(ps):
                    if grads[i] is None:
                        continue
                    lr, wd = (1e-3, 0.01) if i < 2 else (5e-4, 0.0)
                    step = t - 1 if i == 3 else t
                    ref[i], *mom[i] = R.adamw(ref[i], grads[i], *mom[i], step, lr, (0.9, 0.999), 1e-8, wd)
                    got = p if ptype == F32 else opt.state[p]["master"]
                    # three steps of at most lr / (1 - b1) each, 24 u of them, and the weight's own
                    R.check(got.detach(), ref[i], 3 * 24 * R.U * (10 * lr) + 10 * R.U * ref[i].abs(), f"{bits} {t} {i}")
        assert opt.state[ps[0]]["step"] == 3 and opt.state[ps[3]]["step"] == 2
        if bits == 8:
            assert opt.state[ps[0]]["exp_avg"].dtype == E4M3 and opt.state[ps[0]]["exp_avg_scale"].dtype == E8M0
        for p in ps:
            assert torch.isfinite(p).all()


def test_saved_weight_is_guarded(S):
    """A backward pass that saved a weight which the step then changed fails."""
    p = torch.nn.Parameter(torch.ones(64, device="cuda"))
    x = torch.randn(10, 64, device="cuda", requires_grad=True)
    y = S.layer_norm(x, p)
    z = torch.zeros(64, device="cuda")
    S.adamw_step([p.detach()], [torch.ones(64, device="cuda")], [z.clone()], [z.clone()], 1)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()


def test_refusals(S):
    def call(**over):
        z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
        a = dict(params=[z(40)], grads=[z(40)], exp_avgs=[z(40)], exp_avg_sqs=[z(40)], step=1)
        a.update(over)
        S.adamw_step(**a)

    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    call()
    call(params=[], grads=[], exp_avgs=[], exp_avg_sqs=[])
    for over, what in ((dict(grads=[]), "one tensor for each"), (dict(grads=[z(41)]), "number of elements"),
                       (dict(grads=[z(40).half()]), "unsupported dtype"), (dict(exp_avgs=[z(40).bfloat16()]), "moments"),
                       (dict(exp_avg_sqs=[z(39)]), "number of elements"), (dict(params=[z(80)[::2]]), "contiguous"),
                       (dict(params=[torch.zeros(40)]), "CUDA"), (dict(grads=[torch.zeros(40)]), "must be on"),
                       (dict(masters=[z(40).bfloat16()]), "masters"), (dict(exp_avg_scales=[z(2)]), "no scales"),
                       (dict(step=torch.ones(1, device="cuda")), "step as a tensor"),
                       (dict(lr=torch.ones(2, device="cuda")), "lr as a tensor")):
        with pytest.raises(ValueError, match=what):
            call(**over)
    m, v, ms, vs = ([q] for q in _zero8(40))
    with pytest.raises(ValueError, match="need exp_avg_scales"):
        call(exp_avgs=m, exp_avg_sqs=v)
    with pytest.raises(ValueError, match="number of elements"):
        call(exp_avgs=m, exp_avg_sqs=v, exp_avg_scales=ms, exp_avg_sq_scales=[vs[0][:1]])
    for over in (dict(step=0), dict(lr=-1.0), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=-1e-8),
                 dict(weight_decay=float("nan")), dict(lr=float("inf"))):
        with pytest.raises(S.Subm3dError):
            call(**over)
    p = z(40)
    for over in (dict(params=[p], grads=[p]), dict(params=[p], exp_avgs=[p]), dict(exp_avgs=[p], exp_avg_sqs=[p]),
                 dict(params=[p, p], grads=[z(40), z(40)], exp_avgs=[z(40), z(40)], exp_avg_sqs=[z(40), z(40)]),
                 dict(params=[p], masters=[p])):
        with pytest.raises(S.Subm3dError):
            call(**over)
    g = z(40)
    call(params=[z(40), z(40)], grads=[g, g], exp_avgs=[z(40), z(40)], exp_avg_sqs=[z(40), z(40)])  # read twice: fine
    with pytest.raises(ValueError):
        S.AdamW([torch.nn.Parameter(z(3))], state_bits=16)
    with pytest.raises(ValueError):
        S.AdamW([torch.nn.Parameter(z(3))], betas=(0.9, 1.0))
