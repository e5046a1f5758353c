"""The training operators together, as a block's step uses them: layer norm ->
activation -> convolution twice with a skip, rotary positions on the result, the
gradients of all of it, and the AdamW step; eager and as a captured graph."""
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


def _conv64(x, w, nbr):
    """The convolution in 64 bits through the neighbour rows."""
    pad = torch.cat([x, x.new_zeros(1, x.shape[1])])
    rows = pad[nbr.long()]                      # -1: the row of zeros
    return torch.einsum("nkc,okc->no", rows, w.reshape(w.shape[0], 27, -1))


def _norm64(x, w, b, act):
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    return R.act((x - mean) / (var + 1e-5).sqrt() * w + b, act)


def _block(S, c, dtype, seed):
    torch.manual_seed(seed)
    block = S.SubMResBlock3d(c, act="silu", dtype=dtype, device="cuda", norm=True)
    for n in (block.norm1, block.norm2):
        n.weight.copy_(1 + 0.2 * torch.randn(c))
        n.bias.copy_(0.2 * torch.randn(c))
    for p in block.parameters():
        p.requires_grad_(True)
    return block


def test_block_gradients_and_step(S):
    """fp32 on the tiny set: loss, all gradients and the weights after one step against 64
    bits.  The chain is some 27 C + C wide sums in fp32 (the convolution's own bar is 1e-5
    of its scale); three of them in a row stay within 1e-4 of each gradient's scale."""
    c = 16
    coords = torch.from_numpy(WL.tiny_coords()).cuda()
    n = coords.shape[0]
    block = _block(S, c, F32, 0)
    turn = S.VoxelRotary(8)
    x = torch.randn(n, c, device="cuda", requires_grad=True)
    r = torch.randn(n, c, device="cuda")
    opt = S.AdamW(block.parameters(), lr=1e-2, weight_decay=0.1)
    before = {k: p.detach().double() for k, p in block.named_parameters()}
    st = S.SparseTensor(coords, x, 16)
    out = turn(block(st))
    (out.feats * r).sum().backward()

    nbr = st.get_map("subm0").nbr
    ref = {k: v.clone().requires_grad_(True) for k, v in before.items()}
    x64 = x.detach().double().requires_grad_(True)
    h = _conv64(_norm64(x64, ref["norm1.weight"], ref["norm1.bias"], "silu"), ref["conv1.weight"], nbr)
    h = _conv64(_norm64(h, ref["norm2.weight"], ref["norm2.bias"], "silu"), ref["conv2.weight"], nbr) + x64
    y64 = R.rotary(h.view(n, 2, 8), coords[:, 1:], 10000.0, (1, 1, 1), True, False)[0].reshape(n, c)
    (y64 * r.double()).sum().backward()

    def close(got, want, what):
        bar = 1e-4 * (want.abs() + want.square().mean().sqrt())
        R.check(got, want, bar, what)

    close(out.feats.detach(), y64.detach(), "output")
    close(x.grad, x64.grad, "x")
    grads = {}
    for k, p in block.named_parameters():
        close(p.grad, ref[k].grad, k)
        grads[k] = p.grad.clone()
    opt.step()
    for k, p in block.named_parameters():
        want, _, _ = R.adamw(before[k], grads[k], torch.zeros_like(before[k]), torch.zeros_like(before[k]), 1, 1e-2,
                             (0.9, 0.999), 1e-8, 0.1)
        R.check(p.detach(), want, 16 * R.U * 1e-2 + 4 * R.U * want.abs(), k)


def test_block_without_gradients(S):
    """Inference fuses the skip add; it equals the recorded form up to the second rounding of
    bf16 (half a step of conv2's output)."""
    coords = torch.from_numpy(WL.make_workload("shell").coords).cuda()
    block = _block(S, 64, BF, 1)
    x = torch.randn(coords.shape[0], 64, device="cuda").to(BF)
    st = S.SparseTensor(coords, x, 64)
    y = block(st).feats.detach()
    with torch.no_grad():
        z = block(st).feats
    step = 2.0 ** -8
    bound = step * (y.double() - x.double()).abs() + 2 * step * y.double().abs() + 1e-6
    R.check(z, y.double(), bound)
    plain = S.SubMResBlock3d(64, device="cuda")         # the block as it was
    assert plain.norm1 is None and plain.conv1.bias is not None
    assert set(dict(plain.named_parameters())) == {"conv1.weight", "conv1.bias", "conv2.weight", "conv2.bias"}


@pytest.mark.parametrize("bits", [32, 8])
def test_training_runs(S, bits):
    """A few steps in bf16 with masters: the moments exist, the weights move and stay finite."""
    coords = torch.from_numpy(WL.make_workload("shell").coords).cuda()
    block = _block(S, 64, BF, 2)
    convs = [block.conv1.weight, block.conv2.weight]
    norms = [p for k, p in block.named_parameters() if "norm" in k]
    opt = S.AdamW([dict(params=convs, master_weights=True, state_bits=bits), dict(params=norms, weight_decay=0.0)])
    x = torch.randn(coords.shape[0], 64, device="cuda").to(BF)
    target = torch.randn_like(x)
    cache = {}
    before = [p.detach().clone() for p in block.parameters()]
    for _ in range(4):
        opt.zero_grad()
        y = block(S.SparseTensor(coords, x, 64, cache=cache))
        (y.feats.float() - target.float()).square().mean().backward()
        opt.step()
    for p, q in zip(block.parameters(), before):
        assert torch.isfinite(p).all() and not torch.equal(p, q)
    assert opt.state[convs[0]]["step"] == 4


def test_captured_step(S):
    """One graph of norm forward and backward, rotary there and back, and a step with a device
    step number, replayed three times: the bits of three eager rounds.  Two graphs that hold
    the same calls do not disturb each other."""
    n, c = 3001, 96
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    mk = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, dy = mk(n, c).to(BF), mk(n, c).to(BF)
    pos = torch.randint(0, 99, (n, 3), device="cuda", generator=g, dtype=torch.int32)

    def fresh():
        w = [1 + 0.1 * torch.arange(c, device="cuda") / c, 0.1 * torch.arange(c, device="cuda") / c]
        m = [torch.zeros(c, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(4)]
        s = [torch.zeros(3, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu) for _ in range(4)]
        return dict(w=w, m=m[:2], v=m[2:], ms=s[:2], vs=s[2:], t=torch.zeros(1, dtype=torch.int32, device="cuda"),
                    y=torch.empty_like(x), dx=torch.empty_like(x))

    def once(st):
        y, mean, rstd = S.layer_norm_forward(x, st["w"][0], st["w"][1], act="silu")
        st["y"].copy_(S.rotary(y.view(n, 6, 16), pos).view(n, c))
        back = S.rotary(dy.view(n, 6, 16), pos, inverse=True).view(n, c)
        dx, dw, db = S.layer_norm_backward(back, x, mean, rstd, st["w"][0], st["w"][1], act="silu")
        st["dx"].copy_(dx)
        st["t"].add_(1)
        S.adamw_step(st["w"], [dw, db], st["m"], st["v"], st["t"], lr=1e-2, exp_avg_scales=st["ms"],
                     exp_avg_sq_scales=st["vs"], seed=4)

    def all_of(st):
        out = [st["y"].clone(), st["dx"].clone(), *[w.clone() for w in st["w"]]]
        return out + [q.view(torch.uint8).clone() for k in ("m", "v", "ms", "vs") for q in st[k]]

    eager = fresh()
    for _ in range(3):
        once(eager)
    want = all_of(eager)

    side = torch.cuda.Stream()
    states = [fresh(), fresh()]
    graphs = []
    for st in states:
        warm = fresh()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            once(warm)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            once(st)
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for st in states:
        for p, q in zip(all_of(st), want):
            assert torch.equal(p, q)

    opt = S.AdamW([torch.nn.Parameter(torch.ones(8, device="cuda"))])
    opt.param_groups[0]["params"][0].grad = torch.ones(8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="frozen"):
        with torch.cuda.graph(graph):
            opt.step()


def test_two_threads(S):
    """Calls from two host threads on two streams: the bits of calls one after another."""
    import threading
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    data = [torch.randn(20_000 + 13 * k, 128, device="cuda", generator=g).to(BF) for k in range(2)]
    w, b = torch.rand(128, device="cuda"), torch.rand(128, device="cuda")
    pos = [torch.randint(0, 64, (d.shape[0], 3), device="cuda", dtype=torch.int32) for d in data]

    def work(k):
        y, mean, rstd = S.layer_norm_forward(data[k], w, b, act="gelu")
        grads = S.layer_norm_backward(data[k], data[k], mean, rstd, w, b, act="gelu")
        return y, *grads, S.rotary(y.view(-1, 2, 64), pos[k])

    want = [work(0), work(1)]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def run(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[k] = work(k)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(k,)) for k in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    for p, q in zip(got, want):
        assert all(torch.equal(s, t) for s, t in zip(p, q))


def test_first_call_is_a_captured_one():
    """A fresh process whose first calls of the library are captured ones (kernels are loaded,
    and given their shared memory, inside the capture)."""
    import subprocess
    import sys

    code = """
import torch, sparse_voxel_conv_b200 as S
x = torch.randn(300, 128, device='cuda').bfloat16()
w, b = torch.ones(128, device='cuda'), torch.zeros(128, device='cuda')
pos = torch.zeros(300, 3, dtype=torch.int32, device='cuda')
m, v, g = (torch.zeros(128, device='cuda') for _ in range(3))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y, mean, rstd = S.layer_norm_forward(x, w, b, act='silu')
    grads = S.layer_norm_backward(y, x, mean, rstd, w, b, act='silu')
    z = S.rotary(y.view(300, 2, 64), pos)
    S.adamw_step([w], [g], [m], [v], 1, lr=0.0)
graph.replay()
torch.cuda.synchronize()
want, m1, r1 = S.layer_norm_forward(x, w, b, act='silu')
assert torch.equal(y, want) and torch.equal(z.view(300, 128), y)
assert all(torch.equal(p, q) for p, q in zip(grads, S.layer_norm_backward(y, x, m1, r1, w, b, act='silu')))
"""
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout + p.stderr


def test_without_autograd_modes(S):
    """Under inference_mode and no_grad, with out= and in place."""
    x = torch.randn(100, 64, device="cuda")
    pos = torch.randint(0, 9, (100, 3), device="cuda", dtype=torch.int32)
    want, turned = S.layer_norm(x), S.rotary(x, pos)
    for mode in (torch.inference_mode, torch.no_grad):
        with mode():
            p = x.clone()
            assert torch.equal(S.layer_norm(p, out=p), want) and torch.equal(p, want)
            q = x.clone()
            assert torch.equal(S.rotary(q, pos, out=q), turned)
            w, g, m, v = (torch.ones(8, device="cuda") for _ in range(4))
            S.adamw_step([w], [g], [m], [v], 1)
            assert torch.isfinite(w).all()


def test_gradients_that_are_not_contiguous(S):
    """The optimizer takes a gradient of any layout."""
    a, b = (torch.nn.Parameter(torch.ones(6, 8, device="cuda")) for _ in range(2))
    g = torch.randn(8, 6, device="cuda")
    a.grad, b.grad = g.t(), g.t().contiguous()
    S.AdamW([a]).step()
    S.AdamW([b]).step()
    assert torch.equal(a, b)


def test_another_current_device(S, monkeypatch):
    """Tensors of a device that is not the current one: the call is made again with theirs
    current (here told by a first answer that names another one)."""
    import sparse_voxel_conv_b200.norm as norm
    import sparse_voxel_conv_b200.optim as optim
    import sparse_voxel_conv_b200.positions as positions

    x, dy = torch.randn(50, 64, device="cuda"), torch.randn(50, 64, device="cuda")
    w, b = torch.rand(64, device="cuda"), torch.rand(64, device="cuda")
    pos = torch.randint(0, 9, (50, 3), device="cuda", dtype=torch.int32)

    def calls():
        y, mean, rstd = S.layer_norm_forward(x, w, b, act="silu")
        out = [y, *S.layer_norm_backward(dy, x, mean, rstd, w, b, act="silu"), S.layer_norm(x, w, b), S.rotary(x, pos)]
        p, g, m, v = (torch.ones(40, device="cuda") for _ in range(4))
        S.adamw_step([p], [g], [m], [v], 2)
        return out + [p, m, v]

    want = calls()
    asked = []
    for module in (norm, optim, positions):
        real = module._current_device

        def first_another(real=real):
            asked.append(None)
            return 99 if len(asked) % 2 else real()

        monkeypatch.setattr(module, "_current_device", first_another)
    got = calls()
    assert len(asked) == 10 and all(torch.equal(p, q) for p, q in zip(got, want))
