"""The training operators where their parts meet: a saved and resumed optimizer, a block
with and without recorded gradients, and calls at the edges of what the documents allow."""
import copy
import io

import pytest
import torch

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
