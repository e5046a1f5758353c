"""What the training operators' Python layer decides before any kernel runs.  CPU only."""
import copy
import io

import pytest
import torch


@pytest.fixture(scope="module")
def S():
    from sparse_voxel_conv_b200 import build
    build.build()
    import sparse_voxel_conv_b200 as S
    return S


def _through_file(obj):
    f = io.BytesIO()
    torch.save(obj, f)
    f.seek(0)
    return torch.load(f, weights_only=False)


def _seeds_of(opt, monkeypatch):
    """The seeds of the calls that one step() makes."""
    import sparse_voxel_conv_b200.optim as optim
    seeds = []
    monkeypatch.setattr(optim, "adamw_step", lambda *a, seed, **k: seeds.append(seed & 0xFFFFFFFF))
    for group in opt.param_groups:
        for p in group["params"]:
            p.grad = torch.ones_like(p)
    opt.step()
    return seeds


@pytest.mark.parametrize("bits", [32, 8])
def test_optimizer_keeps_its_seed(S, bits, monkeypatch):
    """Copied, saved whole, or loaded into an optimizer that was made with another seed, the
    optimizer goes on with the stream of rounding bits that it had."""
    make = lambda **k: S.AdamW([dict(params=[torch.nn.Parameter(torch.ones(40))]),  # noqa: E731
                                dict(params=[torch.nn.Parameter(torch.ones(7))], lr=1e-4)], state_bits=bits, **k)
    want = [5, 5 + 0x632BE5A7]
    opt = make(seed=5)
    assert opt.seed == 5 and _seeds_of(opt, monkeypatch) == want
    for other in (copy.deepcopy(opt), _through_file(opt)):
        assert other.seed == 5 and _seeds_of(other, monkeypatch) == want
        assert other.state[other.param_groups[0]["params"][0]]["step"] == 2
    resumed = make()
    assert resumed.seed == 0 and _seeds_of(resumed, monkeypatch) == [0, 0x632BE5A7]
    resumed.load_state_dict(opt.state_dict())
    assert resumed.seed == 5 and _seeds_of(resumed, monkeypatch) == want
    # a group that joins later takes part in the same stream
    resumed.add_param_group(dict(params=[torch.nn.Parameter(torch.ones(3))]))
    assert _seeds_of(resumed, monkeypatch) == want + [(5 + 2 * 0x632BE5A7) & 0xFFFFFFFF]
    # a state that was saved without a seed: the constructor's
    old = opt.state_dict()
    for group in old["param_groups"]:
        group.pop("seed", None)
    later = make(seed=9)
    later.load_state_dict(old)
    assert later.seed == 9 and _seeds_of(later, monkeypatch)[0] == 9
    later.seed = 11
    assert _seeds_of(later, monkeypatch)[0] == 11


def test_stride_of_a_single_row(S):
    """A single row's stride says nothing: it is the row's own width to the library."""
    from sparse_voxel_conv_b200.norm import _rows
    buf = torch.zeros(4, 131)
    for x in (buf[:1, :64], buf[3:, 2:66], buf[1:2], buf[:0, :64]):
        t, stride = _rows(x, "x")
        assert t is x and (stride == x.shape[1] or not len(x))
    for x in (buf[:2, :64], buf[1:, 2:66]):
        t, stride = _rows(x, "x")
        assert t is x and stride == 131


def test_tangents_are_refused(S):
    """Forward-mode tangents, which no kernel carries on, are not dropped without a word."""
    from torch.autograd import forward_ad
    x, w, b = torch.randn(4, 16), torch.ones(16), torch.zeros(16)
    pos, where = torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4, 3)
    with forward_ad.dual_level():
        dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
        for call in (lambda: S.layer_norm(dual(x)), lambda: S.layer_norm(x, dual(w), b),
                     lambda: S.layer_norm(x, w, dual(b)), lambda: S.LayerNorm(16)(dual(x)),
                     lambda: S.rotary(dual(x), pos), lambda: S.rotary(x, dual(where))):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call()
            with torch.no_grad(), pytest.raises(NotImplementedError, match="forward-mode"):
                call()
        for call in (lambda: S.layer_norm(x, w, b), lambda: S.rotary(x, pos)):  # nothing to drop
            with pytest.raises(ValueError, match="CUDA"):
                call()
    for f in (lambda t: S.layer_norm(t, w, b), lambda t: S.rotary(t, pos)):
        with pytest.raises(NotImplementedError, match="forward-mode"):
            torch.func.jvp(f, (x,), (torch.ones_like(x),))


def test_recorded_outputs_are_refused(S):
    """out= may not be a tensor of a recorded graph, whose gradient would go on as if nothing
    had been written; without recording it may."""
    x, pos = torch.randn(4, 16), torch.zeros(4, 3, dtype=torch.int32)
    leaf = torch.zeros(4, 16, requires_grad=True)
    for out in (leaf, leaf * 1):
        for call in (lambda: S.layer_norm(x, out=out), lambda: S.layer_norm_forward(x, out=out),
                     lambda: S.rotary(x, pos, out=out)):
            with pytest.raises(ValueError, match="recorded"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):      # as far as the CPU goes
                call()


def test_positions_have_no_gradient(S):
    """Positions that ask for a gradient are refused where one would be recorded."""
    x, where = torch.randn(4, 16), torch.zeros(4, 3, requires_grad=True)
    for t in (x, x.clone().requires_grad_(True)):
        with pytest.raises(ValueError, match="positions have no gradient"):
            S.rotary(t, where)
        for quiet in (where.detach(), where):
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):      # as far as the CPU goes
                S.rotary(t, quiet)


def test_block_that_was_saved_whole_before_it_had_norms(S):
    """A SubMResBlock3d object from a file that knows no norms runs as the block without them."""
    block = S.SubMResBlock3d(16, dtype=torch.float32)
    old = copy.deepcopy(block)
    del old.__dict__["norm1"]
    x = S.SparseTensor(torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, 16), 4)
    for b in (block, old, _through_file(old)):
        with pytest.raises(ValueError, match="CUDA"):       # as far as the CPU goes
            b(x)
