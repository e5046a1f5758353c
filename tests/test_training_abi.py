"""The training operators' entry points refuse bad arguments on the host, and the
binding refuses host tensors.  CPU only: no call here reaches a kernel."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def abi():
    from sparse_voxel_conv_b200 import build
    build.build()
    from sparse_voxel_conv_b200 import _abi
    return _abi


A = 1 << 20     # 256-byte aligned fake addresses, far apart; never dereferenced on these paths


def at(i):
    return A + (i << 32)


NORM = ["x", "n", "channels", "x_stride", "dtype", "weight", "bias", "affine_dtype", "eps", "act", "y", "mean", "rstd",
        "stream"]
NORM_OK = dict(x=at(0), n=10, channels=64, x_stride=64, dtype=1, weight=at(1), bias=at(2), affine_dtype=0, eps=1e-5,
               act=0, y=at(3), mean=at(4), rstd=at(5), stream=None)


def test_layer_norm(abi):
    f = lambda **o: abi.lib.subm3d_layer_norm(*[{**NORM_OK, **o}[k] for k in NORM])  # noqa: E731
    bad = abi.SUBM3D_E_INVALID
    for over in (dict(n=-1), dict(channels=0), dict(x_stride=63), dict(dtype=2), dict(act=7), dict(affine_dtype=5),
                 dict(dtype=0, affine_dtype=1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                 dict(mean=None), dict(rstd=None), dict(x=None), dict(y=None), dict(x=at(0) + 1), dict(y=at(3) + 1),
                 dict(weight=at(1) + 2), dict(mean=at(4) + 2), dict(y=at(0) + 2), dict(y=at(0), x_stride=72),
                 dict(y=at(1)), dict(mean=at(3)), dict(mean=at(5) + 4), dict(y=at(0) - 2)):
        assert f(**over) == bad, over
    assert f(channels=(1 << 24) + 1, x_stride=1 << 25) == abi.SUBM3D_E_UNSUPPORTED
    assert f(n=1 << 40, x_stride=1 << 20) == abi.SUBM3D_E_UNSUPPORTED
    assert f(n=0) == abi.SUBM3D_OK and f(n=0, x=None, y=None) == abi.SUBM3D_OK


GRAD = ["dy", "dy_stride", "x", "x_stride", "n", "channels", "dtype", "mean", "rstd", "weight", "bias", "affine_dtype",
        "act", "dx", "dweight", "dbias", "workspace", "workspace_bytes", "stream"]


def test_layer_norm_backward(abi):
    ws = abi.subm3d_layer_norm_workspace_bytes(100_000, 64)
    assert ws >= 2 * 2 * 64 * 4
    assert abi.subm3d_layer_norm_workspace_bytes(10, 64) == 0       # one block needs none
    assert abi.subm3d_layer_norm_workspace_bytes(100, 1 << 24) >= 2 * 2 * 4 << 24
    assert abi.subm3d_layer_norm_workspace_bytes(-1, 64) == 0 and abi.subm3d_layer_norm_workspace_bytes(10, 0) == 0
    assert abi.subm3d_layer_norm_workspace_bytes(0, 64) == 0
    ok = dict(dy=at(0), dy_stride=64, x=at(1), x_stride=64, n=100_000, channels=64, dtype=1, mean=at(2), rstd=at(3),
              weight=at(4), bias=at(5), affine_dtype=0, act=0, dx=at(6), dweight=at(7), dbias=at(8), workspace=at(9),
              workspace_bytes=ws, stream=None)
    f = lambda **o: abi.lib.subm3d_layer_norm_backward(*[{**ok, **o}[k] for k in GRAD])  # noqa: E731
    for over in (dict(n=-1), dict(channels=0), dict(x_stride=63), dict(dy_stride=10), dict(dtype=3), dict(act=-1),
                 dict(dtype=0, affine_dtype=1), dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None),
                 dict(workspace=None), dict(workspace_bytes=ws - 1), dict(workspace=at(9) + 8), dict(dx=at(0)),
                 dict(dx=at(1)), dict(dweight=at(8)), dict(dweight=at(9)), dict(dx=at(6) + 1), dict(dbias=at(8) + 2),
                 dict(dweight=at(4)), dict(dx=at(2) - 8)):
        assert f(**over) == abi.SUBM3D_E_INVALID, over
    assert f(channels=(1 << 24) + 1, x_stride=1 << 25, dy_stride=1 << 25) == abi.SUBM3D_E_UNSUPPORTED
    assert f(dx=None, dweight=None, dbias=None) == abi.SUBM3D_OK        # nothing is wanted


ROT = ["x", "x_row", "x_head", "n", "heads", "head_dim", "dtype", "positions", "positions_f32", "pos_stride", "axes",
       "axis_pairs", "theta", "halves", "inverse", "y", "y_row", "y_head", "stream"]


def test_rotary(abi):
    pairs = lambda *p: (ctypes.c_int32 * len(p))(*p)  # noqa: E731
    ok = dict(x=at(0), x_row=128, x_head=64, n=10, heads=2, head_dim=64, dtype=1, positions=at(1), positions_f32=0,
              pos_stride=4, axes=3, axis_pairs=pairs(10, 10, 10), theta=1e4, halves=0, inverse=0, y=at(2), y_row=128,
              y_head=64, stream=None)
    f = lambda **o: abi.lib.subm3d_rotary(*[{**ok, **o}[k] for k in ROT])  # noqa: E731
    for over in (dict(n=-1), dict(heads=-1), dict(head_dim=0), dict(dtype=9), dict(axes=0), dict(axes=5),
                 dict(axis_pairs=None), dict(axis_pairs=pairs(20, 10, 3)), dict(axis_pairs=pairs(-1, 1, 1)),
                 dict(axis_pairs=pairs(2 ** 31 - 1, 2 ** 31 - 1, 4)), dict(theta=0.0), dict(theta=-1.0),
                 dict(theta=float("nan")), dict(theta=float("inf")), dict(x=None), dict(y=None), dict(positions=None),
                 dict(x=at(0) + 1), dict(y=at(2) + 1), dict(positions=at(1) + 2), dict(x_row=-1), dict(pos_stride=-4),
                 dict(y_row=127), dict(y_head=63), dict(y_row=0), dict(y=at(0) + 128), dict(y=at(0), y_row=192),
                 dict(y=at(1))):
        assert f(**over) == abi.SUBM3D_E_INVALID, over
    assert f(head_dim=63) == abi.SUBM3D_E_UNSUPPORTED and f(head_dim=514) == abi.SUBM3D_E_UNSUPPORTED
    assert f(x_row=1 << 45) == abi.SUBM3D_E_UNSUPPORTED
    assert f(n=0) == abi.SUBM3D_OK and f(heads=0) == abi.SUBM3D_OK


def test_adamw(abi):
    T, C = abi.AdamWTensor, abi.AdamWStep

    def f(step=None, count=2, **over):
        c = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1, param_dtype=0, grad_dtype=0,
                 state_bits=8, seed=0)
        c.update(step or {})
        ts = (T * 2)()
        for i in range(2):
            d = dict(param=at(10 * i), grad=at(10 * i + 1), exp_avg=at(10 * i + 2), exp_avg_sq=at(10 * i + 3),
                     exp_avg_scale=at(10 * i + 4), exp_avg_sq_scale=at(10 * i + 5), master=at(10 * i + 6), n=100)
            if i == 1:
                d.update(over)
            for k, v in d.items():
                setattr(ts[i], k, v)
        return abi.lib.subm3d_adamw(ts, count, ctypes.byref(C(**c)), None)

    bad = abi.SUBM3D_E_INVALID
    for step in (dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(eps=-1.0),
                 dict(weight_decay=-1.0), dict(step=0), dict(param_dtype=2), dict(grad_dtype=-1), dict(state_bits=16),
                 dict(step_device=A + 2), dict(lr_device=A + 1), dict(beta2=float("nan")), dict(step_device=at(10))):
        assert f(step) == bad, step
    for over in (dict(n=-1), dict(param=None), dict(grad=None), dict(exp_avg=None), dict(exp_avg_sq=None),
                 dict(exp_avg_scale=None), dict(exp_avg_sq_scale=None), dict(param=at(10) + 2), dict(grad=at(11) + 1),
                 dict(master=at(16) + 2), dict(param=at(0) + 396), dict(grad=at(0)), dict(exp_avg=at(10)),
                 dict(exp_avg_scale=at(12) + 96), dict(exp_avg_sq_scale=at(14) + 3), dict(master=at(6) - 396),
                 dict(exp_avg=at(2) + 99)):
        assert f(**over) == bad, over
    assert f(n=(1 << 40) + 1) == abi.SUBM3D_E_UNSUPPORTED
    assert f(count=-1) == bad and abi.lib.subm3d_adamw(None, 1, ctypes.byref(C()), None) == bad
    assert f(count=0) == abi.SUBM3D_OK


def test_host_tensors_are_refused(abi):
    import sparse_voxel_conv_b200 as S
    x = torch.zeros(4, 16)
    for call in (lambda: S.layer_norm(x), lambda: S.layer_norm_forward(x),
                 lambda: S.layer_norm_backward(x, x, torch.zeros(4), torch.zeros(4)),
                 lambda: S.rotary(x, torch.zeros(4, 3, dtype=torch.int32)),
                 lambda: S.adamw_step([x], [x], [x], [x], 1), lambda: S.LayerNorm(16)(x),
                 lambda: S.VoxelRotary(16)(S.SparseTensor(torch.zeros(4, 4, dtype=torch.int32), x, 4))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    p = torch.nn.Parameter(x)
    p.grad = x.clone()
    with pytest.raises(ValueError, match="CUDA"):
        S.AdamW([p]).step()
