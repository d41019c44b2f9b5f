"""Rotary positions without a GPU: refusals of the entry points, the table, and the references by their definitions."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import local_linear_attention_flashlla_gb300 as lla
from local_linear_attention_flashlla_gb300 import build as lla_build
from oracle.cache_ref import frequencies, rotary_backward_ref, rotary_ref, turn_angles
from oracle.lla_ref import lla_grad_ref, lla_ref


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(lla.library_path()):
        lla_build.build()
    return lla.load_library()


def _call(lib, backward=False, **kw):
    a = dict(dtype=0, dy_dtype=0, count=1, B=1, n=4, d=64, pos=64, ps=0, turns=128, rot=64, il=0, m=1.0, eps=-1.0, cu=None,
             shift=None, S=0, ws=None, wsb=0, x=256, dy=512, out=1024, gain=None, dgain=None, xs=(0, 64, 256), ys=(0, 64, 256),
             os=(0, 64, 256), heads=4, rows=True)
    a.update(kw)
    rows = (lla.lla_rotary_rows * max(a["count"], 1))()
    for r in rows:
        r.x, r.dy, r.out, r.gain, r.dgain, r.heads = a["x"], a["dy"], a["out"], a["gain"], a["dgain"], a["heads"]
        r.x_stride[:], r.dy_stride[:], r.out_stride[:] = a["xs"], a["ys"], a["os"]
    rows = rows if a["rows"] else ctypes.POINTER(lla.lla_rotary_rows)()
    common = (rows, a["count"], a["B"], a["n"], a["d"], a["pos"], a["ps"], a["turns"], a["rot"], a["il"], a["m"], a["eps"], a["cu"],
              a["shift"], a["S"])
    if backward:
        return lib.lla_rotary_backward(a["dtype"], a["dy_dtype"], *common, a["ws"], a["wsb"], None)
    return lib.lla_rotary(a["dtype"], *common, None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(rows=False), dict(pos=None), dict(turns=None), dict(count=0), dict(count=5), dict(d=48), dict(d=256), dict(B=0),
    dict(n=0), dict(B=1 << 16, n=1 << 16), dict(rot=0), dict(rot=63), dict(rot=66), dict(m=0.0), dict(m=float("nan")),
    dict(m=float("inf")), dict(eps=float("nan")), dict(eps=float("inf")), dict(ps=3), dict(pos=66), dict(turns=132), dict(cu=64),
    dict(shift=64, S=1), dict(cu=64, shift=64, S=0), dict(cu=64, shift=64, S=1, B=2), dict(cu=66, shift=64, S=1), dict(out=None),
    dict(x=None, eps=1e-6), dict(x=264, eps=1e-6), dict(out=1032), dict(heads=0), dict(heads=70000), dict(os=(0, 60, 256)),
    dict(xs=(0, 64, 254), eps=0.0), dict(gain=128), dict(gain=130, eps=1e-6),
])
def test_refusals(lib, backward, bad):
    assert _call(lib, backward, **bad) == lla.LLA_ERR_INVALID_ARG
    assert lib.lla_last_error().decode()


@pytest.mark.parametrize("bad", [dict(dy=None), dict(dy=520), dict(ys=(0, 64, 252)), dict(dtype=1, dy_dtype=0), dict(dy_dtype=3),
                                 dict(dgain=128), dict(eps=1e-6, dgain=128, ws=256, wsb=16), dict(eps=1e-6, dgain=128, ws=264, wsb=1 << 30)])
def test_backward_refusals(lib, bad):
    assert _call(lib, True, **bad) == lla.LLA_ERR_INVALID_ARG
    assert lib.lla_last_error().decode()


def test_workspace_size(lib):
    assert lib.lla_rotary_backward_workspace_size(2, 128) == 2 * lib.lla_rotary_backward_workspace_size(1, 128) > 0
    assert lib.lla_rotary_backward_workspace_size(0, 128) == lib.lla_rotary_backward_workspace_size(5, 128) == 0
    assert lib.lla_rotary_backward_workspace_size(1, 100) == 0


@pytest.mark.parametrize("bad", [dict(dim=0), dict(dim=7), dict(dim=8, base=0.0), dict(dim=8, base=math.inf), dict(dim=8, factor=0.0),
                                 dict(dim=8, scaling="other"), dict(dim=8, scaling="parts", low=4.0, high=4.0),
                                 dict(dim=8, scaling="parts", original=0)])
def test_table_refusals(bad):
    with pytest.raises(lla.LLAError):
        lla.rotary_table(**bad, device="cpu")


@pytest.mark.parametrize("scaling", [None, "linear", "ntk", "parts"])
@pytest.mark.parametrize("dim,base,factor", [(2, 10000.0, 2.0), (24, 500.0, 4.0), (128, 10000.0, 16.0), (64, 1e6, 1.0)])
def test_table_holds_the_frequencies(scaling, dim, base, factor):
    """Turns per position, in units of 2^-64: within the reference's float64 roundings (a few 2^-53 of the frequency, times
    ln(base^..) <= 14 for the power's), and half a unit."""
    t = lla.rotary_table(dim, base, scaling=scaling, factor=factor, device="cpu")
    f, m = frequencies(dim, base, scaling, factor)
    assert t.dim == dim and math.isclose(t.magnitude, m, rel_tol=1e-15)
    got = np.array([x / 2.0 ** 64 * 2 * np.pi for x in t.turns.tolist()])
    assert (np.abs(got - f) <= 64 * 2.0 ** -53 * f + 2.0 ** -62).all()


def test_table_is_exact_to_the_last_bit():
    """A power of two whose frequencies are rational: 2^(-i) radians a position."""
    t = lla.rotary_table(16, 2.0 ** 8, device="cpu")
    two_pi = 2 * Fraction(3141592653589793238462643383279502884197, 10 ** 39)
    for i, x in enumerate(t.turns.tolist()):
        assert abs(Fraction(x) - Fraction(1, 2 ** i) / two_pi * 2 ** 64) <= Fraction(51, 100)
    assert lla.rotary_table(8, magnitude=0.5, device="cpu").magnitude == 0.5


def test_angles_of_far_positions():
    turns = [1 << 62, 3, -(1 << 61)]
    a = turn_angles([0, 1, 2 ** 31 - 1, -5], turns)
    assert np.allclose(a[:, 0], [0, np.pi / 2, -np.pi / 2, -np.pi / 2])
    assert np.allclose(a[2, 1], 2 * np.pi * 3 * (2 ** 31 - 1) / 2.0 ** 64)
    assert np.allclose(a[:, 2], [0, -np.pi / 4, np.pi / 4, -3 * np.pi / 4])


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_by_its_definition(interleaved):
    """A rotation keeps lengths and relative positions; the gradient is that of central differences."""
    rng = np.random.default_rng(0)
    x, ang = rng.standard_normal((5, 3, 16)), rng.standard_normal((5, 1, 6))
    y = rotary_ref(x, ang, interleaved=interleaved)
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[..., 12:], x[..., 12:])
    same = rotary_ref(x, ang + 0.7, interleaved=interleaved)
    assert np.allclose(y @ y.transpose(0, 2, 1), same @ same.transpose(0, 2, 1))
    gain, dy, eps = 1 + 0.3 * rng.standard_normal(16), rng.standard_normal(x.shape), 1e-3
    f = lambda x, g: (dy * rotary_ref(x, ang, g, eps, interleaved, 1.3)).sum()  # noqa: E731
    dx, dgain = rotary_backward_ref(dy, x, ang, gain, eps, interleaved, 1.3)
    for at in [(0, 0, 0), (1, 2, 7), (4, 1, 15), (3, 0, 11)]:
        e = np.zeros_like(x)
        e[at] = 1e-5
        assert abs((f(x + e, gain) - f(x - e, gain)) / 2e-5 - dx[at]) < 1e-8
        e = np.zeros(16)
        e[at[2]] = 1e-5
        assert abs((f(x, gain + e) - f(x, gain - e)) / 2e-5 - dgain[at[2]]) < 1e-8


def test_binding_refuses_cpu_tensors_and_bad_calls():
    x, p, t = torch.zeros(4, 2, 16), torch.zeros(4, dtype=torch.int32), lla.rotary_table(16, device="cpu")
    for call in (lambda: lla.rotary(x, p, t), lambda: lla.rotary_backward(x, x, p, t), lambda: lla.rotary([x] * 5, p, t),
                 lambda: lla.rotary_backward(x, None, p, t, eps=1e-6), lambda: lla.rotary(x, p, t.turns)):
        with pytest.raises(lla.LLAError):
            call()


def test_marshalling_module_refuses_what_does_not_fit():
    """Without a GPU nothing fits (tensors lie on the CPU): every call says so, and leaves no error set."""
    m = lla._bind()
    if not m:
        pytest.skip("the marshalling module is not built here")
    x, p, t, g = torch.zeros(4, 2, 16), torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.int64), torch.ones(16)
    c, s, i = torch.zeros(2, 1, 8, 16), torch.zeros(2, 1, 8), torch.zeros(1, dtype=torch.int32)
    for dev in (0, -1):
        assert m.rotary(dev, x, p, t, 16, 1.0, g, 1e-6, False, None, None, x, 0) == -1
        assert m.rotary(dev, (x, x), p, t, 16, 1.0, None, None, False, None, None, (x,), 0) == -1
        assert m.rotary(dev, (), p, t, 16, 1.0, None, None, False, None, None, (), 0) == -1
        assert m.rotary_backward(dev, x, x, p, t, 16, 1.0, g, 1e-6, False, None, None, x, g, 0, 0, 0) == -1
        assert m.weigh(dev, x, x[:, :, 0], c, s, s, None, None, p[None], p, i, 1.0, 1, 1.0, 0, True, 0, 0, 0, None) == -1
        assert m.evict(dev, s, s, None, None, c, c, p[None], i, i, None, 0, 0, 0) == -1
        assert m.trim(dev, i, i, p[None], p, i, 16, None, i, i, i, 0) == -1
    assert m.rotary(0, None, p, t, 16, 1.0, None, None, False, None, None, x, 0) == -1
    assert m.rotary(0, x, p, t, 16, "one", None, None, False, None, None, x, 0) == -1
    assert m.weigh(0, x, x, c, s, s, None, None, p[None], p, i, "tau", 1, 1.0, 0, True, 0, 0, 0, None) == -1
    assert m.rotary(0) == m.rotary_backward() == m.weigh(1, 2) == m.evict() == m.trim(0) == -1
    with pytest.raises(TypeError):
        m.init_bounded(1)


def test_gradient_of_rotated_attention_by_differences():
    """The formulas of a training step (norm, rotation, attention and their gradients) against central differences in 64 bits:
    step 1e-5, so the third derivative's term is about 1e-10 and the rounding 1e-16 / 1e-5 of the loss; 1e-6 of it is asked for."""
    rng = np.random.default_rng(5)
    H, n, d, rot, tau, lam = 2, 9, 8, 6, 0.4, 0.1
    x, v, w = rng.standard_normal((2, 1, H, n, d)), rng.standard_normal((1, H, n, d)), rng.standard_normal((1, H, n, d))
    gain = 1 + 0.2 * rng.standard_normal((2, d))
    ang = np.arange(n)[:, None] * np.array([1.0, 0.3, 0.07])

    def loss(x, gain):
        q, k = (rotary_ref(x[i], ang, gain[i], 1e-6) for i in range(2))
        return (lla_ref(q, k, v, tau, lam)[0].reshape(w.shape) * w).sum()

    q, k = (rotary_ref(x[i], ang, gain[i], 1e-6) for i in range(2))
    back = [rotary_backward_ref(g, x[i], ang, gain[i], 1e-6) for i, g in enumerate(lla_grad_ref(q, k, v, w, tau, lam)[:2])]
    for _ in range(6):
        u, g = rng.standard_normal(x.shape), rng.standard_normal(gain.shape)
        step = 1e-5
        diff = (loss(x + step * u, gain + step * g) - loss(x - step * u, gain - step * g)) / (2 * step)
        own = sum((back[i][0] * u[i]).sum() + (back[i][1] * g[i]).sum() for i in range(2))
        assert abs(diff - own) <= 1e-6 * max(1.0, sum(np.abs(back[i][0] * u[i]).sum() for i in range(2)))
