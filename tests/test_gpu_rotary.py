"""Rotary positions on the GPU against float64, element by element.

With u = 2^-24 and a row's fp32 arithmetic: the normalised value carries (d / 2 + 2) u from the mean of squares, 4 u from the
reciprocal root and 3 u from products.  An angle, fixed-point, is off by 2^-32 turns at most; as an fp32 argument by u pi; its
sine and cosine by 4 u each, and 1 u from the magnitude; the two products and their sum by 3 u.  So an output is within
m (|a| + |b|) (d / 2 + 24) u of the pair's exact (a, b), and rounded once (2^-8 of itself in bf16, u in fp32).
Gradients: dx = rs (h - n mean(h n)), n the unit row, |n| <= sqrt(d): the first term errs as above with |g gain| in place of the
pair, the mean's d products and its sum add (d + 8) u mean|h n|, times |n|; all of it rs (2 d + 64) u (|h| + |n| mean|h n|).
A gain's gradient is a sum of R rows in fp32, in chains of at most `chain` (a lane's rows) and trees: (chain + 64 + d) u of the sum
of magnitudes; a chain is no longer than the rows themselves.
"""
import numpy as np
import pytest
import torch

import local_linear_attention_flashlla_gb300 as lla
from oracle.cache_ref import rotary_backward_ref, rotary_ref, turn_angles
from oracle.lla_ref import lla_grad_ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24


def half_step(dtype):
    return 2.0 ** -8 if dtype == "bf16" else U


def make(shape, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DT[dtype]).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def angles_of(positions, table, rows3):
    a = turn_angles(positions.cpu().numpy(), table.turns.tolist())
    return a[:, None] if rows3 else a[..., None, :, :] if a.ndim == 3 else a


def pair_sum(u, rot, interleaved):
    """|a| + |b| of every column's pair."""
    m = np.abs(u).copy()
    h = rot // 2
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, h), slice(h, rot))
    s = m[..., a] + m[..., b]
    m[..., a], m[..., b] = s, s
    return m


def check_forward(y, x, ang, table, dtype, gain, eps, interleaved):
    d = x.shape[-1]
    ref = rotary_ref(f64(x), ang, None if gain is None else f64(gain), eps, interleaved, table.magnitude)
    u = rotary_ref(f64(x), ang * 0, None if gain is None else f64(gain), eps, interleaved, 1.0)
    tol = half_step(dtype) * np.abs(ref) + max(abs(table.magnitude), 1) * pair_sum(u, table.dim, interleaved) * (d / 2 + 24) * U + 1e-37
    got = f64(y)
    assert y.dtype is x.dtype and y.shape == x.shape
    assert np.isfinite(got).all()
    worst = (np.abs(got - ref) / tol).max()
    assert worst <= 1.0, worst


def check_backward(dx, dgain, dy, x, ang, table, dtype, gain, eps, interleaved, chain=4096):
    ref, rg = rotary_backward_ref(f64(dy), None if x is None else f64(x), ang, None if gain is None else f64(gain), eps, interleaved,
                                  table.magnitude)
    d, m = dy.shape[-1], max(abs(table.magnitude), 1)
    g = m * pair_sum(f64(dy), table.dim, interleaved)
    if eps is None:
        tol = g * (d / 2 + 24) * U
    else:
        s = 1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + eps)
        n, h = np.abs(f64(x) * s), g * (1.0 if gain is None else np.abs(f64(gain)))
        tol = s * (2 * d + 64) * U * (h + n * (n * h).mean(-1, keepdims=True))
    got = f64(dx)
    assert np.isfinite(got).all()
    worst = (np.abs(got - ref) / (tol + half_step(dtype) * np.abs(ref) + 1e-37)).max()
    assert worst <= 1.0, worst
    if gain is None:
        assert dgain is None
        return
    mag = (g * n).reshape(-1, d).sum(0)
    rows = got.size // d
    worst = (np.abs(f64(dgain) - rg) / ((min(chain, rows) + 64 + 2 * d) * U * mag + 1e-37)).max()
    assert worst <= 1.0, worst


# tokens, heads of the tensors, head dim, rotary columns
SHAPES = [(1, (1,), 128, 128), (5, (4, 1), 128, 128), (33, (3, 2, 5), 64, 64), (7, (2, 1, 2, 1), 32, 32), (50, (5,), 16, 16), (9, (6, 3), 128, 64),
          (9, (6, 3), 128, 96), (12, (2, 1), 64, 2), (12, (2, 1), 64, 50), (3, (17,), 32, 12), (130, (1, 1), 16, 6), (2, (40, 8, 40), 128, 32)]


@pytest.mark.parametrize("T,heads,d,rot", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [None, "plain", "gain"])
def test_token_rows(lla_gpu, T, heads, d, rot, dtype, interleaved, norm):
    """Slices of one fused projection, in one launch, each as by itself; the gradient with dy of both types."""
    table = lla.rotary_table(rot, scaling="parts", factor=4.0, original=64)
    fused = make((T, (sum(heads) + 1) * d), dtype, T)
    xs = [t.reshape(T, h, d) for h, t in zip(heads, fused.split([h * d for h in heads] + [d], 1))]
    gains = [1 + 0.3 * make((d,), "fp32", 5 + i) for i in range(len(heads))] if norm == "gain" else None
    eps = None if norm is None else 1e-6
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 37 + 11
    ang = angles_of(pos, table, True)
    before = fused.clone()
    ys = lla.rotary(xs, pos, table, gain=gains, eps=eps, interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(fused, before) and isinstance(ys, tuple)
    for i, (x, y) in enumerate(zip(xs, ys)):
        gain = None if gains is None else gains[i]
        check_forward(y, x, ang, table, dtype, gain, eps, interleaved)
        assert torch.equal(y, lla.rotary(x, pos, table, gain=gain, eps=eps, interleaved=interleaved))
    for dy_dtype in {dtype, "fp32"}:
        dys = [make(x.shape, dy_dtype, 90 + i) for i, x in enumerate(xs)]
        dxs, dgains = lla.rotary_backward(dys, xs, pos, table, gain=gains, eps=eps, interleaved=interleaved)
        for i in range(len(xs)):
            check_backward(dxs[i], None if dgains is None else dgains[i], dys[i], xs[i], ang, table, dtype,
                           None if gains is None else gains[i], eps, interleaved)
            assert dxs[i].dtype is xs[i].dtype
    lla.lla_sync_status()


@pytest.mark.parametrize("B,H,n,d", [(2, 3, 70, 128), (3, 1, 1, 64), (1, 5, 129, 16), (2, 2, 31, 32)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("batched", [False, True])
def test_training_layout(lla_gpu, B, H, n, d, dtype, batched):
    table = lla.rotary_table(d)
    x, y2 = make((B, H, n, d), dtype), make((B, 2 * H, n, d), dtype, 4)[:, ::2]        # every second head of a larger tensor
    gains = [1 + 0.3 * make((d,), "fp32", 7), None]
    pos = torch.randint(0, 100000, (B, n) if batched else (n,), dtype=torch.int32, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    ang = angles_of(pos, table, False)
    out = lla.rotary((x, y2), pos, table, gain=gains, eps=1e-6)
    for i, t in enumerate((x, y2)):
        check_forward(out[i], t, ang, table, dtype, gains[i], 1e-6, False)
    dy = [make((B, H, n, d), "fp32", 11), make((B, H, n, d), "fp32", 12).transpose(2, 3).contiguous().transpose(2, 3)]
    dx, dg = lla.rotary_backward(dy, (x, y2), pos, table, gain=gains, eps=1e-6)
    assert dg[1] is None
    for i, t in enumerate((x, y2)):
        check_backward(dx[i], dg[i], dy[i], t, ang, table, dtype, gains[i], 1e-6, False)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [128, 30])
def test_far_and_negative_positions(lla_gpu, interleaved, rot):
    pos = torch.tensor([0, 1, -1, 4095, 131072, 2 ** 24 + 1, 2 ** 30 - 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    x, table = make((9, 2, 128), "fp32"), lla.rotary_table(rot, 500000.0)
    check_forward(lla.rotary(x, pos, table, interleaved=interleaved), x, angles_of(pos, table, True), table, "fp32", None, None, interleaved)


@pytest.mark.parametrize("S,T", [(1, 6), (3, 20), (64, 64), (200, 1000), (5000, 700)])
def test_shift_by_sequence(lla_gpu, S, T):
    """Positions moved by what was evicted; empty sequences, and padding rows behind the last sequence, which keep theirs."""
    rng = np.random.default_rng(S)
    cu = np.concatenate([[0], np.sort(rng.integers(0, T - 1, S))])
    shift = rng.integers(0, 10 ** 6, S)
    pos = rng.integers(0, 4000, T)
    moved = pos.copy()
    for s in range(S):
        moved[cu[s]:cu[s + 1]] += shift[s]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    x, table = make((T, 2, 64), "bf16"), lla.rotary_table(64)
    got = lla.rotary(x, i32(pos), table, cu_q=i32(cu), shift=i32(shift))
    assert torch.equal(got, lla.rotary(x, i32(moved), table))
    dy = make((T, 2, 64), "bf16", 9)
    assert torch.equal(lla.rotary_backward(dy, x, i32(pos), table, cu_q=i32(cu), shift=i32(shift))[0],
                       lla.rotary_backward(dy, None, i32(moved), table)[0])


@pytest.mark.parametrize("dtype,rot,interleaved", [("bf16", 128, False), ("bf16", 20, False), ("fp32", 128, True), ("fp32", 10, False)])
def test_in_place(lla_gpu, dtype, rot, interleaved):
    T, d = 300, 128
    fused = make((T, 7, d), dtype)
    x, pos, table = fused[:, 1:5], torch.arange(T, dtype=torch.int32, device="cuda"), lla.rotary_table(rot)
    gain = 1 + 0.3 * make((d,), "fp32", 3)
    want = lla.rotary(x, pos, table, gain=gain, eps=1e-6, interleaved=interleaved)
    rest = fused[:, [0, 5, 6]].clone()
    dy = make(x.shape, dtype, 5)
    want_dx, want_dg = lla.rotary_backward(dy, x, pos, table, gain=gain, eps=1e-6, interleaved=interleaved)
    got_dx, got_dg = lla.rotary_backward(dy, x, pos, table, gain=gain, eps=1e-6, interleaved=interleaved, dx=dy)
    assert got_dx is dy and torch.equal(dy, want_dx) and torch.equal(got_dg, want_dg)
    assert lla.rotary(x, pos, table, gain=gain, eps=1e-6, interleaved=interleaved, out=x) is x
    assert torch.equal(x, want) and torch.equal(fused[:, [0, 5, 6]], rest)


def test_rows_of_zeros_and_large_values(lla_gpu):
    """A row of zeros stays one (eps), and its gradient is dy's over sqrt(eps); magnitudes to 2^60 neither overflow nor vanish."""
    table, pos = lla.rotary_table(64), torch.arange(3, dtype=torch.int32, device="cuda")
    x = make((3, 1, 64), "fp32")
    x[0] = 0
    x[1] *= 2.0 ** 60
    x[2] *= 2.0 ** -10
    check_forward(lla.rotary(x, pos, table, eps=1e-6), x, angles_of(pos, table, True), table, "fp32", None, 1e-6, False)
    dy = make(x.shape, "fp32", 2)
    dx, _ = lla.rotary_backward(dy, x, pos, table, eps=1e-6)
    check_backward(dx, None, dy, x, angles_of(pos, table, True), table, "fp32", None, 1e-6, False)


def test_many_rows_gain_gradient_has_the_same_bits_every_run(lla_gpu):
    B, H, n, d = 2, 16, 3001, 128
    x, dy, pos = make((B, H, n, d), "bf16"), make((B, H, n, d), "fp32", 1), torch.arange(n, dtype=torch.int32, device="cuda")
    gain, table = 1 + 0.3 * make((d,), "fp32", 3), lla.rotary_table(d)
    a = lla.rotary_backward(dy, x, pos, table, gain=gain, eps=1e-6)
    ws = torch.full((lla.lla_rotary_backward_workspace_size(1, d),), 255, dtype=torch.uint8, device="cuda")
    b = lla.rotary_backward(dy, x, pos, table, gain=gain, eps=1e-6, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_backward(a[0], a[1], dy, x, angles_of(pos, table, False), table, "bf16", gain, 1e-6, False)


def test_capture_streams_and_two_at_once(lla_gpu):
    T, d = 40, 64
    x, pos, table = make((T, 4, d), "bf16"), torch.arange(T, dtype=torch.int32, device="cuda"), lla.rotary_table(d)
    gain, out, dy, dx = 1 + 0.3 * make((d,), "fp32", 3), torch.empty_like(x), make(x.shape, "bf16", 8), torch.empty_like(x)
    step = lambda: (lla.rotary(x, pos, table, gain=gain, eps=1e-6, out=out),  # noqa: E731
                    lla.rotary_backward(dy, x, pos, table, gain=gain, eps=1e-6, dx=dx)[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, dgain = step()
    for k in range(3):
        x.copy_(make(x.shape, "bf16", 20 + k))
        pos += 1000
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), dx.clone(), dgain.clone()
        y, want = step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], y) and torch.equal(got[1], dx) and torch.equal(got[2], want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = lla.rotary(x, pos, table, stream=side)
    b = lla.rotary(x, pos, table)
    ga = lla.rotary_backward(dy, x, pos, table, gain=gain, eps=1e-6, stream=side)[1]
    gb = lla.rotary_backward(dy, x, pos, table, gain=gain, eps=1e-6)[1]
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(ga, gb)


def test_binding_refusals(lla_gpu):
    x, pos, t = make((4, 2, 64), "bf16"), torch.zeros(4, dtype=torch.int32, device="cuda"), lla.rotary_table(64)
    gain = torch.ones(64, device="cuda")
    bad = [lambda: lla.rotary(x, pos.long(), t), lambda: lla.rotary(x, pos[:3], t), lambda: lla.rotary(x, pos.cpu(), t),
           lambda: lla.rotary(x.half(), pos, t), lambda: lla.rotary(x[0], pos, t), lambda: lla.rotary([x, x.float()], pos, t),
           lambda: lla.rotary([x, x[:3]], pos, t), lambda: lla.rotary(x, pos, t, gain=gain), lambda: lla.rotary(x, pos, t, eps=-1.0, gain=gain),
           lambda: lla.rotary(x, pos, t, eps=-1.0), lambda: lla.rotary(x, pos, t, eps=float("nan")), lambda: lla.rotary_backward(x, x, pos, t, eps=-1.0),
           lambda: lla.rotary(x, pos, t, eps=0.0, gain=gain[:32]), lambda: lla.rotary(x, pos, t, eps=0.0, gain=gain.bfloat16()),
           lambda: lla.rotary([x, x], pos, t, eps=0.0, gain=[gain]), lambda: lla.rotary(x, pos, t, out=torch.empty_like(x).float()),
           lambda: lla.rotary(x, pos, t, out=torch.empty(4, 2, 65, device="cuda", dtype=torch.bfloat16)[..., 1:]),
           lambda: lla.rotary([], pos, t), lambda: lla.rotary_backward([], None, pos, t), lambda: lla.rotary([x] * 5, pos, t),
           lambda: lla.rotary(x, pos, t, out=torch.empty_like(x)[:1].expand(4, 2, 64)), lambda: lla.rotary(x, pos, t, shift=pos), lambda: lla.rotary(x, pos, t, shift=pos, cu_q=pos),
           lambda: lla.rotary(x, pos, lla.rotary_table(128)), lambda: lla.rotary(make((4, 2, 48), "bf16"), pos, lla.rotary_table(48)),
           lambda: lla.rotary(x[:0], pos[:0], t), lambda: lla.rotary_backward(x, x, pos[:2], t),
           lambda: lla.rotary_backward(x.half(), x, pos, t), lambda: lla.rotary_backward(x[:, :1], x, pos, t),
           lambda: lla.rotary_backward(x, x, pos, t, eps=0.0, gain=gain, workspace=gain)]
    for i, f in enumerate(bad):
        with pytest.raises(lla.LLAError):
            f()
            pytest.fail(f"call {i} was not refused")
    torch.cuda.synchronize()
    lla.lla_sync_status()


def test_both_ways_of_marshalling_give_the_same_bits(lla_gpu, monkeypatch):
    T, d = 33, 64
    fused = make((T, 9 * d), "bf16")
    xs = [t.reshape(T, -1, d) for t in fused.split([4 * d, 2 * d, 3 * d], 1)]
    pos, table = torch.arange(T, dtype=torch.int32, device="cuda"), lla.rotary_table(d)
    gains = [1 + 0.3 * make((d,), "fp32", i) for i in range(3)]
    cu, shift = torch.tensor([0, 10, 30], dtype=torch.int32, device="cuda"), torch.tensor([5, 9], dtype=torch.int32, device="cuda")
    dys = [make(x.shape, "fp32", 7) for x in xs]
    four, dy4, pos4 = make((2, 3, T, d), "fp32"), make((2, 3, T, d), "fp32", 1), pos[None].repeat(2, 1)

    def calls():
        lla.rotary_backward(dys[0], xs[0], pos, table, gain=gains[0], eps=0.1)        # (the thread's scratch is there from now on)
        return [lla.rotary(xs, pos, table, gain=gains, eps=1e-6, cu_q=cu, shift=shift), (lla.rotary(xs[1], pos, table, interleaved=True),),
                lla.rotary((xs[0], xs[2]), pos, table, gain=(None, gains[0]), eps=0.1), (lla.rotary(four, pos4, table, eps=0.0),),
                (lla.rotary(four, pos, table),), *[(*r[0], *[g for g in r[1] or () if g is not None]) for r in
                                                   (lla.rotary_backward(dys, xs, pos, table, gain=gains, eps=1e-6, cu_q=cu, shift=shift),
                                                    lla.rotary_backward(dys[:2], xs[:2], pos, table, gain=(None, gains[1]), eps=1e-6),
                                                    lla.rotary_backward(dys, xs, pos, table, eps=1e-6), lla.rotary_backward(dys, None, pos, table))],
                (lla.rotary_backward(dy4, four, pos4, table, gain=gains[0], eps=0.0)[1],)]

    fast = calls()
    one = lla.rotary_backward([dys[0]], [xs[0]], pos, table, gain=gains[0], eps=1e-6)
    assert isinstance(one[0], tuple) and isinstance(one[1], tuple)
    assert lla.rotary_backward(dys[:1], xs[:1], pos, table, gain=[None], eps=1e-6)[1] is None
    monkeypatch.setattr(lla, "_BIND", False)
    for a, b in zip(fast, calls()):
        assert len(a) == len(b) and all(x.dtype is y.dtype and torch.equal(x, y) for x, y in zip(a, b))
    two = lla.rotary_backward([dys[0]], [xs[0]], pos, table, gain=gains[0], eps=1e-6)
    assert torch.equal(one[0][0], two[0][0]) and torch.equal(one[1][0], two[1][0])


@pytest.mark.parametrize("B,H,n,d,rot,interleaved", [(1, 2, 40, 32, 32, False), (2, 1, 33, 64, 24, True)])
def test_training_step(lla_gpu, B, H, n, d, rot, interleaved):
    """Rotated, normalised queries and keys through the attention and back: gradients of the unrotated rows and of the gains.

    The oracle's attention gradients are taken at the rotated rows that the GPU made (checked by themselves).  dq and dk are
    within 1e-3 of their RMS, floored at 1e-2 RMS(dout), the bound of a forward and a backward call in series; the way back through
    rotation and norm is linear in them.
    """
    tau, lam, caps = d ** -0.5, 0.1, (4 * d + 64, 1e-6)
    xs = [make((B, H, n, d), "fp32", i) for i in range(2)]
    v, dout = make((B, H, n, d), "fp32", 2), make((B, H, n, d), "fp32", 3)
    gains = [1 + 0.3 * make((d,), "fp32", 4 + i) for i in range(2)]
    pos, table = torch.arange(n, dtype=torch.int32, device="cuda"), lla.rotary_table(rot)
    kw = dict(gain=gains, eps=1e-6, interleaved=interleaved)
    q, k = lla.rotary(xs, pos, table, **kw)
    _, rho, denom = lla.forward(q, k, v, tau, lam, *caps, path=lla.LLA_PATH_FP32)
    dq, dk, _ = lla.backward(q, k, v, rho, denom, dout, tau, lam, *caps, path=lla.LLA_PATH_FP32)
    dxs, dgains = lla.rotary_backward([dq, dk], xs, pos, table, **kw)
    torch.cuda.synchronize()
    lla.lla_sync_status()
    ang = angles_of(pos, table, False)
    for x, y, gain in zip(xs, (q, k), gains):
        check_forward(y, x, ang, table, "fp32", gain, 1e-6, interleaved)
    grads = lla_grad_ref(f64(q), f64(k), f64(v), f64(dout), tau, lam)[:2]
    floor = 1e-2 * np.sqrt((f64(dout) ** 2).mean())
    for x, g, gain, dx, dgain, own in zip(xs, grads, gains, dxs, dgains, (dq, dk)):
        check_backward(dx, dgain, own, x, ang, table, "fp32", gain, 1e-6, interleaved)
        ref, rg = rotary_backward_ref(g, f64(x), ang, f64(gain), 1e-6, interleaved)
        off = pair_sum(np.full(g.shape, 1e-3 * max(np.sqrt((g ** 2).mean()), floor)), rot, interleaved)
        size = pair_sum(g, rot, interleaved)
        s = 1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + 1e-6)
        m = np.abs(f64(x) * s)
        h = (off + (2 * d + 64) * U * size) * np.abs(f64(gain))
        worst = (np.abs(f64(dx) - ref) / (s * (h + m * (m * h).mean(-1, keepdims=True)) + U * np.abs(ref))).max()
        assert worst <= 1.0, worst
        worst = (np.abs(f64(dgain) - rg) / ((off + (B * H * n + 64 + 2 * d) * U * size) * m).reshape(-1, d).sum(0)).max()
        assert worst <= 1.0, worst


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_broadcast_inputs(lla_gpu, dtype):
    """Rows that are one row repeated: a gradient of ones expanded, and x the same for all heads or positions."""
    B, H, n, d = 2, 3, 21, 64
    pos, table = torch.arange(n, dtype=torch.int32, device="cuda"), lla.rotary_table(d)
    gain = 1 + 0.3 * make((d,), "fp32", 3)
    ones = torch.ones((), dtype=DT[dtype], device="cuda").expand(B, H, n, d)
    ang = angles_of(pos, table, False)
    for x in (make((B, 1, n, d), dtype).expand(B, H, n, d), make((B, H, 1, d), dtype, 1).expand(B, H, n, d), make((1, H, n, d), dtype, 2).expand(B, H, n, d)):
        check_forward(lla.rotary(x, pos, table, gain=gain, eps=1e-6), x, ang, table, dtype, gain, 1e-6, False)
        for dy in (ones, ones.float(), make((B, 1, 1, d), dtype, 5).expand(B, H, n, d)):
            dx, dgain = lla.rotary_backward(dy, x, pos, table, gain=gain, eps=1e-6)
            check_backward(dx, dgain, dy, x, ang, table, dtype, gain, 1e-6, False)
