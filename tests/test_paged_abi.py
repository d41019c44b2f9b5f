"""The paged-cache entry points refuse bad arguments on the host, before anything is launched (no GPU
needed), and the references they are tested against agree with the Parallax oracle."""
import numpy as np
import pytest

import local_linear_attention_flashlla_gb300 as lla
from local_linear_attention_flashlla_gb300 import build as lla_build
from oracle.lla_ref import parallax_ref
from oracle.paged_ref import paged_parallax_ref, paged_plan_ref


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(lla.library_path()):
        lla_build.build()
    return lla.load_library()


def _plan(lib, **kw):
    a = dict(ctx=16, new=32, S=4, page=16, table=48, W=8, free=64, F=32, count=80, T=9, kv=96, cu=112, slots=128,
             pos=144, granted=160, left=176)
    a.update(kw)
    return lib.lla_paged_plan(a["ctx"], a["new"], a["S"], a["page"], a["table"], a["W"], a["free"], a["F"], a["count"],
                              a["T"], a["kv"], a["cu"], a["slots"], a["pos"], a["granted"], a["left"], None)


@pytest.mark.parametrize("bad", [
    dict(ctx=None), dict(new=None), dict(table=None), dict(free=None), dict(count=None), dict(kv=None), dict(cu=None),
    dict(slots=None), dict(granted=None), dict(left=None), dict(ctx=18), dict(slots=132), dict(pos=2), dict(S=0),
    dict(S=8193), dict(page=0), dict(page=4), dict(page=24), dict(page=512), dict(W=0), dict(W=1 << 26), dict(F=0),
    dict(T=0), dict(T=-3),
])
def test_plan_refusals(lib, bad):
    assert _plan(lib, **bad) == lla.LLA_ERR_INVALID_ARG
    assert lib.lla_last_error().decode()


def _append(lib, **kw):
    a = dict(dtype=0, k=16, v=32, slots=48, kc=64, vc=80, T=4, Hkv=2, d=64, page=16, P=3, ks=128, vs=128, ps=2048)
    a.update(kw)
    return lib.lla_paged_append(a["dtype"], a["k"], a["v"], a["slots"], a["kc"], a["vc"], a["T"], a["Hkv"], a["d"],
                                a["page"], a["P"], a["ks"], a["vs"], a["ps"], None)


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None), dict(k=24), dict(vc=8), dict(slots=52),
    dict(dtype=2), dict(d=48), dict(d=0), dict(page=12), dict(T=0), dict(Hkv=0), dict(P=0), dict(ks=120), dict(vs=130),
    dict(ps=2047), dict(ps=2052), dict(ps=2056), dict(ks=-128), dict(P=1 << 30, ps=2048),
])
def test_append_refusals(lib, bad):
    assert _append(lib, **bad) == lla.LLA_ERR_INVALID_ARG
    assert lib.lla_last_error().decode()


def _attend(lib, **kw):
    a = dict(dtype=0, path=0, q=16, r=32, kc=48, vc=64, table=80, cu=96, kv=112, out=128, T=4, S=2, Hq=4, Hkv=2, d=64,
             page=16, P=3, W=4, max_new=2, qs=256, rs=256, ps=2048, tau=0.1, causal=1, ws=None, wsb=0)
    a.update(kw)
    return lib.lla_paged_parallax(a["dtype"], a["path"], a["q"], a["r"], a["kc"], a["vc"], a["table"], a["cu"], a["kv"],
                                  a["out"], a["T"], a["S"], a["Hq"], a["Hkv"], a["d"], a["page"], a["P"], a["W"],
                                  a["max_new"], a["qs"], a["rs"], a["ps"], a["tau"], a["causal"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(r=None), dict(kc=None), dict(vc=None), dict(table=None), dict(cu=None), dict(kv=None),
    dict(out=None), dict(q=24), dict(r=40), dict(kc=8), dict(out=132), dict(table=82), dict(cu=97), dict(kv=3),
    dict(T=0), dict(S=0), dict(S=(1 << 20) + 1), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(Hq=4096, Hkv=2, qs=1 << 20),
    dict(d=48), dict(d=256), dict(page=7), dict(page=1024), dict(P=0), dict(W=0), dict(W=1 << 25), dict(max_new=0),
    dict(qs=255), dict(rs=252), dict(qs=260), dict(ps=1024), dict(ps=2050), dict(ps=2056), dict(ps=2560), dict(tau=0.0), dict(tau=-1.0),
    dict(tau=float("nan")), dict(tau=float("inf")), dict(dtype=4), dict(path=3), dict(path=-1), dict(T=1 << 29),
])
def test_attention_refusals(lib, bad):
    assert _attend(lib, **bad) == lla.LLA_ERR_INVALID_ARG
    assert lib.lla_last_error().decode()


def test_attention_tensor_path_needs_bf16_and_supported_dim(lib):
    assert _attend(lib, dtype=1, path=lla.LLA_PATH_TENSOR) == lla.LLA_ERR_UNSUPPORTED
    assert _attend(lib, d=32, path=lla.LLA_PATH_TENSOR) == lla.LLA_ERR_UNSUPPORTED


def test_workspace_size(lib):
    size = lib.lla_paged_parallax_workspace_size
    assert size(0, 0, 64, 64, 16, 16, 128, 64, 64, 1) > 0
    assert size(1, 0, 64, 64, 16, 4, 32, 16, 64, 5) > 0
    assert size(0, 0, 64, 64, 15, 4, 128, 64, 64, 1) == 0       # heads
    assert size(0, 0, 64, 64, 16, 4, 128, 65, 64, 1) == 0       # page size
    assert size(1, lla.LLA_PATH_TENSOR, 64, 64, 16, 4, 128, 64, 64, 1) == 0


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    i = torch.zeros(4, dtype=torch.int32)
    c = torch.zeros(2, 1, 16, 64)
    x = torch.zeros(4, 1, 64)
    with pytest.raises(lla.LLAError):
        lla.paged_plan(i, i, torch.zeros(4, 3, dtype=torch.int32), i, i[:1], 16, 4)
    with pytest.raises(lla.LLAError):
        lla.paged_append(x, x, torch.zeros(4, dtype=torch.int64), c, c)
    with pytest.raises(lla.LLAError):
        lla.paged_parallax(x, x, c, c, torch.zeros(1, 2, dtype=torch.int32), i[:2], i[:1], 0.1, 4)


def test_marshalling_module_hands_back_what_it_does_not_know(lib):
    """csrc/paged_bind.c never raises on an argument and launches nothing for one that is not as expected."""
    torch = pytest.importorskip("torch")
    from local_linear_attention_flashlla_gb300 import _bind
    m = _bind()
    if not m:
        pytest.skip("built without a C compiler or the Python headers")
    i = torch.zeros(4, dtype=torch.int32)
    c, x, s = torch.zeros(2, 1, 16, 64), torch.zeros(4, 1, 64), torch.zeros(4, dtype=torch.int64)
    tb = torch.zeros(1, 2, dtype=torch.int32)
    for k in (c, None, 3, "cache", c[0], c.half(), c.transpose(1, 2)):            # CPU tensors: device -1, never 0
        assert m.append(0, x, x, s, k, k, 0) == -1
        assert m.parallax(0, x, x, k, k, tb, i[:2], i[:1], x, 0.1, 1, True, 0, 0, 0, 0) == -1
    assert m.append(-1, x, x, s, c, c, 0) == -1
    assert m.parallax(0, x, x, c, c, tb, i[:2], i[:1], x, "tau", 1, True, 0, 0, 0, 0) == -1
    assert m.parallax(0, x, x, c, c, tb, i[:2], i[:1], x, 0.1, 1 << 80, True, 0, 0, 0, 0) == -1
    assert m.plan(0, i, i, tb, i, i[:1], 16, 4, i, i, s, i, i, i, 0) == -1
    assert m.plan(0, None, i, tb, i, i[:1], 16, 4, i, i, s, i, i, i, 0) == -1
    assert m.plan(0, i) == -1 and m.append() == -1 and m.parallax(0) == -1


def test_token_rows_are_taken_as_they_lie_or_copied():
    """The binding's row check, on CPU tensors: packed heads at any 16-byte token stride pass as they are."""
    torch = pytest.importorskip("torch")
    from local_linear_attention_flashlla_gb300 import _token_rows
    base = torch.arange(5 * 3 * 2 * 16, dtype=torch.float32).view(5, 6, 16)
    t, stride = _token_rows(base[:, 2:4], "x", base, 2, 16)
    assert stride == 96 and t.data_ptr() == base[:, 2:4].data_ptr()
    flip = torch.arange(2 * 5 * 16, dtype=torch.float32).view(2, 5, 16).transpose(0, 1)     # heads not packed
    t, stride = _token_rows(flip, "x", base, 2, 16)
    assert stride == 32 and t.is_contiguous() and torch.equal(t, flip)
    odd = torch.arange(1 + 5 * 32, dtype=torch.float32)[1:].view(5, 2, 16)                   # base not 16-byte aligned
    t, stride = _token_rows(odd, "x", base, 2, 16)
    assert stride == 32 and t.data_ptr() % 16 == 0 and torch.equal(t, odd)
    one = base[0, :2].expand(4, 2, 16)                                                       # token stride 0
    t, stride = _token_rows(one, "x", base, 2, 16)
    assert stride == 32 and torch.equal(t, one)
    for bad in (base, base[:, :2, :8], base[0, :2], base[:, :2].double()):
        with pytest.raises(lla.LLAError):
            _token_rows(bad, "x", base, 2, 16)


@pytest.mark.parametrize("causal", [True, False])
def test_attention_reference_is_the_parallax_oracle(causal):
    rng = np.random.default_rng(3)
    n, d, page, P = 11, 16, 8, 4
    q, r, k, v = (rng.standard_normal((1, 2, n, d)) for _ in range(4))
    kc, vc = np.full((P, 2, page, d), np.nan), np.full((P, 2, page, d), np.nan)
    table = np.array([[2, 0, -1]])
    for x in range(n):
        kc[table[0, x // page], :, x % page] = k[0, :, x]
        vc[table[0, x // page], :, x % page] = v[0, :, x]
    rows = lambda t: t[0].transpose(1, 0, 2)  # noqa: E731
    out, mag, keys = paged_parallax_ref(rows(q), rows(r), kc, vc, table, [0, n], [n], 0.3, causal=causal)
    if causal:
        ref = parallax_ref(q, k, v, r, 0.3).reshape(2, n, d).transpose(1, 0, 2)
        assert np.abs(out - ref).max() < 1e-12 and list(keys) == list(range(1, n + 1))
    else:
        ref = parallax_ref(q[:, :, -1:].repeat(n, 2), k, v, r[:, :, -1:].repeat(n, 2), 0.3).reshape(2, n, d)
        assert np.abs(out[-1] - ref[:, -1]).max() < 1e-12
    assert (mag >= np.abs(out) - 1e-12).all()


def test_plan_reference_by_hand():
    # page 8: 5 + 4 tokens -> a second page; 8 + 1 -> a second page; 3 + 0; then one that finds the list empty
    r = paged_plan_ref([5, 8, 3, 16], [4, 1, 0, 1], [[7, -1], [6, -1], [5, -1], [4, 3]], [10, 11], 2, 8, 8)
    assert r["granted"] == [1, 1, 1, 0] and r["kv_lens"] == [9, 9, 3, 16] and r["cu_q"] == [0, 4, 5, 5, 6]
    assert r["table"].tolist() == [[7, 11], [6, 10], [5, -1], [4, 3]] and r["free_left"] == 0
    assert r["slots"].tolist() == [61, 62, 63, 88, 80, -1, -1, -1]
    assert r["positions"].tolist() == [5, 6, 7, 8, 8, 16, 0, 0]
