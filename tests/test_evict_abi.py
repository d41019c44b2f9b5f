"""Bounded caches without a GPU: refusals of the entry points, and the references by their definitions."""
import numpy as np
import pytest
import torch

import local_linear_attention_flashlla_gb300 as lla
from local_linear_attention_flashlla_gb300 import build as lla_build
from oracle.cache_ref import paged_evict_ref, paged_trim_ref, paged_weigh_ref


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(lla.library_path()):
        lla_build.build()
    return lla.load_library()


def _weigh(lib, **kw):
    a = dict(dtype=0, q=16, lse=32, kc=48, sc=64, so=64, pos=80, drop=96, table=112, cu=128, kv=144, ok=None, T=4, S=2, Hq=4, Hkv=2, d=64,
             page=16, P=3, W=4, max_new=2, qs=256, ps=2048, tau=0.1, decay=1.0, last=0, causal=1, ws=None, wsb=0)
    a.update(kw)
    return lib.lla_paged_weigh(a["dtype"], a["q"], a["lse"], a["kc"], a["sc"], a["so"], a["pos"], a["drop"], a["table"], a["cu"],
                               a["kv"], a["ok"], a["T"], a["S"], a["Hq"], a["Hkv"], a["d"], a["page"], a["P"], a["W"], a["max_new"], a["qs"],
                               a["ps"], a["tau"], a["decay"], a["last"], a["causal"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(lse=None), dict(kc=None), dict(sc=None), dict(so=None), dict(table=None), dict(cu=None), dict(kv=None),
    dict(q=24), dict(kc=40), dict(lse=34), dict(sc=65), dict(so=66), dict(pos=81), dict(drop=98), dict(ok=177), dict(table=113), dict(T=0),
    dict(S=0), dict(S=(1 << 20) + 1), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(d=48), dict(page=7), dict(page=512), dict(P=0),
    dict(W=0), dict(W=1 << 25), dict(max_new=0), dict(qs=255), dict(qs=252), dict(ps=1024), dict(ps=2050), dict(tau=0.0), dict(tau=1e-31),
    dict(tau=float("nan")), dict(tau=float("inf")), dict(decay=-0.5), dict(decay=float("nan")), dict(decay=float("inf")), dict(last=-1),
    dict(dtype=2), dict(T=1 << 29), dict(Hq=4096, qs=1 << 20), dict(P=1 << 30),
])
def test_weigh_refusals(lib, bad):
    assert _weigh(lib, **bad) == lla.LLA_ERR_INVALID_ARG
    assert lib.lla_last_error().decode()


def _evict(lib, **kw):
    a = dict(dtype=0, sc=64, so=64, pos=80, po=80, kc=48, vc=32, table=112, kv=144, keep=160, drop=None, S=2, Hkv=2, d=64, page=16, P=3,
             W=4, ps=2048, sinks=1, recent=1)
    a.update(kw)
    return lib.lla_paged_evict(a["dtype"], a["sc"], a["so"], a["pos"], a["po"], a["kc"], a["vc"], a["table"], a["kv"], a["keep"],
                               a["drop"], a["S"], a["Hkv"], a["d"], a["page"], a["P"], a["W"], a["ps"], a["sinks"], a["recent"], None)


@pytest.mark.parametrize("bad", [
    dict(sc=None), dict(so=None), dict(kc=None), dict(vc=None), dict(table=None), dict(kv=None), dict(keep=None), dict(pos=None),
    dict(po=None), dict(pos=None, po=None), dict(pos=None, po=None, sinks=0), dict(sc=65), dict(so=66), dict(pos=82), dict(po=81),
    dict(kc=40), dict(vc=8), dict(table=113), dict(kv=142), dict(keep=161), dict(drop=99), dict(dtype=2), dict(d=8), dict(page=0),
    dict(page=24), dict(S=0), dict(S=(1 << 20) + 1), dict(Hkv=0), dict(Hkv=65536), dict(P=0), dict(W=0), dict(W=1 << 26), dict(ps=1024),
    dict(ps=2052), dict(sinks=-1), dict(recent=-1), dict(S=1 << 20, Hkv=1024, ps=1 << 20),
])
def test_evict_refusals(lib, bad):
    assert _evict(lib, **bad) == lla.LLA_ERR_INVALID_ARG
    assert lib.lla_last_error().decode()


def _trim(lib, **kw):
    a = dict(kv=16, keep=32, S=2, page=16, table=48, W=4, free=64, F=8, count=80, drop=96, nl=16, nd=96, left=80)
    a.update(kw)
    return lib.lla_paged_trim(a["kv"], a["keep"], a["S"], a["page"], a["table"], a["W"], a["free"], a["F"], a["count"], a["drop"],
                              a["nl"], a["nd"], a["left"], None)


@pytest.mark.parametrize("bad", [
    dict(kv=None), dict(keep=None), dict(table=None), dict(free=None), dict(count=None), dict(nl=None), dict(left=None), dict(nd=None),
    dict(kv=17), dict(keep=33), dict(table=50), dict(free=66), dict(count=81), dict(drop=97), dict(nl=18), dict(nd=98), dict(left=82),
    dict(S=0), dict(S=8193), dict(page=4), dict(page=48), dict(W=0), dict(W=1 << 26), dict(F=0),
])
def test_trim_refusals(lib, bad):
    assert _trim(lib, **bad) == lla.LLA_ERR_INVALID_ARG
    assert lib.lla_last_error().decode()


def test_workspace_size(lib):
    size = lambda dtype=0, Hq=4, d=64, page=16, most=2: lib.lla_paged_weigh_workspace_size(dtype, 4, 2, Hq, 2, d, page, 4, most)  # noqa: E731
    assert size() > 0 and size(dtype=1) > 0
    assert size(Hq=5) == size(d=10) == size(page=9) == size(dtype=7) == size(most=0) == 0


def test_binding_refuses_cpu_tensors():
    z, i = torch.zeros(2, 1, 8, 16), torch.zeros(1, 2, dtype=torch.int32)
    s = torch.zeros(2, 1, 8)
    for f in (lambda: lla.paged_weigh(z[:, :, 0], s, z, s, i, i[0], i[0, :1], 1.0, 1), lambda: lla.paged_evict(s, z, z, i, i[0, :1], i[0, :1]),
              lambda: lla.paged_trim(i[0, :1], i[0, :1], i, i[0], i[0, :1], 8)):
        with pytest.raises(lla.LLAError):
            f()


def test_weigh_reference_is_the_softmax_summed():
    """Scores of a prompt sum to its rows (each row's weights sum to one); a second step adds and decays."""
    rng = np.random.default_rng(0)
    k, q, n, G = rng.standard_normal((3, 2, 8, 4)), rng.standard_normal((20, 4, 4)), 20, 2
    table, keys = np.array([[2, 0, 1]]), np.concatenate([k[2], k[0], k[1]], 1)[:, :20]
    logit = np.einsum("thd,hjd->thj", q, keys[[0, 0, 1, 1]])
    logit = np.where(np.arange(20)[None, None] > np.arange(20)[:, None, None], -np.inf, logit)
    lse = np.log(np.exp(logit).sum(-1))
    s, p, mag = paged_weigh_ref(q, lse, k, np.full((3, 2, 8), 5.0), table, [0, n], [n], 1.0, positions=np.full((3, 2, 8), -1), dropped=[100])
    assert np.isclose(mag.sum(), n * G * 2) and np.isclose(s[table[0, 2], :, 4:], 5.0).all()
    assert p[2, 0].tolist() == list(range(100, 108)) and p[1, 1].tolist() == [116, 117, 118, 119, -1, -1, -1, -1]
    one = paged_weigh_ref(q[19:], lse[19:], k, s, table, [0, 1], [n], 1.0, decay=0.5)[0]
    assert np.isclose(one[1, 0, 3], np.exp(logit[19, :2, 19] - lse[19, :2]).sum())      # the step's own token starts anew
    assert np.isclose(one[2, 0, 0], 0.5 * s[2, 0, 0] + np.exp(logit[19, :2, 0] - lse[19, :2]).sum())
    few = paged_weigh_ref(q, lse, k, s, table, [0, n], [n], 1.0, last=3)[2]
    assert np.isclose(few.sum(), 3 * G * 2)


def test_evict_reference_keeps_the_best_and_fills_holes():
    s = np.array([[[5, 1, np.nan, 4, 1, 9, -np.inf, 4]]], np.float64)
    got = paged_evict_ref(s, [[0]], [8], [4], 8, 1)
    assert got[0, 0] == [0, 5, 7, 3]                           # 9, 5, 4 (slot 3), 4 (slot 7): 1 and 2 leave
    assert paged_evict_ref(s, [[0]], [3], [4], 8, 1)[0, 0] == [0, 1, 2]
    pos = np.arange(8).reshape(1, 1, 8)
    assert paged_evict_ref(s, [[0]], [8], [4], 8, 1, pos, [0], sinks=2, recent=1)[0, 0] == [0, 1, 5, 7]
    assert paged_evict_ref(np.zeros((1, 1, 8)), [[0]], [8], [3], 8, 1)[0, 0] == [0, 1, 2]


def test_trim_reference():
    r = paged_trim_ref([20, 8, 0, 17], [9, 50, 3, 0], [[4, 5, 6], [7, -1, -1], [-1] * 3, [1, -1, 2]], [9, 0, 0, 0], 1, 8, [1, 2, 3, 4])
    assert r == dict(kv_lens=[9, 8, 0, 0], dropped=[12, 2, 3, 21], free_left=4, free_pages=[9, 6, 1, 2], full=False)
