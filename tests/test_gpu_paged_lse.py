"""The logsumexp of paged_parallax against float64, row by row.

A logit tau q.k is a sum of d products in fp32 (bf16 operands multiply exactly) and is scaled once or twice: within
(d + 8) 2^-24 tau sum |q_c k_c| of itself, sum |q_c k_c| <= |q||k| <= scale d knorm by construction.  The exponent's argument
(a logit less a reference point) rounds by 2 2^-24 of the largest logit's size, each exponential by 2^-22, the sum of the weights by
(keys + parts) 2^-24 at most, all relative to the sum, that is absolute in its logarithm; the logarithm and its sum with the
reference point by 4 2^-24 (|lse| + 8).
"""
import numpy as np
import pytest
import torch

import local_linear_attention_flashlla_gb300 as lla
from oracle.paged_ref import gather_pages
from test_gpu_paged import KINDS, Case, paths

pytestmark = pytest.mark.gpu


def lse_ref(c):
    out = np.full((c.q.shape[0], c.Hq), np.nan)
    q, G = c.q.double().numpy(), c.Hq // c.Hkv
    for s, L in enumerate(c.kv):
        lo, hi = int(c.cu[s]), int(c.cu[s + 1])
        K = gather_pages(c.kc.double().numpy(), c.table[s], L)
        sees = np.clip(L - (hi - lo) + np.arange(hi - lo) + 1, 0, L) if c.causal else np.full(hi - lo, L)
        for h in range(c.Hq):
            x = np.where(np.arange(L)[None] >= sees[:, None], -np.inf, c.tau * (q[lo:hi, h] @ K[h // G].T))
            top = x.max(1, initial=-np.inf)
            with np.errstate(divide="ignore"):
                out[lo:hi, h] = np.log(np.exp(x - np.where(np.isfinite(top), top, 0.0)[:, None]).sum(1)) + np.where(
                    np.isfinite(top), top, 0.0)
    return out


def check(c, got):
    ref, u = lse_ref(c), 2.0 ** -24
    got = got.double().cpu().numpy()
    mine = ~np.isnan(ref)
    none = mine & np.isneginf(ref)
    assert np.isneginf(got[none]).all()
    mine &= ~none
    logit = c.tau * c.scale * c.d * c.knorm
    tol = u * ((c.d + 10) * logit + max(c.kv) + 152 + 8 + 4 * (np.abs(ref) + 8))
    assert (np.abs(got - ref)[mine] <= tol[mine]).all(), np.nanmax((np.abs(got - ref) / tol)[mine])
    return ref


def run(c, path=lla.LLA_PATH_AUTO, **kw):
    lse = torch.full(c.q.shape[:2], 7.0, device="cuda")
    out = lla.paged_parallax(**c.device(), path=path, lse=lse, **kw)
    plain = lla.paged_parallax(**c.device(), path=path, **kw)
    torch.cuda.synchronize()
    lla.lla_sync_status()
    rows = slice(0, int(c.cu[-1]))
    assert torch.equal(out[rows], plain[rows])
    assert (lse[int(c.cu[-1]):] == 7.0).all()
    return lse


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("bf16", 16), ("fp32", 128), ("fp32", 64),
                                     ("fp32", 32), ("fp32", 16)])
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("G,Hkv,page", [(1, 3, 16), (4, 2, 64), (3, 1, 8)])
def test_logsumexp(lla_gpu, dtype, d, kind, G, Hkv, page):
    new, kv = KINDS[kind]
    c = Case(new, kv, G * Hkv, Hkv, d, page, dtype, pad=2)
    for path, _ in paths(dtype, d):
        check(c, run(c, path))


@pytest.mark.parametrize("dtype,d,path", [("bf16", 128, lla.LLA_PATH_TENSOR), ("bf16", 64, lla.LLA_PATH_TENSOR),
                                          ("bf16", 64, lla.LLA_PATH_FP32), ("fp32", 32, lla.LLA_PATH_AUTO)])
@pytest.mark.parametrize("new", [[1], [7], [40], [200]])
def test_parts_of_many_ctas_and_cross_attention(lla_gpu, dtype, d, path, new):
    check(*(lambda c: (c, run(c, path)))(Case(new, [9000], 4, 2, d, 32, dtype)))
    check(*(lambda c: (c, run(c, path)))(Case(new, [700], 4, 2, d, 32, dtype, causal=False)))


@pytest.mark.parametrize("new,kv", [([1, 1, 1], [0, 5, 0]), ([20, 3, 40, 2], [4, 0, 39, 0]), ([0, 1, 0], [3, 4, 0])])
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (32, "fp32")])
def test_rows_without_keys(lla_gpu, new, kv, d, dtype):
    check(*(lambda c: (c, run(c)))(Case(new, kv, 4, 2, d, 16, dtype, pad=3)))


@pytest.mark.parametrize("new", [[1, 2], [150, 9]])
def test_large_logits(lla_gpu, new):
    check(*(lambda c: (c, run(c)))(Case(new, [400, 300], 4, 2, 128, 16, scale=20.0)))


def test_marshalling_in_python_and_refusals(lla_gpu, monkeypatch):
    c = Case([1, 3], [40, 90], 4, 2, 64, 16)
    a = run(c)
    monkeypatch.setattr(lla, "_BIND", False)
    assert torch.equal(a, run(c))
    for bad in (torch.zeros(4, 4), torch.zeros(4, 4, device="cuda", dtype=torch.float64), torch.zeros(4, 3, device="cuda"),
                torch.zeros(4, 8, device="cuda")[:, ::2]):
        with pytest.raises(lla.LLAError):
            lla.paged_parallax(**c.device(), lse=bad)
