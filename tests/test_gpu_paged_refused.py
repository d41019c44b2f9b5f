"""A step in which the free list runs out: what the plan refused leaves the caches and the other sequences alone, and its
rows hold what include/lla.h says (attention as the last of the positions cached before)."""
import math

import numpy as np
import pytest
import torch

import local_linear_attention_flashlla_gb300 as lla
from oracle.paged_ref import paged_plan_ref
from test_gpu_paged import DT, Case, _i32, paths

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("fp32", 32), ("fp32", 128)])
@pytest.mark.parametrize("new,ctx,free", [([1, 1, 1, 1], [31, 16, 40, 32], 1), ([20, 90, 3, 30], [10, 50, 13, 200], 4),
                                          ([40, 2, 3], [5, 30, 0], 2), ([50, 1], [9, 64], 0)])
def test_refused_sequences(lla_gpu, dtype, d, new, ctx, free):
    page, Hq, Hkv, S, W = 16, 4, 2, len(new), 20
    rng = np.random.default_rng(d + S)
    T, dt = sum(new) + 2, DT[dtype]
    ids, at = rng.permutation(100), 0
    table = np.full((S, W), -1)
    for s in range(S):
        held = -(-ctx[s] // page)
        table[s, :held] = ids[at:at + held]
        at += held
    stack = ids[at:at + max(free, 1)]
    ref = paged_plan_ref(ctx, new, table, stack, free, page, T)
    assert 0 in ref["granted"]
    tb = _i32(table)
    pl = lla.paged_plan(_i32(ctx), _i32(new), tb, _i32(stack), _i32([free]), page, T)

    unit = lambda *sh: (lambda x: x / np.sqrt((x * x).mean(-1, keepdims=True)))(rng.standard_normal(sh))  # noqa: E731
    make = lambda x: torch.tensor(x, dtype=torch.float32).to(dt)  # noqa: E731
    kc, vc = make(np.full((100, Hkv, page, d), np.nan)), make(np.full((100, Hkv, page, d), np.nan))
    for s in range(S):
        for x in range(ctx[s]):
            kc[table[s, x // page], :, x % page] = make(unit(Hkv, d))
            vc[table[s, x // page], :, x % page] = make(rng.standard_normal((Hkv, d)))
    before = kc.clone(), vc.clone()
    k, v = make(unit(T, Hkv, d)), make(rng.standard_normal((T, Hkv, d)))
    kc, vc = kc.cuda(), vc.cuda()
    lla.paged_append(k.cuda(), v.cuda(), pl.slots, kc, vc)
    # the caches: the granted tokens' positions and nothing else
    want = before[0].clone(), before[1].clone()
    for t, slot in enumerate(ref["slots"]):
        if slot >= 0:
            want[0][slot // page, :, slot % page], want[1][slot // page, :, slot % page] = k[t], v[t]
    for got, w in zip((kc, vc), want):
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=77.0), torch.nan_to_num(w, nan=77.0))

    # attention: every row against the definition at kv_lens as planned (a refused sequence: ctx)
    c = Case.__new__(Case)
    c.new, c.kv, c.cu, c.causal, c.dtype, c.d, c.page = new, ref["kv_lens"], np.array(ref["cu_q"]), True, dtype, d, page
    c.Hq, c.Hkv, c.tau, c.scale, c.knorm = Hq, Hkv, 1 / math.sqrt(d), 1.0, 1.0
    c.q, c.probe, c.kc, c.vc, c.table = make(unit(T, Hq, d)), make(unit(T, Hq, d) / math.sqrt(d)), *want, ref["table"]
    for path, tensor in paths(dtype, d):
        out = torch.full((T, Hq, d), 123.0, dtype=dt, device="cuda")
        lla.paged_parallax(c.q.cuda(), c.probe.cuda(), kc, vc, tb, pl.cu_q, pl.kv_lens, c.tau, max(new), path=path, out=out)
        torch.cuda.synchronize()
        lla.lla_sync_status()                      # a refusal is not an error
        got = c.check(out, tensor)
        assert (got[sum(new):] == 123.0).all()
        for s in range(S):
            if not ref["granted"][s]:
                early = max(new[s] - ctx[s], 0)    # rows before the first cached position
                assert (got[c.cu[s]:c.cu[s] + early] == 0).all()
        # the granted sequences' rows do not depend on the refused ones
        keep = [s for s in range(S) if ref["granted"][s]]
        if keep:
            rows = np.concatenate([np.arange(c.cu[s], c.cu[s + 1]) for s in keep])
            cu = np.concatenate([[0], np.cumsum([new[s] for s in keep])])
            alone = lla.paged_parallax(c.q[rows].cuda(), c.probe[rows].cuda(), kc, vc, _i32(ref["table"][keep]), _i32(cu),
                                       _i32([ref["kv_lens"][s] for s in keep]), c.tau, max(new), path=path)
            torch.cuda.synchronize()
            a, b = alone.double().cpu().numpy(), got[rows]
            # both are within their bound of the same value (cuts of the work differ, so bits may)
            half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -20
            assert np.linalg.norm(a - b) <= 4 * half * np.linalg.norm(b) + 1e-30
