"""Eviction where no histogram is made: all scores that count are equal, or more positions are mandatory than are kept.

The counts of mandatory positions and of ties are then exchanged between the block's warps one right after the other; every
run has to give the definition's result bit by bit, with blocks of both sizes and with clusters.
"""
import numpy as np
import pytest
import torch

import local_linear_attention_flashlla_gb300 as lla
from test_gpu_evict import Evict
from test_gpu_paged import _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,sinks,recent", [("equal", 0, 0), ("equal", 3, 5), ("random", 40, 400), ("random", 0, 10 ** 9)])
@pytest.mark.parametrize("S,Hkv", [(1, 3), (5, 8), (40, 8), (100, 7)])
def test_evict_without_a_histogram_every_run_alike(lla_gpu, kind, sinks, recent, S, Hkv):
    rng = np.random.default_rng(S + sinks)
    kv = [int(x) for x in rng.integers(2, 700, S)]
    keep = [int(rng.integers(1, min(n, 60))) for n in kv]              # few kept: most warps have no tie to count
    e = Evict(kv, keep, Hkv, 16, 16, "bf16", kind, sinks, recent, seed=S)
    k, v, s, p = (t.cuda() for t in e.want())
    fresh = [t.cuda() for t in (e.kc, e.vc, e.scores, e.positions)]
    args = _i32(e.table), _i32(kv), _i32(keep)
    kw = dict(dropped=_i32(e.dropped), sinks=sinks, recent=recent)
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for _ in range(60):
        kc, vc, sc, pos = (t.clone() for t in fresh)
        lla.paged_evict(sc, kc, vc, *args, positions=pos, **kw)
        for got, want in ((kc, k), (vc, v), (sc, s), (pos, p)):
            same &= (got == want).all()
    torch.cuda.synchronize()
    lla.lla_sync_status()
    assert bool(same)
