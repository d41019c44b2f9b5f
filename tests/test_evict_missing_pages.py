"""Eviction beside table entries that are no pages: such a slot below the kept length takes no row, so that many fewer positions are
kept, and none of those is left behind it to be trimmed away."""
import numpy as np
import pytest
import torch

from oracle.cache_ref import paged_evict_ref


def test_reference_keeps_as_many_as_there_are_places():
    s = np.array([[[5, 1, 9, 4, 1, 9, 2, 4]], [[7, 3, 3, 0, 8, 6, 7, 1]]], np.float64)
    # slots 0 .. 7 without a page; 8 .. 15 are page 1, 16 .. 23 page 0; 12 are kept: four places, for 9, 9, 8 and a 7
    got = paged_evict_ref(s, [[-1, 1, 0]], [24], [12], 8, 1)[0, 0]
    assert got == [0, 1, 2, 3, 4, 5, 6, 7, 8, 12, 18, 21]
    assert paged_evict_ref(s, [[9, 1, 0]], [24], [12], 8, 1)[0, 0] == got
    assert paged_evict_ref(s, [[1, -1, 0]], [24], [3], 8, 1)[0, 0] == [4, 18, 21]               # none missing below the kept length
    assert paged_evict_ref(s, [[-1, -1, 0]], [24], [12], 8, 1)[0, 0] == list(range(12))         # no place at all


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["random", "ties", "equal", "odd"])
@pytest.mark.parametrize("sinks,recent", [(0, 0), (3, 20), (0, 10 ** 9)])
@pytest.mark.parametrize("S,Hkv", [(3, 2), (90, 7)])
def test_evict_keeps_the_best_that_have_a_place(lla_gpu, kind, sinks, recent, S, Hkv):
    import local_linear_attention_flashlla_gb300 as lla
    from test_gpu_evict import Evict
    from test_gpu_paged import _i32
    rng = np.random.default_rng(S)
    kv = [300, 90, 1000] + [int(x) for x in rng.integers(20, 400, S - 3)]
    keep = [100, 60, 130] + [int(rng.integers(1, n)) for n in kv[3:]]
    e = Evict(kv, keep, Hkv, 16, 16, "bf16", kind, sinks, recent, seed=S)
    drop = rng.random(e.table.shape) < 0.15
    drop[0, :7] = True                                         # no place below the kept length
    drop[1] = False
    drop[2, 30:] = True                                        # many behind it
    e.table = np.where(drop, np.where(rng.random(drop.shape) < 0.5, -1, e.P + 3), e.table)
    want = e.want()
    kc, vc, sc, pos = (t.cuda() for t in (e.kc, e.vc, e.scores, e.positions))
    kw = dict(dropped=_i32(e.dropped), sinks=sinks, recent=recent) if sinks or recent else {}
    if kw:
        kw["positions"] = pos
    lla.paged_evict(sc, kc, vc, _i32(e.table), _i32(kv), _i32(keep), **kw)
    with pytest.raises(lla.LLAError) as x:
        lla.lla_sync_status()
    assert x.value.status == lla.LLA_ERR_INVALID_ARG
    same = lambda a, b: torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))  # noqa: E731
    assert all(same(a, b) for a, b in zip((kc, vc, sc), want)) and (not kw or same(pos, want[3]))
