"""The scores and lengths of a bounded cache over many steps, followed on the host position by position.

Prompts, chunks and single tokens of four sequences through two layers: planned, rotated, cached, attended, weighed, evicted,
trimmed.  A position's score is followed in float64: after a step's weights it is decay * score (0 for a new position) plus
the sum of the definition's weights on the cached keys; eviction moves scores with their rows, so that the slot which claims a position
must hold that position's score, whatever happened before.  What eviction keeps is the definition's choice on the scores that the
device held.  Tolerance: a step's weights as in test_gpu_evict.py, and what a score was off before, decayed.
"""
import numpy as np
import pytest
import torch

import local_linear_attention_flashlla_gb300 as lla
from oracle.cache_ref import paged_evict_ref, paged_weigh_ref
from test_gpu_paged import DT, _i32

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("dtype,d,Hq,Hkv,decay", [("bf16", 128, 4, 2, 0.9), ("bf16", 64, 3, 3, 1.0), ("fp32", 32, 4, 1, 0.9), ("bf16", 32, 2, 1, 0.0)])
def test_scores_follow_their_positions(lla_gpu, dtype, d, Hq, Hkv, decay):
    torch.manual_seed(d)
    page, S, layers, W, F, dt = 16, 4, 2, 24, 90, DT[dtype]
    table, free, count = _i32(np.full((S, W), -1)), _i32(np.arange(F)), _i32([F])
    bound, tau, sinks, recent = [40, 90, 64, 7], d ** -0.5, 2, 10
    kv, drop, keep = _i32([0] * S), _i32([0] * S), _i32(bound)
    caches = [[torch.full((F, Hkv, page, d), float("nan"), device="cuda", dtype=dt) for _ in range(2)] for _ in range(layers)]
    state = [(torch.full((F, Hkv, page), float("nan"), device="cuda"), torch.full((F, Hkv, page), -1, dtype=torch.int32, device="cuda")) for _ in range(layers)]
    rope = lla.rotary_table(d)
    known = [[[{} for _ in range(Hkv)] for _ in range(S)] for _ in range(layers)]        # position: (score, how far it may be off)
    total, f64 = np.zeros(S, int), lambda t: t.double().cpu().numpy()  # noqa: E731
    for new in [[60, 33, 5, 20], [1, 1, 1, 1], [30, 0, 100, 2], [1, 1, 1, 0], [1, 7, 1, 1], [3, 120, 1, 9], [1, 1, 0, 1], [0, 2, 1, 1], [1, 1, 1, 1]]:
        T, most = sum(new), max(new)
        plan = lla.paged_plan(kv, _i32(new), table, free, count, page, T + 2, kv_lens=kv, free_left=count)
        assert plan.granted.tolist() == [1] * S
        lens, cu, tb = kv.tolist(), plan.cu_q.tolist(), table.cpu().numpy()
        for l in range(layers):
            q0, k0, r0, v = (torch.randn(T + 2, h, d, device="cuda").to(dt) for h in (Hq, Hkv, Hq, Hkv))
            q, k, r = lla.rotary((q0, k0, r0), plan.positions, rope, eps=1e-6, cu_q=plan.cu_q, shift=drop)
            kc, vc = caches[l]
            lla.paged_append(k, v, plan.slots, kc, vc)
            lse = torch.empty(T + 2, Hq, device="cuda")
            lla.paged_parallax(q, r * d ** -0.5, kc, vc, table, plan.cu_q, kv, tau, most, lse=lse)
            scores, positions = state[l]
            lla.paged_weigh(q, lse, kc, scores, table, plan.cu_q, kv, tau, most, positions=positions, dropped=drop, decay=decay,
                            granted=plan.granted)
            torch.cuda.synchronize()
            qh, kh, lh = f64(q), f64(kc), f64(lse)
            weights = paged_weigh_ref(qh, lh, kh, np.zeros(scores.shape), tb, cu, lens, tau)[2]
            # |q| and |k| are at most sqrt(d) after the norm, and a rounding more
            rel = U * ((d + 30) * tau * d * 1.01 + 3 * np.abs(lh[:T]).max(initial=0.0) + most * (Hq // Hkv) + 32)
            got, pos = f64(scores), positions.cpu().numpy()
            for s in range(S):
                for h in range(Hkv):
                    mine, here = known[l][s][h], {}
                    for j in range(lens[s]):
                        at = tb[s, j // page], h, j % page
                        p, fresh = int(pos[at]), j >= lens[s] - new[s]
                        assert p not in here and (p == total[s] + j - (lens[s] - new[s]) if fresh else p in mine)
                        if new[s] == 0:
                            here[p] = mine[p]
                        else:
                            old, off = (0.0, 0.0) if fresh or decay == 0 else mine[p]
                            ref = decay * old + weights[at]
                            here[p] = ref, decay * off + rel * weights[at] + 2 * U * ref + 1e-37
                        assert abs(got[at] - here[p][0]) <= here[p][1]
                    assert set(here) == set(mine) | set(range(total[s], total[s] + new[s]))
                    known[l][s][h] = here
        total += new
        for l in range(layers):
            scores, positions = state[l]
            before, pos = scores.cpu().numpy().copy(), positions.cpu().numpy().copy()
            want = paged_evict_ref(before, tb, lens, bound, page, Hkv, pos, drop.tolist(), sinks, recent)
            lla.paged_evict(scores, *caches[l], table, kv, keep, positions=positions, dropped=drop, sinks=sinks, recent=recent)
            after, moved = scores.cpu().numpy(), positions.cpu().numpy()
            for (s, h), source in want.items():
                stay = {}
                for j, x in enumerate(source):
                    at, frm = (tb[s, j // page], h, j % page), (tb[s, x // page], h, x % page)
                    assert moved[at] == pos[frm] and after[at] == before[frm]
                    stay[int(pos[frm])] = known[l][s][h][int(pos[frm])]
                assert len(stay) == min(lens[s], bound[s])
                known[l][s][h] = stay
        lla.paged_trim(kv, keep, table, free, count, page, dropped=drop, new_lens=kv, new_dropped=drop, free_left=count)
        torch.cuda.synchronize()
        lla.lla_sync_status()
        assert kv.tolist() == [min(a, b) for a, b in zip(total.tolist(), bound)] and (kv + drop).tolist() == total.tolist()
        held = [x for s in range(S) for x in table[s, : -(-int(kv[s]) // page)].tolist()]
        assert sorted(held + free.tolist()[: int(count)]) == list(range(F))
