"""Bounded caches on the GPU: attention weights summed into scores, eviction, trimming, against oracle/cache_ref.py.

Eviction and trimming are exact.  A score's tolerance, u = 2^-24: a weight exp(tau q.k - lse) has a logit within
(d + 16) u tau sum |q_c k_c| (d fp32 sums, the products exact or within 12 u as three of 11 bits, the scale's rounding), the scaled
lse's rounding and the difference's within 3 u |lse| + u |logit|, the exponential within 2^-22; the sum of R weights is within
R u.  All of it is relative to the sum of the weights; the decayed old score and its sum add 2 u of it.
"""
import numpy as np
import pytest
import torch

import local_linear_attention_flashlla_gb300 as lla
from oracle.cache_ref import paged_evict_ref, paged_trim_ref, paged_weigh_ref, rotary_ref, turn_angles
from oracle.paged_ref import paged_parallax_ref
from test_gpu_paged import DT, KINDS, Case, _i32
from test_gpu_paged_lse import lse_ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


# ------------------------------------------------------------------------------------------ weigh
class Weigh:
    """A Case with lse, scores and positions; rows of no sequence hold NaN in q and lse."""

    def __init__(self, c, seed=0):
        self.c, T = c, c.q.shape[0]
        rng = np.random.default_rng(seed)
        lse = lse_ref(c)
        self.lse = torch.tensor(lse, dtype=torch.float32)
        c.q[int(c.cu[-1]):] = float("nan")
        self.scores = torch.tensor(rng.random((c.P, c.Hkv, c.page)) * 3, dtype=torch.float32)
        self.positions = torch.full((c.P, c.Hkv, c.page), -9, dtype=torch.int32)
        self.dropped = rng.integers(0, 1000, len(c.kv))
        assert T == len(lse)

    def device(self):
        c = self.c
        return dict(q=c.q.cuda(), lse=self.lse.cuda(), k_cache=c.kc.cuda(), block_table=_i32(c.table), cu_q=_i32(c.cu), kv_lens=_i32(c.kv),
                    tau=c.tau, max_new=max(max(c.new), 1), causal=c.causal, dropped=_i32(self.dropped))

    def check(self, got, positions, decay=1.0, last=0, before=None):
        c = self.c
        ref, ref_pos, mag = paged_weigh_ref(c.q.double().numpy(), self.lse.double().numpy(), c.kc.double().numpy(),
                                            self.scores.double().numpy(), c.table, c.cu, c.kv, c.tau, decay, last, c.causal,
                                            self.positions.numpy(), self.dropped)
        got = got.double().cpu().numpy()
        written = np.zeros(got.shape, bool)
        for s, L in enumerate(c.kv):
            if c.new[s]:
                for j in range(L):
                    written[c.table[s, j // c.page], :, j % c.page] = True
        untouched = (self.scores if before is None else before).double().numpy()
        assert np.array_equal(got[~written], untouched[~written])
        logit = c.tau * c.scale * c.d * c.knorm
        finite = self.lse[torch.isfinite(self.lse)].abs()
        most = max(min(n, last) if last else n for n in c.new) * (c.Hq // c.Hkv)
        rel = U * ((c.d + 30) * logit + 3 * (float(finite.max()) if finite.numel() else 0.0) + most + 32)
        tol = rel * mag + 2 * U * np.abs(ref) + 1e-37
        worst = (np.abs(got - ref) / tol)[written]
        assert worst.size == 0 or worst.max() <= 1.0, worst.max()
        assert np.array_equal(positions.cpu().numpy(), ref_pos)

    def run(self, decay=1.0, last=0, **kw):
        pos = self.positions.cuda()
        scores = self.scores.cuda()
        got = lla.paged_weigh(**{**self.device(), **kw}, scores=scores, positions=pos, decay=decay, last=last)
        torch.cuda.synchronize()
        lla.lla_sync_status()
        assert got is scores
        self.check(got, pos, decay, last)
        before = torch.full_like(self.scores, -3.0)
        out, pos2 = before.cuda(), self.positions.cuda()
        assert lla.paged_weigh(**{**self.device(), **kw}, scores=self.scores.cuda(), positions=pos2, decay=decay, last=last, out=out) is out
        self.check(out, pos2, decay, last, before)
        return got


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("bf16", 16), ("fp32", 128), ("fp32", 64),
                                     ("fp32", 32), ("fp32", 16)])
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("G,Hkv,page", [(1, 3, 16), (4, 2, 64), (3, 1, 8), (16, 1, 128)])
def test_weigh(lla_gpu, dtype, d, kind, G, Hkv, page):
    new, kv = KINDS[kind]
    Weigh(Case(new, kv, G * Hkv, Hkv, d, page, dtype, pad=2, wide=3)).run(decay=0.75)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 32)])
@pytest.mark.parametrize("last", [1, 5, 33, 1000])
@pytest.mark.parametrize("new,kv", [([1, 200, 0, 40], [90, 200, 9, 700]), ([300], [300])])
def test_weigh_by_the_last_tokens(lla_gpu, dtype, d, last, new, kv):
    Weigh(Case(new, kv, 6, 2, d, 16, dtype)).run(last=last)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 32)])
@pytest.mark.parametrize("new,kv", [([5, 40, 1], [77, 1, 130]), ([1, 1], [500, 33]), ([300], [129])])
@pytest.mark.parametrize("last,decay", [(0, 1.0), (7, 0.0)])
def test_weigh_cross_attention(lla_gpu, dtype, d, new, kv, last, decay):
    Weigh(Case(new, kv, 4, 2, d, 16, dtype, causal=False)).run(last=last, decay=decay)


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (32, "fp32")])
@pytest.mark.parametrize("new,kv", [([1, 1, 1], [0, 5, 0]), ([20, 3, 40, 2], [4, 0, 39, 0]), ([0, 1, 0], [3, 4, 0]), ([200, 3], [70, 5])])
@pytest.mark.parametrize("last", [0, 2])
def test_weigh_rows_without_keys(lla_gpu, new, kv, last, d, dtype):
    Weigh(Case(new, kv, 4, 2, d, 16, dtype, pad=3)).run(last=last)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("fp32", 64)])
@pytest.mark.parametrize("new,G", [([1], 2), ([7], 4), ([40], 1), ([40], 5), ([300], 2), ([129], 8)])
def test_weigh_one_long_sequence(lla_gpu, dtype, d, new, G):
    """Few tiles and many rows: tiles that several CTAs share, and their join."""
    Weigh(Case(new, [3001], G, 1, d, 32, dtype)).run(decay=0.5)
    Weigh(Case(new, [450], G, 1, d, 32, dtype)).run(decay=0.5)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp32", 32)])
@pytest.mark.parametrize("most", [1, 3, 40])
def test_weigh_more_sequences_than_threads(lla_gpu, dtype, d, most):
    rng = np.random.default_rng(most)
    S = 700 if most == 1 else 300
    new = rng.integers(0, most + 1, S)
    kv = new + rng.integers(0, 60, S)
    Weigh(Case(new, kv, 2, 1, d, 8, dtype, pad=9)).run()


def test_weigh_large_logits_and_rows_of_nothing(lla_gpu):
    w = Weigh(Case([3, 150], [90, 300], 4, 2, 128, 16, scale=20.0))
    w.lse[1], w.lse[20, 2] = float("-inf"), float("-inf")
    w.run()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 32)])
@pytest.mark.parametrize("new,kv", [([30, 45], [200, 70]), ([200], [300]), ([3, 1], [90, 5])])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_weigh_nan_and_infinity_in_masked_places(lla_gpu, dtype, d, new, kv, bad):
    """A key that only the last token sees, and a row without weights (lse -inf), hold NaN or infinity; slots behind the lengths hold
    NaN already.  Every other score is as if they did not."""
    w = Weigh(Case(new, kv, 2, 1, d, 16, dtype))
    c = w.c
    w.lse[0] = -float("inf")
    clean = lla.paged_weigh(**w.device(), scores=w.scores.cuda())
    args = w.device()
    args["q"][0] = bad
    page, at = int(c.table[0, (kv[0] - 1) // 16]), (kv[0] - 1) % 16
    args["k_cache"][page, :, at] = bad
    pos = w.positions.cuda()
    got = lla.paged_weigh(**args, scores=w.scores.cuda(), positions=pos)
    torch.cuda.synchronize()
    lla.lla_sync_status()
    alone = torch.isnan(got) | torch.isinf(got)
    alone[page, :, at] = False
    assert not alone.any() and not torch.equal(got[page, :, at], clean[page, :, at])
    got[page, :, at] = clean[page, :, at]
    w.check(got, pos)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 32)])
@pytest.mark.parametrize("new,ctx,free", [([1, 1, 1, 1], [31, 16, 40, 32], 1), ([20, 90, 3, 30], [10, 50, 13, 200], 4), ([50, 1], [64, 64], 0)])
def test_weigh_leaves_refused_sequences_alone(lla_gpu, monkeypatch, dtype, d, new, ctx, free):
    """A plan that runs out of pages: refused sequences keep the scores and positions of what they have cached; the others' are as
    in a call without them."""
    page, Hq, Hkv, S = 16, 4, 2, len(new)
    held = [-(-n // page) for n in ctx]
    ids = np.random.default_rng(d).permutation(sum(held) + max(free, 1))
    table, at = np.full((S, 20), -1), 0
    for s in range(S):
        table[s, :held[s]] = ids[at:at + held[s]]
        at += held[s]
    tb = _i32(table)
    pl = lla.paged_plan(_i32(ctx), _i32(new), tb, _i32(ids[at:at + max(free, 1)]), _i32([free]), page, sum(new))
    granted = pl.granted.tolist()
    assert 0 in granted
    gen = torch.Generator().manual_seed(d)
    P, T = len(ids), sum(new)
    kc, q = (torch.randn(sh, generator=gen).to(DT[dtype]).cuda() for sh in ((P, Hkv, page, d), (T, Hq, d)))
    lse, old = torch.rand((T, Hq), generator=gen).cuda() + 5, torch.rand((P, Hkv, page), generator=gen).cuda()
    args = dict(block_table=tb, cu_q=pl.cu_q, kv_lens=pl.kv_lens, tau=d ** -0.5, max_new=max(new), decay=0.5)
    keep = [s for s in range(S) if granted[s]]
    want, want_pos = old.clone(), torch.full((P, Hkv, page), -7, dtype=torch.int32, device="cuda")
    if keep:
        cu = pl.cu_q.tolist()
        rows = torch.cat([torch.arange(cu[s], cu[s + 1]) for s in keep]).cuda()
        lla.paged_weigh(q[rows], lse[rows], kc, want, tb[keep], _i32(np.concatenate([[0], np.cumsum([new[s] for s in keep])])),
                        pl.kv_lens[keep], d ** -0.5, max(new), positions=want_pos, decay=0.5)
    for way in (None, False):
        if way is False:
            monkeypatch.setattr(lla, "_BIND", False)
        scores, pos = old.clone(), torch.full_like(want_pos, -7)
        lla.paged_weigh(q, lse, kc, scores, positions=pos, granted=pl.granted, **args)
        torch.cuda.synchronize()
        lla.lla_sync_status()
        for s in range(S):
            for c in range(held[s]):
                if not granted[s]:
                    assert torch.equal(scores[table[s, c]], old[table[s, c]]) and (pos[table[s, c]] == -7).all()
        # a weight's sum may be cut elsewhere: 200 rows' fp32 sums
        assert torch.equal(pos, want_pos) and ((scores - want).abs() <= 256 * U * want.abs()).all()
    with pytest.raises(lla.LLAError):
        lla.paged_weigh(q, lse, kc, scores, granted=pl.granted[:1], **args)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp32", 32)])
@pytest.mark.parametrize("new,kv", [([1, 1, 1], [5, 70, 300]), ([40, 90], [60, 150])])
def test_weigh_strided_rows_and_interleaved_caches(lla_gpu, dtype, d, new, kv):
    w = Weigh(Case(new, kv, 4, 2, d, 16, dtype))
    a = w.run()
    both = torch.stack([w.c.kc, w.c.vc], 1).cuda()
    wide = torch.randn(len(w.c.q), 7, d).to(w.c.q.dtype)
    wide[:, 2:6] = w.c.q
    assert torch.equal(a, w.run(k_cache=both[:, 0], q=wide.cuda()[:, 2:6]))
    odd = torch.randn(len(w.c.q), 4 * d + 1).to(w.c.q.dtype)[:, 1:]             # rows that are copied
    odd.copy_(w.c.q.reshape(len(odd), -1))
    assert torch.equal(a, w.run(q=odd.cuda().reshape(len(odd), 4, d)))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 32)])
@pytest.mark.parametrize("new,kv", [([1], [4000]), ([1] * 40, [300] * 40), ([500, 3], [900, 40])])
def test_weigh_same_bits_every_run_and_with_any_workspace(lla_gpu, dtype, d, new, kv):
    w = Weigh(Case(new, kv, 4, 2, d, 16, dtype))
    a = w.run()
    size = lla.lla_paged_weigh_workspace_size(0 if dtype == "bf16" else 1, 1, 1, 4, 2, d, 16, 1, max(new))
    for fill in (0, 255):
        ws = torch.full((size + 64,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(a, w.run(workspace=ws))
    w.run(max_new=max(new) + 500)              # larger than needed: another kernel may serve it, in another order of the sums


def test_weigh_captured_and_replayed_with_other_lengths(lla_gpu):
    """A captured call follows the lengths on the device; two graphs and an eager call on one stream share nothing."""
    d, S, most = 128, 5, 70
    cases = [Weigh(Case(n, k, 4, 2, d, 16, pad=most * S - sum(n))) for n, k in
             (([70, 1, 0, 33, 9], [300, 40, 20, 33, 500]), ([1, 1, 1, 1, 1], [30, 400, 2, 77, 500]), ([0, 70, 70, 0, 2], [0, 70, 300, 0, 9]))]
    P, W = max(w.c.P for w in cases), max(w.c.table.shape[1] for w in cases)

    def fields(w):
        f = w.device()
        table, kc = torch.full((S, W), -1, dtype=torch.int32), torch.full((P, 2, 16, d), float("nan"), dtype=torch.bfloat16)
        sc, po = torch.zeros(P, 2, 16), torch.full((P, 2, 16), -9, dtype=torch.int32)
        table[:, :w.c.table.shape[1]] = torch.tensor(w.c.table)
        kc[:w.c.P], sc[:w.c.P] = w.c.kc, w.scores
        return {**f, "block_table": table.cuda(), "k_cache": kc.cuda(), "scores": sc.cuda(), "positions": po.cuda(), "max_new": most}

    live = [fields(cases[0]), fields(cases[1])]
    graphs = []
    for f in live:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lla.paged_weigh(**f, decay=0.5)
        graphs.append(g)
    for i, w in enumerate(cases + cases[::-1]):
        f = live[i % 2]
        for k, v in fields(w).items():
            if torch.is_tensor(v):
                f[k].copy_(v)
        eager = fields(cases[(i + 1) % 3])
        graphs[i % 2].replay()
        lla.paged_weigh(**eager, decay=0.5)
        torch.cuda.synchronize()
        w.check(f["scores"][:w.c.P], f["positions"][:w.c.P], 0.5)
        e = cases[(i + 1) % 3]
        e.check(eager["scores"][:e.c.P], eager["positions"][:e.c.P], 0.5)
    lla.lla_sync_status()


def test_weigh_two_calls_at_once(lla_gpu):
    w = Weigh(Case([200, 3], [900, 40], 4, 2, 128, 16))
    want = w.run()
    side = torch.cuda.Stream()
    f, g = ({**w.device(), "scores": w.scores.cuda()} for _ in range(2))
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        f["scores"].copy_(w.scores)
        side.wait_stream(torch.cuda.current_stream())
        a = lla.paged_weigh(**f, stream=side)
        b = lla.paged_weigh(**{**g, "scores": w.scores.cuda()})
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want)


def test_weigh_and_evict_past_32_bit_offsets(lla_gpu):
    """A bf16 cache of 9 GB whose last pages are one sequence's."""
    page, Hkv, d = 64, 8, 128
    P = (1 << 32) // (page * Hkv * d) + 2
    kc = torch.zeros(P, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    scores, pos = torch.zeros(P, Hkv, page, device="cuda"), torch.full((P, Hkv, page), -1, dtype=torch.int32, device="cuda")
    small = torch.randn(2, Hkv, page, d, device="cuda").bfloat16()
    kc[P - 2:] = small
    q = torch.randn(1, Hkv, d, device="cuda").bfloat16()
    table, L = _i32([[P - 1, P - 2]]), 100
    lse = torch.randn(1, Hkv, device="cuda") + 5
    lla.paged_weigh(q, lse, kc, scores, table, _i32([0, 1]), _i32([L]), 0.1, 1, positions=pos)
    near, npos = torch.zeros(2, Hkv, page, device="cuda"), torch.full((2, Hkv, page), -1, dtype=torch.int32, device="cuda")
    lla.paged_weigh(q, lse, small, near, _i32([[1, 0]]), _i32([0, 1]), _i32([L]), 0.1, 1, positions=npos)
    torch.cuda.synchronize()
    assert torch.equal(scores[P - 2:], near) and torch.equal(pos[P - 2:], npos) and near.count_nonzero() == L * Hkv
    assert scores.count_nonzero() == L * Hkv
    vc = kc.clone()
    lla.paged_evict(scores, kc, vc, table, _i32([L]), _i32([30]))
    sv = small.clone()
    lla.paged_evict(near, small, sv, _i32([[1, 0]]), _i32([L]), _i32([30]))
    torch.cuda.synchronize()
    assert torch.equal(kc[P - 2:], small) and torch.equal(vc[P - 2:], sv) and torch.equal(scores[P - 2:], near)
    lla.lla_sync_status()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 32)])
@pytest.mark.parametrize("new", [[1, 1], [30, 80]])
def test_weigh_bad_lengths_and_pages_are_cut_and_reported(lla_gpu, dtype, d, new):
    w = Weigh(Case(new, [90, 130], 4, 2, d, 16, dtype))
    for bad in (dict(kv_lens=_i32([90, 5000])), dict(kv_lens=_i32([-4, 130])), dict(cu_q=_i32([0, new[0], 4000])), dict(cu_q=_i32([3, 1, 2])),
                dict(max_new=max(new) - 1) if max(new) > 1 else dict(cu_q=_i32([-1, 1, 2])),
                dict(block_table=_i32(np.where(w.c.table == w.c.table[1, 2], 10 ** 6, w.c.table))),
                dict(block_table=_i32(np.where(w.c.table == w.c.table[0, 1], -1, w.c.table)))):
        lla.paged_weigh(**{**w.device(), **bad}, scores=w.scores.cuda())
        with pytest.raises(lla.LLAError) as e:
            lla.lla_sync_status()
        assert e.value.status == lla.LLA_ERR_INVALID_ARG
    w.run()


def test_weigh_binding_refusals(lla_gpu):
    w = Weigh(Case([1, 2], [9, 30], 4, 2, 64, 16))
    f = {**w.device(), "scores": w.scores.cuda()}
    for bad in (dict(q=f["q"].float()), dict(q=f["q"][:, :3]), dict(q=f["q"][0]), dict(lse=f["lse"][:, :2]), dict(lse=f["lse"].double()),
                dict(scores=f["scores"][:2]), dict(scores=f["scores"].half()), dict(out=f["scores"][:, :1]), dict(positions=f["scores"]),
                dict(dropped=f["dropped"].long()), dict(block_table=f["block_table"][0]), dict(cu_q=f["cu_q"][:2]), dict(kv_lens=f["kv_lens"].cpu()),
                dict(tau=0.0), dict(decay=-1.0), dict(last=-2), dict(last=2 ** 32), dict(max_new=0), dict(max_new=2 ** 32 + 5), dict(k_cache=f["k_cache"].cpu()), dict(k_cache=f["k_cache"].half()),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(lla.LLAError):
            lla.paged_weigh(**{**f, **bad})
            pytest.fail(f"not refused: {list(bad)}")


# ------------------------------------------------------------------------------------------ evict
class Evict:
    def __init__(self, kv, keep, Hkv, d, page, dtype, kind="random", sinks=0, recent=0, seed=0, wide=0):
        rng = np.random.default_rng(seed)
        self.kv, self.keep, self.Hkv, self.page, self.sinks, self.recent = kv, keep, Hkv, page, sinks, recent
        need = [-(-n // page) for n in kv]
        self.P = sum(need) + 2
        ids, at = rng.permutation(self.P), 0
        self.table = np.full((len(kv), max(max(need), 1) + wide), -5)
        for s, n in enumerate(need):
            self.table[s, :n] = ids[at:at + n]
            at += n
        sc = np.exp(2 * rng.standard_normal((self.P, Hkv, page))).astype(np.float32)
        if kind == "ties":
            sc = rng.integers(0, 4, sc.shape).astype(np.float32) * np.where(rng.random(sc.shape) < 0.5, 1.0, -1.0).astype(np.float32)
        elif kind == "equal":
            sc[:] = 1.5
        elif kind == "odd":
            odd = np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, -1e-42, 3.0], np.float32)
            sc = np.where(rng.random(sc.shape) < 0.6, odd[rng.integers(0, len(odd), sc.shape)], sc).astype(np.float32)
        elif kind == "close":
            sc = (np.float32(1.0) + rng.integers(0, 40, sc.shape) * np.float32(2.0 ** -23)).astype(np.float32)
        self.scores = torch.tensor(sc)
        self.dropped = rng.integers(0, 50, len(kv))
        self.positions = torch.full((self.P, Hkv, page), -1, dtype=torch.int32)
        for s, n in enumerate(kv):
            for h in range(Hkv):
                p = np.sort(rng.permutation(int(self.dropped[s]) + n)[:n])
                rng.shuffle(p[: n // 2])
                j = np.arange(n)
                self.positions[self.table[s, j // page], h, j % page] = torch.tensor(p, dtype=torch.int32)
        self.kc, self.vc = (torch.tensor(rng.standard_normal((self.P, Hkv, page, d)), dtype=torch.float32).to(DT[dtype]) for _ in range(2))

    def want(self):
        ref = paged_evict_ref(self.scores.numpy(), self.table, self.kv, self.keep, self.page, self.Hkv,
                              self.positions.numpy() if self.sinks or self.recent else None, self.dropped, self.sinks, self.recent)
        k, v, s, p = self.kc.clone(), self.vc.clone(), self.scores.clone(), self.positions.clone()
        for (q, h), source in ref.items():
            to = torch.tensor([j for j, x in enumerate(source) if x != j], dtype=torch.long)
            frm = torch.tensor([x for j, x in enumerate(source) if x != j], dtype=torch.long)
            row = torch.tensor(self.table[q]).long()
            a, b = row[to // self.page], row[frm // self.page]
            for new, old in ((k, self.kc), (v, self.vc), (s, self.scores), (p, self.positions)):
                new[a, h, to % self.page] = old[b, h, frm % self.page]
        return k, v, s, p

    def run(self, positions=True, interleaved=False):
        k, v, s, p = self.want()
        both = torch.stack([self.kc, self.vc], 1).cuda()
        kc, vc = (both[:, 0], both[:, 1]) if interleaved else (self.kc.cuda(), self.vc.cuda())
        sc, pos = self.scores.cuda(), self.positions.cuda()
        kw = dict(positions=pos, dropped=_i32(self.dropped), sinks=self.sinks, recent=self.recent) if positions else {}
        args = _i32(self.table), _i32(self.kv), _i32(self.keep)
        lla.paged_evict(sc, kc, vc, *args, **kw)
        torch.cuda.synchronize()
        lla.lla_sync_status()
        same = lambda a, b: torch.equal(a.cpu().contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))  # noqa: E731
        assert same(kc, k) and same(vc, v) and same(sc, s)
        if positions:
            assert same(pos, p)
        # elsewhere: the kept slots are given, others left
        kc, vc, sc, pos = self.kc.cuda(), self.vc.cuda(), self.scores.cuda(), self.positions.cuda()
        so, po = torch.full_like(sc, 7.0), torch.full_like(pos, 7)
        kw = dict(kw, positions=pos, positions_out=po) if positions else {}
        lla.paged_evict(sc, kc, vc, *args, **kw, scores_out=so)
        torch.cuda.synchronize()
        assert same(kc, k) and same(vc, v) and same(sc, self.scores) and same(pos, self.positions)
        kept = torch.zeros(so.shape, dtype=torch.bool)
        for q, n in enumerate(self.kv):
            j = np.arange(min(n, max(self.keep[q], 0)))
            kept[self.table[q, j // self.page], :, j % self.page] = True
        assert same(so, torch.where(kept, s, torch.full_like(s, 7.0)))
        if positions:
            assert same(po, torch.where(kept, p, torch.full_like(p, 7)))


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "odd", "close"])
@pytest.mark.parametrize("dtype,d,Hkv,page", [("bf16", 128, 3, 16), ("fp32", 128, 1, 64), ("bf16", 16, 2, 8), ("fp32", 32, 5, 256)])
def test_evict(lla_gpu, kind, dtype, d, Hkv, page):
    kv, keep = [0, 1, 7, 40, 513, 1024, 1500, 90, 3000, 33], [4, 1, 3, 0, 512, 1000, 600, 200, 17, -2]
    Evict(kv, keep, Hkv, d, page, dtype, kind).run(positions=False)
    Evict(kv, keep, Hkv, d, page, dtype, kind, sinks=3, recent=20, seed=1, wide=2).run(interleaved=True)


@pytest.mark.parametrize("sinks,recent", [(0, 5), (4, 0), (100, 300), (0, 10 ** 9), (10 ** 9, 0)])
def test_evict_first_and_last_positions(lla_gpu, sinks, recent):
    """More of them than are kept, too: then the lowest slots."""
    Evict([400, 50, 1200], [100, 50, 900], 2, 64, 16, "bf16", sinks=sinks, recent=recent).run()


@pytest.mark.parametrize("S,Hkv", [(1, 1), (1, 3), (9, 8), (60, 8)])
def test_evict_by_clusters_of_every_size(lla_gpu, S, Hkv):
    rng = np.random.default_rng(S)
    kv = rng.integers(100, 700, S)
    Evict(list(kv), list(rng.integers(1, 300, S)), Hkv, 32, 16, "bf16", "ties", 2, 9).run()


@pytest.mark.parametrize("keep", [5, 11000, 13000, 39999])
@pytest.mark.parametrize("kind", ["random", "ties"])
def test_evict_longer_than_shared_memory(lla_gpu, keep, kind):
    Evict([40000], [keep], 1, 16, 64, "bf16", kind, 4, 50).run()
    Evict([300, 20000] * 3, [100, min(keep, 19000)] * 3, 2, 16, 64, "bf16", kind).run(positions=False)


def test_evict_slots_without_a_page_and_lengths_beyond_the_table(lla_gpu):
    e = Evict([64, 100], [20, 50], 2, 64, 16, "bf16")
    for table, kv in ((np.where(e.table == e.table[0, 1], -1, e.table), [64, 100]), (np.where(e.table == e.table[1, 3], 10 ** 6, e.table), [64, 100]),
                      (e.table, [64, 10 ** 6])):
        kc, vc, sc = e.kc.cuda(), e.vc.cuda(), e.scores.cuda()
        lla.paged_evict(sc, kc, vc, _i32(table), _i32(kv), _i32(e.keep))
        with pytest.raises(lla.LLAError) as x:
            lla.lla_sync_status()
        assert x.value.status == lla.LLA_ERR_INVALID_ARG
    kc = e.kc.cuda()
    lla.paged_evict(e.scores.cuda(), kc, e.vc.cuda(), _i32(e.table), _i32([-3, 40]), _i32(e.keep))
    with pytest.raises(lla.LLAError):
        lla.lla_sync_status()
    assert torch.equal(kc.cpu(), e.kc)                          # nothing to evict


def test_evict_captured_with_other_lengths_and_on_a_stream(lla_gpu):
    kv, keep = [300, 40, 900], [100, 40, 256]
    e = Evict(kv, keep, 2, 64, 16, "bf16", sinks=2, recent=5)
    kc, vc, sc, pos = e.kc.cuda(), e.vc.cuda(), e.scores.cuda(), e.positions.cuda()
    lens, left, table, drop = _i32([0, 0, 0]), _i32([0, 0, 0]), _i32(e.table), _i32(e.dropped)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lla.paged_evict(sc, kc, vc, table, lens, left, positions=pos, dropped=drop, sinks=2, recent=5)
    for a, b in ((kv, keep), ([300, 40, 70], [299, 0, 60]), ([17, 0, 900], [16, 5, 1])):
        e.kv, e.keep = a, b
        for t, x in ((kc, e.kc), (vc, e.vc), (sc, e.scores), (pos, e.positions)):
            t.copy_(x)
        lens.copy_(_i32(a))
        left.copy_(_i32(b))
        g.replay()
        torch.cuda.synchronize()
        for t, x in zip((kc, vc, sc, pos), e.want()):
            assert torch.equal(t.cpu(), x)
    side = torch.cuda.Stream()
    for t, x in ((kc, e.kc), (vc, e.vc), (sc, e.scores), (pos, e.positions)):
        t.copy_(x)
    side.wait_stream(torch.cuda.current_stream())
    lla.paged_evict(sc, kc, vc, table, lens, left, positions=pos, dropped=drop, sinks=2, recent=5, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(kc.cpu(), e.want()[0])
    lla.lla_sync_status()


def test_evict_binding_refusals(lla_gpu):
    e = Evict([30], [9], 2, 64, 16, "bf16")
    f = dict(scores=e.scores.cuda(), k_cache=e.kc.cuda(), v_cache=e.vc.cuda(), block_table=_i32(e.table), kv_lens=_i32([30]), keep=_i32([9]))
    for bad in (dict(scores=f["scores"].double()), dict(scores=f["scores"][:1]), dict(scores_out=f["scores"].cpu()), dict(positions=f["scores"]),
                dict(v_cache=f["v_cache"].float()), dict(v_cache=f["v_cache"][:, :1]), dict(block_table=f["block_table"][0]), dict(keep=f["keep"].long()),
                dict(keep=_i32([9, 9])), dict(kv_lens=f["kv_lens"].cpu()), dict(sinks=1), dict(recent=1), dict(recent=-1), dict(sinks=2 ** 32), dict(recent=-2 ** 32), dict(dropped=f["scores"]),
                dict(positions_out=torch.zeros_like(f["scores"], dtype=torch.int32))):
        with pytest.raises(lla.LLAError):
            lla.paged_evict(**{**f, **bad})
            pytest.fail(f"not refused: {list(bad)}")


# ------------------------------------------------------------------------------------------- trim
@pytest.mark.parametrize("S,page,hi,cap,count", [(1, 8, 0, 4, 2), (1, 256, 5000, 40, 0), (7, 16, 400, 300, 11), (64, 64, 4200, 9000, 1),
                                                 (65, 16, 900, 9000, 5), (700, 8, 300, 99000, 77), (8192, 16, 200, 99000, 0), (33, 16, 700, 30, 3),
                                                 (100, 16, 700, 200, 0), (5, 8, 90, 100, -3), (5, 8, 90, 20, 99)])
def test_trim(lla_gpu, S, page, hi, cap, count):
    rng = np.random.default_rng(S + page)
    kv, keep = rng.integers(0, hi + 1, S), rng.integers(-3, hi + 2, S)
    W = max(-(-hi // page), 1)
    table = rng.integers(0, 10 ** 6, (S, W))
    table[rng.random((S, W)) < 0.05] = -1
    free, dropped = rng.integers(0, 1000, cap), rng.integers(0, 1000, S)
    ref = paged_trim_ref(kv, keep, table, free, count, page, dropped)
    f, n, tb = _i32(free), _i32([count]), _i32(table)
    r = lla.paged_trim(_i32(kv), _i32(keep), tb, f, n, page, dropped=_i32(dropped))
    torch.cuda.synchronize()
    assert r.kv_lens.tolist() == ref["kv_lens"] and r.dropped.tolist() == ref["dropped"] and r.free_left.tolist() == [ref["free_left"]]
    assert f.tolist() == ref["free_pages"] and np.array_equal(tb.cpu().numpy(), table) and n.tolist() == [count]
    if ref["full"]:
        with pytest.raises(lla.LLAError) as e:
            lla.lla_sync_status()
        assert e.value.status == lla.LLA_ERR_INVALID_ARG
    lla.lla_sync_status()


def test_trim_in_place_in_a_graph_with_the_plan(lla_gpu):
    """Captured: plan a token for every sequence, trim what is beyond its bound: pages go round and none is lost."""
    S, page, W, F = 70, 8, 9, 500
    rng = np.random.default_rng(3)
    kv, keep = _i32([0] * S), _i32(rng.integers(0, 60, S))
    table, free, count, drop = _i32(np.full((S, W), -1)), _i32(rng.permutation(F)), _i32([F]), _i32([0] * S)
    new = _i32(rng.integers(0, 9, S))
    T = int(new.sum())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lla.paged_plan(kv, new, table, free, count, page, T, kv_lens=kv, free_left=count)
        lla.paged_trim(kv, keep, table, free, count, page, dropped=drop, new_lens=kv, new_dropped=drop, free_left=count)
    for step in range(30):
        g.replay()
        torch.cuda.synchronize()
        n, held = int(count), [(-(-L // page)) for L in kv.tolist()]
        ids = free.tolist()[:n] + [x for s, h in enumerate(held) for x in table[s, :h].tolist()]
        assert sorted(ids) == list(range(F))
        assert kv.tolist() == [min(a, b) for a, b in zip((new * (step + 1)).tolist(), keep.tolist())]
        assert (kv + drop).tolist() == (new * (step + 1)).tolist()
    lla.lla_sync_status()


def test_trim_lengths_beyond_the_table_and_refusals(lla_gpu):
    f = dict(kv_lens=_i32([100, -4]), keep=_i32([5, 5]), block_table=_i32([[1, 2], [3, 4]]), free_pages=_i32([0] * 8), free_count=_i32([0]), page_size=16)
    r = lla.paged_trim(**f)
    with pytest.raises(lla.LLAError):
        lla.lla_sync_status()
    assert r.kv_lens.tolist() == [5, 0] and r.dropped.tolist() == [27, 0] and f["free_pages"].tolist()[:1] == [2] and r.free_left.tolist() == [1]
    for bad in (dict(keep=_i32([5])), dict(kv_lens=f["kv_lens"].long()), dict(block_table=_i32([1, 2])), dict(block_table=_i32([[1, 2]])),
                dict(free_pages=f["free_pages"].cpu()), dict(free_count=_i32([0, 0])), dict(page_size=12), dict(page_size=2 ** 32 + 16), dict(dropped=_i32([1])),
                dict(new_lens=_i32([1])), dict(new_dropped=f["kv_lens"].float()), dict(free_left=_i32([]))):
        with pytest.raises(lla.LLAError):
            lla.paged_trim(**{**f, **bad})
            pytest.fail(f"not refused: {list(bad)}")


# --------------------------------------------------------------------------------------- together
@pytest.mark.parametrize("dtype,d,Hq,Hkv", [("bf16", 128, 4, 2), ("bf16", 64, 2, 2), ("fp32", 32, 3, 1)])
def test_serving_with_bounded_caches(lla_gpu, dtype, d, Hq, Hkv):
    """Prompts, chunks and single tokens of three sequences through two layers: rotated, cached, attended, weighed, evicted,
    trimmed.  After every step each slot must hold the rotated key and the value of the position it claims, the attention
    equals the definition on what is cached, and no page is lost."""
    torch.manual_seed(d)
    page, S, layers, W, F, dt = 16, 3, 2, 20, 64, DT[dtype]
    table, free, count = _i32(np.full((S, W), -1)), _i32(np.arange(F)), _i32([F])
    kv, drop, keep, tau = _i32([0] * S), _i32([0] * S), _i32([40, 90, 64]), d ** -0.5
    caches = [[torch.full((F, Hkv, page, d), float("nan"), device="cuda", dtype=dt) for _ in range(2)] for _ in range(layers)]
    state = [(torch.full((F, Hkv, page), float("nan"), device="cuda"), torch.full((F, Hkv, page), -1, dtype=torch.int32, device="cuda")) for _ in range(layers)]
    rope, gain = lla.rotary_table(d, scaling="linear", factor=2.0), 1 + 0.2 * torch.randn(d, device="cuda")
    seen = [[([], []) for _ in range(S)] for _ in range(layers)]          # every token's rotated key and value
    total = np.zeros(S, int)
    for step, new in enumerate([[60, 33, 5], [1, 1, 1], [30, 0, 100], [1, 1, 1], [1, 7, 1], [3, 64, 1], [1, 1, 0], [1, 1, 1]]):
        T, pad = sum(new), 2
        plan = lla.paged_plan(kv, _i32(new), table, free, count, page, T + pad, kv_lens=kv, free_left=count)
        assert plan.granted.tolist() == [1] * S
        for l in range(layers):
            fused = torch.randn(T + pad, (2 * Hq + 2 * Hkv) * d, device="cuda").to(dt)
            q0, k0, r0, v = (t.reshape(T + pad, -1, d) for t in fused.split([Hq * d, Hkv * d, Hq * d, Hkv * d], 1))
            q, k, r = lla.rotary((q0, k0, r0), plan.positions, rope, gain=(None, gain, None), eps=1e-6, cu_q=plan.cu_q, shift=drop)
            r *= d ** -0.5
            kc, vc = caches[l]
            lla.paged_append(k, v, plan.slots, kc, vc)
            lse = torch.empty(T + pad, Hq, device="cuda")
            out = lla.paged_parallax(q, r, kc, vc, table, plan.cu_q, kv, tau, max(new), lse=lse)
            lla.paged_weigh(q, lse, kc, state[l][0], table, plan.cu_q, kv, tau, max(new), positions=state[l][1], dropped=drop)
            torch.cuda.synchronize()
            cu, lens = plan.cu_q.tolist(), kv.tolist()
            f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
            ref, mag, _ = paged_parallax_ref(f64(q), f64(r), f64(kc), f64(vc), table.cpu().numpy(), cu, lens, tau)
            assert (np.abs(f64(out)[:T] - ref[:T]) <= (2.0 ** -7 if dtype == "bf16" else 2.0 ** -15) * (np.abs(ref) + 2 * mag)[:T]).all()
            for s in range(S):
                at = total[s] + np.arange(new[s])
                ang = turn_angles(at, rope.turns.tolist())[:, None]
                want = rotary_ref(f64(k0[cu[s]:cu[s + 1]]), ang, f64(gain), 1e-6)
                got = f64(k[cu[s]:cu[s + 1]])
                assert np.abs(got - want).max(initial=0) <= 2.0 ** -7 * 6
                seen[l][s][0].extend(k[cu[s]:cu[s + 1]].cpu())
                seen[l][s][1].extend(v[cu[s]:cu[s + 1]].cpu())
            # what all rows gave sums to the rows: every weight reached some score, and none that a slot did not have
            weights = state[l][0]
            assert torch.isfinite(weights[table[1, 0].long()]).all() or lens[1] < page
        total += new
        for l in range(layers):
            lla.paged_evict(state[l][0], *caches[l], table, kv, keep, positions=state[l][1], dropped=drop, sinks=2, recent=10)
        lla.paged_trim(kv, keep, table, free, count, page, dropped=drop, new_lens=kv, new_dropped=drop, free_left=count)
        torch.cuda.synchronize()
        lla.lla_sync_status()
        lens, tb = kv.tolist(), table.tolist()
        assert lens == [min(a, b) for a, b in zip(total.tolist(), keep.tolist())] or step > 1
        assert (kv + drop).tolist() == total.tolist()
        held = [x for s in range(S) for x in tb[s][: -(-lens[s] // page)]]
        assert sorted(held + free.tolist()[: int(count)]) == list(range(F))
        for l in range(layers):
            kc, vc = (c.cpu() for c in caches[l])
            pos = state[l][1].cpu()
            for s in range(S):
                for h in range(Hkv):
                    at = [(tb[s][j // page], j % page) for j in range(lens[s])]
                    mine = [int(pos[p, h, i]) for p, i in at]
                    assert len(set(mine)) == len(mine)
                    assert set(range(min(2, lens[s]))) <= set(mine) and set(range(max(total[s] - 10, 0), total[s])) <= set(mine)
                    for (p, i), x in zip(at, mine):
                        assert torch.equal(kc[p, h, i], seen[l][s][0][x][h]) and torch.equal(vc[p, h, i], seen[l][s][1][x][h])


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "odd", "close"])
def test_evict_of_many_heads(lla_gpu, kind):
    """Enough (sequence, key head) pairs for the kernel with small blocks: lengths around its windows' borders, and one beyond
    what it holds in shared memory."""
    rng = np.random.default_rng(5)
    kv = [0, 1, 3, 511, 512, 513, 2047, 2048, 2049, 2560, 4097, 10240, 10241, 12000] + list(rng.integers(1, 300, 66))
    keep = [5, 1, 1, 200, 511, 512, 2046, 1000, 2048, 2049, 4096, 9000, 10240, 11000] + list(rng.integers(0, 200, 66))
    Evict(kv, keep, 8, 16, 16, "bf16", kind, sinks=2, recent=9).run()
    Evict(kv[:8] + kv[14:], keep[:8] + keep[14:], 9, 32, 8, "fp32", kind, seed=3).run(positions=False)


def test_both_ways_of_marshalling_give_the_same_bits(lla_gpu, monkeypatch):
    def calls():
        w = Weigh(Case([3, 40], [90, 300], 4, 2, 64, 16))
        w.run()
        a = w.run(decay=0.5, last=2)
        e = Evict([300, 40], [100, 9], 2, 64, 16, "bf16", "ties", 2, 9)
        e.run(interleaved=True)
        e.sinks = e.recent = 0
        e.run(positions=False)
        f = _i32([0] * 20)
        t = lla.paged_trim(_i32([40, 90]), _i32([10, 0]), _i32([[1, 2, 3, 4, 5, 6]] * 2), f, _i32([3]), 16)
        return a, f, *t

    fast = calls()
    monkeypatch.setattr(lla, "_BIND", False)
    for a, b in zip(fast, calls()):
        assert torch.equal(a, b)
