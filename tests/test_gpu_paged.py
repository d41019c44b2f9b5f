"""Paged-cache operators on the GPU against integer and float64 references (oracle/paged_ref.py).

Planning is exact.  Append is a copy: exact.

Attention tolerances, element by element.  Let mag = (1 + M) sum_j p_j |v_j| + sum_j p_j |t_j - c| |v_j|,
M = max_j |t_j - c| (the reference returns it): a one-pass evaluation with a centre s0 among the row's t
values sums terms of at most that total size, |c - s0| <= M being the factor on the first sum.
* out is rounded once to its type: eps/2 |ref|, eps/2 = 2^-8 for bf16, 2^-24 for fp32.
* products and sums in fp32: (keys + 2 d + 32) 2^-24 relative on every term (the dot products q.k and
  probe.k, the running sums and their rescaling), times 1 + tau |q||k| for the exponent's argument,
  whose absolute error is the logit's.  |q| and |k| are at most sqrt(d) by construction (unit RMS) times
  the scale a test multiplies them by.
* tensor path: the weights p and p (t - s0) enter the value product in bf16: 2^-8 relative each.
These are worst cases; a second check bounds the relative 2-norm of the whole error: independent
roundings of 2^-8 at most, twice (weights and output), stay below 2^-7 for bf16; for fp32 outputs below
8 sqrt(keys + d) 2^-24 (1 + tau |q||k|) of the norm of mag.
"""
import math

import numpy as np
import pytest
import torch

import local_linear_attention_flashlla_gb300 as lla
from oracle.paged_ref import paged_parallax_ref, paged_plan_ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------- plan
def _plan_case(seed, S, page, T_extra, ctx_hi, new_hi, width, count, cap=None):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_hi + 1, S)
    new = rng.integers(0, new_hi + 1, S)
    width = width or -(-(ctx_hi + new_hi) // page) + 1
    held = -(-ctx // page)
    ids = rng.permutation(int(held.sum()) + (cap or 4096))
    table = np.full((S, width), -7)
    at = 0
    for s in range(S):
        h = min(int(held[s]), width)
        table[s, :h] = ids[at:at + h]
        at += h
    free = ids[at:at + (cap or 4096)]
    return ctx, new, table, free, len(free) if count is None else count, max(1, int(new.sum()) + T_extra)


def _check_plan(ctx, new, table, free, count, page, T, got, got_table):
    ref = paged_plan_ref(ctx, new, table, free, count, page, T)
    for name in ("kv_lens", "cu_q", "slots", "positions", "granted"):
        assert np.array_equal(getattr(got, name).cpu().numpy(), np.asarray(ref[name])), name
    assert int(got.free_left) == ref["free_left"]
    assert np.array_equal(got_table.cpu().numpy(), ref["table"])
    return ref


@pytest.mark.parametrize("S,page,extra,ctx_hi,new_hi,width,count", [
    (1, 8, 0, 0, 1, None, None), (1, 256, 3, 5000, 5000, None, None), (7, 16, 0, 40, 40, None, None),
    (64, 64, 0, 4095, 1, None, None), (1025, 16, 5, 300, 3, None, None), (100, 8, 9000, 10, 30, None, None),
    (33, 16, 0, 100, 700, None, 50), (33, 16, 1, 100, 700, None, 0), (40, 8, -200, 60, 20, None, None),
    (20, 8, 4, 90, 90, 9, None), (512, 32, 0, 4000, 250, None, 1500), (8192, 16, 7, 100, 2, None, None),
    (50, 16, 0, 64, 64, None, 100000), (50, 16, 0, 64, 64, None, -5), (3, 8, 20000, 10, 10, None, None),
])
def test_plan(lla_gpu, S, page, extra, ctx_hi, new_hi, width, count):
    ctx, new, table, free, count, T = _plan_case(S + page, S, page, extra, ctx_hi, new_hi, width, count)
    tb = _i32(table)
    got = lla.paged_plan(_i32(ctx), _i32(new), tb, _i32(free), _i32([count]), page, T)
    torch.cuda.synchronize()
    _check_plan(ctx, new, table, free, count, page, T, got, tb)
    lla.lla_sync_status()


def test_plan_negative_lengths_and_missing_pages(lla_gpu):
    ctx, new = np.array([-3, 20, 5, 9]), np.array([4, -2, 0, 3])
    table = np.array([[-1, -1], [1, 2], [3, -1], [-1, 4]])       # sequence 3's first page is missing
    tb = _i32(table)
    got = lla.paged_plan(_i32(ctx), _i32(new), tb, _i32([8, 9]), _i32([2]), 16, 9)
    _check_plan(ctx, new, table, [8, 9], 2, 16, 9, got, tb)
    assert got.slots.tolist()[:4] == [144, 145, 146, 147] and got.slots.tolist()[4:] == [-1] * 5


def test_plan_in_place_decode_loop_in_a_graph(lla_gpu):
    """kv_lens = ctx_lens and free_left = free_count: thirty captured steps continue one another."""
    ctx, new, table, free, count, T = _plan_case(5, 70, 8, 3, 50, 1, 20, None, cap=300)
    new = np.ones_like(new)
    T = len(new) + 3
    c, n, tb, f, k = _i32(ctx), _i32(new), _i32(table), _i32(free), _i32([count])
    out = [torch.empty(T, dtype=torch.int64, device="cuda"), torch.empty(T, dtype=torch.int32, device="cuda")]
    cu, gr = torch.empty(71, dtype=torch.int32, device="cuda"), torch.empty(70, dtype=torch.int32, device="cuda")
    step = lambda: lla.paged_plan(c, n, tb, f, k, 8, T, kv_lens=c, free_left=k, slots=out[0], positions=out[1],  # noqa: E731
                                  cu_q=cu, granted=gr)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    assert c.tolist() == ctx.tolist()
    for _ in range(30):
        ref = paged_plan_ref(ctx, new, table, free, count, 8, T)
        g.replay()
        torch.cuda.synchronize()
        assert c.tolist() == ref["kv_lens"] and k.tolist() == [ref["free_left"]] and gr.tolist() == ref["granted"]
        assert np.array_equal(out[0].cpu().numpy(), ref["slots"]) and np.array_equal(tb.cpu().numpy(), ref["table"])
        ctx, table, count = np.array(ref["kv_lens"]), ref["table"], ref["free_left"]


# ----------------------------------------------------------------------------------------- append
@pytest.mark.parametrize("S,new_hi,count", [(255, 1, None), (256, 3, None), (257, 3, None), (256, 3, 40), (256, 9, None),
                                            (30, 64, None), (31, 70, 20), (1024, 2, None), (1024, 5, 300)])
def test_plan_where_the_block_size_changes(lla_gpu, S, new_hi, count):
    """Up to 256 sequences and 1024 rows a small block plans, beyond either a large one; from 1025 sequences on a thread
    has several."""
    ctx, new, table, free, count, T = _plan_case(S + new_hi, S, 8, 2, 100, new_hi, None, count)
    for rows in {T, max(1024, T), max(1025, T)}:          # more rows than the step's tokens: a padded batch
        tb = _i32(table)
        got = lla.paged_plan(_i32(ctx), _i32(new), tb, _i32(free), _i32([count]), 8, rows)
        torch.cuda.synchronize()
        _check_plan(ctx, new, table, free, count, 8, rows, got, tb)


@pytest.mark.parametrize("dtype,d,Hkv,page,T", [("bf16", 128, 8, 16, 1), ("bf16", 16, 1, 8, 77), ("fp32", 32, 3, 64, 300),
                                                ("bf16", 64, 5, 256, 1000), ("fp32", 128, 2, 32, 4097)])
def test_append(lla_gpu, dtype, d, Hkv, page, T):
    torch.manual_seed(T)
    P = T // page + 4
    both = torch.randn(P, 2, Hkv, page, d, device="cuda").to(DT[dtype])      # keys and values of a page side by side
    before = both.clone()
    kc, vc = both[:, 0], both[:, 1]
    fused = torch.randn(T, 3 * Hkv, d, device="cuda").to(DT[dtype])
    k, v = fused[:, Hkv:2 * Hkv], fused[:, 2 * Hkv:]
    slots = torch.randperm(P * page, device="cuda")[:T]
    slots[torch.rand(T, device="cuda") < 0.2] = -1
    lla.paged_append(k, v, slots, kc, vc)
    torch.cuda.synchronize()
    lla.lla_sync_status()
    ok = slots >= 0
    at = slots[ok]
    before[:, 0][at // page, :, at % page] = k[ok]
    before[:, 1][at // page, :, at % page] = v[ok]
    assert torch.equal(both, before)


def test_append_slot_out_of_range_is_skipped_and_reported(lla_gpu):
    kc, vc = torch.zeros(2, 1, 8, 64, device="cuda"), torch.zeros(2, 1, 8, 64, device="cuda")
    k = torch.ones(3, 1, 64, device="cuda")
    lla.paged_append(k, k, torch.tensor([15, 16, 1 << 40], device="cuda"), kc, vc)
    with pytest.raises(lla.LLAError) as e:
        lla.lla_sync_status()
    assert e.value.status == lla.LLA_ERR_INVALID_ARG
    assert kc.sum().item() == 64 and vc[1, 0, 7].sum().item() == 64
    lla.lla_sync_status()


def test_append_past_32_bit_offsets(lla_gpu):
    """Slots whose element offset lies past 2^32 (a bf16 cache of 9 GB each)."""
    page, Hkv, d = 64, 8, 128
    P = (1 << 32) // (page * Hkv * d) + 2
    kc = torch.zeros(P, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    k = torch.randn(2, Hkv, d, device="cuda").bfloat16()
    lla.paged_append(k, -k, torch.tensor([(P - 1) * page + 3, 5], device="cuda"), kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc[P - 1, :, 3], k[0]) and torch.equal(vc[P - 1, :, 3], -k[0])
    assert torch.equal(kc[0, :, 5], k[1]) and kc[P - 1].count_nonzero() == k[0].count_nonzero()
    # and the attention that reads it: one sequence whose only page is the last one
    for path in (lla.LLA_PATH_AUTO, lla.LLA_PATH_FP32):
        lla.paged_append(k[:1].contiguous(), -k[:1], torch.tensor([(P - 1) * page], device="cuda"), kc, vc)
        q = torch.randn(1, Hkv, d, device="cuda").bfloat16()
        out = lla.paged_parallax(q, torch.zeros_like(q), kc, vc, _i32([[P - 1]]), _i32([0, 1]), _i32([1]), 0.1, 1,
                                 path=path)
        torch.cuda.synchronize()
        assert torch.equal(out[0], -k[0])          # one key: its value, whatever the logit
    lla.lla_sync_status()


# -------------------------------------------------------------------------------------- attention
class Case:
    """Random rows and caches; every cache position that is no sequence's holds NaN."""

    def __init__(self, new, kv, Hq, Hkv, d, page, dtype="bf16", causal=True, pad=0, seed=0, scale=1.0, kshift=0.0,
                 wide=0, probe_scale=None):
        rng = np.random.default_rng(seed + 17 * d + Hq)
        self.new, self.kv, self.causal, self.dtype, self.d, self.page = list(new), list(kv), causal, dtype, d, page
        self.Hq, self.Hkv, self.tau, self.scale = Hq, Hkv, 1.0 / math.sqrt(d), scale
        self.cu = np.concatenate([[0], np.cumsum(new)])
        T = int(self.cu[-1]) + pad
        unit = lambda *sh: (lambda x: x / np.sqrt((x * x).mean(-1, keepdims=True)))(rng.standard_normal(sh))  # noqa: E731
        dt = DT[dtype]
        self.q = torch.tensor(unit(T, Hq, d) * scale, dtype=torch.float32).to(dt)
        self.probe = torch.tensor(unit(T, Hq, d) * (1 / math.sqrt(d) if probe_scale is None else probe_scale),
                                  dtype=torch.float32).to(dt)
        need = [-(-n // page) for n in kv]
        self.P = sum(need) + 3
        ids = rng.permutation(self.P)
        W = max(max(need), 1) + wide
        self.table = np.full((len(kv), W), -1)
        kc = np.full((self.P, Hkv, page, d), np.nan, np.float32)
        vc = kc.copy()
        at = 0
        for s, n in enumerate(kv):
            self.table[s, :need[s]] = ids[at:at + need[s]]
            at += need[s]
            k, v = unit(n, Hkv, d) + kshift, rng.standard_normal((n, Hkv, d))
            for lp in range(need[s]):
                m = min(page, n - lp * page)
                kc[self.table[s, lp], :, :m] = k[lp * page:lp * page + m].transpose(1, 0, 2)
                vc[self.table[s, lp], :, :m] = v[lp * page:lp * page + m].transpose(1, 0, 2)
        self.kc, self.vc = torch.tensor(kc).to(dt), torch.tensor(vc).to(dt)
        self.knorm = 1.0 + abs(kshift)

    def device(self):
        return dict(q=self.q.cuda(), probe=self.probe.cuda(), k_cache=self.kc.cuda(), v_cache=self.vc.cuda(),
                    block_table=_i32(self.table), cu_q=_i32(self.cu), kv_lens=_i32(self.kv), tau=self.tau,
                    max_new=max(max(self.new), 1), causal=self.causal)

    def ref(self, seqs=None):
        return paged_parallax_ref(self.q.double().numpy(), self.probe.double().numpy(), self.kc.double().numpy(),
                                  self.vc.double().numpy(), self.table, self.cu, self.kv, self.tau, self.causal, seqs)

    def check(self, out, tensor, seqs=None):
        ref, mag, keys = self.ref(seqs)
        got = out.double().cpu().numpy()
        mine = ~np.isnan(ref)
        assert np.isfinite(got[mine]).all()
        u, bf = 2.0 ** -24, 2.0 ** -8
        logit = 1.0 + self.tau * self.scale * self.d * self.knorm
        fp = (keys[:, None, None] + 2 * self.d + 32) * u * logit
        tol = (bf if self.dtype == "bf16" else u) * np.abs(ref) + (fp + (2 * bf if tensor else 0.0)) * mag + 1e-30
        worst = (np.abs(got - ref) / tol)[mine]
        assert worst.max() <= 1.0, f"worst error is {worst.max():.3g} of its bound"
        diff, norm = np.linalg.norm((got - ref)[mine]), np.linalg.norm(ref[mine])
        if self.dtype == "bf16" and norm > 0:
            # the roundings' sizes go with the terms: mag over |ref| is above 1 where terms cancel
            assert diff <= 2.0 ** -7 * max(norm, np.linalg.norm(mag[mine]) / math.sqrt(max(keys.max(), 1))), diff / norm
        else:
            most = 8 * math.sqrt(keys.max() + self.d) * u * logit
            assert diff <= most * np.linalg.norm(mag[mine]) + 1e-30
        return got


def run(c, path=lla.LLA_PATH_AUTO, **kw):
    out = lla.paged_parallax(**{**c.device(), **kw}, path=path)
    torch.cuda.synchronize()
    lla.lla_sync_status()
    return out


def paths(dtype, d):
    tensor = dtype == "bf16" and d in (64, 128)
    return ([(lla.LLA_PATH_TENSOR, True)] if tensor else []) + [(lla.LLA_PATH_FP32, False)]


KINDS = {                      # new tokens, cached positions with them
    "decode": ([1] * 9, [1, 2, 8, 63, 64, 65, 200, 777, 1000]),
    "drafts": ([3, 5, 1, 5], [3, 400, 129, 64]),
    "chunk": ([70, 1, 0, 200, 33], [70, 300, 50, 513, 900]),
    "prompts": ([128, 129, 1, 300], [128, 129, 1, 300]),
}


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("bf16", 16), ("fp32", 128),
                                     ("fp32", 64), ("fp32", 32), ("fp32", 16)])
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("G,Hkv,page", [(1, 3, 16), (4, 2, 64), (3, 1, 8), (16, 1, 128)])
def test_attention(lla_gpu, dtype, d, kind, G, Hkv, page):
    new, kv = KINDS[kind]
    c = Case(new, kv, G * Hkv, Hkv, d, page, dtype, pad=3)
    for path, tensor in paths(dtype, d):
        c.check(run(c, path), tensor)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("G,most", [(1, 9), (3, 5), (16, 1), (4, 5), (5, 6), (1, 32)])
def test_up_to_32_rows_to_a_key_head(lla_gpu, d, causal, G, most):
    """Sets of eight rows, full and ragged; lengths about a warp's share of a block, a block and a range border;
    logits that grow with the position, sequences without keys or with fewer keys than tokens."""
    new = [most, 1, most, most, 0, most, max(most - 1, 1), most]
    kv = [most, 15, 47, 64 + 17, 30, max(most - 3, 0), 700, 5001]
    c = Case(new, kv, 2 * G, 2, d, 16, "bf16", causal=causal, pad=2, scale=1.5)
    for s, n in enumerate(c.kv):
        for x in range(0, n, 7):
            c.kc[c.table[s, x // 16], :, x % 16] *= 0.2 + 1.3 * x / n
    c.knorm = 1.5
    out = torch.full((len(c.q), 2 * G, d), 123.0, dtype=torch.bfloat16, device="cuda")
    got = c.check(run(c, lla.LLA_PATH_TENSOR, out=out), True)
    assert (got[c.cu[-1]:] == 123.0).all()
    assert torch.equal(out, run(c, lla.LLA_PATH_TENSOR, out=out.clone()))


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("G,most", [(1, 1), (3, 5), (4, 8), (1, 70)])
def test_fp32_sets_of_rows(lla_gpu, d, G, most):
    """Sets of eight fp32 rows.  Products of halves (d = 32, 64) are off by at most 3 2^-22 = 12 2^-24 of themselves: in
    the logit, in t and in the value product 36 2^-24 of the terms together, within the 32 + 2 d of the bound."""
    new, kv = [most, 1, most, 0, most], [most, 300, 65 + most, 10, 2500]
    c = Case(new, kv, 2 * G, 2, d, 16, "fp32", pad=2, scale=1.5)
    out = torch.full((len(c.q), 2 * G, d), 123.0, device="cuda")
    got = c.check(run(c, out=out), False)
    assert (got[c.cu[-1]:] == 123.0).all()


def test_fp32_products_hold_more_than_two_terms_of_11_bits(lla_gpu):
    """One key: out is its value, to fp32's last bits although each half has 11 (one or two products would leave 2^-11
    or 2^-12 of it)."""
    for d in (32, 64, 128):
        c = Case([1] * 40, [1] * 40, 4, 2, d, 8, "fp32")
        got = run(c).double().cpu().numpy()
        assert np.abs(got / c.ref()[0] - 1).max() <= 2.0 ** -20


def test_fp32_attention_past_32_bit_offsets(lla_gpu):
    """A page whose elements lie past 2^32 (an fp32 cache of 17 GB each): one key, so out is its value to 3 2^-22."""
    page, Hkv, d = 64, 8, 64
    P = (1 << 32) // (page * Hkv * d) + 2
    kc = torch.zeros(P, Hkv, page, d, device="cuda")
    vc = torch.zeros_like(kc)
    k = torch.randn(1, Hkv, d, device="cuda")
    lla.paged_append(k, -k, torch.tensor([(P - 1) * page], device="cuda"), kc, vc)
    out = lla.paged_parallax(torch.randn_like(k), torch.zeros_like(k), kc, vc, _i32([[P - 1]]), _i32([0, 1]), _i32([1]), 0.1, 1)
    torch.cuda.synchronize()
    lla.lla_sync_status()
    assert (out / -k - 1).abs().max() <= 2.0 ** -20


@pytest.mark.parametrize("d", [32, 64])
def test_fp32_captured_step_replays_with_other_lengths(lla_gpu, d):
    c = Case([1, 5, 1], [200, 70, 900], 4, 2, d, 16, "fp32")
    a = c.device()
    shorter = [150, 66, 3]
    want = [run(c), None]
    short = Case([1, 5, 1], shorter, 4, 2, d, 16, "fp32")
    short.kc, short.vc, short.table = c.kc, c.vc, c.table
    short.q, short.probe, short.P = c.q, c.probe, c.P
    want[1] = run(short)
    out, lens = torch.empty_like(a["q"]), a["kv_lens"].clone()
    a["kv_lens"] = lens
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        lla.paged_parallax(**a, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lla.paged_parallax(**a, out=out)
    for kv, ref in ((c.kv, want[0]), (shorter, want[1]), (c.kv, want[0])):
        lens.copy_(_i32(kv))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    lla.lla_sync_status()


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** 100])
def test_fp32_values_of_any_size(lla_gpu, size):
    """The scale of the values is that of the result: a power of two leaves the same bits."""
    c = Case([1, 5], [50, 200], 4, 2, 64, 16, "fp32")
    a = c.device()
    plain = run(c)
    assert torch.equal(plain * size, run(c, v_cache=a["v_cache"] * size))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 32)])
@pytest.mark.parametrize("new,kv", [([5, 40, 1], [77, 1, 130]), ([1, 1], [500, 33]), ([300], [129])])
def test_cross_attention(lla_gpu, dtype, d, new, kv):
    c = Case(new, kv, 4, 2, d, 32, dtype, causal=False)
    for path, tensor in paths(dtype, d):
        c.check(run(c, path), tensor)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,kv", [([1, 1, 1], [0, 5, 0]), ([20, 3, 40, 2], [4, 0, 39, 0]), ([0, 1, 0], [3, 4, 0])])
def test_rows_without_keys_are_zero_and_padding_is_left(lla_gpu, new, kv, causal):
    for dtype, d in (("bf16", 128), ("bf16", 64), ("fp32", 16)):
        c = Case(new, kv, 2, 1, d, 16, dtype, causal=causal, pad=7)
        for path, tensor in paths(dtype, d):
            out = torch.full((len(c.q), 2, d), 123.0, dtype=DT[dtype], device="cuda")
            got = c.check(run(c, path, out=out), tensor)
            sees = c.ref()[2]
            rows = np.arange(len(c.q)) < c.cu[-1]
            assert (got[rows & (sees == 0)] == 0).all()
            assert (got[~rows] == 123.0).all()


@pytest.mark.parametrize("dtype,d,path", [("bf16", 128, lla.LLA_PATH_TENSOR), ("bf16", 64, lla.LLA_PATH_TENSOR),
                                          ("fp32", 64, lla.LLA_PATH_FP32)])
@pytest.mark.parametrize("new,Hq", [([1], 2), ([1], 8), ([1], 24), ([40], 2)])
def test_long_cache_shared_by_many_ctas(lla_gpu, dtype, d, path, new, Hq):
    c = Case(new, [12345], Hq, 2, d, 64, dtype)
    c.check(run(c, path), path == lla.LLA_PATH_TENSOR)


@pytest.mark.parametrize("d,path,dtype", [(128, lla.LLA_PATH_TENSOR, "bf16"), (64, lla.LLA_PATH_TENSOR, "bf16"),
                                          (32, lla.LLA_PATH_FP32, "fp32")])
@pytest.mark.parametrize("new", [[1, 2], [150, 9]])
def test_growing_maximum_and_large_logits(lla_gpu, d, path, dtype, new):
    """Keys scaled up along the sequence: the running maximum grows in every block (logits to about +-60)."""
    c = Case(new, [700, 333], 2, 1, d, 16, dtype, scale=2.0)
    for s, n in enumerate(c.kv):
        for x in range(n):
            c.kc[c.table[s, x // 16], :, x % 16] *= 0.05 + 3.0 * x / n
    c.knorm = 3.1
    c.check(run(c, path), path == lla.LLA_PATH_TENSOR)


@pytest.mark.parametrize("d,path,dtype", [(128, lla.LLA_PATH_TENSOR, "bf16"), (64, lla.LLA_PATH_TENSOR, "bf16"),
                                          (128, lla.LLA_PATH_FP32, "fp32")])
@pytest.mark.parametrize("new", [[1], [90]])
def test_common_key_component_along_the_probe(lla_gpu, d, path, dtype, new):
    """Keys with a mean far from zero: probe.k has a large common part that the centre takes out."""
    c = Case(new, [800], 2, 1, d, 32, dtype, kshift=4.0)
    c.probe = (c.probe.float().abs() * 2).to(c.probe.dtype)
    ref, _, _ = c.ref()
    out = run(c, path)
    c.check(out, path == lla.LLA_PATH_TENSOR)
    got = out.double().cpu().numpy()
    # with the centre, the rounding of p (t - s0) stays that of a spread of a few units, as without the shift
    assert np.linalg.norm(got - ref) / np.linalg.norm(ref) < (2.0 ** -6 if dtype == "bf16" else 1e-4)


def test_zero_probe_is_softmax(lla_gpu):
    c = Case([1, 40], [300, 200], 4, 2, 128, 16, probe_scale=0.0)
    c.check(run(c), True)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp32", 32)])
@pytest.mark.parametrize("new,kv", [([1, 1, 1], [5, 70, 300]), ([40, 90], [60, 150])])
def test_strided_rows_and_interleaved_caches(lla_gpu, dtype, d, new, kv):
    c = Case(new, kv, 6, 2, d, 16, dtype, wide=5)
    a = c.device()
    fused = torch.zeros(len(c.q), 20, d, dtype=c.q.dtype, device="cuda")
    fused[:, 3:9], fused[:, 12:18] = a["q"], a["probe"]
    both = torch.full((c.P, 2, 2, 16, d), float("nan"), dtype=c.q.dtype, device="cuda")
    both[:, 0], both[:, 1] = a["k_cache"], a["v_cache"]
    for path, tensor in paths(dtype, d):
        plain = run(c, path)
        other = run(c, path, q=fused[:, 3:9], probe=fused[:, 12:18], k_cache=both[:, 0], v_cache=both[:, 1])
        assert torch.equal(plain, other)
        heads_first = a["q"].transpose(0, 1).contiguous().transpose(0, 1)      # heads not packed: copied
        assert torch.equal(plain, run(c, path, q=heads_first))
        c.check(plain, tensor)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 32)])
@pytest.mark.parametrize("new,kv", [([1], [4000]), ([1] * 40, [300] * 40), ([500, 3], [900, 40])])
def test_same_bits_every_run_and_with_any_workspace(lla_gpu, dtype, d, new, kv):
    c = Case(new, kv, 4, 2, d, 16, dtype)
    for path, tensor in paths(dtype, d):
        first = run(c, path)
        size = lla.lla_paged_parallax_workspace_size(0 if dtype == "bf16" else 1, path, len(c.q), len(new), 4, 2, d, 16,
                                                     c.table.shape[1], max(new))
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")      # NaN bits
        for _ in range(3):
            assert torch.equal(first, run(c, path, workspace=ws))
        with pytest.raises(lla.LLAError):
            run(c, path, workspace=ws[:-256])


def test_capture_and_replay_with_other_lengths(lla_gpu):
    """One captured call, replayed after the lengths, the table and the rows changed in place."""
    for dtype, d in (("bf16", 128), ("bf16", 64), ("fp32", 32)):
        for new_a, new_b in (([1, 1, 1], [1, 0, 1]), ([60, 2, 31], [3, 80, 0])):
            a = Case(new_a, [900, 70, 200], 4, 2, d, 16, dtype, seed=1, pad=40)
            b = Case(new_b, [100, 333, 5], 4, 2, d, 16, dtype, seed=2, pad=40)
            T, P, W = max(len(a.q), len(b.q)), max(a.P, b.P), max(a.table.shape[1], b.table.shape[1])
            st = None
            for c in (a, b):
                pads = lambda t, n, v: torch.cat([t, torch.full((n - len(t), *t.shape[1:]), v, dtype=t.dtype)])  # noqa: E731
                c.q, c.probe = pads(c.q, T, 0.0), pads(c.probe, T, 0.0)
                c.kc, c.vc = pads(c.kc, P, float("nan")), pads(c.vc, P, float("nan"))
                c.table = np.pad(c.table, ((0, 0), (0, W - c.table.shape[1])), constant_values=-1)
                dev = c.device()
                dev["max_new"] = max(new_a + new_b)
                if st is None:
                    st = dev
                    out = lla.paged_parallax(**st)
                    torch.cuda.synchronize()
                    g = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(g):
                        lla.paged_parallax(**st, out=out)
                else:
                    for k, v in dev.items():
                        if torch.is_tensor(v):
                            st[k].copy_(v)
                out.zero_()
                g.replay()
                torch.cuda.synchronize()
                lla.lla_sync_status()
                c.check(out, dtype == "bf16")


def test_two_calls_at_once_and_on_a_given_stream(lla_gpu):
    cs = [Case([1] * 8, [1500] * 8, 4, 2, 128, 16, seed=5), Case([200, 10], [400, 600], 4, 2, 128, 16, seed=6)]
    dev = [c.device() for c in cs]
    want = [run(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [lla.paged_parallax(**d, stream=s) for d, s in zip(dev, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    lla.lla_sync_status()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 32)])
@pytest.mark.parametrize("most", [1, 3, 40])
def test_more_sequences_than_threads(lla_gpu, dtype, d, most):
    """1100 short sequences, empty ones among them: a thread of the work division sums several."""
    rng = np.random.default_rng(most)
    new = rng.integers(0, most + 1, 1100)
    kv = new + rng.integers(0, 60, 1100) * (rng.random(1100) < 0.7)
    c = Case(new.tolist(), kv.tolist(), 4, 2, d, 8, dtype, pad=1)
    for path, tensor in paths(dtype, d):
        c.check(run(c, path), tensor)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 32)])
@pytest.mark.parametrize("new,kv,G", [([1, 1], [300, 70], 4), ([5, 20], [300, 200], 4), ([130, 40], [130, 400], 3)])
def test_rows_of_others_and_padding_do_not_reach_a_sequence(lla_gpu, dtype, d, new, kv, G):
    """NaN in padding rows, and other queries in the last sequence, leave the first one's bits as they were."""
    c = Case(new, kv, 2 * G, 2, d, 16, dtype, pad=30)
    for path, tensor in paths(dtype, d):
        a = c.device()
        first = run(c, path)
        q, r = a["q"].clone(), a["probe"].clone()
        q[c.cu[-1]:], r[c.cu[-1]:] = float("nan"), float("nan")
        q[c.cu[1]:c.cu[-1]] *= 3
        other = run(c, path, q=q, probe=r)
        assert torch.equal(first[:c.cu[1]], other[:c.cu[1]])
        assert torch.isfinite(other[:c.cu[-1]]).all()


def test_both_ways_of_marshalling_give_the_same_bits(lla_gpu, monkeypatch):
    """The calls through csrc/paged_bind.c and through Python launch the same."""
    c = Case([1, 4, 1], [300, 70, 130], 4, 2, 64, 16, pad=2)
    ctx, new, table, free, count, T = _plan_case(3, 20, 16, 2, 60, 5, None, None)

    def all_calls():
        tb = _i32(table)
        pl = lla.paged_plan(_i32(ctx), _i32(new), tb, _i32(free), _i32([count]), 16, T)
        kc, vc = torch.zeros(5000, 2, 16, 64, device="cuda"), torch.zeros(5000, 2, 16, 64, device="cuda")
        k = torch.arange(T * 128, dtype=torch.float32, device="cuda").view(T, 2, 64)
        lla.paged_append(k, -k, pl.slots, kc, vc)
        return [*pl, tb, kc, vc, run(c)[:6]]

    assert lla._bind()
    fast = all_calls()
    monkeypatch.setattr(lla, "_BIND", False)
    slow = all_calls()
    assert all(torch.equal(a, b) for a, b in zip(fast, slow))


def test_max_new_may_be_larger(lla_gpu):
    for d in (64, 128):
        c = Case([1, 1, 2], [300, 70, 130], 4, 2, d, 16, pad=5)
        c.check(run(c, max_new=len(c.q)), True)


def test_scratch_of_one_stream_grows_and_is_used_again(lla_gpu):
    small, large = Case([1] * 3, [700, 40, 90], 4, 2, 128, 16), Case([100] * 4, [900] * 4, 4, 2, 128, 16)
    want = [run(small), run(large)]
    for _ in range(3):
        got = [lla.paged_parallax(**c.device()) for c in (small, large, small)]
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[0])
    lla.lla_sync_status()


def test_two_host_threads_on_one_stream(lla_gpu):
    import threading
    cs = [Case([1], [6000], 4, 2, 128, 16, seed=7), Case([150], [2000], 4, 2, 128, 16, seed=8)]
    dev, want, bad = [c.device() for c in cs], [run(c) for c in cs], []

    def work(i):
        outs = [lla.paged_parallax(**dev[i]) for _ in range(60)]
        torch.cuda.synchronize()
        bad.extend(k for k, o in enumerate(outs) if not torch.equal(o, want[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    lla.lla_sync_status()
    assert not bad


def test_two_graphs_and_eager_calls_share_nothing(lla_gpu):
    cs = [Case([1] * 4, [2500, 90, 10, 700], 4, 2, 128, 16, seed=3), Case([120, 9], [700, 300], 4, 2, 128, 16, seed=4)]
    dev, want = [c.device() for c in cs], [run(c) for c in cs]
    outs, graphs = [torch.zeros_like(w) for w in want], []
    for d, o in zip(dev, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lla.paged_parallax(**d, out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = [lla.paged_parallax(**d) for d in dev]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs + eager, want + want))
    lla.lla_sync_status()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 32)])
@pytest.mark.parametrize("new", [[1, 1], [30, 80]])
def test_bad_lengths_and_pages_are_cut_and_reported(lla_gpu, dtype, d, new):
    """What the device arrays hold is never followed outside the tensors: the kernels compare every
    length and page id with what the tensors hold before they use it."""
    c = Case(new, [100, 90], 2, 1, d, 16, dtype)
    T, W = len(c.q), c.table.shape[1]
    bad_page = c.table.copy()
    bad_page[0, 2] = 1 << 30
    neg_page = c.table.copy()
    neg_page[0, 3] = -5
    for path, _ in paths(dtype, d):
        good = run(c, path)
        for kw in (dict(block_table=_i32(bad_page)), dict(block_table=_i32(neg_page)),
                   dict(kv_lens=_i32([W * 16 + 9, 90])), dict(kv_lens=_i32([-4, 90])),
                   dict(cu_q=_i32([0, new[0], T + 50])), dict(cu_q=_i32([-7, new[0], T])),
                   dict(cu_q=_i32([0, T + 5, new[0]])),
                   dict(max_new=new[1] - 1) if new[1] > 1 else dict(cu_q=_i32([1 << 30, 0, T]))):
            a = {**c.device(), **kw}
            if "kv_lens" in kw and int(kw["kv_lens"][0]) > 0:
                a["block_table"] = _i32(np.where(c.table < 0, 0, c.table))
            out = lla.paged_parallax(**a, path=path)
            with pytest.raises(lla.LLAError) as e:
                lla.lla_sync_status()
            assert e.value.status == lla.LLA_ERR_INVALID_ARG, kw
            if "block_table" in kw:                      # the other sequence is not touched by it
                assert torch.equal(out[new[0]:], good[new[0]:])
        assert torch.equal(good, run(c, path))


def test_binding_refusals(lla_gpu):
    c = Case([1, 1], [30, 40], 4, 2, 64, 16)
    a = c.device()
    for kw in (dict(q=a["q"].float()), dict(q=a["q"][:, :3]), dict(probe=a["probe"][:1]), dict(v_cache=a["v_cache"][:-1]),
               dict(k_cache=a["k_cache"].transpose(1, 2)), dict(block_table=a["block_table"].long()),
               dict(block_table=a["block_table"][0]), dict(cu_q=a["cu_q"][:-1]), dict(kv_lens=a["kv_lens"].cpu()),
               dict(out=a["q"].float()), dict(out=a["q"][:1]), dict(tau=0.0), dict(max_new=0),
               dict(workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(lla.LLAError):
            lla.paged_parallax(**{**a, **kw})
    s = torch.zeros(2, dtype=torch.int64, device="cuda")
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    for args in ((k, k[:1], s), (k, k, s.int()), (k, k, s[:1]), (k.float(), k.float(), s), (k[:, :1], k[:, :1], s)):
        with pytest.raises(lla.LLAError):
            lla.paged_append(*args, a["k_cache"], a["v_cache"])
    i = _i32([1, 2])
    for kw in (dict(new=i[:1]), dict(table=i), dict(count=i), dict(page=10), dict(rows=0), dict(slots=i)):
        g = dict(new=i, table=_i32([[1, 2], [3, 4]]), count=i[:1], page=16, rows=3, slots=None)
        g.update(kw)
        with pytest.raises(lla.LLAError):
            lla.paged_plan(i, g["new"], g["table"], i, g["count"], g["page"], g["rows"], slots=g["slots"])


# ---------------------------------------------------------------------------------- the run of them
@pytest.mark.parametrize("dtype,d,Hq,Hkv", [("bf16", 128, 4, 2), ("bf16", 64, 2, 2), ("fp32", 32, 3, 1)])
def test_serving_steps_equal_the_whole_sequences(lla_gpu, dtype, d, Hq, Hkv):
    """Chunks of prompts, then single tokens, through plan, append and attention, in shuffled batches:
    every row equals the same row of the causal Parallax forward on the whole sequence."""
    rng = np.random.default_rng(d)
    torch.manual_seed(d)
    lens, page, W = [150, 37, 260], 16, 20
    S, G, tau, dt = len(lens), Hq // Hkv, d ** -0.5, DT[dtype]
    unit = lambda x: x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    q = [unit(torch.randn(n, Hq, d, device="cuda")).to(dt) for n in lens]
    r = [(unit(torch.randn(n, Hq, d, device="cuda")) * tau).to(dt) for n in lens]
    k = [unit(torch.randn(n, Hkv, d, device="cuda")).to(dt) for n in lens]
    v = [torch.randn(n, Hkv, d, device="cuda").to(dt) for n in lens]
    whole = []
    for s in range(S):
        shared = lambda x: x.transpose(0, 1)[None].repeat_interleave(G, 1)  # noqa: E731
        whole.append(lla.parallax_forward(q[s].transpose(0, 1)[None], shared(k[s]), shared(v[s]),
                                          r[s].transpose(0, 1)[None].float(), tau, path=lla.LLA_PATH_FP32)[0].transpose(0, 1))
    P = 40
    kc = torch.full((P, Hkv, page, d), float("nan"), dtype=dt, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    table = torch.full((S, W), -1, dtype=torch.int32, device="cuda")
    free, left, ctx = _i32(rng.permutation(P)), _i32([P]), _i32([0] * S)
    done, first = [0] * S, True
    while any(a < n for a, n in zip(done, lens)):
        new = [min(n - a, int(rng.integers(0, 90)) if a < n // 2 else int(rng.integers(0, 3))) for a, n in zip(done, lens)]
        if sum(new) == 0:
            continue
        T = sum(new) + 2
        pl = lla.paged_plan(ctx, _i32(new), table, free, left, page, T, kv_lens=ctx, free_left=left)
        rows = lambda xs: torch.cat([x[a:a + n] for x, a, n in zip(xs, done, new)] + [x_pad(xs)])  # noqa: E731
        x_pad = lambda xs: torch.zeros(2, *xs[0].shape[1:], dtype=dt, device="cuda")  # noqa: E731
        lla.paged_append(rows(k), rows(v), pl.slots, kc, vc)
        out = lla.paged_parallax(rows(q), rows(r), kc, vc, table, pl.cu_q, pl.kv_lens, tau, max(new))
        torch.cuda.synchronize()
        lla.lla_sync_status()
        at = 0
        for s in range(S):
            want = whole[s][done[s]:done[s] + new[s]].double()
            got = out[at:at + new[s]].double()
            # both sides are within the bounds above of the same value: rounding of bf16 weights and outputs
            # (2^-7 of the norm each side), or fp32 sums
            assert (got - want).norm() <= (2.0 ** -6 if dtype == "bf16" else 2e-5) * want.norm() + 1e-30
            at += new[s]
        done = [a + n for a, n in zip(done, new)]
    assert ctx.tolist() == lens and int(left) == P - sum(-(-n // page) for n in lens)
