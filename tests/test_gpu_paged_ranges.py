"""Paged operators at the ends of their ranges: small fp32 magnitudes, cross attention at every head dim, tiles of copied
rows that several CTAs share, plans of many rows."""
import numpy as np
import pytest
import torch

import local_linear_attention_flashlla_gb300 as lla
from oracle.paged_ref import paged_plan_ref
from test_gpu_paged import Case, _i32, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [32, 64])
@pytest.mark.parametrize("new", [[1, 1], [5, 40]])
def test_fp32_halves_of_small_operands(lla_gpu, d, new):
    """x in [2^e, 2^(e+1)) is cut into 11 bits and a lower half, a multiple of 2^(e-23) below 2^(e-11), of which the products
    hold 11 bits, and nothing below 2^-136.  From e = -113 on the second says nothing that the first does not: queries and
    probes (of 2^-10 at least) scaled by 2^-103 against keys scaled by 2^103 give the same bits.  At e = -114 every lower half
    may lose its last bit, 2^-23 of x as elsewhere: the bounds hold."""
    c = Case(new, [200, 333], 4, 2, d, 16, "fp32")
    for name in ("q", "probe"):
        t = getattr(c, name)
        setattr(c, name, torch.where(t < 0, -1.0, 1.0) * t.abs().clamp(min=2.0 ** -10))
    c.scale = 1.01                                 # sqrt(1 + 2^-20): what the clamp adds to a row's RMS is less
    scaled = lambda x: run(c, q=c.q.cuda() * x, probe=c.probe.cuda() * x, k_cache=c.kc.cuda() / x)  # noqa: E731
    plain = run(c)
    c.check(plain, False)
    assert torch.equal(plain, scaled(2.0 ** -103))
    c.check(scaled(2.0 ** -104), False)


@pytest.mark.parametrize("dtype,d", [("fp32", 16), ("fp32", 64), ("fp32", 128), ("bf16", 32)])
@pytest.mark.parametrize("new,kv", [([5, 40, 1], [77, 1, 130]), ([1, 1], [500, 33]), ([9], [4000])])
def test_cross_attention_of_the_other_kernels(lla_gpu, dtype, d, new, kv):
    c = Case(new, kv, 6, 2, d, 32, dtype, causal=False, pad=2)
    out = torch.full((len(c.q), 6, d), 123.0, dtype=c.q.dtype, device="cuda")
    got = c.check(run(c, out=out), False)
    assert (got[c.cu[-1]:] == 123.0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [3, 6, 12])
@pytest.mark.parametrize("causal", [True, False])
def test_copied_rows_in_tiles_that_many_ctas_share(lla_gpu, d, G, causal):
    """Groups of heads that do not divide a tile (its rows are copied one by one) over long caches."""
    c = Case([45, 150], [20011, 3000], 2 * G, 2, d, 16, "bf16", causal=causal, pad=1, seed=G)
    c.check(run(c, lla.LLA_PATH_TENSOR), True)


@pytest.mark.parametrize("S,new_hi,page,pad", [(3, 60000, 16, 0), (200, 1500, 8, 5000), (1100, 300, 256, 1)])
def test_plan_of_more_rows_than_2_to_the_16(lla_gpu, S, new_hi, page, pad):
    rng = np.random.default_rng(S)
    ctx, new = rng.integers(0, 3000, S), rng.integers(0, new_hi + 1, S)
    new[0] = new_hi
    T = int(new.sum()) + pad
    assert T > 65536
    held, need = -(-ctx // page), -(-(ctx + new) // page)
    ids = rng.permutation(int(need.sum()))
    table = np.full((S, int(need.max()) + 1), -1)
    at = 0
    for s in range(S):
        table[s, :held[s]] = ids[at:at + held[s]]
        at += held[s]
    free = ids[at:]
    for count in (len(free), len(free) // 2):
        ref = paged_plan_ref(ctx, new, table, free, count, page, T)
        tb = _i32(table)
        got = lla.paged_plan(_i32(ctx), _i32(new), tb, _i32(free), _i32([count]), page, T)
        torch.cuda.synchronize()
        for name in ("kv_lens", "cu_q", "slots", "positions", "granted"):
            assert np.array_equal(getattr(got, name).cpu().numpy(), np.asarray(ref[name])), name
        assert int(got.free_left) == ref["free_left"] and np.array_equal(tb.cpu().numpy(), ref["table"])
