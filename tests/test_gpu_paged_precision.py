"""Weights of the bf16 decode kernel up to 16 query rows to a key head: held to 2^-16, as two bf16 halves.

bf16 has 8 significant bits: the upper half of a weight is off by at most 2^-8 of it, and that rest, rounded again, by at most
2^-8 of itself.  So the value products are within 2^-16 of their terms twice (p and p (t - s0)), which is below the fp32
sums' bound of the tests of every kernel: outputs are within their own rounding, 2^-8, and that bound."""
import numpy as np
import pytest
import torch

import local_linear_attention_flashlla_gb300 as lla
from test_gpu_paged import Case, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("G,most", [(1, 1), (1, 8), (8, 1), (3, 2), (16, 1), (4, 4), (1, 13), (5, 3)])
def test_up_to_16_rows_are_off_by_the_outputs_rounding(lla_gpu, d, causal, G, most):
    new, kv = [most, 1, most, 0, most], [most, 15, 300, 30, 5001]
    c = Case(new, kv, 2 * G, 2, d, 16, "bf16", causal=causal, pad=2, seed=G)
    out = run(c, lla.LLA_PATH_TENSOR)
    sums = (1 + 2 * d + 32) * 2.0 ** -24 * (1 + c.tau * d)      # the bound's part for a row that sees one key
    assert 2 * 2.0 ** -16 <= sums
    got = c.check(out, False)
    # the 2-norm: roundings of the output alone are independent and uniform, 2^-8 / sqrt(3) of a value at most
    ref = c.ref()[0]
    mine = ~np.isnan(ref)
    assert np.linalg.norm((got - ref)[mine]) <= 2.0 ** -8 / np.sqrt(3) * np.linalg.norm(ref[mine])


@pytest.mark.parametrize("d", [64, 128])
def test_weights_that_differ_by_less_than_bf16(lla_gpu, d):
    """Two kinds of keys whose logits differ by 2^-7: their weights round to one or to two bf16 values, and the difference of
    their sums is most of the output (values of opposite sign)."""
    c = Case([1] * 6, [512] * 6, 2, 1, d, 16, "bf16", probe_scale=0.0)
    base = c.kc[c.table[0, 0], 0, 0].float()
    for s in range(6):
        for x in range(512):
            at = (int(c.table[s, x // 16]), 0, x % 16)
            c.kc[at] = (base * (1.0 if x % 2 else 0.99)).to(torch.bfloat16)
            c.vc[at] = (c.vc[at].float().abs() * (1 if x % 2 else -1)).to(torch.bfloat16)
    c.check(run(c, lla.LLA_PATH_TENSOR), False)
