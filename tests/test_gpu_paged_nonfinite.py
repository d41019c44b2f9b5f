"""A NaN that a row's formula reads reaches that row, whatever its bits: paged attention neither multiplies it as a number
nor drops it.  0x7fffffff is what CUDA arithmetic produces, 0x7f800001 has nothing but its last bit."""
import numpy as np
import pytest
import torch

from test_gpu_paged import Case, paths, run

pytestmark = pytest.mark.gpu

BITS = {"fp32": (torch.int32, (0x7fffffff, -1, 0x7fc00000, 0x7f800001, -0x7fffff)),
        "bf16": (torch.int16, (0x7fff, -1, 0x7fc0, 0x7f81))}
ALL = [("fp32", 16), ("fp32", 32), ("fp32", 64), ("fp32", 128), ("bf16", 32), ("bf16", 64), ("bf16", 128)]
KINDS = {"decode": ([1, 1], [70, 9]), "long": ([1], [3000]), "chunk": ([40, 1], [100, 20]), "ragged": ([9, 1], [200, 33])}


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("dtype,d", ALL)
def test_nan_reaches_the_rows_that_read_it(lla_gpu, dtype, d, kind):
    new, kv = KINDS[kind]
    c = Case(new, kv, 4, 2, d, 16, dtype, pad=1)
    word, patterns = BITS[dtype]
    n, L, last = new[0], kv[0], d - 3

    def with_bits(t, where, bits):
        t = t.clone()
        t.view(word)[where] = bits
        assert torch.isnan(t[where]).item()
        return t.cuda()

    for path, _ in paths(dtype, d):
        good = run(c, path)
        for bits in patterns:
            # a query or a probe: its row and head, and no other
            for name in ("q", "probe"):
                out = run(c, path, **{name: with_bits(getattr(c, name), (n - 1, 3, last), bits)})
                assert torch.isnan(out[n - 1, 3]).all(), (name, hex(bits))
                rest = out.clone()
                rest[n - 1, 3] = good[n - 1, 3]
                assert torch.equal(rest[:c.cu[-1]], good[:c.cu[-1]])
            # a key or a value that every row of the sequence sees (key head 1: query heads 2 and 3)
            for x in (0, L - n):
                at = (int(c.table[0, x // 16]), 1, x % 16, last)
                out = run(c, path, k_cache=with_bits(c.kc, at, bits))
                assert torch.isnan(out[:n, 2:]).all(), ("key", hex(bits))
                out = run(c, path, v_cache=with_bits(c.vc, at, bits))
                assert torch.isnan(out[:n, 2:, last]).all(), ("value", hex(bits))
                cols = np.arange(d) != last
                assert torch.equal(out[:n, 2:][..., cols], good[:n, 2:][..., cols])
                assert torch.equal(out[:n, :2], good[:n, :2]) and torch.equal(out[n:c.cu[-1]], good[n:c.cu[-1]])
