"""Sequences of one tensor beside bare tensors in the rotary calls: x alone says whether tuples come back, and each result has its
tensor's shape, whichever way the call is marshalled."""
import pytest
import torch

import local_linear_attention_flashlla_gb300 as lla

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(1, 2, 64), (3, 2, 64), (1, 2, 5, 64), (2, 2, 5, 64)])
@pytest.mark.parametrize("marshalled", ["c", "python"])
def test_sequences_of_one_tensor(lla_gpu, monkeypatch, shape, marshalled):
    if marshalled == "python":
        monkeypatch.setattr(lla, "_BIND", False)
    n = shape[0] if len(shape) == 3 else shape[2]
    x, dy = (torch.randn(shape, device="cuda").bfloat16() for _ in range(2))
    table, pos, gain = lla.rotary_table(64), torch.arange(n, dtype=torch.int32, device="cuda") + 3, torch.rand(64, device="cuda")
    want, wantg = lla.rotary_backward(dy, x, pos, table, gain=gain, eps=1e-6)       # (grows the scratch that the C way needs)
    assert want.shape == x.shape and wantg.shape == gain.shape
    for dys in (dy, (dy,), [dy]):
        for g in (gain, (gain,)):
            dx, dg = lla.rotary_backward(dys, x, pos, table, gain=g, eps=1e-6)
            assert torch.is_tensor(dx) and torch.is_tensor(dg) and dx.shape == x.shape
            assert torch.equal(dx, want) and torch.equal(dg, wantg)
            for xs in ((x,), [x]):
                dx, dg = lla.rotary_backward(dys, xs, pos, table, gain=g, eps=1e-6)
                assert isinstance(dx, tuple) and isinstance(dg, tuple) and len(dx) == len(dg) == 1 and dx[0].shape == x.shape
                assert torch.equal(dx[0], want) and torch.equal(dg[0], wantg)
    turned, none = lla.rotary_backward(dy, None, pos, table)
    assert turned.shape == x.shape and none is None
    both, none = lla.rotary_backward((dy,), None, pos, table)
    assert isinstance(both, tuple) and torch.equal(both[0], turned) and none is None
    y = lla.rotary(x, pos, table, gain=(gain,), eps=1e-6)
    assert torch.is_tensor(y) and y.shape == x.shape
    z = lla.rotary((x,), pos, table, gain=gain, eps=1e-6)
    assert isinstance(z, tuple) and torch.equal(z[0], y)
    torch.cuda.synchronize()
    lla.lla_sync_status()
