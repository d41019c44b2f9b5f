"""What lla_sync_status returns where a paged call met a bad argument and a bounded wait gave up."""
import pytest
import torch

import local_linear_attention_flashlla_gb300 as lla

pytestmark = pytest.mark.gpu


def _append_out_of_range():
    cache = torch.zeros(2, 1, 8, 64, device="cuda")
    row = torch.ones(1, 1, 64, device="cuda")
    lla.paged_append(row, row, torch.tensor([99], device="cuda"), cache, cache.clone())


@pytest.mark.parametrize("timeout_first", [True, False])
def test_timeout_is_not_hidden_by_a_bad_argument(lla_gpu, timeout_first):
    lla.lla_sync_status()
    steps = [lla.lla_selftest_device_timeout, _append_out_of_range]
    for step in steps if timeout_first else steps[::-1]:
        step()
    with pytest.raises(lla.LLAError) as e:
        lla.lla_sync_status()
    assert e.value.status == lla.LLA_ERR_DEVICE_TIMEOUT
    assert "wait gave up" in str(e.value) and "a paged call met" in str(e.value)
    lla.lla_sync_status()                          # both were cleared
    _append_out_of_range()
    with pytest.raises(lla.LLAError) as e:
        lla.lla_sync_status()
    assert e.value.status == lla.LLA_ERR_INVALID_ARG
    lla.lla_sync_status()
