"""GPU checks of calls of the paged cache at their edges."""
import pytest
import torch

import mhc_hyper_connection_pre_gb300 as mhc

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mhc.load_library()
    assert mhc.device_status() == 0
    yield
    assert mhc.device_status() == 0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_fork_of_a_batch_that_has_ended():
    """Nobody goes on: empty tables, the caches as they were; and a batch may begin after it."""
    cache = mhc.kv_cache(4, 1, 16, 64)
    got = mhc.kv_fork(cache, _i32([[0, 1], [2, -1]]), _i32([20, 3]), _i32([]), room=1)
    assert got["block_table"].shape == (0, 2) and got["seq_lens"].shape == (0,)
    got = mhc.kv_fork(cache, got["block_table"], got["seq_lens"], _i32([]), room=_i32([]))
    assert got["block_table"].shape == (0, 2)
    got = mhc.kv_fork(cache, got["block_table"], got["seq_lens"], _i32([-1]), room=17)
    assert got["block_table"].tolist() == [[0, 1]] and got["seq_lens"].tolist() == [0]
    assert not cache["k"].view(torch.uint8).any()
