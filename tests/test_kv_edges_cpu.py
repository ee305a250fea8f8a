"""The K/V step's host side on host-only pools, beside test_kv_step_cpu.py."""
import pytest

from linear_attention_state_lsc_gb300 import lsc as L

from _util import gpu_present
from test_kv_step_cpu import DEV, batch, pool_of


def test_no_workspace_size_without_a_device(lsc):
    """The need depends on the device's SMs: a host-only pool has no answer, not 0."""
    if gpu_present():
        pytest.skip("a pool made here is a device pool")
    pool = pool_of()
    a = L.kv_attend_args(batch(), 4, DEV, DEV, L.LSC_BF16, 0.125)
    assert L.lsc_kv_attend_workspace_bytes(pool, a)[0] == L.LSC_ERR_CUDA
    L.lsc_kv_pool_destroy(pool)
