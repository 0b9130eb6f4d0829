"""The test hook of the attention kernel's bounded waits: its refusals (no GPU)."""
import pytest

from trellis_quantized_moe_exl3_gb300 import _lib, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def test_attention_wait_hook_validation(L):
    f = L.exl3_test_set_attention_wait_fault
    for barrier, budget in ((-2, 1000000), (0, 0), (1, 999999), (3, 1 << 40), (0, -1)):
        assert f(barrier, budget) == _lib.EXL3_ERR_ARG
    assert f(2, 2000000) == _lib.EXL3_OK
    assert f(-1, 0) == _lib.EXL3_OK
