"""CPU checks of the test hook that stalls one thread block of qkq_attention_kv8."""
import pytest

qkq = pytest.importorskip("transform_rope_head_b200")


def test_limits():
    hook = qkq.lib().qkq_selftest_attention_kv8_stall
    assert hook(10 ** 8 + 1, 0) == -1 and hook(2 ** 64 - 1, 0) == -1 and hook(1000, -1) == -1
    try:
        assert hook(1, 3) == 0 and hook(10 ** 8, 0) == 0
    finally:
        assert hook(0, 0) == 0
