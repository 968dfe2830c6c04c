"""Splits that a 4-bit cache makes room for, read off its bytes (on the CPU)."""
import ctypes

import pytest

from test_serving_ops_abi import lib  # noqa: F401 (fixture)


def most_splits(lib, B, H, Dh, T, D):  # noqa: F811
    """Rows of Dh + 2 floats per (b, h) beside the blocks, the lengths and the counters."""
    n = ctypes.c_size_t()
    assert lib.ratp_cache_bytes_q4(B, H, Dh, T, D, 0, None, ctypes.byref(n)) == 0
    up = lambda x: -(-x // 256) * 256
    block = 32 * 2 * (Dh // 2 + Dh // 8)
    rest = n.value - up(B * H * -(-(T // D) // 32) * block) - up(4 * B) - up(4 * (B * H + B))
    return rest // (B * H * (Dh + 2) * 4)


@pytest.mark.parametrize("Dh", [64, 128])
def test_a_single_long_head_gets_more_splits(lib, Dh):  # noqa: F811
    assert 100 <= most_splits(lib, 1, 1, Dh, 1 << 20, 1) <= 256
    assert 64 < most_splits(lib, 1, 2, Dh, 1 << 18, 1) <= 128


def test_splits_of_many_heads(lib):  # noqa: F811
    assert most_splits(lib, 64, 16, 128, 33024, 64) == 1
    assert most_splits(lib, 4, 32, 128, 32768 + 64, 4) == 9
    assert most_splits(lib, 1, 16, 128, 1 << 17, 4) == 64
