"""Sizes at the edge of what the experts' and adapters' entry points admit, refused on the host
(no GPU needed: pointers are never dereferenced)."""

import ctypes as C

import pytest

from weight_only_bit_02_amd import _abi

FAKE = C.c_void_p(0x7F0000000000)
SHAPE = 2


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


@pytest.mark.parametrize("kernel", range(6))
def test_largest_x(lib, kernel):
    """X and an adapter's A stay below 2^31 values: a buffer descriptor covers 2^32 - 1 bytes."""
    for f in (lib.awq_linear_w4a16_grouped, lib.awq_linear_w4a16_grouped_gated_silu):
        call = lambda x_rows, K: f(FAKE, x_rows, FAKE, None, 16, 1, 4, FAKE, FAKE, FAKE, 64, K, None, FAKE, None,
                                   kernel, None)
        assert call(1 << 24, 128) == SHAPE and call(1 << 17, 1 << 14) == SHAPE
    lora = lambda M, K, rank: lib.awq_linear_w4a16_lora(FAKE, M, FAKE, FAKE, FAKE, 16, K, None, FAKE, FAKE, FAKE, 2, rank,
                                                        FAKE, None, FAKE, FAKE, 1 << 40, None, kernel, None)
    assert lora(1 << 17, 1 << 14, 8) == SHAPE and lora(1, 1 << 23, 256) == SHAPE


@pytest.mark.parametrize("T,N", [((1 << 29) - 1, 64), ((1 << 28) - 1, 128), ((1 << 30) - 1, 4), ((1 << 32) // 65, 65)])
def test_combine_of_more_blocks_than_a_launch(lib, T, N):
    """T N just below 2^35 (2^32): its whole blocks of threads are 2^32 threads."""
    assert lib.awq_moe_combine(FAKE, FAKE, FAKE, FAKE, 4, T, 1, N, None, FAKE, None) == SHAPE
