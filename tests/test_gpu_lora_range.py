"""Scaled first products (scale X A^T) at the end of the fp32 range."""

import numpy as np
import pytest

import synthetic_inputs as si
import weight_only_bit_02_amd as awq
from tests.grouped_ref import packed_numpy
from tests.gpu_util import host, to_dev

pytestmark = pytest.mark.gpu

KERNELS = [(5, "skinny"), (70, "gemm64"), (70, "gemm64k"), (130, "gemm128"), (260, "gemm256")]
N, K, R = 40, 256, 8


def _run(M, kernel, first, scale):
    """An adapter with one rank: X A^T = first for every row; outputs 0 .. 19 take it, the others not."""
    (qw, sc, zb), _ = packed_numpy(N, K, 128, 4, 7)
    w = awq.PackedLinear(to_dev(qw), to_dev(sc), to_dev(zb), N, K)
    X = si.activations(M, K, offset=M)
    X[:, 0] = 1.0
    A, B = np.zeros((1, R, K), np.float16), np.zeros((1, N, R), np.float16)
    A[0, 2, 0] = first
    B[0, :N // 2, 2] = 1.0
    lora = awq.LoraAdapters(to_dev(A), to_dev(B), to_dev(np.array([scale], np.float32)))
    run = lambda a: host(awq.linear_w4a16_lora(to_dev(X), w, lora, to_dev(np.full(M, a, np.int32)), kernel=kernel))
    return run(0), run(-1)


@pytest.mark.parametrize("M,kernel", KERNELS)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_overflow_is_infinite(M, kernel, sign):
    """scale X A^T past the largest fp32: Inf of its sign in the outputs that take it."""
    got, _ = _run(M, kernel, 4.0, sign * 3.0e38)
    assert np.all(got[:, :N // 2] == sign * np.inf)


@pytest.mark.parametrize("M,kernel", KERNELS)
@pytest.mark.parametrize("scale", [2.0 ** 125, 2.0 ** 126, 1.5 * 2.0 ** 126, 2.0 ** 127, 3.0e38])
def test_largest_finite_products(M, kernel, scale):
    """Finite up to the largest fp32: outputs whose B is zero are those of the linear alone."""
    got, alone = _run(M, kernel, 1.0, scale)
    assert np.all(got[:, :N // 2] == np.inf)
    assert np.array_equal(got[:, N // 2:], alone[:, N // 2:])


@pytest.mark.parametrize("M,kernel", KERNELS)
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_nonfinite_rank_beside_large_ones(M, kernel, bad):
    """A rank of X A^T that is Inf or NaN beside one past the range of fp16: the outputs are Inf of the first's
    sign, or NaN, not the difference of two infinities."""
    (qw, sc, zb), _ = packed_numpy(N, K, 128, 4, 7)
    w = awq.PackedLinear(to_dev(qw), to_dev(sc), to_dev(zb), N, K)
    X = si.activations(M, K, offset=M)
    X[:, 0] = 1.0
    A, B = np.zeros((1, R, K), np.float16), np.ones((1, N, R), np.float16)
    A[0, 2, 0], A[0, 5, 0] = bad, -np.sign(bad) * 1000.0 if bad == bad else 1000.0
    lora = awq.LoraAdapters(to_dev(A), to_dev(B), to_dev(np.array([1000.0], np.float32)))
    # X is finite and meets the zeros of A elsewhere: rank 2 is the bad value, rank 5 is +-10^6
    got = host(awq.linear_w4a16_lora(to_dev(X), w, lora, to_dev(np.zeros(M, np.int32)), kernel=kernel))
    assert np.array_equal(got, np.full((M, N), bad, np.float16), equal_nan=True)
