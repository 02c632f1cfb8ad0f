"""The largest X that the experts' and adapters' linears admit: its last values are read as what they are."""

import numpy as np
import pytest
import torch

import weight_only_bit_02_amd as awq
from tests.grouped_ref import linear_bound, linear_reference, lora_reference, packed_numpy
from tests.gpu_util import DEV, host, to_dev

pytestmark = pytest.mark.gpu

M, N, K = (1 << 17) - 1, 16, 1 << 14  # one row below 2^31 values


def _inputs():
    (qw, sc, zb), Wd = packed_numpy(N, K, 128, 4, 1)
    row = np.random.default_rng(2).standard_normal(K).astype(np.float16)
    row[-8:] = [0, 0, 0, 0, 0, 0, 500, -700]
    X = torch.zeros((M, K), dtype=torch.float16, device=DEV)
    X[-1] = to_dev(row)
    X[0] = to_dev(-row)
    return (to_dev(qw), to_dev(sc), to_dev(zb)), Wd, X, row


def test_largest_input():
    packed, Wd, X, row = _inputs()
    ids = torch.zeros(M, dtype=torch.int32, device=DEV)
    groups = awq.group_rows(ids, 1)
    w = awq.PackedExperts(*(t[None] for t in packed), 1, N, K)
    y, S = linear_reference(row[None], Wd)
    bound = linear_bound(y, S, K)
    for kernel in ("gemm64", "gemm128", "gemm256", "gemm64k", "auto"):
        Y = awq.linear_w4a16_grouped(X, w, groups, kernel=kernel)
        assert np.all(np.abs(host(Y[-1:]).astype(np.float64) - y) <= bound), kernel
        assert torch.equal(Y[0], -Y[-1]) and not Y[1:-1].any(), kernel

    A = np.zeros((1, 8, K), np.float16)
    A[0, :, -2:] = np.random.default_rng(3).standard_normal((8, 2))
    B = np.random.default_rng(4).standard_normal((1, N, 8)).astype(np.float16)
    scale = np.ones(1, np.float32)
    ids[:-1] = -1
    y, bound = lora_reference(row[None], Wd, A, B, scale, [0])
    Y = host(awq.linear_w4a16_lora(X, awq.PackedLinear(*packed, N, K),
                                   awq.LoraAdapters(to_dev(A), to_dev(B), to_dev(scale)), ids)[-1:])
    assert np.all(np.abs(Y.astype(np.float64) - y) <= bound)
