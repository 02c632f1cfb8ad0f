"""The streaming kernel and the adapters' first product over K: few and many waves of a block, K in
several parts, rings that are filled again, and the columns split among the XCDs."""

import numpy as np
import pytest

import synthetic_inputs as si
from tests import test_gpu_lora as lora
from tests.test_gpu_grouped import _experts, _run

pytestmark = pytest.mark.gpu

FORMATS = [(4, 128), (4, 32), (8, 128), (8, 64), (3, 128), (3, 64)]
STEPS = [1024, 1152, 2048, 2176, 4096, 4480, 11008]  # two, four, eight waves; then parts


@pytest.mark.parametrize("w_bit,group", FORMATS)
@pytest.mark.parametrize("K", STEPS)
@pytest.mark.parametrize("gated", [False, True])
def test_experts(K, w_bit, group, gated):
    w, Wd = _experts(3, 72, K, group, w_bit, seed=K)
    _run(w, Wd, [5, 0, 17], gated, "skinny", 2, 2, seed=K + 1)
    _run(w, Wd, [0, 1, 0], gated, "skinny", None, 0, seed=K + 2)


@pytest.mark.parametrize("w_bit,group", FORMATS)
@pytest.mark.parametrize("K", STEPS)
@pytest.mark.parametrize("r", [16, 40])
def test_adapters(K, w_bit, group, r):
    case = lora._case(72, K, 20, r, group, w_bit, seed=K)
    for M, kind in ((1, "same"), (17, "mixed"), (48, "mixed"), (64, "runs")):
        lora._check(case, si.activations(M, K, offset=M), lora._ids(kind, M, 20, M), "skinny", grouped=M == 48)


@pytest.mark.parametrize("M,kernel", [(70, "gemm64"), (70, "gemm64k"), (130, "gemm128"), (260, "gemm256")])
@pytest.mark.parametrize("r", [16, 32])
@pytest.mark.parametrize("K", [4096, 11008])
def test_adapters_many_rows(K, r, M, kernel):
    case = lora._case(40, K, 5, r, seed=K)
    lora._check(case, si.activations(M, K, offset=M), lora._ids("mixed", M, 5, M), kernel, grouped=True)


@pytest.mark.parametrize("K", [2176, 4224])
@pytest.mark.parametrize("w_bit", [4, 8, 3])
def test_many_column_chunks(w_bit, K):
    """Columns for every XCD's share with eight waves a block, K in one part and in two."""
    w, Wd = _experts(2, 4216, K, 128, w_bit, seed=w_bit)
    for gated in (False, True):
        _run(w, Wd, [17, 3], gated, "skinny", None, 1, seed=41)
    case = lora._case(4216, K, 5, 24, 128, w_bit, seed=50)
    for M in (1, 48):
        lora._check(case, si.activations(M, K, offset=M), lora._ids("mixed", M, 5, M), "skinny")
