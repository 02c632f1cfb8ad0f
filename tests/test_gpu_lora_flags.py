"""NONFINITE_INPUT of the linear with adapters: the adapters' scales, with and without rows of theirs."""

import numpy as np
import pytest
import torch

import synthetic_inputs as si
import weight_only_bit_02_amd as awq
from tests.grouped_ref import packed_numpy
from tests.gpu_util import DEV, flags_tensor, host, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L", [1, 300])
@pytest.mark.parametrize("M", [3, 100])
def test_scales(L, M):
    (qw, sc, zb), _ = packed_numpy(64, 128, 128, 4, 13)
    w = awq.PackedLinear(to_dev(qw), to_dev(sc), to_dev(zb), 64, 128)
    A, B = torch.ones(L, 8, 128, device=DEV).half(), torch.ones(L, 64, 8, device=DEV).half()
    X, ids = to_dev(si.activations(M, 128, offset=M)), torch.zeros(M, dtype=torch.int32, device=DEV)

    def flag(value, at):
        scale = torch.full((L,), 3.0e38, device=DEV)  # the largest scales are no Inf
        scale[at] = value
        f = flags_tensor()
        awq.linear_w4a16_lora(X, w, awq.LoraAdapters(A, B, scale), ids, flags=f)
        return int(host(f)[0])
    for at in (0, L - 1):
        assert flag(-3.0e38, at) == 0
        for value in (np.inf, -np.inf, np.nan):
            assert flag(value, at) == 1
