"""The streaming kernel's weights are exact for every group size: its error is that of fp32 sums and of the
one rounding of the result (the GEMM's operands are rounded to fp16 besides, see grouped_ref.linear_bound)."""

import numpy as np
import pytest
import torch

import oracle
import synthetic_inputs as si
import weight_only_bit_02_amd as awq
from tests.grouped_ref import TINY, U, linear_reference, packed_numpy
from tests.gpu_util import DEV, host, to_dev

pytestmark = pytest.mark.gpu

FORMATS = [(b, g) for b in (4, 8, 3) for g in (128, 64, 32)]
M = 16


def _inside(Y, y, bound):
    bad = np.abs(Y - y) > bound
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].tolist(), Y[bad][:5], y[bad][:5], bound[bad][:5])


# Products of fp16 values with the two fp16 parts of a weight (which hold it whole) are exact in fp32; K
# of them, or the two parts' 2 K, and the scales of partial sums make fewer than 2 K roundings to fp32,
# 2^-24 each (2^-23 if a matrix core truncates), of sums that S bounds (1 + 2^-11 for the first parts).
def _sums(S, K):
    return S * (2 * K * 2.0 ** -23)


@pytest.mark.parametrize("w_bit,group", FORMATS)
@pytest.mark.parametrize("N,K", [(600, 128), (512, 384)])
@pytest.mark.parametrize("std", [0.02, 3e-5])
def test_linear(std, N, K, w_bit, group):
    """Results near zero beside large products show the operands' roundings; tiny weights, whose second
    parts are the smallest fp16 values."""
    g = np.random.default_rng(K)
    qw, sc, zb, _ = oracle.quantize_pack((g.standard_normal((N, K)) * std).astype(np.float16), group=group, w_bit=w_bit)
    q, z, s = oracle.unpack(qw, sc, zb, K)
    Wd = oracle.dequantize(q, z, s)
    X = g.standard_normal((M, K)).astype(np.float16)
    y, S = linear_reference(X, Wd)
    bound = _sums(S, K) + np.abs(y) * U + TINY
    if std == 0.02:
        assert (np.abs(y) * U < S * 2.0 ** -14).sum() > 50  # results where the operands' roundings would show
    packed = (to_dev(qw.view(np.int32)), to_dev(sc), to_dev(zb))
    x, ids = to_dev(X), torch.zeros(M, dtype=torch.int32, device=DEV)
    Y = awq.linear_w4a16_grouped(x, awq.PackedExperts(*(t[None] for t in packed), 1, N, K, group, w_bit),
                                 awq.group_rows(ids, 1), kernel="skinny")
    _inside(host(Y).astype(np.float64), y, bound)
    lora = awq.LoraAdapters(torch.zeros(1, 8, K, device=DEV).half(), torch.zeros(1, N, 8, device=DEV).half(),
                            torch.zeros(1, device=DEV))
    Y = awq.linear_w4a16_lora(x, awq.PackedLinear(*packed, N, K, group, w_bit), lora, ids - 1, kernel="skinny")
    _inside(host(Y).astype(np.float64), y, bound)


@pytest.mark.parametrize("w_bit,group", FORMATS)
def test_gated(w_bit, group):
    N, K = 800, 256
    (qw, sc, zb), Wd = packed_numpy(N, K, group, w_bit, 3)
    X = si.activations(M, K, offset=3, heavy_tail=False)
    y, S = linear_reference(X, Wd)
    d, nh = _sums(S, K), N // 2
    gate, up, dg, du = y[:, :nh], y[:, nh:], d[:, :nh], d[:, nh:]
    h = oracle.silu(gate) * up
    # |SiLU'| <= 1.1; the fp32 SiLU is good to 2^-18
    bound = 1.1 * dg * (np.abs(up) + du) + np.abs(oracle.silu(gate)) * du + np.abs(h) * (U + 2.0 ** -18) + TINY
    w = awq.PackedExperts(to_dev(qw)[None], to_dev(sc)[None], to_dev(zb)[None], 1, N, K, group, w_bit)
    groups = awq.group_rows(torch.zeros(M, dtype=torch.int32, device=DEV), 1)
    Y = awq.linear_w4a16_grouped_gated_silu(to_dev(X), w, groups, kernel="skinny")
    _inside(host(Y).astype(np.float64), h, bound)
