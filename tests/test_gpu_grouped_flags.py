"""What raises NONFINITE_INPUT in the experts' linears: the rows that an output is made of."""

import numpy as np
import pytest
import torch

import synthetic_inputs as si
import weight_only_bit_02_amd as awq
from tests.grouped_ref import group_reference, packed_numpy
from tests.gpu_util import flags_tensor, host, to_dev

pytestmark = pytest.mark.gpu

E, N, K = 3, 64, 256


def _weights():
    parts = [packed_numpy(N, K, 128, 4, e) for e in range(E)]
    return awq.PackedExperts(*(to_dev(np.stack([p[0][i] for p in parts])) for i in range(3)), E, N, K)


@pytest.mark.parametrize("f", [awq.linear_w4a16_grouped, awq.linear_w4a16_grouped_gated_silu])
@pytest.mark.parametrize("n,live", [(1, 0), (1, 1), (9, 4), (3000, 2999), (3000, 1), (3000, 0)])
def test_rows_without_a_group_are_not_looked_at(f, n, live):
    w = _weights()
    ids = np.full(n, -1, np.int32)
    ids[:live] = np.random.default_rng(n).integers(0, E, live)
    groups = awq.RowGroups(*(to_dev(a) for a in group_reference(ids, E)))
    X = si.activations(n, K, offset=n)
    X[live:] = np.nan
    flags = flags_tensor()
    f(to_dev(X), w, groups, flags=flags)
    assert int(host(flags)[0]) == 0
    for row in {0, live - 1} if live else ():
        Z = X.copy()
        Z[row, K - 1] = np.inf
        flags.zero_()
        f(to_dev(Z), w, groups, flags=flags)
        assert int(host(flags)[0]) == 1


def test_gathered_rows_are_all_looked_at():
    w = _weights()
    groups = awq.RowGroups(*(to_dev(a) for a in group_reference(np.array([0, -1, -1, 1], np.int32), E)))
    X = si.activations(4, K, offset=1)
    X[1, 3] = np.nan
    flags = flags_tensor()
    awq.linear_w4a16_grouped(to_dev(X), w, groups, fan=1, flags=flags)
    assert int(host(flags)[0]) == 1


@pytest.mark.parametrize("value", [-(2 ** 31), -1, 2 ** 31 - 1])
def test_wrong_offsets_stay_in_bounds(value):
    """The last offset says anything: the rows looked at stay within X."""
    w = _weights()
    X = to_dev(si.activations(5, K, offset=2))
    order = torch.arange(5, dtype=torch.int32, device=X.device)
    groups = awq.RowGroups(to_dev(np.array([0, 1, 2, value], np.int32)), order, order)
    flags = flags_tensor()
    awq.linear_w4a16_grouped(X, w, groups, flags=flags)
    assert int(host(flags)[0]) == 0


@pytest.mark.parametrize("masked", [2, 40])
def test_block_with_padded_tokens(masked):
    """gate|up leaves the rows of padded tokens as they were; the down linear does not take them for input."""
    T, top = 60, 2
    g = np.random.default_rng(3)
    logits = g.standard_normal((T, E)).astype(np.float32)
    logits[:masked] = -np.inf
    r = awq.moe_route(to_dev(logits), top)
    up, down = _weights(), _weights()
    flags = flags_tensor()
    x = to_dev(si.activations(T, K, offset=4))
    h = torch.full((T * top, N // 2), float("nan"), dtype=torch.float16, device=x.device)
    awq.linear_w4a16_grouped_gated_silu(x, up, r.groups, fan=top, out=h, flags=flags)
    wide = torch.full((T * top, K), float("nan"), dtype=torch.float16, device=x.device)
    live = int(host(r.groups.offsets)[-1])
    assert live == (T - masked) * top
    wide[:live] = h[:live].repeat(1, K // (N // 2))
    awq.linear_w4a16_grouped(wide, down, r.groups, flags=flags)
    assert int(host(flags)[0]) == 0
