"""GPU parity of the router and the grouping of rows (awq_moe_route, awq_group_rows)."""

import numpy as np
import pytest
import torch

import weight_only_bit_02_amd as awq
from tests.gpu_util import DEV, flags_tensor, guarded, host, to_dev
from tests.grouped_ref import group_reference, route_reference

pytestmark = pytest.mark.gpu

I32, F32 = torch.int32, torch.float32


def _out_groups(n, groups):
    outs = [guarded((groups + 1,), I32), guarded((n,), I32), guarded((n,), I32)]
    return awq.RowGroups(*(o for o, _ in outs)), lambda: [c() for _, c in outs]


def _check_groups(got, ids, groups):
    for name, g, r in zip(("offsets", "order", "pos"), (got.offsets, got.order, got.pos),
                          group_reference(ids.reshape(-1), groups)):
        assert np.array_equal(host(g), r), name


@pytest.mark.parametrize("n", [1, 63, 64, 65, 1000, 8192, 8193, 20011, 600000])
@pytest.mark.parametrize("groups", [1, 2, 33, 512])
def test_group_rows(n, groups):
    g = np.random.default_rng(n + groups)
    ids = g.integers(-1, groups, n).astype(np.int32)
    ids[g.random(n) < 0.02] = groups + 7   # out of range on either side: no group
    ids[g.random(n) < 0.02] = -(2 ** 31)
    out, check = _out_groups(n, groups)
    got = awq.group_rows(to_dev(ids), groups, out=out)
    _check_groups(got, ids, groups)
    check()


@pytest.mark.parametrize("n,fill", [(1, -1), (5000, -1), (5000, 3), (9000, 0), (9000, -1)])
def test_group_rows_of_one_kind(n, fill):
    """All rows in one group, or in none."""
    ids = np.full(n, fill, np.int32)
    _check_groups(awq.group_rows(to_dev(ids), 8), ids, 8)


def _route(x, k, renorm, flags=None, E=None):
    T, E = x.shape
    n = T * k
    w, cw = guarded((T, k), F32)
    i, ci = guarded((T, k), I32)
    gr, cg = _out_groups(n, E)
    r = awq.moe_route(x, k, renormalize=renorm, out=awq.Routing(w, i, gr), flags=flags)
    torch.cuda.synchronize()
    cw(), ci(), cg()
    return r


def _check_route(r, x, k, renorm, E):
    w, ids, tol = route_reference(x.astype(np.float64), k, renorm)
    assert np.array_equal(host(r.ids), ids)
    assert np.all(np.abs(host(r.weights).astype(np.float64) - w) <= tol)
    _check_groups(r.groups, ids, E)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (2, 3, 3), (63, 65, 2), (64, 128, 64), (65, 128, 8),
                                   (300, 60, 6), (1000, 256, 5), (257, 512, 64), (4111, 8, 2)])
def test_route(T, E, k, half):
    g = np.random.default_rng(T * E + k)
    x = (g.standard_normal((T, E)) * 3).astype(np.float16 if half else np.float32)
    if half and T > 8:
        x[::3] = np.round(x[::3])  # many ties
    for renorm in (True, False):
        _check_route(_route(to_dev(x), k, renorm), x, k, renorm, E)


@pytest.mark.parametrize("T", [5, 200])
@pytest.mark.parametrize("half", [True, False])
def test_route_masks(T, half):
    """Masked experts (-inf), padded tokens (all -inf), the type's lowest value, equal rows."""
    E, k = 70, 6
    dt = np.float16 if half else np.float32
    g = np.random.default_rng(7)
    x = g.standard_normal((T, E)).astype(dt)
    x[0] = -np.inf
    x[1] = -np.inf
    x[1, [3, 66]] = [1.0, 2.0]     # fewer experts than choices
    x[2] = np.finfo(dt).min        # all equal at the lowest value
    x[3, 1:] = np.finfo(dt).min    # one real logit
    x[4] = 0.0
    flags = flags_tensor()
    for renorm in (True, False):
        _check_route(_route(to_dev(x), k, renorm, flags), x, k, renorm, E)
    assert int(host(flags)[0]) == 0


@pytest.mark.parametrize("T", [4, 100])
@pytest.mark.parametrize("half", [True, False])
def test_route_nonfinite(T, half):
    """NaN counts as -inf, +inf as the largest finite value; both raise the flag."""
    E, k = 40, 4
    dt = np.float16 if half else np.float32
    x = np.random.default_rng(9).standard_normal((T, E)).astype(dt)
    x[0, 5] = np.nan
    x[1, [7, 30]] = np.inf
    x[2] = np.nan
    flags = flags_tensor()
    r = _route(to_dev(x), k, True, flags)
    assert int(host(flags)[0]) == 1
    ref = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(dt).max)).astype(dt)
    _check_route(r, ref, k, True, E)


@pytest.mark.parametrize("half", [True, False])
def test_route_strided_rows(half):
    """Logits as columns of a wider matrix, at an address of the element's alignment only."""
    T, E, k = 77, 33, 3
    x = np.random.default_rng(3).standard_normal((T, 51)).astype(np.float16 if half else np.float32)
    _check_route(_route(to_dev(x)[:, 5:5 + E], k, True), x[:, 5:5 + E], k, True, E)


def test_route_runs_are_identical():
    x = torch.randn(3000, 128, device=DEV).half()
    a, b = awq.moe_route(x, 8), awq.moe_route(x, 8)
    for s, t in ((a.weights, b.weights), (a.ids, b.ids), (a.groups.order, b.groups.order)):
        assert torch.equal(s, t)


@pytest.mark.parametrize("groups", [3, 400])
def test_group_rows_of_a_very_large_batch(groups):
    """More rows per block than its threads hold at once."""
    n = 2_200_003
    ids = np.random.default_rng(groups).integers(-1, groups + 1, n).astype(np.int32)
    _check_groups(awq.group_rows(to_dev(ids), groups), ids, groups)


def test_route_of_a_very_large_batch():
    x = np.random.default_rng(1).standard_normal((70001, 40)).astype(np.float32)
    _check_route(_route(to_dev(x), 32, True), x, 32, True, 40)
