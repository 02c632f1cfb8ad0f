"""GPU parity of the experts' linears and the combine against fp64 forms."""

import numpy as np
import pytest
import torch

import synthetic_inputs as si
import weight_only_bit_02_amd as awq
from tests.gpu_util import DEV, flags_tensor, guarded, host, to_dev
from tests.grouped_ref import (U, TINY, gated_reference, group_reference, linear_bound, linear_reference,
                               packed_numpy)

pytestmark = pytest.mark.gpu

KERNELS = ["skinny", "gemm64", "gemm128", "gemm256", "gemm64k", "auto"]
FORMATS = [(4, 128), (4, 64), (4, 32), (8, 128), (8, 64), (8, 32), (3, 128), (3, 64), (3, 32)]


def _experts(E, N, K, group, w_bit, seed):
    parts = [packed_numpy(N, K, group, w_bit, seed + e) for e in range(E)]
    stack = [to_dev(np.stack([p[0][i] for p in parts])) for i in range(3)]
    return awq.PackedExperts(*stack, E, N, K, group, w_bit), [p[1] for p in parts]


def _groups(sizes, rng, tail=0):
    """A batch whose group e has sizes[e] rows, in random order, `tail` rows without one."""
    ids = np.concatenate([np.full(s, e) for e, s in enumerate(sizes)] + [np.full(tail, -1)]).astype(np.int32)
    ids = rng.permutation(ids)
    ref = group_reference(ids, len(sizes))
    return awq.RowGroups(*(to_dev(a) for a in ref)), ref


FILL = -77.0


def _run(w, Wd, sizes, gated, kernel, fan, tail, seed):
    rng = np.random.default_rng(seed)
    n = sum(sizes) + tail
    tail += -n % (fan or 1)
    n = sum(sizes) + tail
    groups, (offsets, order, _) = _groups(sizes, rng, tail)
    X = si.activations(n // fan if fan else n, w.K, offset=seed)
    outs = w.N // 2 if gated else w.N
    out, check = guarded((n, outs), torch.float16)
    out.fill_(FILL)
    f = awq.linear_w4a16_grouped_gated_silu if gated else awq.linear_w4a16_grouped
    Y = host(f(to_dev(X), w, groups, fan=fan, out=out, kernel=kernel)).astype(np.float64)
    check()
    xs = X[order // fan] if fan else X
    for e in range(len(sizes)):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            continue
        if gated:
            y, bound = gated_reference(xs[lo:hi], Wd[e])
        else:
            y, S = linear_reference(xs[lo:hi], Wd[e])
            bound = linear_bound(y, S, w.K)
        bad = np.abs(Y[lo:hi] - y) > bound
        assert not bad.any(), (e, np.argwhere(bad)[:5].tolist(), Y[lo:hi][bad][:5], y[bad][:5])
    assert np.all(Y[offsets[-1]:] == FILL)  # rows without a group are left as they were


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("w_bit,group", FORMATS)
def test_formats(w_bit, group, gated, kernel):
    w, Wd = _experts(5, 70, 384, group, w_bit, seed=10)
    _run(w, Wd, [3, 0, 40, 1, 9], gated, kernel, None, 4, seed=11)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("sizes", [[1], [0, 0, 1], [32, 33, 0, 31], [64, 65, 63], [8, 9, 16, 17], [130, 257, 5, 0, 129]])
def test_ragged_sizes(sizes, gated, kernel):
    """Every row-tile body and accumulator bucket, groups that end inside and on a tile."""
    w, Wd = _experts(len(sizes), 300 if gated else 259, 256, 128, 4, seed=20)
    _run(w, Wd, sizes, gated, kernel, None, 0, seed=21)


@pytest.mark.parametrize("w_bit", [8, 3])
@pytest.mark.parametrize("gated", [False, True])
def test_ragged_sizes_other_widths(w_bit, gated):
    w, Wd = _experts(4, 260, 256, 64, w_bit, seed=23)
    for kernel in KERNELS:
        _run(w, Wd, [200, 33, 0, 70], gated, kernel, None, 3, seed=24)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("N,K", [(1, 128), (2, 128), (7, 1152), (513, 640)])
def test_odd_shapes(N, K, kernel):
    """One and few outputs, one and an odd number of K steps; weights of odd sizes in a stack."""
    w, Wd = _experts(3, N, K, 128, 4, seed=30)
    _run(w, Wd, [5, 20, 66], False, kernel, None, 0, seed=31)
    if N % 2 == 0:
        _run(w, Wd, [5, 20, 66], True, kernel, None, 0, seed=32)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fan", [1, 2, 6])
def test_gathered_rows(fan, gated, kernel):
    w, Wd = _experts(6, 128, 256, 128, 4, seed=40)
    _run(w, Wd, [11, 0, 70, 35, 1, 3], gated, kernel, fan, 6, seed=41)


@pytest.mark.parametrize("kernel", KERNELS)
def test_many_groups(kernel):
    """More groups than a wave has lanes, most of them empty."""
    rng = np.random.default_rng(5)
    sizes = [int(s) for s in rng.integers(0, 4, 150) * (rng.random(150) < 0.3)]
    sizes[149] = 2
    w, Wd = _experts(150, 33, 128, 128, 4, seed=50)
    _run(w, Wd, sizes, False, kernel, None, 1, seed=51)


@pytest.mark.parametrize("kernel", KERNELS)
def test_no_rows_in_any_group(kernel):
    w, Wd = _experts(3, 64, 128, 128, 4, seed=60)
    _run(w, Wd, [0, 0, 0], False, kernel, None, 9, seed=61)
    _run(w, Wd, [0, 0, 0], True, kernel, 3, 9, seed=61)


@pytest.mark.parametrize("w_bit,group", [(4, 128), (4, 64), (4, 32), (3, 128), (8, 128)])
@pytest.mark.parametrize("gated", [False, True])
def test_one_group_equals_the_plain_linear(w_bit, group, gated):
    """The GEMM tiles multiply the same fp16 operands in the same order along K."""
    N, K, M = 512, 1152, 300
    w, _ = _experts(1, N, K, group, w_bit, seed=70)
    p = awq.PackedLinear(w.qweight[0], w.scales[0], w.zeros[0], N, K, group, w_bit)
    X = to_dev(si.activations(M, K, offset=71))
    ids = awq.group_rows(torch.zeros(M, dtype=torch.int32, device=DEV), 1)
    f, h = ((awq.linear_w4a16_gated_silu, awq.linear_w4a16_grouped_gated_silu) if gated
            else (awq.linear_w4a16, awq.linear_w4a16_grouped))
    ref = f(X, p, kernel="gemm")
    for kernel in ("gemm64", "gemm128", "gemm256"):
        assert torch.equal(h(X, w, ids, kernel=kernel), ref)
        assert torch.equal(h(X, w, ids, fan=1, kernel=kernel), ref)


@pytest.mark.parametrize("kernel", ["skinny", "gemm64", "gemm128", "gemm256", "gemm64k"])
def test_wrong_device_contents_stay_in_bounds(kernel):
    """Offsets and orders that say anything: no write outside the output, no fault."""
    E, N, K, n = 4, 40, 256, 50
    w, _ = _experts(E, N, K, 128, 4, seed=80)
    X = to_dev(si.activations(n, K, offset=81))
    for offsets in ([0, 10, 20, 30, 10 ** 9], [-5, 60, 2, 2 ** 31 - 1, 7], [2 ** 31 - 1, -(2 ** 31), 0, 9, 9]):
        for o in (None, 2 ** 31 - 1, -3):
            order = np.arange(n, dtype=np.int32) if o is None else np.full(n, o, np.int32)
            g = awq.RowGroups(to_dev(np.array(offsets, np.int32)), to_dev(order), to_dev(order))
            out, check = guarded((n, N), torch.float16)
            awq.linear_w4a16_grouped(X, w, g, fan=1, out=out, kernel=kernel)
            check()


def test_flags():
    w, _ = _experts(2, 32, 128, 128, 4, seed=90)
    X = si.activations(6, 128, offset=91)
    groups, _ = _groups([3, 3], np.random.default_rng(1))
    f = flags_tensor()
    awq.linear_w4a16_grouped(to_dev(X), w, groups, flags=f)
    assert int(host(f)[0]) == 0
    X[5, 127] = np.inf
    awq.linear_w4a16_grouped(to_dev(X), w, groups, flags=f)
    assert int(host(f)[0]) == 1
    f.zero_()
    w.scales[1, 31, 0] = float("nan")
    awq.linear_w4a16_grouped_gated_silu(to_dev(si.activations(6, 128, offset=91)), w, groups, flags=f)
    assert int(host(f)[0]) == 1


@pytest.mark.parametrize("kernel", KERNELS)
def test_nonfinite_row_stays_in_its_row(kernel):
    """An Inf or NaN row of X reaches no other row; a group's weights reach no other group."""
    w, Wd = _experts(2, 64, 256, 128, 4, seed=95)
    X = si.activations(70, 256, offset=96)
    groups, (offsets, _, _) = _groups([40, 30], np.random.default_rng(2))
    clean = host(awq.linear_w4a16_grouped(to_dev(X), w, groups, kernel=kernel))
    X[3, 9], X[50, 0] = np.nan, np.inf
    got = host(awq.linear_w4a16_grouped(to_dev(X), w, groups, kernel=kernel))
    rest = [i for i in range(70) if i not in (3, 50)]
    assert np.array_equal(got[rest].view(np.uint16), clean[rest].view(np.uint16))
    assert not np.isfinite(got[3]).any()


def test_pack_experts():
    E, N, K = 3, 5, 256   # scales of one expert: 20 bytes, no multiple of 16
    W = to_dev(np.stack([si.weights(N, K, offset=e) for e in range(E)]))
    s = (torch.rand(E, K, device=DEV) + 0.5).half()
    for w_bit, group in ((4, 128), (3, 32), (8, 64)):
        for scales in (None, s[0], s):
            w = awq.quantize_pack_experts(W, scales, group_size=group, w_bit=w_bit)
            for e in range(E):
                se = scales if scales is None or scales.dim() == 1 else scales[e].contiguous()
                p = awq.quantize_pack(W[e].contiguous(), se, group_size=group, w_bit=w_bit)
                for a, b in ((w.qweight, p.qweight), (w.scales, p.scales), (w.zeros, p.zeros)):
                    assert torch.equal(a[e], b)


# ------------------------------------------------------------------ combine

@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (1, 8, 4096), (3, 5, 7), (130, 2, 264), (33, 64, 24), (700, 6, 1000)])
@pytest.mark.parametrize("add", [False, True])
def test_combine(T, k, N, add):
    rng = np.random.default_rng(T + N)
    E = 64
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    ids[rng.random((T, k)) < 0.2] = -1
    offsets, order, pos = group_reference(ids.reshape(-1), E)
    P = rng.standard_normal((T * k, N)).astype(np.float16)
    P[offsets[-1]:] = np.nan           # rows without an expert: whatever they hold, unread
    w = rng.random((T, k)).astype(np.float32)
    a = rng.standard_normal((T, N)).astype(np.float16) if add else None
    groups = awq.RowGroups(to_dev(offsets), to_dev(order), to_dev(pos))
    out, check = guarded((T, N), torch.float16)
    Y = host(awq.moe_combine(to_dev(P), to_dev(w), groups, add=to_dev(a) if add else None, out=out))
    check()
    p = pos.reshape(T, k)
    on = p < offsets[-1]
    terms = np.where(on[..., None], P.astype(np.float64)[p] * w.astype(np.float64)[..., None], 0.0)
    y, S = terms.sum(1), np.abs(terms).sum(1)
    if add:
        y, S = y + a, S + np.abs(a)
    # fp32 fma over k + 1 terms, then one rounding to fp16
    assert np.all(np.abs(Y - y) <= S * (k + 1) * 2.0 ** -24 + np.abs(y) * U + TINY)


def test_combine_in_place_and_wrong_positions():
    T, k, N = 9, 3, 16
    P = torch.randn(T * k, N, device=DEV).half()
    w = torch.rand(T, k, device=DEV)
    g = awq.group_rows(torch.arange(T * k, dtype=torch.int32, device=DEV) % 4, 4)
    add = torch.randn(T, N, device=DEV).half()
    ref = awq.moe_combine(P, w, g, add=add)
    assert torch.equal(awq.moe_combine(P, w, g, add=add, out=add), ref)
    g.pos.fill_(2 ** 31 - 1)
    g.offsets.fill_(2 ** 31 - 1)
    assert not awq.moe_combine(P, w, g).any()
    g.pos.fill_(-4)
    assert not awq.moe_combine(P, w, g).any()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("w_bit,group", [(4, 128), (4, 32), (8, 64), (3, 128)])
@pytest.mark.parametrize("K", [128, 256, 640, 1664, 4480])
def test_numbers_of_k_steps(K, w_bit, group, kernel):
    """From a single K step, fewer than the waves and buffers that share them, to several rounds."""
    w, Wd = _experts(4, 72, K, group, w_bit, seed=K)
    _run(w, Wd, [5, 0, 33, 70], False, kernel, None, 3, seed=K + 1)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("w_bit,K", [(4, 128), (4, 640), (8, 384), (3, 256)])
@pytest.mark.parametrize("kernel", ["skinny", "gemm64k", "auto"])
def test_many_column_chunks(kernel, w_bit, K, gated):
    """Enough columns that every XCD takes its share of the chunks, the last one partly filled."""
    w, Wd = _experts(3, 4216, K, 128, w_bit, seed=40 + w_bit)
    _run(w, Wd, [17, 0, 40], gated, kernel, 2, 2, seed=41)
