"""Scores of any size that a scale below 1e20 can give: the softmax is a choice of the largest one, and
every output is a number."""

import pytest
import torch

import weight_only_bit_02_amd as awq

from . import kv_exact
from .gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("scale", [1e5, 1e7, 1e9, 1e13, 9e19])
@pytest.mark.parametrize("D,group,share,n,length", [
    (128, 128, 2, 1, 3000), (64, 32, 3, 2, 500), (128, 32, 2, 1, 3000), (256, 64, 4, 6, 500),  # streamed
    (128, 128, 20, 1, 700), (128, 64, 12, 2, 700), (128, 32, 9, 3, 700),                       # in tiles of 32 rows
    (128, 128, 1, 200, 300), (64, 64, 4, 60, 900), (256, 128, 1, 70, 300),                     # tiles
])
def test_choice(D, group, share, n, length, scale, sign):
    gen = torch.Generator(DEV).manual_seed(D + n)
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.arange(-(-length // 16), **i32)[None]
    cache = awq.alloc_kv_cache(table.shape[1], 1, D, DEV, page_size=16, group=group)
    whole = awq.KVBatch(torch.tensor([0, length], **i32), torch.tensor([length], **i32), table)
    kv = torch.randn(length, 2, D, generator=gen, device=DEV)
    if sign < 0:
        kv[:, 0] = kv[:, 0].abs() + 1  # all scores far below zero
    kv = kv.half()
    awq.kv_append(cache, whole, kv[:, :1], kv[:, 1:])
    # each query one channel of the keys: one product, exact; different ones differ by 2^-11 or more of their size
    q = torch.zeros(n, share, D, dtype=torch.float16, device=DEV)
    q.scatter_(2, torch.randint(0, D, (n, share, 1), generator=gen, device=DEV), float(sign))
    lse = torch.empty(n, share, device=DEV)
    y = awq.attention_kv4(q, cache, awq.KVBatch(torch.tensor([0, n], **i32), whole.lengths, table), scale=scale, lse=lse)
    assert bool(y.isfinite().all()) and bool(lse.isfinite().all())
    k, v, _ = kv_exact.tokens(awq, cache, whole, 0, length)
    low, high = torch.zeros(2, n, share, D, dtype=torch.float64)
    want_lse = torch.zeros(n, share, dtype=torch.float64)
    for i in range(n):
        for h in range(share):
            s = (k[:length - n + i + 1, 0] @ q[i, h].cpu().double())
            best = v[:length - n + i + 1, 0][s == s.max()]
            low[i, h], high[i, h] = best.amin(0), best.amax(0)
            want_lse[i, h] = s.max() * scale
    # Ties lie anywhere between: equal keys of different codes and scales, n_1 s_1 = n_2 s_2, have the scores n_1 fl(s_1 c) and
    # n_2 fl(s_2 c), rounded, in the streaming form; they differ by up to 2^-23 of their size, a unit of log2 from 2^23 on.
    # A probability is rounded to fp16 in the tile form (2^-11) while the sum keeps it, then the output (2^-11); as
    # hi + lo with the values' scales 2^-22 of values (below 8) that may cancel.
    off = 2.0 ** -10 * 1.01 * torch.maximum(low.abs(), high.abs()) + 2.0 ** -19
    y = y.cpu().double()
    assert bool((y >= low - off).all()) and bool((y <= high + off).all())
    # (the scale itself is rounded to fp32, times 1 / ln 2, ln 2; the log of a few ties is below 2)
    assert bool(((lse.cpu().double() - want_lse).abs() <= 2.0 ** -21 * want_lse.abs() + 2).all())


FORMS = [(128, 128, 2, 5), (128, 64, 5, 4), (64, 32, 1, 20), (128, 32, 2, 6), (256, 64, 7, 4), (256, 128, 1, 3),
         (128, 128, 2, 90), (64, 64, 8, 30), (256, 64, 2, 60)]


def one_sequence(k, v, group):
    length, D = k.shape
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.arange(-(-length // 16), **i32)[None]
    cache = awq.alloc_kv_cache(table.shape[1], 1, D, DEV, page_size=16, group=group)
    whole = awq.KVBatch(torch.tensor([0, length], **i32), torch.tensor([length], **i32), table)
    awq.kv_append(cache, whole, k[:, None].half(), v[:, None].half())
    return cache, whole


@pytest.mark.parametrize("D,group,share,n", FORMS)
def test_rows_of_different_size(D, group, share, n):
    """Rows whose scores are zero, some tens and some 2^30 in one tile: each as if it were alone."""
    gen = torch.Generator(DEV).manual_seed(D + n)
    length, scale = 400, 1e9
    kv = torch.randn(2, length, D, generator=gen, device=DEV)
    cache, whole = one_sequence(*kv, group)
    q = torch.zeros(n * share, D, dtype=torch.float16, device=DEV)
    size = torch.tensor([0.0, 2.0 ** -24, 1.0, -1.0], dtype=torch.float16, device=DEV)[torch.arange(n * share, device=DEV) % 4]
    q.scatter_(1, torch.randint(0, D, (n * share, 1), generator=gen, device=DEV), size[:, None])
    q = q.view(n, share, D)
    lse = torch.empty(n, share, device=DEV)
    rows = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    y = awq.attention_kv4(q, cache, awq.KVBatch(rows, whole.lengths, whole.page_table), scale=scale, lse=lse)
    kvs = kv_exact.tokens(awq, cache, whole, 0, length)
    out, want_lse, bound, lse_bound = kv_exact.attention(q.cpu().double(), kvs, scale, True, 0, D // group <= 2, n * share > 64)
    far = size.cpu().abs().view(n, share) == 1
    for i, h in far.nonzero().tolist():  # one product, exact: the bound of a score's sum does not apply (test_choice)
        bound[i, h] = 2.0 ** -10 * 1.01 * out[i, h].abs() + 2.0 ** -19
        lse_bound[i, h] = 2.0 ** -21 * want_lse[i, h].abs() + 2
    kv_exact.check(y, lse, (out, want_lse, bound, lse_bound))


@pytest.mark.parametrize("D,group,share,n", FORMS)
@pytest.mark.parametrize("first", [0, 1, 200, 399])
def test_tokens_of_different_size(D, group, share, n, first):
    """Tokens that score -2^30 or so, before or among tokens that score zero: the latter's mean, exactly weighed."""
    gen = torch.Generator(DEV).manual_seed(D + n + first)
    length = 400
    k, v = torch.randn(2, length, D, generator=gen, device=DEV)
    k[:, 0] = -k[:, 0].abs() - 1
    zero = torch.arange(length, device=DEV) >= first
    if first == 1:
        zero = torch.rand(length, generator=gen, device=DEV) < 0.2
        zero[0] = True
    k[zero, 0] = 0
    cache, whole = one_sequence(k, v, group)
    q = torch.zeros(n, share, D, dtype=torch.float16, device=DEV)
    q[:, :, 0] = 1
    rows = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    lse = torch.empty(n, share, device=DEV)
    y = awq.attention_kv4(q, cache, awq.KVBatch(rows, whole.lengths, whole.page_table), scale=1e9, lse=lse).cpu().double()
    _, values, _ = kv_exact.tokens(awq, cache, whole, 0, length)
    zero = zero.cpu()
    for i in range(n):
        seen = zero[:length - n + i + 1].nonzero()[:, 0]
        if len(seen) == 0:
            continue  # (its largest score is -2^30: test_choice)
        vv = values[seen, 0]
        # equal probabilities, one rounding for all of them; 2^-22 of the values from hi + lo; the sums' and the output's own
        off = 2.0 ** -11 * vv.mean(0).abs() + (2.0 ** -22 + len(seen) * 2.0 ** -24) * vv.abs().mean(0)
        bound = off + 2.0 ** -11 * (vv.mean(0).abs() + off) + 2.0 ** -25
        assert bool(((y[i] - vv.mean(0)).abs() <= bound).all())
        want = torch.tensor(float(len(seen))).log()
        assert bool(((lse[i].cpu() - want).abs() <= 2.0 ** -20 + len(seen) * 2.0 ** -24).all())
