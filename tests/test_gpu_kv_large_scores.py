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
    want = torch.zeros(n, share, D, dtype=torch.float64)
    want_lse = torch.zeros(n, share, dtype=torch.float64)
    for i in range(n):
        for h in range(share):
            s = (k[:length - n + i + 1, 0] @ q[i, h].cpu().double())
            best = s == s.max()  # ties are halved
            want[i, h] = v[:length - n + i + 1, 0][best].mean(0)
            want_lse[i, h] = s.max() * scale
    # ties have one probability, rounded to fp16 in the tile form (2^-11) while the sum keeps it, then the output's own
    # rounding (2^-11); as hi + lo with the values' scales 2^-22 of ties whose values (below 8) may cancel
    assert bool(((y.cpu().double() - want).abs() <= 2.0 ** -10 * 1.01 * want.abs() + 2.0 ** -19).all())
    # (the scale itself is rounded to fp32, times 1 / ln 2, ln 2; the log of a few ties is below 2)
    assert bool(((lse.cpu().double() - want_lse).abs() <= 2.0 ** -21 * want_lse.abs() + 2).all())
