"""Tokens that no row of a tile sees may hold anything, like pages that nobody wrote: those before the
window lie in the same 64 tokens, or the same step, as the first ones that are seen."""

import pytest
import torch

import weight_only_bit_02_amd as awq

from . import kv_exact
from .gpu_util import DEV

pytestmark = pytest.mark.gpu

INF, NAN, LARGEST = 0x7C00, 0x7FFF, 0x6C40  # LARGEST: 4352


@pytest.mark.parametrize("D,group,share,n,length,window", [
    (128, 128, 4, 1, 300, 100),
    (128, 64, 16, 1, 300, 5),
    (128, 32, 4, 1, 300, 100),
    (64, 64, 3, 7, 700, 130),
    (64, 32, 20, 3, 130, 1),
    (256, 128, 2, 1, 300, 63),
    (256, 64, 5, 6, 200, 40),
    (128, 128, 2, 100, 400, 90),   # tiles
    (128, 32, 4, 40, 1000, 77),
    (64, 64, 4, 70, 600, 33),
    (64, 32, 8, 300, 300, 20),     # (windows that reach the start: nothing is stale)
    (256, 128, 2, 90, 500, 120),
])
@pytest.mark.parametrize("page", [16, 64])
def test_before_the_window(D, group, share, n, length, window, page):
    gen = torch.Generator(DEV).manual_seed(D + group + n)
    i32 = dict(dtype=torch.int32, device=DEV)
    wide = -(-length // page)
    table = torch.randperm(wide, generator=gen, device=DEV).to(torch.int32)[None]
    cache = awq.alloc_kv_cache(wide, 1, D, DEV, page_size=page, group=group)
    whole = awq.KVBatch(torch.tensor([0, length], **i32), torch.tensor([length], **i32), table)
    kv = torch.randn(length, 2, D, generator=gen, device=DEV).half()
    awq.kv_append(cache, whole, kv[:, :1], kv[:, 1:])
    q = torch.randn(n, share, D, generator=gen, device=DEV).half()
    batch = awq.KVBatch(torch.tensor([0, n], **i32), whole.lengths, table)

    def run():
        lse = torch.empty(n, share, device=DEV)
        return awq.attention_kv4(q, cache, batch, window=window, lse=lse), lse

    want = kv_exact.attention(q.cpu().double(), kv_exact.tokens(awq, cache, whole, 0, length), D ** -0.5, True, window,
                              D // group <= 2, n * share > 64)
    kv_exact.check(*run(), want)
    stale = torch.arange(max(0, length - n - window + 1), device=DEV)
    at, place = table[0, stale // page].long(), stale % page
    results = []
    for param in (0, INF, NAN, LARGEST):
        for name in ("k_params", "v_params"):
            getattr(cache, name)[at, :, :, place] = param
        results.append(run())
        kv_exact.check(*results[-1], want)
    for y, lse in results[1:]:
        assert torch.equal(y, results[0][0]) and torch.equal(lse, results[0][1])
