"""Rows before position 0 are no tokens: without a causal mask too they attend to nothing, in both
forms of the attention, beside rows of the same tile that see every token."""

import pytest
import torch

import weight_only_bit_02_amd as awq

from . import kv_exact
from .gpu_util import DEV, guarded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [0, 3, 20])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D,group,share,n,lengths", [
    (128, 128, 1, [3, 2, 2], [1, 0, 2]),       # streamed, 16 rows
    (128, 32, 5, [6, 1], [4, 40]),             # 32 rows
    (64, 64, 2, [20, 9, 30], [5, 300, 18]),
    (256, 128, 3, [7, 7], [6, 7]),
    (128, 64, 4, [90, 80, 70], [30, 0, 1]),    # tiles
    (64, 32, 8, [70, 40], [33, 5]),
    (256, 64, 2, [100, 3], [36, 2]),
])
def test_rows_before_the_sequence(D, group, share, n, lengths, causal, window):
    gen = torch.Generator(DEV).manual_seed(D + group + share)
    i32 = dict(dtype=torch.int32, device=DEV)
    wide = max(-(-x // 16) for x in lengths)
    table = torch.arange(len(n) * wide, **i32).view(len(n), wide)
    cache = awq.alloc_kv_cache(len(n) * wide, 1, D, DEV, page_size=16, group=group)
    ends = [sum(lengths[:s]) for s in range(len(n) + 1)]
    whole = awq.KVBatch(torch.tensor(ends, **i32), torch.tensor(lengths, **i32), table)
    kv = torch.randn(ends[-1], 2, D, generator=gen, device=DEV).half()
    awq.kv_append(cache, whole, kv[:, :1], kv[:, 1:])
    rows = [sum(n[:s]) for s in range(len(n) + 1)]
    q = torch.randn(rows[-1], share, D, generator=gen, device=DEV).half()
    batch = awq.KVBatch(torch.tensor(rows, **i32), whole.lengths, table)
    out, out_check = guarded(q.shape, torch.float16)
    lse, lse_check = guarded(q.shape[:2], torch.float32)
    awq.attention_kv4(q, cache, batch, causal=causal, window=window, out=out, lse=lse)
    out_check(), lse_check()
    for s in range(len(n)):
        r = slice(rows[s], rows[s + 1])
        if lengths[s] == 0:
            assert bool((out[r] == 0).all()) and bool(torch.isneginf(lse[r]).all())
            continue
        want = kv_exact.attention(q[r].cpu().double(), kv_exact.tokens(awq, cache, whole, s, lengths[s]), D ** -0.5, causal,
                                  window, D // group <= 2, n[s] * share > 64)
        kv_exact.check(out[r], lse[r], want)
