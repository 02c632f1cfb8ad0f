"""Rows with one token far above all others, whose value is zero: the output is made of
probabilities of 2^-20 to 2^-30 alone."""

import pytest
import torch

import weight_only_bit_02_amd as awq

from . import kv_exact
from .gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nats", [14, 16, 18])
@pytest.mark.parametrize("D,group,share,n", [
    (128, 32, 2, 1), (256, 64, 3, 2), (256, 32, 1, 20),              # streamed, scales in the operands
    (128, 128, 2, 1), (64, 32, 20, 1),                               # streamed, scales on the probabilities
    (128, 128, 2, 80), (64, 64, 4, 40), (256, 64, 2, 50),            # tiles
])
def test_one_token_above_all(D, group, share, n, nats):
    length = 4000
    gen = torch.Generator(DEV).manual_seed(nats + D)
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.arange(-(-length // 64), **i32)[None]
    cache = awq.alloc_kv_cache(table.shape[1], 1, D, DEV, group=group)
    whole = awq.KVBatch(torch.tensor([0, length], **i32), torch.tensor([length], **i32), table)
    kv = torch.randn(length, 2, D, generator=gen, device=DEV) * torch.tensor([[0.1], [1.0]], device=DEV)
    kv[:, 1] += 1  # a sum that does not average out
    kv[0, 0], kv[0, 1] = 1, 0
    kv = kv.half()
    awq.kv_append(cache, whole, kv[:, :1], kv[:, 1:])
    # the first token's keys are all one: it scores `nats`, the others within half a nat or so
    q = (torch.randn(n, share, D, generator=gen, device=DEV) * 0.2 + nats * D ** -0.5).half()
    lse = torch.empty(n, share, device=DEV)
    y = awq.attention_kv4(q, cache, awq.KVBatch(torch.tensor([0, n], **i32), whole.lengths, table), lse=lse)
    want = kv_exact.attention(q.cpu().double(), kv_exact.tokens(awq, cache, whole, 0, length), D ** -0.5, True, 0,
                              D // group <= 2, n * share > 64)
    kv_exact.check(y, lse, want)
