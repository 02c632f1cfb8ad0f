"""The 4-bit cache and its attention at the ends of their ranges: parameters past 4 GiB, page tables far
wider than the sequences, as many rows as the streaming form takes."""

import pytest
import torch

import weight_only_bit_02_amd as awq

from . import kv_exact
from .gpu_util import DEV

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("D,group", [(64, 32), (128, 32), (256, 64)])
def test_parameters_beyond_4_gib(D, group):
    """Pages whose parameters lie past 2^32 bytes (codes past 2^34) hold and give what the first pages do."""
    heads, size = 32, 256
    pages = (1 << 32) // (heads * (D // group) * size * 2) + 5
    need = 2 * pages * heads * size * (D // 2 + 2 * (D // group))
    if torch.cuda.mem_get_info()[0] < need + (8 << 30):
        pytest.skip("needs %d GiB" % (need >> 30))
    cache = awq.alloc_kv_cache(pages, heads, D, DEV, page_size=size, group=group)
    assert cache.v_params.numel() * 2 > 1 << 32
    gen = torch.Generator(DEV).manual_seed(D)
    lengths = [500, 300]
    kv = torch.randn(800, 2 * heads, D, generator=gen, device=DEV).half()
    rows, at = torch.tensor([0, 500, 800], **I32), torch.tensor(lengths, **I32)
    outs = []
    for first in (0, pages - 4):
        table = torch.tensor([[first, first + 1], [first + 3, first + 2]], **I32)
        batch = awq.KVBatch(rows, at, table)
        awq.kv_append(cache, batch, kv[:, :heads], kv[:, heads:])
        got = list(awq.kv_read(cache, batch, 800))
        for n in (1, 9, 140):  # streamed, streamed in tiles of 32 rows, tiles
            q = torch.randn(2 * n, heads, D, generator=torch.Generator(DEV).manual_seed(n), device=DEV).half()
            got.append(awq.attention_kv4(q, cache, awq.KVBatch(torch.tensor([0, n, 2 * n], **I32), at, table)))
        outs.append(got)
    for a, b in zip(*outs):
        assert torch.equal(a, b) and bool((a != 0).any())
    del cache
    torch.cuda.empty_cache()


def one_sequence(D, group, length, wide, seed=0, size=16):
    gen = torch.Generator(DEV).manual_seed(seed + D + group)
    table = torch.full((1, wide), -1, **I32)
    need = -(-length // size)
    table[0, :need] = torch.randperm(need, generator=gen, device=DEV).to(torch.int32)
    cache = awq.alloc_kv_cache(need, 2, D, DEV, page_size=size, group=group)
    whole = awq.KVBatch(torch.tensor([0, length], **I32), torch.tensor([length], **I32), table)
    kv = torch.randn(length, 4, D, generator=gen, device=DEV).half()
    awq.kv_append(cache, whole, kv[:, :2], kv[:, 2:])
    return gen, cache, whole


@pytest.mark.parametrize("D,group,share,n", [(128, 128, 4, 1), (128, 32, 1, 1), (64, 64, 20, 2), (256, 128, 2, 70),
                                             (128, 64, 8, 40)])
@pytest.mark.parametrize("length", [1, 77, 600])
def test_wide_page_tables(D, group, share, n, length):
    """A table for 131072 tokens and sequences of a few: work is planned for what the table can hold."""
    gen, cache, whole = one_sequence(D, group, length, 8192)
    n = min(n, length)
    q = torch.randn(n, 2 * share, D, generator=gen, device=DEV).half()
    lse = torch.empty(n, 2 * share, device=DEV)
    y = awq.attention_kv4(q, cache, awq.KVBatch(torch.tensor([0, n], **I32), whole.lengths, whole.page_table), lse=lse)
    want = kv_exact.attention(q.cpu().double(), kv_exact.tokens(awq, cache, whole, 0, length), D ** -0.5, True, 0,
                              D // group <= 2, n * share > 64)
    kv_exact.check(y, lse, want)


@pytest.mark.parametrize("D,group,share,n", [(128, 128, 1, 100), (128, 64, 2, 64), (64, 64, 3, 30), (128, 32, 2, 50)])
def test_as_many_rows_as_are_streamed(D, group, share, n):
    """65 to 128 rows of one sequence at few heads are streamed, with probabilities as hi + lo."""
    gen, cache, whole = one_sequence(D, group, 300, 19)
    q = torch.randn(n, 2 * share, D, generator=gen, device=DEV).half()
    lse = torch.empty(n, 2 * share, device=DEV)
    y = awq.attention_kv4(q, cache, awq.KVBatch(torch.tensor([0, n], **I32), whole.lengths, whole.page_table), lse=lse)
    want = kv_exact.attention(q.cpu().double(), kv_exact.tokens(awq, cache, whole, 0, 300), D ** -0.5, True, 0,
                              D // group <= 2, False)
    kv_exact.check(y, lse, want)
