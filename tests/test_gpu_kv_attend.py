"""Attention over the 4-bit cache against the plain 64-bit form, at the sizes and masks where it
can go wrong: one token to several chunks, ragged sequences, empty rows, holes in the page
table, windows, shared heads, every head size and group."""

import math

import numpy as np
import pytest
import torch

import weight_only_bit_02_amd as awq

from . import kv_ref
from .gpu_util import DEV, guarded, host, to_dev
from .kv_util import batch_of, filled, on_device, strided

pytestmark = pytest.mark.gpu


def attend(D, group, size, heads, share, n, lengths, causal=True, window=0, scale=None, seed=0, holes=(), wide=None,
           q_gain=1.0, k_gain=1.0, v_gain=1.0, max_rows=None, extra_rows=0):
    rng = np.random.default_rng(seed)
    b, pages, table, rows = batch_of(awq, n, lengths, size, rng, wide=wide, holes=holes, max_rows=max_rows)
    c = filled(pages, heads, size, D, group, table, lengths, rng, k_gain, v_gain)
    T = int(rows[-1]) + extra_rows
    q = (rng.standard_normal((T, heads * share, D)) * q_gain).astype(np.float16)
    out, check = guarded((T, heads * share, D), torch.float16)
    lse, lse_check = guarded((T, heads * share), torch.float32)
    out.fill_(9)
    lse.fill_(9)
    awq.attention_kv4(strided(q), on_device(awq, c), b, scale=scale, causal=causal, window=window, out=out, lse=lse)
    scale = 1 / math.sqrt(D) if scale is None else scale
    y, l = host(out).astype(np.float64), host(lse).astype(np.float64)
    check(), lse_check()
    for s in range(len(n)):
        if n[s] == 0:
            continue
        kv = kv_ref.tokens(c, table[s], lengths[s])
        r = slice(rows[s], rows[s + 1])
        # probabilities are rounded to fp16 where the rows are many
        want, want_lse, bound, lse_bound = kv_ref.attention(q[r].astype(np.float64), kv, scale, causal, window,
                                                            n[s] * share > 64)
        none = np.isinf(want_lse)
        assert np.array_equal(np.isneginf(l[r]), none), s
        assert np.all(y[r][none] == 0)
        off = np.abs(y[r] - want) - bound
        assert np.all(off <= 0), (s, off.max(), np.abs(want).max())
        assert np.all(np.abs(l[r] - want_lse)[~none] <= lse_bound[~none]), s
    assert np.all(y[rows[-1]:] == 9) and np.all(l[rows[-1]:] == 9)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("share,n,lengths", [
    (1, [1], [1]),
    (4, [1, 1, 1], [15, 16, 17]),
    (7, [1, 2, 1], [63, 130, 300]),
    (16, [1], [65]),
    (20, [1, 3], [64, 257]),
])
def test_few_rows(D, group, share, n, lengths):
    if group > D:
        pytest.skip("a group is within a head")
    attend(D, group, 16, 2, share, n, lengths, seed=D + group + share)


@pytest.mark.parametrize("size", [16, 32, 64, 256])
def test_page_sizes(size):
    attend(128, 128, size, 1, 4, [1, 2, 1, 1], [255, 513, size, size + 1], seed=size)


@pytest.mark.parametrize("n,lengths", [([40], [40]), ([100, 1, 17], [100, 90, 300]), ([1, 65, 0, 33], [5, 129, 7, 64])])
@pytest.mark.parametrize("D,share", [(128, 1), (128, 3), (64, 5), (256, 2)])
def test_many_rows(D, share, n, lengths):
    attend(D, 64, 32, 2, share, n, lengths, seed=D + share)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [1, 5, 64, 100, 10 ** 12])
def test_windows(causal, window):
    attend(128, 128, 16, 1, 2, [1, 9, 30, 1], [700, 300, 30, 3], causal=causal, window=window, seed=window % 1000)


def test_without_mask():
    attend(64, 64, 16, 2, 2, [5, 70], [90, 70], causal=False)


def test_empty_rows():
    """An empty sequence, rows before position 0, a sequence whose pages are gone, and one whose
    pages in the window are gone."""
    attend(128, 128, 16, 1, 4, [1, 3, 2, 1], [0, 1, 30, 90], window=16, holes=[(2, 0), (2, 1), (3, 4), (3, 5)])
    attend(128, 32, 16, 1, 4, [2], [0], wide=1)


def test_holes():
    attend(128, 128, 16, 2, 2, [1, 20, 1], [200, 100, 47], holes=[(0, 3), (0, 4), (1, 0), (2, 2)], seed=5)


def test_lengths_beyond_the_table():
    """A length that the table cannot hold counts for positions; the tokens are those it holds."""
    rng = np.random.default_rng(1)
    b, pages, table, rows = batch_of(awq, [2], [64], 16, rng)
    c = filled(pages, 1, 16, 128, 128, table, [64], rng)
    q = rng.standard_normal((2, 2, 128)).astype(np.float16)
    dev = on_device(awq, c)
    b.lengths.fill_(1000)
    y = awq.attention_kv4(to_dev(q), dev, b)
    want, _, bound, _ = kv_ref.attention(q.astype(np.float64), kv_ref.tokens(c, table[0], 64), 1 / math.sqrt(128), False,
                                         0, False)
    assert np.all(np.abs(host(y) - want) <= bound)


@pytest.mark.parametrize("D,group,share", [(64, 32, 8), (64, 64, 1), (128, 128, 8), (128, 32, 2), (256, 128, 4), (256, 32, 3)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50), (False, 130)])
def test_tiles(D, group, share, causal, window):
    """More rows than a wave's, a block's and a work list's piece; short sequences among them."""
    attend(D, group, 16, 1, share, [150, 1, 67, 9], [170, 600, 700, 9], causal=causal, window=window, seed=D + group)


def test_tiles_holes():
    attend(128, 64, 16, 1, 4, [40, 100], [200, 100], seed=6, holes=[(0, 0), (0, 5), (0, 12), (1, 0), (1, 1), (1, 2), (1, 6)])
    attend(64, 64, 32, 1, 2, [60], [290], seed=7, holes=[(0, p) for p in range(9)])
    attend(256, 64, 16, 1, 2, [60], [290], seed=8, holes=[(0, 1), (0, 17)])


@pytest.mark.parametrize("n,length", [(3, 700), (1, 1), (0, 0), (150, 200)])
def test_one_sequence_and_rows_behind_it(n, length):
    """A single sequence with fewer rows than the tensors: what they have says little."""
    attend(128, 64, 16, 1, 2, [n], [length], extra_rows=230, seed=10 + n)


def test_tiles_rows_before_the_sequence():
    attend(128, 128, 16, 1, 4, [90, 80, 70], [30, 0, 1], seed=9)


@pytest.mark.parametrize("D,heads,share,n,lengths,window", [
    (128, 8, 4, [700, 1300], [700, 2000], 0),      # pieces of items, joined
    (128, 32, 4, [700, 1300], [700, 2000], 0),     # whole items
    (128, 2, 1, [257, 1, 300], [5000, 4000, 301], 0),
    (64, 2, 8, [130, 256], [9000, 300], 1000),
    (256, 2, 2, [64, 500], [3001, 777], 0),
])
def test_prompts(D, heads, share, n, lengths, window):
    """Long ones, against 64-bit products on the GPU of the values that the cache holds."""
    rng = np.random.default_rng(12)
    b, pages, table, rows = batch_of(awq, n, lengths, 64, rng)
    dev = awq.alloc_kv_cache(pages, heads, D, DEV)
    T = int(rows[-1])
    whole = awq.KVBatch(to_dev(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)), b.lengths, b.page_table)
    gen = torch.Generator(DEV).manual_seed(1)
    kv = torch.randn(sum(lengths), 2 * heads, D, generator=gen, device=DEV).half()
    awq.kv_append(dev, whole, kv[:, :heads], kv[:, heads:])
    q = torch.randn(T, heads * share, D, generator=gen, device=DEV).half()
    lse = torch.empty(T, heads * share, device=DEV)
    y = awq.attention_kv4(q, dev, b, window=window, lse=lse)
    assert torch.equal(y, awq.attention_kv4(q, dev, b, window=window))
    k, v = (x.double() for x in awq.kv_read(dev, whole, sum(lengths)))
    ends = np.cumsum(lengths)
    for s in range(len(n)):
        r = slice(int(ends[s]) - lengths[s], int(ends[s]))
        p = torch.arange(lengths[s] - n[s], lengths[s], device=DEV)[:, None]
        t = torch.arange(lengths[s], device=DEV)
        see = (t <= p) & (t > p - (window or 1 << 30))
        for h in range(heads * share):
            kk, vv = k[r, h // share].contiguous(), v[r, h // share].contiguous()
            x = q[rows[s]:rows[s + 1], h].double()
            sc = (x @ kk.t().contiguous() / math.sqrt(D)).masked_fill(~see, -math.inf)
            size = (x.abs() @ kk.t().contiguous().abs() / math.sqrt(D)).amax(1, keepdim=True)
            want_lse = torch.logsumexp(sc, 1)
            w = torch.exp(sc - want_lse[:, None])
            want, spread = w @ vv, w @ vv.abs()
            # the bound of kv_ref.attention; 15 scale of a few thousand normal values is below 12
            e = (D + 8) * 2.0 ** -24 * size + 2.0 ** -21 + see.sum(1, keepdim=True) * 2.0 ** -24
            top = torch.exp(sc.amax(1) - want_lse)[:, None]
            least = (2.0 ** -24 * vv.abs().sum(0) + lengths[s] * 2.0 ** -31 * 12) * top
            off = (2 * e + 2.0 ** -11) * spread + least
            bound = off + 2.0 ** -11 * (want.abs() + off) + 2.0 ** -25
            got = y[rows[s]:rows[s + 1], h].double()
            assert bool(((got - want).abs() <= bound).all()), (s, h)
            got = lse[rows[s]:rows[s + 1], h].double()
            assert bool(((got - want_lse).abs() <= e[:, 0] + 2.0 ** -22 * (want_lse.abs() + sc.amax(1).abs() + 1)).all()), (s, h)


@pytest.mark.parametrize("D,group,n", [(128, 128, 1), (128, 64, 5), (64, 64, 1), (256, 128, 2), (128, 32, 1), (128, 128, 80)])
def test_values_of_many_magnitudes(D, group, n):
    """Values whose scales rise by 2^14 along the sequence, fall by as much, and differ by group: the
    smallest count where the large ones have no probability."""
    rng = np.random.default_rng(13)
    length = 600
    b, pages, table, rows = batch_of(awq, [n, n], [length, length], 16, rng)
    c = kv_ref.Cache(pages, 1, 16, D, group, rng)
    q = rng.standard_normal((2 * n, 2, D)).astype(np.float16)
    for s in range(2):
        for t in range(length):
            up = t if s == 0 else length - 1 - t
            k = rng.standard_normal((1, D)) * 0.5 - 0.6 * q[s * n, :1] * (up / length)  # large values: unlikely
            gain = 2.0 ** (14 * up / length - 7) * (1 + 15 * (np.arange(D) < group))
            c.put(table[s, t // 16], t % 16, k.astype(np.float16), (rng.standard_normal((1, D)) * gain).astype(np.float16))
    y = host(awq.attention_kv4(to_dev(q), on_device(awq, c), b))
    for s in range(2):
        r = slice(rows[s], rows[s + 1])
        want, _, bound, _ = kv_ref.attention(q[r].astype(np.float64), kv_ref.tokens(c, table[s], length), 1 / math.sqrt(D),
                                             True, 0, 2 * n > 64)
        assert np.all(np.abs(y[r] - want) <= bound)


@pytest.mark.parametrize("q_gain,k_gain,v_gain", [(30, 8, 1), (0, 1, 1), (1e-4, 1, 100), (1, 1, 2000), (1, 1, 1e-3)])
def test_ranges(q_gain, k_gain, v_gain):
    """One token that takes all, equal probabilities, large and small values."""
    attend(128, 128, 16, 1, 3, [1, 6], [400, 70], q_gain=q_gain, k_gain=k_gain, v_gain=v_gain)


def test_scores_that_rise_and_fall():
    """Running maxima: keys that grow along the sequence, and that shrink."""
    rng = np.random.default_rng(2)
    D, length = 128, 900
    b, pages, table, rows = batch_of(awq, [1, 1], [length, length], 16, rng)
    c = kv_ref.Cache(pages, 1, 16, D, 128, rng)
    q = np.abs(rng.standard_normal((2, 4, D))).astype(np.float16)
    for s in range(2):
        for t in range(length):
            gain = (t if s == 0 else length - t) / 60
            c.put(table[s, t // 16], t % 16, (np.abs(rng.standard_normal((1, D))) * gain).astype(np.float16),
                  rng.standard_normal((1, D)).astype(np.float16))
    lse = torch.empty(2, 4, device=DEV)
    y = host(awq.attention_kv4(to_dev(q), on_device(awq, c), b, lse=lse))
    for s in range(2):
        kv = kv_ref.tokens(c, table[s], length)
        want, wl, bound, lb = kv_ref.attention(q[s:s + 1].astype(np.float64), kv, 1 / math.sqrt(D), True, 0, False)
        assert np.all(np.abs(y[s:s + 1] - want) <= bound)
        assert np.all(np.abs(host(lse)[s:s + 1] - wl) <= lb)


@pytest.mark.parametrize("D,group,n", [(128, 128, 1), (64, 64, 1), (128, 64, 9), (256, 128, 1), (128, 32, 1), (128, 128, 70)])
def test_small_outputs_of_long_sequences(D, group, n):
    """40000 tokens of nearly equal probabilities, values around zero: the output is a hundredth of
    them, and its error against the 64-bit form is that of its rounding."""
    length = 40000
    b, pages, _, _ = batch_of(awq, [n], [length], 64, np.random.default_rng(14))
    dev = awq.alloc_kv_cache(pages, 1, D, DEV, group=group)
    kv = torch.randn(length, 2, D, generator=torch.Generator(DEV).manual_seed(7), device=DEV).half()
    whole = awq.KVBatch(torch.tensor([0, length], dtype=torch.int32, device=DEV), b.lengths, b.page_table)
    awq.kv_append(dev, whole, kv[:, :1], kv[:, 1:])
    q = (torch.randn(n, 1, D, generator=torch.Generator(DEV).manual_seed(8), device=DEV) / 4).half()
    y = awq.attention_kv4(q, dev, b)[:, 0].double()
    k, v = (t[:, 0].double() for t in awq.kv_read(dev, whole, length))
    s = q[:, 0].double() @ k.t().contiguous() / math.sqrt(D)
    t = torch.arange(length, device=DEV)[None]
    s = s.masked_fill(t > length - n + torch.arange(n, device=DEV)[:, None], -math.inf)
    want = torch.softmax(s, 1) @ v
    # fp16 outputs are off by 2^-11 of themselves at most, 2^-12.6 on the mean square; probabilities
    # rounded to fp16 (many rows) add 2^-12.6 of a random sum as large as the output
    assert ((y - want).norm() / want.norm()).item() < (2.0 ** -11 if n > 64 else 2.0 ** -12)


def test_nonfinite_query_keeps_to_its_row():
    rng = np.random.default_rng(3)
    b, pages, table, _ = batch_of(awq, [2, 1], [300, 40], 16, rng)
    c = on_device(awq, filled(pages, 2, 16, 128, 128, table, [300, 40], rng))
    q = rng.standard_normal((3, 8, 128)).astype(np.float16)
    good = host(awq.attention_kv4(to_dev(q), c, b))
    for bad in (np.nan, np.inf):
        x = q.copy()
        x[1, 5, 7] = bad
        y = host(awq.attention_kv4(to_dev(x), c, b))
        same = np.ones((3, 8), bool)
        same[1, 5] = False
        assert np.array_equal(y[same].view(np.uint16), good[same].view(np.uint16))
        assert np.isnan(y[1, 5]).any()


@pytest.mark.parametrize("S", [1, 70, 700])
def test_many_sequences_same_bits(S):
    """A sequence's output does not depend on the batch that it is in beyond rounding, and the same
    call gives the same bits; work lists of several steps."""
    rng = np.random.default_rng(4)
    lengths = [int(x) for x in rng.integers(1, 700, S)]
    n = [int(x) for x in rng.integers(0, 2, S)]
    n[-1] = 1
    b, pages, table, rows = batch_of(awq, n, lengths, 64, rng)
    dev = awq.alloc_kv_cache(pages, 2, 128, DEV)
    T = int(rows[-1])
    whole = awq.KVBatch(to_dev(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)), b.lengths, b.page_table)
    kv = torch.randn(sum(lengths), 4, 128, generator=torch.Generator(DEV).manual_seed(1), device=DEV).half()
    awq.kv_append(dev, whole, kv[:, :2], kv[:, 2:])
    q = torch.randn(T, 8, 128, generator=torch.Generator(DEV).manual_seed(2), device=DEV).half()
    y = awq.attention_kv4(q, dev, b, out=torch.zeros(T, 8, 128, dtype=torch.float16, device=DEV))
    assert torch.equal(y, awq.attention_kv4(q, dev, b))
    k, v = (x.double() for x in awq.kv_read(dev, whole, sum(lengths)))
    ends = np.cumsum(lengths)
    for s in range(S):
        if n[s] == 0:
            continue
        r = slice(ends[s] - lengths[s], ends[s])
        x = q[rows[s]].double().view(2, 4, 128)
        w = torch.softmax(torch.einsum("hgd,thd->hgt", x.cpu(), k[r].cpu()) / math.sqrt(128), 2)
        want = torch.einsum("hgt,thd->hgd", w, v[r].cpu()).reshape(8, 128)
        # kv_ref.attention's bound; 15 scale of a few thousand normal values is below 12
        size = torch.einsum("hgd,thd->hgt", x.cpu().abs(), k[r].cpu().abs()).max().item() / math.sqrt(128)
        e = 136 * 2.0 ** -24 * size + 2.0 ** -21 + lengths[s] * 2.0 ** -24
        spread = torch.einsum("hgt,thd->hgd", w, v[r].cpu().abs()).reshape(8, 128)
        off = (2 * e + 2.0 ** -22) * spread + lengths[s] * 2.0 ** -31 * 12
        bound = off + 2.0 ** -11 * (want.abs() + off) + 2.0 ** -25
        assert bool(((y[rows[s]].double().cpu() - want).abs() <= bound).all()), s


def test_row_bound_too_small_stays_in_bounds():
    """A max_rows that some sequence passes is the caller's mistake; nothing is written out of range."""
    rng = np.random.default_rng(11)
    b, pages, table, rows = batch_of(awq, [9, 40], [70, 40], 16, rng, max_rows=2)
    c = on_device(awq, filled(pages, 1, 16, 128, 128, table, [70, 40], rng))
    out, check = guarded((49, 2, 128), torch.float16)
    awq.attention_kv4(torch.zeros(49, 2, 128, dtype=torch.float16, device=DEV), c, b, out=out)
    check()
