"""The cache, the attention over it and the linears around them as a server runs them: step after
step, in captured graphs, on several streams; and contents that no correct caller passes."""

import math

import numpy as np
import pytest
import torch

import weight_only_bit_02_amd as awq

from . import kv_ref
from .gpu_util import DEV, guarded, host, to_dev
from .kv_util import NAMES, batch_of, filled, on_device, same, strided
from .test_gpu_graphs import _refill
from .test_gpu_kv_append import table_of

pytestmark = pytest.mark.gpu

HEADS, SHARE, D, HIDDEN = 2, 3, 64, 256
Q = HEADS * SHARE


def layer(seed):
    g = torch.Generator(DEV).manual_seed(seed)
    qkv = torch.randn((Q + 2 * HEADS) * D, HIDDEN, generator=g, device=DEV) / 16
    o = torch.randn(HIDDEN, Q * D, generator=g, device=DEV) / 20
    return awq.quantize_pack(qkv.half()), awq.quantize_pack(o.half())


def step(x, qkv, o, cache, batch, rope, workspace=None):
    """A decoder layer's attention: (q rotated, k, v, attention's output, the layer's)."""
    q, k, v = awq.linear_w4a16(x, qkv).view(len(x), -1, D).split([Q, HEADS, HEADS], dim=1)
    q = awq.kv_append(cache, batch, k, v, q, rope, out=q)
    y = awq.attention_kv4(q, cache, batch, workspace=workspace)
    return q, k, v, y, awq.linear_w4a16(y.view(len(x), -1), o)


def room(batch, T, q_heads=Q, heads=HEADS, dim=D, size=16):
    S, wide = batch.page_table.shape
    most = T if batch.max_rows is None else min(T, batch.max_rows)
    n = awq.attention_kv4_workspace_size(T, S, most, wide * size, q_heads, heads, dim)
    return torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)


def test_decoding():
    """Prompts of two sequences, then tokens one at a time, then two at a time: every step's cache and
    attention against the 64-bit form of what the linear put out."""
    rng = np.random.default_rng(20)
    qkv, o = layer(1)
    tab = table_of(128, D, rng)
    rope = awq.Rotary(to_dev(tab))
    table = np.array([[3, 0, 5, 7, 8, -1], [1, 6, 4, 2, -1, -1]], np.int32)
    c = kv_ref.Cache(9, HEADS, 16, D, D, rng)
    cache = on_device(awq, c)
    lengths = [0, 0]
    for n in [(40, 13), (1, 1), (1, 1), (1, 0), (2, 2), (7, 30)]:
        lengths = [a + b for a, b in zip(lengths, n)]
        rows = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        batch = awq.KVBatch(to_dev(rows), to_dev(np.array(lengths, np.int32)), to_dev(table), max(n))
        x = to_dev(rng.standard_normal((int(rows[-1]), HIDDEN)).astype(np.float16))
        plain = host(awq.linear_w4a16(x, qkv)).reshape(len(x), -1, D)
        q, k, v, y, out = step(x, qkv, o, cache, batch, rope)
        at = np.concatenate([np.arange(l - m, l) for l, m in zip(lengths, n)])
        kr = kv_ref.rotate(plain[:, Q:Q + HEADS], tab[at], False)
        assert np.array_equal(host(q).view(np.uint16), kv_ref.rotate(plain[:, :Q], tab[at], False).view(np.uint16))
        for s in range(2):
            for i in range(n[s]):
                p = lengths[s] - n[s] + i
                c.put(table[s, p // 16], p % 16, kr[rows[s] + i], plain[rows[s] + i, Q + HEADS:])
        assert same(cache, c) == []
        for s in range(2):
            if n[s]:
                r = slice(rows[s], rows[s + 1])
                want, _, bound, _ = kv_ref.attention(host(q)[r].astype(np.float64), kv_ref.tokens(c, table[s], lengths[s]),
                                                     1 / math.sqrt(D), True, 0, max(n) * SHARE > 64)
                assert np.all(np.abs(host(y)[r] - want) <= bound)
        assert torch.equal(out, awq.linear_w4a16(y.view(len(x), -1), o))


@pytest.mark.parametrize("T,max_rows", [(3, 1), (3, None), (60, None)])
def test_step_in_a_graph(T, max_rows):
    """One capture serves growing sequences: rows, lengths and pages change between replays."""
    rng = np.random.default_rng(21)
    qkv, o = layer(2)
    rope = awq.Rotary(to_dev(table_of(400, D, rng)), True)
    S, wide = 3, 20
    pages = S * wide
    cache = awq.alloc_kv_cache(pages, HEADS, D, DEV, page_size=16)
    for name in NAMES:
        getattr(cache, name).zero_()
    batch = awq.KVBatch(torch.zeros(S + 1, dtype=torch.int32, device=DEV), torch.zeros(S, dtype=torch.int32, device=DEV),
                        torch.zeros((S, wide), dtype=torch.int32, device=DEV), max_rows)
    x = torch.zeros(T, HIDDEN, dtype=torch.float16, device=DEV)
    ko = torch.empty(T, HEADS, D, dtype=torch.float16, device=DEV)
    vo, workspace = torch.empty_like(ko), room(batch, T)

    def update(i):
        _refill(x, 60 + i, 1.0)
        if max_rows == 1:
            n = np.ones(S, int)
        else:
            n = rng.multinomial(T, [0.2, 0.5, 0.3])
        lengths = n + rng.integers(0, 16 * wide - T, S)
        batch.rows.copy_(to_dev(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)))
        batch.lengths.copy_(to_dev(lengths.astype(np.int32)))
        batch.page_table.copy_(to_dev(rng.permutation(pages).reshape(S, wide).astype(np.int32)))

    def run():
        q, _, _, y, out = step(x, qkv, o, cache, batch, rope, workspace)
        awq.kv_read(cache, batch, out=(ko, vo))
        return q, y, out, ko, vo

    update(0)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs = run()
        for i in range(4):
            update(i)
            kept = [getattr(cache, name).clone() for name in NAMES]
            ref = [r.clone() for r in run()]
            after = [getattr(cache, name).clone() for name in NAMES]
            for name, t in zip(NAMES, kept):
                getattr(cache, name).copy_(t)
            torch.cuda.synchronize()
            for r in outs:
                r.view(torch.uint8).fill_(0xA5)
            workspace.fill_(0xA5)
            graph.replay()
            torch.cuda.synchronize()
            for r, want in zip(outs, ref):
                assert torch.equal(r.view(torch.uint8), want.view(torch.uint8)), i
            for name, want in zip(NAMES, after):
                assert torch.equal(getattr(cache, name), want), (i, name)
        del graph


def random_cache(pages, heads, dim, size, seed):
    """A cache with random contents (every 16-bit word of the parameters a scale in [2^-4, 1))."""
    g = torch.Generator(DEV).manual_seed(seed)
    c = awq.alloc_kv_cache(pages, heads, dim, DEV, page_size=size)
    for name in ("k_codes", "v_codes"):
        t = getattr(c, name)
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV).byte())
    for name in ("k_params", "v_params"):
        t = getattr(c, name)
        t.copy_((0x2C00 + torch.randint(0, 0x1000, t.shape, generator=g, device=DEV)).short())
    return c


def lists(seqs, n, length, size, seed, max_rows=None):
    """Sequences with n rows and about `length` tokens each, pages in any order."""
    rng = np.random.default_rng(seed)
    lengths = rng.integers(length // 2, length, seqs)
    b, pages, _, rows = batch_of(awq, [n] * seqs, [int(x) for x in lengths], size, rng, max_rows=max_rows)
    return b, pages, int(rows[-1])


def test_two_graphs_with_one_workspace():
    """Two captured calls of different shapes take turns with one workspace."""
    a, pages, Ta = lists(2, 1, 3000, 16, 22, 1)
    b, more, Tb = lists(1, 90, 700, 16, 23)
    cache = random_cache(max(pages, more), HEADS, D, 16, 24)
    ws = max((room(a, Ta), room(b, Tb)), key=len)
    calls = [(torch.zeros(Ta, Q, D, dtype=torch.float16, device=DEV), a), (torch.zeros(Tb, Q, D, dtype=torch.float16, device=DEV), b)]
    graphs, outs = [], []
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for q, batch in calls:
            awq.attention_kv4(q, cache, batch, workspace=ws)
            torch.cuda.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=stream):
                outs.append(awq.attention_kv4(q, cache, batch, workspace=ws))
        for i in range(4):
            for q, _ in calls:
                _refill(q, 70 + i, 1.0)
            ref = [awq.attention_kv4(q, cache, batch) for q, batch in calls]
            ws.fill_(0xFF)
            for o in outs:
                o.fill_(7)
            for k in (0, 1, 0) if i % 2 else (1, 0, 1):
                graphs[k].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(o, r) for o, r in zip(outs, ref))
        graphs.clear()


@pytest.mark.parametrize("n,max_rows", [(1, 1), (50, None)])
def test_calls_at_once(n, max_rows):
    """Appends to different pages and attention on three streams at the same time."""
    parts = []
    for i in range(3):
        b, pages, T = lists(4, n, 900, 16, 30 + i, max_rows)
        cache = random_cache(pages, HEADS, D, 16, 40 + i)
        x = torch.randn(T, Q + 2 * HEADS, D, generator=torch.Generator(DEV).manual_seed(i), device=DEV).half()
        parts.append((b, cache, x))
    rope = awq.Rotary(to_dev(table_of(1000, D, np.random.default_rng(25))))

    def run(b, cache, x):
        q, k, v = x.split([Q, HEADS, HEADS], dim=1)
        q = awq.kv_append(cache, b, k, v, q, rope)
        return awq.attention_kv4(q, cache, b)

    ref = [run(*p) for p in parts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [[] for _ in parts]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(run(*parts[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, r) for part, r in zip(outs, ref) for o in part)


@pytest.mark.parametrize("n,length,max_rows", [(1, 400, 1), (1, 9000, 1), (40, 400, None), (300, 2000, None)])
def test_strided_output(n, length, max_rows):
    """Rows of outputs and queries with room between them, which stays as it was; the output in the
    queries' place."""
    b, pages, T = lists(3, n, length, 32, 26, max_rows)
    cache = random_cache(pages, HEADS, 128, 32, 27)
    q = torch.randn(T, Q, 128, generator=torch.Generator(DEV).manual_seed(3), device=DEV).half()
    want = awq.attention_kv4(q, cache, b)
    buf = torch.full((T, Q * 128 + 24), 7.0, dtype=torch.float16, device=DEV)
    out = buf[:, 8:8 + Q * 128].unflatten(1, (Q, 128))
    assert awq.attention_kv4(strided(host(q), 16), cache, b, out=out) is out
    assert torch.equal(out, want)
    assert bool((buf[:, :8] == 7).all()) and bool((buf[:, 8 + Q * 128:] == 7).all())
    assert awq.attention_kv4(q, cache, b, out=q) is q  # in place
    assert torch.equal(q, want)


def test_shared_pages():
    """Two sequences with the same prefix, and one that holds a page twice."""
    rng = np.random.default_rng(28)
    table = np.array([[4, 2, 0, -1], [4, 2, 1, -1], [3, 4, 3, 4]], np.int32)
    lengths, n = [40, 45, 64], [1, 2, 1]
    rows = np.array([0, 1, 3, 4], np.int32)
    c = filled(5, HEADS, 16, D, D, np.arange(5, dtype=np.int32)[None], [80], rng)
    b = awq.KVBatch(to_dev(rows), to_dev(np.array(lengths, np.int32)), to_dev(table), 2)
    q = rng.standard_normal((4, Q, D)).astype(np.float16)
    y = host(awq.attention_kv4(to_dev(q), on_device(awq, c), b))
    for s in range(3):
        r = slice(rows[s], rows[s + 1])
        want, _, bound, _ = kv_ref.attention(q[r].astype(np.float64), kv_ref.tokens(c, table[s], lengths[s]),
                                             1 / math.sqrt(D), True, 0, False)
        assert np.all(np.abs(y[r] - want) <= bound)


@pytest.mark.parametrize("T,max_rows", [(12, 12), (200, None)])
def test_wrong_contents_stay_in_bounds(T, max_rows):
    """Rows that fall, overlap, are negative or pass the tensors, lengths and pages of any value: what
    comes out is not specified, nothing outside the tensors is touched."""
    rng = np.random.default_rng(29)
    pages, size, wide, S = 6, 16, 5, 5
    rope = awq.Rotary(to_dev(table_of(50, D, rng)))
    big = 2 ** 31 - 1
    rows_list = [[0, T, 0, T, 0, T], [0, -5, 3, big, -big, T], [5, 4, 3, 2, 1, 0], [big] * 6, [-big] * 6,
                 [0, 2 * T, 3 * T, 4, 4, T], [T, T, T, T, T, T]]
    for rows in rows_list:
        bufs, checks = [], []
        for shape, dtype in [((pages, HEADS, size, D // 2), torch.uint8), ((pages, HEADS, 1, size), torch.int16)] * 2:
            t, check = guarded(shape, dtype)
            t.zero_()
            bufs.append(t), checks.append(check)
        cache = awq.KVCache(*bufs, D)
        table = rng.choice([0, 1, 5, 6, -1, big, -big - 1], (S, wide)).astype(np.int32)
        lengths = rng.choice([0, 1, 70, 81, big, -3, -big], S).astype(np.int32)
        b = awq.KVBatch(to_dev(np.array(rows, np.int32)), to_dev(lengths), to_dev(table), max_rows)
        x = torch.randn(T, Q + 2 * HEADS, D, device=DEV).half()
        q, k, v = x.split([Q, HEADS, HEADS], dim=1)
        out, c0 = guarded((T, Q, D), torch.float16)
        y, c1 = guarded((T, Q, D), torch.float16)
        lse, c2 = guarded((T, Q), torch.float32)
        ko, c3 = guarded((T, HEADS, D), torch.float16)
        vo, c4 = guarded((T, HEADS, D), torch.float16)
        ws = room(b, T)
        wide_ws = torch.full((ws.numel() + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
        out.zero_()
        awq.kv_append(cache, b, k, v, q, rope, out=out)
        awq.attention_kv4(out, cache, b, out=y, lse=lse, workspace=wide_ws[:ws.numel()])
        awq.kv_read(cache, b, out=(ko, vo))
        torch.cuda.synchronize()
        for check in checks + [c0, c1, c2, c3, c4]:
            check()
        assert bool((wide_ws[ws.numel():] == 0x5A).all())


def test_many_sequences_and_heads():
    """The largest number of sequences, and of query heads."""
    S = 65536
    rng = np.random.default_rng(31)
    lengths = rng.integers(1, 4, S).astype(np.int32)
    cache = random_cache(S, 1, D, 16, 32)
    table = rng.permutation(S).astype(np.int32)[:, None]
    b = awq.KVBatch(torch.arange(S + 1, dtype=torch.int32, device=DEV), to_dev(lengths), to_dev(table), 1)
    q = torch.randn(S, 1, D, generator=torch.Generator(DEV).manual_seed(5), device=DEV).half()
    lse = torch.empty(S, 1, device=DEV)
    y = awq.attention_kv4(q, cache, b, lse=lse)
    whole = awq.KVBatch(torch.arange(0, 3 * S + 1, 3, dtype=torch.int32, device=DEV),
                        torch.full((S,), 3, dtype=torch.int32, device=DEV), b.page_table, 3)
    k, v = (t.view(S, 3, D).double() for t in awq.kv_read(cache, whole, 3 * S))
    s = (k * q.double()).sum(2) / math.sqrt(D)
    s = s.masked_fill(torch.arange(3, device=DEV)[None] >= b.lengths[:, None], -math.inf)
    want = (torch.softmax(s, 1)[:, :, None] * v).sum(1)
    # kv_ref.attention's bound; scales are below 1
    size = (k.abs() * q.double().abs()).sum(2).amax(1, keepdim=True) / math.sqrt(D)
    e = (D + 8) * 2.0 ** -24 * size + 2.0 ** -21 + 3 * 2.0 ** -24
    off = (2 * e + 2.0 ** -22) * (torch.softmax(s, 1)[:, :, None] * v.abs()).sum(1) + 3 * 2.0 ** -31 * 15
    assert bool(((y[:, 0].double() - want).abs() <= off + 2.0 ** -11 * (want.abs() + off) + 2.0 ** -25).all())
    wl = torch.logsumexp(s, 1, keepdim=True)
    assert bool(((lse.double() - wl).abs() <= e + 2.0 ** -22 * (wl.abs() + s.amax(1, keepdim=True).abs() + 1)).all())

    b, pages, table, rows = batch_of(awq, [1, 2], [40, 3], 16, rng)
    c = filled(pages, 1, 16, D, D, table, [40, 3], rng)
    q = rng.standard_normal((3, 1024, D)).astype(np.float16)
    y = host(awq.attention_kv4(to_dev(q), on_device(awq, c), b))
    for s in range(2):
        r = slice(rows[s], rows[s + 1])
        want, _, bound, _ = kv_ref.attention(q[r].astype(np.float64), kv_ref.tokens(c, table[s], [40, 3][s]),
                                             1 / math.sqrt(D), True, 0, True)
        assert np.all(np.abs(y[r] - want) <= bound)


@pytest.mark.parametrize("n", [1, 80])
def test_attention_beyond_4_gib(n):
    """Pages whose codes and parameters lie past 2^32 bytes give what pages at the start give."""
    heads, size, dim = 32, 256, 128
    pages = (1 << 32) // (heads * size * dim // 2) + 5
    cache = awq.alloc_kv_cache(pages, heads, dim, DEV, page_size=size)
    small = random_cache(4, heads, dim, size, 33)
    for name in NAMES:
        getattr(cache, name)[:4].copy_(getattr(small, name))
        getattr(cache, name)[pages - 4:].copy_(getattr(small, name))
    q = torch.randn(2 * n, heads, dim, generator=torch.Generator(DEV).manual_seed(6), device=DEV).half()
    outs = []
    for first in (0, pages - 4):
        b = awq.KVBatch(to_dev(np.array([0, n, 2 * n], np.int32)), to_dev(np.array([500, 300], np.int32)),
                        to_dev(np.array([[first, first + 1], [first + 3, first + 2]], np.int32)))
        outs.append(awq.attention_kv4(q, cache, b))
    assert torch.equal(*outs) and bool((outs[0] != 0).any())


def test_refusals_on_the_device():
    """Arguments that the binding passes on: the library's refusal, with nothing launched."""
    rng = np.random.default_rng(34)
    b, pages, _, _ = batch_of(awq, [1], [20], 16, rng)
    cache = random_cache(pages, HEADS, D, 16, 35)
    q = torch.zeros(1, Q, D, dtype=torch.float16, device=DEV)
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(window=-1)):
        with pytest.raises(awq.AwqError):
            awq.attention_kv4(q, cache, b, **bad)
    with pytest.raises(awq.AwqError):  # rows of 16 bytes
        awq.attention_kv4(torch.zeros(2 * Q * D + 8, dtype=torch.float16, device=DEV)[4:4 + Q * D].view(1, Q, D), cache, b)
    with pytest.raises(awq.AwqError):  # query heads by key heads
        awq.attention_kv4(torch.zeros(1, 3, D, dtype=torch.float16, device=DEV), cache, b)
    with pytest.raises(ValueError):
        awq.kv_append(cache, b, q[:, :HEADS], q[:, :HEADS], q)
    with pytest.raises(ValueError):
        awq.attention_kv4(q.transpose(1, 2), cache, b)
