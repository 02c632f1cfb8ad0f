"""The key / value cache's entry points reject bad arguments on the host before anything is
enqueued (no GPU needed: every call here fails validation), and so does their binding."""

import ctypes as C

import pytest
import torch

import weight_only_bit_02_amd as awq
from weight_only_bit_02_amd import _abi

A = 0x7F0000000000  # 16-byte aligned, never dereferenced
NULL, SHAPE, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


def cache(k=A, kp=A, v=A, vp=A, pages=10, size=16, heads=2, dim=128, group=128):
    return _abi.KvCache(k, kp, v, vp, pages, size, heads, dim, group)


def batch(rows=A, lengths=A, table=A, n=5, seqs=2, wide=4, most=5):
    return _abi.KvBatch(rows, lengths, table, n, seqs, wide, most)


def calls(lib):
    """The three entry points as functions of a cache and a batch, all else right."""
    return {
        "append": lambda c, b: lib.awq_kv_append(c, b, A, 256, A, 256, A, 512, 4, A, 512, A, 100, 128, 0, None, None),
        "read": lambda c, b: lib.awq_kv_read(c, b, A, A, None),
        "attend": lambda c, b: lib.awq_attention_kv4(A, 512, 4, c, b, 0.1, 1, 0, A, 512, None, None, 0, None),
    }



@pytest.mark.parametrize("name", ["append", "read", "attend"])
def test_cache_and_batch(lib, name):
    f = calls(lib)[name]
    assert f(None, batch()) == NULL and f(cache(), None) == NULL
    for k in ("k", "kp", "v", "vp"):
        assert f(cache(**{k: None}), batch()) == NULL
        assert f(cache(**{k: A + 8}), batch()) == MISALIGNED
    for k in ("rows", "lengths", "table"):
        assert f(cache(), batch(**{k: None})) == NULL
        assert f(cache(), batch(**{k: A + 4})) == MISALIGNED
    for dim in (0, -64, 32, 80, 96, 192, 512):
        assert f(cache(dim=dim), batch()) == UNSUPPORTED
    for group in (0, -32, 16, 48, 256):
        assert f(cache(group=group), batch()) == UNSUPPORTED
    assert f(cache(dim=64), batch()) == UNSUPPORTED  # groups of 128 in heads of 64
    for size in (0, 1, 8, 15, 17, 48, 8192, -16):
        assert f(cache(size=size), batch()) == UNSUPPORTED
    for pages in (0, -1, 1 << 31):
        assert f(cache(pages=pages), batch()) == SHAPE
    for heads in (0, -1, 1025):
        assert f(cache(heads=heads), batch()) == SHAPE
    for n in (0, -1, 1 << 22):
        assert f(cache(), batch(n=n)) == SHAPE
    for seqs in (0, -1, 65537):
        assert f(cache(), batch(seqs=seqs)) == SHAPE
    for wide in (0, -1, (1 << 30) // 16):
        assert f(cache(), batch(wide=wide)) == SHAPE
    for most in (0, -1, 6):
        assert f(cache(), batch(most=most)) == SHAPE


def test_append(lib):
    def call(k=A, k_ld=256, v=A, v_ld=256, q=A, q_ld=512, qh=4, out=A, out_ld=512, tab=A, positions=100, R=128, inter=0,
             flags=None, c=cache(), b=batch()):
        return lib.awq_kv_append(c, b, k, k_ld, v, v_ld, q, q_ld, qh, out, out_ld, tab, positions, R, inter, flags, None)
    assert call(k=None) == NULL and call(v=None) == NULL
    assert call(q=None) == NULL and call(out=None) == NULL  # one of the two
    assert call(tab=None) == NULL
    assert call(inter=2) == UNSUPPORTED and call(inter=-1) == UNSUPPORTED
    for ld in ("k_ld", "v_ld"):
        for x in (0, -256, 255, 252, 260, 1 << 31):
            assert call(**{ld: x}) == SHAPE
    for ld in ("q_ld", "out_ld"):
        for x in (0, 256, 511, 516, 1 << 31):
            assert call(**{ld: x}) == SHAPE
    assert call(qh=0) == SHAPE and call(qh=-1) == SHAPE and call(qh=1025, q_ld=1 << 20, out_ld=1 << 20) == SHAPE
    for R in (0, 8, 24, 130, 144, 256, -16):
        assert call(R=R) == SHAPE
    assert call(positions=0) == SHAPE and call(positions=1 << 31) == SHAPE
    for p in ("k", "v", "q", "out", "tab"):
        assert call(**{p: A + 8}) == MISALIGNED
    assert call(flags=A + 2) == MISALIGNED
    # fewer than 2^32 threads: 2^21 rows of 4 + 2 x 2 heads of 128 are 2^21 x 2 waves; 2^22 - 1 of 1024 + 4 are too many
    assert call(qh=1024, q_ld=1 << 17, out_ld=1 << 17, b=batch(n=(1 << 22) - 1, most=1)) == SHAPE


def test_read(lib):
    assert lib.awq_kv_read(cache(), batch(), None, A, None) == NULL
    assert lib.awq_kv_read(cache(), batch(), A, None, None) == NULL
    assert lib.awq_kv_read(cache(), batch(), A + 8, A, None) == MISALIGNED
    assert lib.awq_kv_read(cache(), batch(), A, A + 2, None) == MISALIGNED
    assert lib.awq_kv_read(cache(heads=1024), batch(n=(1 << 22) - 1, most=1), A, A, None) == SHAPE


def test_attend(lib):
    def call(q=A, q_ld=512, qh=4, scale=0.1, causal=1, window=0, out=A, out_ld=512, lse=None, ws=A, wsb=1 << 30, c=cache(),
             b=batch()):
        return lib.awq_attention_kv4(q, q_ld, qh, c, b, scale, causal, window, out, out_ld, lse, ws, wsb, None)
    assert call(q=None) == NULL and call(out=None) == NULL
    assert call(causal=2) == UNSUPPORTED
    for scale in (0.0, -1.0, float("nan"), float("inf"), 1e20):
        assert call(scale=scale) == UNSUPPORTED
    assert call(window=-1) == SHAPE
    for qh in (0, -2, 1, 3, 1026):
        assert call(qh=qh, q_ld=1 << 18, out_ld=1 << 18) == SHAPE
    for ld in ("q_ld", "out_ld"):
        for x in (0, 256, 511, 516, 1 << 31):
            assert call(**{ld: x}) == SHAPE
    assert call(q=A + 8) == MISALIGNED and call(out=A + 8) == MISALIGNED and call(lse=A + 2) == MISALIGNED
    assert call(b=batch(n=1 << 21, most=1), qh=8, q_ld=1024, out_ld=1024) == SHAPE  # n_rows q_heads reaches 2^24
    need = lib.awq_attention_kv4_workspace_size(5, 2, 5, 100 * 16, 4, 2, 128)
    assert need > 0
    b = batch(wide=100)
    assert call(b=b, ws=None, wsb=0) == WORKSPACE and call(b=b, wsb=need - 1) == WORKSPACE
    assert call(b=b, ws=A + 8, wsb=need) == WORKSPACE


def test_workspace_sizes(lib):
    f = lib.awq_attention_kv4_workspace_size
    assert f(1, 1, 1, 16, 1, 1, 64) == 0  # nothing to split
    assert f(64, 64, 1, 100000, 64, 8, 128) > 0
    for bad in ((0, 1, 1, 999, 4, 2, 128), (5, 0, 1, 999, 4, 2, 128), (5, 1, 0, 999, 4, 2, 128), (5, 1, 6, 999, 4, 2, 128),
                (5, 1, 1, 0, 4, 2, 128), (5, 1, 1, 1 << 30, 4, 2, 128), (5, 1, 1, 999, 3, 2, 128), (5, 1, 1, 999, 0, 2, 128),
                (5, 1, 1, 999, 4, 0, 128), (5, 1, 1, 999, 4, 2, 96), (1 << 22, 1, 1, 999, 4, 2, 128),
                (5, 65537, 1, 999, 4, 2, 128), (1 << 20, 65536, 1, (1 << 30) - 1, 8, 8, 128)):
        assert f(*bad) == 0, bad


def test_binding_refuses_host_tensors_and_shapes():
    c = awq.alloc_kv_cache(4, 2, 128, "cpu", page_size=16, group=64)
    assert c.k_codes.shape == (4, 2, 16, 64) and c.v_params.shape == (4, 2, 2, 16) and c.group == 64
    assert awq.alloc_kv_cache(4, 2, 64, "cpu").group == 64
    assert c.nbytes() == 4 * 2 * 16 * (128 + 4 * 2)
    i32 = torch.zeros(2, dtype=torch.int32)
    b = awq.KVBatch(i32, i32[:1], torch.zeros(1, 1, dtype=torch.int32))
    x = torch.zeros(1, 2, 128, dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        awq.kv_append(c, b, x, x)
    with pytest.raises(ValueError, match="GPU"):
        awq.attention_kv4(x, c, b)
    with pytest.raises(ValueError, match="GPU"):
        awq.kv_read(c, b, 1)
    with pytest.raises(TypeError):
        awq.kv_append(c, b, None, x)
    with pytest.raises(TypeError):
        awq.attention_kv4(None, c, b)
