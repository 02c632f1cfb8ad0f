"""The expert and adapter entry points reject bad arguments on the host before anything is
enqueued (no GPU needed: every call here fails validation), and so does their binding."""

import ctypes as C

import pytest
import torch

import weight_only_bit_02_amd as awq
from weight_only_bit_02_amd import _abi

FAKE = C.c_void_p(0x7F0000000000)      # 16-byte aligned, never dereferenced
FAKE_ODD = C.c_void_p(0x7F0000000008)  # misaligned
FAKE_2 = C.c_void_p(0x7F0000000002)
NULL, SHAPE, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


def test_group_rows(lib):
    def call(ids=FAKE, n=100, groups=4, offsets=FAKE, order=FAKE, pos=FAKE, ws=None, wsb=0):
        return lib.awq_group_rows(ids, n, groups, offsets, order, pos, ws, wsb, None)
    assert call(ids=None) == NULL and call(offsets=None) == NULL and call(order=None) == NULL
    assert call(n=0) == SHAPE and call(n=-1) == SHAPE and call(n=1 << 30) == SHAPE
    assert call(groups=0) == SHAPE and call(groups=513) == SHAPE and call(groups=-1) == SHAPE
    for k in ("ids", "offsets", "order", "pos"):
        assert call(**{k: FAKE_ODD}) == MISALIGNED
    need = lib.awq_group_rows_workspace_size(8193, 4)
    assert need > 0 and lib.awq_group_rows_workspace_size(8192, 4) == 0
    assert lib.awq_group_rows_workspace_size(0, 4) == 0 and lib.awq_group_rows_workspace_size(9000, 513) == 0
    assert call(n=8193) == WORKSPACE and call(n=8193, ws=FAKE, wsb=need - 1) == WORKSPACE
    assert call(n=8193, ws=FAKE_ODD, wsb=need) == WORKSPACE


def test_moe_route(lib):
    def call(x=FAKE, type=0, T=8, E=16, ld=16, k=2, renorm=1, w=FAKE, ids=FAKE, offsets=FAKE, order=FAKE, pos=FAKE,
             ws=None, wsb=0, flags=None):
        return lib.awq_moe_route(x, type, T, E, ld, k, renorm, w, ids, offsets, order, pos, ws, wsb, flags, None)
    for k in ("x", "w", "ids", "offsets", "order", "pos"):
        assert call(**{k: None}) == NULL
    assert call(type=2) == UNSUPPORTED and call(type=-1) == UNSUPPORTED and call(renorm=2) == UNSUPPORTED
    assert call(T=0) == SHAPE and call(E=0) == SHAPE and call(E=513, ld=513) == SHAPE and call(ld=15) == SHAPE
    assert call(k=0) == SHAPE and call(k=17) == SHAPE and call(E=128, ld=128, k=65) == SHAPE
    assert call(T=1 << 29, k=2) == SHAPE
    for k in ("w", "ids", "offsets", "order", "pos"):
        assert call(**{k: FAKE_ODD}) == MISALIGNED
    assert call(x=FAKE_2, type=1) == MISALIGNED and call(flags=FAKE_2) == MISALIGNED
    assert lib.awq_moe_route_workspace_size(64, 16) == 0
    need = lib.awq_moe_route_workspace_size(65, 16)
    assert need > 0 and call(T=65) == WORKSPACE and call(T=65, ws=FAKE, wsb=need - 1) == WORKSPACE


@pytest.mark.parametrize("gated", [False, True])
def test_grouped_linear(lib, gated):
    f = lib.awq_linear_w4a16_grouped_gated_silu if gated else lib.awq_linear_w4a16_grouped

    def call(X=FAKE, x_rows=10, offsets=FAKE, order=None, n=10, fan=1, groups=4, q=FAKE, sc=FAKE, z=FAKE, N=64, K=256,
             cfg=None, Y=FAKE, flags=None, kernel=0):
        return f(X, x_rows, offsets, order, n, fan, groups, q, sc, z, N, K, cfg, Y, flags, kernel, None)
    for k in ("X", "offsets", "q", "sc", "z", "Y"):
        assert call(**{k: None}) == NULL
        assert call(**{k: FAKE_ODD}) == MISALIGNED
    assert call(order=FAKE_ODD) == MISALIGNED and call(flags=FAKE_2) == MISALIGNED
    assert call(n=0) == SHAPE and call(n=1 << 30, x_rows=1 << 29) == SHAPE and call(x_rows=0) == SHAPE
    assert call(x_rows=9) == SHAPE                               # fewer rows than positions
    assert call(order=FAKE, x_rows=4, fan=2) == SHAPE            # 4 tokens x 2 < 10 positions
    assert call(order=FAKE, fan=0) == SHAPE and call(order=FAKE, fan=-2) == SHAPE
    assert call(groups=0) == SHAPE and call(groups=513) == SHAPE
    assert call(N=0) == SHAPE and call(K=100) == SHAPE and call(K=0) == SHAPE
    assert call(x_rows=1 << 28, K=256) == SHAPE                  # X of 2^36 values
    assert call(N=(1 << 31) - 2, n=1 << 20, x_rows=1 << 20) == SHAPE  # more tiles than a grid holds
    assert call(kernel=6) == UNSUPPORTED and call(kernel=-1) == UNSUPPORTED
    assert call(kernel=1, n=65537, x_rows=65537) == SHAPE
    if gated:
        assert call(N=63) == SHAPE
    for bad in (dict(w_bit=5), dict(group_size=16), dict(zero_point=2)):
        assert call(cfg=C.byref(_abi.config(**bad))) == UNSUPPORTED


def test_combine(lib):
    def call(P=FAKE, w=FAKE, pos=FAKE, offsets=FAKE, groups=4, T=8, k=2, N=64, add=None, Y=FAKE):
        return lib.awq_moe_combine(P, w, pos, offsets, groups, T, k, N, add, Y, None)
    for k in ("P", "w", "pos", "offsets", "Y"):
        assert call(**{k: None}) == NULL
        assert call(**{k: FAKE_ODD}) == MISALIGNED
    assert call(add=FAKE_ODD) == MISALIGNED
    assert call(groups=0) == SHAPE and call(groups=513) == SHAPE
    assert call(T=0) == SHAPE and call(k=0) == SHAPE and call(k=65) == SHAPE and call(T=1 << 29, k=2) == SHAPE
    assert call(N=0) == SHAPE and call(N=1 << 31) == SHAPE and call(T=1 << 20, N=1 << 18) == SHAPE


def test_lora(lib):
    def call(X=FAKE, M=4, q=FAKE, sc=FAKE, z=FAKE, N=64, K=256, cfg=None, A=FAKE, B=FAKE, s=FAKE, L=3, r=16, ids=FAKE,
             order=None, Y=FAKE, ws=FAKE, wsb=1 << 20, flags=None, kernel=0):
        return lib.awq_linear_w4a16_lora(X, M, q, sc, z, N, K, cfg, A, B, s, L, r, ids, order, Y, ws, wsb, flags, kernel,
                                         None)
    for k in ("X", "q", "sc", "z", "A", "B", "s", "ids", "Y"):
        assert call(**{k: None}) == NULL
        assert call(**{k: FAKE_ODD}) == MISALIGNED
    assert call(order=FAKE_ODD) == MISALIGNED and call(flags=FAKE_2) == MISALIGNED
    assert call(M=0) == SHAPE and call(M=1 << 30) == SHAPE and call(N=0) == SHAPE and call(K=130) == SHAPE
    assert call(L=0) == SHAPE and call(L=513) == SHAPE
    for r in (0, 4, 12, 264, -8):
        assert call(r=r) == SHAPE
        assert lib.awq_linear_w4a16_lora_workspace_size(4, r) == 0
    need = lib.awq_linear_w4a16_lora_workspace_size(4, 16)
    assert need >= 4 * 16 * 4 and lib.awq_linear_w4a16_lora_workspace_size(0, 16) == 0
    assert call(ws=None) == WORKSPACE and call(wsb=need - 1) == WORKSPACE and call(ws=FAKE_ODD) == WORKSPACE
    assert call(kernel=6) == UNSUPPORTED and call(M=65, kernel=1) == SHAPE
    assert call(cfg=C.byref(_abi.config(w_bit=2))) == UNSUPPORTED


def test_limits_of_grids_and_offsets(lib):
    def linear(n, N, K, kernel):
        return lib.awq_linear_w4a16_grouped(FAKE, n, FAKE, None, n, 1, 4, FAKE, FAKE, FAKE, N, K, None, FAKE, None, kernel,
                                            None)
    assert linear(1 << 22, 1 << 20, 128, 0) == SHAPE              # 2^29 tiles
    assert linear(1 << 20, 1 << 16, 128, 5) == SHAPE              # 2^26 of the narrowest ones

    def lora(M, N, K, rank):
        return lib.awq_linear_w4a16_lora(FAKE, M, FAKE, FAKE, FAKE, N, K, None, FAKE, FAKE, FAKE, 2, rank, FAKE, None, FAKE,
                                         FAKE, 1 << 40, None, 0, None)
    assert lora(1, 8, 1 << 26, 64) == SHAPE                       # one adapter's A of 2^32 values
    assert lora(1 << 23, 1 << 20, 128, 8) == SHAPE

    def combine(T, N):
        return lib.awq_moe_combine(FAKE, FAKE, FAKE, FAKE, 4, T, 2, N, None, FAKE, None)
    assert combine(1 << 20, (1 << 12) + 1) == SHAPE and combine(1 << 20, 1 << 15) == SHAPE


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 8, dtype=torch.float16)
    ids = torch.zeros(4, dtype=torch.int32)
    groups = awq.RowGroups(torch.zeros(3, dtype=torch.int32), ids, ids)
    w = awq.PackedExperts(ids, x, ids, 2, 8, 128)
    for call in (lambda: awq.moe_route(x, 2), lambda: awq.group_rows(ids, 2),
                 lambda: awq.linear_w4a16_grouped(x, w, groups), lambda: awq.moe_combine(x, x.float(), groups),
                 lambda: awq.linear_w4a16_lora(x, w, awq.LoraAdapters(x, x, x), ids)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        awq.moe_route([[1.0]], 1)
    with pytest.raises(ValueError):
        awq.linear_w4a16_grouped_gated_silu(x, awq.PackedExperts(ids, x, ids, 2, 7, 128), groups)
