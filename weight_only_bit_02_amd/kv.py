"""Key / value cache in 4 bits and the attention over it: binding of that part of the C ABI
(argument marshalling only).

    cache = alloc_kv_cache(pages, kv_heads, head_dim, device)      # one per layer
    batch = KVBatch(rows, lengths, page_table, max_rows)           # one per step, for all layers
    q, k, v = linear_w4a16(x, qkv).view(T, -1, head_dim).split([q_heads, kv_heads, kv_heads], dim=1)
    q = kv_append(cache, batch, k, v, q, Rotary(cos_sin))          # rotated; k and v are in the cache
    y = attention_kv4(q, cache, batch)                             # [T][q_heads][head_dim]

Every function checks that its tensors live on one GPU and have the expected dtype, shape and
strides, launches on that GPU's current stream, allocates the outputs and workspaces it is not
given, and raises AwqError on a non-OK status. The contents of rows, lengths and page_table
stay on the device and are not looked at here.
"""

from __future__ import annotations

import math
from dataclasses import dataclass

import torch

from . import _abi
from .awq import GROUP
from .grouped import _check, _first, _flags, _launch, _workspace, _workspace_size


@dataclass
class KVCache:
    """Keys and values of one layer, 4-bit codes in pages (see awq.h for the layout)."""
    k_codes: torch.Tensor   # uint8 [pages][kv_heads][page_size][head_dim / 2]
    k_params: torch.Tensor  # int16 [pages][kv_heads][head_dim / group][page_size]: scale and zero
    v_codes: torch.Tensor   # as k_codes, in the values' own order
    v_params: torch.Tensor  # as k_params
    group: int = GROUP

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.k_codes, self.k_params, self.v_codes, self.v_params))


@dataclass
class KVBatch:
    """Rows of a step by sequence, the newest tokens of each, on the device."""
    rows: torch.Tensor        # int32 [S + 1]: sequence s has rows [rows[s], rows[s + 1])
    lengths: torch.Tensor     # int32 [S]: tokens in the cache, those of the rows among them
    page_table: torch.Tensor  # int32 [S][max_pages]; -1: no page
    # no sequence has more rows; None: as many as there are, which takes a decoding batch (1) half as long again
    max_rows: int | None = None


@dataclass
class Rotary:
    """Rotation by position: cos of rotary_dim / 2 angles, then sin, for every position."""
    table: torch.Tensor        # fp32 [positions][rotary_dim]
    interleaved: bool = False  # pairs (2 i, 2 i + 1) instead of (i, i + rotary_dim / 2)


def alloc_kv_cache(pages: int, kv_heads: int, head_dim: int, device, page_size: int = 64,
                   group: int | None = None) -> KVCache:
    """An empty cache (its memory is not cleared: what lies behind a sequence is never used).
    group: channels that share a scale; None: 128, or the head's 64."""
    group = min(GROUP, head_dim) if group is None else group
    codes = dict(size=(pages, kv_heads, page_size, head_dim // 2), dtype=torch.uint8, device=device)
    params = dict(size=(pages, kv_heads, head_dim // group, page_size), dtype=torch.int16, device=device)
    return KVCache(torch.empty(**codes), torch.empty(**params), torch.empty(**codes), torch.empty(**params), group)


def _cache(c, device):
    pages, heads, size, half = c.k_codes.shape
    params = (pages, heads, 2 * half // c.group if c.group > 0 else 0, size)
    codes = c.k_codes.shape
    return _abi.KvCache(_check(c.k_codes, torch.uint8, codes, "k_codes", device),
                        _check(c.k_params, torch.int16, params, "k_params", device),
                        _check(c.v_codes, torch.uint8, codes, "v_codes", device),
                        _check(c.v_params, torch.int16, params, "v_params", device),
                        pages, size, heads, 2 * half, c.group)


def _batch(b, n_rows, device):
    if not isinstance(b.page_table, torch.Tensor) or b.page_table.dim() != 2:
        raise ValueError("page_table must be [S][max_pages]")
    S, wide = b.page_table.shape
    most = n_rows if b.max_rows is None else min(b.max_rows, n_rows)
    return _abi.KvBatch(_check(b.rows, torch.int32, (S + 1,), "rows", device),
                        _check(b.lengths, torch.int32, (S,), "lengths", device),
                        _check(b.page_table, torch.int32, (S, wide), "page_table", device), n_rows, S, wide, most)


def _heads(t, rows, heads, dim, name, device):
    """(address, stride) of rows of heads: fp16 [rows][heads][dim], the rows may be strided."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.float16:
        raise TypeError(f"{name} must be torch.float16, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.shape != (rows, heads, dim):
        raise ValueError(f"{name} must have shape {(rows, heads, dim)}, got {tuple(t.shape)}")
    ld, by_head, by_dim = t.stride()
    if by_dim != 1 or heads > 1 and by_head != dim or rows > 1 and ld < heads * dim:
        raise ValueError(f"{name} must have contiguous heads, and rows that do not overlap")
    return t.data_ptr(), ld if rows > 1 else heads * dim


def _dims(cache):
    if not isinstance(cache.k_codes, torch.Tensor) or cache.k_codes.dim() != 4:
        raise ValueError("k_codes must be [pages][kv_heads][page_size][head_dim / 2]")
    return cache.k_codes.shape[1], 2 * cache.k_codes.shape[3]


def kv_append(cache: KVCache, batch: KVBatch, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor | None = None,
              rope: Rotary | None = None, out: torch.Tensor | None = None,
              flags: torch.Tensor | None = None) -> torch.Tensor | None:
    """awq_kv_append: keys and values fp16 [T][kv_heads][head_dim] (rows may be strided: parts of
    the q|k|v linear's output) into the cache, keys rotated by position; q [T][q_heads][head_dim]
    is rotated too, into out (may be q). Returns out, or None without q."""
    dev = _first(k, (torch.float16,), 3, "k")
    heads, dim = _dims(cache)
    T = k.shape[0]
    kp, kl = _heads(k, T, heads, dim, "k", dev)
    vp, vl = _heads(v, T, heads, dim, "v", dev)
    qp = ql = op = ol = qh = 0
    if q is not None:
        if rope is None:
            raise ValueError("q is only taken to be rotated: rope is missing")
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be [T][q_heads][head_dim]")
        qh = q.shape[1]
        qp, ql = _heads(q, T, qh, dim, "q", dev)
        if out is None:
            out = torch.empty((T, qh, dim), dtype=torch.float16, device=dev)
        op, ol = _heads(out, T, qh, dim, "out", dev)
    elif out is not None:
        raise ValueError("out is the rotated q: q is missing")
    tp = positions = rotary = 0
    if rope is not None:
        if not isinstance(rope.table, torch.Tensor) or rope.table.dim() != 2:
            raise ValueError("rope.table must be [positions][rotary_dim]")
        positions, rotary = rope.table.shape
        tp = _check(rope.table, torch.float32, (positions, rotary), "rope.table", dev)
    _launch("awq_kv_append", dev, _cache(cache, dev), _batch(batch, T, dev), kp, kl, vp, vl, qp or None, ql, qh,
            op or None, ol, tp or None, positions, rotary, int(bool(rope is not None and rope.interleaved)),
            _flags(flags, dev))
    return out


def kv_read(cache: KVCache, batch: KVBatch, n_rows: int | None = None,
            out: tuple[torch.Tensor, torch.Tensor] | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """awq_kv_read: what the cache holds for the batch's rows, keys and values fp16
    [n_rows][kv_heads][head_dim], exactly. n_rows (rows of the batch) or out is needed."""
    heads, dim = _dims(cache)
    dev = _first(cache.k_codes, (torch.uint8,), 4, "k_codes")
    if out is None:
        if n_rows is None:
            raise ValueError("n_rows or out is needed: the batch's rows stand on the device")
        half = dict(dtype=torch.float16, device=dev)
        out = torch.empty((n_rows, heads, dim), **half), torch.empty((n_rows, heads, dim), **half)
    k, v = out
    T = k.shape[0] if n_rows is None else n_rows
    kp = _check(k, torch.float16, (T, heads, dim), "k", dev)
    vp = _check(v, torch.float16, (T, heads, dim), "v", dev)
    _launch("awq_kv_read", dev, _cache(cache, dev), _batch(batch, T, dev), kp, vp)
    return k, v


def attention_kv4_workspace_size(n_rows: int, seqs: int, max_rows: int, max_tokens: int, q_heads: int,
                                 kv_heads: int, head_dim: int) -> int:
    """Bytes of workspace (a uint8 tensor) that attention_kv4 takes; max_tokens: what a row of
    the page table can hold. 0: none."""
    return _workspace_size("awq_attention_kv4_workspace_size", n_rows, seqs, max_rows, max_tokens, q_heads, kv_heads,
                           head_dim)


def attention_kv4(q: torch.Tensor, cache: KVCache, batch: KVBatch, scale: float | None = None, causal: bool = True,
                  window: int = 0, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """awq_attention_kv4: attention of q fp16 [T][q_heads][head_dim] (rows may be strided), the
    batch's rows, over their sequences in the cache. scale: 1 / sqrt(head_dim) by default;
    out: may be q; window: only the last so many tokens up to the row's own (0: all); lse fp32 [T][q_heads]
    (optional): log of the sums of exponentials. workspace: attention_kv4_workspace_size bytes,
    one for each of the calls that overlap."""
    dev = _first(q, (torch.float16,), 3, "q")
    heads, dim = _dims(cache)
    T, qh, _ = q.shape
    qp, ql = _heads(q, T, qh, dim, "q", dev)
    c, b = _cache(cache, dev), _batch(batch, T, dev)
    if out is None:
        out = torch.empty((T, qh, dim), dtype=torch.float16, device=dev)
    op, ol = _heads(out, T, qh, dim, "out", dev)
    lp = None if lse is None else _check(lse, torch.float32, (T, qh), "lse", dev)
    wp, wn, _keep = _workspace(workspace, attention_kv4_workspace_size(T, b.seqs, b.max_rows, b.max_pages * c.page_size,
                                                                      qh, heads, dim), dev)
    _launch("awq_attention_kv4", dev, qp, ql, qh, c, b, 1 / math.sqrt(dim) if scale is None else scale,
            int(bool(causal)), window, op, ol, lp, wp, wn)
    return out
