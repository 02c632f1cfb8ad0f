"""Batches of the key / value cache for the GPU tests."""

import numpy as np
import torch

from . import kv_ref
from .gpu_util import DEV, to_dev

NAMES = ("k_codes", "k_params", "v_codes", "v_params")


def on_device(awq, c):
    """A kv_ref.Cache as the binding's KVCache."""
    return awq.KVCache(to_dev(c.k_codes), to_dev(c.k_params.view(np.int16)), to_dev(c.v_codes),
                       to_dev(c.v_params.view(np.int16)), c.group)


def same(dev_cache, c):
    """Whether the device's cache is the host's, byte for byte."""
    return [n for n in NAMES if not np.array_equal(getattr(dev_cache, n).cpu().numpy().view(getattr(c, n).dtype),
                                                   getattr(c, n))]


def batch_of(awq, n, lengths, size, rng, spare=2, wide=None, max_rows=None, holes=()):
    """A KVBatch of sequences with n rows each; (batch, pages, table, rows). holes: (sequence,
    page number) pairs that have no page."""
    need = [-(-x // size) for x in lengths]
    wide = wide or max(need + [1])
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(n), wide), -1, np.int32)
    at = 0
    for s, k in enumerate(need):
        k = min(k, wide)
        table[s, :k] = order[at:at + k]
        at += k
    for s, p in holes:
        table[s, p] = rng.choice([-1, pages, 2 ** 31 - 1, -2 ** 31])
    rows = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    b = awq.KVBatch(to_dev(rows), to_dev(np.array(lengths, np.int32)), to_dev(table), max_rows)
    return b, pages, table, rows


def filled(pages, heads, size, D, group, table, lengths, rng, k_gain=1.0, v_gain=1.0):
    """A cache with random tokens wherever the sequences have a page."""
    c = kv_ref.Cache(pages, heads, size, D, group, rng)
    for s, length in enumerate(lengths):
        for t in range(length):
            if t // size < table.shape[1] and 0 <= table[s, t // size] < pages:
                k = (rng.standard_normal((heads, D)) * k_gain).astype(np.float16)
                k[:, D // 3] *= np.float16(4)
                c.put(table[s, t // size], t % size, k,
                      (rng.standard_normal((heads, D)) * v_gain).astype(np.float16))
    return c


def strided(x, extra=8):
    """x [T][H][D] as rows with `extra` values behind each."""
    T, H, D = x.shape
    t = torch.full((T, H * D + extra), 7.0, dtype=torch.float16, device=DEV)
    t[:, :H * D] = to_dev(x).view(T, H * D)
    return t[:, :H * D].unflatten(1, (H, D))
