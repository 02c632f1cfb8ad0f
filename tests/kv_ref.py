"""Plain 64-bit forms of the 4-bit key / value cache and of the attention over it (NumPy), and
the error bounds of the latter. They share no code with the library."""

import math

import numpy as np

NIBBLE = [0, 4, 1, 5, 2, 6, 3, 7]


def quantize(x, group):
    """fp16 [..., D] -> codes [..., D], scales and zeros [..., D / group]."""
    v = x.astype(np.float64).reshape(*x.shape[:-1], -1, group)
    lo, hi = np.minimum(v.min(-1), 0.0), np.maximum(v.max(-1), 0.0)
    sc = ((hi - lo).astype(np.float32) / np.float32(15)).astype(np.float64)
    m, e = np.frexp(sc)
    sc = np.clip(np.ldexp(np.ceil(m * 128), e - 7), 2.0 ** -14, 4352.0)
    z = np.clip(np.rint(-lo / sc), 0, 15)
    q = np.clip(np.rint(v / sc[..., None]) + z[..., None], 0, 15)
    return q.astype(np.int64).reshape(x.shape), sc, z.astype(np.int64)


def params(sc, z):
    return (sc.astype(np.float16).view(np.uint16) | z.astype(np.uint16)).astype(np.uint16)


def rotate(x, table, interleaved):
    """x fp16 [T][H][D] by rows of table fp32 [T][R] (cos, then sin)."""
    R = table.shape[1]
    y = x.copy()
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        c, s = table[:, i].astype(np.float64)[:, None], table[:, R // 2 + i].astype(np.float64)[:, None]
        u, w = x[:, :, a].astype(np.float64), x[:, :, b].astype(np.float64)
        with np.errstate(over="ignore", invalid="ignore"):
            y[:, :, a] = (u * c - w * s).astype(np.float32).astype(np.float16)
            y[:, :, b] = (w * c + u * s).astype(np.float32).astype(np.float16)
    return y


def k_place(D):
    """(byte, shift) of each channel in a token's row of key codes."""
    d = np.arange(D)
    nibble = 8 * ((d % 32 // 8) * (D // 32) + d // 32) + np.array(NIBBLE)[d % 8]
    return nibble // 2, 4 * (nibble % 2)


def v_place(D, place):
    """(byte, shift) of each channel of the token at `place` in a page's value codes of one head."""
    d, i = np.arange(D), place % 16
    cell = (((i // 4) * 16 + d % 16) * (D // 64) + d // 64) * 4 + i % 4
    nibble = d // 16 % 4
    return (place // 16) * 8 * D + 2 * cell + nibble // 2, 4 * (nibble % 2)


class Cache:
    """The four arrays of a cache on the host."""

    def __init__(self, pages, heads, size, D, group, rng):
        self.pages, self.heads, self.size, self.D, self.group = pages, heads, size, D, group
        self.k_codes, self.v_codes = (rng.integers(0, 256, (pages, heads, size, D // 2)).astype(np.uint8) for _ in "kv")
        # what no token wrote may be anything: NaN and infinite scales among it
        self.k_params, self.v_params = (rng.choice(np.array([0x7C00, 0x7FFF, 0xFFFF, 0x3C05], np.uint16),
                                                   (pages, heads, D // group, size)) for _ in "kv")

    def put(self, page, place, k, v):
        """One token's fp16 keys and values [heads][D]."""
        for name, x in (("k", k), ("v", v)):
            q, sc, z = quantize(x, self.group)
            codes = getattr(self, name + "_codes")[page].reshape(self.heads, -1)
            if name == "k":
                at, shift = k_place(self.D)
                at = at + place * (self.D // 2)
            else:
                at, shift = v_place(self.D, place)
            for d in range(self.D):
                codes[:, at[d]] = codes[:, at[d]] & ~(15 << shift[d]) & 255 | q[:, d] << shift[d]
            getattr(self, name + "_params")[page, :, :, place] = params(sc, z)

    def get(self, name, page, place):
        """One token's values, float64 [heads][D]."""
        codes = getattr(self, name + "_codes")[page].reshape(self.heads, -1)
        if name == "k":
            at, shift = k_place(self.D)
            at = at + place * (self.D // 2)
        else:
            at, shift = v_place(self.D, place)
        p = getattr(self, name + "_params")[page, :, :, place]
        sc = (p & 0xFFF0).astype(np.uint16).view(np.float16).astype(np.float64).repeat(self.group, 1)
        return ((codes[:, at] >> shift & 15).astype(np.int64) - (p & 15).astype(np.int64).repeat(self.group, 1)) * sc


def tokens(cache, table_row, length):
    """Keys and values of a sequence [length][heads][D], the ranges 15 scale of the values' groups, and
    which tokens have a page."""
    k, v, v_range = (np.zeros((length, cache.heads, cache.D)) for _ in "kvr")
    there = np.zeros(length, bool)
    for t in range(length):
        at = t // cache.size
        if at < len(table_row) and 0 <= table_row[at] < cache.pages:
            k[t], v[t] = cache.get("k", table_row[at], t % cache.size), cache.get("v", table_row[at], t % cache.size)
            p = cache.v_params[table_row[at], :, :, t % cache.size]
            sc = (p & 0xFFF0).astype(np.uint16).view(np.float16).astype(np.float64)
            v_range[t] = 15 * sc.repeat(cache.group, 1)
            there[t] = True
    return k, v, v_range, there


def attention(q, kv, scale, causal, window, rounded):
    """Rows q [n][q_heads][D] at the end of a sequence (kv: what tokens() gives): (out, lse, bound of
    |out - exact|, of lse).

    The bounds. Terms q (code - zero), or q times the value, are exact as products of short numbers; a
    kernel may multiply their sums by the scale in fp32. D of them are added with an error of at most
    D 2^-24 of the sum of their sizes; scales, softmax scale, the maximum and the exponential (two units
    of 2^-23) are a few roundings of the score more: a probability is off by at most
    e = (D + 8) 2^-24 softmax_scale sum |q| |k| + 2^-21, relatively.
    Numerator and denominator have that error each, and that of adding n numbers, n 2^-24.
    Probabilities (or probabilities times scale) go to the second product as fp16 hi + lo: 2^-22
    relative, and 2^-25 absolute in units where the largest scale times a probability of one is 2^6 or
    more, times code - zero: 2^-31 of 15 scale. rounded = True: or as fp16 beside exact values, 2^-11
    relative, 2^-24 absolute of the largest probability. The output is rounded to fp16: 2^-11 relative,
    2^-25 absolute."""
    k, v, v_range, there = kv
    n, heads, D = q.shape
    share, length = heads // k.shape[1], k.shape[0]
    out, lse = np.zeros((n, heads, D)), np.full((n, heads), -np.inf)
    bound, lse_bound = np.zeros((n, heads, D)), np.zeros((n, heads))
    t = np.arange(length)
    for i in range(n):
        p = length - n + i
        see = there.copy()
        if causal:
            see &= t <= p
        if window:
            see &= t > p - window
        if not see.any():
            continue
        for h in range(heads):
            kk, vv = k[see, h // share], v[see, h // share]
            vr = v_range[see, h // share]
            s = scale * (kk @ q[i, h])
            size = (scale * (np.abs(kk) @ np.abs(q[i, h]))).max()
            top = s.max()
            w = np.exp(s - top)
            w_sum = w.sum()
            out[i, h], lse[i, h] = w @ vv / w_sum, top + math.log(w_sum)
            e = (D + 8) * 2.0 ** -24 * size + 2.0 ** -21 + see.sum() * 2.0 ** -24
            off = (2 * e + 2.0 ** -22) * (w @ np.abs(vv)) / w_sum + see.sum() * 2.0 ** -31 * vr.max() / w_sum
            if rounded:
                off = off + 2.0 ** -11 * (w @ np.abs(vv)) / w_sum + 2.0 ** -24 * np.abs(vv).sum(0) / w_sum
            bound[i, h] = off + 2.0 ** -11 * (np.abs(out[i, h]) + off) + 2.0 ** -25
            lse_bound[i, h] = e + 2.0 ** -22 * (abs(lse[i, h]) + abs(top) + 1)
    return out, lse, bound, lse_bound
