"""Attention over tokens of the 4-bit cache in 64 bits, with error bounds that hold for every row
by what that row itself sees. Shares no code with the library."""

import math

import torch


def tokens(awq, cache, batch, s, length):
    """Sequence s of a batch: keys and values [length][heads][D] and the values' scales
    [length][heads][D / group], in 64 bits on the CPU."""
    size = cache.k_codes.shape[2]
    one = awq.KVBatch(torch.tensor([0, length], dtype=torch.int32, device=batch.rows.device),
                      torch.tensor([length], dtype=torch.int32, device=batch.rows.device), batch.page_table[s:s + 1].clone())
    k, v = (t.cpu().double() for t in awq.kv_read(cache, one, length))
    t = torch.arange(length)
    page = batch.page_table[s].cpu().long()[t // size]
    sc = (cache.v_params.cpu()[page, :, :, t % size] & -16).view(torch.float16).double()
    return k, v, sc


def attention(q, kv, scale, causal, window, folded, rounded):
    """Rows q [n][q_heads][D] at the end of a sequence: (out, lse, bound of |out - exact|, of lse).

    The error of a score is that of adding D exact products and of a few roundings; with the
    exponential's and that of adding the numbers themselves, a term of numerator or denominator is
    off by at most e = (D + 8) 2^-24 scale sum |q| |k| + 2^-21 + n 2^-24, relatively. A probability goes to
    the second product as fp16 hi + lo (2^-22 relative) or as one fp16 (rounded: 2^-11), 2^-25 absolute in
    units in which the largest one is 2^7 or more: 2^-32 of the value. Folded: the probability times the
    value's scale does so, in units in which the largest such product that the row has in the group is
    2^6 or more: 2^-31 of 15 times it. The output is rounded to fp16."""
    k, v, sc = kv
    n, heads, D = q.shape
    share, length = heads // k.shape[1], k.shape[0]
    t = torch.arange(length)
    out, lse = torch.zeros(n, heads, D, dtype=torch.float64), torch.full((n, heads), -math.inf, dtype=torch.float64)
    bound, lse_bound = torch.zeros_like(out), torch.zeros_like(lse)
    for i in range(n):
        p = length - n + i
        if p < 0:
            continue  # no token
        see = torch.ones(length, dtype=torch.bool)
        if causal:
            see &= t <= p
        if window:
            see &= t > p - window
        for h in range(heads):
            kk, vv, ss = k[see, h // share], v[see, h // share], sc[see, h // share]
            if len(kk) == 0:
                continue
            s = scale * (kk @ q[i, h])
            size = (scale * (kk.abs() @ q[i, h].abs())).max()
            top = s.max()
            w = torch.exp(s - top)
            w_sum = w.sum()
            out[i, h], lse[i, h] = w @ vv / w_sum, top + w_sum.log()
            e = (D + 8) * 2.0 ** -24 * size + 2.0 ** -21 + len(kk) * 2.0 ** -24
            if folded:
                least = len(kk) * 2.0 ** -31 * 15 * (w[:, None] * ss).amax(0).repeat_interleave(D // ss.shape[1])
            else:
                least = 2.0 ** -32 * vv.abs().sum(0)
            off = (2 * e + (2.0 ** -11 if rounded else 2.0 ** -22)) * (w @ vv.abs()) / w_sum + least / w_sum
            bound[i, h] = off + 2.0 ** -11 * (out[i, h].abs() + off) + 2.0 ** -25
            lse_bound[i, h] = e + 2.0 ** -22 * (lse[i, h].abs() + top.abs() + 1)
    return out, lse, bound, lse_bound


def check(y, lse, want):
    """Asserts that outputs and log-sum-exp are within the bounds of attention()."""
    out, want_lse, bound, lse_bound = want
    y, lse = y.cpu().double(), lse.cpu().double()
    none = torch.isneginf(want_lse)
    assert torch.equal(torch.isneginf(lse), none)
    assert bool((y[none] == 0).all())
    off = (y - out).abs()
    assert bool((off <= bound).all()), ((off / bound).nan_to_num(nan=math.inf).max().item(), off.max().item())
    assert bool(((lse - want_lse).abs() <= lse_bound)[~none].all())
