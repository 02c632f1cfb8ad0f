"""Plain fp64 forms of the expert and adapter operators, and the error bounds of the kernels.

Bounds count the roundings the kernels make (u = 2^-11, half a step of fp16):
* a dequantized operand (q - z) sc is rounded to fp16 once at most: u S, S = sum |x| |w|;
* fp32 accumulation over K products: K 2^-23 S covers any order and truncating adders;
* the result is rounded to fp16 once: u |y|, and half the smallest subnormal, 2^-25.
"""

import numpy as np

import oracle

U = 2.0 ** -11
TINY = 2.0 ** -25


def packed_numpy(N, K, group, w_bit, seed):
    """A packed weight of normal values (oracle layout) and its fp64 dequantization."""
    g = np.random.default_rng(seed)
    W = (g.standard_normal((N, K)) * 0.02).astype(np.float16)
    qw, sc, zb, _ = oracle.quantize_pack(W, group=group, w_bit=w_bit)
    q, z, s = oracle.unpack(qw, sc, zb, K)
    return (qw.view(np.int32), sc, zb), oracle.dequantize(q, z, s)


def group_reference(ids, groups):
    key = np.where((ids < 0) | (ids >= groups), groups, ids)
    order = np.argsort(key, kind="stable")
    pos = np.empty_like(order)
    pos[order] = np.arange(len(order))
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=groups + 1)[:groups])])
    return offsets.astype(np.int32), order.astype(np.int32), pos.astype(np.int32)


def route_reference(x, k, renorm):
    """(weights fp64, ids, error bound of the weights) of fp64 logits x [T][E]."""
    T, E = x.shape
    ids = np.argsort(-x, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(x, ids, 1)
    live = np.isfinite(top[:, :1])
    m = np.where(live, top[:, :1], 0.0)
    with np.errstate(over="ignore"):
        e = np.exp(top - m)
        total = e.sum(1, keepdims=True) if renorm else np.exp(x - m).sum(1, keepdims=True)
    w = np.where(live & np.isfinite(top), e / np.where(live, total, 1.0), 0.0)
    ids = np.where(np.isfinite(top), ids, -1).astype(np.int32)
    # the rounded difference l - m moves exp by |l - m| 2^-24; expf and the division are good
    # to 2 ulp; the sum has at most E roundings, each term the error of its own exponential
    # (e^-d d <= 0.37): together below (|l - m| + E + 8) 2^-24, relative
    dist = np.where(np.isfinite(top), m - top, 0.0)
    return w, ids, w * (dist + E + 8) * 2.0 ** -24 + 2.0 ** -149


def linear_reference(X, Wd):
    X = X.astype(np.float64)
    return X @ Wd.T, np.abs(X) @ np.abs(Wd).T


def linear_bound(y, S, K):
    return S * (U + K * 2.0 ** -23) + np.abs(y) * U + TINY


def gated_reference(X, Wd):
    """(h, bound) of SiLU(g) u from the bounds of g and u before their fp16 rounding."""
    y, S = linear_reference(X, Wd)
    nh = Wd.shape[0] // 2
    d = S * (U + Wd.shape[1] * 2.0 ** -23)
    g, u, dg, du = y[:, :nh], y[:, nh:], d[:, :nh], d[:, nh:]
    h = oracle.silu(g) * u
    # |SiLU'| <= 1.1; the fp32 SiLU itself is good to 2^-18 (hardware exp and reciprocal)
    bound = 1.1 * dg * (np.abs(u) + du) + np.abs(oracle.silu(g)) * du + np.abs(h) * (U + 2.0 ** -18) + TINY
    return h, bound


def lora_reference(X, Wd, A, B, scale, ids):
    """(y, bound): the linear plus each row's adapter. A [L][r][K], B [L][N][r]."""
    y, S = linear_reference(X, Wd)
    K, r = Wd.shape[1], A.shape[1]
    bound = S * (U + (K + r) * 2.0 ** -23)
    Xd = X.astype(np.float64)
    for i, a in enumerate(ids):
        if 0 <= a < A.shape[0]:
            Ad, Bd, s = A[a].astype(np.float64), B[a].astype(np.float64), float(scale[a])
            h, hS = s * (Ad @ Xd[i]), abs(s) * (np.abs(Ad) @ np.abs(Xd[i]))
            y[i] += Bd @ h
            # h: fp32 over K products, one product with the scale; then hi + lo keeps 2^-22 of
            # the row's largest |h|; the second product accumulates 2 r terms in fp32
            dh = hS * (K + 2) * 2.0 ** -23 + np.abs(h).max(initial=0.0) * 2.0 ** -22
            bound[i] += np.abs(Bd) @ dh + (np.abs(Bd) @ np.abs(h)) * (2 * r + 4) * 2.0 ** -23
    return y, bound + np.abs(y) * U + TINY
