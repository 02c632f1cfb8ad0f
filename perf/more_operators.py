"""The paged key/value cache held in 4 bits and the attention over it, as measured cases.

Three kinds of case:

* ``append``  new tokens' keys and values into the cache (rotated by position, quantized),
              their queries rotated on the way; returned with the values the cache then holds;
* ``attend``  attention of the newest rows of every sequence over its tokens in the cache;
* ``read``    tokens of the cache back as fp16.

``run`` computes them in elementary torch operations in 32 bits (rotation and quantizer in 64,
where a rounding decides a code), or, where ``own`` is set, through the framework. ``exact``
computes them from their definitions in 64 bits.

The cache: per token and head, each group of ``group`` channels has a scale of 7 significant
bits and a zero, one 16-bit word (the fp16 bits of the scale, the zero in the low four), and
4-bit codes: value = (code - zero) scale, exact in fp16.

* key codes: a token's row of D / 8 words of 32 bits; word h (D / 32) + s holds channels
  32 s + 8 h + i, i < 8, channel i in nibble (0, 4, 1, 5, 2, 6, 3, 7)[i];
* value codes: 16 tokens together, as 16-bit words [4][16][D / 64][4]: word (h, c, w, i) holds
  token 4 h + i's channels c + 16 (4 w + j) in nibble j;
* scales and zeros: [group][token of the page].
"""

import math

import torch

own = False

DEV = "cuda"
OUTLIERS, GAIN = 0.02, 6.0   # of a head's key channels, 2% are 6 times larger
BASE = 10000.0               # of the rotation's angles

# --------------------------------------------------------------------------- cases


def listed():
    return [
        # one token of a decoding step of one sequence, all heads with keys of their own
        dict(name="append one token", kind="append", S=1, n_lo=1, n_hi=1, len_lo=1000, len_hi=1000, Hq=32, Hkv=32,
             D=128, group=128, page=16, rotary=128, interleaved=False),
        # a decoding batch with shared key heads, smaller groups
        dict(name="append decode batch", kind="append", S=64, n_lo=1, n_hi=1, len_lo=7, len_hi=6000, Hq=64, Hkv=8,
             D=128, group=32, page=64, rotary=128, interleaved=False),
        # prompts of different lengths, interleaved rotation of half the channels
        dict(name="append prompts", kind="append", S=5, n_lo=120, n_hi=2000, len_lo=150, len_hi=2500, Hq=32, Hkv=32,
             D=128, group=64, page=32, rotary=64, interleaved=True),
        # one token of a young sequence: latency alone
        dict(name="attend one token", kind="attend", S=1, n_lo=1, n_hi=1, len_lo=77, len_hi=77, Hq=32, Hkv=32, D=128,
             group=128, page=16, causal=True, window=0),
        # a decoding batch, every head with keys of its own, ragged lengths
        dict(name="attend decode batch", kind="attend", S=24, n_lo=1, n_hi=1, len_lo=300, len_hi=4000, Hq=32, Hkv=32,
             D=128, group=128, page=64, causal=True, window=0),
        # a decoding batch with eight shared key heads in groups of 32, very ragged lengths
        dict(name="attend decode shared heads", kind="attend", S=64, n_lo=1, n_hi=1, len_lo=1, len_hi=9000, Hq=64,
             Hkv=8, D=128, group=32, page=16, causal=True, window=0),
        # one long context: few rows, the work is split over the length
        dict(name="attend one long sequence", kind="attend", S=1, n_lo=1, n_hi=1, len_lo=131071, len_hi=131071, Hq=64,
             Hkv=8, D=128, group=128, page=256, causal=True, window=0),
        # several drafted tokens a sequence under a sliding window, narrow heads
        dict(name="attend drafts in a window", kind="attend", S=16, n_lo=3, n_hi=6, len_lo=900, len_hi=12000, Hq=32,
             Hkv=8, D=64, group=64, page=32, causal=True, window=4096),
        # a fresh prompt
        dict(name="attend prompt", kind="attend", S=1, n_lo=4096, n_hi=4096, len_lo=4096, len_hi=4096, Hq=32, Hkv=32,
             D=128, group=128, page=64, causal=True, window=0),
        # prompts' pieces behind long histories, shared heads, groups of 64, ragged
        dict(name="attend prompt pieces", kind="attend", S=3, n_lo=257, n_hi=1024, len_lo=2000, len_hi=12345, Hq=64,
             Hkv=8, D=128, group=64, page=128, causal=True, window=0),
        # a prefix that another engine takes over
        dict(name="read prefix", kind="read", S=1, n_lo=8192, n_hi=8192, len_lo=8192, len_hi=8192, Hkv=8, D=128,
             group=128, page=64),
        # the latest tokens of many sequences
        dict(name="read latest", kind="read", S=32, n_lo=1, n_hi=50, len_lo=60, len_hi=3000, Hkv=32, D=128, group=32,
             page=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST_FLOPS = 2.5e11      # of the largest listed cases
MOST_BYTES = 1.5e8
MOST_SCORES = 6e8        # of the plain form, padded
MOST_CACHE = 2.5e8       # padded values of the keys


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        n, length = _sizes(c)
        padded = c["S"] * max(length) * c["Hkv"] * c["D"]
        if w["flops"] > MOST_FLOPS or w["bytes"] > MOST_BYTES or padded > MOST_CACHE:
            continue
        if c["kind"] == "attend" and c["S"] * max(n) * max(length) * c["Hq"] > MOST_SCORES:
            continue
        return c


def _draw(rng):
    kind = rng.choice(["append", "append", "attend", "attend", "attend", "attend", "attend", "read"])
    D = rng.choice([64, 128, 128, 128, 256])
    group = rng.choice([g for g in (32, 64, 128, 128) if g <= D])
    Hkv = rng.choice([1, 2, 4, 8, 8, 32])
    Hq = Hkv * rng.choice([1, 1, 2, 3, 4, 7, 8] if Hkv < 32 else [1, 1, 2])
    c = dict(kind=kind, D=D, group=group, Hkv=Hkv, page=rng.choice([16, 32, 64, 128, 256]))
    rows = rng.choice(["one", "few", "many"])
    c["S"] = _log_int(rng, 1, 8 if rows == "many" else 100)
    if rows == "one":
        c["n_lo"] = c["n_hi"] = 1
    else:
        c["n_lo"], c["n_hi"] = sorted(_log_int(rng, 1, 9 if rows == "few" else 2000) for _ in range(2))
    # histories behind the rows, none included
    c["len_lo"], c["len_hi"] = sorted(c["n_hi"] + rng.choice([0, _log_int(rng, 1, 20000)]) for _ in range(2))
    if kind == "read":
        return c
    c["Hq"] = Hq
    if kind == "append":
        return dict(c, rotary=rng.choice([D, D, D // 2]), interleaved=rng.random() < 0.3)
    return dict(c, causal=rng.random() < 0.85, window=rng.choice([0, 0, 0, _log_int(rng, 1, 5000)]))


def _sizes(c):
    """Rows and length of every sequence: spread over the case's ranges by the golden ratio."""
    def at(s, lo, hi):
        return lo + int((hi - lo + 1) * ((s * 0.6180339887498949 + 0.37) % 1.0))
    n = [at(s, c["n_lo"], c["n_hi"]) for s in range(c["S"])]
    return n, [max(n[s], at(3 * s + 1, c["len_lo"], c["len_hi"])) for s in range(c["S"])]


# --------------------------------------------------------------------------- inputs

_NIBBLE = (0, 4, 1, 5, 2, 6, 3, 7)


def _quantize(x, group):
    """Codes (int32, x's shape) and parameters (int32 [..., D / group]) of fp16 values."""
    v = x.double().unflatten(-1, (-1, group))
    lo, hi = v.amin(-1).clamp(max=0.0), v.amax(-1).clamp(min=0.0)
    # a tensor divides; a number would be multiplied by its reciprocal
    sc = ((hi - lo) / torch.tensor(15.0, dtype=torch.float64, device=v.device)).float()
    bits = (sc.view(torch.int32) + 0x1FFFF) & ~0x1FFFF
    sc = bits.view(torch.float32).clamp(2.0 ** -14, 4352.0)
    z = (-lo / sc.double()).round().clamp(0, 15)
    q = ((v / sc.double()[..., None]).round() + z[..., None]).clamp(0, 15)
    return q.to(torch.int32).flatten(-2), sc.half().view(torch.int16).to(torch.int32) | z.to(torch.int32)


def _nibbles(t, order):
    return sum(t[..., i] << (4 * at) for i, at in enumerate(order))


def _pack_k(q):
    """Codes [..., D] of keys to the rows' bytes [..., D / 2]."""
    D = q.shape[-1]
    words = _nibbles(q.unflatten(-1, (D // 32, 4, 8)), _NIBBLE).transpose(-1, -2)  # [..., h, s]
    return words.contiguous().flatten(-2).view(torch.uint8)


def _v_cell(q):
    """Codes [..., D] of one token's values as its 16-bit words [..., 16, D / 64]."""
    D = q.shape[-1]
    return _nibbles(q.unflatten(-1, (D // 64, 4, 16)).transpose(-1, -2), range(4)).transpose(-1, -2).to(torch.int16)


def _cache(gen, pages, c):
    """Pages full of tokens: keys with a few large channels, values, a hundred MB at a time."""
    Hkv, P, D, g = c["Hkv"], c["page"], c["D"], c["group"]
    out = dict(k_codes=torch.empty(pages, Hkv, P, D // 2, dtype=torch.uint8, device=DEV),
               v_codes=torch.empty(pages, Hkv, P, D // 2, dtype=torch.uint8, device=DEV),
               k_params=torch.empty(pages, Hkv, D // g, P, dtype=torch.int16, device=DEV),
               v_params=torch.empty(pages, Hkv, D // g, P, dtype=torch.int16, device=DEV))
    gain = torch.where(torch.rand(Hkv, 1, D, generator=gen, device=DEV) < OUTLIERS, GAIN, 1.0)
    some = max(1, 25_000_000 // (Hkv * P * D))
    for p in range(0, pages, some):
        n = min(some, pages - p)
        for which in ("k", "v"):
            x = torch.randn(n, Hkv, P, D, generator=gen, device=DEV)
            q, par = _quantize((x * gain if which == "k" else x * 0.5).half(), g)
            out[which + "_params"][p:p + n] = par.transpose(2, 3).to(torch.int16)
            if which == "k":
                out["k_codes"][p:p + n] = _pack_k(q)
            else:  # [.., unit, h, i, c, w] -> [.., unit, h, c, w, i]
                cells = _v_cell(q).unflatten(2, (P // 16, 4, 4)).permute(0, 1, 2, 3, 5, 6, 4).contiguous()
                out["v_codes"][p:p + n] = cells.view(torch.uint8).view(n, Hkv, P, D // 2)
    return out


def _table(rows, rotary):
    """cos and sin of the rotation's angles, fp32 [rows][rotary]: cos first."""
    freq = BASE ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device=DEV) / rotary)
    angle = torch.arange(rows, dtype=torch.float64, device=DEV)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    n, length = _sizes(c)
    S, P, T = c["S"], c["page"], sum(n)
    wide = -(-max(length) // P)
    need = [-(-x // P) for x in length]
    order = torch.randperm(sum(need) + 1, generator=gen, device=DEV).to(torch.int32)  # one page is nobody's
    table = torch.full((S, wide), -1, dtype=torch.int32)
    at = 0
    order_host = order.cpu()
    for s in range(S):
        table[s, :need[s]] = order_host[at:at + need[s]]
        at += need[s]
    rows = torch.tensor([sum(n[:s]) for s in range(S + 1)], dtype=torch.int32)
    s = dict(case=c, rows=rows.to(DEV), lengths=torch.tensor(length, dtype=torch.int32).to(DEV), table=table.to(DEV),
             most=max(n), longest=max(length), **_cache(gen, sum(need) + 1, c))
    half = dict(dtype=torch.float16, device=DEV)
    if c["kind"] == "append":  # the rows of a q|k|v linear
        Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=gen, device=DEV)
        qkv[:, Hq:Hq + Hkv] *= torch.where(torch.rand(Hkv, D, generator=gen, device=DEV) < OUTLIERS, GAIN, 1.0)
        s.update(qkv=qkv.half(), rope=_table(max(length), c["rotary"]), q_out=torch.empty(T, Hq, D, **half),
                 k_out=torch.empty(T, Hkv, D, **half), v_out=torch.empty(T, Hkv, D, **half))
    elif c["kind"] == "read":
        s.update(k_out=torch.empty(T, c["Hkv"], c["D"], **half), v_out=torch.empty(T, c["Hkv"], c["D"], **half))
    else:
        s.update(q=torch.randn(T, c["Hq"], c["D"], generator=gen, device=DEV).half(),
                 out=torch.empty(T, c["Hq"], c["D"], **half),
                 lse=torch.empty(T, c["Hq"], dtype=torch.float32, device=DEV))
    return s


# --------------------------------------------------------------------------- the operators


def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own_run(state, kind)
    return _PLAIN[kind](state)


def _own_run(s, kind):
    import weight_only_bit_02_amd as awq

    c = s["case"]
    cache = awq.KVCache(s["k_codes"], s["k_params"], s["v_codes"], s["v_params"], c["group"])
    batch = awq.KVBatch(s["rows"], s["lengths"], s["table"], s["most"])
    if kind == "append":
        q, k, v = s["qkv"].split([c["Hq"], c["Hkv"], c["Hkv"]], dim=1)
        q = awq.kv_append(cache, batch, k, v, q=q, rope=awq.Rotary(s["rope"], c["interleaved"]), out=s["q_out"])
        k, v = awq.kv_read(cache, batch, out=(s["k_out"], s["v_out"]))
        return dict(q=q, k=k, v=v)
    if kind == "read":
        k, v = awq.kv_read(cache, batch, out=(s["k_out"], s["v_out"]))
        return dict(k=k, v=v)
    out = awq.attention_kv4(s["q"], cache, batch, causal=c["causal"], window=c["window"], out=s["out"], lse=s["lse"])
    return dict(out=out, lse=s["lse"])


def _owners(s, T):
    """(sequence, position, page, place in the page) of every row."""
    rows, lengths = s["rows"].long(), s["lengths"].long()
    t = torch.arange(T, device=rows.device)
    seq = torch.searchsorted(rows, t, right=True) - 1
    p = lengths[seq] - (rows[seq + 1] - t)
    P = s["case"]["page"]
    return seq, p, s["table"][seq, p // P].long(), p % P


def _rotate(x, table, interleaved):
    """x fp16 [T][H][D], its first channels rotated by cos | sin fp32 [T][R]."""
    R = table.shape[1]
    cos, sin = table.double()[:, None].chunk(2, dim=2)
    v = x[..., :R].double()
    a, b = (v[..., 0::2], v[..., 1::2]) if interleaved else v.chunk(2, dim=2)
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r.float().half(), x[..., R:]], -1)


def _values(q, par, group):
    """(code - zero) scale in fp32 (exact) from codes [..., D] and parameters [..., D / group]."""
    sc = (par & 0xFFF0).to(torch.int16).view(torch.float16).float()
    v = q.unflatten(-1, (-1, group)) - (par & 15)[..., None]
    return (v.float() * sc[..., None]).flatten(-2)


def _plain_append(s):
    c, g = s["case"], s["case"]["group"]
    T, D = s["qkv"].shape[0], c["D"]
    seq, p, page, place = _owners(s, T)
    q, k, v = s["qkv"].split([c["Hq"], c["Hkv"], c["Hkv"]], dim=1)
    table = s["rope"][p]
    q, k = _rotate(q, table, c["interleaved"]), _rotate(k, table, c["interleaved"])
    kq, kp = _quantize(k, g)
    vq, vp = _quantize(v, g)
    s["k_codes"][page, :, place] = _pack_k(kq)
    s["k_params"][page, :, :, place] = kp.to(torch.int16)
    s["v_params"][page, :, :, place] = vp.to(torch.int16)
    cells = s["v_codes"].view(torch.int16).view(-1, c["Hkv"], c["page"] // 16, 4, 16, D // 64, 4)
    cells[page, :, place // 16, place // 4 % 4, :, :, place % 4] = _v_cell(vq)
    return dict(q=q, k=_values(kq, kp, g).half(), v=_values(vq, vp, g).half())


def _unpack_k(rows, D):
    """Key codes int32 [..., D] of row bytes [..., D / 2]."""
    w = rows.contiguous().view(torch.int32).unflatten(-1, (4, D // 32)).transpose(-1, -2)  # [..., s, h]
    return torch.stack([(w >> (4 * at)) & 15 for at in _NIBBLE], -1).flatten(-3)


def _unpack_v(pages, D):
    """Value codes int32 [..., P, D] of pages' bytes [..., P, D / 2]."""
    P = pages.shape[-2]
    w = pages.contiguous().view(torch.int16).flatten(-2).unflatten(-1, (P // 16, 4, 16, D // 64, 4)).to(torch.int32)
    w = torch.stack([(w >> (4 * j)) & 15 for j in range(4)], -1)          # [..., u, h, c, w, i, j]
    n = w.dim() - 6
    return w.permute(*range(n), n, n + 1, n + 4, n + 3, n + 5, n + 2).flatten(-3).flatten(n, n + 2)


def _plain_read(s):
    c, g = s["case"], s["case"]["group"]
    T, D, P = s["k_out"].shape[0], c["D"], c["page"]
    _, _, page, place = _owners(s, T)
    kp, vp = (s[n][page, :, :, place].int() for n in ("k_params", "v_params"))
    cells = s["v_codes"].view(torch.int16).view(-1, c["Hkv"], P // 16, 4, 16, D // 64, 4)
    w = cells[page, :, place // 16, place // 4 % 4, :, :, place % 4].int()  # [T][Hkv][16][D / 64]
    vq = torch.stack([(w >> (4 * j)) & 15 for j in range(4)], -1).permute(0, 1, 3, 4, 2).flatten(2)
    return dict(k=_values(_unpack_k(s["k_codes"][page, :, place], D), kp, g).half(), v=_values(vq, vp, g).half())


def _plain_attend(s):
    c, g, T = s["case"], s["case"]["group"], s["q"].shape[0]
    S, Hq, Hkv, D, n, L = c["S"], c["Hq"], c["Hkv"], c["D"], s["most"], s["longest"]
    at = s["table"].long().clamp(min=0)
    # keys and values of every sequence, [S][Hkv][tokens][D]
    kp, vp = (s[x][at].permute(0, 2, 1, 4, 3).flatten(2, 3).int() for x in ("k_params", "v_params"))
    k = _values(_unpack_k(s["k_codes"][at], D).transpose(1, 2).flatten(2, 3), kp, g)[:, :, :L]
    v = _values(_unpack_v(s["v_codes"][at], D).transpose(1, 2).flatten(2, 3), vp, g)[:, :, :L]
    rows, lengths = s["rows"].long(), s["lengths"].long()
    i = torch.arange(n, device=k.device)
    row = rows[:-1, None] + i                                             # [S][n]
    inside = row < rows[1:, None]
    q = s["q"].float()[row.clamp(max=T - 1)].unflatten(2, (Hkv, -1))      # [S][n][Hkv][Hq / Hkv][D]
    q = q.permute(0, 2, 3, 1, 4).flatten(0, 1).flatten(1, 2)              # [S Hkv][heads n][D]
    x = torch.bmm(q, k.flatten(0, 1).transpose(1, 2).contiguous()) * (1 / math.sqrt(D))
    p = (lengths - (rows[1:] - rows[:-1]))[:, None] + i                   # positions [S][n]
    t = torch.arange(L, device=k.device)
    see = (t < lengths[:, None, None]) & inside[..., None]
    if c["causal"]:
        see = see & (t <= p[..., None])
    if c["window"]:
        see = see & (t > p[..., None] - c["window"])
    x = x.view(S, Hkv, Hq // Hkv, n, L).masked_fill_(~see[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    e = x.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.bmm(e.view(S * Hkv, -1, L), v.flatten(0, 1)).view(S, Hkv, Hq // Hkv, n, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).flatten(2, 3)
    lse = (total.log() + top)[..., 0].permute(0, 3, 1, 2).flatten(2, 3)
    # back to the rows of the batch
    seq = torch.searchsorted(rows, torch.arange(T, device=k.device), right=True) - 1
    j = torch.arange(T, device=k.device) - rows[seq]
    return dict(out=o[seq, j].half(), lse=lse[seq, j])


_PLAIN = dict(append=_plain_append, read=_plain_read, attend=_plain_attend)


# --------------------------------------------------------------------------- what each has to do


def _token_bytes(c):
    """A token's keys and values in the cache."""
    return c["Hkv"] * (c["D"] + 4 * (c["D"] // c["group"]))


def work(case):
    c = case
    n, length = _sizes(c)
    T = sum(n)
    if c["kind"] == "read":
        return dict(bytes=T * (_token_bytes(c) + 4 * c["Hkv"] * c["D"]), flops=4 * T * c["Hkv"] * c["D"])
    if c["kind"] == "append":  # and read back
        heads = c["Hq"] + c["Hkv"]
        return dict(bytes=T * (2 * c["D"] * (heads + c["Hkv"]) + 2 * c["D"] * c["Hq"] + 2 * _token_bytes(c)
                               + 4 * c["rotary"] + 4 * c["Hkv"] * c["D"]),
                    flops=T * (3 * heads * c["rotary"] + 16 * c["Hkv"] * c["D"]))
    seen, tokens = 0, 0
    for a, b in zip(n, length):
        p0, w = b - a, c["window"] or b + a
        tokens += b - max(0, p0 - w + 1)
        if c["causal"]:
            seen += sum(min(p0 + i + 1, w) for i in range(a))
        else:
            seen += sum(b - max(0, p0 + i - w + 1) for i in range(a))
    return dict(bytes=tokens * _token_bytes(c) + T * c["Hq"] * (4 * c["D"] + 4), flops=4.0 * seen * c["Hq"] * c["D"])


# --------------------------------------------------------------------------- in 64 bits


def _cell64(s, which, page, place):
    """Values [len(page)][Hkv][D] of tokens of the cache, from the format's definition."""
    c = s["case"]
    D, g, P, Hkv = c["D"], c["group"], c["page"], c["Hkv"]
    d = torch.arange(D, device=DEV)
    par = s[which + "_params"].long()[page, :, :, place] & 0xFFFF            # [n][Hkv][D / g]
    exponent, fraction = (par >> 10).double(), ((par >> 4) & 63).double()
    scale = torch.exp2(exponent - 15) * (1 + fraction / 64)
    if which == "k":
        row = s["k_codes"][page, :, place].long()                            # [n][Hkv][D / 2]
        nibble = (8 * ((d % 32 // 8) * (D // 32) + d // 32)                  # 8 nibbles a word
                  + torch.tensor([0, 4, 1, 5, 2, 6, 3, 7], device=DEV)[d % 8])
        code = (row[..., nibble // 2] >> (4 * (nibble % 2))) & 15
    else:
        i = place % 16
        cell = ((((i // 4)[:, None] * 16 + d % 16) * (D // 64) + d // 64) * 4 + (i % 4)[:, None])  # [n][D]
        at = (place // 16 * 8 * D)[:, None] + 2 * cell + (d // 16 % 4 >= 2)
        flat = s["v_codes"].view(s["v_codes"].shape[0], Hkv, -1)
        byte = flat[page[:, None, None], torch.arange(Hkv, device=DEV)[None, :, None], at[:, None]].long()
        code = (byte >> (4 * (d // 16 % 2))) & 15
    return (code - (par & 15)[..., d // g]).double() * scale[..., d // g]


def _quantized64(x, g):
    """The values that the cache holds for fp16 x [...][D]."""
    v = x.double().reshape(*x.shape[:-1], -1, g)
    lo = torch.minimum(v.min(-1, keepdim=True).values, torch.zeros((), dtype=torch.float64, device=DEV))
    hi = torch.maximum(v.max(-1, keepdim=True).values, torch.zeros((), dtype=torch.float64, device=DEV))
    mantissa, exponent = torch.frexp(torch.div(hi - lo, torch.full_like(lo, 15.0)).float().double())
    scale = (torch.ceil(mantissa * 128) * torch.exp2(exponent.double() - 7)).clamp(2.0 ** -14, 4352)
    zero = torch.round(-lo / scale).clamp(0, 15)
    code = (torch.round(v / scale) + zero).clamp(0, 15)
    return ((code - zero) * scale).reshape(x.shape)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    n, length = _sizes(c)
    P, D = c["page"], c["D"]
    if c["kind"] == "append":
        pos = torch.cat([torch.arange(b - a, b, device=DEV) for a, b in zip(n, length)])
        R, out = c["rotary"], []
        for x in s["qkv"].split([c["Hq"], c["Hkv"]] + [c["Hkv"]], dim=1)[:2]:
            y = x.double().clone()
            for j in range(R // 2):
                a, b = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + R // 2)
                cos, sin = s["rope"][pos, j].double()[:, None], s["rope"][pos, R // 2 + j].double()[:, None]
                u, w = x[..., a].double(), x[..., b].double()
                y[..., a], y[..., b] = u * cos - w * sin, w * cos + u * sin
            out.append(y.float().half())
        v = s["qkv"][:, c["Hq"] + c["Hkv"]:]
        return dict(q=out[0].double(), k=_quantized64(out[1], c["group"]), v=_quantized64(v, c["group"]))
    table = s["table"].cpu()

    def tokens(i, lo, hi):
        t = torch.arange(lo, hi)
        return table[i, t // P].long().to(DEV), (t % P).to(DEV)

    if c["kind"] == "read":
        both = [tokens(i, b - a, b) for i, (a, b) in enumerate(zip(n, length))]
        page, place = torch.cat([x for x, _ in both]), torch.cat([x for _, x in both])
        return dict(k=_cell64(s, "k", page, place), v=_cell64(s, "v", page, place))
    share = c["Hq"] // c["Hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for i, (a, b) in enumerate(zip(n, length)):
        page, place = tokens(i, 0, b)
        k, v = (torch.cat([_cell64(s, w, x, y) for x, y in zip(page.split(8192), place.split(8192))]) for w in "kv")
        p = torch.arange(b - a, b, device=DEV)[:, None]
        t = torch.arange(b, device=DEV)
        see = torch.ones(a, b, dtype=torch.bool, device=DEV)
        if c["causal"]:
            see &= t <= p
        if c["window"]:
            see &= p - t < c["window"]
        for h in range(c["Hq"]):
            x = s["q"][at:at + a, h].double() @ k[:, h // share].t().contiguous() / math.sqrt(D)
            x = x.masked_fill(~see, -math.inf)
            lse[at:at + a, h] = torch.logsumexp(x, 1)
            w = torch.exp(x - lse[at:at + a, h][:, None])
            out[at:at + a, h] = torch.where(torch.isnan(w), 0.0, w) @ v[:, h // share]
        at += a
    return dict(out=out, lse=lse)
