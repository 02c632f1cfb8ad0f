"""The mixture-of-experts and adapter operators beside the packed linear, as measured cases.

Five kinds of case:

* ``route``   router logits to the chosen experts, their weights and the rows in expert order;
* ``group``   rows put in group order by their group ids (one adapter id per row);
* ``experts`` the products of a ragged batch in expert order with stacked packed weights,
              plain (down projection) or as the fused gate|up pair;
* ``combine`` the weighted sum that takes expert outputs back to token order;
* ``lora``    the packed linear with a low-rank adapter of its own for every row.

``run`` computes them in elementary torch operations in 32 bits, or, where ``own`` is set,
through the framework. ``exact`` computes them from their definitions in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
W_STD = 0.02           # weights ~ N(0, 0.02^2), as everywhere in this repository
OUTLIERS, GAIN = 0.01, 20.0  # 1% of the input channels are 20 times larger

# --------------------------------------------------------------------------- cases


def listed():
    return [
        # one token of a decoding step picks 8 of 64 experts: latency alone
        dict(name="route one token", kind="route", T=1, E=64, k=8, half=True, renorm=True, pad=0.0),
        # a prefill batch of odd length with padded rows, fp32 router output
        dict(name="route prefill", kind="route", T=8191, E=128, k=8, half=False, renorm=True, pad=0.05),
        # the rows of a prefill batch by the adapter of their request, some without one
        dict(name="group adapter rows", kind="group", n=2048, L=32, none=0.2),
        # one token: eight experts with one row each, gate|up of each streamed once
        dict(name="experts one token gated", kind="experts", gated=True, T=1, E=64, k=8, N=2048, K=2048,
             w_bit=4, group=128, gather=True, pad=0.0),
        # a decoding batch: a few rows on nearly every expert, down projection
        dict(name="experts decode batch", kind="experts", gated=False, T=48, E=64, k=8, N=4096, K=1024,
             w_bit=4, group=128, gather=False, pad=0.0),
        # a prefill batch on eight wide experts: matrix-core bound, the largest case
        dict(name="experts prefill gated", kind="experts", gated=True, T=4096, E=8, k=2, N=22016, K=4096,
             w_bit=4, group=128, gather=True, pad=0.0),
        # ragged prefill on many narrow experts, 8-bit codes in small groups, padded rows
        dict(name="experts prefill 8-bit", kind="experts", gated=False, T=1999, E=64, k=6, N=2048, K=1152,
             w_bit=8, group=64, gather=False, pad=0.03),
        # the end of a decoding step's block for a small batch
        dict(name="combine decode", kind="combine", T=16, k=8, N=4096, add=True, pad=0.0),
        # the same for a prefill batch
        dict(name="combine prefill", kind="combine", T=4096, k=8, N=4096, add=False, pad=0.02),
        # one token of one request with an adapter
        dict(name="lora one token", kind="lora", M=1, N=4096, K=4096, w_bit=4, group=128, L=8, r=16, none=0.0,
             runs=False),
        # a decoding batch: every row another request, adapters mixed at random
        dict(name="lora decode batch", kind="lora", M=48, N=11008, K=4096, w_bit=4, group=128, L=32, r=32,
             none=0.1, runs=False),
        # prefill: a few requests of different lengths, each with its adapter
        dict(name="lora prefill", kind="lora", M=2048, N=4096, K=4096, w_bit=4, group=128, L=16, r=16, none=0.1,
             runs=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST_FLOPS = 2.0 * 8192 * 22016 * 4096   # of the largest listed case
MOST_BYTES = 4.0e8
MOST_WEIGHTS = 8 * 22016 * 4096


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        if c["kind"] == "experts" and c["E"] * c["N"] * c["K"] > MOST_WEIGHTS:
            continue
        if w["flops"] <= MOST_FLOPS and w["bytes"] <= MOST_BYTES:
            return c


def _draw(rng):
    kind = rng.choice(["route", "group", "experts", "experts", "experts", "combine", "lora", "lora", "lora"])
    E = rng.choice([4, 8, 16, 32, 60, 64, 96, 128])
    k = rng.randint(1, min(8, E))
    pad = rng.choice([0.0, 0.0, 0.05, 0.3])
    bits = dict(w_bit=rng.choice([4, 4, 4, 8, 3]), group=rng.choice([128, 128, 64, 32]))
    if kind == "route":
        E = rng.choice([E, rng.randint(1, 256)])
        return dict(kind=kind, T=_log_int(rng, 1, 12000), E=E, k=rng.randint(1, min(8, E)), half=rng.random() < 0.5,
                    renorm=rng.random() < 0.6, pad=pad)
    if kind == "group":
        return dict(kind=kind, n=_log_int(rng, 1, 60000), L=_log_int(rng, 1, 500), none=rng.choice([0.0, 0.1, 0.5]))
    if kind == "combine":
        return dict(kind=kind, T=_log_int(rng, 1, 6000), k=k, N=_log_int(rng, 1, 8192), add=rng.random() < 0.5, pad=pad)
    if kind == "experts":
        gated = rng.random() < 0.5
        N = _log_int(rng, 2, 8192) if rng.random() < 0.5 else 128 * _log_int(rng, 1, 64)
        return dict(kind=kind, gated=gated, T=_log_int(rng, 1, 4096), E=E, k=k, N=N + N % 2 if gated else N,
                    K=128 * _log_int(rng, 1, 32), gather=rng.random() < 0.6, pad=pad, **bits)
    return dict(kind=kind, M=_log_int(rng, 1, 4096), N=_log_int(rng, 1, 12000) if rng.random() < 0.5 else 128 * _log_int(rng, 1, 64),
                K=128 * _log_int(rng, 1, 40), L=_log_int(rng, 1, 64), r=rng.choice([8, 16, 16, 24, 32, 64, 128]),
                none=rng.choice([0.0, 0.1, 0.5]), runs=rng.random() < 0.5, **bits)


# --------------------------------------------------------------------------- inputs

# Where the codes of a 128-channel block lie in its 32-bit words: per channel the word, the
# shift and the mask (3-bit codes: bits 0-1 in words 0-7, bit 2 in words 8-11).
_NIBBLE = [0, 4, 1, 5, 2, 6, 3, 7]


def _planes(w_bit):
    if w_bit == 4:
        return [([c // 8 for c in range(128)], [4 * _NIBBLE[c % 8] for c in range(128)], 15, 0)]
    if w_bit == 8:
        return [([c // 4 for c in range(128)], [8 * (c % 4) for c in range(128)], 255, 0)]
    return [([c // 16 for c in range(128)], [2 * (c % 16 // 2) + 16 * (c % 2) for c in range(128)], 3, 0),
            ([8 + c // 32 for c in range(128)], [c % 32 // 2 + 16 * (c % 2) for c in range(128)], 1, 2)]


def _tables(w_bit):
    """_planes with its lists on the device: (word, shift, mask, place of the bits)."""
    return [(torch.tensor(at, device=DEV), torch.tensor(shift, dtype=torch.int32, device=DEV), mask, up)
            for at, shift, mask, up in _planes(w_bit)]


def _pack(codes, w_bit):
    """Codes [rows][K] (int64) to the packed words int32 [rows][K w_bit / 32]."""
    rows, K = codes.shape
    words = torch.zeros(rows, K // 128, 4 * w_bit, dtype=torch.int64, device=codes.device)
    blocks = codes.view(rows, K // 128, 128)
    for at, shift, mask, up in _tables(w_bit):
        words.index_add_(2, at, ((blocks >> up) & mask) << shift.long())
    return words.to(torch.int32).view(rows, K * w_bit // 32)


def _packed_weight(gen, N, K, w_bit, group):
    """A weight of normal values in the packed format: codes, fp16 scales, zero points."""
    w = torch.randn(N, K // group, group, generator=gen, device=DEV) * W_STD
    lo, hi, top = w.amin(2), w.amax(2), 2 ** w_bit - 1
    scales = ((hi - lo) / top).clamp_min(2.0 ** -14).half()
    z = (-lo / scales.float()).round().clamp(0, top)
    codes = ((w / scales.float()[..., None]).round() + z[..., None]).clamp(0, top).to(torch.int64).view(N, K)
    z = z.to(torch.uint8)
    if w_bit != 8:
        z = torch.nn.functional.pad(z, (0, z.shape[1] % 2))
        z = z[:, 0::2] | (z[:, 1::2] << 4)
    return _pack(codes, w_bit), scales.contiguous(), z.contiguous()


def _activations(gen, rows, K):
    x = torch.randn(rows, K, generator=gen, device=DEV)
    x[:, torch.randperm(K, generator=gen, device=DEV)[:max(1, round(OUTLIERS * K))]] *= GAIN
    return x.half()


def _logits(gen, T, E, pad):
    """Router logits: some experts are liked more than others; padded rows hold -inf."""
    x = torch.randn(T, E, generator=gen, device=DEV) * 1.5 + torch.randn(E, generator=gen, device=DEV) * 0.5
    out = torch.rand(T, generator=gen, device=DEV) < pad
    return x.masked_fill(out[:, None], -math.inf)


def _grouped(ids, groups):
    """(offsets, order, pos) of group ids: rows in group order, those of no group last."""
    key = torch.where((ids < 0) | (ids >= groups), groups, ids).to(torch.int64)
    order = torch.sort(key, stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=order.device)
    count = torch.zeros(groups + 1, dtype=torch.int64, device=ids.device).index_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([count.new_zeros(1), count[:groups].cumsum(0)])
    return offsets.to(torch.int32), order.to(torch.int32), pos.to(torch.int32)


def _routed(gen, c):
    """The ids, weights and groups of a routed batch (for the operators behind the router)."""
    return _route(_logits(gen, c["T"], c["E"], c["pad"]), c["k"], True)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    i32 = dict(dtype=torch.int32, device=DEV)
    if c["kind"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        x = _logits(gen, T, E, c["pad"])
        return dict(case=c, logits=x.half() if c["half"] else x, weights=torch.empty(T, k, device=DEV),
                    ids=torch.empty(T, k, **i32), offsets=torch.empty(E + 1, **i32), order=torch.empty(T * k, **i32),
                    pos=torch.empty(T * k, **i32))
    if c["kind"] == "group":
        n = c["n"]
        ids = torch.randint(0, c["L"], (n,), generator=gen, device=DEV)
        ids[torch.rand(n, generator=gen, device=DEV) < c["none"]] = -1
        return dict(case=c, ids=ids.to(torch.int32), offsets=torch.empty(c["L"] + 1, **i32), order=torch.empty(n, **i32),
                    pos=torch.empty(n, **i32))
    if c["kind"] == "experts":
        r = _routed(gen, c)
        E, N, K, rows = c["E"], c["N"], c["K"], c["T"] * c["k"]
        x = _activations(gen, c["T"] if c["gather"] else rows, K)
        parts = [_packed_weight(gen, N, K, c["w_bit"], c["group"]) for _ in range(E)]
        qweight, scales, zeros = (torch.stack(p) for p in zip(*parts))
        sizes = (r["offsets"][1:] - r["offsets"][:-1]).tolist()
        return dict(case=c, x=x, qweight=qweight, scales=scales, zeros=zeros, tables=_tables(c["w_bit"]),
                    offsets=r["offsets"], order=r["order"], pos=r["pos"], most=max(sizes + [1]),
                    out=torch.zeros(rows, N // 2 if c["gated"] else N, dtype=torch.float16, device=DEV))
    if c["kind"] == "combine":
        r = _routed(gen, dict(c, E=max(16, c["k"])))
        y = (torch.randn(c["T"] * c["k"], c["N"], generator=gen, device=DEV) * 0.5).half()
        add = torch.randn(c["T"], c["N"], generator=gen, device=DEV).half() if c["add"] else None
        return dict(case=c, y=y, weights=r["weights"], offsets=r["offsets"], order=r["order"], pos=r["pos"], add=add,
                    out=torch.empty(c["T"], c["N"], dtype=torch.float16, device=DEV))
    M, N, K, L, rank = c["M"], c["N"], c["K"], c["L"], c["r"]
    ids = torch.randint(0, L, (M,), generator=gen, device=DEV)
    ids[torch.rand(M, generator=gen, device=DEV) < c["none"]] = -1
    if c["runs"]:  # the rows of one request are neighbours: six lengths
        cuts = torch.rand(5, generator=gen, device=DEV).mul(M).sort().values
        ids = ids[:6].repeat(6)[torch.searchsorted(cuts, torch.arange(M, device=DEV).float())]
    qweight, scales, zeros = _packed_weight(gen, N, K, c["w_bit"], c["group"])
    a = (torch.randn(L, rank, K, generator=gen, device=DEV) / math.sqrt(K)).half()
    b = (torch.randn(L, N, rank, generator=gen, device=DEV) * 0.05).half()
    scale = torch.rand(L, generator=gen, device=DEV) + 0.5
    offsets, order, pos = _grouped(ids, L)
    return dict(case=c, x=_activations(gen, M, K), qweight=qweight, scales=scales, zeros=zeros, a=a, b=b, scale=scale,
                tables=_tables(c["w_bit"]), ids=ids.to(torch.int32), offsets=offsets, order=order, pos=pos,
                out=torch.empty(M, N, dtype=torch.float16, device=DEV))


# --------------------------------------------------------------------------- the operators


def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own_run(state, kind)
    return _PLAIN[kind](state)


def _own_run(s, kind):
    import weight_only_bit_02_amd as awq

    c = s["case"]
    if kind == "route":
        r = awq.moe_route(s["logits"], c["k"], renormalize=c["renorm"],
                          out=awq.Routing(s["weights"], s["ids"], awq.RowGroups(s["offsets"], s["order"], s["pos"])))
        return dict(weights=r.weights, ids=r.ids, offsets=r.groups.offsets, order=r.groups.order, pos=r.groups.pos)
    if kind == "group":
        g = awq.group_rows(s["ids"], c["L"], out=awq.RowGroups(s["offsets"], s["order"], s["pos"]))
        return dict(offsets=g.offsets, order=g.order, pos=g.pos)
    groups = awq.RowGroups(s["offsets"], s["order"], s["pos"])
    if kind == "experts":
        w = awq.PackedExperts(s["qweight"], s["scales"], s["zeros"], c["E"], c["N"], c["K"], c["group"], c["w_bit"])
        f = awq.linear_w4a16_grouped_gated_silu if c["gated"] else awq.linear_w4a16_grouped
        return f(s["x"], w, groups, fan=c["k"] if c["gather"] else None, out=s["out"])
    if kind == "combine":
        return awq.moe_combine(s["y"], s["weights"], groups, add=s["add"], out=s["out"])
    w = awq.PackedLinear(s["qweight"], s["scales"], s["zeros"], c["N"], c["K"], c["group"], c["w_bit"])
    return awq.linear_w4a16_lora(s["x"], w, awq.LoraAdapters(s["a"], s["b"], s["scale"]), s["ids"], groups=groups,
                                 out=s["out"])


def _route(logits, k, renorm):
    x = logits.float()
    E = x.shape[1]
    best, ids = torch.sort(x, dim=1, descending=True, stable=True)
    top, ids = best[:, :k], ids[:, :k]
    some = torch.isfinite(best[:, :1])
    e = torch.exp(x - torch.where(some, best[:, :1], 0.0))
    chosen = torch.exp(top - torch.where(some, best[:, :1], 0.0))
    total = (chosen if renorm else e).sum(1, keepdim=True)
    weights = torch.where(some, chosen / torch.where(some, total, 1.0), 0.0)
    ids = torch.where(torch.isfinite(top), ids, -1).to(torch.int32)
    offsets, order, pos = _grouped(ids.reshape(-1), E)
    return dict(weights=weights, ids=ids, offsets=offsets, order=order, pos=pos)


def _plain_route(s):
    return _route(s["logits"], s["case"]["k"], s["case"]["renorm"])


def _plain_group(s):
    offsets, order, pos = _grouped(s["ids"], s["case"]["L"])
    return dict(offsets=offsets, order=order, pos=pos)


def _unpacked(s, which=slice(None)):
    """The dequantized weight (q - z) sc in fp32, [..., N, K] (exact in 24 bits)."""
    c, qweight, scales, zeros = s["case"], s["qweight"][which], s["scales"][which], s["zeros"][which]
    w_bit, group, K = c["w_bit"], c["group"], c["K"]
    words = qweight.view(*qweight.shape[:-1], K // 128, 4 * w_bit)
    codes = sum(((words[..., at] >> shift) & mask) << up for at, shift, mask, up in s["tables"])
    z = zeros if w_bit == 8 else torch.stack([zeros & 15, zeros >> 4], -1).flatten(-2)[..., :K // group]
    codes = codes.view(*qweight.shape[:-1], K // group, group)
    return ((codes - z[..., None].int()).float() * scales[..., None].float()).flatten(-2)


def _plain_experts(s):
    c, offsets = s["case"], s["offsets"].long()
    E, rows = c["E"], s["out"].shape[0]
    p = torch.arange(rows, device=offsets.device)
    e = torch.searchsorted(offsets, p, right=True) - 1
    inside = e < E
    e = e.clamp(max=E - 1)
    few = rows < E  # one product for each row with its expert's weight, else one for each expert
    most = 1 if few else s["most"]
    at = p[:, None] if few else offsets[:-1, None] + torch.arange(most, device=offsets.device)
    row = s["order"].long()[at.clamp(max=rows - 1)] // c["k"] if c["gather"] else at.clamp(max=rows - 1)
    w = _unpacked(s, e) if few else _unpacked(s)
    y = torch.bmm(s["x"].float()[row], w.transpose(1, 2).contiguous())
    if c["gated"]:
        g, u = y.chunk(2, dim=2)
        y = g / (1 + torch.exp(-g)) * u
    flat = p if few else e * most + (p - offsets[e]).clamp(max=most - 1)
    return torch.where(inside[:, None], y.flatten(0, 1)[flat], 0.0).half()


def _plain_combine(s):
    pos = s["pos"].view(s["case"]["T"], -1).long()
    w = torch.where(pos < s["offsets"][-1], s["weights"], 0.0)
    y = (s["y"].float()[pos] * w[..., None]).sum(1)
    return (y if s["add"] is None else y + s["add"].float()).half()


def _plain_lora(s):
    c = s["case"]
    x = s["x"].float()
    L, rank = c["L"], c["r"]
    y = x @ _unpacked(s).t()
    # every adapter's A on every row, all but the row's own masked, then every adapter's B
    h = (x @ s["a"].float().view(L * rank, -1).t()).view(-1, L, rank) * s["scale"][:, None]
    mine = s["ids"][:, None] == torch.arange(L, device=x.device)
    h = torch.where(mine[..., None], h, 0.0).flatten(1)
    return (y + h @ s["b"].float().transpose(1, 2).reshape(L * rank, -1)).half()


_PLAIN = dict(route=_plain_route, group=_plain_group, experts=_plain_experts, combine=_plain_combine, lora=_plain_lora)


# --------------------------------------------------------------------------- what each has to do


def _weight_bytes(c):
    return c["N"] * c["K"] * c["w_bit"] / 8 + c["N"] * (c["K"] // c["group"]) * (2 + (1 if c["w_bit"] == 8 else 0.5))


def work(case):
    c = case
    if c["kind"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return dict(bytes=T * E * (2 if c["half"] else 4) + T * k * 16 + 4 * (E + 1), flops=T * E * 3)
    if c["kind"] == "group":
        return dict(bytes=12 * c["n"] + 4 * (c["L"] + 1), flops=c["n"])
    if c["kind"] == "experts":
        rows = round(c["T"] * (1 - c["pad"])) * c["k"]
        active = c["E"] * (1 - (1 - c["k"] / c["E"]) ** max(1, round(c["T"] * (1 - c["pad"]))))  # experts with a row
        outs = c["N"] // 2 if c["gated"] else c["N"]
        x = (c["T"] if c["gather"] else rows) * c["K"]
        return dict(bytes=active * _weight_bytes(c) + 2 * (x + rows * outs), flops=2.0 * rows * c["N"] * c["K"])
    if c["kind"] == "combine":
        rows = c["T"] * c["k"] * (1 - c["pad"])
        return dict(bytes=2 * c["N"] * (rows + c["T"] * (2 if c["add"] else 1)) + 8 * c["T"] * c["k"],
                    flops=2.0 * rows * c["N"])
    rows = c["M"] * (1 - c["none"])
    used = min(6, c["L"]) if c["runs"] else c["L"] * (1 - (1 - 1 / c["L"]) ** rows)  # adapters with a row
    return dict(bytes=_weight_bytes(c) + 2 * c["M"] * (c["K"] + c["N"]) + 2 * used * c["r"] * (c["K"] + c["N"]),
                flops=2.0 * c["M"] * c["N"] * c["K"] + 2.0 * rows * c["r"] * (c["N"] + c["K"]))


# --------------------------------------------------------------------------- in 64 bits


def _rows64(c, qweight, scales, zeros):
    """One packed weight [N][K] from the definition of the format, channel by channel."""
    N, K, g = c["N"], c["K"], c["group"]
    w = torch.empty(N, K, dtype=torch.float64, device=DEV)
    q = qweight.to(torch.int64) & 0xFFFFFFFF
    for j in range(128):
        if c["w_bit"] == 4:
            code = q[:, j // 8::16] >> (4 * (j % 8 // 2 + 4 * (j % 2))) & 15
        elif c["w_bit"] == 8:
            code = q[:, j // 4::32] >> (8 * (j % 4)) & 255
        else:
            code = (q[:, j // 16::12] >> (2 * (j // 2 % 8) + 16 * (j % 2)) & 3) + (
                4 * (q[:, 8 + j // 32::12] >> (j // 2 % 16 + 16 * (j % 2)) & 1))
        w[:, j::128] = code.double()
    for i in range(K // g):
        z = zeros[:, i] if c["w_bit"] == 8 else (zeros[:, i // 2] >> (4 * (i % 2))) & 15
        w[:, i * g:(i + 1) * g] = (w[:, i * g:(i + 1) * g] - z.double()[:, None]) * scales[:, i].double()[:, None]
    return w


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "group":
        return None  # whole numbers
    if c["kind"] == "route":
        x = s["logits"].double()
        live = torch.isfinite(x).any(1)
        p = torch.zeros_like(x)
        p[live] = torch.softmax(x[live], 1)
        chosen = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :c["k"]]
        w = p.gather(1, chosen)
        if c["renorm"]:
            w[live] /= w[live].sum(1, keepdim=True)
        return dict(weights=w, ids=None, offsets=None, order=None, pos=None)
    if c["kind"] == "experts":
        y = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        at = s["offsets"].tolist()
        for e in range(c["E"]):
            if at[e] == at[e + 1]:
                continue
            p = torch.arange(at[e], at[e + 1], device=DEV)
            x = s["x"][s["order"][p].long() // c["k"]] if c["gather"] else s["x"][p]
            t = x.double() @ _rows64(c, s["qweight"][e], s["scales"][e], s["zeros"][e]).t()
            if c["gated"]:
                t = t[:, :c["N"] // 2] * torch.sigmoid(t[:, :c["N"] // 2]) * t[:, c["N"] // 2:]
            y[p] = t
        return y
    if c["kind"] == "combine":
        y = torch.zeros(c["T"], c["N"], dtype=torch.float64, device=DEV) if s["add"] is None else s["add"].double()
        last = s["offsets"][-1]
        for j in range(c["k"]):
            p = s["pos"].view(-1, c["k"])[:, j].long()
            y = y + s["y"][p].double() * (s["weights"][:, j].double() * (p < last))[:, None]
        return y
    x = s["x"].double()
    y = x @ _rows64(c, s["qweight"], s["scales"], s["zeros"]).t()
    for a in range(c["L"]):
        m = (s["ids"] == a).nonzero()[:, 0]
        if m.numel():
            y[m] += float(s["scale"][a]) * (x[m] @ s["a"][a].double().t()) @ s["b"][a].double().t()
    return y
