"""Experts and adapters: binding of the grouped part of the C ABI (argument marshalling only).

    r = moe_route(logits, top_k)                                   # [T][E] router output
    h = linear_w4a16_grouped_gated_silu(X, gate_up, r.groups, fan=top_k)
    p = linear_w4a16_grouped(h, down, r.groups)
    y = moe_combine(p, r.weights, r.groups, add=residual)          # [T][N]

    y = linear_w4a16_lora(X, w, LoraAdapters(A, B, scale), ids)    # ids: adapter of each row

Every function checks that its tensors live on one GPU, have the expected dtype and shape
and are contiguous, launches on that GPU's current stream, allocates the outputs and
workspaces it is not given, and raises AwqError on a non-OK status. The contents of ids,
offsets and orders stay on the device and are not looked at here.
"""

from __future__ import annotations

import ctypes as C
import functools
from dataclasses import dataclass

import torch

from . import _abi
from .awq import GROUP, PackedLinear, alloc_packed, quantize_pack

MAX_GROUPS = 512  # AWQ_MAX_GROUPS

_GROUPED_KERNELS = {"auto": 0, "skinny": 1, "gemm64": 2, "gemm128": 3, "gemm256": 4, "gemm64k": 5}


def _check(t, dtype, shape, name, device):
    """The address of a tensor that is what the call needs; these run on every call of a
    decoding step, so what is right takes one pass and only a wrong tensor is looked at again."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device.index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _first(t, dtypes, dims, name):
    """Checks the tensor that fixes a call's device; returns that device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions")
    return t.device


def _flags(flags, device):
    return None if flags is None else _check(flags, torch.int32, (1,), "flags", device)


def _workspace(workspace, nbytes, device):
    """(pointer, bytes) of the caller's workspace, or of a new one on the current stream."""
    if nbytes == 0:
        return None, 0, None
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    else:
        if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8:
            raise TypeError("workspace must be a uint8 tensor")
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on {device}")
    return workspace.data_ptr(), workspace.numel(), workspace


def _stream_of(index):
    return torch.cuda.current_stream(index).cuda_stream


# The handle without a Stream object around it (0.1 us instead of 2.7, of the 8 that a call takes).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_of)


@functools.lru_cache(maxsize=None)
def _function(name):
    return getattr(_abi.load(), name)


def _launch(name, device, *args):
    """Calls an entry point on the device's current stream, whatever device is current."""
    fn = _function(name)
    index = device.index
    if torch.cuda.current_device() == index:
        status = fn(*args, _current_stream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _current_stream(index))
    if status:
        _abi.check(name, status)


@functools.lru_cache(maxsize=1024)
def _workspace_size(name, *sizes):
    return getattr(_abi.load(), name)(*sizes)


@functools.lru_cache(maxsize=None)
def _config(group: int, w_bit: int):
    return C.pointer(_abi.config(group_size=group, w_bit=w_bit))


# ------------------------------------------------------------------ routing and grouping

@dataclass
class RowGroups:
    """Rows of a batch in group order, on the device."""
    offsets: torch.Tensor  # int32 [groups + 1]: group e has positions [offsets[e], offsets[e + 1])
    order: torch.Tensor    # int32 [n]: the row at each position (rows without a group last)
    pos: torch.Tensor      # int32 [n]: the position of each row


@dataclass
class Routing:
    """The router's choices for T tokens; groups holds the T top_k (token, choice) pairs."""
    weights: torch.Tensor  # fp32 [T][top_k]
    ids: torch.Tensor      # int32 [T][top_k], -1: no expert
    groups: RowGroups


def _alloc_groups(n, groups, device):
    i32 = dict(dtype=torch.int32, device=device)
    return RowGroups(torch.empty(groups + 1, **i32), torch.empty(n, **i32), torch.empty(n, **i32))


def group_rows_workspace_size(n: int, n_groups: int) -> int:
    """Bytes of workspace (a uint8 tensor) that group_rows takes for n rows; 0: none."""
    return _workspace_size("awq_group_rows_workspace_size", n, n_groups)


def moe_route_workspace_size(T: int, E: int) -> int:
    """Bytes of workspace (a uint8 tensor) that moe_route takes for logits [T][E]; 0: none."""
    return _workspace_size("awq_moe_route_workspace_size", T, E)


def group_rows(ids: torch.Tensor, n_groups: int, out: RowGroups | None = None,
               workspace: torch.Tensor | None = None) -> RowGroups:
    """awq_group_rows: int32 ids [n] (outside [0, n_groups): no group) to the rows in group
    order, stable; rows without a group come last. workspace: group_rows_workspace_size bytes,
    one for each of the calls that overlap."""
    dev = _first(ids, (torch.int32,), 1, "ids")
    n = ids.shape[0]
    ip = _check(ids, torch.int32, (n,), "ids", dev)
    if out is None:
        out = _alloc_groups(n, max(n_groups, 0), dev)
    op = _check(out.offsets, torch.int32, (n_groups + 1,), "out.offsets", dev)
    rp = _check(out.order, torch.int32, (n,), "out.order", dev)
    pp = _check(out.pos, torch.int32, (n,), "out.pos", dev)
    wp, wn, _keep = _workspace(workspace, group_rows_workspace_size(n, n_groups), dev)
    _launch("awq_group_rows", dev, ip, n, n_groups, op, rp, pp, wp, wn)
    return out


def moe_route(logits: torch.Tensor, top_k: int, renormalize: bool = True, out: Routing | None = None,
              flags: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> Routing:
    """awq_moe_route: router logits [T][E] (fp16 or fp32; rows may be strided) to the top_k
    experts of each token, their softmax weights, and the pairs in expert order. workspace:
    moe_route_workspace_size bytes, one for each of the calls that overlap."""
    dev = _first(logits, (torch.float16, torch.float32), 2, "logits")
    T, E = logits.shape
    ld = logits.stride(0) if T > 1 else E
    if E > 1 and logits.stride(1) != 1 or ld < E:
        raise ValueError("logits must have contiguous rows that do not overlap")
    n = T * top_k
    if out is None:
        out = Routing(torch.empty((T, max(top_k, 0)), dtype=torch.float32, device=dev),
                      torch.empty((T, max(top_k, 0)), dtype=torch.int32, device=dev),
                      _alloc_groups(max(n, 0), E, dev))
    wtp = _check(out.weights, torch.float32, (T, top_k), "out.weights", dev)
    ip = _check(out.ids, torch.int32, (T, top_k), "out.ids", dev)
    op = _check(out.groups.offsets, torch.int32, (E + 1,), "out.groups.offsets", dev)
    rp = _check(out.groups.order, torch.int32, (n,), "out.groups.order", dev)
    pp = _check(out.groups.pos, torch.int32, (n,), "out.groups.pos", dev)
    wp, wn, _keep = _workspace(workspace, moe_route_workspace_size(T, E), dev)
    _launch("awq_moe_route", dev, logits.data_ptr(), 0 if logits.dtype == torch.float16 else 1, T, E, ld,
            top_k, int(bool(renormalize)), wtp, ip, op, rp, pp, wp, wn, _flags(flags, dev))
    return out


# ------------------------------------------------------------------ experts

@dataclass
class PackedExperts:
    """E packed weights of one [N][K] linear each, stacked (see PackedLinear)."""
    qweight: torch.Tensor  # int32 [E][N][K w_bit / 32]
    scales: torch.Tensor   # fp16 [E][N][G], G = K / group
    zeros: torch.Tensor    # uint8 [E][N][ceil(G/2)] (3/4-bit) or [E][N][G] (8-bit)
    E: int
    N: int
    K: int
    group: int = GROUP
    w_bit: int = 4

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.qweight, self.scales, self.zeros))

    def expert(self, e: int) -> PackedLinear:
        """Expert e as a PackedLinear (views; as arguments of the linears their addresses
        have to be 16-byte aligned, which odd N and few groups can miss)."""
        return PackedLinear(self.qweight[e], self.scales[e], self.zeros[e], self.N, self.K, self.group,
                            self.w_bit)


def quantize_pack_experts(W: torch.Tensor, s: torch.Tensor | None = None, zero_point: bool = True,
                          group_size: int = GROUP, w_bit: int = 4,
                          flags: torch.Tensor | None = None) -> PackedExperts:
    """awq_quantize_pack of E stacked weights W fp16 [E][N][K]; s (optional): the input
    channel scales, fp16 [K] for all experts or [E][K]."""
    dev = _first(W, (torch.float16,), 3, "W")
    E, N, K = W.shape
    _check(W, torch.float16, (E, N, K), "W", dev)
    each = isinstance(s, torch.Tensor) and s.dim() != 1
    if s is not None:
        _check(s, torch.float16, (E, K) if each else (K,), "s", dev)
    if flags is not None:
        _check(flags, torch.int32, getattr(flags, "shape", None), "flags", dev)
    with torch.cuda.device(dev):  # quantize_pack launches on the current device
        if each:
            parts = [quantize_pack(W[e], s[e], flags, zero_point=zero_point, group_size=group_size, w_bit=w_bit)
                     for e in range(E)]
            qweight, scales, zeros = (torch.stack(t) for t in zip(*((p.qweight, p.scales, p.zeros) for p in parts)))
        else:
            p = quantize_pack(W.view(E * N, K), s, flags, out=alloc_packed(E * N, K, dev, group_size, w_bit),
                              zero_point=zero_point, group_size=group_size, w_bit=w_bit)
            qweight, scales, zeros = (t.view(E, N, -1) for t in (p.qweight, p.scales, p.zeros))
    return PackedExperts(qweight, scales, zeros, E, N, K, group_size, w_bit)


def _packed(w, lead, device):
    G = w.K // w.group
    return (_check(w.qweight, torch.int32, (*lead, w.N, w.K * w.w_bit // 32), "qweight", device),
            _check(w.scales, torch.float16, (*lead, w.N, G), "scales", device),
            _check(w.zeros, torch.uint8, (*lead, w.N, G if w.w_bit == 8 else (G + 1) // 2), "zeros", device))


def _grouped(name, X, w, groups, fan, outs, out, flags, kernel):
    dev = _first(X, (torch.float16,), 2, "X")
    rows, K = X.shape
    if K != w.K:
        raise ValueError("X and the packed weights disagree on K")
    xp = _check(X, torch.float16, (rows, K), "X", dev)
    n = groups.order.shape[0]
    if fan is None:
        rp = None
        if rows != n:
            raise ValueError("X must have one row per position (or pass fan to gather them)")
    else:
        if fan < 1 or rows * fan != n:
            raise ValueError("fan times the rows of X must be the number of positions")
        rp = _check(groups.order, torch.int32, (n,), "groups.order", dev)
    op = _check(groups.offsets, torch.int32, (w.E + 1,), "groups.offsets", dev)
    qp, sp, zp = _packed(w, (w.E,), dev)
    if out is None:
        out = torch.empty((n, outs), dtype=torch.float16, device=dev)
    yp = _check(out, torch.float16, (n, outs), "out", dev)
    _launch(name, dev, xp, rows, op, rp, n, fan or 1, w.E, qp, sp, zp, w.N, K, _config(w.group, w.w_bit), yp,
            _flags(flags, dev), _GROUPED_KERNELS[kernel])
    return out


def linear_w4a16_grouped(X: torch.Tensor, w: PackedExperts, groups: RowGroups, fan: int | None = None,
                         out: torch.Tensor | None = None, flags: torch.Tensor | None = None,
                         kernel: str = "auto") -> torch.Tensor:
    """awq_linear_w4a16_grouped: every expert's linear on its rows, Y [n][N] in group order.
    X holds the rows in group order, or (fan = choices per token) one row per token, taken
    through groups.order. Rows without a group are left as they are in out; X in group order
    need not hold any there, and flags does not look at them."""
    return _grouped("awq_linear_w4a16_grouped", X, w, groups, fan, w.N, out, flags, kernel)


def linear_w4a16_grouped_gated_silu(X: torch.Tensor, w: PackedExperts, groups: RowGroups,
                                    fan: int | None = None, out: torch.Tensor | None = None,
                                    flags: torch.Tensor | None = None,
                                    kernel: str = "auto") -> torch.Tensor:
    """awq_linear_w4a16_grouped_gated_silu: SiLU(x W_gate^T) * (x W_up^T) of every expert's
    gate|up weight on its rows, Y [n][N/2] in group order; arguments as linear_w4a16_grouped."""
    if w.N % 2:
        raise ValueError("a gate|up weight has an even number of rows")
    return _grouped("awq_linear_w4a16_grouped_gated_silu", X, w, groups, fan, w.N // 2, out, flags, kernel)


def moe_combine(P: torch.Tensor, weights: torch.Tensor, groups: RowGroups, add: torch.Tensor | None = None,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """awq_moe_combine: Y[t] = add[t] + sum_j weights[t][j] P[pos of pair (t, j)], fp16 [T][N];
    pairs without an expert add nothing. out may be add."""
    dev = _first(P, (torch.float16,), 2, "P")
    if weights.dim() != 2:
        raise ValueError("weights must be [T][top_k]")
    T, k = weights.shape
    n, N = P.shape
    pp = _check(P, torch.float16, (T * k, N), "P", dev)
    wp = _check(weights, torch.float32, (T, k), "weights", dev)
    op = _check(groups.pos, torch.int32, (T * k,), "groups.pos", dev)
    fp = _check(groups.offsets, torch.int32, tuple(groups.offsets.shape[:1]), "groups.offsets", dev)
    ap = None if add is None else _check(add, torch.float16, (T, N), "add", dev)
    if out is None:
        out = torch.empty((T, N), dtype=torch.float16, device=dev)
    yp = _check(out, torch.float16, (T, N), "out", dev)
    _launch("awq_moe_combine", dev, pp, wp, op, fp, groups.offsets.shape[0] - 1, T, k, N, ap, yp)
    return out


# ------------------------------------------------------------------ adapters

@dataclass
class LoraAdapters:
    """Low-rank adapters of one [N][K] linear, stacked: W_a = W + scale[a] B_a A_a."""
    A: torch.Tensor      # fp16 [adapters][rank][K]
    B: torch.Tensor      # fp16 [adapters][N][rank]
    scale: torch.Tensor  # fp32 [adapters]


def linear_w4a16_lora_workspace_size(M: int, rank: int) -> int:
    """Bytes of workspace (a uint8 tensor) that linear_w4a16_lora takes for M rows."""
    return _workspace_size("awq_linear_w4a16_lora_workspace_size", M, rank)


def linear_w4a16_lora(X: torch.Tensor, w: PackedLinear, lora: LoraAdapters, ids: torch.Tensor,
                      groups: RowGroups | None = None, out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, flags: torch.Tensor | None = None,
                      kernel: str = "auto") -> torch.Tensor:
    """awq_linear_w4a16_lora: Y = X deq(W)^T + scale[a] (X A_a^T) B_a^T with a = ids[i] for
    row i (int32; outside [0, adapters): the linear alone). groups (group_rows(ids, adapters))
    brings the rows of an adapter together: worth it for large batches of mixed rows, kept
    by the caller over the layers of a step. workspace: linear_w4a16_lora_workspace_size
    bytes, one for each of the calls that overlap."""
    dev = _first(X, (torch.float16,), 2, "X")
    M, K = X.shape
    if K != w.K:
        raise ValueError("X and the packed weight disagree on K")
    if not isinstance(lora.A, torch.Tensor) or lora.A.dim() != 3:
        raise ValueError("lora.A must be [adapters][rank][K]")
    L, rank, _ = lora.A.shape
    xp = _check(X, torch.float16, (M, K), "X", dev)
    ap = _check(lora.A, torch.float16, (L, rank, K), "lora.A", dev)
    bp = _check(lora.B, torch.float16, (L, w.N, rank), "lora.B", dev)
    cp = _check(lora.scale, torch.float32, (L,), "lora.scale", dev)
    ip = _check(ids, torch.int32, (M,), "ids", dev)
    rp = None if groups is None else _check(groups.order, torch.int32, (M,), "groups.order", dev)
    qp, sp, zp = _packed(w, (), dev)
    if out is None:
        out = torch.empty((M, w.N), dtype=torch.float16, device=dev)
    yp = _check(out, torch.float16, (M, w.N), "out", dev)
    wp, wn, _keep = _workspace(workspace, linear_w4a16_lora_workspace_size(M, rank), dev)
    _launch("awq_linear_w4a16_lora", dev, xp, M, qp, sp, zp, w.N, K, _config(w.group, w.w_bit), ap, bp, cp, L,
            rank, ip, rp, yp, wp, wn, _flags(flags, dev), _GROUPED_KERNELS[kernel])
    return out
