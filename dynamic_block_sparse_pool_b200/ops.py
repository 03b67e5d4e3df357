"""PyTorch-facing calls of libdsa.

PyTorch supplies device memory and the current CUDA stream; every step of
the computation runs in libdsa's kernels.  Tensors are [B, H, N, D],
contiguous, bf16 or fp32, on one CUDA device.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import NamedTuple, Optional, Tuple

import torch

from . import _lib
from ._lib import check, lib

Csr = Tuple[torch.Tensor, torch.Tensor]


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(t: torch.Tensor):
    # the handle alone: a Stream object costs 2 us, as much as a launch
    return torch._C._cuda_getCurrentRawStream(t.device.index)


_HERE = contextlib.nullcontext()


def _on(t: torch.Tensor):
    """t's device as the current one."""
    return _HERE if t.device.index == torch._C._cuda_getDevice() else torch.cuda.device(t.device)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return _lib.DSA_BF16
    if t.dtype == torch.float32:
        return _lib.DSA_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _check_qkv(*ts: torch.Tensor):
    t0 = ts[0]
    if t0.dim() != 4:
        raise ValueError("expected [B, H, N, D] tensors")
    for t in ts:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")
        if t.shape != t0.shape or t.dtype != t0.dtype or t.device != t0.device:
            raise ValueError("q, k, v must share shape, dtype and device")
    return t0.shape


def _check_csr(csr: Optional[Csr], rows: int):
    if csr is None:
        return None, None
    rp, col = csr
    for t in (rp, col):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("CSR tensors must be contiguous int32 CUDA tensors")
    if rp.numel() != rows + 1:
        raise ValueError(f"row_ptr must have {rows + 1} entries, got {rp.numel()}")
    return rp, col


def n_blocks(N: int, block: int) -> int:
    return (N + block - 1) // block


def workspace_size(op: int, B: int, H: int, N: int, D: int, block: int) -> int:
    return int(lib().dsa_workspace_size(op, B, H, N, D, block))


def pool_score(q: torch.Tensor, k: torch.Tensor, block: int, scale: Optional[float] = None,
               cand: Optional[Csr] = None, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """P [B*H, nB, nB] fp32: row softmax of scale * (block means of Q).(block means of K)."""
    B, H, N, D = _check_qkv(q, k)
    nB = n_blocks(N, block)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    crp, ccol = _check_csr(cand, B * H * nB)
    if out is None:
        out = torch.empty(B * H, nB, nB, device=q.device, dtype=torch.float32)
    ws_bytes = workspace_size(_lib.DSA_OP_POOL_SCORE, B, H, N, D, block)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), device=q.device, dtype=torch.uint8)
    st = lib().dsa_pool_score(q.data_ptr(), k.data_ptr(), _dtype_code(q), B, H, N, D, block,
                              scale, _ptr(crp), _ptr(ccol), out.data_ptr(), workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(), _stream(q))
    check(st, "dsa_pool_score")
    return out


def pool_score_hier(q: torch.Tensor, k: torch.Tensor, block: int, sub: int,
                    scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """P [B*H, nB, nB] fp32: the two-level estimate (pooled scores over
    sub-blocks of block/sub rows, folded back into block rows); sub = 1 is
    pool_score's P."""
    B, H, N, D = _check_qkv(q, k)
    nB = n_blocks(N, block)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        out = torch.empty(B * H, nB, nB, device=q.device, dtype=torch.float32)
    op = _lib.DSA_OP_POOL_SCORE_HIER4 if sub == 4 else _lib.DSA_OP_POOL_SCORE_HIER2
    ws_bytes = workspace_size(op, B, H, N, D, block)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), device=q.device, dtype=torch.uint8)
    st = lib().dsa_pool_score_hier(q.data_ptr(), k.data_ptr(), _dtype_code(q), B, H, N, D, block,
                                   sub, scale, out.data_ptr(), workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(), _stream(q))
    check(st, "dsa_pool_score_hier")
    return out


def select_topp(probs: torch.Tensor, p: float, cand: Optional[Csr] = None,
                row_ptr: Optional[torch.Tensor] = None, col_idx: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None) -> Csr:
    """CSR (row_ptr [rows+1], col_idx [capacity rows*nB]) of the Top-p block sets."""
    if probs.dtype != torch.float32 or not probs.is_cuda or not probs.is_contiguous():
        raise ValueError("probs must be a contiguous fp32 CUDA tensor")
    nB = probs.shape[-1]
    rows = probs.numel() // nB
    crp, ccol = _check_csr(cand, rows)
    dev = probs.device
    if row_ptr is None:
        row_ptr = torch.empty(rows + 1, device=dev, dtype=torch.int32)
    if col_idx is None:
        col_idx = torch.empty(rows * nB, device=dev, dtype=torch.int32)
    ws_bytes = rows * 33 * 4
    if workspace is None:
        workspace = torch.empty(ws_bytes, device=dev, dtype=torch.uint8)
    st = lib().dsa_select_topp(probs.data_ptr(), rows, nB, float(p), _ptr(crp), _ptr(ccol),
                               row_ptr.data_ptr(), col_idx.data_ptr(), workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), _stream(probs))
    check(st, "dsa_select_topp")
    return row_ptr, col_idx


def row_order(row_ptr: torch.Tensor, B: int, H: int, nB: int,
              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """int32 [B*H*nB]: each head's rows by descending block count (ties by
    row index), as global row indices; the order attn_fwd takes them in."""
    rows = B * H * nB
    if (row_ptr.dtype != torch.int32 or not row_ptr.is_cuda or not row_ptr.is_contiguous()
            or row_ptr.numel() != rows + 1):
        raise ValueError("row_ptr must be a contiguous int32 CUDA tensor of B*H*nB + 1 entries")
    if out is None:
        out = torch.empty(rows, device=row_ptr.device, dtype=torch.int32)
    elif (out.dtype != torch.int32 or out.device != row_ptr.device or not out.is_contiguous()
          or out.numel() != rows):
        raise ValueError("out must be a contiguous int32 tensor of B*H*nB entries on row_ptr's device")
    st = lib().dsa_row_order(row_ptr.data_ptr(), B, H, nB, out.data_ptr(), _stream(row_ptr))
    check(st, "dsa_row_order")
    return out


def attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, row_ptr: torch.Tensor,
             col_idx: torch.Tensor, block: int, scale: Optional[float] = None,
             out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
             blk_lse: Optional[torch.Tensor] = None, want_lse: bool = True,
             want_blk_lse: bool = True, order: Optional[torch.Tensor] = None):
    """(O [B,H,N,D], lse [B,H,N] or None, blk_lse [nnz, block] or None).

    Without `order` this is dsa_attn_fwd (rows in index order); with it,
    dsa_attn_fwd_ordered: `order` (row_order's output) is the order in which
    the persistent CTAs take the rows, and changes no output.  When blk_lse
    is wanted but not given, nnz is read from row_ptr (one device-to-host
    copy)."""
    B, H, N, D = _check_qkv(q, k, v)
    nB = n_blocks(N, block)
    _check_csr((row_ptr, col_idx), B * H * nB)
    if order is not None and (order.dtype != torch.int32 or order.device != q.device
                              or not order.is_contiguous() or order.numel() != B * H * nB):
        raise ValueError("order must be a contiguous int32 tensor of B*H*nB entries on q's device")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    if want_lse and lse is None:
        lse = torch.empty(B, H, N, device=q.device, dtype=torch.float32)
    if want_blk_lse and blk_lse is None:
        nnz = int(row_ptr[-1].item())
        blk_lse = torch.empty(max(nnz, 1), block, device=q.device, dtype=torch.float32)
    if order is None:
        st = lib().dsa_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype_code(q), B, H, N,
                                D, block, scale, row_ptr.data_ptr(), col_idx.data_ptr(),
                                out.data_ptr(), _ptr(lse), _ptr(blk_lse), _stream(q))
        check(st, "dsa_attn_fwd")
    else:
        st = lib().dsa_attn_fwd_ordered(q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype_code(q), B,
                                        H, N, D, block, scale, row_ptr.data_ptr(),
                                        col_idx.data_ptr(), order.data_ptr(), out.data_ptr(),
                                        _ptr(lse), _ptr(blk_lse), _stream(q))
        check(st, "dsa_attn_fwd_ordered")
    return out, lse, blk_lse


def attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
             dout: torch.Tensor, lse: torch.Tensor, row_ptr: torch.Tensor, col_idx: torch.Tensor,
             block: int, scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None):
    """(dQ, dK, dV) [B, H, N, D] of attn_fwd's O for a fixed mask, given dO.

    bf16 with block 128 runs on the tensor cores (P and dS as bf16 hi + lo
    terms); fp32 and block 64 in exact fp32 on CUDA cores."""
    B, H, N, D = _check_qkv(q, k, v)
    for t in (out, dout):
        if t.shape != q.shape or t.dtype != q.dtype or not t.is_contiguous():
            raise ValueError("out and dout must match q")
    nB = n_blocks(N, block)
    _check_csr((row_ptr, col_idx), B * H * nB)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    ws_bytes = workspace_size(_lib.DSA_OP_ATTN_BWD, B, H, N, D, block)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), device=q.device, dtype=torch.uint8)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    st = lib().dsa_attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                            dout.data_ptr(), lse.data_ptr(), _dtype_code(q), B, H, N, D, block,
                            scale, row_ptr.data_ptr(), col_idx.data_ptr(), dq.data_ptr(),
                            dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(),
                            workspace.numel() * workspace.element_size(), _stream(q))
    check(st, "dsa_attn_bwd")
    return dq, dk, dv


def block_mass(lse: torch.Tensor, blk_lse: torch.Tensor, row_ptr: torch.Tensor, block: int,
               mass: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mass [nnz] (capacity blk_lse.shape[0]): exact softmax mass of each selected block."""
    B, H, N = lse.shape
    if mass is None:
        mass = torch.empty(blk_lse.shape[0], device=lse.device, dtype=torch.float32)
    st = lib().dsa_block_mass(lse.data_ptr(), blk_lse.data_ptr(), B, H, N, block,
                              row_ptr.data_ptr(), mass.data_ptr(), _stream(lse))
    check(st, "dsa_block_mass")
    return mass


def mass_to_probs(row_ptr: torch.Tensor, col_idx: torch.Tensor, mass: torch.Tensor, nB: int,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """probs [rows, nB] fp32: each row's exact block masses at their columns, 0 elsewhere."""
    rows = row_ptr.numel() - 1
    _check_csr((row_ptr, col_idx), rows)
    if mass.dtype != torch.float32 or not mass.is_cuda:
        raise ValueError("mass must be an fp32 CUDA tensor")
    if out is None:
        out = torch.empty(rows, nB, device=mass.device, dtype=torch.float32)
    st = lib().dsa_mass_to_probs(row_ptr.data_ptr(), col_idx.data_ptr(), mass.data_ptr(), rows, nB,
                                 out.data_ptr(), _stream(mass))
    check(st, "dsa_mass_to_probs")
    return out


def hilbert_order(T: int, H: int, W: int, n_prefix: int = 0) -> torch.Tensor:
    """Host int32 [n_prefix + T*H*W]: perm[i] = original index of the token at
    position i along the 3-D Hilbert curve (text prefix first)."""
    perm = torch.empty(n_prefix + T * H * W, dtype=torch.int32)
    check(lib().dsa_hilbert_order(T, H, W, n_prefix, perm.data_ptr()), "dsa_hilbert_order")
    return perm


def gilbert_order(T: int, H: int, W: int, n_prefix: int = 0) -> torch.Tensor:
    """Host int32 [n_prefix + T*H*W]: perm[i] = original index of the token at
    position i along the generalised Hilbert curve of the T x H x W grid
    (consecutive grid tokens are grid neighbours; text prefix first)."""
    perm = torch.empty(n_prefix + T * H * W, dtype=torch.int32)
    check(lib().dsa_gilbert_order(T, H, W, n_prefix, perm.data_ptr()), "dsa_gilbert_order")
    return perm


def permute_tokens(x: torch.Tensor, perm: torch.Tensor, inverse: bool = False,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gather (dst[i] = src[perm[i]]) or scatter (dst[perm[i]] = src[i]) of the
    token rows of x [B, H, N, D]; perm: device int32 [N]."""
    if x.dim() != 4 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA tensor [B, H, N, D]")
    B, H, N, D = x.shape
    if perm.dtype != torch.int32 or not perm.is_cuda or perm.numel() != N:
        raise ValueError("perm must be a device int32 tensor of N entries")
    if out is None:
        out = torch.empty_like(x)
    st = lib().dsa_permute_tokens(x.data_ptr(), out.data_ptr(), _dtype_code(x), B, H, N, D,
                                  perm.data_ptr(), 1 if inverse else 0, _stream(x))
    check(st, "dsa_permute_tokens")
    return out


class HilbertOrder:
    """The Hilbert token order of one grid, kept on the device.  curve:
    "hilbert" (the enclosing power-of-two cube's curve, restricted to the
    grid) or "gilbert" (the curve generalised to the grid's own box)."""

    def __init__(self, T: int, H: int, W: int, n_prefix: int = 0, device=None,
                 curve: str = "hilbert"):
        if curve not in ("hilbert", "gilbert"):
            raise ValueError(f"unknown curve {curve!r}")
        self.host = (hilbert_order if curve == "hilbert" else gilbert_order)(T, H, W, n_prefix)
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None \
            else torch.device(device)
        self.perm = self.host.to(dev)

    def gather(self, x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        return permute_tokens(x, self.perm, False, out)

    def scatter(self, x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        return permute_tokens(x, self.perm, True, out)


# ------------------------------------------------- around the attention --

def _check_workspace(ws: torch.Tensor, t: torch.Tensor) -> None:
    if ws.device != t.device or not ws.is_contiguous():
        raise ValueError("the workspace must be contiguous and on the tensors' device")


def _int32(what: str, v) -> int:
    v = int(v)
    if not -2**31 <= v < 2**31:  # ctypes would take the low 32 bits
        raise ValueError(f"{what} = {v} does not fit in 32 bits")
    return v


class Act8(NamedTuple):
    """Activation rows of D values in 8 bits: the value held is code * scale."""

    codes: torch.Tensor        # int8 [..., D]
    scales: torch.Tensor       # fp32 [...]


def _check_act8(a: Act8) -> None:
    c, s = a
    if c.dtype != torch.int8 or s.dtype != torch.float32 or not c.is_cuda or s.device != c.device:
        raise ValueError("8-bit rows are int8 codes and fp32 scales on one CUDA device")
    if not c.is_contiguous() or not s.is_contiguous() or c.shape[:-1] != s.shape:
        raise ValueError("codes [..., D] and scales [...] must be contiguous and match")


def pack8(x: torch.Tensor) -> Act8:
    """The rows of x [..., D] (contiguous, bf16 or fp32) in 8 bits: one scale
    amax / 127 for each row, half-even rounding."""
    if not x.is_cuda or not x.is_contiguous() or x.dim() < 1:
        raise ValueError("x must be a contiguous CUDA tensor [..., D]")
    dt, shape, n = _dtype_code(x), x.shape, x.numel()
    D = shape[-1]
    codes, scales = x.new_empty(shape, dtype=torch.int8), x.new_empty(shape[:-1], dtype=torch.float32)
    if n > 0:
        with _on(x):
            st = lib().dsa_pack8(x.data_ptr(), dt, n // D, D, codes.data_ptr(), scales.data_ptr(), _stream(x))
        check(st, "dsa_pack8")
    return Act8(codes, scales)


def unpack8(a: Act8, dtype: torch.dtype = torch.bfloat16,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values that 8-bit rows stand for, as bf16 or fp32."""
    _check_act8(a)
    codes, scales = a
    if out is None:
        out = codes.new_empty(codes.shape, dtype=dtype)
    elif out.shape != codes.shape or out.device != codes.device or not out.is_contiguous():
        raise ValueError("out must be contiguous, of the codes' shape and device")
    dt, n, D = _dtype_code(out), codes.numel(), codes.shape[-1]
    if n > 0:
        with _on(out):
            st = lib().dsa_unpack8(codes.data_ptr(), scales.data_ptr(), dt, n // D, D, out.data_ptr(), _stream(out))
        check(st, "dsa_unpack8")
    return out


def rope_table(positions: int, pairs: int, theta: float = 10000.0, device=None) -> torch.Tensor:
    """fp32 [positions, pairs, 2] on the device: cos and sin of p * theta^(-i / pairs)."""
    positions, pairs = _int32("positions", positions), _int32("pairs", pairs)
    if positions < 1 or pairs < 1:
        raise ValueError("positions and pairs must be at least 1")
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if dev.type != "cuda":
        raise ValueError(f"the rotation tables live on a CUDA device, not on {dev}")
    t = torch.empty(positions, pairs, 2, dtype=torch.float32, device=dev)
    with _on(t):
        st = lib().dsa_rope_table_f64(positions, pairs, ctypes.byref(ctypes.c_double(theta)), t.data_ptr(), _stream(t))
    check(st, "dsa_rope_table_f64")
    return t


class RopePlan:
    """Positions and rotation tables of the tokens of one layout, on the device.

    pos     [N, axes] or [B, N, axes] integers, up to three axes (a grid's
            t, y, x, or one axis of plain positions); below 0: the axis'
            pairs of that token do not turn.
    pairs   rotated pairs of each axis, in the order of the pairs of a row;
            at most D/2 in all, the rest do not turn.
    theta   base of the frequencies, one for all axes or one for each.
    halves  False: pair m is elements (2m, 2m+1); True: (m, m + D/2).
    lengths positions that each axis' table covers (default: those in pos)."""

    def __init__(self, pos: torch.Tensor, pairs, theta=10000.0, halves: bool = False,
                 lengths=None, device=None):
        pairs = [int(p) for p in pairs]
        if not 1 <= len(pairs) <= 3 or min(pairs) < 0 or max(pairs) < 1:
            raise ValueError("pairs: one to three axes, at least one of them with a pair")
        thetas = list(theta) if isinstance(theta, (tuple, list)) else [theta] * len(pairs)
        if len(thetas) != len(pairs) or (lengths is not None and len(lengths) != len(pairs)):
            raise ValueError("theta and lengths must match the axes of pairs")
        dev = device if device is not None else pos.device if pos.is_cuda else \
            torch.device("cuda", torch.cuda.current_device())
        if lengths is None:
            flat = pos.reshape(-1, pos.shape[-1])
            top = flat.amax(0).tolist() if flat.numel() else [0] * flat.shape[-1]
            lengths = [max(int(t), 0) + 1 for t in top[:len(pairs)]]
            lengths += [1] * (len(pairs) - len(lengths))
        self.pairs = tuple(pairs + [0] * (3 - len(pairs)))
        self.lengths = tuple([int(n) for n in lengths] + [1] * (3 - len(pairs)))
        self.halves = bool(halves)
        self.table = torch.cat([rope_table(n, p, t, dev).reshape(-1, 2) for n, p, t in
                                zip(self.lengths, pairs, thetas) if p])
        self._axes = (ctypes.c_int32 * 6)(*self.pairs, *self.lengths)
        self.pos = self._positions(pos, dev)

    @staticmethod
    def _positions(pos: torch.Tensor, dev) -> torch.Tensor:
        if pos.dim() not in (2, 3) or not 1 <= pos.shape[-1] <= 3 or pos.is_floating_point():
            raise ValueError("pos must be integers [N, axes] or [B, N, axes], up to three axes")
        if pos.dtype == torch.int64:  # what 32 bits cannot hold stays past every table
            pos = pos.clamp(-1, 2**31 - 1)
        pos = pos.to(device=dev, dtype=torch.int32)
        if pos.shape[-1] < 3:
            pos = torch.nn.functional.pad(pos, (0, 3 - pos.shape[-1]), value=-1)
        return (pos if pos.dim() == 3 else pos[None]).contiguous()

    @classmethod
    def grid(cls, T: int, H: int, W: int, head_dim: int, n_prefix: int = 0, pairs=None,
             theta=10000.0, halves: bool = False, order: Optional[torch.Tensor] = None, t0: int = 0,
             device=None) -> "RopePlan":
        """The tokens of a T x H x W grid in row-major (t, y, x) order, behind
        n_prefix text tokens that do not turn; `order` (hilbert_order's or
        gilbert_order's perm) lists them in that order instead, t0 is the
        first frame's position.  By default the axes share the D/2 pairs
        evenly, the t axis taking what is left over."""
        if pairs is None:
            third = head_dim // 2 // 3
            pairs = (head_dim // 2 - 2 * third, third, third)
        t, y, x = torch.meshgrid(torch.arange(T), torch.arange(H), torch.arange(W), indexing="ij")
        pos = torch.full((n_prefix + T * H * W, 3), -1, dtype=torch.int32)
        pos[n_prefix:] = torch.stack([t.reshape(-1) + t0, y.reshape(-1), x.reshape(-1)], 1).int()
        if order is not None:
            pos = pos[order.cpu().long()]
        return cls(pos, pairs, theta, halves, device=device)

    def at(self, pos: torch.Tensor) -> "RopePlan":
        """The same tables for other tokens: pos as in the constructor, within
        the tables' lengths (a position past them is reported by
        device_status and does not turn)."""
        new = object.__new__(RopePlan)
        new.__dict__.update(self.__dict__)
        new.pos = self._positions(pos, self.table.device)
        return new


def _token_rows(x: torch.Tensor, what: str):
    """Strides of b, n, h of token-major rows [B, N, H, D], D contiguous."""
    n, st = x.shape, x.stride()
    if len(n) != 4 or not x.is_cuda or (n[3] > 1 and st[3] != 1):
        raise ValueError(f"{what} must be a CUDA tensor [B, N, H, D] with contiguous rows")
    return _strides3(n, st)


def _strides3(n, st):
    return st[0] if n[0] > 1 else 0, st[1] if n[1] > 1 else 0, st[2] if n[2] > 1 else 0


_Int64x6 = ctypes.c_int64 * 6


def _strides6(a, b):
    return _Int64x6(*a, *b)


def _check_norm_rope(xq, xk, wq, wk, plan: RopePlan):
    """(q data, k data, q scales, k scales, B, N, Hq, Hk, D) of either kind of x."""
    if isinstance(xq, Act8) != isinstance(xk, Act8):
        raise ValueError("xq and xk must both be tensors or both be 8-bit rows")
    sq = sk = None
    if isinstance(xq, Act8):
        _check_act8(xq)
        _check_act8(xk)
        (xq, sq), (xk, sk) = xq, xk
    if xq.dim() != 4 or xk.dim() != 4 or xq.dtype != xk.dtype or xq.device != xk.device:
        raise ValueError("xq and xk must be [B, N, H, D] of one dtype on one device")
    B, N, Hq, D = xq.shape
    if xk.shape[0] != B or xk.shape[1] != N or xk.shape[3] != D:
        raise ValueError("xq and xk must share B, N and D")
    for w in (wq, wk):
        if w is not None and (w.dtype != torch.float32 or w.device != xq.device or w.numel() != D
                              or not w.is_contiguous()):
            raise ValueError("weights must be contiguous fp32 [D] on x's device")
    if plan.pos.device != xq.device or plan.pos.shape[1] != N or plan.pos.shape[0] not in (1, B):
        raise ValueError(f"the plan's positions {tuple(plan.pos.shape)} do not fit B = {B}, N = {N} on x's device")
    return xq, xk, sq, sk, B, N, Hq, xk.shape[2], D


def qk_norm_rope(xq, xk, wq: Optional[torch.Tensor], wk: Optional[torch.Tensor], plan: RopePlan,
                 eps: float = 1e-6, save8: bool = False, dtype: torch.dtype = torch.bfloat16):
    """(q, k) [B, H, N, D]: each head's row of xq, xk [B, N, H, D] normalised
    by its root mean square, times wq or wk [D] (fp32, None: ones), turned by
    its token's position.

    xq and xk may be strided views (the fused projection's output), or Act8
    rows that an earlier call saved (q and k then come in `dtype`).  save8:
    also returns the rows of xq and xk in 8 bits, (q, k, xq8, xk8)."""
    dx, dk, sq, sk, B, N, Hq, Hk, D = _check_norm_rope(xq, xk, wq, wk, plan)
    from8 = sq is not None
    if save8 and from8:
        raise ValueError("save8: xq and xk already are 8-bit rows")
    dt = dtype if from8 else dx.dtype
    q = dx.new_empty((B, Hq, N, D), dtype=dt)
    k = dx.new_empty((B, Hk, N, D), dtype=dt)
    code = _dtype_code(q)
    st6 = _strides6(_token_rows(dx, "xq"), _token_rows(dk, "xk"))
    q8 = k8 = Act8(None, None)
    if save8:
        q8, k8 = (Act8(dx.new_empty((B, N, h, D), dtype=torch.int8),
                       dx.new_empty((B, N, h), dtype=torch.float32)) for h in (Hq, Hk))
    if B * N > 0:
        with _on(dx):
            st = lib().dsa_qk_norm_rope(
                dx.data_ptr(), dk.data_ptr(), _ptr(sq), _ptr(sk), st6, code, B, N, Hq, Hk, D,
                _ptr(wq), _ptr(wk), float(eps), plan.table.data_ptr(), plan.pos.data_ptr(),
                1 if plan.pos.shape[0] > 1 else 0, plan._axes, int(plan.halves), q.data_ptr(),
                k.data_ptr(), _ptr(q8.codes), _ptr(q8.scales), _ptr(k8.codes), _ptr(k8.scales),
                _stream(dx))
        check(st, "dsa_qk_norm_rope")
    return (q, k, q8, k8) if save8 else (q, k)


def qk_norm_rope_bwd(dq: torch.Tensor, dk: torch.Tensor, xq, xk, wq: Optional[torch.Tensor],
                     wk: Optional[torch.Tensor], plan: RopePlan, eps: float = 1e-6,
                     dxq: Optional[torch.Tensor] = None, dxk: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None):
    """(dxq, dxk [B, N, H, D], dwq, dwk fp32 [D]): qk_norm_rope's gradients for
    dq, dk [B, H, N, D].  xq, xk as the forward took them, or the Act8 rows it
    saved.  dxq and dxk may be given, strided views of a fused buffer among
    them."""
    vq, vk, sq, sk, B, N, Hq, Hk, D = _check_norm_rope(xq, xk, wq, wk, plan)
    for g, h in ((dq, Hq), (dk, Hk)):
        if tuple(g.shape) != (B, h, N, D) or not g.is_contiguous() or g.device != vq.device or \
                g.dtype != dq.dtype:
            raise ValueError("dq and dk must be contiguous [B, H, N, D] of one dtype on x's device")
    if sq is None and vq.dtype != dq.dtype:
        raise ValueError("dq and dk must have x's dtype")
    code = _dtype_code(dq)
    outs = []
    for d, h in ((dxq, Hq), (dxk, Hk)):
        if d is None:
            d = dq.new_empty((B, N, h, D))
        elif tuple(d.shape) != (B, N, h, D) or d.dtype != dq.dtype or d.device != dq.device:
            raise ValueError("dxq and dxk must be [B, N, H, D] of dq's dtype and device")
        elif any(d.shape[i] > 1 and d.stride(i) == 0 for i in range(3)):
            raise ValueError("rows of dxq and dxk must not overlap")
        outs.append(d)
    dxq, dxk = outs
    st6 = _strides6(_token_rows(vq, "xq"), _token_rows(vk, "xk"))
    dst6 = _strides6(_token_rows(dxq, "dxq"), _token_rows(dxk, "dxk"))
    dwq, dwk = dq.new_empty(D, dtype=torch.float32), dq.new_empty(D, dtype=torch.float32)
    if B * N == 0:
        return dxq, dxk, dwq.zero_(), dwk.zero_()
    if workspace is None:
        workspace = dq.new_empty(int(lib().dsa_qk_norm_rope_bwd_workspace_size(D)), dtype=torch.uint8)
    _check_workspace(workspace, dq)
    with _on(dq):
        st = lib().dsa_qk_norm_rope_bwd(
            dq.data_ptr(), dk.data_ptr(), vq.data_ptr(), vk.data_ptr(), _ptr(sq), _ptr(sk), st6,
            code, B, N, Hq, Hk, D, _ptr(wq), _ptr(wk), float(eps), plan.table.data_ptr(),
            plan.pos.data_ptr(), 1 if plan.pos.shape[0] > 1 else 0, plan._axes,
            int(plan.halves), dxq.data_ptr(), dxk.data_ptr(), dst6, dwq.data_ptr(),
            dwk.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
            _stream(dq))
    check(st, "dsa_qk_norm_rope_bwd")
    return dxq, dxk, dwq, dwk


def _check_window(q, k, v, out=None, dout=None):
    """B, H, Hk, Nq, Nk, D of q [B, H, Nq, D] and k, v [B, Hk, Nk, D]."""
    for t in (q, k, v):
        if t.dim() != 4 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous CUDA tensors [B, H, N, D]")
        if t.dtype != q.dtype or t.device != q.device or t.shape[0] != q.shape[0] or t.shape[3] != q.shape[3]:
            raise ValueError("q, k, v must share B, D, dtype and device")
    if k.shape != v.shape:
        raise ValueError("k and v must share their shape")
    for t in (out, dout):
        if t is not None and (t.shape != q.shape or t.dtype != q.dtype or t.device != q.device
                              or not t.is_contiguous()):
            raise ValueError("out and dout must match q")
    B, H, Nq, D = q.shape
    return B, H, k.shape[1], Nq, k.shape[2], D


def _check_lse(lse, q):
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != q.shape[:3] or lse.device != q.device
                            or not lse.is_contiguous()):
        raise ValueError("lse must be contiguous fp32 [B, H, Nq] on q's device")


def _check_mask(q_offset, left, right, sink):
    return _int32("q_offset", q_offset), _int32("left", left), _int32("right", right), _int32("sink", sink)


def window_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, left: int = -1, right: int = 0,
                    sink: int = 0, q_offset: Optional[int] = None, scale: Optional[float] = None,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    want_lse: bool = True):
    """(O [B, H, Nq, D], lse [B, H, Nq] or None): softmax attention in which key
    u is visible to the query at position t = q_offset + i iff u <= t + right
    and (u < sink or u >= t - left); a negative bound is no bound.

    q [B, H, Nq, D], k and v [B, Hk, Nk, D] with Hk dividing H.  q_offset
    defaults to Nk - Nq: the queries are the newest tokens."""
    B, H, Hk, Nq, Nk, D = _check_window(q, k, v, out)
    _check_lse(lse, q)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    q_offset, left, right, sink = _check_mask(Nk - Nq if q_offset is None else q_offset, left, right, sink)
    if out is None:
        out = torch.empty_like(q)
    if want_lse and lse is None:
        lse = q.new_empty((B, H, Nq), dtype=torch.float32)
    with _on(q):
        st = lib().dsa_window_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype_code(q), B, H, Hk, Nq,
                                       Nk, D, scale, q_offset, left, right, sink, out.data_ptr(), _ptr(lse),
                                       _stream(q))
    check(st, "dsa_window_attn_fwd")
    return out, lse


def window_attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                    dout: torch.Tensor, lse: torch.Tensor, left: int = -1, right: int = 0, sink: int = 0,
                    q_offset: Optional[int] = None, scale: Optional[float] = None,
                    workspace: Optional[torch.Tensor] = None):
    """(dQ, dK, dV) of window_attn_fwd's O for its gradient dout, with the O and
    lse it gave and the same mask; dK and dV summed over shared heads."""
    B, H, Hk, Nq, Nk, D = _check_window(q, k, v, out, dout)
    if lse is None:
        raise ValueError("the forward's lse is required")
    _check_lse(lse, q)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    q_offset, left, right, sink = _check_mask(Nk - Nq if q_offset is None else q_offset, left, right, sink)
    dt = _dtype_code(q)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if workspace is None:
        n = int(lib().dsa_window_attn_bwd_workspace_size(dt, B, H, Hk, Nq, Nk, D, q_offset, left, right, sink))
        workspace = q.new_empty(max(n, 16), dtype=torch.uint8)
    _check_workspace(workspace, q)
    with _on(q):
        st = lib().dsa_window_attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                       dout.data_ptr(), lse.data_ptr(), dt, B, H, Hk, Nq, Nk, D, scale,
                                       q_offset, left, right, sink, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                       workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                       _stream(q))
    check(st, "dsa_window_attn_bwd")
    return dq, dk, dv


def window_attn_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, lens: torch.Tensor,
                       left: int = -1, sink: int = 0, scale: Optional[float] = None,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """O [B, H, Nq, D] of each stream's newest Nq tokens (up to 128) over its
    cache: window_attn_fwd with right = 0 and q_offset = lens[b] - Nq.

    k_cache, v_cache [B, Hk, cap, D] may be strided (rows of D contiguous);
    lens int32 [B] on the device counts the keys in each cache, the new tokens'
    among them.  lse, if given, receives the log-sums [B, H, Nq]."""
    if q.dim() != 4 or not q.is_cuda or not q.is_contiguous():
        raise ValueError("q must be a contiguous CUDA tensor [B, H, Nq, D]")
    B, H, Nq, D = q.shape
    for t in (k_cache, v_cache):
        if t.dim() != 4 or t.dtype != q.dtype or t.device != q.device or t.shape != k_cache.shape \
                or t.shape[0] != B or t.shape[3] != D or t.stride(3) != 1:
            raise ValueError("caches must be [B, Hk, cap, D] of q's dtype and device with contiguous rows")
    if lens.dtype != torch.int32 or lens.device != q.device or lens.shape != (B,) or not lens.is_contiguous():
        raise ValueError("lens must be contiguous int32 [B] on q's device")
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or out.device != q.device or not out.is_contiguous():
        raise ValueError("out must match q")
    _check_lse(lse, q)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    st6 = _strides6(*(_strides3(t.shape, t.stride()) for t in (k_cache, v_cache)))
    Hk, cap, dt = k_cache.shape[1], k_cache.shape[2], _dtype_code(q)
    left, sink = _int32("left", left), _int32("sink", sink)
    if workspace is None:
        n = int(lib().dsa_window_attn_decode_workspace_size(dt, B, H, Hk, Nq, cap, D, left, sink))
        workspace = q.new_empty(n, dtype=torch.uint8) if n else None
    if workspace is not None:
        _check_workspace(workspace, q)
    with _on(q):
        st = lib().dsa_window_attn_decode(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), st6,
                                          dt, B, H, Hk, Nq, cap, D, scale, lens.data_ptr(), left,
                                          sink, out.data_ptr(), _ptr(lse), _ptr(workspace),
                                          0 if workspace is None else workspace.numel() * workspace.element_size(),
                                          _stream(q))
    check(st, "dsa_window_attn_decode")
    return out


def selftest_wait_timeout(limit_ns: int = 1_000_000, device: Optional[torch.device] = None) -> None:
    """Launch the failure-detection self-test: a bounded wait that runs out
    after limit_ns and records a wait timeout (dsa_device_status then raises)."""
    s = torch.cuda.current_stream(device).cuda_stream
    check(lib().dsa_selftest_wait_timeout(int(limit_ns), s), "dsa_selftest_wait_timeout")


def selftest_exp2_poly(x: torch.Tensor) -> torch.Tensor:
    """2^x by the attention softmax's FMA-pipe exponential (fp32 CUDA tensor)."""
    if not (x.is_cuda and x.dtype == torch.float32):
        raise ValueError("x must be a float32 CUDA tensor")
    x = x.contiguous()
    y = torch.empty_like(x)
    s = torch.cuda.current_stream(x.device).cuda_stream
    check(lib().dsa_selftest_exp2_poly(x.data_ptr(), y.data_ptr(), x.numel(), s), "dsa_selftest_exp2_poly")
    return y


def device_status(device: Optional[torch.device] = None) -> None:
    """Synchronises the current stream and raises DSAError if a kernel flagged bad input."""
    s = torch.cuda.current_stream(device).cuda_stream
    check(lib().dsa_device_status(s), "dsa_device_status")


class SparseAttention(NamedTuple):
    out: torch.Tensor          # [B, H, N, D]
    lse: torch.Tensor          # [B, H, N]
    probs: torch.Tensor        # [B*H, nB, nB]
    row_ptr: torch.Tensor      # [B*H*nB + 1]
    col_idx: torch.Tensor      # [nnz]
    mass: torch.Tensor         # [nnz]


def sparse_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, p: float,
                     block: int = 128, scale: Optional[float] = None,
                     cand: Optional[Csr] = None) -> SparseAttention:
    """Whole pipeline: pooled scores -> Top-p selection -> sparse attention
    (rows taken longest first within each head) -> block mass."""
    B, H, N, _ = q.shape
    probs = pool_score(q, k, block, scale, cand)
    row_ptr, col_idx = select_topp(probs, p, cand)
    order = row_order(row_ptr, B, H, n_blocks(N, block))
    out, lse, blk = attn_fwd(q, k, v, row_ptr, col_idx, block, scale, order=order)
    mass = block_mass(lse, blk, row_ptr, block)
    nnz = blk.shape[0] if int(row_ptr[-1].item()) > 0 else 0
    return SparseAttention(out, lse, probs, row_ptr, col_idx[:nnz], mass[:nnz])
