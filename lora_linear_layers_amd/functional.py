"""Python entry points with the C ABI's names (include/lora_linear.h).

Each call validates tensor placement/contiguity, allocates outputs (and the
workspace when none is passed) with torch, and calls the library on the
current HIP stream.  Row-major shapes:

    X [M, d_in]   W [d_out, d_in]   A [r, d_in]   B [d_out, r]   Y, dY [M, d_out]

scale is s = alpha / r.  dA and dB come back in fp32.
"""
from __future__ import annotations

import contextlib

import torch
from torch.autograd.function import once_differentiable

from . import _lib as L


def _dims(X, W_rows, W_cols, A, B):
    M, d_in = X.shape
    r = A.shape[0]
    if A.shape != (r, d_in) or B.shape != (W_rows, r) or W_cols != d_in:
        raise ValueError("shape mismatch: X [M,d_in], W [d_out,d_in], A [r,d_in], B [d_out,r]")
    return M, d_in, W_rows, r


def lora_linear_fwd(X, W, A, B, scale: float, Y=None, ws=None):
    """Y = X W^T + scale (X A^T) B^T."""
    L._contig(X, W, A, B, Y)
    M, d_in, d_out, r = _dims(X, W.shape[0], W.shape[1], A, B)
    dt = L._dtype_code(X)
    if Y is None:
        Y = torch.empty(M, d_out, dtype=X.dtype, device=X.device)
    ws = L._workspace(L.OP_FWD, dt, M, d_in, d_out, r, X.device, ws)
    L._check("lora_linear_fwd", L.lib().lora_linear_fwd(
        dt, M, d_in, d_out, r, float(scale), L._ptr(X), L._ptr(W), L._ptr(A), L._ptr(B), L._ptr(Y),
        L._ptr(ws), ws.numel(), L._stream(X.device)))
    return Y


def lora_linear_fwd_noalloc(X, W, A, B, scale: float, Y=None):
    """lora_linear_fwd with the library's static scratch instead of a
    workspace (for callers that cannot allocate device memory; Y is allocated
    here only when the caller passes none)."""
    L._contig(X, W, A, B, Y)
    M, d_in, d_out, r = _dims(X, W.shape[0], W.shape[1], A, B)
    dt = L._dtype_code(X)
    if Y is None:
        Y = torch.empty(M, d_out, dtype=X.dtype, device=X.device)
    L._check("lora_linear_fwd_noalloc", L.lib().lora_linear_fwd_noalloc(
        dt, M, d_in, d_out, r, float(scale), L._ptr(X), L._ptr(W), L._ptr(A), L._ptr(B), L._ptr(Y),
        L._stream(X.device)))
    return Y


def lora_linear_bwd(X, W, A, B, scale: float, dY, need_dX: bool = True, ws=None, out=None):
    """(dX or None, dA fp32, dB fp32) for upstream gradient dY; X A^T is recomputed."""
    L._contig(X, W, A, B, dY)
    M, d_in, d_out, r = _dims(X, W.shape[0], W.shape[1], A, B)
    dt = L._dtype_code(X)
    if out is None:
        dX = torch.empty(M, d_in, dtype=X.dtype, device=X.device) if need_dX else None
        dA = torch.empty(r, d_in, dtype=torch.float32, device=X.device)
        dB = torch.empty(d_out, r, dtype=torch.float32, device=X.device)
    else:
        dX, dA, dB = out
    ws = L._workspace(L.OP_BWD, dt, M, d_in, d_out, r, X.device, ws)
    L._check("lora_linear_bwd", L.lib().lora_linear_bwd(
        dt, M, d_in, d_out, r, float(scale), L._ptr(X), L._ptr(W), L._ptr(A), L._ptr(B), L._ptr(dY), L._ptr(dX),
        L._ptr(dA), L._ptr(dB), L._ptr(ws), ws.numel(), L._stream(X.device)))
    return dX, dA, dB


def rope_cache(max_pos: int, head_dim: int = 128, theta: float = 500000.0, device="cuda"):
    """(cos, sin) fp32 [max_pos, head_dim/2], filled on the device in fp64."""
    cos = torch.empty(max_pos, head_dim // 2, dtype=torch.float32, device=device)
    sin = torch.empty_like(cos)
    L._check("lora_rope_cache", L.lib().lora_rope_cache(max_pos, head_dim, float(theta), L._ptr(cos), L._ptr(sin),
                                                        L._stream(cos.device)))
    return cos, sin


def lora_qk_rope_fwd(X, W, A, B, scale: float, positions, cos, sin, head_dim: int = 128, Y=None, ws=None):
    """RoPE(X W^T + scale (X A^T) B^T) with the rotation as the GEMM epilogue."""
    L._contig(X, W, A, B, positions, cos, sin, Y)
    M, d_in, d_out, r = _dims(X, W.shape[0], W.shape[1], A, B)
    dt = L._dtype_code(X)
    if positions.dtype != torch.int32 or positions.numel() != M:
        raise ValueError("positions must be int32 [M]")
    if Y is None:
        Y = torch.empty(M, d_out, dtype=X.dtype, device=X.device)
    ws = L._workspace(L.OP_ROPE_FWD, dt, M, d_in, d_out, r, X.device, ws)
    L._check("lora_qk_rope_fwd", L.lib().lora_qk_rope_fwd(
        dt, M, d_in, d_out, r, float(scale), L._ptr(X), L._ptr(W), L._ptr(A), L._ptr(B), head_dim,
        L._ptr(positions), L._ptr(cos), L._ptr(sin), cos.shape[0], L._ptr(Y), L._ptr(ws), ws.numel(),
        L._stream(X.device)))
    return Y


def lora_qk_rope_bwd(X, W, A, B, scale: float, positions, cos, sin, dY, head_dim: int = 128,
                     need_dX: bool = True, ws=None):
    """Backward of lora_qk_rope_fwd: inverse rotation of dY, then the LoRA backward."""
    L._contig(X, W, A, B, positions, cos, sin, dY)
    M, d_in, d_out, r = _dims(X, W.shape[0], W.shape[1], A, B)
    dt = L._dtype_code(X)
    dX = torch.empty(M, d_in, dtype=X.dtype, device=X.device) if need_dX else None
    dA = torch.empty(r, d_in, dtype=torch.float32, device=X.device)
    dB = torch.empty(d_out, r, dtype=torch.float32, device=X.device)
    ws = L._workspace(L.OP_ROPE_BWD, dt, M, d_in, d_out, r, X.device, ws)
    L._check("lora_qk_rope_bwd", L.lib().lora_qk_rope_bwd(
        dt, M, d_in, d_out, r, float(scale), L._ptr(X), L._ptr(W), L._ptr(A), L._ptr(B), head_dim,
        L._ptr(positions), L._ptr(cos), L._ptr(sin), cos.shape[0], L._ptr(dY), L._ptr(dX), L._ptr(dA), L._ptr(dB),
        L._ptr(ws), ws.numel(), L._stream(X.device)))
    return dX, dA, dB


def nf4_lora_linear_fwd(X, codes, absmax, table16, A, B, scale: float, d_out: int, blocksize: int = 64,
                        Y=None, ws=None):
    """Forward with the NF4 base weight dequantised inside the GEMM load stage."""
    L._contig(X, codes, absmax, A, B, Y)
    M, d_in = X.shape
    r = A.shape[0]
    if X.dtype != torch.bfloat16:
        raise TypeError("NF4 path takes bf16 activations")
    if Y is None:
        Y = torch.empty(M, d_out, dtype=X.dtype, device=X.device)
    ws = L._workspace(L.OP_NF4_FWD, L.LORA_BF16, M, d_in, d_out, r, X.device, ws)
    tab = L._table_ptr(table16)
    L._check("nf4_lora_linear_fwd", L.lib().nf4_lora_linear_fwd(
        M, d_in, d_out, r, float(scale), L._ptr(X), L._ptr(codes), L._ptr(absmax), blocksize, tab, L._ptr(A),
        L._ptr(B), L._ptr(Y), L._ptr(ws), ws.numel(), L._stream(X.device)))
    return Y


def nf4_lora_linear_bwd(X, codes, absmax, table16, A, B, scale: float, dY, blocksize: int = 64,
                        need_dX: bool = True, ws=None):
    """(dX or None, dA, dB) with the NF4 base weight; no dW."""
    L._contig(X, codes, absmax, A, B, dY)
    M, d_in = X.shape
    d_out = dY.shape[1]
    r = A.shape[0]
    dX = torch.empty(M, d_in, dtype=X.dtype, device=X.device) if need_dX else None
    dA = torch.empty(r, d_in, dtype=torch.float32, device=X.device)
    dB = torch.empty(d_out, r, dtype=torch.float32, device=X.device)
    ws = L._workspace(L.OP_NF4_BWD, L.LORA_BF16, M, d_in, d_out, r, X.device, ws)
    tab = L._table_ptr(table16)
    L._check("nf4_lora_linear_bwd", L.lib().nf4_lora_linear_bwd(
        M, d_in, d_out, r, float(scale), L._ptr(X), L._ptr(codes), L._ptr(absmax), blocksize, tab, L._ptr(A),
        L._ptr(B), L._ptr(dY), L._ptr(dX), L._ptr(dA), L._ptr(dB), L._ptr(ws), ws.numel(), L._stream(X.device)))
    return dX, dA, dB


def nf4_dequant(codes, absmax, table16, n: int, blocksize: int = 64):
    """bf16 [n] from NF4 codes with the GEMM load stage's own routine."""
    out = torch.empty(n, dtype=torch.bfloat16, device=codes.device)
    tab = L._table_ptr(table16)
    L._check("nf4_dequant", L.lib().nf4_dequant(L._ptr(codes), L._ptr(absmax), blocksize, n, tab, L._ptr(out),
                                                L._stream(codes.device)))
    return out


def lora_dropout_fwd(X, W, A, B, scale: float, p: float, keep, Y=None, ws=None):
    """Y = X W^T + scale (D A^T) B^T, D = X * keep / (1 - p); keep is the packed
    uint8 bit mask [M, d_in / 8] (bit b of byte (i, j) keeps element (i, 8 j + b))."""
    L._contig(X, W, A, B, keep, Y)
    M, d_in, d_out, r = _dims(X, W.shape[0], W.shape[1], A, B)
    _check_keep(keep, M, d_in)
    dt = L._dtype_code(X)
    if Y is None:
        Y = torch.empty(M, d_out, dtype=X.dtype, device=X.device)
    ws = L._workspace(L.OP_DROPOUT_FWD, dt, M, d_in, d_out, r, X.device, ws)
    L._check("lora_dropout_fwd", L.lib().lora_dropout_fwd(
        dt, M, d_in, d_out, r, float(scale), float(p), L._ptr(keep), L._ptr(X), L._ptr(W), L._ptr(A), L._ptr(B),
        L._ptr(Y), L._ptr(ws), ws.numel(), L._stream(X.device)))
    return Y


def lora_dropout_bwd(X, W, A, B, scale: float, p: float, keep, dY, need_dX: bool = True, ws=None):
    """(dX or None, dA fp32, dB fp32) of lora_dropout_fwd with the same keep mask."""
    L._contig(X, W, A, B, keep, dY)
    M, d_in, d_out, r = _dims(X, W.shape[0], W.shape[1], A, B)
    _check_keep(keep, M, d_in)
    dt = L._dtype_code(X)
    dX = torch.empty(M, d_in, dtype=X.dtype, device=X.device) if need_dX else None
    dA = torch.empty(r, d_in, dtype=torch.float32, device=X.device)
    dB = torch.empty(d_out, r, dtype=torch.float32, device=X.device)
    ws = L._workspace(L.OP_DROPOUT_BWD, dt, M, d_in, d_out, r, X.device, ws)
    L._check("lora_dropout_bwd", L.lib().lora_dropout_bwd(
        dt, M, d_in, d_out, r, float(scale), float(p), L._ptr(keep), L._ptr(X), L._ptr(W), L._ptr(A), L._ptr(B),
        L._ptr(dY), L._ptr(dX), L._ptr(dA), L._ptr(dB), L._ptr(ws), ws.numel(), L._stream(X.device)))
    return dX, dA, dB


def lora_dropout_mask(M: int, d_in: int, p: float, seed: int, offset: int = 0, device="cuda"):
    """The packed keep mask [M, d_in / 8] (uint8) that the Philox dropout entry
    points draw for (seed, offset), generated on the device."""
    keep = torch.empty(M, d_in // 8, dtype=torch.uint8, device=device)
    L._check("lora_dropout_mask", L.lib().lora_dropout_mask(M, d_in, float(p), int(seed), int(offset),
                                                            L._ptr(keep), L._stream(keep.device)))
    return keep


def lora_dropout_philox_fwd(X, W, A, B, scale: float, p: float, seed: int, offset: int = 0, Y=None, ws=None):
    """lora_dropout_fwd with the keep mask drawn on the device from Philox4x32-10
    (seed, offset), as lora_dropout_mask draws it."""
    L._contig(X, W, A, B, Y)
    M, d_in, d_out, r = _dims(X, W.shape[0], W.shape[1], A, B)
    dt = L._dtype_code(X)
    if Y is None:
        Y = torch.empty(M, d_out, dtype=X.dtype, device=X.device)
    ws = L._workspace(L.OP_DROPOUT_FWD, dt, M, d_in, d_out, r, X.device, ws)
    L._check("lora_dropout_philox_fwd", L.lib().lora_dropout_philox_fwd(
        dt, M, d_in, d_out, r, float(scale), float(p), int(seed), int(offset), L._ptr(X), L._ptr(W), L._ptr(A),
        L._ptr(B), L._ptr(Y), L._ptr(ws), ws.numel(), L._stream(X.device)))
    return Y


def lora_dropout_philox_bwd(X, W, A, B, scale: float, p: float, seed: int, dY, offset: int = 0,
                            need_dX: bool = True, ws=None):
    """(dX or None, dA fp32, dB fp32) of lora_dropout_philox_fwd with the same
    (seed, offset): the mask is drawn again, not stored."""
    L._contig(X, W, A, B, dY)
    M, d_in, d_out, r = _dims(X, W.shape[0], W.shape[1], A, B)
    dt = L._dtype_code(X)
    dX = torch.empty(M, d_in, dtype=X.dtype, device=X.device) if need_dX else None
    dA = torch.empty(r, d_in, dtype=torch.float32, device=X.device)
    dB = torch.empty(d_out, r, dtype=torch.float32, device=X.device)
    ws = L._workspace(L.OP_DROPOUT_BWD, dt, M, d_in, d_out, r, X.device, ws)
    L._check("lora_dropout_philox_bwd", L.lib().lora_dropout_philox_bwd(
        dt, M, d_in, d_out, r, float(scale), float(p), int(seed), int(offset), L._ptr(X), L._ptr(W), L._ptr(A),
        L._ptr(B), L._ptr(dY), L._ptr(dX), L._ptr(dA), L._ptr(dB), L._ptr(ws), ws.numel(), L._stream(X.device)))
    return dX, dA, dB


def _check_keep(keep, M, d_in):
    if keep.dtype != torch.uint8 or keep.numel() != M * d_in // 8:
        raise ValueError("keep must be a uint8 bit mask of M * d_in / 8 bytes")


def lora_transpose(W, out=None):
    """W^T (bf16) through the library's tiled transpose, e.g. the frozen
    weight's transpose that group members take as W_t."""
    L._contig(W, out)
    if W.dtype != torch.bfloat16 or W.dim() != 2:
        raise TypeError("bf16 matrix expected")
    rows, cols = W.shape
    if out is None:
        out = torch.empty(cols, rows, dtype=W.dtype, device=W.device)
    L._check("lora_transpose", L.lib().lora_transpose(L._ptr(W), rows, cols, L._ptr(out), L._stream(W.device)))
    return out


def lora_merge(W, A, B, scale: float, out=None, ws=None):
    """W + scale B A in W's dtype (out may be W itself); -scale unmerges."""
    L._contig(W, A, B, out)
    d_out, d_in = W.shape
    r = A.shape[0]
    if A.shape != (r, d_in) or B.shape != (d_out, r):
        raise ValueError("shape mismatch: W [d_out,d_in], A [r,d_in], B [d_out,r]")
    dt = L._dtype_code(W)
    if out is None:
        out = torch.empty_like(W)
    ws = L._workspace(L.OP_MERGE, dt, 0, d_in, d_out, r, W.device, ws)
    L._check("lora_merge", L.lib().lora_merge(dt, d_out, d_in, r, float(scale), L._ptr(W), L._ptr(A), L._ptr(B),
                                              L._ptr(out), L._ptr(ws), ws.numel(), L._stream(W.device)))
    return out


def _group_members(X, members):
    """ctypes array of lora_group_member from dicts with keys A, B, scale and
    either W or (codes, absmax), plus an optional rope flag."""
    n = len(members)
    if not 1 <= n <= L.GROUP_MAX:
        raise ValueError(f"a group holds 1..{L.GROUP_MAX} projections")
    arr = (L.GroupMember * n)()
    M, d_in = X.shape
    for g, m in enumerate(members):
        A, B = m["A"], m["B"]
        W, codes, absmax, Wt = m.get("W"), m.get("codes"), m.get("absmax"), m.get("W_t")
        L._contig(A, B, W, codes, absmax, Wt)
        r, d_out = A.shape[0], B.shape[0]
        if A.shape != (r, d_in) or B.shape != (d_out, r) or (W is not None and W.shape != (d_out, d_in)):
            raise ValueError("shape mismatch: X [M,d_in], W [d_out,d_in], A [r,d_in], B [d_out,r]")
        if (W is None) == (codes is None):
            raise ValueError("each member takes exactly one of W and NF4 codes")
        e = arr[g]
        e.d_out, e.r, e.scale, e.rope = d_out, r, float(m["scale"]), int(bool(m.get("rope", False)))
        if Wt is not None and (Wt.shape != (d_in, d_out) or Wt.dtype != torch.bfloat16):
            raise ValueError("W_t must be the bf16 [d_in, d_out] transpose of W")
        e.W, e.W_nf4, e.absmax, e.W_t = (L._ptr(t) for t in (W, codes, absmax, Wt))
        e.A, e.B = L._ptr(A), L._ptr(B)
    return arr


def _group_ws(backward, dt, M, d_in, arr, device, ws):
    if ws is not None:
        return _check_ws(device, ws)
    n = int(L.lib().lora_group_workspace_bytes(int(backward), dt, M, d_in, len(arr), arr))
    return torch.empty(max(n, 1), dtype=torch.uint8, device=device)


def _group_rope(positions, cos, sin, M):
    if positions is None:
        return None, None, None, 0
    L._contig(positions, cos, sin)
    if positions.dtype != torch.int32 or positions.numel() != M:
        raise ValueError("positions must be int32 [M]")
    return L._ptr(positions), L._ptr(cos), L._ptr(sin), cos.shape[0]


def lora_group_fwd(X, members, positions=None, cos=None, sin=None, table16=None, head_dim: int = 128, ws=None,
                   Ys=None):
    """[Y_1, .., Y_n] of projections sharing X, the rank-r panels in one pass over X."""
    L._contig(X)
    M, d_in = X.shape
    dt = L._dtype_code(X)
    arr = _group_members(X, members)
    if Ys is None:
        Ys = [torch.empty(M, arr[g].d_out, dtype=X.dtype, device=X.device) for g in range(len(arr))]
    for g, Y in enumerate(Ys):
        L._contig(Y)
        if Y.shape != (M, arr[g].d_out) or Y.dtype != X.dtype:
            raise ValueError("Y shape or dtype mismatch")
        arr[g].Y = L._ptr(Y)
    pos, c, s, max_pos = _group_rope(positions, cos, sin, M)
    tab = L._table_ptr(table16) if table16 is not None else None
    ws = _group_ws(False, dt, M, d_in, arr, X.device, ws)
    L._check("lora_group_fwd", L.lib().lora_group_fwd(
        dt, M, d_in, len(arr), arr, L._ptr(X), head_dim, pos, c, s, max_pos, tab, L._ptr(ws), ws.numel(),
        L._stream(X.device)))
    return Ys


def lora_group_bwd(X, members, dYs, positions=None, cos=None, sin=None, table16=None, head_dim: int = 128,
                   need_dX: bool = True, ws=None, outs=None):
    """[(dX_g or None, dA_g fp32, dB_g fp32)] per member; dX_g is the member's own
    input gradient (the caller sums them)."""
    L._contig(X, *dYs)
    M, d_in = X.shape
    dt = L._dtype_code(X)
    arr = _group_members(X, members)
    if len(dYs) != len(arr):
        raise ValueError("one dY per member")
    res = []
    for g in range(len(arr)):
        d_out, r = arr[g].d_out, arr[g].r
        if dYs[g].shape != (M, d_out):
            raise ValueError("dY shape mismatch")
        if outs is None:
            dX = torch.empty(M, d_in, dtype=X.dtype, device=X.device) if need_dX else None
            dA = torch.empty(r, d_in, dtype=torch.float32, device=X.device)
            dB = torch.empty(d_out, r, dtype=torch.float32, device=X.device)
        else:
            dX, dA, dB = outs[g]
            L._contig(dX, dA, dB)
            if (dX is not None and dX.shape != (M, d_in)) or dA.shape != (r, d_in) or dB.shape != (d_out, r) \
                    or dA.dtype != torch.float32 or dB.dtype != torch.float32:
                raise ValueError("output shape or dtype mismatch")
        arr[g].dY, arr[g].dX, arr[g].dA, arr[g].dB = L._ptr(dYs[g]), L._ptr(dX), L._ptr(dA), L._ptr(dB)
        res.append((dX, dA, dB))
    pos, c, s, max_pos = _group_rope(positions, cos, sin, M)
    tab = L._table_ptr(table16) if table16 is not None else None
    ws = _group_ws(True, dt, M, d_in, arr, X.device, ws)
    L._check("lora_group_bwd", L.lib().lora_group_bwd(
        dt, M, d_in, len(arr), arr, L._ptr(X), head_dim, pos, c, s, max_pos, tab, L._ptr(ws), ws.numel(),
        L._stream(X.device)))
    return res


def _swiglu_ws(backward, dt, M, d_in, arr, device, ws):
    if ws is not None:
        return _check_ws(device, ws)
    n = int(L.lib().lora_swiglu_workspace_bytes(int(backward), dt, M, d_in, arr))
    return torch.empty(max(n, 1), dtype=torch.uint8, device=device)


def lora_swiglu_fwd(X, members, table16=None, H=None, store_gu: bool = True, ws=None):
    """(H, G, U) for the gate (members[0]) and up (members[1]) projections of X:
    H = silu(G) * U; G and U come back (for the backward) when store_gu, else None."""
    L._contig(X, H)
    if len(members) != 2:
        raise ValueError("SwiGLU takes the gate and the up projection")
    M, d_in = X.shape
    dt = L._dtype_code(X)
    arr = _group_members(X, members)
    d = arr[0].d_out
    if H is None:
        H = torch.empty(M, d, dtype=X.dtype, device=X.device)
    G = U = None
    if store_gu:
        G = torch.empty(M, d, dtype=X.dtype, device=X.device)
        U = torch.empty(M, d, dtype=X.dtype, device=X.device)
        arr[0].Y, arr[1].Y = L._ptr(G), L._ptr(U)
    tab = L._table_ptr(table16) if table16 is not None else None
    ws = _swiglu_ws(False, dt, M, d_in, arr, X.device, ws)
    L._check("lora_swiglu_fwd", L.lib().lora_swiglu_fwd(dt, M, d_in, arr, L._ptr(X), tab, L._ptr(H), L._ptr(ws),
                                                        ws.numel(), L._stream(X.device)))
    return H, G, U


def lora_swiglu_bwd(X, members, dH, G, U, table16=None, need_dX: bool = True, ws=None):
    """(dX or None, [(dA_gate, dB_gate), (dA_up, dB_up)]); dX sums both input gradients."""
    L._contig(X, dH, G, U)
    if len(members) != 2:
        raise ValueError("SwiGLU takes the gate and the up projection")
    M, d_in = X.shape
    dt = L._dtype_code(X)
    arr = _group_members(X, members)
    d = arr[0].d_out
    for t in (dH, G, U):
        if t.shape != (M, d):
            raise ValueError("dH, G and U must be [M, d_out]")
    dX = torch.empty(M, d_in, dtype=X.dtype, device=X.device) if need_dX else None
    grads = []
    for g in range(2):
        dA = torch.empty(arr[g].r, d_in, dtype=torch.float32, device=X.device)
        dB = torch.empty(d, arr[g].r, dtype=torch.float32, device=X.device)
        arr[g].dA, arr[g].dB = L._ptr(dA), L._ptr(dB)
        grads.append((dA, dB))
    tab = L._table_ptr(table16) if table16 is not None else None
    ws = _swiglu_ws(True, dt, M, d_in, arr, X.device, ws)
    L._check("lora_swiglu_bwd", L.lib().lora_swiglu_bwd(
        dt, M, d_in, arr, L._ptr(X), tab, L._ptr(dH), L._ptr(G), L._ptr(U), L._ptr(dX), L._ptr(ws), ws.numel(),
        L._stream(X.device)))
    return dX, grads


# ---------------------------------------------------------------------------
# one projection with bias, activation and residual
# ---------------------------------------------------------------------------
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def _epi_member(X, member):
    """(device, M, d_in, d_out, r, the ctypes member) of a projection, its tensors checked against X."""
    dev, same = _gpu(X), (X.dtype,)
    if X.dim() != 2:
        raise ValueError("X must be [M, d_in]")
    A, B, W, codes, absmax, Wt = (member.get(k) for k in ("A", "B", "W", "codes", "absmax", "W_t"))
    (M, d_in), r, d_out = X.shape, A.shape[0], B.shape[0]
    _check(dev, "X", X, same)
    _check(dev, "A", A, same, r * d_in)
    _check(dev, "B", B, same, d_out * r)
    if (W is None) == (codes is None):
        raise ValueError("a member takes exactly one of W and NF4 codes")
    if A.dim() != 2 or B.dim() != 2 or (W is not None and W.shape != (d_out, d_in)):
        raise ValueError("shape mismatch: X [M,d_in], W [d_out,d_in], A [r,d_in], B [d_out,r]")
    if W is not None:
        _check(dev, "W", W, same)
    else:
        _check(dev, "codes", codes, (torch.uint8,), d_out * d_in // 2)
        if absmax is None:
            raise ValueError("codes need absmax")
        _check(dev, "absmax", absmax, _F32, d_out * d_in // 64)
    if Wt is not None:
        _check(dev, "W_t", Wt, (torch.bfloat16,), d_out * d_in)
        if Wt.shape != (d_in, d_out):
            raise ValueError("W_t must be the bf16 [d_in, d_out] transpose of W")
    return dev, M, d_in, d_out, r, _epi_struct(member, r, d_out)


def _epi_struct(member, r, d_out):
    get = member.get
    return L.GroupMember(d_out, r, member["scale"], 1 if get("rope") else 0, L._ptr(get("W")), L._ptr(get("codes")),
                         L._ptr(get("absmax")), L._ptr(member["A"]), L._ptr(member["B"]), None, None, None, None, None,
                         L._ptr(get("W_t")))


def _epi_ws(backward, dt, M, d_in, m, e, device, ws):
    """(workspace, its bytes)"""
    if ws is not None:
        return _check_ws(device, ws, ws.nbytes), ws.nbytes
    n = int(L.lib().lora_linear_epi_workspace_bytes(int(backward), dt, M, d_in, m, e))
    return torch.empty(max(n, 1), dtype=torch.uint8, device=device), n


def lora_linear_epi_fwd(X, member, act: str = "none", bias=None, residual=None, table16=None, Y=None,
                        store_z: bool = False, ws=None):
    """(Y, Z or None): Y = act(Z) + residual, Z = X W^T + scale (X A^T) B^T + bias, for a member as lora_group_fwd
    takes them (W or NF4 codes and absmax, A, B, scale).  Z comes back (for the backward) when store_z.  Y may be the
    residual."""
    dt = L._dtype_code(X)
    dev, M, d_in, d_out, r, m = _epi_member(X, member)
    same = (X.dtype,)
    if bias is not None:
        _check(dev, "bias", bias, same, d_out)
    if residual is not None:
        _check(dev, "residual", residual, same, M * d_out)
    if Y is None:
        Y = torch.empty(M, d_out, dtype=X.dtype, device=dev)
    else:
        _check(dev, "Y", Y, same, M * d_out)
    Z = torch.empty(M, d_out, dtype=X.dtype, device=dev) if store_z else None
    m.Y = L._ptr(Y)
    e = L.Epilogue(_choice("act", ACTIVATIONS, act), L._ptr(bias), L._ptr(residual), L._ptr(Z))
    tab = L._table_ptr(table16) if table16 is not None else None
    ws, ws_bytes = _epi_ws(False, dt, M, d_in, m, e, dev, ws)
    with _on(dev):
        L._check("lora_linear_epi_fwd", L.lib().lora_linear_epi_fwd(
            dt, M, d_in, m, e, L._ptr(X), tab, L._ptr(ws), ws_bytes, L._stream(dev)))
    return Y, Z


def lora_linear_epi_bwd(X, member, dY, act: str = "none", Z=None, need_dX: bool = True, need_dbias: bool = False,
                        table16=None, ws=None):
    """(dX or None, dA fp32, dB fp32, dbias fp32 or None) of lora_linear_epi_fwd; Z: its pre-activation (not needed
    with act "none").  The residual's gradient is dY."""
    dt = L._dtype_code(X)
    dev, M, d_in, d_out, r, m = _epi_member(X, member)
    same = (X.dtype,)
    _check(dev, "dY", dY, same, M * d_out)
    if Z is not None:
        _check(dev, "Z", Z, same, M * d_out)
    return _epi_bwd(dt, dev, M, d_in, d_out, r, m, X, dY, act, Z, need_dX, need_dbias, table16, ws)


def _epi_bwd(dt, dev, M, d_in, d_out, r, m, X, dY, act, Z, need_dX, need_dbias, table16=None, ws=None):
    """lora_linear_epi_bwd of checked tensors."""
    dX = torch.empty(M, d_in, dtype=X.dtype, device=dev) if need_dX else None
    dA = torch.empty(r, d_in, dtype=torch.float32, device=dev)
    dB = torch.empty(d_out, r, dtype=torch.float32, device=dev)
    dbias = torch.empty(d_out, dtype=torch.float32, device=dev) if need_dbias else None
    m.dY, m.dX, m.dA, m.dB = L._ptr(dY), L._ptr(dX), L._ptr(dA), L._ptr(dB)
    e = L.Epilogue(_choice("act", ACTIVATIONS, act), None, None, L._ptr(Z))
    tab = L._table_ptr(table16) if table16 is not None else None
    ws, ws_bytes = _epi_ws(True, dt, M, d_in, m, e, dev, ws)
    with _on(dev):
        L._check("lora_linear_epi_bwd", L.lib().lora_linear_epi_bwd(
            dt, M, d_in, m, e, L._ptr(X), tab, L._ptr(dbias), L._ptr(ws), ws_bytes, L._stream(dev)))
    return dX, dA, dB, dbias


class LoraLinearEpiFunction(torch.autograd.Function):
    """Y = LoraLinearEpiFunction.apply(X, W, A, B, bias, residual, scale, act, W_t): gradients for X, A, B, bias and
    residual (W frozen; bias and residual may be None; W_t: W's transpose, where the caller keeps one for dX)."""

    @staticmethod
    def forward(ctx, X, W, A, B, bias, residual, scale, act="none", W_t=None):
        member = {"W": W, "A": A, "B": B, "scale": scale, "W_t": W_t}
        # (the residual's gradient alone needs no Z)
        Y, Z = lora_linear_epi_fwd(X, member, act, bias, residual,
                                   store_z=act != "none" and any(ctx.needs_input_grad[i] for i in (0, 2, 3, 4)))
        ctx.save_for_backward(X, W, A, B, Z, W_t)
        ctx.dims, ctx.scale, ctx.act = (*X.shape, *B.shape), scale, act
        ctx.shapes = [None if t is None else t.shape for t in (bias, residual)]
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        dev, same, (M, d_in, d_out, r) = dY.device, dY.dtype, ctx.dims
        X, W, A, B, Z, W_t = _kept(ctx, dev, (same, (M, d_in)), (same, (d_out, d_in)), (same, (r, d_in)), (same, (d_out, r)),
                                   (same, (M, d_out)), (torch.bfloat16, (d_in, d_out)))
        dY = dY.contiguous()
        _check(dev, "the gradient of Y", dY, (X.dtype,), M * d_out)
        bias, residual = ctx.shapes
        need_dX, _, need_dA, need_dB, need_dbias, need_dR = ctx.needs_input_grad[:6]
        dX = dA = dB = dbias = dR = None
        if need_dX or need_dA or need_dB or need_dbias:
            m = _epi_struct({"W": W, "A": A, "B": B, "scale": ctx.scale, "W_t": W_t}, r, d_out)
            dX, dA, dB, dbias = _epi_bwd(L._dtype_code(X), dev, M, d_in, d_out, r, m, X, dY, ctx.act, Z, need_dX,
                                         need_dbias)
            # (each gradient in a storage of its own)
            dA = dA.to(A.dtype) if need_dA else None
            dB = dB.to(B.dtype) if need_dB else None
            dbias = dbias.to(X.dtype).view(bias) if need_dbias else None
        if need_dR:  # dY itself, or a copy: autograd would keep a view of it, the caller's memory
            dR = dY if dY.shape == residual else dY.clone().view(residual)
        return (dX, None, dA, dB, dbias, dR, None, None, None)


class LoraLinearFunction(torch.autograd.Function):
    """Autograd wrapper: gradients for X, A and B (W frozen); A and B grads in fp32."""

    @staticmethod
    def forward(ctx, X, W, A, B, scale):
        ctx.save_for_backward(X, W, A, B)
        ctx.scale = scale
        return lora_linear_fwd(X, W, A, B, scale)

    @staticmethod
    def backward(ctx, dY):
        X, W, A, B = ctx.saved_tensors
        dX, dA, dB = lora_linear_bwd(X, W, A, B, ctx.scale, dY.contiguous(), need_dX=ctx.needs_input_grad[0])
        return dX, None, dA.to(A.dtype), dB.to(B.dtype), None


# ---------------------------------------------------------------------------
# token log-probabilities and the losses that read them
# ---------------------------------------------------------------------------
class _OtherDevice:
    """Makes a device current for one call (launches go to the current device)."""

    def __init__(self, index):
        self.index = index

    def __enter__(self):
        self.back = torch.cuda.current_device()
        torch.cuda.set_device(self.index)

    def __exit__(self, *_):
        torch.cuda.set_device(self.back)


_HERE = contextlib.nullcontext()


def _on(device):
    return _HERE if device.index == torch.cuda.current_device() else _OtherDevice(device.index)


def _check(device, name, t, dtypes, numel=None):
    """t is on the device, contiguous, of one of the dtypes and of numel values."""
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} values, not {numel}")


def _check_ws(device, ws, nbytes=None):
    """A caller's workspace: on the device or pinned, with nbytes (its elements' number by default) behind its first
    element, however it is laid out.  The library is told that size and checks it."""
    if ws.device != device and not ws.is_pinned():
        raise ValueError(f"ws is on {ws.device}, not on {device}")
    if ws.untyped_storage().nbytes() - ws.storage_offset() * ws.element_size() < (ws.numel() if nbytes is None else nbytes):
        raise ValueError("ws holds fewer bytes than it has elements")
    return ws


def _kept(ctx, device, *as_saved):
    """The saved tensors, still contiguous, on the device and of the dtype and shape that as_saved gives for each:
    saved-tensor hooks may give back any others, and their addresses go to the library."""
    saved = ctx.saved_tensors
    for t, (dtype, shape) in zip(saved, as_saved):
        if t is not None and (t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous()):
            raise ValueError("a saved tensor came back with another device, dtype, shape or strides")
    return saved


def _gpu(t):
    if not t.is_cuda:
        raise ValueError("tensors must be on a GPU")
    return t.device


_F32, _I64, _MASK = (torch.float32,), (torch.int64,), (torch.bool, torch.uint8)


def _logits_ld(name, z):
    if z.dim() != 2:
        raise ValueError(f"{name} must be [n, vocab]")
    n, vocab = z.shape
    if vocab > 1 and z.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return n, vocab, (z.stride(0) if n > 1 else vocab)


def lora_token_logp_fwd(logits, targets, inv_temp: float = 1.0):
    """(logp fp32 [n], stats fp32 [n, 2]) of int64 targets [n] under the rows of logits [n, vocab] (rows may be
    strided); stats holds each row's maximum logit and the log of its shifted sum, which the backward takes."""
    n, vocab, ld = _logits_ld("logits", logits)
    dev = _gpu(logits)
    _check(dev, "targets", targets, _I64, n)
    dt = L._dtype_code(logits)
    logp = torch.empty(n, dtype=torch.float32, device=dev)
    stats = torch.empty(n, 2, dtype=torch.float32, device=dev)
    with _on(dev):
        L._check("lora_token_logp_fwd", L.lib().lora_token_logp_fwd(
            dt, n, vocab, L._ptr(logits), ld, L._ptr(targets), float(inv_temp), L._ptr(logp), L._ptr(stats),
            L._stream(dev)))
    return logp, stats


def lora_token_logp_bwd(logits, targets, stats, dlogp, inv_temp: float = 1.0, dlogits=None):
    """dlogits in the dtype of logits for the upstream gradient dlogp fp32 [n]; dlogits may be logits itself."""
    n, vocab, ld = _logits_ld("logits", logits)
    dev = _gpu(logits)
    _check(dev, "targets", targets, _I64, n)
    _check(dev, "stats", stats, _F32, 2 * n)
    _check(dev, "dlogp", dlogp, _F32, n)
    dt = L._dtype_code(logits)
    if dlogits is None:
        dlogits, ldd = torch.empty(n, vocab, dtype=logits.dtype, device=dev), vocab
    else:
        nd, vd, ldd = _logits_ld("dlogits", dlogits)
        if (nd, vd) != (n, vocab) or dlogits.dtype != logits.dtype or dlogits.device != dev:
            raise ValueError("dlogits must have the shape, dtype and device of logits")
    with _on(dev):
        L._check("lora_token_logp_bwd", L.lib().lora_token_logp_bwd(
            dt, n, vocab, L._ptr(logits), ld, L._ptr(targets), float(inv_temp), L._ptr(stats), L._ptr(dlogp),
            L._ptr(dlogits), ldd, L._stream(dev)))
    return dlogits


def _loss_ws(loss, n_seq, n_tokens, logp, ws):
    """(workspace, its bytes)"""
    if ws is not None:
        return _check_ws(logp.device, ws, ws.nbytes), ws.nbytes
    nbytes = L.lib().lora_loss_workspace_bytes(loss, n_seq, n_tokens)
    return logp.new_empty(nbytes // 4), nbytes


PREFERENCE_KINDS = {"sigmoid": 0, "hinge": 1, "ipo": 2}
POLICY_REDUCTIONS = {"sequence": 0, "token": 1, "constant": 2}


def _choice(name, table, value):
    if value not in table:
        raise ValueError(f"{name} must be one of {', '.join(table)}")
    return table[value]


def _check_tokens(dev, n, cu, ref_logp, mask):
    _check(dev, "cu", cu, _I64)
    if ref_logp is not None:
        _check(dev, "ref_logp", ref_logp, _F32, n)
    if mask is not None:
        _check(dev, "mask", mask, _MASK, n)


def _pairs(cu):
    """P of the 2 P + 1 offsets of response pairs."""
    S = cu.numel() - 1
    if S < 2 or S % 2:
        raise ValueError("cu must hold 2 P + 1 offsets")
    return S // 2


def lora_preference_loss_fwd(logp, cu, beta: float, ref_logp=None, mask=None, kind: str = "sigmoid",
                             label_smoothing: float = 0.0, average: bool = False, ws=None):
    """(loss, pair_loss [P], rewards [2 P], coef [2 P]) of P pairs over packed sequences: logp (and ref_logp) fp32
    [n], cu int64 [2 P + 1] with the chosen responses first, then the rejected ones in the same order; mask bool or
    uint8 [n] (tokens that count).  coef goes to lora_preference_loss_bwd."""
    n, dev = logp.numel(), _gpu(logp)
    _check(dev, "logp", logp, _F32)
    _check_tokens(dev, n, cu, ref_logp, mask)
    P = _pairs(cu)
    S = 2 * P
    new = logp.new_empty
    loss, pair_loss, rewards, coef = new(()), new(P), new(S), new(S)
    ws, ws_bytes = _loss_ws(0, S, n, logp, ws)
    with _on(dev):
        L._check("lora_preference_loss_fwd", L.lib().lora_preference_loss_fwd(
            _choice("kind", PREFERENCE_KINDS, kind), P, n, float(beta), float(label_smoothing), int(average),
            L._ptr(cu), L._ptr(mask), L._ptr(logp), L._ptr(ref_logp), L._ptr(loss), L._ptr(pair_loss),
            L._ptr(rewards), L._ptr(coef), L._ptr(ws), ws_bytes, L._stream(dev)))
    return loss, pair_loss, rewards, coef


def lora_preference_loss_bwd(coef, cu, n_tokens: int, mask=None, dloss=None):
    """dlogp fp32 [n_tokens] of lora_preference_loss_fwd; dloss: fp32 scalar tensor (None: 1)."""
    dev, P = _gpu(coef), _pairs(cu)
    _check(dev, "coef", coef, _F32, 2 * P)
    _check_tokens(dev, n_tokens, cu, None, mask)
    if dloss is not None:
        _check(dev, "dloss", dloss, _F32, 1)
    dlogp = coef.new_empty(n_tokens)
    with _on(dev):
        L._check("lora_preference_loss_bwd", L.lib().lora_preference_loss_bwd(
            P, n_tokens, L._ptr(cu), L._ptr(mask), L._ptr(coef), L._ptr(dloss), L._ptr(dlogp),
            L._stream(dev)))
    return dlogp


def _policy_checks(logp, cu, advantages, old_logp, ref_logp, mask, per_token):
    n, S, dev = logp.numel(), cu.numel() - 1, _gpu(logp)
    if S < 1:
        raise ValueError("cu must hold S + 1 offsets")
    _check(dev, "logp", logp, _F32)
    _check_tokens(dev, n, cu, ref_logp, mask)
    _check(dev, "advantages", advantages, _F32, n if per_token else S)
    if old_logp is not None:
        _check(dev, "old_logp", old_logp, _F32, n)
    return n, S, dev


def lora_policy_loss_fwd(logp, cu, advantages, old_logp=None, ref_logp=None, mask=None, eps_low: float = 0.2,
                         eps_high: float = 0.2, beta: float = 0.0, reduction: str = "sequence", norm: float = 1.0,
                         per_token: bool = False, ws=None):
    """(loss, stats [4], weight [S]) of the clipped policy loss over packed sequences: logp (old_logp, ref_logp)
    fp32 [n], cu int64 [S + 1], advantages fp32 [S], or [n] with per_token; stats: the policy part, the KL part, the
    share of clipped tokens, the number of tokens.  weight goes to lora_policy_loss_bwd."""
    n, S, dev = _policy_checks(logp, cu, advantages, old_logp, ref_logp, mask, per_token)
    new = logp.new_empty
    loss, stats, weight = new(()), new(4), new(S)
    ws, ws_bytes = _loss_ws(1, S, n, logp, ws)
    with _on(dev):
        L._check("lora_policy_loss_fwd", L.lib().lora_policy_loss_fwd(
            _choice("reduction", POLICY_REDUCTIONS, reduction), S, n, float(eps_low), float(eps_high), float(beta),
            float(norm), L._ptr(cu), L._ptr(mask), L._ptr(logp), L._ptr(old_logp), L._ptr(ref_logp),
            L._ptr(advantages), int(per_token), L._ptr(loss), L._ptr(stats), L._ptr(weight), L._ptr(ws), ws_bytes,
            L._stream(dev)))
    return loss, stats, weight


def lora_policy_loss_bwd(logp, cu, advantages, weight, old_logp=None, ref_logp=None, mask=None, eps_low: float = 0.2,
                         eps_high: float = 0.2, beta: float = 0.0, per_token: bool = False, dloss=None):
    """dlogp fp32 [n] of lora_policy_loss_fwd, given its weight and the same inputs; dloss: fp32 scalar tensor."""
    n, S, dev = _policy_checks(logp, cu, advantages, old_logp, ref_logp, mask, per_token)
    _check(dev, "weight", weight, _F32, S)
    if dloss is not None:
        _check(dev, "dloss", dloss, _F32, 1)
    dlogp = logp.new_empty(n)
    with _on(dev):
        L._check("lora_policy_loss_bwd", L.lib().lora_policy_loss_bwd(
            S, n, float(eps_low), float(eps_high), float(beta), L._ptr(cu), L._ptr(mask), L._ptr(logp),
            L._ptr(old_logp), L._ptr(ref_logp), L._ptr(advantages), int(per_token), L._ptr(weight), L._ptr(dloss),
            L._ptr(dlogp), L._stream(dev)))
    return dlogp


def _f32c(t):
    return t.to(torch.float32).contiguous()


class LoraTokenLogpFunction(torch.autograd.Function):
    """logp = LoraTokenLogpFunction.apply(logits, targets, inv_temp); gradient for logits."""

    @staticmethod
    def forward(ctx, logits, targets, inv_temp=1.0):
        logp, stats = lora_token_logp_fwd(logits, targets, inv_temp)
        ctx.save_for_backward(logits, targets, stats)
        ctx.inv_temp = inv_temp
        return logp

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogp):
        logits, targets, stats = ctx.saved_tensors
        return lora_token_logp_bwd(logits, targets, stats, _f32c(dlogp), ctx.inv_temp), None, None


class LoraHeadLogpFunction(torch.autograd.Function):
    """logp = LoraHeadLogpFunction.apply(X, W, A, B, scale, targets, inv_temp): the log-probabilities of targets under
    a LoRA head projection (W [vocab, d_in] frozen), the logits kept in X's dtype between the two; gradients for
    X, A and B."""

    @staticmethod
    def forward(ctx, X, W, A, B, scale, targets, inv_temp=1.0):
        with _on(_gpu(X)):
            logits = lora_linear_fwd(X, W, A, B, scale)
        logp, stats = lora_token_logp_fwd(logits, targets, inv_temp)
        ctx.save_for_backward(X, W, A, B, logits, targets, stats)
        ctx.scale, ctx.inv_temp = scale, inv_temp
        return logp

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogp):
        X, W, A, B, logits, targets, stats = ctx.saved_tensors
        dlogits = lora_token_logp_bwd(logits, targets, stats, _f32c(dlogp), ctx.inv_temp)
        with _on(X.device):
            dX, dA, dB = lora_linear_bwd(X, W, A, B, ctx.scale, dlogits, need_dX=ctx.needs_input_grad[0])
        return dX, None, dA.to(A.dtype), dB.to(B.dtype), None, None, None


class LoraPreferenceLossFunction(torch.autograd.Function):
    """(loss, pair_loss, rewards) = LoraPreferenceLossFunction.apply(logp, ref_logp, cu, mask, beta, kind,
    label_smoothing, average); gradient of loss for logp (the reference is frozen, the other outputs are for logs).
    logp may have any shape, its tokens in order."""

    @staticmethod
    def forward(ctx, logp, ref_logp, cu, mask, beta, kind="sigmoid", label_smoothing=0.0, average=False):
        loss, pair_loss, rewards, coef = lora_preference_loss_fwd(logp, cu, beta, ref_logp, mask, kind,
                                                                  label_smoothing, average)
        ctx.save_for_backward(cu, mask, coef)
        ctx.shape = logp.shape
        ctx.mark_non_differentiable(pair_loss, rewards)
        return loss, pair_loss, rewards

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, *_):
        cu, mask, coef = ctx.saved_tensors
        d = lora_preference_loss_bwd(coef, cu, ctx.shape.numel(), mask, _f32c(dloss))
        return (d.view(ctx.shape),) + (None,) * 7


class LoraPolicyLossFunction(torch.autograd.Function):
    """(loss, stats) = LoraPolicyLossFunction.apply(logp, old_logp, ref_logp, cu, advantages, mask, eps_low, eps_high,
    beta, reduction, norm, per_token); gradient of loss for logp, which may have any shape, its tokens in order."""

    @staticmethod
    def forward(ctx, logp, old_logp, ref_logp, cu, advantages, mask, eps_low=0.2, eps_high=0.2, beta=0.0,
                reduction="sequence", norm=1.0, per_token=False):
        loss, stats, weight = lora_policy_loss_fwd(logp, cu, advantages, old_logp, ref_logp, mask, eps_low, eps_high,
                                                   beta, reduction, norm, per_token)
        ctx.save_for_backward(logp, old_logp, ref_logp, cu, advantages, mask, weight)
        ctx.args = dict(eps_low=eps_low, eps_high=eps_high, beta=beta, per_token=per_token)
        ctx.mark_non_differentiable(stats)
        return loss, stats

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, *_):
        logp, old_logp, ref_logp, cu, advantages, mask, weight = ctx.saved_tensors
        d = lora_policy_loss_bwd(logp, cu, advantages, weight, old_logp, ref_logp, mask, dloss=_f32c(dloss), **ctx.args)
        return (d.view(logp.shape),) + (None,) * 11


# ---------------------------------------------------------------------------
# the norm in front of the projections, and activations kept in 8 bits
# ---------------------------------------------------------------------------
_F8 = (torch.float8_e4m3fn, torch.uint8)


def _rows(name, dev, t, shape, dtypes):
    """The row stride of a [M, d] tensor with contiguous rows."""
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, not on {dev}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    M, d = shape
    if d > 1 and M > 0 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.stride(0) if M > 1 else d


def lora_rmsnorm_fwd(X, weight, eps: float = 1e-5, residual=None, pack: bool = False, need_y: bool = True, H=None):
    """(Y, H, rstd, codes, scale8): H = X + residual (X itself without one), rstd = 1 / sqrt(mean(H^2) + eps) fp32 [M],
    Y = H rstd weight (None unless need_y), and Y as lora_act8_pack keeps it where pack (else None, None).  X and
    residual [M, d] may have a row stride; H, where given, receives the sum and may be X or the residual."""
    dev, same = _gpu(X), (X.dtype,)
    dt = L._dtype_code(X)
    if X.dim() != 2:
        raise ValueError("X must be [M, d]")
    M, d = X.shape
    ldx = _rows("X", dev, X, X.shape, same)
    _check(dev, "weight", weight, same, d)
    ldr = 0
    if residual is not None:
        ldr = _rows("residual", dev, residual, X.shape, same)
        if H is None:
            H = torch.empty(M, d, dtype=X.dtype, device=dev)
    if H is not None:
        _check(dev, "H", H, same, M * d)
    new = lambda t: torch.empty(M, d, dtype=t, device=dev)  # noqa: E731
    Y = new(X.dtype) if need_y else None
    codes = new(torch.float8_e4m3fn) if pack else None
    rstd = torch.empty(M, dtype=torch.float32, device=dev)
    scale8 = torch.empty(M, dtype=torch.float32, device=dev) if pack else None
    with _on(dev):
        L._check("lora_rmsnorm_fwd", L.lib().lora_rmsnorm_fwd(
            dt, M, d, float(eps), L._ptr(X), ldx, L._ptr(residual), ldr, L._ptr(weight), L._ptr(H), L._ptr(Y),
            L._ptr(codes), L._ptr(scale8), L._ptr(rstd), L._stream(dev)))
    return Y, X if H is None else H, rstd, codes, scale8


def lora_rmsnorm_bwd(H, weight, rstd, dY, dH=None, need_dX: bool = True, need_dweight: bool = True,
                     dweight_dtype=torch.float32, ws=None):
    """(dX or None, dweight or None) of lora_rmsnorm_fwd from its H and rstd; dH: the gradient of H itself, where the
    residual stream goes on.  dX is the gradient of X and of the residual."""
    dev, same = _gpu(H), (H.dtype,)
    if H.dim() != 2:
        raise ValueError("H must be [M, d]")
    M, d = H.shape
    _check(dev, "H", H, same)
    _check(dev, "weight", weight, same, d)
    _check(dev, "rstd", rstd, _F32, M)
    _check(dev, "dY", dY, same, M * d)
    if dH is not None:
        _check(dev, "dH", dH, same, M * d)
    return _rmsnorm_bwd(H, weight, rstd, dY, dH, need_dX, need_dweight, dweight_dtype, ws)


def _rmsnorm_bwd(H, weight, rstd, dY, dH, need_dX, need_dweight, dweight_dtype, ws=None):
    """lora_rmsnorm_bwd of checked tensors."""
    if not need_dX and not need_dweight:
        return None, None
    dt, dev, (M, d) = L._dtype_code(H), H.device, H.shape
    dX = torch.empty_like(H) if need_dX else None
    dw, ws_bytes = None, 0
    if need_dweight:
        dw = torch.empty(d, dtype=dweight_dtype, device=dev)
        if ws is None:
            ws_bytes = int(L.lib().lora_rmsnorm_workspace_bytes(M, d))
            ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
        else:
            ws_bytes = _check_ws(dev, ws, ws.nbytes).nbytes
    with _on(dev):
        L._check("lora_rmsnorm_bwd", L.lib().lora_rmsnorm_bwd(
            dt, M, d, L._ptr(H), L._ptr(weight), L._ptr(rstd), L._ptr(dY), L._ptr(dH), L._ptr(dX), L._ptr(dw),
            0 if dw is None else L._dtype_code(dw), L._ptr(ws), ws_bytes, L._stream(dev)))
    return dX, dw


class LoraRmsNormFunction(torch.autograd.Function):
    """(Y, H) = LoraRmsNormFunction.apply(X, residual, weight, eps, pack), or (Y, H, codes, scale8) with pack: Y the
    norm of H = X + residual, or of X where residual is None (H is then None); gradients for X, residual and weight
    from those of Y and H.  codes and scale8 keep Y in 8 bits, for LoraLinearAct8Function."""

    @staticmethod
    def forward(ctx, X, residual, weight, eps=1e-5, pack=False):
        Y, H, rstd, codes, scale8 = lora_rmsnorm_fwd(X, weight, eps, residual, pack)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(H.contiguous(), weight, rstd)
        ctx.weight = weight.shape
        H = H if residual is not None else None
        if not pack:
            return Y, H
        ctx.mark_non_differentiable(codes, scale8)
        return Y, H, codes, scale8

    @staticmethod
    @once_differentiable
    def backward(ctx, dY, dH, *_):
        need_X, need_R, need_w = ctx.needs_input_grad[:3]
        if dY is None:  # the stream alone went on
            return dH if need_X else None, dH if need_R else None, None, None, None
        # (autograd checked the gradients' type, shape and device)
        same = dY.dtype
        H, weight, rstd = _kept(ctx, dY.device, (same, dY.shape), (same, ctx.weight), (torch.float32, dY.shape[:1]))
        dX, dw = _rmsnorm_bwd(H, weight, rstd, dY.contiguous(), None if dH is None else dH.contiguous(),
                              need_X or need_R, need_w, weight.dtype)
        return dX if need_X else None, dX if need_R else None, None if dw is None else dw.view_as(weight), None, None


def lora_act8_pack(X):
    """(codes float8_e4m3fn [M, d], scale8 fp32 [M]) of X [M, d] (rows may be strided): row t is codes[t] * scale8[t],
    scale8[t] the smallest power of two that keeps the row at or below 448."""
    dev = _gpu(X)
    dt = L._dtype_code(X)
    if X.dim() != 2:
        raise ValueError("X must be [M, d]")
    M, d = X.shape
    ldx = _rows("X", dev, X, X.shape, (X.dtype,))
    codes = torch.empty(M, d, dtype=torch.float8_e4m3fn, device=dev)
    scale8 = torch.empty(M, dtype=torch.float32, device=dev)
    with _on(dev):
        L._check("lora_act8_pack", L.lib().lora_act8_pack(dt, M, d, L._ptr(X), ldx, L._ptr(codes), L._ptr(scale8),
                                                          L._stream(dev)))
    return codes, scale8


def _packed(codes, scale8, M=None):
    dev = _gpu(codes)
    if codes.dim() != 2:
        raise ValueError("codes must be [M, d]")
    _check(dev, "codes", codes, _F8, None if M is None else M * codes.shape[1])
    _check(dev, "scale8", scale8, _F32, codes.shape[0])
    return dev, codes.shape


def lora_act8_unpack(codes, scale8, dtype=torch.bfloat16):
    """codes * scale8 [M, d] in bf16 or fp32 (exact, but for bf16 values below 2^-125 and what was rounded to 2^128)."""
    dev, (M, d) = _packed(codes, scale8)
    X = torch.empty(M, d, dtype=dtype, device=dev)
    with _on(dev):
        L._check("lora_act8_unpack", L.lib().lora_act8_unpack(L._dtype_code(X), M, d, L._ptr(codes), L._ptr(scale8),
                                                              L._ptr(X), L._stream(dev)))
    return X


def lora_act8_linear_bwd(codes, scale8, member, dY, need_dX: bool = True, table16=None, grad_dtype=torch.float32,
                         ws=None):
    """(dX or None, dA, dB) of a projection whose input was kept as codes and scale8 (lora_act8_pack, or
    lora_rmsnorm_fwd with pack), for a member as lora_linear_epi_bwd takes it; dA and dB in grad_dtype."""
    dev, (M, d_in) = _packed(codes, scale8)
    A, B = member["A"], member["B"]
    if A.dim() != 2 or B.dim() != 2 or dY.dim() != 2:
        raise ValueError("shape mismatch: codes [M,d_in], W [d_out,d_in], A [r,d_in], B [d_out,r], dY [M,d_out]")
    # (a [0, d_in] tensor of the layer's type stands for X in the checks of the member)
    _, _, _, d_out, r, m = _epi_member(dY.new_empty(0, d_in), member)
    if A.shape != (r, d_in) or B.shape != (d_out, r) or dY.shape != (M, d_out):
        raise ValueError("shape mismatch: codes [M,d_in], W [d_out,d_in], A [r,d_in], B [d_out,r], dY [M,d_out]")
    _check(dev, "dY", dY, (dY.dtype,), M * d_out)
    return _act8_bwd(codes, scale8, m, dY, M, d_in, d_out, r, need_dX, table16, grad_dtype, ws)


def _act8_bwd(codes, scale8, m, dY, M, d_in, d_out, r, need_dX, table16, grad_dtype, ws=None):
    """lora_act8_linear_bwd of checked tensors."""
    dev, dt, new = dY.device, L._dtype_code(dY), torch.empty
    dX = new(M, d_in, dtype=dY.dtype, device=dev) if need_dX else None
    dA, dB = new(r, d_in, dtype=grad_dtype, device=dev), new(d_out, r, dtype=grad_dtype, device=dev)
    m.dY, m.dX, m.dA, m.dB = L._ptr(dY), L._ptr(dX), L._ptr(dA), L._ptr(dB)
    tab, gt = L._table_ptr(table16) if table16 is not None else None, L._dtype_code(dA)
    if ws is None:
        ws_bytes = L.lib().lora_act8_linear_workspace_bytes(dt, M, d_in, m, gt)
        ws = new(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    else:
        ws_bytes = _check_ws(dev, ws, ws.nbytes).nbytes
    with _on(dev):
        L._check("lora_act8_linear_bwd", L.lib().lora_act8_linear_bwd(
            dt, M, d_in, m, L._ptr(codes), L._ptr(scale8), tab, gt, L._ptr(ws), ws_bytes, L._stream(dev)))
    return dX, dA, dB


class LoraLinearAct8Function(torch.autograd.Function):
    """Y = LoraLinearAct8Function.apply(X, W, A, B, scale, codes, scale8, W_t): LoraLinearFunction that keeps its input
    in 8 bits for the backward (a quarter of fp32's bytes, half of bf16's): codes and scale8 where the caller has them
    (the norm's, one checkpoint for all the projections that read it), else X packed here.  Y and dX are those of X itself;
    dA and dB are of the kept values."""

    @staticmethod
    def forward(ctx, X, W, A, B, scale, codes=None, scale8=None, W_t=None):
        Y, _ = lora_linear_epi_fwd(X, {"W": W, "A": A, "B": B, "scale": scale, "W_t": W_t})
        if any(ctx.needs_input_grad[i] for i in (0, 2, 3)):
            if codes is None:
                codes, scale8 = lora_act8_pack(X)
            else:
                if codes.shape != X.shape or codes.device != X.device:
                    raise ValueError("codes must have X's shape and device")
                _packed(codes, scale8)
            ctx.save_for_backward(codes, scale8, W, A, B, W_t)
            ctx.dims, ctx.code, ctx.rows = (*X.shape, *B.shape), codes.dtype, scale8.shape
        ctx.scale = scale
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        same, (M, d_in, d_out, r) = dY.dtype, ctx.dims
        codes, scale8, W, A, B, W_t = _kept(ctx, dY.device, (ctx.code, (M, d_in)), (torch.float32, ctx.rows), (same, (d_out, d_in)),
                                            (same, (r, d_in)), (same, (d_out, r)), (torch.bfloat16, (d_in, d_out)))
        dY = dY.contiguous()  # (its type, shape and device are Y's)
        m = _epi_struct({"W": W, "A": A, "B": B, "scale": ctx.scale, "W_t": W_t}, r, d_out)
        need_dX, _, need_dA, need_dB = ctx.needs_input_grad[:4]
        dX, dA, dB = _act8_bwd(codes, scale8, m, dY, M, d_in, d_out, r, need_dX, None, A.dtype)
        return dX, None, dA if need_dA else None, dB if need_dB else None, None, None, None, None


# ---------------------------------------------------------------------------
# an adapter of its own for every row
# ---------------------------------------------------------------------------
_I32 = (torch.int32,)


def _multi_dims(X, W, A, B, scales, index):
    dev, same = _gpu(X), (X.dtype,)
    dt = L._dtype_code(X)
    if X.dim() != 2 or W.dim() != 2 or A.dim() != 3 or B.dim() != 3:
        raise ValueError("shape mismatch: X [M,d_in], W [d_out,d_in], A [n,r,d_in], B [n,d_out,r]")
    (M, d_in), d_out, (n, r, _) = X.shape, W.shape[0], A.shape
    if W.shape != (d_out, d_in) or A.shape != (n, r, d_in) or B.shape != (n, d_out, r):
        raise ValueError("shape mismatch: X [M,d_in], W [d_out,d_in], A [n,r,d_in], B [n,d_out,r]")
    for name, t in (("X", X), ("W", W), ("A", A), ("B", B)):
        _check(dev, name, t, same)
    _check(dev, "scales", scales, _F32, n)
    _check(dev, "index", index, _I32, M)
    return dt, dev, M, d_in, d_out, n, r


def _multi_ws(backward, dt, M, d_in, d_out, n, r, have_wt, need_dX, dev, ws):
    """(workspace, its bytes)"""
    if ws is not None:
        return _check_ws(dev, ws, ws.nbytes), ws.nbytes
    nb = int(L.lib().lora_multi_workspace_bytes(backward, dt, M, d_in, d_out, n, r, have_wt, need_dX))
    return torch.empty(max(nb, 1), dtype=torch.uint8, device=dev), nb


def lora_multi_fwd(X, W, A, B, scales, index, Y=None, ws=None):
    """Y [M, d_out]: row t is W x_t + scales[a] B[a] (A[a] x_t) with a = index[t] (int32 [M]; outside [0, n): W x_t
    alone), for n adapters A [n, r, d_in], B [n, d_out, r] and fp32 scales [n] over one frozen W [d_out, d_in]."""
    dims = _multi_dims(X, W, A, B, scales, index)
    if Y is not None:
        _check(dims[1], "Y", Y, (X.dtype,), dims[2] * dims[4])
    return _multi_fwd(dims, X, W, A, B, scales, index, Y, ws)


def _multi_fwd(dims, X, W, A, B, scales, index, Y=None, ws=None):
    """lora_multi_fwd of checked tensors."""
    dt, dev, M, d_in, d_out, n, r = dims
    if Y is None:
        Y = torch.empty(M, d_out, dtype=X.dtype, device=dev)
    ws, ws_bytes = _multi_ws(0, dt, M, d_in, d_out, n, r, 0, 0, dev, ws)
    with _on(dev):
        L._check("lora_multi_fwd", L.lib().lora_multi_fwd(
            dt, M, d_in, d_out, n, r, L._ptr(X), L._ptr(W), L._ptr(A), L._ptr(B), L._ptr(scales), L._ptr(index),
            L._ptr(Y), L._ptr(ws), ws_bytes, L._stream(dev)))
    return Y


def lora_multi_bwd(X, W, A, B, scales, index, dY, need_dX: bool = True, W_t=None, grad_dtype=torch.float32, ws=None):
    """(dX or None, dA [n, r, d_in], dB [n, d_out, r]) of lora_multi_fwd, the adapters' gradients in grad_dtype (zeros for
    an adapter without rows); W_t: W's transpose (bf16), where the caller keeps one."""
    dims = _multi_dims(X, W, A, B, scales, index)
    _, dev, M, d_in, d_out, _, _ = dims
    _check(dev, "dY", dY, (X.dtype,), M * d_out)
    _multi_wt(dev, W_t, d_in, d_out)
    return _multi_bwd(dims, X, W, A, B, scales, index, dY, need_dX, W_t, grad_dtype, ws)


def _multi_wt(dev, W_t, d_in, d_out):
    if W_t is not None:
        _check(dev, "W_t", W_t, (torch.bfloat16,), d_in * d_out)
        if W_t.shape != (d_in, d_out):
            raise ValueError("W_t must be the bf16 [d_in, d_out] transpose of W")


def _multi_bwd(dims, X, W, A, B, scales, index, dY, need_dX, W_t, grad_dtype, ws=None):
    """lora_multi_bwd of checked tensors."""
    dt, dev, M, d_in, d_out, n, r = dims
    dX = torch.empty_like(X) if need_dX else None
    dA = torch.empty(n, r, d_in, dtype=grad_dtype, device=dev)
    dB = torch.empty(n, d_out, r, dtype=grad_dtype, device=dev)
    ws, ws_bytes = _multi_ws(1, dt, M, d_in, d_out, n, r, int(W_t is not None), int(need_dX), dev, ws)
    with _on(dev):
        L._check("lora_multi_bwd", L.lib().lora_multi_bwd(
            dt, M, d_in, d_out, n, r, L._ptr(X), L._ptr(W), L._ptr(W_t), L._ptr(A), L._ptr(B), L._ptr(scales),
            L._ptr(index), L._ptr(dY), L._ptr(dX), L._ptr(dA), L._ptr(dB), L._dtype_code(dA), L._ptr(ws), ws_bytes,
            L._stream(dev)))
    return dX, dA, dB


class LoraMultiFunction(torch.autograd.Function):
    """Y = LoraMultiFunction.apply(X, W, A, B, scales, index, W_t): lora_multi_fwd with gradients for X, A and B (W frozen);
    a backward takes 2^21 rows at most."""

    @staticmethod
    def forward(ctx, X, W, A, B, scales, index, W_t=None):
        ctx.dims = dims = _multi_dims(X, W, A, B, scales, index)
        _multi_wt(dims[1], W_t, dims[3], dims[4])
        ctx.save_for_backward(X, W, A, B, scales, index, W_t)
        ctx.rows = scales.shape, index.shape
        return _multi_fwd(dims, X, W, A, B, scales, index)

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        same, (_, _, M, d_in, d_out, n, r), (ns, ni) = dY.dtype, ctx.dims, ctx.rows
        X, W, A, B, scales, index, W_t = _kept(
            ctx, dY.device, (same, (M, d_in)), (same, (d_out, d_in)), (same, (n, r, d_in)), (same, (n, d_out, r)),
            (torch.float32, ns), (torch.int32, ni), (torch.bfloat16, (d_in, d_out)))
        need_dX, _, need_dA, need_dB = ctx.needs_input_grad[:4]
        dX, dA, dB = _multi_bwd(ctx.dims, X, W, A, B, scales, index, dY.contiguous(), need_dX, W_t, X.dtype)
        return dX, None, dA if need_dA else None, dB if need_dB else None, None, None, None
