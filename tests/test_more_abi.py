"""Refusals of the norm, 8-bit and adapter-per-token entry points: validation comes before any HIP call, so no GPU is needed."""
import ctypes
import math

import pytest

import lora_linear_layers_amd as L
from lora_linear_layers_amd import _lib

OK, ENULL, ESHAPE, EALIGN, EDTYPE, EWS, EDEV = 0, -1, -2, -3, -4, -5, -6
P = 1 << 20  # an aligned address that nothing reads


def _norm(lib, dtype=1, M=4, d=64, eps=1e-5, X=P, ldx=64, R=None, ldr=0, w=P, H=None, Y=P, codes=None, s8=None, rstd=None):
    return lib.lora_rmsnorm_fwd(dtype, M, d, eps, X, ldx, R, ldr, w, H, Y, codes, s8, rstd, None)


def test_norm_validation():
    lib = L.load()
    assert _norm(lib, dtype=2) == EDTYPE
    assert _norm(lib, d=0) == ESHAPE
    assert _norm(lib, d=32769, ldx=32769) == ESHAPE
    assert _norm(lib, M=-1) == ESHAPE
    assert _norm(lib, M=1 << 31) == ESHAPE
    assert _norm(lib, ldx=63) == ESHAPE
    assert _norm(lib, R=P, ldr=63) == ESHAPE
    for eps in (-1e-9, math.nan, math.inf):
        assert _norm(lib, eps=eps) == ESHAPE
    assert _norm(lib, X=None) == ENULL
    assert _norm(lib, w=None) == ENULL
    assert _norm(lib, Y=None) == ENULL  # no output at all
    assert _norm(lib, codes=P) == ENULL
    assert _norm(lib, s8=P) == ENULL
    assert _norm(lib, X=P + 1) == EALIGN
    assert _norm(lib, dtype=0, Y=P + 2) == EALIGN
    assert _norm(lib, rstd=P + 2) == EALIGN


def test_norm_bwd_validation():
    lib = L.load()

    def call(dtype=1, M=4, d=64, H=P, w=P, rstd=P, dY=P, dH=None, dX=P, dw=None, wt=0, ws=None, n=0):
        return lib.lora_rmsnorm_bwd(dtype, M, d, H, w, rstd, dY, dH, dX, dw, wt, ws, n, None)
    assert call(dtype=5) == EDTYPE
    assert call(dw=P, wt=3, ws=P, n=1 << 30) == EDTYPE
    assert call(d=40000) == ESHAPE
    assert call(H=None) == ENULL
    assert call(rstd=None) == ENULL
    assert call(dX=None) == ENULL
    assert call(dY=P + 1) == EALIGN
    need = lib.lora_rmsnorm_workspace_bytes(4, 64)
    assert need > 0 and lib.lora_rmsnorm_workspace_bytes(-1, 64) == 0 and lib.lora_rmsnorm_workspace_bytes(4, 0) == 0
    assert call(dw=P) == EWS
    assert call(dw=P, ws=P, n=need - 1) == EWS
    assert call(dw=P, ws=P + 8, n=need) == EALIGN


def test_act8_validation():
    lib = L.load()
    assert lib.lora_act8_pack(2, 4, 64, P, 64, P, P, None) == EDTYPE
    assert lib.lora_act8_pack(1, 4, 64, P, 60, P, P, None) == ESHAPE
    assert lib.lora_act8_pack(1, 4, 64, None, 64, P, P, None) == ENULL
    assert lib.lora_act8_pack(1, 4, 64, P, 64, P, None, None) == ENULL
    assert lib.lora_act8_pack(1, 4, 64, P + 1, 64, P, P, None) == EALIGN
    assert lib.lora_act8_unpack(1, 4, 64, P, None, P, None) == ENULL
    assert lib.lora_act8_unpack(1, 4, 64, P + 4, P, P, None) == EALIGN
    assert lib.lora_act8_unpack(1, 4, 0, P, P, P, None) == ESHAPE
    member = _lib.GroupMember(32, 8, 1.0, 0, P, None, None, P, P, None, P, P, P, P, None)

    def call(m=member, dtype=1, M=4, d_in=64, codes=P, s8=P, gt=0, ws=P, n=1 << 30):
        return lib.lora_act8_linear_bwd(dtype, M, d_in, m, codes, s8, None, gt, ws, n, None)
    assert call(dtype=2) == EDTYPE
    assert call(gt=3) == EDTYPE
    assert call(d_in=12) == ESHAPE
    assert call(d_in=32776) == ESHAPE
    assert call(m=None) == ENULL
    assert call(codes=None) == ENULL
    assert call(codes=P + 8) == EALIGN
    assert call(s8=None) == ENULL
    assert call(s8=P + 2) == EALIGN
    assert call(ws=None) == EWS
    need = lib.lora_act8_linear_workspace_bytes(1, 4, 64, member, 0)
    assert need > 0 and call(n=need - 1) == EWS
    assert lib.lora_act8_linear_workspace_bytes(1, 4, 12, member, 0) == 0
    rope = _lib.GroupMember(128, 8, 1.0, 1, P, None, None, P, P, None, P, P, P, P, None)
    assert call(m=rope) == ESHAPE
    no_grad = _lib.GroupMember(32, 8, 1.0, 0, P, None, None, P, P, None, P, P, None, P, None)
    assert call(m=no_grad) == ENULL


def test_multi_validation():
    lib = L.load()

    def fwd(dtype=1, M=4, k=64, d=64, n=3, r=8, X=P, W=P, A=P, B=P, s=P, idx=P, Y=P, ws=P, nb=1 << 30):
        return lib.lora_multi_fwd(dtype, M, k, d, n, r, X, W, A, B, s, idx, Y, ws, nb, None)

    def bwd(dtype=1, M=4, n=3, W_t=None, dY=P, dX=P, dA=P, dB=P, gt=0, ws=P, nb=1 << 30):
        return lib.lora_multi_bwd(dtype, M, 64, 64, n, 8, P, P, W_t, P, P, P, P, dY, dX, dA, dB, gt, ws, nb, None)
    assert fwd(dtype=2) == EDTYPE
    for kw in (dict(k=12), dict(d=0), dict(r=0), dict(r=12), dict(r=136), dict(n=0), dict(n=4097), dict(M=-1), dict(M=1 << 31),
               dict(k=(1 << 20) + 8), dict(d=(1 << 20) + 8)):
        assert fwd(**kw) == ESHAPE, kw
    for kw in (dict(X=None), dict(W=None), dict(A=None), dict(B=None), dict(s=None), dict(idx=None), dict(Y=None)):
        assert fwd(**kw) == ENULL, kw
    for kw in (dict(X=P + 8), dict(B=P + 4), dict(s=P + 2), dict(idx=P + 1), dict(ws=P + 8)):
        assert fwd(**kw) == EALIGN, kw
    need = lib.lora_multi_workspace_bytes(0, 1, 4, 64, 64, 3, 8, 0, 0)
    assert need > 0 and fwd(nb=need - 1) == EWS and fwd(ws=None) == EWS
    assert lib.lora_multi_workspace_bytes(0, 1, 4, 64, 64, 3, 12, 0, 0) == 0
    assert bwd(gt=2) == EDTYPE
    assert bwd(dA=None) == ENULL
    assert bwd(dY=None) == ENULL
    assert bwd(W_t=P + 2) == EALIGN
    assert bwd(dX=P + 8) == EALIGN
    need = lib.lora_multi_workspace_bytes(1, 1, 4, 64, 64, 3, 8, 0, 1)
    assert bwd(nb=need - 1) == EWS
    # what the caller keeps (W^T) and does not ask for (dX) takes no room
    big = [lib.lora_multi_workspace_bytes(1, 1, 4096, 4096, 4096, 8, 16, *a) for a in ((0, 1), (1, 1), (1, 0))]
    assert big[0] >= big[1] + 2 * 4096 * 4096 and big[1] > big[2]


def test_act8_workspace_of_a_refused_gradient_type():
    lib = L.load()
    member = _lib.GroupMember(32, 8, 1.0, 0, P, None, None, P, P, None, P, P, P, P, None)
    assert lib.lora_act8_linear_workspace_bytes(1, 4, 64, member, 1) >= lib.lora_act8_linear_workspace_bytes(1, 4, 64, member, 0) > 0
    for bad in (-1, 2, 3):
        assert lib.lora_act8_linear_workspace_bytes(1, 4, 64, member, bad) == 0


def test_multi_backward_rows():
    lib = L.load()
    assert lib.lora_multi_workspace_bytes(1, 1, 1 << 21, 64, 64, 2, 8, 0, 1) > 0
    for dtype in (0, 1):
        assert lib.lora_multi_workspace_bytes(1, dtype, (1 << 21) + 1, 64, 64, 2, 8, 0, 1) == 0
        assert lib.lora_multi_workspace_bytes(0, dtype, (1 << 21) + 1, 64, 64, 2, 8, 0, 0) > 0
        assert lib.lora_multi_bwd(dtype, (1 << 21) + 1, 64, 64, 2, 8, P, P, None, P, P, P, P, P, P, P, P, 0, P, 1 << 40, None) == ESHAPE


def test_norm_in_place_needs_rows_of_the_width():
    """Outputs have rows of d elements: over an input with longer rows they would overwrite rows not yet read."""
    lib = L.load()
    X, R, far = P, P + 4096, P + 8192
    for kw in (dict(ldx=72, H=X), dict(ldx=72, Y=X), dict(R=R, ldr=72, H=R), dict(R=R, ldr=72, Y=R), dict(R=R, ldr=64, ldx=72, H=X)):
        assert _norm(lib, **{"Y": far, **kw}) == ESHAPE, kw
    # a single row, rows of d elements, or other memory: refused for the alignment of rstd alone
    for kw in (dict(ldx=72, H=X, M=1), dict(H=X), dict(ldx=72, H=far + 4096), dict(R=R, ldr=64, H=R, ldx=72), dict(Y=X)):
        assert _norm(lib, **{"Y": far, "rstd": P + 2, **kw}) == EALIGN, kw
