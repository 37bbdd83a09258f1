"""The residual RMS norm, rows kept in 8 bits and the LoRA backward that reads
them, against their definitions in 64 bits, element by element.

Tolerances, h = half a step of the type relative to the value (bf16 2^-8, fp32
2^-24), u = 2^-24.  A row's sum of squares: a thread adds up to 32 elements one
after the other, then at most 10 joins, so 42 u of a sum of positive terms, half
of that in rstd, and rstd, h rstd and (h rstd) w add 4 u: y is off by 32 u and h.
dX = rstd (g - xh c) + dH with c = mean(g xh): 48 u of every term's magnitude, and
h; dw: at most 64 rows a block, 32 blocks a thread and 32 threads in a row: 128 + 8
additions, 160 u of the sum of magnitudes, and h.  8 bits: half a step is 2^-4 of the
value, or 2^-10 of the scale below 2^-6 of it.  LoRA gradients: P and Q are rounded
once (h), a contraction of n products accumulates at most (n + 2) u."""
import math

import pytest
import torch

U = 2.0 ** -24
H = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DTYPES = [torch.bfloat16, torch.float32]
F8 = torch.float8_e4m3fn
pytestmark = pytest.mark.gpu


def _near(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((err / tol.clamp(min=1e-300)).max()))


def _randn(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def _pow2(e):
    """2^e in 64 bits, from its exponent field (a device's pow is off by a bit)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def pack64(v):
    """(codes as fp64 values, scale) of the rows of v (fp64), from the definition."""
    size = torch.where(torch.isfinite(v), v.abs(), 0.0).amax(1, keepdim=True)
    m, e = torch.frexp(size.cpu())  # size = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
    e = torch.where(size.cpu() > 0, (e - 9 + (m > 0.875)).clamp(min=-126), 0)
    scale = _pow2(e).to(v.device)
    x = v / scale
    a = x.abs()
    k = torch.floor(torch.log2(torch.where(torch.isfinite(a), a, 1.0).clamp(min=2.0 ** -6)))
    step = _pow2(k - 3)
    return torch.where(torch.isfinite(x), torch.round(x / step) * step, math.nan), scale.squeeze(1)


def _same_codes(codes, want):
    got = codes.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


def check_norm(lib, X, w, eps, res, pack, **kw):
    dt = X.dtype
    x0, r0 = X.clone(), None if res is None else res.clone()
    Y, Hh, rstd, codes, s8 = lib.lora_rmsnorm_fwd(X, w, eps, residual=res, pack=pack, **kw)
    torch.cuda.synchronize()
    h = x0.double() if r0 is None else (x0.float() + r0.float()).to(dt).double()
    if r0 is not None:
        assert torch.equal(Hh.double(), h)
    r = 1 / torch.sqrt(h.square().mean(1) + eps)
    _near(rstd, r, 24 * U * r, "rstd")
    y = h * r[:, None] * w.double()
    _near(Y, y, (32 * U + H[dt]) * y.abs() + 1e-37, "Y")
    if pack:
        c, s = pack64(y)
        # the scale of a row whose largest value lies on the border of a power of two may be either
        border = (y.abs().amax(1) / s - 448).abs() < 448 * 64 * U
        border |= (y.abs().amax(1) / s - 224).abs() < 224 * 64 * U
        assert torch.equal(s8.double()[~border], s[~border])
        got = codes.double() * s8.double()[:, None]
        half = torch.maximum(2.0 ** -4 * y.abs() * (1 + 2.0 ** -6), 2.0 ** -10 * s8.double()[:, None])
        _near(got, y, half + 32 * U * y.abs(), "codes")
        # and the nearest code but for values next to the middle of two
        assert (codes.double() != c)[~border].double().mean() < 1e-3
    return Hh, rstd


WIDTHS = [1, 7, 8, 33, 120, 128, 129, 256, 264, 512, 520, 1001, 1024, 2048, 2056, 4096, 5000, 8192, 8200, 16384, 16391, 32768]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", WIDTHS)
def test_norm_widths(lib, dtype, d):
    for M, res, pack in ((1, False, False), (5, True, True), (37, False, True)):
        X = _randn(d + M, M, d, dtype=dtype) * 3
        R = _randn(d + M + 1, M, d, dtype=dtype) if res else None
        w = 1 + 0.3 * _randn(d + M + 2, d)
        check_norm(lib, X, w.to(dtype), 1e-5, R, pack)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,pad,off", [(256, 8, 0), (4096, 64, 0), (250, 3, 1), (1024, 8, 1), (4096, 1, 0)])
def test_norm_strided_rows(lib, dtype, d, pad, off):
    M = 19
    big = [_randn(i, M, d + pad + off, dtype=dtype) for i in (1, 2)]
    X, R = (b[:, off:off + d] for b in big)
    w = _randn(3, d + 1, dtype=dtype)[1:]  # at its element's alignment only
    check_norm(lib, X, w, 1e-6, R, True)
    codes, s8 = lib.lora_act8_pack(X)
    c, s = pack64(X.double())
    _same_codes(codes, c)
    assert torch.equal(s8.double(), s)


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_in_place(lib, dtype):
    X, R, w = _randn(1, 33, 1024, dtype=dtype), _randn(2, 33, 1024, dtype=dtype), _randn(3, 1024, dtype=dtype)
    want = lib.lora_rmsnorm_fwd(X, w, residual=R, pack=True)
    for out in ("X", "R"):
        x, r = X.clone(), R.clone()
        got = lib.lora_rmsnorm_fwd(x, w, residual=r, pack=True, H=x if out == "X" else r)
        assert got[1] is (x if out == "X" else r)
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_norm_outputs_stay_inside(lib):
    """No value is written beside an output's own: every output a slice between guards."""
    M, d = 7, 1001
    for dtype in DTYPES:
        X, w = _randn(1, M, d, dtype=dtype), _randn(2, d, dtype=dtype)
        n = M * d
        H, Y = (torch.full((n + 64,), 7.0, dtype=dtype, device="cuda") for _ in range(2))
        codes = torch.full((n + 64,), 77, dtype=torch.uint8, device="cuda")
        sc, rs = (torch.full((M + 64,), 7.0, device="cuda") for _ in range(2))
        p, st = lambda t, o: t.data_ptr() + o * t.element_size(), torch.cuda.current_stream().cuda_stream  # noqa: E731
        rc = lib.lib().lora_rmsnorm_fwd(0 if dtype == torch.float32 else 1, M, d, 1e-5, X.data_ptr(), d, X.data_ptr(), d,
                                        w.data_ptr(), p(H, 32), p(Y, 32), p(codes, 32), p(sc, 32), p(rs, 32), st)
        assert rc == 0
        torch.cuda.synchronize()
        for t, k in ((H, n), (Y, n), (codes, n), (sc, M), (rs, M)):
            g = 77 if t.dtype == torch.uint8 else 7.0
            assert bool((t[:32] == g).all()) and bool((t[32 + k:] == g).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_special_rows(lib, dtype):
    d = 512
    X = _randn(1, 8, d, dtype=dtype)
    X[0] = 0
    X[1, 3] = math.inf
    X[2, 5] = math.nan
    X[3] *= 1e-20
    X[4] = 1e15
    w = torch.ones(d, dtype=dtype, device="cuda")
    Y, _, rstd, codes, s8 = lib.lora_rmsnorm_fwd(X, w, 1e-6, pack=True)
    assert bool((Y[0] == 0).all()) and bool((codes[0].float() == 0).all()) and float(s8[0]) == 1.0
    assert float(rstd[1]) == 0 and bool(torch.isnan(Y[1, 3])) and bool((Y[1, 4:] == 0).all())
    assert bool(torch.isnan(codes[1, 3].float())) and bool((codes[1, 4:].float() == 0).all())
    assert bool(torch.isnan(Y[2]).all()) and bool(torch.isnan(codes[2].float()).all()) and float(s8[2]) == 1.0
    for i in (3, 4, 5, 6, 7):
        check_norm(lib, X[i:i + 1], w, 1e-6, None, True)


def check_norm_bwd(lib, X, w, eps, dY, dH):
    dt = X.dtype
    _, Hh, rstd, _, _ = lib.lora_rmsnorm_fwd(X, w, eps)
    dX, dw = lib.lora_rmsnorm_bwd(Hh, w, rstd, dY, dH)
    only, none = lib.lora_rmsnorm_bwd(Hh, w, rstd, dY, dH, need_dweight=False)
    none2, only_w = lib.lora_rmsnorm_bwd(Hh, w, rstd, dY, dH, need_dX=False)
    torch.cuda.synchronize()
    assert none is None and none2 is None and torch.equal(only, dX) and torch.equal(only_w, dw)
    h, g, wd, r = X.double(), dY.double(), w.double(), rstd.double()[:, None]
    xh = h * r
    gw = g * wd
    c, mc = (gw * xh).mean(1, keepdim=True), (gw * xh).abs().mean(1, keepdim=True)
    want = r * (gw - xh * c)
    mag = r * (gw.abs() + xh.abs() * mc)
    if dH is not None:
        want, mag = want + dH.double(), mag + dH.double().abs()
    _near(dX, want, 48 * U * mag + H[dt] * want.abs() + 1e-37, "dX")
    _near(dw, (g * xh).sum(0), 160 * U * (g * xh).abs().sum(0) + 1e-37, "dw")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", WIDTHS)
def test_norm_gradients(lib, dtype, d):
    for M, stream in ((1, True), (37, False), (1100, True)):
        if M * d > 1 << 23:
            continue
        X, dY = _randn(d, M, d, dtype=dtype), _randn(d + 1, M, d, dtype=dtype)
        dH = _randn(d + 2, M, d, dtype=dtype) if stream else None
        check_norm_bwd(lib, X, (1 + 0.3 * _randn(d + 3, d)).to(dtype), 1e-5, dY, dH)


def test_norm_gradient_of_many_rows(lib):
    for M, d in ((65536, 128), (20000, 1000), (8192, 4096)):
        X, dY = _randn(1, M, d, dtype=torch.bfloat16), _randn(2, M, d, dtype=torch.bfloat16)
        check_norm_bwd(lib, X, _randn(3, d, dtype=torch.bfloat16), 1e-5, dY, dY)


def test_norm_gradient_in_place_and_differences(lib):
    """dX may be dH or dY; and the gradient is the forward's slope, by central differences in fp32."""
    M, d = 6, 96
    X, w, dY, dH = (_randn(i, *s) for i, s in ((1, (M, d)), (2, (d,)), (3, (M, d)), (4, (M, d))))
    _, Hh, rstd, _, _ = lib.lora_rmsnorm_fwd(X, w, 1e-5)
    dX, dw = lib.lora_rmsnorm_bwd(Hh, w, rstd, dY, dH)
    p = lambda t: t.data_ptr()  # noqa: E731
    for own in (dH.clone(), dY.clone()):
        a, b = (own, dH) if own.equal(dY) else (dY, own)
        rc = lib.lib().lora_rmsnorm_bwd(0, M, d, p(X), p(w), p(rstd), p(a), p(b), p(own), None, 0, None, 0,
                                        torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        assert torch.equal(own, dX)
    # along random directions V: sum(dY (y(X + t V) - y(X - t V))) / 2 t; curvature t^2 |V|^3 and rounding 2^-24 / t
    t = 2.0 ** -8
    for seed in range(3):
        V, v = _randn(10 + seed, M, d), _randn(20 + seed, d)
        up, dn = (lib.lora_rmsnorm_fwd(X + k * V, w + k * v, 1e-5)[0].double() for k in (t, -t))
        slope = float((dY.double() * (up - dn)).sum() / (2 * t))
        want = float((( dX - dH).double() * V.double()).sum() + (dw.double() * v.double()).sum())
        size = float(dY.double().abs().sum())
        assert abs(slope - want) <= size * (16 * t * t + 64 * U / t), (slope, want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_function(lib, dtype):
    M, d = 40, 264
    leaf = lambda i, *s: _randn(i, *s, dtype=dtype).requires_grad_()  # noqa: E731
    X, R, w = leaf(1, M, d), leaf(2, M, d), leaf(3, d)
    dY, dH = _randn(4, M, d, dtype=dtype), _randn(5, M, d, dtype=dtype)
    F = lib.LoraRmsNormFunction
    Y, Hh, codes, s8 = F.apply(X, R, w, 1e-5, True)
    torch.autograd.backward((Y, Hh), (dY, dH))
    want, ww = lib.lora_rmsnorm_bwd(Hh.detach(), w.detach(), lib.lora_rmsnorm_fwd(Hh.detach(), w.detach())[2], dY, dH)
    assert torch.equal(X.grad, want) and torch.equal(R.grad, want)
    assert torch.equal(w.grad, ww.to(dtype))
    assert X.grad.data_ptr() != R.grad.data_ptr()  # a gradient is nobody else's
    assert not codes.requires_grad and not s8.requires_grad
    # Y alone, H alone, no residual, no weight gradient
    (g,) = torch.autograd.grad(F.apply(X, R, w)[0], X, dY)
    assert torch.equal(g, lib.lora_rmsnorm_bwd(Hh.detach(), w.detach(), lib.lora_rmsnorm_fwd(Hh.detach(), w.detach())[2], dY)[0])
    g = torch.autograd.grad(F.apply(X, R, w)[1], (X, R), dH)
    assert torch.equal(g[0], dH) and torch.equal(g[1], dH)
    Y, none = F.apply(X, None, w.detach(), 1e-5)
    assert none is None
    (g,) = torch.autograd.grad(Y, X, dY)
    x = X.detach()
    assert torch.equal(g, lib.lora_rmsnorm_bwd(x, w.detach(), lib.lora_rmsnorm_fwd(x, w.detach())[2], dY)[0])


def test_norm_empty(lib):
    for dtype in DTYPES:
        X, w = torch.empty(0, 256, dtype=dtype, device="cuda"), torch.ones(256, dtype=dtype, device="cuda")
        Y, Hh, rstd, codes, s8 = lib.lora_rmsnorm_fwd(X, w, residual=X, pack=True)
        assert Y.shape == (0, 256) and codes.shape == (0, 256) and rstd.shape == (0,)
        dX, dw = lib.lora_rmsnorm_bwd(X, w, rstd, X)
        assert dX.shape == (0, 256) and bool((dw == 0).all())
        assert lib.lora_act8_pack(X)[0].shape == (0, 256)
        assert lib.lora_act8_unpack(codes, s8, dtype).shape == (0, 256)


# ---------------------------------------------------------------------------
# 8 bits
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", WIDTHS)
def test_pack_is_exact(lib, dtype, d):
    """Codes, scales and what they stand for, bit for bit, over rows of every size."""
    M = 29
    X = _randn(d, M, d) * torch.exp(12 * _randn(d + 1, M, 1))
    if d > 4:
        X[0] = 0
        X[1, 0], X[1, 1:] = 448.0, 1.0
        X[2, 0] = 449.0
        X[3, 1] = math.inf
        X[4, 2] = math.nan
        X[5] = -math.inf
        X[6, :4] = torch.tensor([464.0, 2.0 ** -6, 2.0 ** -9, 2.0 ** -10 * 1.001])
        X[7] *= 1e-38
        X[8, 0] = 3.0e38
        X[9, :2], X[9, 2:] = torch.tensor([448.0, 2.0 ** -10]), 0.0
    X = X.to(dtype)
    codes, s8 = lib.lora_act8_pack(X)
    c, s = pack64(X.double())
    assert torch.equal(s8.double(), s)
    _same_codes(codes, c)
    for out in DTYPES:
        got, want = lib.lora_act8_unpack(codes, s8, out).double(), c * s[:, None]
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        keep = want.abs() >= 2.0 ** -126  # (below, a type's own small numbers)
        keep |= want == 0
        assert torch.equal(got[keep], want[keep])


def test_every_code(lib):
    """Each of the 256 codes decodes as torch's float8 does, and packs back to itself."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(1, 256)
    ref = codes.view(F8).float()
    got = lib.lora_act8_unpack(codes, torch.ones(1, device="cuda"), torch.float32)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)) and torch.equal(torch.nan_to_num(got), torch.nan_to_num(ref))
    again, s8 = lib.lora_act8_pack(got)
    assert float(s8[0]) == 1.0
    ok = ~torch.isnan(ref)
    assert torch.equal(again.view(torch.uint8)[ok], codes[ok])


def _lora(seed, M, k, d, r, dtype):
    X = (_randn(seed, M, k) * torch.exp(_randn(seed + 9, M, 1))).to(dtype)
    W = (_randn(seed + 1, d, k) / math.sqrt(k)).to(dtype)
    A, B = (_randn(seed + 2, r, k) / math.sqrt(k)).to(dtype), (0.1 * _randn(seed + 3, d, r)).to(dtype)
    return X, W, A, B, _randn(seed + 4, M, d, dtype=dtype)


def check_act8_bwd(lib, X, W, A, B, scale, dY, member=None, Wd=None, table=None, **kw):
    dt = dY.dtype
    codes, s8 = lib.lora_act8_pack(X)
    member = member or {"W": W, "A": A, "B": B, "scale": scale}
    dX, dA, dB = lib.lora_act8_linear_bwd(codes, s8, member, dY, table16=table, **kw)
    torch.cuda.synchronize()
    c, s = pack64(X.double())
    K, w, a, b, g = c * s[:, None], (W if Wd is None else Wd).double(), A.double(), B.double(), dY.double()
    (M, k), (d, r) = K.shape, b.shape
    P, Q = scale * (K @ a.T), scale * (g @ b)
    magP, magQ = abs(scale) * (K.abs() @ a.abs().T), abs(scale) * (g.abs() @ b.abs())
    eP = H[dt] * P.abs() + (k + 4) * U * magP
    eQ = H[dt] * Q.abs() + (d + 4) * U * magQ
    want = g @ w + Q @ a
    t = eQ @ a.abs() + (d + r + 2) * U * (g.abs() @ w.abs() + magQ @ a.abs())
    if dX is not None:
        _near(dX, want, t + H[dt] * (want.abs() + t) + 1e-37, "dX")
    _near(dA, Q.T @ K, eQ.T @ K.abs() + (M + 2) * U * (magQ.T @ K.abs()) + 1e-37, "dA")
    if not kw:  # in 16 bits: the same rounded
        low = lib.lora_act8_linear_bwd(codes, s8, member, dY, table16=table, grad_dtype=torch.bfloat16)
        assert torch.equal(low[1], dA.bfloat16()) and torch.equal(low[2], dB.bfloat16())
    _near(dB, g.T @ P, g.abs().T @ eP + (M + 2) * U * (g.abs().T @ magP) + 1e-37, "dB")
    return dX, dA, dB


SHAPES = [(1, 64, 64, 8), (3, 8, 16, 1), (17, 72, 40, 5), (64, 256, 128, 16), (100, 1024, 512, 24), (128, 128, 4096, 64),
          (300, 1024, 1024, 16), (513, 512, 776, 64), (1000, 2048, 264, 128), (1025, 784, 512, 33), (700, 520, 640, 130),
          (2048, 1024, 1024, 256)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_act8_backward(lib, shape, dtype):
    X, W, A, B, dY = _lora(sum(shape), *shape, dtype)
    check_act8_bwd(lib, X, W, A, B, 0.75, dY)
    check_act8_bwd(lib, X, W, A, B, 0.75, dY, need_dX=False)


def test_act8_backward_large(lib):
    X, W, A, B, dY = _lora(5, 4096, 4096, 1024, 64, torch.bfloat16)
    one = check_act8_bwd(lib, X, W, A, B, 0.25, dY)
    two = check_act8_bwd(lib, X, W, A, B, 0.25, dY, member={"W": W, "W_t": lib.lora_transpose(W), "A": A, "B": B, "scale": 0.25})
    for a, b in zip(one[1:], two[1:]):
        assert torch.equal(a, b)


def test_act8_backward_nf4(lib):
    M, k, d, r = 600, 256, 192, 16
    X, _, A, B, dY = _lora(8, M, k, d, r, torch.bfloat16)
    g = torch.Generator().manual_seed(3)
    codes = torch.randint(0, 256, (d * k // 2,), generator=g, dtype=torch.uint8).cuda()
    absmax = (0.5 + torch.rand(d * k // 64, generator=g)).cuda() / math.sqrt(k)
    table = [(i - 7.5) / 7.5 for i in range(16)]
    W = lib.nf4_dequant(codes, absmax, table, d * k).view(d, k)
    m = {"codes": codes, "absmax": absmax, "A": A, "B": B, "scale": 0.5}
    check_act8_bwd(lib, X, None, A, B, 0.5, dY, member=m, Wd=W, table=table)


def test_act8_empty_and_refusals(lib):
    X, W, A, B, dY = _lora(1, 0, 64, 32, 8, torch.bfloat16)
    codes, s8 = lib.lora_act8_pack(X)
    dX, dA, dB = lib.lora_act8_linear_bwd(codes, s8, {"W": W, "A": A, "B": B, "scale": 1.0}, dY)
    assert dX.shape == (0, 64) and bool((dA == 0).all()) and bool((dB == 0).all())
    X, W, A, B, dY = _lora(1, 4, 64, 32, 8, torch.bfloat16)
    codes, s8 = lib.lora_act8_pack(X)
    m = {"W": W, "A": A, "B": B, "scale": 1.0}
    with pytest.raises(ValueError):
        lib.lora_act8_linear_bwd(codes[:3], s8, m, dY)
    with pytest.raises(ValueError):
        lib.lora_act8_linear_bwd(codes, s8, m, dY[:3])
    with pytest.raises(TypeError):
        lib.lora_act8_linear_bwd(X, s8, m, dY)
    with pytest.raises(TypeError):
        lib.lora_act8_linear_bwd(codes, s8, m, dY.float())
    with pytest.raises(ValueError):
        lib.lora_act8_linear_bwd(codes, s8.cpu(), m, dY)
    with pytest.raises(lib.LoraError):
        lib.lora_act8_linear_bwd(codes, s8, m, dY, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        lib.lora_act8_pack(X.half())
    with pytest.raises(ValueError):
        lib.lora_act8_pack(X.t())
    with pytest.raises(ValueError):
        lib.lora_act8_pack(X.cpu())
    with pytest.raises(lib.LoraError):
        lib.lora_act8_pack(torch.zeros(1, 32776, device="cuda"))
    with pytest.raises(ValueError):
        lib.lora_rmsnorm_fwd(X, torch.ones(63, dtype=X.dtype, device="cuda"))
    with pytest.raises(ValueError):
        lib.lora_rmsnorm_fwd(X, torch.ones(64, dtype=X.dtype, device="cuda"), residual=X[:2])
    with pytest.raises(TypeError):
        lib.lora_rmsnorm_fwd(X, torch.ones(64, device="cuda"))
    with pytest.raises(lib.LoraError):
        lib.lora_rmsnorm_fwd(X, torch.ones(64, dtype=X.dtype, device="cuda"), eps=-1.0)
    w, rstd = torch.ones(64, dtype=X.dtype, device="cuda"), torch.ones(4, device="cuda")
    with pytest.raises(ValueError):
        lib.lora_rmsnorm_bwd(X, w, rstd[:3], X)
    with pytest.raises(lib.LoraError):
        lib.lora_rmsnorm_bwd(X, w, rstd, X, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES)
def test_act8_function(lib, dtype):
    X, W, A, B, dY = _lora(3, 200, 256, 128, 16, dtype)
    X, A, B = (t.requires_grad_() for t in (X, A, B))
    Y = lib.LoraLinearAct8Function.apply(X, W, A, B, 0.5)
    Yl, _ = lib.lora_linear_epi_fwd(X.detach(), {"W": W, "A": A.detach(), "B": B.detach(), "scale": 0.5})
    assert torch.equal(Y, Yl)
    saved = Y.grad_fn.saved_tensors
    assert saved[0].dtype == F8 and all(t is None or t.data_ptr() != X.data_ptr() for t in saved)  # X itself is not kept
    Y.backward(dY)
    codes, s8 = lib.lora_act8_pack(X.detach())
    dX, dA, dB = lib.lora_act8_linear_bwd(codes, s8, {"W": W, "A": A.detach(), "B": B.detach(), "scale": 0.5}, dY)
    assert torch.equal(X.grad, dX) and torch.equal(A.grad, dA.to(dtype)) and torch.equal(B.grad, dB.to(dtype))
    # a checkpoint that the caller has
    y = lib.LoraLinearAct8Function.apply(X, W, A, B, 0.5, codes, s8)
    for g, w in zip(torch.autograd.grad(y, (X, A, B), dY), (X.grad, A.grad, B.grad)):
        assert torch.equal(g, w)
    with pytest.raises(ValueError):
        lib.LoraLinearAct8Function.apply(X, W, A, B, 0.5, codes[:100], s8[:100])


def test_block_run(lib):
    """Norm with its 8-bit output, two projections of it from one checkpoint, and back: the gradients of the block
    against 64 bits, eagerly and captured into a graph, on a stream of its own."""
    M, d, f, r = 520, 512, 768, 16
    dt = torch.bfloat16
    X, R, w = _randn(1, M, d, dtype=dt), _randn(2, M, d, dtype=dt), (1 + 0.2 * _randn(3, d)).to(dt)
    W = [(_randn(4 + i, f, d) / math.sqrt(d)).to(dt) for i in range(2)]
    A = [(_randn(6 + i, r, d) / math.sqrt(d)).to(dt) for i in range(2)]
    B = [(0.1 * _randn(8 + i, f, r)).to(dt) for i in range(2)]
    dY = [_randn(10 + i, M, f, dtype=dt) for i in range(2)]
    dHn = _randn(12, M, d, dtype=dt)

    def step():
        Y, Hh, rstd, codes, s8 = lib.lora_rmsnorm_fwd(X, w, residual=R, pack=True)
        outs, g, dsum = [], [], None
        for i in range(2):
            m = {"W": W[i], "A": A[i], "B": B[i], "scale": 0.5}
            outs.append(lib.lora_linear_epi_fwd(Y, m)[0])
            dX, dA, dB = lib.lora_act8_linear_bwd(codes, s8, m, dY[i])
            g += [dA, dB]
            dsum = dX if dsum is None else dsum + dX
        return (*outs, *g, *lib.lora_rmsnorm_bwd(Hh, w, rstd, dsum, dHn))

    want = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(other, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(3):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
    # in 64 bits, the kept values in the adapters' gradients
    h = (X.float() + R.float()).to(dt).double().requires_grad_()
    wd = w.double().requires_grad_()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-5) * wd
    K = pack64(y.detach())
    K = K[0] * K[1][:, None]
    dy = 0
    for i in range(2):
        Q, P = 0.5 * (dY[i].double() @ B[i].double()), 0.5 * (K @ A[i].double().T)
        dy = dy + dY[i].double() @ W[i].double() + Q @ A[i].double()
        for got, ref in ((want[2 + 2 * i], Q.T @ K), (want[3 + 2 * i], dY[i].double().T @ P)):
            assert float((got.double() - ref).norm() / ref.norm()) < 2.0 ** -7  # Q or P rounded, codes on a border
    gh, gw = torch.autograd.grad(y, (h, wd), dy)
    for got, ref in ((want[6], gh + dHn.double()), (want[7], gw)):
        assert float((got.double() - ref).norm() / ref.norm()) < 2.0 ** -7


def test_side_stream_does_not_need_its_own_device_guard(lib):
    """Calls run on the current stream: work queued before them there is seen."""
    X, w = _randn(1, 256, 512), torch.ones(512, device="cuda")
    want = lib.lora_rmsnorm_fwd(X * 3, w)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        Z = X.clone()
        for _ in range(3):
            torch.cuda._sleep(100000)
        Z.mul_(3)
        got = lib.lora_rmsnorm_fwd(Z, w)[0]
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_codes_are_those_of_the_exact_values(lib, dtype):
    """Among 4 million values some lie within fp32's error of the middle of two codes, and some rows' largest next to a
    power of two's border: all are rounded as the exact value is."""
    M, d = 2048, 2048
    X, R, w = _randn(1, M, d, dtype=dtype) * 3, _randn(2, M, d, dtype=dtype), (1 + 0.3 * _randn(3, d)).to(dtype)
    _, Hh, rstd, codes, s8 = lib.lora_rmsnorm_fwd(X, w, 1e-5, residual=R, pack=True)
    h = Hh.double()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + torch.tensor(1e-5).double().item()) * w.double()
    c, s = pack64(y)
    assert torch.equal(s8.double(), s)
    assert torch.equal(codes.double(), c)
    # and the other outputs are the same without them
    Y, Hp, rp, _, _ = lib.lora_rmsnorm_fwd(X, w, 1e-5, residual=R)
    assert torch.equal(Y, lib.lora_rmsnorm_fwd(X, w, 1e-5, residual=R, pack=True)[0]) and torch.equal(rp, rstd) and torch.equal(Hp, Hh)
    # rows whose largest value is 448 or 224 to 32 bits, above or below it by less
    d = 4
    X = torch.zeros(2000, d)
    X[:, 0] = torch.arange(1, 2001) / 7.0
    X = X.to(dtype).cuda()
    for target in (1.75, 1.75 * 2 ** 8):
        w = torch.full((d,), target / 2, device="cuda").to(dtype)
        _, _, _, codes, s8 = lib.lora_rmsnorm_fwd(X, w, 0.0, pack=True)
        h = X.double()
        c, s = pack64(h / torch.sqrt(h.square().mean(1, keepdim=True)) * w.double())
        near = (h[:, 0] / torch.sqrt(h.square().mean(1)) * w.double()[0] / target - 1).abs() < 1e-15  # (64 bits' own border)
        assert torch.equal(s8.double()[~near], s[~near]) and torch.equal(codes.double()[~near], c[~near])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 1001, 4096])
def test_norm_magnitudes(lib, dtype, d):
    """Rows whose squares lie outside fp32's range."""
    w = (1 + 0.3 * _randn(1, d)).to(dtype)
    X = _randn(2, 5, d) * torch.tensor([1e30, 1e-30, 3e-20, 2e19, 1e37]).cuda()[:, None]
    check_norm(lib, X.to(dtype), w, 0.0, None, True)


def test_act8_function_takes_codes_of_its_input_only(lib):
    X, W = _randn(1, 8, 64, dtype=torch.bfloat16).requires_grad_(), _randn(2, 32, 64, dtype=torch.bfloat16)
    A, B = _randn(3, 8, 64, dtype=torch.bfloat16), _randn(4, 32, 8, dtype=torch.bfloat16)
    codes, s8 = lib.lora_act8_pack(X.detach())
    f = lib.LoraLinearAct8Function.apply
    for bad in ((codes.cpu(), s8.cpu()), (codes[:7], s8[:7]), (codes, s8[:7]), (codes, s8.cpu())):
        with pytest.raises(ValueError):
            f(X, W, A, B, 0.5, *bad)
    with pytest.raises(TypeError):
        f(X, W, A, B, 0.5, codes, s8.double())


def test_more_rows_than_a_launch_takes(lib):
    """2^28 rows and some of 8: blocks of 16 rows and 256 threads, of which a launch takes fewer than 2^24.  Every output
    is that of the rows in parts, bit for bit, past 2^31 elements."""
    M, d, part = (1 << 28) + 37, 8, 1 << 25
    X = torch.randn(M, d, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda", dtype=torch.bfloat16)
    w = _randn(2, d, dtype=torch.bfloat16)
    Y, _, rstd, codes, s8 = lib.lora_rmsnorm_fwd(X, w, residual=X, pack=True)
    pc, ps = lib.lora_act8_pack(X)
    back = lib.lora_act8_unpack(pc, ps)
    bits = lambda t: t.view(torch.uint8)  # noqa: E731
    for a in range(0, M, part):
        x = X[a:a + part]
        y, _, r, c, s = lib.lora_rmsnorm_fwd(x, w, residual=x, pack=True)
        q, e = lib.lora_act8_pack(x)
        rows = slice(a, a + len(x))
        for got, want in ((Y, y), (codes, c), (pc, q), (back, lib.lora_act8_unpack(q, e))):
            assert torch.equal(bits(got[rows]), bits(want))
        for got, want in ((rstd, r), (s8, s), (ps, e)):
            assert torch.equal(got[rows], want)
    # and the parts are right where the launches meet
    x = X[-64:].float()
    h = (x + x).bfloat16().double()
    r = 1 / torch.sqrt(h.square().mean(1) + 1e-5)
    _near(rstd[-64:], r, 2 * U * r, "rstd")
    _near(Y[-64:], h * r[:, None] * w.double(), (4 * U + 2.0 ** -8) * (h * r[:, None] * w.double()).abs(), "Y")
    del X, Y, codes, pc, back
    torch.cuda.empty_cache()


def test_norm_outputs_own_their_storage(lib):
    """Every output is a tensor of its own: the codes' scales may be changed or freed without the backward's rstd."""
    X, w = _randn(1, 16, 64).requires_grad_(), _randn(2, 64)
    outs = [t for t in lib.lora_rmsnorm_fwd(X.detach(), w, residual=X.detach(), pack=True)]
    assert len({t.untyped_storage().data_ptr() for t in outs}) == len(outs)
    Y, Hh, codes, s8 = lib.LoraRmsNormFunction.apply(X, X.detach(), w, 1e-5, True)
    (want,) = torch.autograd.grad(Y, X, torch.ones_like(Y), retain_graph=True)
    s8.mul_(2)
    (got,) = torch.autograd.grad(Y, X, torch.ones_like(Y))
    assert torch.equal(got, want)


def test_norm_codes_beside_a_value_past_the_range(lib):
    """A value past fp32's range is an infinity in Y and no code, and the row's scale is that of the others, also where
    their largest lies on the border of two scales (448 2^-8 here, which 64 bits decide)."""
    big = torch.finfo(torch.float32).max
    X = torch.tensor([[1.0, 1.5, 0.25, 0.5]] * 4, device="cuda")
    r = 1 / math.sqrt((1 + 2.25 + 0.0625 + 0.25) / 4)
    for step in range(-2, 3):
        w0 = torch.tensor(1.75 / r, dtype=torch.float32).view(torch.int32).add(step).view(torch.float32)
        w = torch.tensor([float(w0), big, 1.0, 1.0], device="cuda")
        Y, _, _, codes, s8 = lib.lora_rmsnorm_fwd(X, w, 0.0, pack=True)
        assert bool(torch.isinf(Y[:, 1]).all()) and bool(torch.isnan(codes[:, 1].float()).all())
        h = X.double()
        y = h / torch.sqrt(h.square().mean(1, keepdim=True)) * w.double()
        y[:, 1] = math.inf
        c, s = pack64(y)
        assert torch.equal(s8.double(), s), (step, s8, s)
        _same_codes(codes, c)


def test_act8_backward_past_2_31_elements(lib):
    """Codes of more than 2^31 elements; dY is zero but for some rows at either end and between, whose gradients are
    those of these rows alone."""
    M, k, d, r, scale = (1 << 18) + 300, 8208, 64, 16, 0.5
    gpu = torch.Generator(device="cuda").manual_seed(4)
    X = torch.randn(M, k, generator=gpu, device="cuda", dtype=torch.bfloat16)
    codes, s8 = lib.lora_act8_pack(X)
    rows = torch.cat([torch.arange(a, a + 300, device="cuda") for a in (0, M // 2 - 7, M - 300)])
    x = X[rows]
    del X
    _, W, A, B, dy = _lora(5, 900, k, d, r, torch.bfloat16)
    dY = torch.zeros(M, d, device="cuda", dtype=torch.bfloat16)
    dY[rows] = dy
    _, dA, dB = lib.lora_act8_linear_bwd(codes, s8, {"W": W, "A": A, "B": B, "scale": scale}, dY, need_dX=False)
    c, s = pack64(x.double())
    K, a, b, g, h = c * s[:, None], A.double(), B.double(), dy.double(), 2.0 ** -8
    P, Q, mP, mQ = scale * (K @ a.T), scale * (g @ b), scale * (K.abs() @ a.abs().T), scale * (g.abs() @ b.abs())
    eP, eQ = h * P.abs() + (k + 4) * U * mP, h * Q.abs() + (d + 4) * U * mQ
    _near(dA, Q.T @ K, eQ.T @ K.abs() + 902 * U * (mQ.T @ K.abs()) + 1e-37, "dA")
    _near(dB, g.T @ P, g.abs().T @ eP + 902 * U * (g.abs().T @ mP) + 1e-37, "dB")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", WIDTHS)
def test_norm_is_as_exact_as_its_type(lib, dtype, d):
    """The bounds of sums kept in 64 bits.  The reciprocal root is off by half of the sum's error (44 additions of 2^-53)
    and by 3/2 of the square of its start's (a root and a division in 32 bits, 2^-23): below 2^-44 in all.  rstd is that
    rounded once, u; y = (h rstd) w takes two products more, 3 u and their second order, then the type's half step.  Codes
    and scales are those of the exact y, but for values that 2^-44 of themselves could bring across a border."""
    for M, scale in ((3, 1.0), (64, 1e-12), (257, 1e9)):
        X, R = ((_randn(d + M + i, M, d) * scale).to(dtype) for i in (5, 6))
        w, eps = (1 + 0.3 * _randn(d + M + 7, d)).to(dtype), 1e-6 * scale * scale
        Y, Hh, rstd, codes, s8 = lib.lora_rmsnorm_fwd(X, w, eps, residual=R, pack=True)
        h, e32 = Hh.double(), torch.tensor(eps, dtype=torch.float32).double().item()
        r = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + e32)
        y = h * r * w.double()
        _near(rstd, r[:, 0], (U + 2.0 ** -44) * r[:, 0], "rstd")
        _near(Y, y, (3.001 * U + H[dtype] * (1 + 4 * U)) * y.abs() + 1e-37, "Y")
        (c, s), (lo, sl), (hi, sh) = (pack64(y * (1 + k * 2.0 ** -44)) for k in (0, -1, 1))
        sure = (sl == sh)
        assert torch.equal(s8.double()[sure], s[sure])
        sure = sure[:, None] & (lo == hi)
        assert torch.equal(codes.double()[sure], c[sure]) and float(sure.double().mean()) > 0.999
