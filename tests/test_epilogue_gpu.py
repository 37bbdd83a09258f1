"""The LoRA linear layer with bias, activation and residual in its epilogue,
and its backward, against the definition in 64 bits, element by element.

Tolerances, h = half a step of the type relative to the value (bf16 2^-8, fp32
2^-24), u = 2^-24.  Forward: the panel P = s X A^T is rounded once (h |P| into
|B|), a contraction of n products accumulates at most (n + 2) u of the sum of
their magnitudes; the activations' slopes stay below 1.13 and their own
evaluation is off by at most 2e-5 (bf16 forms) or 16 u (fp32) of |z| + 1;
bias and residual additions add u each, the output h.  Backward: dZ is rounded
once (h) after the same evaluation error times |dY|, P and Q once each; those
go through the products' magnitudes, with the same accumulation error; the
bias gradient is summed before dZ is rounded."""
import math

import numpy as np
import pytest
import torch

from tests.helpers import int_inputs, lora_inputs

U = 2.0 ** -24
H = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
EVAL = {torch.bfloat16: 2e-5, torch.float32: 16 * 2.0 ** -24}
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
K2 = math.sqrt(2 / math.pi)


def cdf64(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2))  # (1 + erf would lose the negative tail)


def act64(z, act):
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: z * cdf64(z),
            "gelu_tanh": lambda: z * torch.sigmoid(2 * K2 * (z + 0.044715 * z ** 3))}[act]()


def grad64(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return cdf64(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    t = torch.tanh(K2 * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * K2 * (1 + 3 * 0.044715 * z * z)


def _near(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((err / tol.clamp(min=1e-300)).max()))


def _weight(lib, X, member, table):
    if "codes" not in member:
        return member["W"].double()
    n = X.shape[1] * member["B"].shape[0]
    return lib.nf4_dequant(member["codes"], member["absmax"], table, n).view(-1, X.shape[1]).double()


def check_fwd(lib, X, member, act, bias, res, table=None, out=None):
    dt = X.dtype
    r0 = None if res is None else res.clone()
    Y, Z = lib.lora_linear_epi_fwd(X, member, act, bias, res, table, Y=out, store_z=True)
    Y2, none = lib.lora_linear_epi_fwd(X, member, act, bias, r0, table)
    torch.cuda.synchronize()
    assert none is None and torch.equal(Y, Y2)  # keeping Z changes nothing
    x, w, a, b, s = X.double(), _weight(lib, X, member, table), member["A"].double(), member["B"].double(), member["scale"]
    P = s * (x @ a.T)
    z = x @ w.T + P @ b.T
    n = X.shape[1] + a.shape[0] + 2
    magP = abs(s) * (x.abs() @ a.abs().T)
    tz = n * U * (x.abs() @ w.abs().T + magP @ b.abs().T) + (H[dt] * P.abs() + n * U * magP) @ b.abs().T
    if bias is not None:
        z = z + bias.double()
        tz = tz + U * z.abs()
    _near(Z, z, tz + H[dt] * z.abs() + 1e-37, "Z")
    y = act64(z, act)
    ty = 1.13 * tz + (EVAL[dt] * (z.abs() + 1) if act not in ("none", "relu") else 0)
    if r0 is not None:
        y = y + r0.double()
        ty = ty + U * y.abs()
    _near(Y, y, ty + H[dt] * (y.abs() + ty) + 1e-37, "Y")
    return Z


def check_bwd(lib, X, member, dY, act, Z, table=None):
    dt = X.dtype
    dX, dA, dB, db = lib.lora_linear_epi_bwd(X, member, dY, act, Z, need_dbias=True, table16=table)
    torch.cuda.synchronize()
    x, w, a, b, s = X.double(), _weight(lib, X, member, table), member["A"].double(), member["B"].double(), member["scale"]
    (M, k), (d, r) = x.shape, b.shape
    g = dY.double()
    dz, e = g, torch.zeros_like(g)
    if act != "none":
        dz = g * grad64(Z.double(), act)
        e = (EVAL[dt] * g.abs() * (Z.double().abs() + 1) if act != "relu" else 0) + U * dz.abs()
    ez = e + (H[dt] * (dz.abs() + e) if act != "none" else 0)
    _near(db, dz.sum(0), (e + (M + 2) * U * dz.abs()).sum(0) + 1e-37, "dbias")
    P, Q = s * (x @ a.T), s * (dz @ b)
    magP, magQ = abs(s) * (x.abs() @ a.abs().T), abs(s) * (dz.abs() @ b.abs())
    eP = H[dt] * P.abs() + (k + 2) * U * magP
    eQ = abs(s) * (ez @ b.abs()) + H[dt] * Q.abs() + (d + 2) * U * magQ
    dXr = dz @ w + Q @ a
    tX = ez @ w.abs() + eQ @ a.abs() + (d + r + 2) * U * (dz.abs() @ w.abs() + magQ @ a.abs())
    _near(dX, dXr, tX + H[dt] * (dXr.abs() + tX) + 1e-37, "dX")
    _near(dA, Q.T @ x, eQ.T @ x.abs() + (M + 2) * U * (Q.abs().T @ x.abs()) + 1e-37, "dA")
    _near(dB, dz.T @ P, ez.T @ P.abs() + (dz.abs() + ez).T @ eP + (M + 2) * U * (dz.abs().T @ P.abs()) + 1e-37, "dB")
    return db


def _inputs(seed, M, k, d, r, dtype):
    X, W, A, B, dY = lora_inputs(seed, M, k, d, r, dtype)
    g = torch.Generator().manual_seed(seed)
    bias = (torch.randn(d, generator=g) * 0.5).to(X.dtype).cuda()
    res = torch.randn(M, d, generator=g).to(X.dtype).cuda()
    return X, {"W": W, "A": A, "B": B, "scale": 16.0 / r}, bias, res, dY


def _nf4(seed, k, d, r, M):
    X, _, A, B, dY = lora_inputs(seed, M, k, 8, r, "bf16")
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (d * k // 2,), generator=g, dtype=torch.uint8).cuda()
    absmax = ((torch.rand(d * k // 64, generator=g) + 0.5) / math.sqrt(k)).cuda()
    B = (torch.randn(d, r, generator=g) * math.sqrt(0.02)).bfloat16().cuda()
    table = [float(v) for v in np.linspace(-1, 1, 16)]
    bias = (torch.randn(d, generator=g) * 0.5).bfloat16().cuda()
    res = torch.randn(M, d, generator=g).bfloat16().cuda()
    dY = torch.randn(M, d, generator=g).bfloat16().cuda()
    return X, {"codes": codes, "absmax": absmax, "A": A, "B": B, "scale": 16.0 / r}, bias, res, dY, table


def _kinds(fn):
    from lora_linear_layers_amd import _lib

    _lib.profile_begin(64)
    try:
        fn()
        torch.cuda.synchronize()
        return set(_lib.profile_report())
    finally:
        _lib.profile_end()


# (M, d_in, d_out, r, the launch that applies the epilogue)
BF16 = [
    (1, 4096, 14336, 16, "few_fwd"), (33, 256, 512, 64, "few_fwd"), (64, 128, 192, 24, "few_fwd"),
    (1, 64, 64, 8, "skinny_fwd"), (16, 1000, 136, 8, "skinny_fwd"), (5, 4096, 12296, 16, "skinny_fwd"),
    (61, 72, 12296, 48, "skinny_fwd"), (40, 512, 768, 5, "split_finish"), (100, 1024, 2048, 16, "split_finish"),
    (129, 520, 136, 3, "split_finish"), (1, 8, 8, 1, "gemm_bf16_128x128_nt_epi"),
    (300, 264, 392, 16, "gemm_bf16_128x128_nt_epi"), (2049, 264, 4104, 12, "gemm_bf16_128x128_nt_epi"),
    # 256 x 256 tiles, ragged or no multiple of the CUs: a block each; two blocks each; whole rounds and two blocks
    # for each of the rest; the ragged tile alone in its column
    (2049, 1024, 4104, 100, "gemm_bf16_256x256_nt_stream"), (2048, 14336, 2056, 100, "gemm_bf16_256x256_nt_stream"),
    (4100, 1600, 4104, 8, "gemm_bf16_256x256_nt_stream"), (4353, 64, 4104, 1, "gemm_bf16_256x256_nt_stream"),
    (2048, 14400, 2048, 24, "gemm_bf16_256x256_nt_stream"),
    # 128 x 256 tiles: whole, ragged in either direction, one row or one group of columns in the last, ranks of two
    # stages, the fewest stages
    (2048, 3200, 2048, 24, "gemm_bf16_128x256_nt_epi"), (2048, 3136, 2056, 16, "gemm_bf16_128x256_nt_epi"),
    (1153, 512, 4096, 3, "gemm_bf16_128x256_nt_epi"), (700, 1024, 4360, 100, "gemm_bf16_128x256_nt_epi"),
    (257, 448, 21512, 8, "gemm_bf16_128x256_nt_epi"), (384, 512, 4088, 256, "gemm_bf16_128x256_nt_epi"),
    (2047, 448, 4096, 1, "gemm_bf16_128x256_nt_epi"),
    # a last stage of 8, 56, 24 columns
    (700, 1032, 4360, 100, "gemm_bf16_128x256_nt_epi"), (2047, 504, 4096, 1, "gemm_bf16_128x256_nt_epi"),
    (2049, 1080, 4104, 100, "gemm_bf16_256x256_nt_stream"), (4100, 1592, 4104, 8, "gemm_bf16_256x256_nt_stream"),
    (4096, 72, 4104, 256, "gemm_bf16_256x256_nt_stream"), (2048, 14344, 2056, 100, "gemm_bf16_256x256_nt_stream"),
    (4090, 136, 4096, 12, "gemm_bf16_256x256_nt_epi"), (4096, 320, 4096, 72, "gemm_bf16_256x256_nt_epi"),
]
F32 = [
    (1, 8, 8, 1, "tiny_f32"), (128, 256, 256, 8, "tiny_f32"), (33, 72, 40, 3, "tiny_f32"),
    (1000, 520, 392, 24, "gemm_f32_64x128_nt_epi"), (33, 520, 1032, 64, "gemm_f32_64x128_nt_epi"),
    (107, 8704, 384, 32, "gemm_f32_64x128_nt_split"), (79, 1096, 1216, 5, "gemm_f32_64x128_nt_split"),
    (2, 2024, 7144, 16, "gemm_f32_64x128_nt_split"), (700, 1024, 256, 256, "gemm_f32_64x128_nt_split"),
    (1, 4104, 8, 1, "gemm_f32_64x128_nt_split"),
]
NF4 = [
    (1, 512, 384, 16, "few_fwd"), (128, 256, 256, 64, "few_fwd"), (200, 512, 1024, 16, "split_finish"),
    (300, 128, 11008, 8, "gemm_nf4_128x128_nt_epi"), (300, 64, 32768, 12, "gemm_nf4_256x256_nt_epi"),
    (700, 192, 640, 16, "gemm_bf16_128x128_nt_epi"), (2048, 256, 4096, 64, "gemm_nf4_256x256_nt_whole_epi"),
]
_id = lambda c: "%dx%dx%dr%d" % c[:4]  # noqa: E731


@pytest.mark.gpu
@pytest.mark.parametrize("case", BF16, ids=_id)
def test_epilogue_bf16(lib, case):
    M, k, d, r, kind = case
    X, m, bias, res, dY = _inputs(100 + M + d, M, k, d, r, "bf16")
    act = ACTS[(M + d // 8) % 5]
    kinds = _kinds(lambda: lib.lora_linear_epi_fwd(X, m, act, bias, res))
    assert kind in kinds, kinds
    Z = check_fwd(lib, X, m, act, bias, res)
    check_bwd(lib, X, m, dY, act, Z)
    check_fwd(lib, X, m, "gelu" if act != "gelu" else "silu", None, res)


@pytest.mark.gpu
@pytest.mark.parametrize("case", F32, ids=_id)
def test_epilogue_f32(lib, case):
    M, k, d, r, kind = case
    X, m, bias, res, dY = _inputs(200 + M + d, M, k, d, r, "f32")
    for act in ("silu", "gelu"):
        kinds = _kinds(lambda: lib.lora_linear_epi_fwd(X, m, act, bias, res))
        assert kind in kinds, kinds
        Z = check_fwd(lib, X, m, act, bias, res)
        check_bwd(lib, X, m, dY, act, Z)


@pytest.mark.gpu
@pytest.mark.parametrize("case", NF4, ids=_id)
def test_epilogue_nf4(lib, case):
    M, k, d, r, kind = case
    X, m, bias, res, dY, table = _nf4(300 + M, k, d, r, M)
    kinds = _kinds(lambda: lib.lora_linear_epi_fwd(X, m, "silu", bias, res, table))
    assert kind in kinds, kinds
    Z = check_fwd(lib, X, m, "silu", bias, res, table)
    check_bwd(lib, X, m, dY, "silu", Z, table)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,res", [(True, True), (True, False), (False, True), (False, False)])
def test_epilogue_forms(lib, dtype, act, bias, res):
    X, m, b, R, dY = _inputs(7, 70, 264, 136, 8, dtype)
    Z = check_fwd(lib, X, m, act, b if bias else None, R if res else None)
    check_bwd(lib, X, m, dY, act, Z)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
def test_epilogue_activation_values(lib, dtype, act):
    # the activation alone over its whole range: W = I, no adapter contribution, so Z = X
    d = 256
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    z = torch.cat([torch.linspace(-12, 12, 300 * d - 8), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 60.0, -60.0, 1e4, -1e4])])
    X = z.view(300, d).to(dt).cuda()
    m = {"W": torch.eye(d).to(dt).cuda(), "A": torch.zeros(8, d, dtype=dt, device="cuda"),
         "B": torch.zeros(d, 8, dtype=dt, device="cuda"), "scale": 1.0}
    Y, Z = lib.lora_linear_epi_fwd(X, m, act, store_z=True)
    assert torch.equal(Z, X)
    want = act64(X.double(), act)
    # relative to the value wherever it is a normal number: the negative tails keep their digits
    tol = (EVAL[dt] * (1 + (X.double() ** 2)) + H[dt]) * want.abs() + 2.0 ** -120
    _near(Y, want, tol, act)
    g = torch.ones_like(X)
    dX, _, _, _ = lib.lora_linear_epi_bwd(X, m, g, act, Z)
    dz = grad64(X.double(), act)
    _near(dX, dz, EVAL[dt] * (X.double().abs() + 1) * (act not in ("none", "relu")) + 2 * H[dt] * dz.abs() + 1e-37, act)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_epilogue_activation_of_huge_values(lib, dtype):
    # the activations' limits at values whose square or cube is no fp32 number: z or 0, slope 1 or 0
    X = torch.zeros(8, 64, dtype=dtype, device="cuda")
    X.view(-1)[:12] = torch.tensor([1e9, 1e13, 1e20, 3e38, 500.0, 95.0, -1e9, -1e13, -1e20, -3e38, -500.0, -120.0])
    m = {"W": torch.eye(64, dtype=dtype, device="cuda"), "A": torch.zeros(8, 64, dtype=dtype, device="cuda"),
         "B": torch.zeros(64, 8, dtype=dtype, device="cuda"), "scale": 1.0}
    for act in ACTS:
        if act == "none":
            continue
        Y, Z = lib.lora_linear_epi_fwd(X, m, act, store_z=True)
        dX, _, _, _ = lib.lora_linear_epi_bwd(X, m, torch.ones_like(X), act, Z)
        y, d, x = Y.view(-1)[:12].double(), dX.view(-1)[:12].double(), X.view(-1)[:12].double()
        up = x > 0
        assert torch.equal(y[up], x[up]) and (y[~up].abs() <= 1e-37).all(), act
        assert (d[up] == 1).all() and (d[~up].abs() <= 1e-37).all(), (act, d)


@pytest.mark.gpu
def test_epilogue_exact_on_integers(lib):
    # small integers: every product, sum, relu and residual is exact, on every kind of tile
    for M, k, d, r in ((4096, 64, 4096, 8), (2050, 1024, 4104, 8), (2048, 3200, 2056, 8), (4100, 1600, 4104, 8), (1, 128, 8192, 32), (300, 264, 392, 16), (40, 512, 768, 5), (9, 64, 64, 8)):
        X, W, A, B, R = int_inputs(5 + M, M, k, d, r, "bf16")
        X = X * (torch.rand(M, k, generator=torch.Generator().manual_seed(M)) < 0.2).cuda()  # |Z| stays below 2^8
        A = A * (torch.arange(k, device="cuda") % 32 == 0)
        bias = R[0].contiguous()
        z = X.double() @ W.double().T + (X.double() @ A.double().T) @ B.double().T + bias.double()
        y = z.clamp(min=0) + R.double()
        keep = (z.abs() <= 256) & (y.abs() <= 256)
        Y, Z = lib.lora_linear_epi_fwd(X, {"W": W, "A": A, "B": B, "scale": 1.0}, "relu", bias, R, store_z=True)
        assert keep.double().mean() > 0.99
        assert torch.equal(Z.double()[keep], z[keep]) and torch.equal(Y.double()[keep], y[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("case", [c for c in BF16 if c[0] in (1, 5, 40, 300, 700, 1153, 2048, 2049, 4090, 4096, 4100)], ids=_id)
def test_epilogue_residual_in_place_and_rows_behind(lib, case):
    M, k, d, r, _ = case
    X, m, bias, res, _ = _inputs(31, M, k, d, r, "bf16")
    buf = torch.full((M + 3, d), 9.0, dtype=X.dtype, device="cuda")
    buf[:M] = res
    want, _ = lib.lora_linear_epi_fwd(X, m, "silu", bias, res)
    got, _ = lib.lora_linear_epi_fwd(X, m, "silu", bias, buf[:M], Y=buf[:M])
    assert torch.equal(got, want) and (buf[M:] == 9).all()


@pytest.mark.gpu
def test_epilogue_plain_layer_bit_for_bit(lib):
    # with nothing in the epilogue it is the layer
    for dtype, M, k, d, r in (("bf16", 4096, 256, 4096, 16), ("bf16", 300, 264, 392, 16), ("bf16", 1, 4096, 14336, 16),
                              ("bf16", 9, 264, 136, 8), ("bf16", 100, 1024, 2048, 16), ("f32", 128, 256, 256, 8),
                              ("f32", 1000, 520, 392, 24)):
        X, m, _, _, dY = _inputs(17, M, k, d, r, dtype)
        Y, _ = lib.lora_linear_epi_fwd(X, m)
        assert torch.equal(Y, lib.lora_linear_fwd(X, m["W"], m["A"], m["B"], m["scale"]))
        got = lib.lora_linear_epi_bwd(X, m, dY)
        want = lib.lora_linear_bwd(X, m["W"], m["A"], m["B"], m["scale"], dY)
        assert all(torch.equal(a, b) for a, b in zip(got[:3], want)) and got[3] is None


@pytest.mark.gpu
@pytest.mark.parametrize("k", [64, 72])  # 256 x 256 tiles of whole stages, with a ragged one
def test_epilogue_offsets_past_32_bits(lib, k):
    # 2^31 elements of Y, Z, the residual, dY and dZ and more, in small integers: every sum is exact whatever its
    # order, so the rows at both ends are those of the same rows alone
    M, d, r = 140003, 16384, 8
    gen = torch.Generator("cuda").manual_seed(k)
    draw = lambda *n: torch.randint(-2, 3, n, generator=gen, device="cuda", dtype=torch.int8).bfloat16()  # noqa: E731
    X, R, dY, bias = draw(M, k), draw(M, d), draw(M, d), draw(d)
    m = {"W": draw(d, k), "A": draw(r, k), "B": draw(d, r), "scale": 1.0}
    Y, Z = lib.lora_linear_epi_fwd(X, m, "relu", bias, R, store_z=True)
    dX, dA, dB, db = lib.lora_linear_epi_bwd(X, m, dY, "relu", Z, need_dbias=True)
    for at in (slice(0, 40), slice(131060, 131090), slice(M - 40, M)):  # (131072 x 16384 = 2^31)
        y, z = lib.lora_linear_epi_fwd(X[at], m, "relu", bias, R[at], store_z=True)
        dx = lib.lora_linear_epi_bwd(X[at], m, dY[at], "relu", z)[0]
        assert torch.equal(Y[at], y) and torch.equal(Z[at], z) and torch.equal(dX[at], dx)
    P = X.float() @ m["A"].float().T  # below 2^9, exact
    dZ = dY * (Z > 0)
    sums, mags = torch.zeros(d, r + 1, device="cuda", dtype=torch.float64), torch.zeros(d, r, device="cuda", dtype=torch.float64)
    for i in range(0, M, 20000):
        g, p = dZ[i:i + 20000].double().T.contiguous(), P[i:i + 20000].bfloat16().double()
        sums += g @ torch.cat([p, torch.ones_like(p[:, :1])], 1)
        mags += g.abs() @ p.abs()
    assert mags.max() < 2 ** 24  # (fp32 sums of integers: exact)
    assert torch.equal(db.double(), sums[:, r]) and torch.equal(dB.double(), sums[:, :r]) and dA.isfinite().all()


@pytest.mark.gpu
def test_epilogue_not_finite(lib):
    X, m, bias, res, _ = _inputs(3, 12, 64, 64, 8, "bf16")
    res[3, 5], res[4, 6], bias[7] = float("nan"), float("inf"), -float("inf")
    for act in ("none", "relu", "silu"):
        Y, _ = lib.lora_linear_epi_fwd(X, m, act, bias, res)
        ok = torch.ones_like(Y, dtype=torch.bool)
        ok[3, 5] = ok[4, 6] = False
        ok[:, 7] = False
        assert Y[ok].isfinite().all() and Y[3, 5].isnan() and Y[4, 6] == float("inf")
    X[2, 0] = float("nan")
    Y, _ = lib.lora_linear_epi_fwd(X, m, "relu", None, None)
    assert Y[2].isnan().all() and Y[:2].isfinite().all() and Y[3:].isfinite().all()


@pytest.mark.gpu
def test_epilogue_no_tokens(lib):
    X, m, bias, res, dY = _inputs(4, 1, 64, 64, 8, "bf16")
    Y, Z = lib.lora_linear_epi_fwd(X[:0], m, "silu", bias, res[:0], store_z=True)
    assert Y.shape == (0, 64)
    dX, dA, dB, db = lib.lora_linear_epi_bwd(X[:0], m, dY[:0], "silu", Z, need_dbias=True)
    assert dX.shape == (0, 64) and (dA == 0).all() and (dB == 0).all() and (db == 0).all()


# dX on the tiles of the forward above: through the caller's W^T, through one made on the way, through an NF4 W
BIG, LOW = "gemm_bf16_256x256_nt_stream", "gemm_bf16_128x256_nt_epi"
DX = [(2048, 2056, 14400, 16, True, BIG), (4100, 4104, 1600, 8, False, BIG), (4100, 4104, 1600, 8, True, BIG),
      (2049, 4104, 2112, 24, False, BIG), (2304, 4096, 2112, 64, None, BIG),
      (2048, 2056, 3136, 16, True, LOW), (2048, 2056, 3200, 16, False, LOW), (700, 4360, 1024, 100, False, LOW),
      (1153, 4096, 448, 3, True, LOW), (640, 4096, 512, 8, None, LOW), (384, 4088, 1024, 24, True, LOW),
      (2049, 4096, 4104, 24, False, BIG), (700, 4096, 1032, 16, False, LOW)]


@pytest.mark.gpu
@pytest.mark.parametrize("case", DX, ids=lambda c: "%dx%dx%dr%d-%s" % c[:5])
def test_epilogue_input_gradient_tiles(lib, case):
    M, k, d, r, kept, kind = case
    table = None
    if kept is None:
        X, m, _, _, dY, table = _nf4(40 + M, k, d, r, M)
    else:
        X, m, _, _, dY = _inputs(40 + M, M, k, d, r, "bf16")
        if kept:
            m["W_t"] = lib.lora_transpose(m["W"])
    Z = torch.randn(M, d, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    kinds = _kinds(lambda: lib.lora_linear_epi_bwd(X, m, dY, "silu", Z, table16=table))
    assert kind in kinds, kinds
    check_bwd(lib, X, m, dY, "silu", Z, table)


@pytest.mark.gpu
def test_epilogue_kept_transpose_of_w(lib):
    X, m, _, _, dY = _inputs(6, 4096, 4096, 256, 16, "bf16")
    Z = torch.randn(4096, 256, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    a = lib.lora_linear_epi_bwd(X, m, dY, "silu", Z, need_dbias=True)
    b = lib.lora_linear_epi_bwd(X, dict(m, W_t=lib.lora_transpose(m["W"])), dY, "silu", Z, need_dbias=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 4096, 14336, 16), (300, 264, 392, 16), (4096, 128, 4096, 16),
                                   (2048, 3200, 2056, 24), (4100, 1600, 4104, 8)], ids=str)
def test_epilogue_repeats_other_stream_and_captured(lib, shape):
    M, k, d, r = shape
    X, m, bias, res, dY = _inputs(8, M, k, d, r, "bf16")

    def step():
        Y, Z = lib.lora_linear_epi_fwd(X, m, "silu", bias, res, store_z=True)
        return (Y, Z) + lib.lora_linear_epi_bwd(X, m, dY, "silu", Z, need_dbias=True)

    first = step()
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        X.mul_(0.5)
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held))


@pytest.mark.gpu
def test_epilogue_function_gradient_against_differences(lib):
    X, m, bias, res, dY = _inputs(9, 5, 16, 8, 2, "f32")
    for act in ("silu", "gelu", "gelu_tanh"):
        leaves = [t.clone().requires_grad_() for t in (X, m["A"], m["B"], bias, res)]
        lib.LoraLinearEpiFunction.apply(leaves[0], m["W"], leaves[1], leaves[2], leaves[3], leaves[4], m["scale"],
                                        act).backward(dY)
        base = [t.detach().double() for t in leaves]

        def loss(v):
            z = v[0] @ m["W"].double().T + m["scale"] * (v[0] @ v[1].T) @ v[2].T + v[3]
            return float(((act64(z, act) + v[4]) * dY.double()).sum())

        for i, t in enumerate(base):
            for j in range(0, t.numel(), max(1, t.numel() // 7)):
                up, dn = [v.clone() for v in base], [v.clone() for v in base]
                up[i].view(-1)[j] += 1e-5
                dn[i].view(-1)[j] -= 1e-5
                num = (loss(up) - loss(dn)) / 2e-5
                assert abs(float(leaves[i].grad.view(-1)[j]) - num) <= 2e-5 * (1 + abs(num)), (act, i, j)


@pytest.mark.gpu
def test_block_head_and_policy_loss(lib):
    """A block and its head as they are used: up projection with bias and SiLU, down projection added to its input, head,
    log-probabilities, policy loss, and back to every adapter, against the same step in 64 bits."""
    d, f, V, r, lens = 128, 264, 520, 8, [30, 1, 0, 44]
    n = sum(lens)
    X, up, b1, _, _ = _inputs(1, n, d, f, r, "f32")
    _, down, b2, _, _ = _inputs(2, n, f, d, r, "f32")
    _, head, _, _, _ = _inputs(3, n, d, V, r, "f32")
    gen = torch.Generator().manual_seed(4)
    t = torch.randint(0, V, (n,), generator=gen).cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), device="cuda")
    adv = torch.tensor([0.8, -0.5, 1.0, -1.1], device="cuda")
    mask = (torch.rand(n, generator=gen) > 0.2).cuda()

    def params():
        return [v.clone() for m in (up, down, head) for v in (m["A"], m["B"])] + [b1.clone(), b2.clone(), X.clone()]

    p = [v.requires_grad_() for v in params()]
    E = lib.LoraLinearEpiFunction.apply
    h = E(p[8], up["W"], p[0], p[1], p[6], None, up["scale"], "silu")
    y = E(h, down["W"], p[2], p[3], p[7], p[8], down["scale"], "none")
    lp = lib.LoraHeadLogpFunction.apply(y, head["W"], p[4], p[5], head["scale"], t)
    noise = 0.3 * torch.randn(n, generator=gen).cuda()
    old = (lp + noise).detach()
    ref = (lp - noise).detach()
    loss, stats = lib.LoraPolicyLossFunction.apply(lp, old, ref, cu, adv, mask, 0.2, 0.2, 0.05, "sequence")
    loss.backward()

    q = [v.detach().cpu().double().requires_grad_() for v in params()]
    W = [m["W"].cpu().double() for m in (up, down, head)]
    lin = lambda x, i, a, b, s: x @ W[i].T + s * (x @ a.T) @ b.T  # noqa: E731
    h = lin(q[8], 0, q[0], q[1], up["scale"]) + q[6]
    y = lin(h * torch.sigmoid(h), 1, q[2], q[3], down["scale"]) + q[7] + q[8]
    z = lin(y, 2, q[4], q[5], head["scale"])
    l64 = torch.log_softmax(z, 1).gather(1, t.cpu()[:, None]).squeeze(1)
    x = l64 - old.cpu().double()
    A = adv.cpu().double()[torch.repeat_interleave(torch.arange(4), torch.tensor(lens))]
    c = x.clamp(math.log1p(-0.2), math.log1p(0.2))
    # (no token may sit at its border within the layers' own error)
    assert min((x - math.log1p(-0.2)).abs().min(), (x - math.log1p(0.2)).abs().min()) > 1e-4
    dd = ref.cpu().double() - l64
    per = (-torch.minimum(x.exp() * A, c.exp() * A) + 0.05 * (dd.exp() - dd - 1)) * mask.cpu()
    o = cu.cpu()
    want = sum(per[o[i]:o[i + 1]].sum() / max(1, int(mask[o[i]:o[i + 1]].sum())) for i in range(4)) / 4
    want.backward()
    # fp32 through three layers: the layers' bar of 1e-5 of the largest value, each
    assert abs(float(loss.detach()) - float(want.detach())) <= 3e-5 * (1 + abs(float(want.detach())))
    for a, b in zip(p, q):
        assert (a.grad.cpu().double() - b.grad).abs().max() <= 3e-5 * b.grad.abs().max()


@pytest.mark.gpu
@pytest.mark.parametrize("k", [3200, 14400])
def test_epilogue_two_calls_at_once(lib, k):
    # the same layer twice on two streams, each call with its own workspace (slots and counters of the split tiles)
    X, m, bias, res, dY = _inputs(12, 2048, k, 2048, 24, "bf16")
    m["W_t"] = lib.lora_transpose(m["W"])

    def step():
        Y, Z = lib.lora_linear_epi_fwd(X, m, "silu", bias, res, store_z=True)
        return (Y, Z) + lib.lora_linear_epi_bwd(X, m, dY, "silu", Z, need_dbias=True)

    want = step()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        for st in streams:
            with torch.cuda.stream(st):
                got.append(step())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(want, g))


@pytest.mark.gpu
def test_epilogue_function_with_kept_transpose(lib):
    X, m, bias, res, dY = _inputs(13, 300, 264, 136, 8, "bf16")
    out = []
    for wt in (None, lib.lora_transpose(m["W"])):
        leaves = [t.clone().requires_grad_() for t in (X, m["A"], m["B"], bias, res)]
        Y = lib.LoraLinearEpiFunction.apply(leaves[0], m["W"], *leaves[1:], m["scale"], "silu", wt)
        out.append([Y] + list(torch.autograd.grad(Y, leaves, dY)))
    assert all(torch.equal(a, b) for a, b in zip(*out))
    assert torch.equal(out[0][5], dY)  # the residual's gradient


def test_calls_run_on_their_tensors_device(monkeypatch):
    from lora_linear_layers_amd import functional as F

    now, seen = [0], []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "set_device", lambda i: (now.__setitem__(0, i), seen.append(i)))
    with F._on(torch.device("cuda:0")):
        assert now == [0]
    assert seen == []
    with pytest.raises(RuntimeError), F._on(torch.device("cuda:3")):
        assert now == [3]
        raise RuntimeError
    assert now == [0] and seen == [3, 0]


@pytest.mark.gpu
def test_host_workspaces_are_refused(lib):
    X, m, _, _, dY = _inputs(3, 12, 64, 64, 8, "bf16")
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    lp, cu = torch.zeros(4, device="cuda"), torch.tensor([0, 2, 4], device="cuda")
    for call in (lambda: lib.lora_linear_epi_fwd(X, m, ws=ws), lambda: lib.lora_linear_epi_bwd(X, m, dY, ws=ws),
                 lambda: lib.lora_preference_loss_fwd(lp, cu, 0.1, ws=ws),
                 lambda: lib.lora_policy_loss_fwd(lp, cu, torch.zeros(2, device="cuda"), ws=ws)):
        with pytest.raises(ValueError, match="ws is on cpu"):
            call()


def test_workspace_of_another_device_is_refused():
    from lora_linear_layers_amd import functional as F

    with pytest.raises(ValueError, match="ws is on cpu"):
        F._check_ws(torch.device("cuda:0"), torch.empty(16, dtype=torch.uint8))


def test_epilogue_refusals():
    import ctypes

    import lora_linear_layers_amd as L
    from lora_linear_layers_amd import _lib

    X = torch.zeros(4, 16)
    m = {"W": torch.zeros(8, 16), "A": torch.zeros(2, 16), "B": torch.zeros(8, 2), "scale": 1.0}
    with pytest.raises(ValueError, match="GPU"):
        L.lora_linear_epi_fwd(X, m)
    lib, P = L.lib(), 0x100000
    tab = (ctypes.c_float * 16)(*range(16))

    def mk(rope=0, d_out=64, r=8, W=P, W_nf4=None, absmax=None, A=P, B=P, Y=P, dY=P, dX=P, dA=P, dB=P, W_t=None):
        return _lib.GroupMember(d_out, r, 1.0, rope, W, W_nf4, absmax, A, B, Y, dY, dX, dA, dB, W_t)

    def ep(act=2, bias=P, res=P, Z=P):
        return _lib.Epilogue(act, bias, res, Z)

    def fwd(dtype=1, M=16, k=64, m=None, e=None, X=P, table=tab, ws=P, wsb=1 << 30):
        return lib.lora_linear_epi_fwd(dtype, M, k, m or mk(), e or ep(), X, table, ws, wsb, None)

    def bwd(dtype=1, M=16, k=64, m=None, e=None, X=P, table=tab, db=P, ws=P, wsb=1 << 30):
        return lib.lora_linear_epi_bwd(dtype, M, k, m or mk(), e or ep(), X, table, db, ws, wsb, None)

    for f in (fwd, bwd):
        assert f(dtype=2) == -4 and f(M=-1) == -2 and f(k=12) == -2 and f(m=mk(r=0)) == -2 and f(m=mk(d_out=12)) == -2
        assert f(m=mk(rope=1)) == -2 and f(m=mk(d_out=2 ** 20 + 8)) == -2 and f(e=ep(act=5)) == -2 and f(e=ep(act=-1)) == -2
        assert f(m=mk(W=None)) == -1 and f(m=mk(A=None)) == -1 and f(X=None) == -1 and f(X=P + 8) == -3
        assert f(dtype=0, m=mk(W_nf4=P, absmax=P)) == -4 and f(m=mk(W_nf4=P)) == -1
        assert f(m=mk(W_nf4=P, absmax=P), table=None) == -1 and f(m=mk(W_nf4=P, absmax=P), k=96) == -2
        assert f(wsb=16) == -5 and f(ws=None) == -5 and f(ws=P + 4) == -3
    assert fwd(m=mk(Y=None)) == -1 and fwd(m=mk(Y=P + 2)) == -3
    assert fwd(e=ep(bias=P + 2)) == -3 and fwd(e=ep(res=P + 4)) == -3 and fwd(e=ep(Z=P + 8)) == -3
    assert bwd(m=mk(dY=None)) == -1 and bwd(m=mk(dA=None)) == -1 and bwd(m=mk(dX=P + 2)) == -3 and bwd(db=P + 4) == -3
    assert bwd(e=ep(Z=None)) == -1 and bwd(m=mk(W_t=P + 2)) == -3
    size = lib.lora_linear_epi_workspace_bytes
    base = lib.lora_workspace_bytes(_lib.OP_BWD, 1, 1000, 512, 768, 16)
    assert size(0, 1, 1000, 512, mk(d_out=768, r=16), ep()) == lib.lora_workspace_bytes(_lib.OP_FWD, 1, 1000, 512, 768, 16)
    # the layer's own, the bias gradient's partials (up to 64 rows) and, with an activation, dZ
    none, act = (size(1, 1, 1000, 512, mk(d_out=768, r=16), ep(act=a)) for a in (0, 2))
    assert base + 768 * 4 <= none <= base + 64 * 768 * 4 and act == none + 1000 * 768 * 2
    assert size(0, 3, 8, 64, mk(), ep()) == 0 and size(0, 1, 8, 12, mk(), ep()) == 0
    if torch.cuda.device_count() == 0:
        assert fwd() == -6 and bwd(e=ep(act=0, Z=None)) == -6


@pytest.mark.gpu
def test_epilogue_adapter_gradient_past_32_bits(lib):
    # dA where dZ has 2^31 elements and more: one token in 64 carries input, the rows at both ends and around
    # element 2^31 among them, so that every sum of integers is exact in fp32 whatever its order
    M, k, d, r = 140003, 64, 16384, 8
    gen = torch.Generator("cuda").manual_seed(3)
    draw = lambda *n: torch.randint(-2, 3, n, generator=gen, device="cuda", dtype=torch.int8).bfloat16()  # noqa: E731
    X, dY, Z = draw(M, k), draw(M, d), draw(M, d)
    rows = torch.arange(M, device="cuda")
    X *= ((rows % 64 == 5) | (rows < 20) | (rows >= M - 20) | ((rows - 131072).abs() < 20))[:, None]
    m = {"W": draw(d, k), "A": draw(r, k), "B": draw(d, r), "scale": 1.0}
    _, dA, _, _ = lib.lora_linear_epi_bwd(X, m, dY, "relu", Z, need_dX=False)
    want, mag = torch.zeros(r, k, device="cuda", dtype=torch.float64), torch.zeros(r, k, device="cuda", dtype=torch.float64)
    for i in range(0, M, 20000):
        x = X[i:i + 20000].double()
        at = x.abs().sum(1) > 0
        q = (dY[i:i + 20000][at] * (Z[i:i + 20000][at] > 0)).double() @ m["B"].double()  # below 2^17, exact
        q = q.bfloat16().double().T.contiguous()  # Q is rounded to bf16, the product's operand
        want += q @ x[at]
        mag += q.abs() @ x[at].abs()
    assert 0 < mag.max() < 2 ** 24
    assert torch.equal(dA.double(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_epilogue_function_gradients_have_their_inputs_shapes(lib, dtype):
    X, m, bias, res, dY = _inputs(14, 20, 64, 72, 8, dtype)
    out = []
    for b, r in ((bias, res), (bias.view(1, 72), res.view(4, 5, 72)), (bias.view(72, 1), res.view(-1))):
        leaves = [t.clone().requires_grad_() for t in (X, m["A"], m["B"], b, r)]
        Y = lib.LoraLinearEpiFunction.apply(leaves[0], m["W"], *leaves[1:], m["scale"], "silu")
        Y.backward(dY)
        assert all(t.grad.shape == t.shape for t in leaves)
        out.append([Y] + [t.grad.reshape(-1) for t in leaves])
    assert all(torch.equal(a, b) for o in out[1:] for a, b in zip(out[0], o))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(20, 72), (4, 5, 72)], ids=str)
def test_epilogue_residual_gradient_is_not_the_callers(lib, shape):
    # the residual's gradient is dY: what a step then does to residual.grad leaves the caller's dY as it was
    X, m, bias, res, dY = _inputs(19, 20, 64, 72, 8, "f32")
    r, keep = res.view(shape).requires_grad_(), dY.clone()
    lib.LoraLinearEpiFunction.apply(X, m["W"], m["A"], m["B"], bias, r, m["scale"]).backward(dY)
    assert torch.equal(r.grad.view(20, 72), dY)
    r.grad.zero_()
    assert torch.equal(dY, keep)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_epilogue_function_gradients_own_their_storage(lib, dtype):
    # one gradient's storage may be freed or resized without the others (sharded training does); and the rounded
    # gradients are the fp32 ones, each rounded once
    X, m, bias, res, dY = _inputs(15, 20, 64, 72, 8, dtype)
    leaves = [t.clone().requires_grad_() for t in (X, m["A"], m["B"], bias, res)]
    lib.LoraLinearEpiFunction.apply(leaves[0], m["W"], *leaves[1:], m["scale"]).backward(dY)
    grads = [t.grad for t in leaves[:4]]
    assert len({g.untyped_storage().data_ptr() for g in grads}) == 4
    assert all(g.untyped_storage().nbytes() == g.numel() * g.element_size() for g in grads)
    dX, dA, dB, db = lib.lora_linear_epi_bwd(X, m, dY, need_dbias=True)
    assert all(torch.equal(g, w.to(X.dtype)) for g, w in zip(grads, (dX, dA, dB, db)))


@pytest.mark.gpu
def test_epilogue_function_does_only_what_is_asked_for(lib, monkeypatch):
    from lora_linear_layers_amd import functional as F

    X, m, bias, res, dY = _inputs(16, 20, 64, 72, 8, "bf16")
    kept, ran = [], []
    fwd, bwd = F.lora_linear_epi_fwd, F._epi_bwd
    monkeypatch.setattr(F, "lora_linear_epi_fwd", lambda *a, **k: (kept.append(k["store_z"]), fwd(*a, **k))[1])
    monkeypatch.setattr(F, "_epi_bwd", lambda *a, **k: (ran.append(1), bwd(*a, **k))[1])
    base = (X, m["A"], m["B"], bias, res)
    for need in ((), (4,), (0,), (1,), (3,), (0, 1, 2, 3, 4)):
        leaves = [t.clone().requires_grad_(i in need) for i, t in enumerate(base)]
        Y = lib.LoraLinearEpiFunction.apply(leaves[0], m["W"], *leaves[1:], m["scale"], "silu")
        if need:
            Y.backward(dY)
        assert kept.pop() == bool(set(need) - {4}) and len(ran) == (1 if set(need) - {4} else 0)
        ran.clear()
        assert [t.grad is not None for t in leaves] == [i in need for i in range(5)]
        if 4 in need:
            assert torch.equal(leaves[4].grad, dY)


def test_epilogue_sizing_refuses_what_the_calls_refuse():
    import lora_linear_layers_amd as L
    from lora_linear_layers_amd import _lib

    size, P = L.lib().lora_linear_epi_workspace_bytes, 0x100000

    def n(bwd, dtype=1, M=1000, k=512, d_out=768, r=16, rope=0, nf4=None, act=2):
        return size(bwd, dtype, M, k, _lib.GroupMember(d_out, r, 1.0, rope, None if nf4 else P, nf4),
                    _lib.Epilogue(act))

    for b in (0, 1):
        assert n(b) > 0 and n(b, nf4=P) > 0
        assert n(b, act=5) == 0 and n(b, act=-1) == 0 and n(b, rope=1) == 0 and n(b, d_out=2 ** 20 + 8) == 0
        assert n(b, nf4=P, dtype=0) == 0 and n(b, nf4=P, k=520) == 0
        assert n(b, r=0) == 0 and n(b, M=-1) == 0


@pytest.mark.gpu
def test_epilogue_workspaces_are_measured_in_bytes(lib):
    from lora_linear_layers_amd import _lib

    X, m, bias, _, dY = _inputs(17, 300, 264, 392, 16, "bf16")
    mem = _lib.GroupMember(392, 16, 1.0, 0, 1)
    size = [lib.lib().lora_linear_epi_workspace_bytes(b, 1, 300, 264, mem, _lib.Epilogue()) for b in (0, 1)]
    assert all(n and n % 4 == 0 for n in size)
    ws = [torch.empty(n // 4, device="cuda") for n in size]
    Y, _ = lib.lora_linear_epi_fwd(X, m, "none", bias, ws=ws[0])
    assert torch.equal(Y, lib.lora_linear_epi_fwd(X, m, "none", bias)[0])
    got, want = lib.lora_linear_epi_bwd(X, m, dY, ws=ws[1]), lib.lora_linear_epi_bwd(X, m, dY)
    assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
    for call in (lambda: lib.lora_linear_epi_fwd(X, m, "none", bias, ws=ws[0][:-1]),
                 lambda: lib.lora_linear_epi_bwd(X, m, dY, ws=ws[1][:-1])):
        with pytest.raises(RuntimeError):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_epilogue_relu_passes_no_gradient_below_zero(lib, dtype):
    # not even an infinite one or a NaN: those where Z <= 0 leave every gradient as zeros there do
    X, m, _, _, dY = _inputs(18, 40, 64, 72, 8, dtype)
    Z = dY.flip(0).contiguous()
    Z[3, 5] = 0.0
    off = Z <= 0
    assert off[3, 5] and off.sum() > 100
    bad = dY.clone()
    bad[off] = torch.tensor([float("inf"), -float("inf"), float("nan")], device="cuda").repeat(int(off.sum()))[:int(off.sum())].to(dY.dtype)
    zero = dY.masked_fill(off, 0.0)
    got = lib.lora_linear_epi_bwd(X, m, bad, "relu", Z, need_dbias=True)
    want = lib.lora_linear_epi_bwd(X, m, zero, "relu", Z, need_dbias=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and got[0].isfinite().all()


def test_workspaces_of_groups_and_pairs_are_taken_as_before():
    # a workspace given to the group and SwiGLU calls: any memory that the device reaches, of at least as many bytes
    # from its first element on as it has elements (which is the size that the library is told)
    from lora_linear_layers_amd import functional as F

    here, buf = torch.device("cpu"), torch.empty(4096, dtype=torch.uint8)
    for f in (F._group_ws, F._swiglu_ws):
        for ws in (buf, buf[::2], buf.view(64, 64).t(), buf.view(torch.float32), buf[16:1040]):
            assert f(False, 1, 8, 64, None, here, ws) is ws
        for ws in (torch.empty(1, dtype=torch.uint8).expand(4096), buf[-64:].as_strided((65,), (0,))):
            with pytest.raises(ValueError, match="fewer bytes"):
                f(False, 1, 8, 64, None, here, ws)
        with pytest.raises(ValueError, match="ws is on cpu"):
            f(False, 1, 8, 64, None, torch.device("cuda:0"), buf)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [("bf16", 1, 4096, 1024, 16), ("bf16", 33, 256, 512, 64), ("bf16", 300, 264, 392, 16),
                                  ("bf16", 2048, 3200, 2056, 24), ("bf16", 2048, 14400, 2048, 24), ("f32", 128, 256, 256, 8),
                                  ("f32", 107, 4352, 384, 32), ("nf4", 128, 256, 256, 64), ("nf4", 640, 4096, 512, 8)], ids=str)
def test_epilogue_backward_without_the_inputs_gradient(lib, case):
    # a first layer's step: no dX, on every path that has one with it
    kind, M, k, d, r = case
    table = None
    if kind == "nf4":
        X, m, _, _, dY, table = _nf4(60 + M, k, d, r, M)
    else:
        X, m, _, _, dY = _inputs(60 + M, M, k, d, r, kind)
    Z = torch.randn(M, d, generator=torch.Generator().manual_seed(5)).to(X.dtype).cuda()

    class NoDX:
        nf4_dequant = staticmethod(lib.nf4_dequant)

        @staticmethod
        def lora_linear_epi_bwd(*a, **kw):
            none, *grads = lib.lora_linear_epi_bwd(*a, need_dX=False, **kw)
            assert none is None
            return (lib.lora_linear_epi_bwd(*a, **kw)[0], *grads)

    check_bwd(NoDX, X, m, dY, "silu", Z, table)


@pytest.mark.gpu
def test_whole_step_captured_and_replayed(lib):
    # epilogue layer, head, log-probabilities and policy loss with every gradient, captured once (no eager graph of the
    # leaves alive then) and replayed on new inputs with eager work between the replays
    d, V, n, r = 128, 520, 96, 8
    X, up, bias, res, _ = _inputs(1, n, d, d, r, "bf16")
    _, head, _, _, _ = _inputs(2, n, d, V, r, "bf16")
    gen = torch.Generator().manual_seed(4)
    t = torch.randint(0, V, (n,), generator=gen).cuda()
    cu = torch.tensor([0, 40, 40, 96], device="cuda")
    adv, old = torch.tensor([0.8, -0.5, 1.0], device="cuda"), (-6 + torch.randn(n, generator=gen)).cuda()
    leaves = [v.clone().requires_grad_() for v in (X, up["A"], up["B"], bias, res, head["A"], head["B"])]

    def step():
        x, a, b, bi, rs, ha, hb = leaves
        y = lib.LoraLinearEpiFunction.apply(x, up["W"], a, b, bi, rs, up["scale"], "silu")
        lp = lib.LoraHeadLogpFunction.apply(y, head["W"], ha, hb, head["scale"], t)
        loss, _ = lib.LoraPolicyLossFunction.apply(lp, old, old, cu, adv, None, 0.2, 0.2, 0.05)
        return [loss.detach(), *torch.autograd.grad(loss, leaves)]

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        with torch.no_grad():
            leaves[0].copy_(torch.roll(leaves[0], 1, 0))
            old.add_(0.05)
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held))
