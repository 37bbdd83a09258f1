"""A projection whose rows each carry an adapter of their own, and its gradients,
against the definition in 64 bits, element by element.

Tolerances, h = half a step of the type relative to the value (bf16 2^-8, fp32
2^-24), u = 2^-24: a strip (s A x, or s B^T dy) is rounded once (h), its product with
the second operand may be rounded once more before the base product is added to it
(h of its magnitude), a contraction of n products accumulates at most (n + 2) u of
the sum of magnitudes, the output is rounded (h)."""
import math

import pytest
import torch

U = 2.0 ** -24
H = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DTYPES = [torch.bfloat16, torch.float32]
pytestmark = pytest.mark.gpu


def _near(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((err / tol.clamp(min=1e-300)).max()))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g)


def _index(g, M, n, order):
    if order == "one":
        return torch.full((M,), n - 1, dtype=torch.int32)
    if order == "none":
        return torch.full((M,), -1, dtype=torch.int32)
    if order == "random":  # a tenth of them without adapter, by indices on either side of the range
        a = torch.randint(0, n, (M,), generator=g, dtype=torch.int32)
        out = torch.tensor([-1, n, n + 70000, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
        return torch.where(torch.rand(M, generator=g) < 0.1, out[torch.arange(M) % 5], a)
    cuts = torch.sort(torch.randint(0, M + 1, (max(1, min(M, 12)),), generator=g)).values
    which = torch.randint(-1, n, (len(cuts) + 1,), generator=g, dtype=torch.int32)
    return which[torch.searchsorted(cuts, torch.arange(M), right=True)]


def make(seed, M, k, d, n, r, dtype, order="packed"):
    g = torch.Generator().manual_seed(seed)
    X, W = _randn(g, M, k), _randn(g, d, k) / math.sqrt(k)
    A, B = _randn(g, n, r, k) / math.sqrt(k), 0.2 * _randn(g, n, d, r)
    dY, scales = _randn(g, M, d), 0.25 + torch.rand(n, generator=g)
    index = _index(g, M, n, order)
    return [t.to(dtype).cuda() for t in (X, W, A, B)] + [scales.cuda(), index.cuda(), dY.to(dtype).cuda()]


def reference(X, W, A, B, scales, index, dY):
    """Y, dX, dA, dB and their tolerances in 64 bits, adapter by adapter."""
    dt, h = X.dtype, H[X.dtype]
    x, w, a, b, s, g = X.double(), W.double(), A.double(), B.double(), scales.double(), dY.double()
    (M, k), (d, _), (n, r, _) = x.shape, w.shape, a.shape
    Y, tY = x @ w.T, (k + r + 4) * U * (x.abs() @ w.abs().T)
    dX, tX = g @ w, (d + r + 4) * U * (g.abs() @ w.abs())
    dA, dB = torch.zeros_like(a), torch.zeros_like(b)
    tA, tB = torch.zeros_like(a), torch.zeros_like(b)
    for i in set(index.tolist()):
        if not 0 <= i < n:
            continue
        rows = torch.nonzero(index == i).squeeze(1)
        xi, gi = x[rows], g[rows]
        P, Q = s[i] * (xi @ a[i].T), s[i] * (gi @ b[i])
        mP, mQ = s[i] * (xi.abs() @ a[i].abs().T), s[i] * (gi.abs() @ b[i].abs())
        eP, eQ = h * P.abs() + (k + 4) * U * mP, h * Q.abs() + (d + 4) * U * mQ
        Y[rows] += P @ b[i].T
        tY[rows] += eP @ b[i].abs().T + ((k + r + 4) * U + h) * (mP @ b[i].abs().T)
        dX[rows] += Q @ a[i]
        tX[rows] += eQ @ a[i].abs() + ((d + r + 4) * U + h) * (mQ @ a[i].abs())
        m = (len(rows) + 4) * U
        dA[i], dB[i] = Q.T @ xi, gi.T @ P
        tA[i] = eQ.T @ xi.abs() + m * (mQ.T @ xi.abs())
        tB[i] = gi.abs().T @ eP + m * (gi.abs().T @ mP)
    fin = lambda v, t: t + h * (v.abs() + t) + 1e-37  # noqa: E731
    return (Y, fin(Y, tY)), (dX, fin(dX, tX)), (dA, tA + 1e-37), (dB, tB + 1e-37)


def check(lib, args, W_t=None):
    X, W, A, B, scales, index, dY = args
    Y = lib.lora_multi_fwd(X, W, A, B, scales, index)
    dX, dA, dB = lib.lora_multi_bwd(X, W, A, B, scales, index, dY, W_t=W_t)
    none, dA2, dB2 = lib.lora_multi_bwd(X, W, A, B, scales, index, dY, need_dX=False)
    torch.cuda.synchronize()
    assert none is None and torch.equal(dA, dA2) and torch.equal(dB, dB2)
    for name, got, (want, tol) in zip(("Y", "dX", "dA", "dB"), (Y, dX, dA, dB), reference(*args)):
        _near(got, want, tol, name)
    return Y, dX, dA, dB


# tokens, d_in, d_out, adapters, rank
SHAPES = [(1, 64, 64, 1, 8), (1, 4096, 512, 16, 16), (2, 8, 16, 3, 8), (7, 72, 40, 5, 24), (16, 256, 512, 64, 16),
          (33, 520, 1032, 7, 40), (48, 1024, 2048, 64, 16), (64, 2048, 768, 100, 8), (65, 128, 256, 9, 64), (100, 64, 4096, 2, 32),
          (129, 384, 264, 30, 128), (200, 1000, 1000, 3, 56), (300, 4096, 1024, 8, 16), (513, 512, 776, 20, 72),
          (1000, 256, 4096, 17, 16), (777, 2560, 3000, 40, 16)]


@pytest.mark.parametrize("order", ["packed", "random", "one", "none"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_shapes(lib, dtype, shape, order):
    check(lib, make(sum(shape), *shape, dtype, order))


@pytest.mark.parametrize("order", ["packed", "random"])
@pytest.mark.parametrize("shape", [(2048, 4096, 4096, 8, 16), (4096, 1024, 4096, 64, 16), (2049, 2048, 4104, 33, 32),
                                   (4352, 1024, 1776, 5, 64), (1537, 4096, 2048, 300, 8), (8192, 512, 2048, 6, 128)])
def test_large(lib, shape, order):
    """128 x 256 and 256 x 256 tiles, whole and ragged, in one block and in two."""
    args = make(sum(shape), *shape, torch.bfloat16, order)
    one = check(lib, args)
    two = lib.lora_multi_bwd(*args, W_t=lib.lora_transpose(args[1]))
    for a, b in zip(one[1:], two):
        assert torch.equal(a, b)


@pytest.mark.parametrize("shape", [(40, 512, 1024, 6, 16), (3000, 512, 4096, 6, 16), (900, 1024, 4096, 12, 8)])
def test_one_adapter_is_the_plain_layer(lib, shape):
    """With every row on one adapter: the layer of that adapter, up to its rounding."""
    X, W, A, B, scales, index, dY = make(5, *shape, torch.bfloat16, "one")
    i = A.shape[0] - 1
    Y = lib.lora_multi_fwd(X, W, A, B, scales, index)
    y = lib.lora_linear_fwd(X, W, A[i], B[i], float(scales[i]))
    assert float((Y.double() - y.double()).norm() / y.double().norm()) < 2.0 ** -8


def test_repeats_bit_for_bit(lib):
    for order in ("packed", "random"):
        args = make(3, 3000, 1024, 2048, 20, 16, torch.bfloat16, order)
        first = check(lib, args)
        for _ in range(3):
            again = (lib.lora_multi_fwd(*args[:6]), *lib.lora_multi_bwd(*args))
            for a, b in zip(first, again):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,k,d", [(20, 256, 512), (150, 256, 384), (2500, 1024, 4096), (4200, 512, 4096)])
def test_infinities_stay_with_their_own(lib, dtype, M, k, d):
    """An infinity or a NaN in a row of X or dY, in an adapter, or in a row without adapter reaches no other adapter
    and no other row."""
    if dtype == torch.float32 and M > 1000:
        pytest.skip("the fp32 kernels take one row at a time whatever the size")
    n, r = 6, 16
    args = make(11, M, k, d, n, r, dtype, "random")
    X, W, A, B, scales, index, dY = args
    index[:4] = torch.tensor([0, 1, -1, 2])
    clean = (lib.lora_multi_fwd(*args[:6]), *lib.lora_multi_bwd(*args))
    X[0, 3], X[2, 5], dY[2, 7] = math.nan, math.inf, math.nan
    dY[1, 2] = -math.inf
    A[3, 2, 1], B[4, 9, 5] = math.inf, math.nan
    Y = lib.lora_multi_fwd(*args[:6])
    dX, dA, dB = lib.lora_multi_bwd(*args)
    torch.cuda.synchronize()
    i = index.cpu()
    own = (i == 3) | (i == 4)  # rows of the adapters with a bad value
    keep = ~own
    keep[[0, 2]] = False
    assert torch.equal(Y[keep], clean[0][keep])
    keep[[0, 1, 2]] = torch.tensor([True, False, False])  # (X plays no part in dX)
    assert torch.equal(dX[keep], clean[1][keep])
    assert bool(torch.isnan(Y[0]).all()) and bool((~torch.isfinite(dX[1])).any())
    assert bool((~torch.isfinite(Y[i == 3])).any(1).all()) and bool((~torch.isfinite(Y[i == 4])).any(1).all())
    for a in (2, 5):
        assert torch.equal(dA[a], clean[2][a]) and torch.equal(dB[a], clean[3][a])
    # the rows' own adapters: not finite where the definition is not
    assert bool((~torch.isfinite(dB[0])).all()) and bool((~torch.isfinite(dA[0][:, 3])).all())
    assert bool((~torch.isfinite(dA[1])).all()) and bool((~torch.isfinite(dB[1][2])).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_function(lib, dtype):
    X, W, A, B, scales, index, dY = make(4, 150, 256, 384, 5, 16, dtype)
    X, A, B = (t.requires_grad_() for t in (X, A, B))
    Y = lib.LoraMultiFunction.apply(X, W, A, B, scales, index)
    Y.backward(dY)
    x, a, b = X.detach(), A.detach(), B.detach()
    assert torch.equal(Y, lib.lora_multi_fwd(x, W, a, b, scales, index))
    for g, w in zip((X.grad, A.grad, B.grad), lib.lora_multi_bwd(x, W, a, b, scales, index, dY, grad_dtype=dtype)):
        assert g.dtype == dtype and torch.equal(g, w)
    (dA,) = torch.autograd.grad(lib.LoraMultiFunction.apply(x, W, A, b, scales, index), A, dY)
    assert torch.equal(dA, A.grad)
    # the gradients in 16 bits are those in 32 rounded
    wide = lib.lora_multi_bwd(x, W, a, b, scales, index, dY)
    for g, w in zip((A.grad, B.grad), wide[1:]):
        assert torch.equal(g, w.to(dtype))


def test_gradients_against_differences(lib):
    X, W, A, B, scales, index, dY = make(9, 24, 64, 48, 4, 8, torch.float32, "random")
    dX, dA, dB = lib.lora_multi_bwd(X, W, A, B, scales, index, dY)
    g, t = torch.Generator().manual_seed(1), 2.0 ** -6
    for which, grad in ((0, dX), (2, dA), (3, dB)):
        V = _randn(g, *grad.shape).cuda()
        f = []
        for k in (t, -t):
            args = [X, W, A, B, scales, index]
            args[which] = args[which] + k * V
            f.append(lib.lora_multi_fwd(*args).double())
        slope, want = float((dY.double() * (f[0] - f[1])).sum() / (2 * t)), float((grad.double() * V.double()).sum())
        # linear in each of them: the rounding of the outputs and of the sums, 100 additions deep, alone
        size = float((dY.double().abs() * f[0].abs().clamp(min=10)).sum())
        assert abs(slope - want) <= size * 100 * U / t, (which, slope, want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_empty(lib, dtype):
    X, W, A, B, scales, index, dY = make(1, 0, 64, 48, 3, 8, dtype)
    assert lib.lora_multi_fwd(X, W, A, B, scales, index).shape == (0, 48)
    for gt in DTYPES:
        dX, dA, dB = lib.lora_multi_bwd(X, W, A, B, scales, index, dY, grad_dtype=gt)
        assert dX.shape == (0, 64) and bool((dA == 0).all()) and bool((dB == 0).all())


def test_stream_graph_and_workspace(lib):
    """On a stream of its own, captured and replayed with new rows' adapters, with one caller's workspace."""
    for M, k, d in ((40, 512, 1024), (700, 512, 4096), (2600, 1024, 4096)):
        X, W, A, B, scales, index, dY = args = make(M, M, k, d, 10, 16, torch.bfloat16)
        want = (lib.lora_multi_fwd(*args[:6]), *lib.lora_multi_bwd(*args))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = (lib.lora_multi_fwd(*args[:6]), *lib.lora_multi_bwd(*args))
        torch.cuda.current_stream().wait_stream(s)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        nb = max(lib.lib().lora_multi_workspace_bytes(b, 1, M, k, d, 10, 16, 0, b) for b in (0, 1))
        ws = torch.full((nb,), 0xA5, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = (lib.lora_multi_fwd(*args[:6], ws=ws), *lib.lora_multi_bwd(*args, ws=ws))
        for seed in range(3):
            index.copy_(_index(torch.Generator().manual_seed(seed), M, 10, "random").cuda())
            ws.fill_(0xFF)
            graph.replay()
            torch.cuda.synchronize()
            want = (lib.lora_multi_fwd(*args[:6]), *lib.lora_multi_bwd(*args))
            for a, b in zip(outs, want):
                assert torch.equal(a, b)


def test_sliced_index_and_scales(lib):
    X, W, A, B, scales, index, dY = make(6, 300, 256, 512, 5, 16, torch.bfloat16)
    big_i, big_s = torch.zeros(303, dtype=torch.int32, device="cuda"), torch.zeros(7, device="cuda")
    big_i[1:301], big_s[1:6] = index, scales
    a = (X, W, A, B, scales, index)
    b = (X, W, A, B, big_s[1:6], big_i[1:301])
    assert torch.equal(lib.lora_multi_fwd(*a), lib.lora_multi_fwd(*b))
    for g, w in zip(lib.lora_multi_bwd(*a, dY), lib.lora_multi_bwd(*b, dY)):
        assert torch.equal(g, w)


def test_refusals(lib):
    X, W, A, B, scales, index, dY = make(1, 10, 64, 48, 3, 8, torch.bfloat16)
    f = lib.lora_multi_fwd
    for bad in ((X[:, :32], W, A, B, scales, index), (X, W, A[:, :, :32], B, scales, index), (X, W, A, B[:2], scales, index),
                (X, W, A, B, scales[:2], index), (X, W, A, B, scales, index[:9]), (X, W, A, B, scales, index.cpu()),
                (X, W, A.transpose(0, 1).contiguous().transpose(0, 1), B, scales, index), (X.cpu(), W, A, B, scales, index)):
        with pytest.raises(ValueError):
            f(*bad)
    for bad in ((X, W, A, B, scales, index.long()), (X, W.float(), A, B, scales, index), (X, W, A, B, scales.double(), index)):
        with pytest.raises(TypeError):
            f(*bad)
    with pytest.raises(lib.LoraError):
        f(X, W, A[:, :4].contiguous(), B[:, :, :4].contiguous(), scales, index)  # rank 4
    with pytest.raises(lib.LoraError):
        f(X, W, A, B, scales, index, ws=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        lib.lora_multi_bwd(X, W, A, B, scales, index, dY[:5])
    with pytest.raises(TypeError):
        lib.lora_multi_bwd(X, W, A, B, scales, index, dY, grad_dtype=torch.float16)


def _norm64(h, w):
    return h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-5) * w


def _rel(got, want, tol, what):
    assert float((got.double() - want).norm()) <= tol * float(want.norm()), what


def test_served_block(lib):
    """A decode step of requests with adapters of their own: residual norm, a projection up and one down, captured once
    and replayed for new tokens, requests and adapters, two of them in turn; a prompt batch by the same calls."""
    k, d, n, r = 512, 1024, 12, 16
    _, W1, A1, B1, s1, _, _ = make(1, 1, k, d, n, r, torch.bfloat16)
    _, W2, A2, B2, s2, _, _ = make(2, 1, d, k, n, r, torch.bfloat16)
    w = (1 + 0.2 * _randn(torch.Generator().manual_seed(3), k)).bfloat16().cuda()

    def block(X, R, index):
        Y, Hh, _, _, _ = lib.lora_rmsnorm_fwd(X, w, residual=R)
        U1 = lib.lora_multi_fwd(Y, W1, A1, B1, s1, index)
        return Hh, lib.lora_multi_fwd(U1, W2, A2, B2, s2, index)

    def inputs(seed, M):
        g = torch.Generator().manual_seed(seed)
        return [_randn(g, M, k).bfloat16().cuda() for _ in range(2)] + [_index(g, M, n, "random").cuda()]

    def proj(y, W, A, B, s, index):
        out = y @ W.double().T
        for i in range(n):
            rows = index == i
            out[rows] += s.double()[i] * (y[rows] @ A[i].double().T) @ B[i].double().T
        return out
    graphs = []
    for M in (5, 40):
        ins = inputs(10 + M, M)
        block(*ins)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = block(*ins)
        graphs.append((M, ins, graph, outs))
    for seed in range(3):
        for M, ins, _, _ in graphs:
            for t, v in zip(ins, inputs(20 + seed, M)):
                t.copy_(v)
        for _, _, graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for M, ins, _, outs in graphs:
            for a, b in zip(outs, block(*ins)):
                assert torch.equal(a, b)
    for M in (5, 40, 700):
        X, R, index = inputs(30, M)
        Hh, Z = block(X, R, index)
        y = _norm64((X.float() + R.float()).bfloat16().double(), w.double())
        want = proj(proj(y, W1, A1, B1, s1, index), W2, A2, B2, s2, index)
        _rel(Z, want, 6 * 2.0 ** -8, M)  # the norm's output, both strips (and their parts) and both outputs rounded


@pytest.mark.parametrize("M", [200, 1100])
def test_trained_block(lib, M):
    """Several adapters trained behind one norm, through the autograd functions, while another graph of the same leaves
    lives."""
    k, d, n, r = 512, 768, 5, 16
    X, W, A, B, s, index, dY = make(7, M, k, d, n, r, torch.bfloat16)
    g = torch.Generator().manual_seed(8)
    R, w = _randn(g, M, k).bfloat16().cuda(), (1 + 0.2 * _randn(g, k)).bfloat16().cuda()
    leaves = [t.requires_grad_() for t in (X, R, w, A, B)]

    def forward():
        Y, Hh = lib.LoraRmsNormFunction.apply(X, R, w, 1e-5, False)
        return lib.LoraMultiFunction.apply(Y, W, A, B, s, index), Hh
    dH = _randn(g, M, k).bfloat16().cuda()
    one, two = forward(), forward()
    first = torch.autograd.grad(one, leaves, (dY, dH))
    for a, b in zip(first, torch.autograd.grad(two, leaves, (dY, dH))):
        assert torch.equal(a, b)
    h = (X.float() + R.float()).bfloat16().detach().double().requires_grad_()
    wd, ad, bd = (t.detach().double().requires_grad_() for t in (w, A, B))
    y = _norm64(h, wd)
    z = y @ W.double().T
    for i in range(n):
        m = (index == i).double()[:, None]
        z = z + m * s.double()[i] * (y @ ad[i].T) @ bd[i].T
    gh, gw, ga, gb = torch.autograd.grad((z, h), (h, wd, ad, bd), (dY.double(), dH.double()), allow_unused=True)
    for got, want, what in zip(first, (gh, gh, gw, ga, gb), ("X", "residual", "weight", "A", "B")):
        _rel(got, want, 4 * 2.0 ** -8, what)  # the norm's output, a strip, dY W and the gradient rounded


# one launch over strips of W's columns, or a stream of W, that adds the rows' strips itself; ranks in steps of 32
@pytest.mark.parametrize("order", ["packed", "random"])
@pytest.mark.parametrize("shape", [(1, 4096, 4096, 3, 128), (16, 1024, 1032, 9, 72), (40, 2048, 2056, 30, 128), (64, 1024, 1024, 64, 64),
                                   (33, 520, 4104, 40, 24), (20, 4096, 4096, 20, 32), (64, 4096, 4104, 64, 24), (5, 4096, 8192, 5, 128),
                                   (48, 4096, 8200, 64, 64), (64, 8192, 4096, 7, 40), (3, 4096, 8192, 2, 16)])
def test_few_rows(lib, shape, order):
    M, k, d, n, r = shape
    args = make(M + k + n, M, k, d, n, r, torch.bfloat16, order)
    Y = lib.lora_multi_fwd(*args[:6])
    (want, tol), *_ = reference(*args)
    _near(Y, want, tol, "Y")
    assert torch.equal(Y, lib.lora_multi_fwd(*args[:6]))


@pytest.mark.parametrize("M,k,d", [(20, 4096, 4096), (40, 4096, 8192), (60, 1024, 1024)])
def test_infinities_of_few_rows_stay_with_their_own(lib, M, k, d):
    test_infinities_stay_with_their_own(lib, torch.bfloat16, M, k, d)


def _large_stack(seed, M, k, d, n, r):
    """Inputs with n adapters on the device, of which the rows carry six and none; and the same with those six alone."""
    g = torch.Generator().manual_seed(seed)
    gpu = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gpu, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    X, W, dY = normal(M, k), normal(d, k).div_(math.sqrt(k)), normal(M, d)
    A, B = normal(n, r, k).div_(math.sqrt(k)), normal(n, d, r).mul_(0.2)
    scales = (0.25 + torch.rand(n, generator=g)).cuda()
    used = torch.tensor([0, 7, n // 2 - 1, n // 2, n - 2, n - 1])
    small = _index(g, M, 6, "random")
    small[(small < 0) | (small >= 6)] = -1
    index = torch.where(small < 0, -1, used[small.clamp(min=0).long()].to(torch.int32))
    used = used.cuda()
    return (X, W, A, B, scales, index.cuda(), dY), (X, W, A[used], B[used], scales[used], small.cuda(), dY), used


@pytest.mark.parametrize("M,k,d,n,r", [(1200, 4096, 14336, 1024, 128), (1200, 1536, 14336, 2048, 64)])
def test_stacks_past_the_product_kernel(lib, M, k, d, n, r):
    """Second operands of 0xE0000000 bytes, which the product with the adapters' columns does not take: the strips' part
    first, then the base product, the last of whose tiles are two blocks' work each.  The workspace holds ones."""
    args, few, _ = _large_stack(n, M, k, d, n, r)
    assert args[3].nbytes >= 0xE0000000
    nb = lib.lib().lora_multi_workspace_bytes(0, 1, M, k, d, n, r, 0, 0)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    (want, tol), *_ = reference(*few)
    for _ in range(2):
        Y = lib.lora_multi_fwd(*args[:6], ws=ws.fill_(0xFF))
        _near(Y, want, tol, "Y")


def test_stacks_past_the_product_kernel_backward(lib):
    M, k, d, n, r = 1200, 14336, 4096, 1024, 128
    args, few, used = _large_stack(5, M, k, d, n, r)
    nb = lib.lib().lora_multi_workspace_bytes(1, 1, M, k, d, n, r, 0, 1)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda").fill_(0xFF)
    dX, dA, dB = lib.lora_multi_bwd(*args, grad_dtype=torch.bfloat16, ws=ws)
    _, (want, tol), (wA, tA), (wB, tB) = reference(*few)
    _near(dX, want, tol, "dX")
    for got, w, t, what in ((dA, wA, tA, "dA"), (dB, wB, tB, "dB")):
        _near(got[used], w, t + 2.0 ** -8 * (w.abs() + t), what)
        assert int((got != 0).flatten(1).any(1).sum()) <= len(used)


@pytest.mark.parametrize("dtype,M,k,d", [(torch.float32, (1 << 24) + 77, 8, 16), (torch.bfloat16, (1 << 24) + 300, 64, 72)])
def test_more_rows_than_a_launch_takes(lib, dtype, M, k, d):
    """Past 2^24 rows: a launch of a block a row would have 2^32 threads.  Workspace of the asked size, between guards."""
    n, r, part = 5, 8, 1 << 20
    gpu = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn(M, k, generator=gpu, device="cuda", dtype=dtype)
    _, W, A, B, scales, _, _ = make(3, 1, k, d, n, r, dtype)
    index = torch.randint(-1, n + 1, (M,), generator=gpu, device="cuda", dtype=torch.int32)
    nb = lib.lib().lora_multi_workspace_bytes(0, 0 if dtype == torch.float32 else 1, M, k, d, n, r, 0, 0)
    room = torch.full((nb + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    Y = lib.lora_multi_fwd(X, W, A, B, scales, index, ws=room[256:256 + nb])
    assert bool((room[:256] == 0xA5).all()) and bool((room[256 + nb:] == 0xA5).all())
    h, one = H[dtype], torch.zeros(1, r, k, dtype=torch.float64, device="cuda")
    a = torch.cat((A.double() * scales.double()[:, None, None], one))  # (row n: none)
    b = torch.cat((B.double(), torch.zeros(1, d, r, dtype=torch.float64, device="cuda")))
    for t in range(0, M, part):
        x, i = X[t:t + part].double(), index[t:t + part].long()
        i = torch.where((i < 0) | (i >= n), n, i)
        want, tol = x @ W.double().T, (k + r + 4) * U * (x.abs() @ W.double().abs().T)
        for e in range(n):
            rows = torch.nonzero(i == e).squeeze(1)
            P, mP = x[rows] @ a[e].T, x[rows].abs() @ a[e].abs().T
            want[rows] += P @ b[e].T
            tol[rows] += (h * P.abs() + (k + 4) * U * mP) @ b[e].abs().T + ((k + r + 4) * U + h) * (mP @ b[e].abs().T)
        _near(Y[t:t + part], want, tol + h * (want.abs() + tol) + 1e-37, t)


# up to 64 rows whose product neither the one-launch kernel nor the W stream takes: dot products for the strips in fp32,
# their part into Y, then the layer's other kernels
DOT_ROWS = [(17, 4096, 1024, 9, 16), (64, 4096, 1024, 16, 64), (33, 2568, 1032, 7, 24), (40, 2056, 8, 3, 8), (64, 8200, 1000, 64, 128)]


@pytest.mark.parametrize("order", ["packed", "random"])
@pytest.mark.parametrize("shape", DOT_ROWS)
def test_few_rows_by_dot_products(lib, shape, order):
    check(lib, make(sum(shape), *shape, torch.bfloat16, order))


@pytest.mark.parametrize("M,k,d", [(40, 4096, 1024), (64, 2568, 1032)])
def test_infinities_of_rows_by_dot_products(lib, M, k, d):
    test_infinities_stay_with_their_own(lib, torch.bfloat16, M, k, d)


@pytest.mark.parametrize("order", ["packed", "random"])
@pytest.mark.parametrize("shape", [(1000, 1000, 4096, 12, 16), (2600, 1000, 4096, 5, 72), (1200, 1544, 14336, 40, 64), (4096, 1000, 4096, 6, 16),
                                   (1000, 4096, 1000, 12, 16), (1200, 14336, 1544, 40, 24), (4096, 4096, 1000, 6, 128)])
def test_ragged_contractions(lib, shape, order):
    """The tile kernels with a last stage of the base product that is not whole, ahead of the adapters' stages: 128 x 256
    and 256 x 256 tiles, a block or two each, Y and dX."""
    check(lib, make(sum(shape), *shape, torch.bfloat16, order))


def test_offsets_past_2_31_elements(lib):
    """X and dX of more than 2^31 elements; dY is zero but for some rows at either end and between."""
    M, k, d, n, r = (1 << 19) + 300, 4104, 64, 6, 16
    gpu = torch.Generator(device="cuda").manual_seed(4)
    X = torch.randn(M, k, generator=gpu, device="cuda", dtype=torch.bfloat16)
    _, W, A, B, scales, _, _ = make(4, 1, k, d, n, r, torch.bfloat16)
    index = torch.randint(-1, n, (M,), generator=gpu, device="cuda", dtype=torch.int32)
    rows = torch.cat([torch.arange(a, a + 300, device="cuda") for a in (0, M // 2 - 7, M - 300)])
    dY = torch.zeros(M, d, device="cuda", dtype=torch.bfloat16)
    dY[rows] = torch.randn(900, d, generator=gpu, device="cuda", dtype=torch.bfloat16)
    Y = lib.lora_multi_fwd(X, W, A, B, scales, index)
    dX, dA, dB = lib.lora_multi_bwd(X, W, A, B, scales, index, dY)
    got = (Y[rows], dX[rows], dA, dB)
    for name, g, (want, tol) in zip(("Y", "dX", "dA", "dB"), got, reference(X[rows], W, A, B, scales, index[rows], dY[rows])):
        _near(g, want, tol, name)
    dX[rows] = 0
    assert not bool(dX.any())
