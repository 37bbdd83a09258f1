"""Token log-probabilities and their gradient against the definition in 64
bits, element by element.

Tolerances (u = 2^-24, one fp32 rounding is off by at most u): an exponential
is off by at most (3 |arg| + 4) u relative (the shifted logit, its product with
tau log2 e, the exponential itself); a row's sum of n = V / threads terms a
thread and the joins of its threads by (n + 24) u more, never fewer than 64
threads.  So log s is off by at most u (V / 64 + 24 + 3 D + 4) + 2 u |log s|,
D = max |tau (z - m)| over the terms that count (e^-D s above 2^-24: D < 40),
and logp by that plus 3 u |tau (z_t - m)|.  A gradient element g (1[j=t] - p)
is off by |g| p times p's relative error, plus one rounding of each of the two
products and the difference, plus the output's rounding (half its eps), plus
|g| 2^-126 where p is below the normals."""
import numpy as np
import pytest
import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _plain(z, t, tau, g=None):
    """logp, m, log s (and dz) in 64 bits on the CPU."""
    z = z.detach().cpu().double()
    t = t.cpu()
    V = z.shape[1]
    m = z.amax(1)
    s = torch.exp((z - m[:, None]) * tau).sum(1)
    has = (t >= 0) & (t < V)
    at = torch.where(has, t, torch.zeros_like(t))
    zt = z.gather(1, at[:, None]).squeeze(1)
    logp = torch.where(has, (zt - m) * tau - s.log(), torch.zeros_like(m))
    if g is None:
        return logp, m, s.log()
    g = torch.where(has, g.cpu().double(), torch.zeros_like(m)) * tau
    p = torch.exp((z - m[:, None]) * tau - s.log()[:, None])
    dz = -g[:, None] * p
    dz[torch.arange(len(t)), at] += g
    return logp, m, s.log(), torch.where(g[:, None] == 0, torch.zeros_like(dz), dz), p, g


def _inputs(seed, n, V, dtype, ignored=True):
    r = torch.Generator().manual_seed(seed)
    z = (torch.randn(n, V, generator=r) * 2.5).to(dtype)
    t = torch.randint(0, V, (n,), generator=r)
    z[torch.arange(n), t] += (torch.rand(n, generator=r) * 16).to(dtype)
    if ignored and n > 2:
        t[n // 3] = -100
        t[n // 2] = V
    return z.cuda(), t.cuda(), torch.randn(n, generator=r).cuda()


def _check(lib, z, t, g, tau, out=None):
    V = z.shape[1]
    z0 = z.clone()
    logp, stats = lib.lora_token_logp_fwd(z, t, tau)
    dz = lib.lora_token_logp_bwd(z, t, stats, g, tau, dlogits=out)
    torch.cuda.synchronize()
    lp, m, ls, d, p, gt = _plain(z0, t, tau, g)
    assert torch.equal(stats[:, 0].cpu().double(), m)
    tol_s = U * (V / 64 + 24 + 3 * 40 + 4 + 2 * ls.abs())
    assert ((stats[:, 1].cpu().double() - ls).abs() <= tol_s).all()
    tol = tol_s + 3 * U * (lp + ls).abs() + U * lp.abs()
    assert ((logp.cpu().double() - lp).abs() <= tol).all()
    arg = ((z0.cpu().double() - m[:, None]) * tau).abs().clamp(max=200) + ls[:, None].abs()
    rel_p = U * (3 * arg + 8) + tol_s[:, None]
    tol_d = gt.abs()[:, None] * (p * rel_p + 3 * U * (p + 1.0 * (d > 0))) + HALF[z.dtype] * d.abs()
    # the hardware exponential flushes p below the smallest normal 2^-126 to 0: |g| p is then at most |g| 2^-126
    # off, and an output below 2^-126 may be flushed itself
    tol_d = tol_d + (gt.abs()[:, None] + 1) * 2.0 ** -126
    err = (dz.cpu().double() - d).abs()
    assert (err <= tol_d).all(), (err - tol_d).max()
    return dz


SHAPES = [(1, 1), (1, 7), (3, 64), (5, 255), (2, 2048), (3, 2049), (24, 32000), (2, 50001), (1100, 2500), (1, 128000)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=[f"{n}x{v}" for n, v in SHAPES])
def test_logp_parity(lib, shape, dtype):
    n, V = shape
    z, t, g = _inputs(11 + n + V, n, V, dtype)
    _check(lib, z, t, g, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("tau", [0.7, 1.25, 8.0])
def test_logp_temperature(lib, tau):
    z, t, g = _inputs(5, 9, 1003, torch.float32)
    _check(lib, z, t, g, tau)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_logp_padded_and_sliced_rows(lib, dtype):
    # rows of a wider buffer, starting one row and 3 columns in: element alignment only
    z, t, g = _inputs(6, 10, 1031, dtype)
    view, tt, gg = z[1:, 3:1004], (t[1:] % 1001).contiguous(), g[1:]
    keep = z.clone()
    out = torch.full((9, 1013), 7.0, dtype=dtype, device="cuda")
    _check(lib, view, tt, gg, 1.0, out=out[:, 5:1006])
    assert torch.equal(z, keep)  # inputs untouched
    assert (out[:, :5] == 7).all() and (out[:, 1006:] == 7).all()  # and what lies beside the rows
    # sliced targets of the whole rows (t[1:] starts 8 bytes into its buffer)
    _check(lib, z[:-1], t[1:], g[1:], 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [77, 4099])
def test_logp_in_place(lib, V, dtype):
    z, t, g = _inputs(8, 33, V, dtype)
    _, stats = lib.lora_token_logp_fwd(z, t)
    apart = lib.lora_token_logp_bwd(z, t, stats, g)
    lib.lora_token_logp_bwd(z, t, stats, g, dlogits=z)
    assert torch.equal(z, apart)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_logp_masked_vocabulary(lib, dtype):
    # columns of -inf and of the type's lowest value have probability 0
    z, t, g = _inputs(9, 6, 3001, dtype, ignored=False)
    t = t % 1000
    z[:, 1000:2000] = -float("inf")
    z[:, 2000:] = torch.finfo(dtype).min
    z[2, :1000] = -float("inf")
    z[2, t[2]] = 0.5  # one finite column
    lp, stats = lib.lora_token_logp_fwd(z, t)
    dz = lib.lora_token_logp_bwd(z, t, stats, g)
    ref, m, ls, d, _, _ = _plain(z, t, 1.0, g)
    assert torch.equal(stats[:, 0].cpu().double(), m)
    assert torch.allclose(lp.cpu().double(), ref, rtol=0, atol=2e-5) and lp[2] == 0
    assert (dz[:, 1000:] == 0).all()
    assert torch.allclose(dz.cpu().double(), d, rtol=HALF[dtype], atol=1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_logp_not_finite(lib, dtype):
    z, t, g = _inputs(10, 6, 2500, dtype, ignored=False)
    z[0] = -float("inf")
    z[1, 17] = float("nan")
    z[2, 2499] = float("inf")
    t[3] = 5
    z[3, 5] = -float("inf")
    lp, stats = lib.lora_token_logp_fwd(z, t)
    dz = lib.lora_token_logp_bwd(z, t, stats, g)
    assert lp[:3].isnan().all() and lp[3] == -float("inf") and lp[4:].isfinite().all()
    assert dz[0].isnan().all() and dz[1].isnan().all() and dz[3:].isfinite().all()
    # rows that carry no gradient are not read
    t[1], g[0], g[2] = -100, 0.0, 0.0
    lp, stats = lib.lora_token_logp_fwd(z, t)
    dz = lib.lora_token_logp_bwd(z, t, stats, g)
    assert lp[1] == 0 and (dz[:3] == 0).all() and dz[3:].isfinite().all()


@pytest.mark.gpu
def test_logp_no_rows(lib):
    z = torch.empty(0, 50, dtype=torch.bfloat16, device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    lp, stats = lib.lora_token_logp_fwd(z, t)
    assert lp.shape == (0,) and stats.shape == (0, 2)
    assert lib.lora_token_logp_bwd(z, t, stats, lp).shape == (0, 50)


@pytest.mark.gpu
def test_logp_offsets_past_32_bits(lib):
    # 2^32 elements and more: rows at both ends against the same rows alone
    n, V = 33100, 130003
    z = torch.empty(n, V, dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, 16517, 33036, n - 1]
    z.zero_()
    small, t_s, g_s = _inputs(12, len(rows), V, torch.bfloat16, ignored=False)
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    g = torch.zeros(n, device="cuda")
    for k, r in enumerate(rows):
        z[r], t[r], g[r] = small[k], t_s[k], g_s[k]
    lp, stats = lib.lora_token_logp_fwd(z, t)
    lp_s, stats_s = lib.lora_token_logp_fwd(small, t_s)
    at = torch.tensor(rows, device="cuda")
    # (the few rows run with other threads a row: sums in another order)
    assert torch.equal(stats[at, 0], stats_s[:, 0]) and torch.allclose(lp[at], lp_s, rtol=0, atol=1e-4)
    dz = lib.lora_token_logp_bwd(z, t, stats, g)
    assert torch.equal(dz[at], lib.lora_token_logp_bwd(small, t_s, stats[at], g_s))
    assert (dz[2] == 0).all() and (dz[n - 2] == 0).all()


@pytest.mark.gpu
def test_logp_function_gradient_against_differences(lib):
    # d/dz of sum g logp: central differences of the 64-bit definition at the same point
    z, t, g = _inputs(13, 3, 11, torch.float32, ignored=False)
    leaf = z.clone().requires_grad_()
    lib.LoraTokenLogpFunction.apply(leaf, t, 0.9).backward(g)
    z64, h = z.cpu().double(), 1e-5
    for i in range(3):
        for j in range(11):
            up, dn = z64.clone(), z64.clone()
            up[i, j] += h
            dn[i, j] -= h
            num = ((_plain(up, t, 0.9)[0] - _plain(dn, t, 0.9)[0]) * g.cpu().double()).sum() / (2 * h)
            assert abs(float(leaf.grad[i, j]) - float(num)) <= 1e-5 * (1 + abs(float(num)))


@pytest.mark.gpu
def test_logp_on_another_stream_and_captured(lib):
    z, t, g = _inputs(14, 40, 3000, torch.bfloat16)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    want = lib.lora_token_logp_fwd(z, t)
    dwant = lib.lora_token_logp_bwd(z, t, want[1], g)
    with torch.cuda.stream(st):
        got = lib.lora_token_logp_fwd(z, t)
        lib.lora_token_logp_bwd(z, t, got[1], g)
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        glp, gst = lib.lora_token_logp_fwd(z, t)
        gdz = lib.lora_token_logp_bwd(z, t, gst, g)
    for k in range(3):
        z.copy_(torch.roll(z, 1, 0))
        t.copy_(torch.roll(t, 1, 0))
        want = lib.lora_token_logp_fwd(z, t)
        dwant = lib.lora_token_logp_bwd(z, t, want[1], g)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(glp, want[0]) and torch.equal(gdz, dwant)


def test_logp_refusals():
    import lora_linear_layers_amd as L

    z, t = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        L.lora_token_logp_fwd(z, t)
    with pytest.raises(ValueError, match="vocab"):
        L.lora_token_logp_fwd(z.view(-1), t)
    with pytest.raises(ValueError, match="rows"):
        L.lora_token_logp_fwd(z.t(), t)
    lib = L.lib()
    P = 0x100000

    def fwd(dtype=1, n=4, V=8, z=P, ld=8, t=P, tau=1.0, lp=P, st=P):
        return lib.lora_token_logp_fwd(dtype, n, V, z, ld, t, tau, lp, st, None)

    def bwd(dtype=1, n=4, V=8, z=P, ld=8, t=P, tau=1.0, st=P, g=P, dz=P, ldd=8):
        return lib.lora_token_logp_bwd(dtype, n, V, z, ld, t, tau, st, g, dz, ldd, None)

    for f in (fwd, bwd):
        assert f(dtype=2) == -4
        assert f(n=-1) == -2 and f(V=0) == -2 and f(ld=7) == -2 and f(V=2 ** 31, ld=2 ** 31) == -2
        assert f(tau=0.0) == -2 and f(tau=-1.0) == -2 and f(tau=float("nan")) == -2 and f(tau=float("inf")) == -2
        assert f(tau=1.1e38) == -2  # tau log2 e would be infinite
        assert f(z=None) == -1 and f(t=None) == -1 and f(st=None) == -1
        assert f(z=P + 1) == -3 and f(dtype=0, z=P + 2) == -3 and f(t=P + 4) == -3 and f(st=P + 2) == -3
    assert fwd(lp=None) == -1 and fwd(lp=P + 2) == -3
    assert bwd(g=None) == -1 and bwd(dz=None) == -1 and bwd(ldd=7) == -2
    assert bwd(dz=P, z=P, ldd=9) == -2  # in place with another stride
    if torch.cuda.device_count() == 0:
        assert fwd(z=P + 2, t=P + 8) == -6  # element alignment is enough: only the device is missing


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [2, 64, 777, 2500, 50001])
@pytest.mark.parametrize("tau", [1.0, 0.75])
def test_logp_of_confident_rows_keeps_its_digits(lib, V, dtype, tau):
    # a target that stands far out: logp = -log(1 + rest) with rest = sum of the others' e^(tau (z_j - z_t)), down to
    # 1e-30, and the target's gradient g (1 - p).  Relative tolerance: rest's terms are off by (3 D + 4) u each, once
    # more for their rescaling on the way (D = the largest tau |z_j - z_t|, at most one rescaling a vector of 4 and one
    # a join, 6 u each), their sum by V / 64 u, log1p and the last products by 16 u
    r = torch.Generator().manual_seed(V)
    margins = [4.0, 9.0, 13.8, 14.5, 17.0, 25.0, 40.0, 80.0]
    n = 3 * len(margins)
    z = (torch.randn(n, V, generator=r) * 0.5).to(dtype)
    t = torch.tensor([(0, V - 1, V // 2 + i % 7)[i % 3] % V for i in range(n)])
    z[torch.arange(n), t] = torch.tensor([margins[i // 3] for i in range(n)]).to(dtype)
    g = torch.randn(n, generator=r).cuda()
    lp, stats = lib.lora_token_logp_fwd(z.cuda(), t.cuda(), tau)
    dz = lib.lora_token_logp_bwd(z.cuda(), t.cuda(), stats, g, tau)
    a = (z.double() - z.double().gather(1, t[:, None])) * tau
    e = a.exp()
    e[torch.arange(n), t] = 0  # (not subtracted afterwards: 1 + rest - 1 would lose the digits here too)
    rest = e.sum(1)
    want = -torch.log1p(rest)
    rel = U * (6 * a.abs().amax(1) + 4 + 6 * (V / 256 + 24) + V / 64 + 16)
    got = lp.cpu().double()
    assert ((got - want).abs() <= rel * want.abs() + 2.0 ** -126).all(), ((got - want) / want).abs().max()
    assert ((stats[:, 1].cpu().double() + want).abs() <= rel * want.abs() + 2.0 ** -126).all()
    at = dz.cpu().double()[torch.arange(n), t]
    wd = g.cpu().double() * tau * rest / (1 + rest)
    assert ((at - wd).abs() <= (rel + HALF[dtype]) * wd.abs() + 2.0 ** -125).all(), ((at - wd) / wd).abs().max()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 5, 9, 64, 2049, 50001])
def test_logp_of_tied_maxima(lib, V, dtype):
    # k elements share the maximum, wherever they lie (one vector, neighbouring ones, the row's ends): the row's sum
    # is k and every tied element's probability 1 / k
    r = torch.Generator().manual_seed(V)
    sets = [[0], [V - 1], [0, V - 1], list(range(min(V, 3))), list(range(min(V, 8))), list(range(max(0, V - 9), V)),
            list(range(V)), torch.randperm(V, generator=r)[:min(V, 40)].tolist()]
    z = torch.full((len(sets), V), -200.0)
    for i, s in enumerate(sets):
        z[i, s] = 3.5
    t = torch.tensor([s[len(s) // 2] for s in sets]).cuda()
    k = torch.tensor([float(len(set(s))) for s in sets]).double()
    z = z.to(dtype).cuda()
    lp, stats = lib.lora_token_logp_fwd(z, t)
    dz = lib.lora_token_logp_bwd(z, t, stats, torch.ones(len(sets), device="cuda"))
    assert (stats[:, 0] == 3.5).all()
    assert ((lp.cpu().double() + k.log()).abs() <= 4 * U * k.log()).all()
    at = dz.cpu().double()[torch.arange(len(sets)), t.cpu()]
    assert ((at - (1 - 1 / k)).abs() <= (HALF[dtype] + 40 * U) * (1 - 1 / k)).all()


@pytest.mark.gpu
def test_logp_infinite_row_with_one_vector(lib):
    # +infinity as the only element, in a vector of its own and beside a NaN: NaN, not a finite sum of the rest
    z = torch.zeros(4, 9, device="cuda")
    z[0, 0] = z[1, 8] = z[2, 3] = float("inf")
    z[3, 1], z[3, 2] = float("inf"), float("nan")
    t = torch.tensor([0, 8, 5, 1], device="cuda")
    lp, _ = lib.lora_token_logp_fwd(z, t)
    assert lp.isnan().all()
    assert lib.lora_token_logp_fwd(z[:1, :1], t[:1])[0].isnan().all()


@pytest.mark.gpu
def test_logp_gradient_on_another_stream(lib):
    z, t, g = _inputs(15, 40, 3000, torch.bfloat16)
    want = lib.lora_token_logp_fwd(z, t)
    dwant = lib.lora_token_logp_bwd(z, t, want[1], g)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = lib.lora_token_logp_fwd(z, t)
        dgot = lib.lora_token_logp_bwd(z, t, got[1], g)
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]) and torch.equal(dwant, dgot)


@pytest.mark.gpu
def test_logp_fp32_logits_past_the_caches(lib):
    # above 256 MB the gradient streams past the caches: the same bits as the same rows alone, and those right
    n, V = 1400, 50001
    small, t_s, g_s = _inputs(16, 8, V, torch.float32, ignored=False)
    z, t, g = small.repeat(n // 8, 1), t_s.repeat(n // 8), g_s.repeat(n // 8)
    assert z.numel() * 4 > 256 << 20
    _check(lib, small.clone(), t_s, g_s, 1.25)
    lp_s, stats_s = lib.lora_token_logp_fwd(small, t_s, 1.25)
    want = lib.lora_token_logp_bwd(small, t_s, stats_s, g_s, 1.25)
    lp, stats = lib.lora_token_logp_fwd(z, t, 1.25)
    assert torch.equal(lp.view(-1, 8), lp_s.expand(n // 8, 8)) and torch.equal(stats, stats_s.repeat(n // 8, 1))
    apart = lib.lora_token_logp_bwd(z, t, stats, g, 1.25)
    assert torch.equal(apart.view(-1, 8, V), want.expand(n // 8, 8, V))
    lib.lora_token_logp_bwd(z, t, stats, g, 1.25, dlogits=z)
    assert torch.equal(z, apart)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,V", [(torch.float32, 8), (torch.bfloat16, 9)], ids=["f32", "bf16"])
def test_logp_more_rows_than_blocks(lib, dtype, V):
    # blocks take several rows (2^20 of them) and the gradient's several segments (2^22): every row against its
    # definition in 64 bits, at the bounds of the head of this file
    n = (1 << 22) + 5
    gen = torch.Generator("cuda").manual_seed(17)
    z = (torch.randn(n, V, generator=gen, device="cuda") * 2.5).to(dtype)
    t = torch.randint(-1, V, (n,), generator=gen, device="cuda")
    g = torch.randn(n, generator=gen, device="cuda")
    lp, stats = lib.lora_token_logp_fwd(z, t)
    dz = lib.lora_token_logp_bwd(z, t, stats, g)
    full = torch.log_softmax(z.double(), 1)
    has = t >= 0
    at = t.clamp(min=0)[:, None]
    want = torch.where(has, full.gather(1, at).squeeze(1), 0.0)
    tol = U * (V / 64 + 24 + 3 * 40 + 4 + 8 * (full.abs().amax(1) + 1))
    assert torch.equal(stats[:, 0], z.float().amax(1))
    assert ((lp.double() - want).abs() <= tol).all()
    gz = torch.where(has, g, 0.0).double()[:, None]
    d = -gz * full.exp()
    d.scatter_add_(1, at, gz)
    err = (dz.double() - d).abs()
    assert (err <= gz.abs() * (tol[:, None] + 8 * U) + HALF[dtype] * d.abs() + 2.0 ** -126).all()
