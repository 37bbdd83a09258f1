"""The preference and the clipped policy loss over packed sequences against
their definitions in 64 bits.

Tolerances (u = 2^-24): the preference loss is formed in 64 bits from fp32
inputs, so an output is off by its one rounding (u) and the sums' own error
(2^-52 of the sum of magnitudes, times beta or 2 u for the ipo loss: covered by
an absolute 1e-9 of that sum); a gradient has three roundings (coef, its
product with dloss).  A policy token's ratio is off by at most
(2 + |x|) 2 u relative (x rounded to fp32, then e^x), the KL term's value by
8 u relative plus 2e-9 of d^2 and its slope by (2 + |d|) 2 u of e^d plus u;
weight, dloss and their product add 3 u."""
import math

import numpy as np
import pytest
import torch

U = 2.0 ** -24
NAN = float("nan")


def _packed(lens, lead=0, tail=0):
    cu = lead + np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    return cu, int(cu[-1]) + tail


def _draw(seed, n):
    r = np.random.default_rng(seed)
    ref = -2.5 * r.exponential(size=n)
    lp = ref + 0.3 * r.normal(size=n)
    old = lp + 0.15 * r.normal(size=n)
    return (lp.astype(np.float32), ref.astype(np.float32), old.astype(np.float32), r.random(n) > 0.25,
            r.normal(size=n).astype(np.float32))


def _dev(*xs):
    return [None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in xs]


# ---------------------------------------------------------------------------
# preference
# ---------------------------------------------------------------------------
def _pref_plain(lp, ref, cu, mask, beta, kind, eps, average, dloss=1.0):
    P, n = (len(cu) - 1) // 2, len(lp)
    D, cnt, mag = np.zeros(2 * P), np.zeros(2 * P), np.zeros(2 * P)
    keep = np.ones(n, bool) if mask is None else mask.astype(bool)
    for s in range(2 * P):
        at = np.arange(cu[s], cu[s + 1])
        at = at[keep[at]]
        x = lp[at].astype(np.float64) - (0 if ref is None else ref[at].astype(np.float64))
        cnt[s] = len(at)
        D[s], mag[s] = math.fsum(x) if np.isfinite(x).all() else x.sum(), np.abs(x).sum()
    per = 1 / np.maximum(cnt, 1) if average else np.ones(2 * P)
    D, mag = D * per, mag * per
    u = D[:P] - D[P:]
    sp = lambda x: np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))  # noqa: E731
    if kind == "sigmoid":
        l = (1 - eps) * sp(-beta * u) + (eps * sp(beta * u) if eps else 0)
        du = -beta * (1 - eps) / (1 + np.exp(beta * u)) + (beta * eps / (1 + np.exp(-beta * u)) if eps else 0)
    elif kind == "hinge":
        l, du = np.maximum(1 - beta * u, 0), np.where(beta * u < 1, -beta, 0.0)
    else:
        l, du = (u - 0.5 / beta) ** 2, 2 * (u - 0.5 / beta)
    coef = np.concatenate([du, -du]) * per / P
    d = np.zeros(n)
    for s in range(2 * P):
        d[cu[s]:cu[s + 1]] = np.where(keep[cu[s]:cu[s + 1]], coef[s] * dloss, 0)
    return l.mean(), l, beta * D, d, mag.sum()


def _near(got, want, rtol, atol):
    got = got.detach().cpu().double().numpy()
    want = np.asarray(want, np.float64)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= rtol * np.abs(want) + atol)
    assert not bad.any(), (got[bad][:4], want[bad][:4], int(bad.sum()))


def _pref_check(lib, lens, kind="sigmoid", eps=0.0, average=False, reference=True, masked=True, beta=0.1, lead=0, tail=0,
                seed=1, dloss=0.5):
    cu, n = _packed(lens, lead, tail)
    lp, ref, _, mask, _ = _draw(seed, n)
    mask = mask if masked else None
    if masked and n:  # what does not count may hold anything
        lp, ref = np.where(mask, lp, NAN), np.where(mask, ref, -np.inf).astype(np.float32)
    if lead:
        lp[:lead] = np.inf
    if tail:
        lp[-tail:] = NAN
    ref = ref if reference else None
    dev = _dev(lp, ref, cu, mask)
    loss, pair, rew, coef = lib.lora_preference_loss_fwd(dev[0], dev[2], beta, dev[1], dev[3], kind, eps, average)
    d = lib.lora_preference_loss_bwd(coef, dev[2], n, dev[3], torch.tensor(dloss, device="cuda"))
    wl, wp, wr, wd, mag = _pref_plain(lp, ref, cu, mask, beta, kind, eps, average, dloss)
    a = 1e-9 * max(mag, 1.0)
    _near(loss, wl, 2 * U, a)
    _near(pair, wp, 2 * U, a)
    _near(rew, wr, 2 * U, a)
    _near(d, wd, 4 * U, 1e-9 * max(mag, 1.0) / max(1, len(lens)))
    return dev, coef


PREF_LENS = {
    "one pair of one token": [1, 1],
    "two pairs": [300, 1, 7, 260],
    "empty ones": [0, 5, 64, 0, 0, 65, 0, 3],
    "all empty": [0, 0],
    "around a chunk": [256, 255, 257, 512, 1, 63],
    "one long among short": [3, 20000, 2, 5, 1, 4],
    "many short": list(np.random.default_rng(5).integers(0, 4, 2 * 3000)),
    "a batch": list(np.random.default_rng(6).integers(200, 900, 2 * 60)),
}


@pytest.mark.gpu
@pytest.mark.parametrize("lens", PREF_LENS.values(), ids=PREF_LENS.keys())
def test_preference_lengths(lib, lens):
    _pref_check(lib, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,eps", [("sigmoid", 0.0), ("sigmoid", 0.2), ("hinge", 0.0), ("ipo", 0.0)])
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("reference,masked", [(True, True), (True, False), (False, True), (False, False)])
def test_preference_kinds(lib, kind, eps, average, reference, masked):
    _pref_check(lib, [40, 0, 333, 12, 80, 1], kind, eps, average, reference, masked, seed=3)


@pytest.mark.gpu
@pytest.mark.parametrize("total", [8191, 8192, 8193, 70000])
def test_preference_both_sides_of_the_small_form(lib, total):
    _pref_check(lib, [total // 3, total // 5, total // 4, total - total // 3 - total // 5 - total // 4], seed=total)


@pytest.mark.gpu
def test_preference_tokens_outside_the_sequences(lib):
    _pref_check(lib, [70, 10, 0, 300], lead=130, tail=700)
    _pref_check(lib, [70, 10, 0, 30000], lead=1300, tail=70000)


@pytest.mark.gpu
def test_preference_all_masked_and_infinite(lib):
    lp, cu = torch.tensor([-1.0, -2.0, -3.0], device="cuda"), torch.tensor([0, 2, 3], device="cuda")
    none = torch.zeros(3, dtype=torch.uint8, device="cuda")
    for average in (False, True):
        loss, pair, rew, coef = lib.lora_preference_loss_fwd(lp, cu, 0.5, mask=none, average=average)
        assert abs(float(loss) - math.log(2)) < 1e-7 and (rew == 0).all()
        assert (lib.lora_preference_loss_bwd(coef, cu, 3, none) == 0).all()
    # a response of probability zero: the margin is infinite, the loss 0 or infinite, never a NaN
    lp[2] = -float("inf")
    loss, _, _, coef = lib.lora_preference_loss_fwd(lp, cu, 0.5)
    assert float(loss) == 0 and (coef == 0).all()
    loss, _, _, coef = lib.lora_preference_loss_fwd(torch.tensor([-float("inf"), 0, 0], device="cuda"), cu, 0.5)
    assert float(loss) == float("inf") and torch.allclose(coef.cpu(), torch.tensor([-0.5, 0.5]))
    lp[0] = NAN
    assert torch.isnan(lib.lora_preference_loss_fwd(lp, cu, 0.5, kind="hinge")[0])


@pytest.mark.gpu
def test_preference_gradient_against_differences(lib):
    cu, n = _packed([4, 3, 5, 2])
    lp, ref, _, mask, _ = _draw(21, n)
    for kind, eps, average in (("sigmoid", 0.1, False), ("ipo", 0.0, True)):
        dev = _dev(lp, ref, cu, mask)
        x = dev[0].requires_grad_()
        loss, pair, rew = lib.LoraPreferenceLossFunction.apply(x, dev[1], dev[2], dev[3], 0.3, kind, eps, average)
        assert not pair.requires_grad and not rew.requires_grad
        loss.backward()
        for t in range(n):
            up, dn = lp.astype(np.float64), lp.astype(np.float64)
            up[t] += 1e-5
            dn[t] -= 1e-5
            f = lambda v: _pref_plain(v, ref, cu, mask, 0.3, kind, eps, average)[0]  # noqa: E731
            assert abs(float(x.grad[t]) - (f(up) - f(dn)) / 2e-5) <= 1e-6


# ---------------------------------------------------------------------------
# policy
# ---------------------------------------------------------------------------
def _policy_plain(lp, old, ref, adv, cu, mask, lo, hi, beta, reduction, norm, per_token, dloss=1.0):
    S, n = len(cu) - 1, len(lp)
    f = lambda v: None if v is None else v.astype(np.float64)  # noqa: E731
    lp, old, ref, adv = f(lp), f(old), f(ref), f(adv)
    keep = np.ones(n, bool) if mask is None else mask.astype(bool)
    seq = np.full(n, -1)
    for s in range(S):
        seq[cu[s]:cu[s + 1]] = s
    keep = keep & (seq >= 0)
    T = np.array([keep[cu[s]:cu[s + 1]].sum() for s in range(S)])
    tot = max(T.sum(), 1)
    w = {"sequence": 1 / (S * np.maximum(T, 1.0)), "token": np.full(S, 1 / tot),
         "constant": np.full(S, 1 / (S * norm))}[reduction]
    pol, kl, cut, d, tol = 0.0, 0.0, 0, np.zeros(n), np.zeros(n)
    mag = 0.0
    for t in np.flatnonzero(keep):
        A = adv[t] if per_token else adv[seq[t]]
        x = 0.0 if old is None else lp[t] - old[t]
        over, under = A > 0 and x > math.log1p(hi), A < 0 and x < (math.log1p(-lo) if lo < 1 else -math.inf)
        r = math.exp(x)
        used = 1 + hi if over else (1 - lo if under else r)
        W = w[seq[t]]
        pol += W * (-used * A if A else 0)
        e = math.expm1(ref[t] - lp[t]) if ref is not None else 0.0
        dd = ref[t] - lp[t] if ref is not None else 0.0
        kl += W * (e - dd)
        cut += over or under
        g = (0 if over or under or A == 0 else -r * A) - beta * e
        d[t] = W * g * dloss
        tol[t] = W * dloss * (abs(r * A) * (2 + abs(x)) * 2 * U + beta * ((e + 1) * (2 + abs(dd)) * 2 * U + U)) + \
            4 * U * abs(d[t]) + 1e-37
        mag += W * (abs(used * A) * (2 + abs(x)) * 2 * U + (e - dd) * 10 * U + dd * dd * 2e-9)
    return pol + beta * kl, (pol, kl, cut / tot, T.sum()), d, tol, mag


def _policy_check(lib, lens, reduction="sequence", per_token=False, beta=0.04, with_old=True, with_ref=True, masked=True,
                  lo=0.2, hi=0.28, lead=0, tail=0, seed=1, dloss=0.5):
    cu, n = _packed(lens, lead, tail)
    S = len(lens)
    lp, ref, old, mask, adv = _draw(seed, n)
    adv = adv if per_token else np.random.default_rng(seed + 1).normal(size=S).astype(np.float32)
    mask = mask if masked else None
    if masked and n:
        lp, old = np.where(mask, lp, NAN), np.where(mask, old, np.inf).astype(np.float32)
        if per_token:
            adv = np.where(mask, adv, NAN).astype(np.float32)
    if lead:
        lp[:lead] = NAN
    if tail:
        lp[-tail:] = np.inf
    old, ref = old if with_old else None, ref if with_ref else None
    L, O, R, A, C, M = _dev(lp, old, ref, adv, cu, mask)
    kw = dict(old_logp=O, ref_logp=R, mask=M, eps_low=lo, eps_high=hi, beta=beta, per_token=per_token)
    loss, stats, weight = lib.lora_policy_loss_fwd(L, C, A, reduction=reduction, norm=37.5, **kw)
    d = lib.lora_policy_loss_bwd(L, C, A, weight, dloss=torch.tensor(dloss, device="cuda"), **kw)
    wl, ws, wd, tol, mag = _policy_plain(lp, old, ref, adv, cu, mask, lo, hi, beta, reduction, 37.5, per_token, dloss)
    _near(loss, wl, 2 * U, mag)
    _near(stats[0], ws[0], 2 * U, mag)
    _near(stats[1], ws[1], 2 * U, mag)
    _near(stats[2:], ws[2:], 2 * U, 0)
    got = d.cpu().double().numpy()
    assert (np.abs(got - wd) <= tol).all(), np.max(np.abs(got - wd) - tol)


POLICY_LENS = {
    "one token": [1],
    "a group": [250, 3, 0, 64, 191, 1, 77, 256],
    "all empty": [0, 0, 0],
    "one long among short": [5, 30000, 0, 2],
    "many short": list(np.random.default_rng(7).integers(0, 4, 5000)),
    "a batch": list(np.random.default_rng(8).integers(100, 700, 60)),
}


@pytest.mark.gpu
@pytest.mark.parametrize("lens", POLICY_LENS.values(), ids=POLICY_LENS.keys())
def test_policy_lengths(lib, lens):
    _policy_check(lib, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("reduction", ["sequence", "token", "constant"])
@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("beta,with_ref", [(0.0, False), (0.0, True), (0.1, True)])
@pytest.mark.parametrize("with_old,masked", [(True, True), (False, False)])
def test_policy_forms(lib, reduction, per_token, beta, with_ref, with_old, masked):
    _policy_check(lib, [30, 0, 100, 1, 65], reduction, per_token, beta, with_old, with_ref, masked, seed=4)


@pytest.mark.gpu
@pytest.mark.parametrize("total", [8191, 8192, 8193])
def test_policy_both_sides_of_the_small_form(lib, total):
    _policy_check(lib, [total // 2, total - total // 2], seed=total)


@pytest.mark.gpu
def test_policy_tokens_outside_the_sequences(lib):
    _policy_check(lib, [70, 10, 0, 300], per_token=True, lead=130, tail=700)
    _policy_check(lib, [70, 10, 0, 9000], lead=1300, tail=3000)


@pytest.mark.gpu
def test_policy_clip_borders(lib):
    # logp - old exactly at, one step inside and one step outside each border, both signs of the advantage
    lo, hi = 0.2, 0.28
    for border in (math.log1p(hi), math.log1p(-lo)):
        b = np.float32(border)
        x = np.array([np.nextafter(b, np.float32(-9)), b, np.nextafter(b, np.float32(9))], np.float32)
        for sign in (1.0, -1.0):
            lp, old = x, np.zeros(3, np.float32)
            L, O, A, C = _dev(lp, old, np.array([sign], np.float32), np.array([0, 3], np.int64))
            loss, stats, w = lib.lora_policy_loss_fwd(L, C, A, old_logp=O, eps_low=lo, eps_high=hi)
            d = lib.lora_policy_loss_bwd(L, C, A, w, old_logp=O, eps_low=lo, eps_high=hi)
            x64 = x.astype(np.float64)
            cut = (x64 > math.log1p(hi)) if sign > 0 else (x64 < math.log1p(-lo))
            assert ((d.cpu().numpy() == 0) == cut).all()
            assert abs(float(stats[2]) - cut.mean()) < 1e-7
    _policy_check(lib, [50, 20], lo=1.0, hi=0.0)  # no lower border; every rise clipped
    _policy_check(lib, [50, 20], lo=0.0, hi=5.0)


@pytest.mark.gpu
def test_policy_zero_advantage_and_overflow(lib):
    # A = 0 leaves the KL term alone even where the ratio overflows; A > 0 is clipped there
    L, O, R, A, C = _dev(np.array([200.0, 200.0, -1.0], np.float32), np.array([0.0, 0.0, -1.0], np.float32),
                         np.array([200.0, 200.0, -1.0], np.float32), np.array([0.0, 2.0, 1.0], np.float32),
                         np.array([0, 1, 2, 3], np.int64))
    loss, stats, w = lib.lora_policy_loss_fwd(L, C, A, old_logp=O, ref_logp=R, beta=0.1, eps_high=0.5)
    assert abs(float(loss) + (0 + 3 + 1) / 3) < 1e-6 and float(stats[1]) == 0
    d = lib.lora_policy_loss_bwd(L, C, A, w, old_logp=O, ref_logp=R, beta=0.1, eps_high=0.5)
    assert (d[:2] == 0).all() and abs(float(d[2]) + 1 / 3) < 1e-6


@pytest.mark.gpu
def test_policy_kl_of_near_equal_policies(lib):
    # e^d - d - 1 of tiny d: d^2 / 2 to fp32, where the plain difference has no digit left
    for d0 in (0.0, 1e-6, 3e-4, 0.01, 0.2499, 0.2501, -0.25, -1e-5, 3.0, -30.0):
        ref = np.array([np.float32(d0)], np.float32)
        L, R, A, C = _dev(np.zeros(1, np.float32), ref, np.zeros(1, np.float32), np.array([0, 1], np.int64))
        kl = float(lib.lora_policy_loss_fwd(L, C, A, ref_logp=R, beta=1.0)[0])
        x = float(ref[0])
        want = math.expm1(x) - x if abs(x) > 0.05 else x * x * (1 / 2 + x / 6 + x * x / 24 + x ** 3 / 120 + x ** 4 / 720)
        assert abs(kl - want) <= 12 * U * want + 2e-9 * x * x * (abs(x) < 0.25) + 3 * U * abs(math.expm1(x)) * (abs(x) >= 0.25)


@pytest.mark.gpu
def test_policy_kl_gradient_of_distant_policies(lib):
    # 1 - e^d keeps its digits where d itself has none left for it, and where the reference's probability is 0
    lp = np.zeros(12, np.float32)
    ref = np.array([-0.49, -0.51, -17.3, -1000.3, -123456.7, -3.0e8, -np.inf, 0.49, 0.51, 17.3, 80.2, 0.0], np.float32)
    L, R, A, C = _dev(lp, ref, np.zeros(12, np.float32), np.arange(13, dtype=np.int64))
    _, _, w = lib.lora_policy_loss_fwd(L, C, A, ref_logp=R, beta=0.5, reduction="constant", norm=1.0)
    got = lib.lora_policy_loss_bwd(L, C, A, w, ref_logp=R, beta=0.5).cpu().double().numpy()
    d = ref.astype(np.float64)
    e = np.array([math.expm1(x) for x in d])
    # the slope's bound of the head of this file, and 3 roundings of the products
    shift = np.where(np.isinf(d), 0, np.abs(d))
    tol = 0.5 / 12 * (np.where(np.isinf(d), 0, np.exp(d)) * (2 + shift) * 2 * U + U) + 4 * U * np.abs(0.5 * e / 12)
    assert (np.abs(got + 0.5 * e / 12) <= tol).all(), got * -24 - e


@pytest.mark.gpu
def test_policy_gradient_against_differences(lib):
    cu, n = _packed([4, 0, 6, 3])
    lp, ref, old, mask, _ = _draw(31, n)
    adv = np.array([0.7, 1.0, -1.2, 0.4], np.float32)
    L, O, R, A, C, M = _dev(lp, old, ref, adv, cu, mask)
    x = L.requires_grad_()
    loss, stats = lib.LoraPolicyLossFunction.apply(x, O, R, C, A, M, 0.2, 0.28, 0.05, "token")
    assert not stats.requires_grad
    loss.backward()
    f = lambda v: _policy_plain(v, old, ref, adv, cu, mask, 0.2, 0.28, 0.05, "token", 1.0, False)[0]  # noqa: E731
    for t in range(n):
        up, dn = lp.astype(np.float64), lp.astype(np.float64)
        up[t] += 1e-6
        dn[t] -= 1e-6
        assert abs(float(x.grad[t]) - (f(up) - f(dn)) / 2e-6) <= 1e-6


# ---------------------------------------------------------------------------
# both
# ---------------------------------------------------------------------------
@pytest.mark.gpu
def test_losses_bad_offsets_stay_in_the_arrays(lib):
    # offsets past the ends are taken as the ends; decreasing ones give some value, and guards stay untouched
    n = 3000
    lp = torch.full((n + 64,), -1.0, device="cuda")
    cu = torch.tensor([-50, 1000, n + 999], device="cuda")
    loss, _, rew, coef = lib.lora_preference_loss_fwd(lp[:n], cu, 1.0)
    assert torch.allclose(rew.cpu(), torch.tensor([-1000.0, -2000.0]))
    out = torch.full((n + 64,), 7.0, device="cuda")
    bad = torch.tensor([2000, 10, 5, 2999, 17], device="cuda")
    _, _, _, coef = lib.lora_preference_loss_fwd(lp[:n], bad, 1.0)
    d = lib.lora_preference_loss_bwd(coef, bad, n)
    adv = torch.ones(4, device="cuda")
    _, _, w = lib.lora_policy_loss_fwd(lp[:n], bad, adv)
    d2 = lib.lora_policy_loss_bwd(lp[:n], bad, adv, w)
    torch.cuda.synchronize()
    assert d.shape == (n,) and d2.shape == (n,) and (out == 7).all()


@pytest.mark.gpu
def test_losses_repeat_bit_for_bit_and_captured(lib):
    lens = list(np.random.default_rng(9).integers(0, 700, 200))
    cu, n = _packed(lens)
    lp, ref, old, mask, _ = _draw(41, n)
    L, R, O, C, M = _dev(lp, ref, old, cu, mask)
    A = torch.randn(len(lens), generator=torch.Generator().manual_seed(1)).cuda()
    g = torch.tensor(1.5, device="cuda")

    def both():
        loss, pair, rew, coef = lib.lora_preference_loss_fwd(L, C, 0.1, R, M)
        d = lib.lora_preference_loss_bwd(coef, C, n, M, g)
        ploss, stats, w = lib.lora_policy_loss_fwd(L, C, A, O, R, M, beta=0.04)
        pd = lib.lora_policy_loss_bwd(L, C, A, w, O, R, M, beta=0.04, dloss=g)
        return loss, pair, rew, d, ploss, stats, pd

    first = both()
    for a, b in zip(first, both()):
        assert torch.equal(a, b)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = both()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for k in range(3):
        L.add_(0.01)
        want = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held))


@pytest.mark.gpu
def test_head_to_preference_loss(lib):
    """A LoRA head's step as it is used: hidden states -> logits -> log-probabilities -> preference loss, and back to
    the adapter, against the same step in 64 bits on the layer's own rounded logits."""
    from tests.helpers import lora_inputs

    lens, d, V, r, s = [40, 9, 25, 33], 128, 520, 8, 2.0
    cu, n = _packed(lens)
    X, W, A, B, _ = lora_inputs(77, n, d, V, r, "f32")
    gen = torch.Generator().manual_seed(3)
    t = torch.randint(0, V, (n,), generator=gen).cuda()
    t[::7] = -100
    C = torch.from_numpy(cu).cuda()
    M = t >= 0
    ref = (-6 + torch.randn(n, generator=gen)).cuda()
    leaves = [v.clone().requires_grad_() for v in (X, A, B)]
    logp = lib.LoraHeadLogpFunction.apply(leaves[0], W, leaves[1], leaves[2], s, t)
    loss, _, _ = lib.LoraPreferenceLossFunction.apply(logp, ref, C, M, 0.1)
    loss.backward()
    l64 = [v.detach().cpu().double().requires_grad_() for v in leaves]
    z = l64[0] @ W.cpu().double().T + s * (l64[0] @ l64[1].T) @ l64[2].T
    lp = torch.log_softmax(z, 1).gather(1, t.cpu().clamp(min=0)[:, None]).squeeze(1)
    D = torch.stack([((lp - ref.cpu().double()) * M.cpu())[cu[i]:cu[i + 1]].sum() for i in range(4)])
    want = -torch.nn.functional.logsigmoid(0.1 * (D[:2] - D[2:])).mean()
    want.backward()
    # fp32 throughout: 1e-5 of the largest value, the layer's own bar
    assert abs(float(loss) - float(want)) <= 1e-5 * abs(float(want))
    for a, b in zip(leaves, l64):
        assert (a.grad.cpu().double() - b.grad).abs().max() <= 1e-5 * b.grad.abs().max()


def test_loss_refusals():
    import lora_linear_layers_amd as L

    lp, cu = torch.zeros(4), torch.tensor([0, 2, 4])
    with pytest.raises(ValueError, match="GPU"):
        L.lora_preference_loss_fwd(lp, cu, 0.1)
    with pytest.raises(ValueError, match="GPU"):
        L.lora_policy_loss_fwd(lp, cu, torch.zeros(2))
    lib, P = L.lib(), 0x100000
    f = lib.lora_loss_workspace_bytes
    assert f(0, 4, 1000) == (4 + 4) * 16 and f(1, 4, 1000) == (4 + 4) * 32
    assert f(2, 4, 10) == 0 and f(0, 0, 10) == 0 and f(0, 4, -1) == 0 and f(0, 2 ** 30 + 1, 1) == 0

    def pref(kind=0, pairs=2, n=100, beta=0.1, eps=0.0, cu=P, lp=P, ref=P, mask=P + 1, loss=P, coef=P, ws=P, wsb=1 << 20):
        return lib.lora_preference_loss_fwd(kind, pairs, n, beta, eps, 0, cu, mask, lp, ref, loss, P, P, coef, ws, wsb,
                                            None)

    assert pref(kind=3) == -2 and pref(kind=-1) == -2 and pref(pairs=0) == -2 and pref(n=-1) == -2
    assert pref(n=2 ** 40) == -2 and pref(pairs=2 ** 29 + 1) == -2
    for bad in (0.0, -1.0, NAN, float("inf")):
        assert pref(beta=bad) == -2
    assert pref(eps=1.0) == -2 and pref(eps=-0.1) == -2 and pref(eps=NAN) == -2 and pref(kind=1, eps=0.1) == -2
    assert pref(cu=None) == -1 and pref(lp=None) == -1 and pref(loss=None) == -1 and pref(coef=None) == -1
    assert pref(cu=P + 4) == -3 and pref(lp=P + 2) == -3 and pref(ref=P + 1) == -3 and pref(ws=P + 8) == -3
    assert pref(ws=None) == -5 and pref(wsb=10) == -5
    g = lib.lora_preference_loss_bwd
    assert g(0, 10, P, P, P, P, P, None) == -2 and g(2, 10, P, P, None, P, P, None) == -1
    assert g(2, 10, P, P, P, P, None, None) == -1 and g(2, 10, P, P, P, P + 2, P, None) == -3

    def pol(red=0, S=3, n=100, lo=0.2, hi=0.2, beta=0.1, norm=1.0, cu=P, lp=P, old=P, ref=P, adv=P, w=P, ws=P,
            wsb=1 << 20):
        return lib.lora_policy_loss_fwd(red, S, n, lo, hi, beta, norm, cu, None, lp, old, ref, adv, 0, P, P, w, ws, wsb,
                                        None)

    assert pol(red=3) == -2 and pol(S=0) == -2 and pol(lo=-0.1) == -2 and pol(lo=1.1) == -2 and pol(hi=-0.1) == -2
    assert pol(hi=float("inf")) == -2 and pol(lo=NAN) == -2 and pol(beta=-1.0) == -2 and pol(beta=NAN) == -2
    assert pol(red=2, norm=0.0) == -2 and pol(red=2, norm=NAN) == -2
    assert pol(ref=None) == -1 and pol(adv=None) == -1 and pol(lp=None) == -1 and pol(w=None) == -1
    assert pol(old=P + 2) == -3 and pol(adv=P + 1) == -3 and pol(wsb=0) == -5
    h = lib.lora_policy_loss_bwd
    assert h(3, 100, 0.2, 0.2, 0.1, P, None, P, P, P, P, 0, None, P, P, None) == -1
    assert h(3, 100, 0.2, 0.2, 0.1, P, None, P, P, P, P, 0, P, P, None, None) == -1
    assert h(3, 100, 2.0, 0.2, 0.1, P, None, P, P, P, P, 0, P, P, P, None) == -2
    if torch.cuda.device_count() == 0:
        assert pref() == -6 and pol() == -6 and pol(ref=None, beta=0.0, old=None) == -6


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 40), (5, 8), (2, 4, 5), (40,)], ids=str)
def test_loss_gradients_have_the_shape_of_logp(lib, shape):
    lens = [12, 9, 9, 10]
    cu, n = _packed(lens)
    lp, ref, old, mask, _ = _draw(51, n)
    L, R, O, C, M = _dev(lp, ref, old, cu, mask)
    adv = torch.tensor([0.7, 1.0, -1.2, 0.4], device="cuda")
    calls = (lambda x: lib.LoraPreferenceLossFunction.apply(x, R, C, M, 0.1)[0],
             lambda x: lib.LoraPolicyLossFunction.apply(x, O, R, C, adv, M, 0.2, 0.28, 0.05)[0])
    for call in calls:
        flat, x = L.clone().requires_grad_(), L.clone().view(shape).requires_grad_()
        call(flat).backward()
        call(x).backward()
        assert x.grad.shape == torch.Size(shape) and torch.equal(x.grad.view(-1), flat.grad)


@pytest.mark.gpu
def test_preference_backward_refuses_an_odd_number_of_sequences(lib):
    with pytest.raises(ValueError, match="2 P"):
        lib.lora_preference_loss_bwd(torch.zeros(3, device="cuda"), torch.tensor([0, 1, 2, 3], device="cuda"), 3)


# ---------------------------------------------------------------------------
# guarded outputs, many tokens, and shapes
# ---------------------------------------------------------------------------
class _Guards:
    """Arrays in the middle of larger ones, to see what is written beside them."""

    def __init__(self):
        self.all = []

    def new(self, n):
        b = torch.full((n + 128,), 7.25, device="cuda")
        self.all.append((b, n))
        return b[64:64 + n]

    def intact(self):
        return all(bool((b[:64] == 7.25).all()) and bool((b[64 + n:] == 7.25).all()) for b, n in self.all)


def _offsets(kind, n, S, seed):
    r = np.random.default_rng(seed)
    if kind == "outside":  # in order, but reaching past both ends of the tokens
        cu = np.sort(r.integers(0, n, S + 1))
        cu[0], cu[-1] = -50, n + 999
        return cu
    if kind == "random":
        return r.integers(-50, n + 51, S + 1)
    return np.sort(r.integers(0, n + 1, S + 1))[::-1].copy()  # decreasing


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["outside", "random", "decreasing"])
@pytest.mark.parametrize("n,S", [(3000, 4), (3000, 130), (8192, 1024), (8193, 4), (70001, 130), (70001, 2050)])
def test_losses_write_nothing_beside_their_outputs(lib, kind, n, S):
    # every output and the workspace between guards, the token arrays NaN behind n: offsets outside the tokens are
    # taken as their ends, disordered ones give some value, and nothing beside the outputs is written
    G = _Guards()
    C = lib.load()
    P = S // 2
    lp = torch.full((n + 256,), NAN, device="cuda")
    ref, old = lp.clone(), lp.clone()
    h = _draw(n + S, n)
    lp[:n], ref[:n], old[:n] = (torch.from_numpy(h[i]).cuda() for i in (0, 1, 2))
    cu_h = _offsets(kind, n, S, n + S)
    cu = torch.from_numpy(cu_h.astype(np.int64)).cuda()
    adv = torch.from_numpy(np.random.default_rng(1).normal(size=S).astype(np.float32)).cuda()
    p = lambda t: t.data_ptr()  # noqa: E731
    wb = [C.lora_loss_workspace_bytes(k, S, n) for k in (0, 1)]
    ws = [G.new(b // 4) for b in wb]
    loss, pair, rew, coef, d = G.new(1), G.new(P), G.new(S), G.new(S), G.new(n)
    assert C.lora_preference_loss_fwd(0, P, n, 0.1, 0.0, 0, p(cu), None, p(lp), p(ref), p(loss), p(pair), p(rew),
                                      p(coef), p(ws[0]), wb[0], None) == 0
    assert C.lora_preference_loss_bwd(P, n, p(cu), None, p(coef), None, p(d), None) == 0
    ploss, stats, weight, pd = G.new(1), G.new(4), G.new(S), G.new(n)
    args = (0.2, 0.28, 0.05)
    assert C.lora_policy_loss_fwd(0, S, n, *args, 1.0, p(cu), None, p(lp), p(old), p(ref), p(adv), 0, p(ploss), p(stats),
                                  p(weight), p(ws[1]), wb[1], None) == 0
    assert C.lora_policy_loss_bwd(S, n, *args, p(cu), None, p(lp), p(old), p(ref), p(adv), 0, p(weight), None, p(pd),
                                  None) == 0
    torch.cuda.synchronize()
    assert G.intact()
    assert not (d == 7.25).any() and not (pd == 7.25).any()  # every token's gradient is written
    if kind == "outside":
        c = np.clip(cu_h, 0, n)
        wl, wp, wr, wd, mag = _pref_plain(h[0], h[1], c, None, 0.1, "sigmoid", 0.0, False)
        a = 1e-9 * max(mag, 1.0)
        _near(loss, [wl], 2 * U, a)
        _near(pair, wp, 2 * U, a)
        _near(rew, wr, 2 * U, a)
        _near(d, wd, 4 * U, a / S)
        wl, wst, wd, tol, mag = _policy_plain(h[0], h[2], h[1], adv.cpu().numpy(), c, None, 0.2, 0.28, 0.05, "sequence",
                                              1.0, False)
        _near(ploss, [wl], 2 * U, mag)
        _near(stats[2:], wst[2:], 2 * U, 0)
        assert (np.abs(pd.cpu().double().numpy() - wd) <= tol).all()


def _walk_chunk(cu, S, N, t0, t1):
    """The stretches (sequence or -1, its first token, from, to) in which a wave walks the tokens [t0, t1): the
    kernels' steps on plain integers, every index checked."""
    clip = lambda t: min(max(t, 0), N)  # noqa: E731
    lo, hi = 0, S
    while S > 64 and hi > lo:  # the first sequence that ends after t0, by a 64-way search
        step = (hi - lo + 63) // 64
        at = [lo + lane * step + step - 1 for lane in range(64)]
        lo += sum(cu[i + 1] <= t0 for i in at if i < hi) * step
        if step == 1:
            break
        hi = min(lo + step, hi)
    base, pos, out = (min(lo, S) if S > 64 else 0), t0, []
    while base < S and pos < t1:
        end = [clip(cu[base + lane + 1]) if base + lane < S else 0 for lane in range(64)]
        first = clip(cu[base])
        while pos < t1:
            todo = [lane for lane in range(64) if end[lane] > pos]
            if not todo:
                break
            lane = todo[0]
            assert base + lane < S
            b = end[lane - 1] if lane else first
            to = min(b if b > pos else end[lane], t1)
            assert to > pos  # every step moves on
            out.append((-1 if b > pos else base + lane, b, pos, to))
            pos = to
        base += 64
    if pos < t1:
        out.append((-1, 0, pos, t1))
    return out


def test_losses_walk_covers_every_token_once():
    # the walk of loss.hip (Walk, first_seq, sum_chunk, sum_sequences) for ordered and disordered offsets: stretches
    # join up over the chunk, and for ordered ones each sequence's parts are where its sum looks for them
    import random

    rng = random.Random(3)
    for k in range(400):
        S, N, ch = rng.choice([1, 2, 63, 64, 65, 130, 300]), rng.choice([1, 5, 64, 257, 1000]), rng.choice([64, 256])
        if k % 3 == 0:
            cu = [rng.randint(-50, N + 50) for _ in range(S + 1)]
        elif k % 3 == 1:
            cu = sorted(rng.randint(0, N) for _ in range(S + 1))
        else:
            cu = sorted(rng.choice([0, N // 3, N // 2, N]) for _ in range(S + 1))
        head, seqp = {}, {}
        for c in range(-(-N // ch)):
            at = c * ch
            for s, b, lo, hi in _walk_chunk(cu, S, N, at, min(at + ch, N)):
                assert lo == at
                at = hi
                if s >= 0:
                    where, key = (head, c) if b < c * ch else (seqp, s)
                    where[key] = where.get(key, 0) + hi - lo
            assert at == min(c * ch + ch, N)
        if k % 3:
            for s in range(S):
                n = cu[s + 1] - cu[s]
                if n:
                    c0, c1 = cu[s] // ch, (cu[s + 1] - 1) // ch
                    assert seqp[s] + sum(head[c] for c in range(c0 + 1, c1 + 1)) == n


def _many_lens(total, seed):
    """Lengths that sum to total: on and beside steps of 256 and chunks of 512 to 4096, empty ones, one of 40 %."""
    r = np.random.default_rng(seed)
    lens = [256, 0, 512, 1024, 4096, 255, 257, 1, 511, 513, 2048, 4095, 4097, 0]
    lens += [int(total * 0.4)]
    left = total - sum(lens)
    while left > 0:
        n = min(left, int(r.choice([r.integers(1, 700), 256, 768, r.integers(3000, 9000)])))
        lens.append(n)
        left -= n
    if len(lens) % 2:
        lens.append(0)
    return lens


@pytest.mark.gpu
@pytest.mark.parametrize("total", [2_200_003, 5_000_001, 20_000_003])
def test_losses_of_many_tokens(lib, total):
    # chunks of several steps (512 tokens above 2.1 M, up to 4096), both losses forward and backward
    lens = _many_lens(total, total)
    S, P = len(lens), len(lens) // 2
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), device="cuda")
    n = int(cu[-1])
    gen = torch.Generator("cuda").manual_seed(5)
    rand = lambda *s: torch.rand(*s, generator=gen, device="cuda")  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    ref = 2.5 * torch.log1p(-rand(n) * 0.999)
    lp = ref + 0.3 * randn(n)
    old = lp + 0.15 * randn(n)
    mask = rand(n) > 0.25
    adv = randn(S)
    g = torch.tensor(0.5, device="cuda")
    seq = torch.repeat_interleave(torch.arange(S, device="cuda"), torch.tensor(lens, device="cuda"))
    m = mask.double()
    # (summed on the CPU: one sequence has millions of the entries, which an atomic sum would add one by one)
    add = lambda v: torch.stack([c.sum() for c in v.cpu().split(lens)]).cuda()  # noqa: E731
    T = add(m)
    # preference, averaged
    loss, pair, rew, coef = lib.lora_preference_loss_fwd(lp, cu, 0.1, ref, mask, average=True)
    d = lib.lora_preference_loss_bwd(coef, cu, n, mask, g)
    x = lp.double() - ref.double()
    D = add(x * m) / T.clamp(min=1)
    u = D[:P] - D[P:]
    want = torch.nn.functional.softplus(-0.1 * u)
    cw = -0.1 * torch.sigmoid(-0.1 * u) / P
    cw = torch.cat([cw, -cw]) / T.clamp(min=1)
    near = lambda a, b, r, t: bool(((a.double() - b).abs() <= r * b.abs() + t).all())  # noqa: E731
    assert near(pair, want, 2 * U, 1e-9) and near(loss, want.mean(), 2 * U, 1e-9) and near(rew, 0.1 * D, 2 * U, 1e-9)
    assert near(d, cw[seq] * m * 0.5, 4 * U, 1e-13)
    # policy, every token alike
    kw = dict(old_logp=old, ref_logp=ref, mask=mask, eps_low=0.2, eps_high=0.28, beta=0.05)
    loss, stats, w = lib.lora_policy_loss_fwd(lp, cu, adv, reduction="token", **kw)
    d = lib.lora_policy_loss_bwd(lp, cu, adv, w, dloss=g, **kw)
    A, y, dd = adv.double()[seq], lp.double() - old.double(), -x
    over, under = (A > 0) & (y > math.log1p(0.28)), (A < 0) & (y < math.log1p(-0.2))
    r, e = y.exp(), torch.expm1(dd)
    pol = torch.where(over, 1.28, torch.where(under, 0.8, r)) * -A
    W = 1 / float(T.sum())
    # (the bounds of the head of this file, token by token)
    mag = W * (m * (pol.abs() * (2 + y.abs()) * 2 * U + (e - dd) * 10 * U + dd * dd * 2e-9)).sum()
    sums = torch.stack([(pol * m).sum() * W, ((e - dd) * m).sum() * W, ((over | under) & mask).sum() * W, T.sum()])
    assert near(stats, sums, 2 * U, torch.stack([mag, mag, 0 * mag, 0 * mag]))
    assert near(loss, sums[0] + 0.05 * sums[1], 2 * U, mag)
    gr = W * 0.5 * (torch.where(over | under, 0.0, -r * A) - 0.05 * e) * m
    tol = W * 0.5 * ((r * A).abs() * (2 + y.abs()) * 2 * U + 0.05 * ((e + 1) * (2 + dd.abs()) * 2 * U + U)) + 4 * U * gr.abs()
    assert bool(((d.double() - gr).abs() <= tol + 1e-37).all())


@pytest.mark.gpu
def test_policy_kl_around_its_series(lib):
    # e^d - 1 - d: a series below |d| = 0.5 (cut after d^9: the rest is below 2.5e-9 of the sum, at d = -0.5; 8
    # roundings of its Horner steps and products), the difference above it.  There e^d is off by (2 + 1.25 |d|) u and
    # its products, e^d - 1 by u of itself and the last difference by u of itself
    d0 = np.array([-0.499, -0.5, -0.501, 0.499, 0.5, 0.501, 0.6, -0.6, 0.75, 1.0, -1.0, 2.0, -2.0, 6.0, -17.0], np.float32)
    for x32 in d0:
        L, R, A, C = _dev(np.zeros(1, np.float32), np.array([x32]), np.zeros(1, np.float32), np.array([0, 1], np.int64))
        kl = float(lib.lora_policy_loss_fwd(L, C, A, ref_logp=R, beta=1.0)[0])
        x = float(x32)
        want = math.expm1(x) - x
        if abs(x) < 0.5:
            tol = 2.5e-9 * want + 10 * U * want
        else:
            tol = math.exp(x) * (2 + 1.25 * abs(x)) * U + abs(math.expm1(x)) * U + 2 * U * want
        assert abs(kl - want) <= tol, (x, kl, want, abs(kl - want) / tol)
