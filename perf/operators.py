"""Cases and plain forms of the operators around a LoRA training step's head and blocks: the fused
LoRA linear layer with bias, activation and residual in its epilogue, the log-probabilities of tokens
from logits, the preference loss of response pairs and the clipped policy loss with a KL term, each
with its gradient.

`run` computes a case in its plain form (elementary torch operations in 32 bits, in 64 where sums and
borders need it), or, where `own` is true, through the package's entry points.  `exact` gives the same
outputs from the definitions in 64 bits."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
# relu's gradient jumps at 0, where the last bit of the pre-activation decides it: steps take the smooth ones
STEP_ACTS = ("none", "silu", "gelu", "gelu_tanh")
STATS = ("policy", "kl", "clipped", "tokens")  # the policy loss's parts, the share of clipped tokens, their number
IGNORED = -100  # a target outside the vocabulary: the row has no token


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _linear(name, M, d_in, d_out, r, dtype, act, bias, residual, train, store_z=False):
    return {"name": name, "op": "linear", "M": M, "d_in": d_in, "d_out": d_out, "r": r, "dtype": dtype, "act": act,
            "bias": bias, "residual": residual, "train": train, "store_z": store_z}


def _logp(name, rows, vocab, dtype, inv_temp, grad):
    return {"name": name, "op": "logp", "rows": rows, "vocab": vocab, "dtype": dtype, "inv_temp": inv_temp,
            "grad": grad}


def _pref(name, pairs, length, kind, average, smoothing, reference):
    return {"name": name, "op": "preference", "pairs": pairs, "length": length, "kind": kind, "average": average,
            "smoothing": smoothing, "reference": reference}


def _policy(name, seqs, length, reduction, per_token, beta):
    return {"name": name, "op": "policy", "seqs": seqs, "length": length, "reduction": reduction,
            "per_token": per_token, "beta": beta}


def listed():
    return [
        # one token of a served MLP projection (Llama-3-8B gate shape): latency, the weight's bytes
        _linear("linear 1 token", 1, 4096, 14336, 16, "bf16", "silu", True, False, False),
        # a packed prompt batch that fills no tile, with the pre-activation kept for a backward
        _linear("linear ragged prompt", 2049, 4096, 4104, 24, "bf16", "gelu_tanh", True, False, False, True),
        # the down projection of the Llama-3-8B MLP at 4 x 2048 tokens, added to the residual stream
        _linear("linear down + residual", 8192, 14336, 4096, 64, "bf16", "none", False, True, False),
        # a training step of a biased projection that ends a block: forward and every gradient
        _linear("linear step bf16", 2048, 4096, 4096, 16, "bf16", "none", True, True, True),
        # the single fp32 layer of 128 tokens, forward and every gradient
        _linear("linear step fp32", 128, 256, 256, 8, "f32", "silu", True, True, True),
        # scoring the answers of a few prompts (reference log-probabilities, no gradient)
        _logp("logp score", 24, 32000, "bf16", 1.0, False),
        # a training step over 4 x 2048 positions of a large vocabulary: forward and the logits' gradient
        _logp("logp step", 8192, 128000, "bf16", 1.0, True),
        # fp32 logits of an odd vocabulary, sampled at a temperature
        _logp("logp step fp32 odd", 2047, 50001, "f32", 1.25, True),
        # one micro-batch of two pairs
        _pref("preference small", 2, 300, "sigmoid", False, 0.0, True),
        # a global batch of pairs packed without padding
        _pref("preference large", 256, 2048, "sigmoid", False, 0.1, True),
        # one prompt with a group of eight sampled answers
        _policy("policy small", 8, 250, "sequence", False, 0.04),
        # a rollout batch, advantages per token, averaged over all tokens
        _policy("policy large", 1024, 2048, "token", True, 0.04),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "logp", "preference", "policy"))
    if op == "linear":
        dtype = rng.choice(("bf16", "bf16", "f32"))
        train = rng.random() < 0.4
        most = 4.8e11 if dtype == "bf16" else 6e10
        if train:
            most /= 4
        while True:
            M = _log_int(rng, 1, 8192)
            d_in, d_out = 8 * _log_int(rng, 8, 1792), 8 * _log_int(rng, 8, 1792)
            if rng.random() < 0.5:
                d_in, d_out = max(64, d_in // 64 * 64), max(64, d_out // 64 * 64)
            if rng.random() < 0.3:
                M = max(1, M // 256) * 256
            if M * d_in * d_out <= most:
                break
        return {k: v for k, v in _linear("", M, d_in, d_out, rng.choice((1, 4, 8, 12, 16, 32, 64, 128)), dtype,
                                         rng.choice(STEP_ACTS if train else ACTS), rng.random() < 0.6, rng.random() < 0.6, train,
                                         not train and rng.random() < 0.4).items() if k != "name"}
    if op == "logp":
        while True:
            rows, vocab = _log_int(rng, 1, 8192), _log_int(rng, 100, 160000)
            if rows * vocab <= 2.5e8:
                break
        return {k: v for k, v in _logp("", rows, vocab, rng.choice(("bf16", "bf16", "f32")),
                                       rng.choice((1.0, 1.0, 0.7, 1.25)), rng.random() < 0.6).items() if k != "name"}
    if op == "preference":
        length = _log_int(rng, 2, 4096)
        pairs = _log_int(rng, 1, max(2, min(512, 500000 // length)))
        kind = rng.choice(("sigmoid", "sigmoid", "hinge", "ipo"))
        smoothing = rng.choice((0.0, 0.0, 0.1)) if kind == "sigmoid" else 0.0
        return {k: v for k, v in _pref("", pairs, length, kind, rng.random() < 0.4, smoothing,
                                       rng.random() < 0.8).items() if k != "name"}
    length = _log_int(rng, 2, 4096)
    seqs = _log_int(rng, 1, max(2, min(1024, 2000000 // length)))
    return {k: v for k, v in _policy("", seqs, length, rng.choice(("sequence", "token", "constant")),
                                     rng.random() < 0.3, rng.choice((0.0, 0.04, 0.1))).items() if k != "name"}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _tokens(count, length):
    """Tokens of `count` packed sequences, the same for every seed."""
    return max(count, int(0.625 * count * length))


def _ragged(count, length, gen):
    """Packed sequences: offsets int64 [count + 1] over _tokens(count, length) tokens, the lengths spread over a
    factor of four, one in eight of them empty when there are eight or more (a response that was cut away)."""
    n = _tokens(count, length)
    share = torch.rand(count, generator=gen, device="cuda", dtype=torch.float64) * 0.75 + 0.25
    if count >= 8:
        share[count // 2 :: 8] = 0
    cu = torch.zeros(count + 1, dtype=torch.int64, device="cuda")
    cu[1:] = (share.cumsum(0) / share.sum() * n).round().long()
    cu[-1] = n
    return cu, n


def prepare(case, seed):
    gen = _generator(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=gen, device="cuda")  # noqa: E731
    state = {"case": dict(case)}
    if case["op"] == "linear":
        M, k, d, r, t = case["M"], case["d_in"], case["d_out"], case["r"], DTYPES[case["dtype"]]
        state["X"] = normal(M, k).to(t)
        state["W"] = (normal(d, k) / math.sqrt(k)).to(t)
        state["A"] = ((rand(r, k) * 2 - 1) / math.sqrt(k)).to(t)
        state["B"] = (normal(d, r) * math.sqrt(0.02)).to(t)
        state["bias"] = (normal(d) * 0.5).to(t) if case["bias"] else None
        state["residual"] = normal(M, d).to(t) if case["residual"] else None
        state["dY"] = normal(M, d).to(t) if case["train"] else None
        state["scale"] = 16.0 / r
    elif case["op"] == "logp":
        n, v, t = case["rows"], case["vocab"], DTYPES[case["dtype"]]
        logits = torch.empty(n, v, dtype=t, device="cuda")
        for i in range(0, n, 1024):  # in pieces: the whole in fp32 would be twice the state
            logits[i : i + 1024] = (normal(min(1024, n - i), v) * 2.5).to(t)
        targets = torch.randint(0, v, (n,), generator=gen, device="cuda")
        # a model that learned something: the target's logit stands out by 0 to 16
        at = torch.arange(n, device="cuda")
        logits[at, targets] += (rand(n) * 16).to(t)
        state["targets"] = torch.where(rand(n) < 0.05, torch.full_like(targets, IGNORED), targets)
        state["logits"] = logits
        state["dlogp"] = normal(n) / n if case["grad"] else None
    else:
        count = 2 * case["pairs"] if case["op"] == "preference" else case["seqs"]
        cu, n = _ragged(count, case["length"], gen)
        state["cu"], state["n"] = cu, n
        state["ref"] = 2.5 * torch.log1p(-rand(n) * 0.999)
        state["logp"] = state["ref"] + 0.3 * normal(n)
        # the prompt's share of each sequence carries no loss
        state["mask"] = rand(n) > 0.25
        if case["op"] == "policy":
            state["old"] = state["logp"] + 0.15 * normal(n)
            state["adv"] = normal(n if case["per_token"] else count)
        state["dloss"] = torch.full((), 0.5, device="cuda")
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    return {"linear": _plain_linear, "logp": _plain_logp, "preference": _plain_preference,
            "policy": _plain_policy}[c["op"]](c, state)


def _run_own(c, s):
    import lora_linear_layers_amd as L

    if c["op"] == "linear":
        if c["train"]:
            leaves = [t.detach().requires_grad_() for t in (s["X"], s["A"], s["B"], s["bias"], s["residual"])
                      if t is not None]
            it = iter(leaves)
            X, A, B = next(it), next(it), next(it)
            bias = next(it) if c["bias"] else None
            res = next(it) if c["residual"] else None
            Y = L.LoraLinearEpiFunction.apply(X, s["W"], A, B, bias, res, s["scale"], c["act"])
            grads = iter(torch.autograd.grad(Y, leaves, s["dY"]))
            out = {"Y": Y.detach(), "dX": next(grads), "dA": next(grads), "dB": next(grads)}
            out["dbias"] = next(grads) if c["bias"] else None
            out["dresidual"] = next(grads) if c["residual"] else None
            return out
        member = {"W": s["W"], "A": s["A"], "B": s["B"], "scale": s["scale"]}
        Y, Z = L.lora_linear_epi_fwd(s["X"], member, act=c["act"], bias=s["bias"], residual=s["residual"],
                                     store_z=c["store_z"])
        return {"Y": Y, "Z": Z}
    if c["op"] == "logp":
        logp, stats = L.lora_token_logp_fwd(s["logits"], s["targets"], c["inv_temp"])
        out = {"logp": logp, "stats": stats}
        if c["grad"]:
            out["dlogits"] = L.lora_token_logp_bwd(s["logits"], s["targets"], stats, s["dlogp"], c["inv_temp"])
        return out
    if c["op"] == "preference":
        ref = s["ref"] if c["reference"] else None
        loss, pair_loss, rewards, coef = L.lora_preference_loss_fwd(
            s["logp"], s["cu"], 0.1, ref_logp=ref, mask=s["mask"], kind=c["kind"], label_smoothing=c["smoothing"],
            average=c["average"])
        dlogp = L.lora_preference_loss_bwd(coef, s["cu"], s["n"], mask=s["mask"], dloss=s["dloss"])
        return {"loss": loss, "pair_loss": pair_loss, "rewards": rewards, "dlogp": dlogp}
    args = dict(old_logp=s["old"], ref_logp=s["ref"], mask=s["mask"], eps_low=0.2, eps_high=0.28, beta=c["beta"],
                per_token=c["per_token"])
    loss, stats, weight = L.lora_policy_loss_fwd(s["logp"], s["cu"], s["adv"], reduction=c["reduction"],
                                                 norm=float(c["length"]), **args)
    dlogp = L.lora_policy_loss_bwd(s["logp"], s["cu"], s["adv"], weight, dloss=s["dloss"], **args)
    return {"loss": loss, **dict(zip(STATS, stats)), "dlogp": dlogp}


# -- plain forms ------------------------------------------------------------
def _act(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return z * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_linear(c, s, wide=torch.float32):
    t = DTYPES[c["dtype"]]
    X, W, A, B = (s[k].to(wide) for k in ("X", "W", "A", "B"))
    P = X @ A.T * s["scale"]
    Z = X @ W.T + P @ B.T
    if s["bias"] is not None:
        Z = Z + s["bias"].to(wide)
    Y = _act(Z, c["act"])
    if s["residual"] is not None:
        Y = Y + s["residual"].to(wide)
    if not c["train"]:
        return {"Y": Y.to(t), "Z": Z.to(t) if c["store_z"] else None}
    dY = s["dY"].to(wide)
    dZ = dY * _act_grad(Z, c["act"])
    Q = dZ @ B * s["scale"]
    return {"Y": Y.to(t), "dX": (dZ @ W + Q @ A).to(t), "dA": (Q.T @ X).to(t), "dB": (dZ.T @ P).to(t),
            "dbias": dZ.sum(0).to(t) if c["bias"] else None, "dresidual": dY.to(t) if c["residual"] else None}


def _plain_logp(c, s):
    z, targets = s["logits"].float(), s["targets"]
    has = (targets >= 0) & (targets < c["vocab"])
    t = torch.where(has, targets, 0).unsqueeze(1)
    top = z.amax(1, keepdim=True)
    e = torch.exp((z - top) * c["inv_temp"])
    logsum = torch.log(e.sum(1, keepdim=True))
    logp = ((z.gather(1, t) - top) * c["inv_temp"] - logsum).squeeze(1)
    out = {"logp": torch.where(has, logp, 0.0), "stats": torch.cat((top, logsum), 1)}
    if c["grad"]:
        g = torch.where(has, s["dlogp"], 0.0).unsqueeze(1) * c["inv_temp"]
        d = e.mul_(torch.exp(-logsum) * -g)
        out["dlogits"] = d.scatter_add_(1, t, g).to(DTYPES[c["dtype"]])
    return out


def _segments(cu, n, count):
    """Each token's sequence (tokens lie in order, every one of them in a sequence)."""
    return torch.searchsorted(cu[1:], torch.arange(n, device=cu.device), right=True)


def _plain_preference(c, s):
    # sums of log-ratios over long responses, and their differences: 64 bits
    pairs, beta, n = c["pairs"], 0.1, s["n"]
    seq = _segments(s["cu"], n, 2 * pairs)
    d = s["logp"].double() - s["ref"].double() if c["reference"] else s["logp"].double()
    m = s["mask"]
    total = torch.zeros(2 * pairs, dtype=torch.float64, device="cuda").index_add_(0, seq, torch.where(m, d, 0.0))
    length = torch.zeros(2 * pairs, dtype=torch.float64, device="cuda").index_add_(0, seq, m.double())
    per = 1 / length.clamp(min=1) if c["average"] else torch.ones_like(length)
    ratio = total * per
    u = ratio[:pairs] - ratio[pairs:]
    eps = c["smoothing"]
    if c["kind"] == "sigmoid":
        soft = lambda x: x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))  # noqa: E731
        pair = (1 - eps) * soft(-beta * u) + eps * soft(beta * u)
        du = beta * (eps / (1 + torch.exp(-beta * u)) - (1 - eps) / (1 + torch.exp(beta * u)))
    elif c["kind"] == "hinge":
        pair = (1 - beta * u).clamp(min=0)
        du = -beta * (beta * u < 1).double()
    else:
        pair = (u - 1 / (2 * beta)) ** 2
        du = 2 * (u - 1 / (2 * beta))
    coef = torch.cat((du, -du)) * per / pairs * s["dloss"].double()
    return {"loss": pair.mean().float(), "pair_loss": pair.float(), "rewards": (beta * ratio).float(),
            "dlogp": torch.where(m, coef[seq], 0.0).float()}


def _plain_policy(c, s):
    # the clip borders are compared in 64 bits, where the difference of two fp32 values is exact
    count, n, m = c["seqs"], s["n"], s["mask"]
    seq = _segments(s["cu"], n, count)
    delta = s["logp"].double() - s["old"].double()
    adv = s["adv"].double() if c["per_token"] else s["adv"].double()[seq]
    over = (adv > 0) & (delta > math.log1p(0.28))
    under = (adv < 0) & (delta < math.log1p(-0.2))
    ratio = torch.exp(delta)
    used = torch.where(over, 1.28, torch.where(under, 0.8, ratio))
    pol = torch.where(adv == 0, 0.0, -used * adv)
    d = s["ref"].double() - s["logp"].double()
    kl = torch.expm1(d) - d
    tokens = torch.zeros(count, dtype=torch.float64, device="cuda").index_add_(0, seq, m.double())
    if c["reduction"] == "sequence":
        w = 1 / (count * tokens.clamp(min=1))
    elif c["reduction"] == "token":
        w = (1 / tokens.sum().clamp(min=1)).expand(count)
    else:
        w = torch.full((count,), 1 / (count * float(c["length"])), dtype=torch.float64, device="cuda")
    wt = torch.where(m, w[seq], 0.0)
    pol_sum, kl_sum = (wt * pol).sum(), (wt * kl).sum()
    clipped = ((over | under) & m).double().sum() / tokens.sum().clamp(min=1)
    grad = torch.where(over | under | (adv == 0), 0.0, -ratio * adv) - c["beta"] * torch.expm1(d)
    return {"loss": (pol_sum + c["beta"] * kl_sum).float(),
            **dict(zip(STATS, torch.stack((pol_sum, kl_sum, clipped, tokens.sum())).float())),
            "dlogp": (wt * grad * s["dloss"].double()).float()}


# ---------------------------------------------------------------------------
# from the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "linear":
        # [X | X A^T s] [W | B]^T in one product; gradients from the chain rule through autograd in 64 bits
        f = lambda k: None if s[k] is None else s[k].double().requires_grad_(c["train"])  # noqa: E731
        X, A, B, bias, res = (f(k) for k in ("X", "A", "B", "bias", "residual"))
        low = torch.matmul(X, A.transpose(0, 1)).mul(s["scale"])
        Z = torch.cat((X, low), 1).matmul(torch.cat((s["W"].double(), B), 1).transpose(0, 1))
        Z = Z if bias is None else Z + bias
        h = {"none": lambda z: z, "relu": lambda z: z.clamp(min=0), "silu": lambda z: z * torch.sigmoid(z),
             "gelu": lambda z: z * torch.special.ndtr(z),
             "gelu_tanh": lambda z: z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))}
        Y = h[c["act"]](Z)
        Y = Y if res is None else Y + res
        if not c["train"]:
            return {"Y": Y, "Z": Z if c["store_z"] else None}
        names = [k for k in (("X", X), ("A", A), ("B", B), ("bias", bias), ("residual", res)) if k[1] is not None]
        grads = torch.autograd.grad(Y, [t for _, t in names], s["dY"].double())
        out = {"Y": Y.detach(), "dbias": None, "dresidual": None}
        out.update({"d" + k: g for (k, _), g in zip(names, grads)})
        return out
    if c["op"] == "logp":
        n, v, tau = c["rows"], c["vocab"], c["inv_temp"]
        logp = torch.zeros(n, dtype=torch.float64, device="cuda")
        stats = torch.empty(n, 2, dtype=torch.float64, device="cuda")
        dlogits = torch.zeros(n, v, dtype=torch.float64, device="cuda") if c["grad"] else None
        for i in range(0, n, 512):
            z = s["logits"][i : i + 512].double()
            t = s["targets"][i : i + 512]
            rows = torch.nonzero((t >= 0) & (t < v)).squeeze(1)
            full = torch.log_softmax(z * tau, 1)
            stats[i : i + 512, 0] = z.max(1).values
            stats[i : i + 512, 1] = torch.logsumexp(z * tau, 1) - z.max(1).values * tau
            logp[i + rows] = full[rows, t[rows]]
            if c["grad"]:
                g = s["dlogp"][i : i + 512].double()[rows] * tau
                part = -full[rows].exp() * g[:, None]
                part[torch.arange(len(rows), device="cuda"), t[rows]] += g
                dlogits[i + rows] = part
        return {"logp": logp, "stats": stats, **({"dlogits": dlogits} if c["grad"] else {})}
    # the two losses: padded [sequence, token] tables, gradients through autograd
    cu, m = s["cu"], s["mask"]
    lens = cu[1:] - cu[:-1]
    count, most = len(lens), max(1, int(lens.max()))
    col = torch.arange(most, device="cuda")
    inside = col[None] < lens[:, None]
    at = (cu[:-1, None] + col[None]).clamp(max=max(0, s["n"] - 1))
    pad = lambda x: torch.where(inside, x.double()[at], 0.0)  # noqa: E731
    keep = inside & m[at]
    x = s["logp"].double().requires_grad_()
    lp = torch.where(keep, x[at], 0.0)
    tokens = keep.sum(1).double()
    if c["op"] == "preference":
        beta, p = 0.1, c["pairs"]
        ref = torch.where(keep, pad(s["ref"]), 0.0) if c["reference"] else torch.zeros_like(lp)
        ratio = (lp - ref).sum(1)
        if c["average"]:
            ratio = ratio / tokens.clamp(min=1)
        u = ratio[:p] - ratio[p:]
        if c["kind"] == "sigmoid":
            e = c["smoothing"]
            pair = -(1 - e) * torch.nn.functional.logsigmoid(beta * u) - e * torch.nn.functional.logsigmoid(-beta * u)
        elif c["kind"] == "hinge":
            pair = torch.relu(1 - beta * u)
        else:
            pair = (u - 0.5 / beta).square()
        loss = pair.mean()
        (g,) = torch.autograd.grad(loss, x, s["dloss"].double())
        return {"loss": loss.detach(), "pair_loss": pair.detach(), "rewards": (beta * ratio).detach(), "dlogp": g}
    adv = pad(s["adv"]) if c["per_token"] else s["adv"].double()[:, None].expand(count, most)
    delta = lp - torch.where(keep, pad(s["old"]), 0.0)
    ratio = torch.exp(delta)
    clipped = torch.exp(delta.clamp(math.log1p(-0.2), math.log1p(0.28)))
    pol = torch.where(keep, -torch.minimum(ratio * adv, clipped * adv), 0.0)
    d = torch.where(keep, pad(s["ref"]), 0.0) - lp
    kl = torch.where(keep, torch.expm1(d) - d, 0.0)
    if c["reduction"] == "sequence":
        mean = lambda v: (v.sum(1) / tokens.clamp(min=1)).sum() / count  # noqa: E731
    elif c["reduction"] == "token":
        mean = lambda v: v.sum() / tokens.sum().clamp(min=1)  # noqa: E731
    else:
        mean = lambda v: v.sum() / (count * float(c["length"]))  # noqa: E731
    loss = mean(pol) + c["beta"] * mean(kl)
    (g,) = torch.autograd.grad(loss, x, s["dloss"].double())
    cut = keep & (((adv > 0) & (delta > math.log1p(0.28))) | ((adv < 0) & (delta < math.log1p(-0.2))))
    stats = torch.stack((mean(pol), mean(kl), cut.sum() / tokens.sum().clamp(min=1), tokens.sum()))
    return {"loss": loss.detach(), **dict(zip(STATS, stats.detach())), "dlogp": g}


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "linear":
        M, k, d, r, e = c["M"], c["d_in"], c["d_out"], c["r"], 2 if c["dtype"] == "bf16" else 4
        weights = k * d + r * (k + d) + (d if c["bias"] else 0)
        values = M * (k + d) + (M * d if c["residual"] else 0) + (M * d if c["store_z"] else 0)
        flops = 2.0 * M * (k * d + r * (k + d))
        if c["train"]:
            values += M * (d + k) + (M * d if c["residual"] else 0)
            weights += r * (k + d) + (d if c["bias"] else 0)
            flops += 2.0 * M * (k * d + 3 * r * (k + d))
        return {"bytes": float(e * (weights + values)), "flops": flops}
    if c["op"] == "logp":
        n, e = c["rows"] * c["vocab"], 2 if c["dtype"] == "bf16" else 4
        return {"bytes": float(n * e * (2 if c["grad"] else 1) + c["rows"] * (8 + 4 + 8)),
                "flops": 4.0 * n + (4.0 * n if c["grad"] else 0.0)}
    count = 2 * c["pairs"] if c["op"] == "preference" else c["seqs"]
    tokens = float(_tokens(count, c["length"]))
    if c["op"] == "preference":
        return {"bytes": tokens * (4 + (4 if c["reference"] else 0) + 1 + 4) + 24 * count, "flops": 4.0 * tokens}
    adv = 4 * tokens if c["per_token"] else 4 * count
    return {"bytes": tokens * (4 * 3 + 1 + 4) + adv + 12 * count, "flops": 20.0 * tokens}
