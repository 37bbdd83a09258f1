"""The autograd functions' backward passes take the addresses of what the forward saved: saved-tensor hooks that give
back tensors of other strides, dtypes or shapes are refused before anything is launched.  On the CPU, with the calls
into the library replaced; on the GPU, hooks that keep copies elsewhere give the same gradients."""
import pytest
import torch

import lora_linear_layers_amd as L
from lora_linear_layers_amd import functional as F

BF16 = torch.bfloat16


def _columns(t):
    """An equal tensor whose rows are not contiguous."""
    return t if t.dim() < 2 else t.transpose(-1, -2).contiguous().transpose(-1, -2)


def _longer(t):
    """Another shape: a row more."""
    return torch.cat((t, t[-1:])) if t.dim() else t


CHANGES = {"columns": _columns, "wider": lambda t: t.double() if t.is_floating_point() else t.long(), "longer": _longer,
           "spaced": lambda t: torch.stack((t, t), -1)[..., 0], "device": lambda t: t.to("meta")}


def _tensors(dev, M=4, k=32, d=24, n=3, r=8):
    g = torch.Generator().manual_seed(1)
    normal = lambda *s: torch.randn(*s, generator=g).to(dev, BF16)  # noqa: E731
    return {"X": normal(M, k), "R": normal(M, k), "w": normal(k), "W": normal(d, k), "A": normal(r, k), "B": normal(d, r),
            "As": normal(n, r, k), "Bs": normal(n, d, r), "bias": normal(d), "scales": torch.ones(n, device=dev),
            "index": torch.arange(M, dtype=torch.int32, device=dev) % n}


def _norm(t):
    return L.LoraRmsNormFunction.apply(t["X"].requires_grad_(), t["R"], t["w"])[0]


def _act8(t):
    return L.LoraLinearAct8Function.apply(t["X"].requires_grad_(), t["W"], t["A"].requires_grad_(), t["B"], 0.5)


def _multi(t):
    return L.LoraMultiFunction.apply(t["X"].requires_grad_(), t["W"], t["As"].requires_grad_(), t["Bs"], t["scales"], t["index"])


def _epi(t):
    return L.LoraLinearEpiFunction.apply(t["X"].requires_grad_(), t["W"], t["A"].requires_grad_(), t["B"], t["bias"], None, 0.5, "silu")


OPS = {"norm": _norm, "act8": _act8, "multi": _multi, "epi": _epi}


@pytest.fixture
def replaced(monkeypatch):
    """The library's part in plain torch; its backward entry points fail the test."""
    def reached(*_, **__):
        pytest.fail("the backward took the tensors as they came")
    linear = lambda X, W: X @ W.T  # noqa: E731
    monkeypatch.setattr(F, "_gpu", lambda t: t.device)
    monkeypatch.setattr(F, "lora_rmsnorm_fwd", lambda X, w, eps, R, pack: (X * w, X + R, X.float().mean(1), None, None))
    monkeypatch.setattr(F, "lora_linear_epi_fwd", lambda X, m, *a, **k: (linear(X, m["W"]), linear(X, m["W"])))
    monkeypatch.setattr(F, "lora_act8_pack", lambda X: (X.to(torch.float8_e4m3fn), X.float().amax(1)))
    monkeypatch.setattr(F, "_multi_fwd", lambda dims, X, W, *a: linear(X, W))
    for name in ("_rmsnorm_bwd", "_act8_bwd", "_multi_bwd", "_epi_bwd"):
        monkeypatch.setattr(F, name, reached)


@pytest.mark.parametrize("change", CHANGES)
@pytest.mark.parametrize("op", OPS)
def test_changed_tensors_are_refused(replaced, op, change):
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, CHANGES[change]):
        Y = OPS[op](_tensors("cpu"))
        with pytest.raises(ValueError, match="saved"):
            Y.backward(torch.ones_like(Y))


@pytest.mark.gpu
@pytest.mark.parametrize("op", OPS)
def test_hooks_on_the_gpu(lib, op):
    """Kept on the host and brought back: the same gradients; in column order: refused."""
    def grads(hooks):
        t = _tensors("cuda", M=40, k=64, d=48)
        with hooks:
            Y = OPS[op](t)
            Y.backward(torch.ones_like(Y))
        return [v.grad for v in t.values() if v.grad is not None]
    want = grads(torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: t))
    assert want
    for pin in (False, True):
        for a, b in zip(grads(torch.autograd.graph.save_on_cpu(pin_memory=pin)), want):
            assert torch.equal(a, b)
    for change in ("columns", "spaced", "wider"):
        with pytest.raises(ValueError, match="saved"):
            grads(torch.autograd.graph.saved_tensors_hooks(lambda t: t, CHANGES[change]))
