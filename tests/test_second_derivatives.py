"""The layers and the norm have no second derivative, and every way of asking for one says so (no GPU needed: the
library's calls do nothing here, what is tested is the graph around them)."""
import pytest
import torch

import nvfp4_quantization_current_gb300 as Q
import nvfp4_quantization_current_gb300.linear as linear
from test_operators_abi import L  # noqa: F401 (a fixture)

K = 128


@pytest.fixture(autouse=True)
def no_kernels(L, monkeypatch):
    monkeypatch.setattr(Q, "_call", lambda name, *args: None)
    monkeypatch.setattr(Q, "_stream", lambda dev: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))


def made(kind):
    """(the call as a function of x, its weights)."""
    kw = dict(device="cpu", dtype=torch.float32)
    r = torch.randn(32, K)
    if kind == "norm_add":
        w = torch.ones(K, requires_grad=True)
        return lambda x: Q.norm_add(x, w)[0], [w]
    if kind == "norm_add, residual":
        w = torch.ones(K, requires_grad=True)
        return lambda x: Q.norm_add(x, w, residual=r)[0], [w]
    if kind == "norm_add, the residual's":
        w = torch.ones(K, requires_grad=True)
        return lambda x: Q.norm_add(r, w, residual=x)[0], [w]
    if kind == "RMSNorm":
        m = linear.RMSNorm(K, **kw)
        return m, list(m.parameters())
    if kind.startswith("NormBlockwiseLinear"):
        m = linear.NormBlockwiseLinear(K, 256, **kw)
        return (m if kind[-1] == "r" else lambda x: m(x, r)[0]), list(m.parameters())
    if kind == "NVFP4Linear":
        m = linear.NVFP4Linear(K, 256, **kw)
        return lambda x: m(x, offset=0), list(m.parameters())
    m = linear.BlockwiseLinear(K, 256, **kw)
    return m, list(m.parameters())


KINDS = ["norm_add", "norm_add, residual", "norm_add, the residual's", "RMSNorm", "NormBlockwiseLinear", "NormBlockwiseLinear, residual",
         "NVFP4Linear", "BlockwiseLinear"]
raises = lambda: pytest.raises(RuntimeError, match="no second derivative")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("loss", [torch.sum, lambda y: y.square().sum()])
@pytest.mark.parametrize("way", ["hvp", "vhp", "hessian", "jvp"])
def test_functional(kind, loss, way):
    f, _ = made(kind)
    x, v = torch.randn(32, K), torch.randn(32, K)
    with raises():
        if way == "jvp":   # the gradient's derivative by the gradient that comes in
            torch.autograd.functional.jvp(f, x, v)
        elif way == "hessian":
            torch.autograd.functional.hessian(lambda x: loss(f(x)), x)
        else:
            getattr(torch.autograd.functional, way)(lambda x: loss(f(x)), x, v)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("leaf", [True, False])
def test_by_every_input(kind, leaf):
    """Gradients of a loss that is linear in the result, differentiated by x (a leaf, or made of one) and by each weight."""
    f, weights = made(kind)
    a = torch.randn(32, K, requires_grad=True)
    x = a if leaf else a * 2
    grads = torch.autograd.grad(f(x).sum(), [x, *weights], create_graph=True)
    for g in grads:
        for t in (a, *weights):
            with raises():
                torch.autograd.grad(g.sum(), t, allow_unused=True, retain_graph=True)
    with raises():
        sum(g.sum() for g in grads).backward()


def test_the_sum_has_its_second_derivative():
    """Where the result is h alone nothing is lost, and nothing raises."""
    for f in (lambda x, r: Q.norm_add(x, torch.ones(K), residual=r)[1], lambda x, r: linear.NormBlockwiseLinear(K, 128, device="cpu", dtype=torch.float32)(x, r)[1]):
        h = torch.randn(32, K)
        x = torch.randn(32, K, requires_grad=True)
        (g,) = torch.autograd.grad((f(x, torch.zeros(32, K)) * x * h).sum(), x, create_graph=True)
        torch.autograd.grad(g.sum(), x)


@pytest.mark.parametrize("kind", KINDS)
def test_nothing_is_kept_without_gradients(kind):
    f, weights = made(kind)
    with torch.no_grad():
        assert f(torch.randn(32, K)).grad_fn is None
    for w in weights:
        w.requires_grad_(False)
    assert f(torch.randn(32, K)).grad_fn is None
