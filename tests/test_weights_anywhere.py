"""Parameters that are views into a flat buffer, on no 16-byte boundary: the library's calls are handed addresses that they
take (no GPU needed)."""
import pytest
import torch

import nvfp4_quantization_current_gb300 as Q
import nvfp4_quantization_current_gb300.linear as linear
from test_operators_abi import L  # noqa: F401 (a fixture)

BF16 = torch.bfloat16


@pytest.fixture
def calls(L, monkeypatch):
    """Calls that compute nothing, but take what the library takes: every address of a tensor here is on a 16-byte boundary."""
    made = []
    bad = set()

    def call(name, *args):
        assert not bad & set(args), name
        made.append(name)

    monkeypatch.setattr(Q, "_call", call)
    monkeypatch.setattr(Q, "_stream", lambda dev: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    return made, bad


def flat(module, bad):
    """The module with its parameters in one buffer, from its second element on."""
    params = list(module.parameters())
    buf = torch.zeros(sum(p.numel() for p in params) + 9, dtype=params[0].dtype)
    at = 1
    for p in params:
        view = buf[at:at + p.numel()].view(p.shape)
        view.copy_(p.data)
        p.data = view
        assert p.data_ptr() % 16
        bad.add(p.data_ptr())
        at += p.numel()
    return module


@pytest.mark.parametrize("kind", ["RMSNorm", "NormBlockwiseLinear", "BlockwiseLinear", "NVFP4Linear"])
@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_weights_of_any_address(kind, dtype, calls):
    made, bad = calls
    kw = dict(device="cpu", dtype=dtype)
    m = flat(linear.RMSNorm(128, **kw) if kind == "RMSNorm" else getattr(linear, kind)(128, 128, **kw), bad)
    x = torch.randn(128, 128, dtype=dtype, requires_grad=True)
    y = m(x, offset=0) if kind == "NVFP4Linear" else m(x)
    y.sum().backward()
    assert made and x.grad is not None and all(p.grad is not None and p.grad.shape == p.shape for p in m.parameters())
    with torch.no_grad():
        m(x, offset=0) if kind == "NVFP4Linear" else m(x)
