"""The norm's two passes report to one status word, given to norm_add or the module's own (no GPU needed: what is tested is
the address that the library's calls are handed)."""
import pytest
import torch

import nvfp4_quantization_current_gb300 as Q
import nvfp4_quantization_current_gb300.linear as linear
from test_operators_abi import L  # noqa: F401 (a fixture)


@pytest.fixture
def words(L, monkeypatch):
    made = []
    monkeypatch.setattr(Q, "_call", lambda name, *args: made.append((name, args[-2])))
    monkeypatch.setattr(Q, "_stream", lambda dev: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    return made


@pytest.mark.parametrize("residual", [False, True])
def test_norm_add_and_its_backward_pass(words, residual):
    status = torch.zeros(1, dtype=torch.int32)
    x, w, r = torch.randn(4, 64, requires_grad=True), torch.ones(64, requires_grad=True), torch.randn(4, 64)
    for word in (status, None):
        y = Q.norm_add(x, w, residual=r if residual else None, status=word)[0]
        y.sum().backward()
        assert words == [(n, None if word is None else word.data_ptr()) for n in ("norm_add", "norm_grad")]
        words.clear()


@pytest.mark.parametrize("residual", [False, True])
def test_module(words, residual):
    m = linear.RMSNorm(64, device="cpu", dtype=torch.float32)
    assert m.status.dtype == torch.int32 and m.status.tolist() == [0]
    x, r = torch.randn(4, 64, requires_grad=True), torch.randn(4, 64)
    y = m(x, r)[0] if residual else m(x)
    y.sum().backward()
    assert words == [(n, m.status.data_ptr()) for n in ("norm_add", "norm_grad")]
    words.clear()
    with torch.no_grad():
        m(x)
    assert words == [("norm_add", m.status.data_ptr())]
    assert [n for n, _ in m.named_parameters()] == ["weight"] and list(m.state_dict()) == ["weight"]
