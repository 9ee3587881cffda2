"""The linear layer and dropout as a model uses them: reports, gradients, masks, strides and shapes."""
import pytest
import torch

import nvfp4_quantization_current_gb300 as Q
from nvfp4_quantization_current_gb300.linear import BlockwiseLinear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Q.lib()


def test_layer_status_reports_casts_and_products():
    layer = BlockwiseLinear(256, 128)
    x = torch.randn(200, 256, device="cuda", dtype=torch.bfloat16)
    layer(x)
    assert layer.status.item() == 0
    y = layer(x)
    y.backward(torch.full_like(y, torch.inf))
    assert layer.status.item() == Q.Q_ST_NONFINITE
    layer.status.zero_()
    x[3, 5] = torch.nan
    layer(x)
    assert layer.status.item() == Q.Q_ST_NONFINITE
    layer.status.zero_()
    x[3, 5] = 0
    try:
        assert Q.lib().selftest_mm_give_up(1) == Q.Q_OK
        layer(x)
    finally:
        Q.lib().selftest_mm_give_up(0)
    assert layer.status.item() == Q.Q_ST_TIMEOUT


def test_captured_training_call_needs_its_offset():
    layer = BlockwiseLinear(256, 128, p=0.5, seed=4, dtype=torch.float32)
    x = torch.randn(128, 256, device="cuda")
    want = layer(x, offset=12)
    assert not torch.equal(layer(x), layer(x))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.no_grad(), torch.cuda.graph(g):
        with pytest.raises(ValueError, match="offset"):
            layer(x)
        y = layer(x, offset=12)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(3, 7), (64, 512)])
def test_drop_add_gradient(dtype, shape):
    """Of x by the same call, of the residual as it is; strided and unaligned gradients; exactly linear, so by differences too."""
    x, r, t = (torch.randn(shape, device="cuda", dtype=dtype, requires_grad=True) for _ in range(3))
    y = Q.drop_add(x, 0.25, 5, 3, residual=r)
    with torch.no_grad():
        assert torch.equal(y, Q.drop_add(x, 0.25, 5, 3, residual=r))
    g = torch.randn(shape[::-1], device="cuda", dtype=dtype).t()
    dx, dr = torch.autograd.grad(y, (x, r), g)
    assert torch.equal(dx, Q.drop_add(g.contiguous(), 0.25, 5, 3)) and torch.equal(dr, g)
    both = torch.cat([t.flatten()[:1], Q.drop_add(x, 0.25, 5, 3).flatten()])   # its gradient begins one element off a boundary
    h = torch.randn_like(both)
    (dx,) = torch.autograd.grad(both, x, h)
    assert torch.equal(dx, Q.drop_add(h[1:].clone().view(shape), 0.25, 5, 3))
    if dtype == torch.float32:   # c = 4/3 is a double's: each product rounds once, by 2^-24 of it
        with torch.no_grad():
            f = Q.drop_add(x + 1, 0.25, 5, 3).double() - Q.drop_add(x, 0.25, 5, 3).double()
            slope = Q.drop_add(torch.ones_like(x), 0.25, 5, 3).double()
            assert bool(((f - slope).abs() <= 2.0 ** -22 * (x.double().abs() + 2) * slope).all())
