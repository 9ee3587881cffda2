"""The linear layer and dropout as a model uses them: reports, gradients, masks, strides and shapes."""
import pytest
import torch

import nvfp4_quantization_current_gb300 as Q
from nvfp4_quantization_current_gb300.linear import BlockwiseLinear
from test_gpu_operators import lossless, mm_bound

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


def off_by_one(t):
    return torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)


@pytest.mark.parametrize("made", [lambda t: t.transpose(0, 1).contiguous().transpose(0, 1), lambda t: t.repeat(1, 1, 2)[..., : t.shape[-1]],
                                  off_by_one])
@pytest.mark.parametrize("rows", [40, 64])
def test_strided_and_unaligned_operands(made, rows):
    layer = BlockwiseLinear(256, 128, p=0.5, seed=2)
    x, r, g = (torch.randn(4, rows, n, device="cuda", dtype=torch.bfloat16) for n in (256, 128, 128))

    def run(f):
        layer.weight.grad = None
        a, b = x.clone().requires_grad_(), r.clone().requires_grad_()
        y = layer(f(a), f(b), offset=0)
        y.backward(f(g))
        return y.detach(), a.grad, b.grad, layer.weight.grad

    assert all(torch.equal(a, b) for a, b in zip(run(made), run(lambda t: t)))


@pytest.mark.parametrize("shape", [(0, 256), (2, 0, 256)])
def test_no_rows(shape):
    layer = BlockwiseLinear(256, 128, p=0.5)
    x, r = (torch.zeros((*shape[:-1], n), device="cuda", dtype=torch.bfloat16, requires_grad=True) for n in (256, 128))
    y = layer(x, r)
    assert y.shape == r.shape
    y.sum().backward()
    assert x.grad.shape == x.shape and r.grad.shape == r.shape
    assert torch.equal(layer.weight.grad, torch.zeros_like(layer.weight))
    layer.main_grad = torch.ones(128, 256, device="cuda")
    layer(x, r).sum().backward()
    assert bool((layer.main_grad == 1).all())


# ---------------------------------------------------------------------------
# gradients that cannot be a little wrong
# ---------------------------------------------------------------------------

def padded(t):
    return torch.nn.functional.pad(t, (0, 0, 0, -t.shape[0] % 128))


@pytest.mark.parametrize("M", [128, 200, 256, 1])
def test_lossless_gradients_are_the_formulas(M):
    """Without dropout, integers whose tiles all reach 7 are cast without loss (and so are zero rows below them, rowwise):
    every sum is exact.  The transposed copy's tiles reach 7 where no row is cut off."""
    layer = BlockwiseLinear(256, 128, dtype=torch.float32)
    rows = -(-M // 128) * 128
    x = lossless((rows, 256), 1)[:M].contiguous().requires_grad_()
    with torch.no_grad():
        layer.weight.copy_(lossless((128, 256), 2))
    dy = lossless((rows, 128), 4)[:M].contiguous()
    y = layer(x)
    assert torch.equal(y.double(), x.double() @ layer.weight.double().T)
    y.backward(dy)
    assert torch.equal(x.grad.double(), dy.double() @ layer.weight.double())
    if M % 128 == 0:
        assert torch.equal(layer.weight.grad.double(), dy.double().T @ x.double())


@pytest.mark.parametrize("M", [1, 100, 128, 200, 384])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradients_are_the_products_of_the_casts(M, p, dtype):
    """Both gradients against the products in 64 bits of what the casts decode to: the cast of the dropped gradient, of x with
    its rows filled up, and of the weight.  Only the products' own tolerance is left, and one rounding of each decoded
    value (2^-24, two factors: 2^-23 of the sum of magnitudes)."""
    torch.manual_seed(M)
    layer = BlockwiseLinear(384, 256, p=p, seed=17, dtype=dtype)
    x = torch.randn(M, 384, device="cuda", dtype=dtype, requires_grad=True)
    dy = torch.randn(M, 256, device="cuda", dtype=dtype)
    layer(x, offset=40).backward(dy)
    g = Q.drop_q_blockwise(padded(dy), p, 17, 40, colwise=True)
    xq = Q.q_blockwise(padded(x.detach()), colwise=True)
    wq = Q.q_blockwise(layer.weight.detach(), "128x128", colwise=True)
    wide = lambda t, d: t.dequantize(d).double()
    for got, a, b, blocks in ((x.grad, wide(g, Q.Q_ROW)[:M], wide(wq, Q.Q_COL), 2), (layer.weight.grad, wide(g, Q.Q_COL), wide(xq, Q.Q_COL), -(-M // 128))):
        ref, mags = a @ b.T, a.abs() @ b.abs().T
        ref, tol = mm_bound(ref, mags, blocks, dtype)
        assert got.dtype == dtype and bool(((got.double() - ref).abs() <= tol + 2.0 ** -22 * mags).all())
    if p > 0:   # and the decoded gradient is the dropped one: a code is off by 2^-4 of its value, or 2^-10 448 / alpha below the normal ones
        keep = Q.drop_add(torch.ones_like(dy, dtype=torch.float32), p, 17, 40).double()
        want = dy.double() * keep
        top = want.view(M, -1, 128).abs().amax(2, keepdim=True).expand(-1, -1, 128).reshape(M, -1)
        assert bool(((wide(g, Q.Q_ROW)[:M] - want).abs() <= want.abs() * 2.0 ** -4 * (1 + 2.0 ** -20) + top * 2.0 ** -10 / 448).all())
