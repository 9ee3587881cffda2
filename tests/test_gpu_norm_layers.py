"""The norm's and the NVFP4 product's layers as a model uses them, alone and in a row: each against its own operators
called by hand, whose results other tests compare with the formulas, and against the formulas where casts lose nothing."""
import pytest
import torch

import nvfp4_quantization_current_gb300 as Q
from nvfp4_quantization_current_gb300.linear import BlockwiseLinear, NormBlockwiseLinear, NVFP4Linear, RMSNorm
from test_gpu_matmul_nvfp4 import reference

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Q.lib()


def new(*shape, dtype=BF16, seed=0):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def rows(t, step):
    return torch.nn.functional.pad(t, (0, 0, 0, -t.shape[0] % step))


# ---------------------------------------------------------------------------
# NVFP4Linear
# ---------------------------------------------------------------------------

def lossless(shape, seed):
    """FP4 values with a 6 in every block of 16 along both axes: the scales are 448, alpha 1, and every code is exact."""
    g = torch.Generator("cuda").manual_seed(seed)
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    x = values[torch.randint(0, 14, shape, generator=g, device="cuda")]
    i = torch.arange(shape[0], device="cuda")
    for k in range(0, shape[1], 16):
        x[i, k + i % 16] = 6.0
    return x


@pytest.mark.parametrize("M", [16, 48, 160])
def test_fp4_layer_of_exact_codes(M):
    """Forward and input gradient are the products of the tensors themselves: the tensors' scales, 1/448 rounded, and their
    two products round by 2^-24 each; a stochastic rounding does not move what needs none."""
    layer = NVFP4Linear(256, 96, dtype=F32)
    with torch.no_grad():
        layer.weight.copy_(lossless((96, 256), 1))
    x, dy = lossless((M, 256), 2).requires_grad_(), lossless((M, 96), 3)
    y = layer(x)
    y.backward(dy)
    for got, want, mags in ((y, x @ layer.weight.T, x.abs() @ layer.weight.abs().T), (x.grad, dy @ layer.weight, dy.abs() @ layer.weight.abs())):
        # sums of 256 products of multiples of 1/4 below 36: exact in FP32 as integers
        assert bool(((got.double() - want.double()).abs() <= 6 * 2.0 ** -24 * want.double().abs()).all())
    assert layer.status.item() == 0


@pytest.mark.parametrize("shape", [(16, 256), (33, 256), (2, 20, 256), (256,), (0, 256), (640, 256)])
@pytest.mark.parametrize("dtype,wt", [(BF16, BF16), (F32, BF16), (BF16, F32)])
def test_fp4_layer_by_hand(shape, dtype, wt):
    layer = NVFP4Linear(256, 96, seed=5, dtype=wt)
    x = new(*shape, dtype=dtype, seed=1).requires_grad_()
    y = layer(x, offset=77)
    dy = new(*shape[:-1], 96, dtype=dtype, seed=2)
    y.backward(dy)
    assert y.shape == (*shape[:-1], 96) and y.dtype == dtype and x.grad.shape == x.shape and layer.weight.grad.dtype == wt
    x2, d2 = x.detach().reshape(-1, 256), dy.reshape(-1, 96)
    M = x2.shape[0]
    w = Q.q_nvfp4(layer.weight.detach(), "16x16", colwise=True)
    if M == 0:
        assert bool((layer.weight.grad == 0).all())
        return
    xr, xc = Q.q_nvfp4_recipe(rows(x2, 32), layer.sign_mask)
    dr, dc = Q.q_nvfp4_recipe(rows(d2, 32), layer.sign_mask, "sr", 5, 77)
    row, col = (lambda t: (t.q_row, t.sb_row, t.s_global)), (lambda t: (t.q_colT, t.sb_colT, t.s_global))
    half = lambda t: 2.0 ** -8 if t.dtype == BF16 else 2.0 ** -24
    for got, a, b, bb, n in ((y.reshape(-1, 96), row(xr), row(w), "16x16", 256), (x.grad.reshape(-1, 256), row(dr), col(w), "16x16", 96),
                             (layer.weight.grad, col(dc), col(xc), "1x16", rows(x2, 32).shape[0])):
        want, mags = reference(*a, "1x16", *b, bb)
        want, mags = want[:got.shape[0]], mags[:got.shape[0]]
        tol = (n * 2.0 ** -23 + 11 * 2.0 ** -24) * mags
        assert bool(((got.double() - want).abs() <= tol + half(got) * (want.abs() + tol)).all())
    again = layer(x, offset=77)
    again.backward(dy)   # the same numbers drawn again: twice the gradient
    assert torch.equal(again, y)


def test_fp4_layer_main_grad_serving_and_status():
    layer = NVFP4Linear(256, 96, seed=3)
    x = new(50, 256, seed=4)
    layer(x, offset=1).float().square().sum().backward()
    want = layer.weight.grad.float()
    layer.weight.grad = None
    layer.main_grad = torch.zeros(96, 256, device="cuda")
    for _ in range(2):
        layer(x, offset=1).float().square().sum().backward()
    assert layer.weight.grad is None
    assert bool(((layer.main_grad - 2 * want).abs() <= 2 * 2.0 ** -8 * want.abs() * (1 + 2.0 ** -8) + 1e-30).all())   # want is rounded to BF16
    copies = layer.quantize_weight(colwise=False)
    with torch.no_grad():
        one = layer(x[:1], copies=copies)
        t = Q.q_nvfp4(rows(x[:1], 16))
        assert torch.equal(one, Q.matmul_nvfp4(t.q_row[:1], t.sb_row[:1], t.s_global, copies.q_row, copies.sb_row, copies.s_global))
    with pytest.raises(ValueError, match="transposed copy"):
        layer(x.clone().requires_grad_(), copies=copies)
    assert layer.status.item() == 0
    x[3, 5] = torch.inf
    layer(x)
    assert layer.status.item() & Q.Q_ST_NONFINITE


@pytest.mark.parametrize("weights", [True, False])
def test_fp4_layer_partial_gradients(weights):
    layer = NVFP4Linear(64, 32, seed=9)
    layer.weight.requires_grad_(weights)
    x = new(40, 64, seed=6).requires_grad_(not weights)
    y = layer(x, offset=3)
    y.backward(new(40, 32, seed=7))
    assert (x.grad is None) == weights and (layer.weight.grad is None) != weights


def test_fp4_layer_draws_and_captures():
    layer = NVFP4Linear(64, 32)
    x = new(64, 64, seed=8).requires_grad_()
    dy = new(64, 32, seed=9)
    grads = [torch.autograd.grad(layer(x), layer.weight, dy)[0] for _ in range(2)]
    assert not torch.equal(*grads)   # drawn per call
    torch.manual_seed(5)
    a = torch.autograd.grad(layer(x), layer.weight, dy)[0]
    torch.manual_seed(5)
    assert torch.equal(torch.autograd.grad(layer(x), layer.weight, dy)[0], a)
    copies = layer.quantize_weight(colwise=False)
    xs = x.detach().clone()
    with torch.no_grad():
        want = layer(xs, copies=copies)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = layer(xs, copies=copies)
        xs.mul_(2)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, layer(xs, copies=copies)) and not torch.equal(y, want)


def test_no_second_derivatives():
    x = new(32, 256, dtype=F32, seed=10).requires_grad_()
    for layer in (NVFP4Linear(256, 96, dtype=F32), NormBlockwiseLinear(256, 128, dtype=F32), RMSNorm(256, dtype=F32)):
        (g,) = torch.autograd.grad(layer(x).square().sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="no second derivative"):
            g.sum().backward()


# ---------------------------------------------------------------------------
# the norm's layers
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("shape", [(128, 256), (100, 256), (3, 50, 256), (256,), (0, 256)])
@pytest.mark.parametrize("dtype,wt", [(BF16, BF16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_layer_by_hand(shape, dtype, wt, residual):
    layer = NormBlockwiseLinear(256, 384, dtype=wt)
    with torch.no_grad():
        layer.norm_weight.copy_(1 + 0.1 * new(256, dtype=wt, seed=1))
    x = new(*shape, dtype=dtype, seed=2).requires_grad_()
    r = new(*shape, dtype=dtype, seed=3).requires_grad_() if residual else None
    out = layer(x, r)
    y, h = out if residual else (out, None)
    dy, dh = new(*shape[:-1], 384, dtype=dtype, seed=4), new(*shape, dtype=dtype, seed=5)
    torch.autograd.backward((y, h) if residual else y, (dy, dh) if residual else dy)
    x2 = rows(x.detach().reshape(-1, 256), 128)
    M = x[..., 0].numel()
    r2 = rows(r.detach().reshape(-1, 256), 128) if residual else None
    t, h2, rstd = Q.norm_q_blockwise(x2, layer.norm_weight.detach(), layer.eps, r2, colwise=True)
    w = layer.quantize_weight()
    assert torch.equal(y.reshape(-1, 384), Q.mm_blockwise(t.q_row[:M], t.s_row[:M], w.q_row, w.s_row, dtype=dtype))
    if residual:
        assert torch.equal(h.reshape(-1, 256), h2[:M])
    d = Q.q_blockwise(rows(dy.reshape(-1, 384), 128), "1x128", colwise=True)
    back = Q.mm_blockwise(d.q_row[:M], d.s_row[:M], w.q_colT, w.s_colT, dtype=dtype)
    dx, dn = Q.norm_grad(back, h2[:M], rstd[:M], layer.norm_weight.detach(), dh.reshape(-1, 256) if residual else None)
    assert torch.equal(x.grad.reshape(-1, 256), dx) and torch.equal(layer.norm_weight.grad, dn)
    if residual:
        assert torch.equal(r.grad, x.grad)
    dw = Q.mm_blockwise(d.q_colT, d.s_colT, t.q_colT, t.s_colT, tile_b="1x128", dtype=wt)
    assert torch.equal(layer.weight.grad, dw) and layer.status.item() == 0


def test_norm_layer_is_norm_then_layer():
    """Near the same thing in two steps: the copies are of the norm in FP32 instead of rounded to bfloat16."""
    layer = NormBlockwiseLinear(256, 128)
    plain, norm = BlockwiseLinear(256, 128), RMSNorm(256)
    with torch.no_grad():
        plain.weight.copy_(layer.weight)
        x, r = new(64, 256, seed=6), new(64, 256, seed=7)
        y, h = layer(x, r)
        z, k = norm(x, r)
        assert torch.equal(h, k)
        want = plain(z).double()
        # a copy's code may fall to the other side of a border: off by 2^-3 of its value instead of 2^-4 (2^-3 + 2^-4 between
        # them), and the results are rounded by 2^-8 each
        mags = z.double().abs() @ plain.weight.double().abs().T
        assert bool(((y.double() - want).abs() <= (2.0 ** -3 + 2.0 ** -4) * mags + 2.0 ** -7 * want.abs()).all())


def test_norm_layer_serving_and_strides():
    layer = NormBlockwiseLinear(256, 128)
    x, r = new(256, 40, seed=8).t(), new(40, 512, seed=9)[:, ::2]
    with torch.no_grad():
        copies = layer.quantize_weight(colwise=False)
        y, h = layer(x, r, copies=copies)
        a, b = layer(x.contiguous(), r.contiguous())
        assert torch.equal(y, a) and torch.equal(h, b)
        with pytest.raises(ValueError, match="residual must"):
            layer(x, r[:, :128])
        odd = torch.empty(40 * 256 + 1, device="cuda", dtype=BF16)[1:].view(40, 256).copy_(x)   # on a 2-byte boundary
        assert torch.equal(layer(odd, r)[0], y)
        assert torch.equal(RMSNorm(256)(odd), RMSNorm(256)(x.contiguous()))
    with pytest.raises(ValueError, match="transposed copy"):
        layer(x.clone().requires_grad_(), copies=copies)
    with pytest.raises(ValueError, match="eps"):
        NormBlockwiseLinear(256, 128, eps=0.0)


def test_gradients_of_the_sum_alone_and_of_the_norm_alone():
    layer = NormBlockwiseLinear(256, 128, dtype=F32)
    norm = RMSNorm(256, dtype=F32)
    for f in (layer, norm):
        x, r = new(8, 256, dtype=F32, seed=10).requires_grad_(), new(8, 256, dtype=F32, seed=11).requires_grad_()
        g = new(8, 256, dtype=F32, seed=12)
        (f(x, r)[1] * g).sum().backward()
        assert torch.equal(x.grad, g) and torch.equal(r.grad, g)
        f(x.detach(), r)[0].sum().backward()   # x has no gradient here: the residual's and the weights' are whole
        assert x.grad is not None and not torch.equal(r.grad, g)


# ---------------------------------------------------------------------------
# all of them in a row
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M", [64, 200])
def test_a_block_of_layers(M):
    """norm + FP8 layer, activation, norm that leaves its largest value, FP4 layer, with the residual stream through both: training
    against the same chain in 64 bits, serving against training's forward pass."""
    torch.manual_seed(0)
    up, norm, down = NormBlockwiseLinear(256, 512), RMSNorm(512), NVFP4Linear(512, 256, seed=1)
    top = torch.zeros(1, device="cuda")
    x, r = new(M, 256, seed=13).requires_grad_(), new(M, 256, seed=14).requires_grad_()

    def block(x, r, copies=(None, None), offset=5):
        y, h = up(x, r, copies=copies[0])
        z = norm(torch.nn.functional.silu(y), amax=top)
        return down(z, offset=offset, copies=copies[1], amax=top) + h

    out = block(x, r)
    out.float().square().mean().backward()
    grads = [t.grad for t in (x, r, up.weight, up.norm_weight, norm.weight, down.weight)]
    assert all(g is not None and bool(g.isfinite().all()) for g in grads) and up.status.item() == down.status.item() == 0
    with torch.no_grad():
        serve = block(x, r, (up.quantize_weight(colwise=False), down.quantize_weight(colwise=False)))
    assert torch.equal(serve, out)
    # the same chain in 64 bits, without casts: the gradients point the same way
    wide = [t.detach().double().requires_grad_() for t in (x, r, up.weight, up.norm_weight, norm.weight, down.weight)]
    X, R, W1, N1, N2, W2 = wide
    h = X + R
    rms = lambda v, w: v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * w
    z = rms(torch.nn.functional.silu(rms(h, N1) @ W1.T), N2)
    (z @ W2.T + h).square().mean().backward()
    for got, want in zip(grads, wide):
        a, b = got.double().flatten(), want.grad.flatten()
        assert float(a @ b / (a.norm() * b.norm())) > 0.9
    # serving in a graph, replayed on other inputs
    xs, rs = x.detach().clone(), r.detach().clone()
    copies = up.quantize_weight(colwise=False), down.quantize_weight(colwise=False)
    with torch.no_grad():
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = block(xs, rs, copies)
        xs.copy_(new(M, 256, seed=15))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, block(xs, rs, copies))


def test_a_captured_training_step():
    """A step with its backward pass captured, replayed on other inputs, against the eager one: the same numbers."""
    torch.manual_seed(1)
    up, norm, down = NormBlockwiseLinear(256, 512), RMSNorm(512), NVFP4Linear(512, 256, seed=1)
    params = [up.weight, up.norm_weight, norm.weight, down.weight]
    up.main_grad = torch.zeros(512, 256, device="cuda")
    xs, rs, ds = new(100, 256, seed=21), new(100, 256, seed=22), new(100, 256, seed=23)

    def step():
        x, r = xs.detach().requires_grad_(), rs.detach().requires_grad_()
        y, h = up(x, r)
        z = norm(torch.nn.functional.silu(y))
        out = down(z, offset=7) + h
        return list(torch.autograd.grad(out, [x, r, *params[1:], up.weight], ds, allow_unused=True))[:-1] + [up.main_grad.clone()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):   # first launches happen outside the capture
        step()
    torch.cuda.synchronize()
    up.main_grad.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in (24, 25):
        for t, s in ((xs, seed), (rs, seed + 10), (ds, seed + 20)):
            t.copy_(new(100, 256, seed=s))
        up.main_grad.zero_()
        g.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in got]
        up.main_grad.zero_()
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(replayed, want)) and len(want) == 6
    assert up.status.item() == down.status.item() == 0
