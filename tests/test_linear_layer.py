"""The linear layer's own logic on the CPU: its four operators are replaced by plain ones on the
oracle's copies, which refuse what the library's refuse."""
import numpy as np
import pytest
import torch

import nvfp4_quantization_current_gb300 as Q
import nvfp4_quantization_current_gb300.linear as linear
import oracle as O
from test_gpu_operators import draws

TILE = {"1x128": O.T1x128, "128x128": O.T128x128}


def contiguous(t):
    if not t.is_contiguous() or t.data_ptr() % 16:
        raise ValueError("input must be contiguous and aligned")
    return t


def tensors(t, tile):
    f = lambda v: None if v is None else torch.from_numpy(v)
    return Q.BlockwiseTensor(f(t.q_row), f(t.s_row), f(t.q_colT), f(t.s_colT), tile)


def decoded(q, s, tile):
    return torch.from_numpy(O.dq_blockwise(q.numpy(), s.numpy(), TILE[tile])).double() if q.numel() else q.double()


class Plain:
    """The operators on CPU tensors; `status` collects what each call was given for it."""

    def __init__(self):
        self.status, self.offsets, self.version = [], [], {}

    def q_blockwise(self, x, tile="1x128", rowwise=True, colwise=False, out=None, status=None):
        self.status.append(status)
        return tensors(O.blockwise(contiguous(x).numpy(), TILE[tile], rowwise, colwise), TILE[tile])

    def mm_blockwise(self, a, s_a, b, s_b, tile_a="1x128", tile_b="128x128", dtype=torch.bfloat16, out=None, accumulate=False,
                     status=None):
        self.status.append(status)
        y = decoded(a, s_a, tile_a) @ decoded(b, s_b, tile_b).T
        if out is None:
            return y.to(dtype)
        return out.copy_(y + out.double() if accumulate else y)

    def kept(self, x, p, seed, offset):
        self.offsets.append((seed, offset))
        T = int(np.rint(p * 65536))
        keep = torch.from_numpy(draws(x.numel(), seed, offset) >= T).view(x.shape)
        return torch.where(keep, x * (65536 / (65536 - T) if T < 65536 else 0.0), 0.0)

    def drop_add(self, x, p, seed, offset=0, residual=None, out=None):
        y = self.kept(contiguous(x), p, seed, offset)
        if residual is not None:
            if residual.shape != x.shape or residual.dtype != x.dtype:
                raise ValueError("residual must have x's shape and dtype")
            y = y + contiguous(residual)
        return y if out is None else out.copy_(y)

    def drop_q_blockwise(self, x, p, seed, offset=0, rowwise=True, colwise=False, out=None, status=None):
        self.status.append(status)
        y = self.kept(contiguous(x), p, seed, offset)
        return tensors(O.blockwise(y.numpy(), O.T1x128, rowwise, colwise), O.T1x128)


@pytest.fixture
def plain(monkeypatch):
    ops = Plain()
    for name in ("q_blockwise", "mm_blockwise", "drop_add", "drop_q_blockwise"):
        monkeypatch.setattr(linear, name, getattr(ops, name))
    return ops


def layer_of(p=0.0, **kw):
    torch.manual_seed(1)
    return linear.BlockwiseLinear(256, 128, p=p, device="cpu", dtype=torch.float32, **kw)


def test_every_cast_and_product_gets_the_layers_status(plain):
    """A wait that ran out, or a non-finite input, is found in the layer's status word, forward and backward."""
    layer = layer_of(p=0.5, seed=3)
    x = torch.randn(256, 256, requires_grad=True)
    layer(x, offset=0).sum().backward()
    assert len(plain.status) == 6   # two casts and a product, a cast and two products
    assert layer.status.dtype == torch.int32 and layer.status.tolist() == [0]
    assert all(s is layer.status for s in plain.status)


@pytest.mark.parametrize("of_y", [lambda y: y.square().sum(), lambda y: y.sum()])
def test_a_second_derivative_is_refused_and_not_lost(plain, of_y):
    """The backward pass has no derivative: a gradient penalty must not train without its part, whether its
    gradient is one of the incoming gradient or of the weight alone (y's sum: dx is the weight's column sums)."""
    layer = layer_of()
    x = torch.randn(128, 256, requires_grad=True)
    r = torch.randn(128, 128, requires_grad=True)
    y = layer(x, r)
    dx, dw = torch.autograd.grad(of_y(y), (x, layer.weight), create_graph=True)
    for g in (dx, dw):
        with pytest.raises(RuntimeError, match="no second derivative"):
            (y.sum() + g.square().sum()).backward(retain_graph=True)
    dr = torch.autograd.grad(of_y(layer(x, r)), r, create_graph=True)[0]
    if dr.requires_grad:   # y squared: the residual's gradient is 2 y, whose own derivative the layer has
        first = torch.autograd.grad(dr.sum(), x, create_graph=True)[0]
        with pytest.raises(RuntimeError, match="no second derivative"):
            torch.autograd.grad(first.sum(), r)
    layer.weight.grad = None
    of_y(layer(x, r)).backward()   # the first derivative alone is as before
    assert torch.equal(x.grad, dx) and torch.equal(layer.weight.grad, dw) and not x.grad.requires_grad


def test_calls_without_an_offset_draw_masks_of_their_own(plain):
    """In training, call by call and layer by layer; the backward pass draws what its forward pass drew."""
    one, two = layer_of(p=0.5), linear.BlockwiseLinear(256, 128, p=0.5, device="cpu", dtype=torch.float32)
    x = torch.randn(128, 256, requires_grad=True)
    masks = [layer(x) != 0 for layer in (one, one, two, two)]
    for i, a in enumerate(masks):
        assert 0.45 < float(a.double().mean()) < 0.55
        assert all(0.4 < float((a == b).double().mean()) < 0.6 for b in masks[:i])
    assert len(set(plain.offsets)) == 4
    assert one.seed != two.seed   # the same offset gives layers masks of their own, too
    assert not torch.equal(one(x, offset=7) != 0, two(x, offset=7) != 0)
    plain.offsets.clear()
    y, z = one(x), one(x)
    y.sum().backward()
    z.sum().backward()
    assert plain.offsets[2:] == plain.offsets[:2] and plain.offsets[0] != plain.offsets[1]
    plain.offsets.clear()
    one.eval()
    assert torch.equal(one(x), one(x)) and plain.offsets == []


def test_masks_follow_torchs_generator_and_checkpointing(plain):
    """The same seed of torch's generator gives the same masks, and so does a recomputed forward pass."""
    from torch.utils.checkpoint import checkpoint
    layer = layer_of(p=0.5)
    x = torch.randn(128, 256, requires_grad=True)

    def grads(f):
        torch.manual_seed(5)
        layer.weight.grad = x.grad = None
        y = f(x)
        y.square().sum().backward()
        return y.detach(), x.grad, layer.weight.grad

    want = grads(layer)
    for reentrant in (False, True):
        assert all(torch.equal(a, b) for a, b in zip(grads(lambda x: checkpoint(layer, x, use_reentrant=reentrant)), want))


def test_a_given_offset_and_seed_are_taken_as_they_are(plain):
    layer = layer_of(p=0.5, seed=9)
    state = torch.get_rng_state()
    layer(torch.randn(128, 256, generator=torch.Generator().manual_seed(1)), offset=0)
    assert plain.offsets == [(9, 0)] and torch.equal(torch.get_rng_state(), state)
    layer_of()   # without dropout nothing is drawn
    torch.manual_seed(3)
    a = torch.rand(1)
    torch.manual_seed(3)
    linear.BlockwiseLinear(128, 128, device="meta")
    assert torch.equal(torch.rand(1), a)


def test_a_residual_of_another_shape_is_refused_and_not_reinterpreted(plain):
    """It has y's shape, or y's rows flattened; one with as many elements only is another tensor."""
    layer = layer_of()
    x = torch.randn(4, 32, 256)
    r = torch.randn(4, 32, 128, requires_grad=True)
    y = layer(x)
    assert torch.allclose(layer(x, r), y + r)
    flat = r.detach().reshape(128, 128).requires_grad_()
    z = layer(x, flat)
    assert z.shape == (4, 32, 128) and torch.equal(z, layer(x, r))
    g = torch.randn(4, 32, 128)
    assert torch.equal(torch.autograd.grad(z, flat, g)[0], g.reshape(128, 128))
    for shape in ((32, 4, 128), (4, 128, 32), (128 * 128,), (4, 32, 64), (64, 256), (32, 128), (128,)):
        with torch.no_grad(), pytest.raises(ValueError, match="residual"):
            layer(x, torch.zeros(shape))


def off_by_one(t):
    """The same values one element off a 16-byte boundary."""
    return torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)


@pytest.mark.parametrize("made", [lambda t: t.transpose(0, 1).contiguous().transpose(0, 1), lambda t: t.repeat(1, 1, 2)[..., : t.shape[-1]],
                                  off_by_one])
def test_strided_and_unaligned_operands_are_those_they_hold(plain, made):
    """x, the residual and the incoming gradient, as a slice, a transpose or a view into a buffer gives them."""
    layer = layer_of(p=0.5, seed=2)
    x, r, g = torch.randn(4, 40, 256), torch.randn(4, 40, 128), torch.randn(4, 40, 128)

    def run(f):
        layer.weight.grad = None
        a, b = x.clone().requires_grad_(), r.clone().requires_grad_()
        y = layer(f(a), f(b), offset=0)
        y.backward(f(g))
        return y.detach(), a.grad, b.grad, layer.weight.grad

    assert all(torch.equal(a, b) for a, b in zip(run(made), run(lambda t: t)))


@pytest.mark.parametrize("shape", [(0, 256), (2, 0, 256)])
def test_no_rows(plain, shape):
    """A batch that came out empty: an empty result, and gradients of zero."""
    layer = layer_of(p=0.5)
    x, r = torch.zeros(shape, requires_grad=True), torch.zeros((*shape[:-1], 128), requires_grad=True)
    y = layer(x, r)
    assert y.shape == r.shape
    y.sum().backward()
    assert x.grad.shape == x.shape and r.grad.shape == r.shape
    assert torch.equal(layer.weight.grad, torch.zeros(128, 256))
    layer.main_grad = torch.ones(128, 256)
    layer(x, r).sum().backward()
    assert torch.equal(layer.main_grad, torch.ones(128, 256))
