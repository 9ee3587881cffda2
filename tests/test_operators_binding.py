"""What the Python binding of the operators on the blockwise copies lets through to the library, on
the CPU: tensors that say they are CUDA ones, and a library call that only notes its arguments."""
import ctypes
import dataclasses

import pytest
import torch

import nvfp4_quantization_current_gb300 as Q
from test_operators_abi import L, fake, mm_args, status_of  # noqa: F401 (L is a fixture)

U8, F32, BF16 = torch.uint8, torch.float32, torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    """The names of the library calls that were made."""
    made = []
    monkeypatch.setattr(Q, "_call", lambda name, *args: made.append(name))
    monkeypatch.setattr(Q, "_stream", lambda dev: None)
    return made


def copies(M, K, tile=Q.Q_T1x128, rowwise=True, colwise=True, **change):
    t = Q.alloc_blockwise(M, K, "cpu", tile, rowwise, colwise)
    t = Q.BlockwiseTensor(*(v if v is None else fake(v.shape, v.dtype) for v in (t.q_row, t.s_row, t.q_colT, t.s_colT)), t.tile)
    return dataclasses.replace(t, **change)


def test_drop_q_blockwise_writes_only_to_copies_of_its_input(calls):
    """Scales of 128x128 tiles are 128 times too few, copies of a smaller tensor end before the kernel's last write."""
    x = fake((256, 384), BF16)
    for out, text in ((copies(256, 384, Q.Q_T128x128), "1x128"), (copies(128, 384), "q_row"), (copies(256, 256), "q_row"),
                      (copies(384, 256), "q_row"), (copies(256, 384, s_row=fake((256, 2), F32)), "s_row"),
                      (copies(256, 384, q_row=fake((256, 384), F32)), "q_row"), (copies(256, 384, s_row=fake((256, 3), BF16)), "s_row"),
                      (copies(256, 384, q_colT=fake((256, 384), U8).t()), "q_colT"), (copies(256, 384, q_colT=fake((256, 384), U8)), "q_colT"),
                      (copies(256, 384, s_colT=fake((384, 1), F32)), "s_colT"),
                      (copies(256, 384, s_colT=torch.empty((384, 2), device="meta")), "s_colT")):
        with pytest.raises(ValueError, match=text):
            Q.drop_q_blockwise(x, 0.1, 0, out=out)
    with pytest.raises(ValueError, match="transposed"):   # asked for, and nowhere to write it
        Q.drop_q_blockwise(x, 0.1, 0, colwise=True, out=copies(256, 384, colwise=False))
    assert calls == []
    for out in (copies(256, 384), copies(256, 384, colwise=False), copies(256, 384, rowwise=False)):   # its directions are written
        assert Q.drop_q_blockwise(x, 0.1, 0, out=out) is out
    assert calls == ["drop_q_blockwise"] * 3


def test_mm_blockwise_wants_its_operands_on_one_device(calls):
    a, s_a, b, s_b = fake((4, 256), U8), fake((4, 2), F32), fake((128, 256), U8), fake((1, 2), F32)
    off = lambda t: torch.empty(t.shape, dtype=t.dtype, device="meta").as_subclass(type(a))
    for args, text in (((a, off(s_a), b, s_b), "a: scales"), ((a, s_a, b, off(s_b)), "b: scales"), ((a, s_a, off(b), off(s_b)), "a is on")):
        with pytest.raises(ValueError, match=text):
            Q.mm_blockwise(*args)
    assert calls == []
    Q.mm_blockwise(a, s_a, b, s_b)
    assert calls == ["mm_blockwise"]


def test_status_is_an_int32_on_the_device(calls):
    """The kernels OR into it: a word of another type or place would be overwritten."""
    a, s_a, b, s_b, x = fake((4, 256), U8), fake((4, 2), F32), fake((128, 256), U8), fake((1, 2), F32), fake((128, 128), BF16)
    for call in (lambda status: Q.mm_blockwise(a, s_a, b, s_b, status=status), lambda status: Q.drop_q_blockwise(x, 0.1, 0, status=status)):
        for status in (fake((1,), U8), fake((1,), torch.int64), fake((0,), torch.int32), torch.zeros(1, dtype=torch.int32, device="meta")):
            with pytest.raises(ValueError, match="status"):
                call(status)
        assert calls == []
        call(fake((1,), torch.int32))
        call(None)
        assert len(calls) == 2
        calls.clear()


def test_give_up_is_for_one_call_and_clears(L):
    """The diagnostic is taken by the next call that launches, and not by one that is refused or empty."""
    try:
        assert L.selftest_mm_give_up(1) == Q.Q_OK
        assert status_of(L, "mm_blockwise", *mm_args(M=0, a=None, s_a=None, c=None))[0] == Q.Q_OK
        assert status_of(L, "mm_blockwise", *mm_args(K=192))[0] == Q.Q_ERR_SHAPE
        assert L.q_selftest_inject_launch_error(1) == Q.Q_OK   # taken here, where nothing is launched after all
        assert status_of(L, "mm_blockwise", *mm_args())[0] == Q.Q_ERR_CUDA
    finally:
        L.q_selftest_inject_launch_error(0)
        L.selftest_mm_give_up(0)


def grad(t):
    return t.requires_grad_()


def test_drop_add_into_a_given_tensor_records_no_gradient_and_says_so(calls):
    """Written to out, the result has no graph: where a gradient is wanted that is refused, as torch does."""
    new = lambda: fake((4, 128), F32)
    for kw in (dict(x=grad(new()), out=new()), dict(x=new(), residual=grad(new()), out=new()), dict(x=new(), out=grad(new()))):
        with pytest.raises(RuntimeError, match="gradient"):
            Q.drop_add(p=0.1, seed=0, **kw)
        assert calls == []
        with torch.no_grad():
            assert Q.drop_add(p=0.1, seed=0, **kw) is kw["out"]
        assert calls.pop() == "drop_add"


def test_drop_add_has_a_gradient(monkeypatch):
    """The library's call is linear in x and the residual, and its backward pass is the same call on the gradient."""
    made, values = [], {}

    def call(name, x, dt, n, residual, p, seed, offset, y, stream):
        made.append((name, p, seed, offset, residual is not None))
        t = lambda a: torch.frombuffer((ctypes.c_float * n).from_address(a), dtype=F32)
        t(y).copy_(t(x) * 3 + (t(residual) if residual else 0))

    monkeypatch.setattr(Q, "_call", call)
    monkeypatch.setattr(Q, "_stream", lambda dev: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))   # autograd hands plain tensors on
    x, r = (torch.randn(4, 24, requires_grad=True) for _ in range(2))
    g = torch.randn(24, 4).t()   # a gradient that is not contiguous
    y = Q.drop_add(x, 0.25, 7, 9, residual=r)
    assert torch.equal(y, x * 3 + r)
    dx, dr = torch.autograd.grad(y, (x, r), g, create_graph=True)
    assert torch.equal(dx, g * 3) and torch.equal(dr, g)
    assert made == [("drop_add", 0.25, 7, 9, True), ("drop_add", 0.25, 7, 9, False)]
    (z,) = torch.autograd.grad(Q.drop_add(r.detach(), 0.25, 7, residual=r), (r,), g)   # the residual's alone: no call
    assert torch.equal(z, g) and len(made) == 3
    w = x * 2
    (second,) = torch.autograd.grad((torch.autograd.grad(Q.drop_add(w, 0.25, 7) ** 2, w, g, create_graph=True)[0]).sum(), x)
    assert torch.allclose(second, 36 * g)   # y = 3 w with w = 2 x: the sum of 18 w g, by x


def test_mm_blockwise_has_no_gradient_and_says_so(calls):
    a, s_a, b, s_b = fake((4, 256), U8), fake((4, 2), F32), fake((128, 256), U8), fake((1, 2), F32)
    for args, out in (((a, grad(s_a.clone()), b, s_b), None), ((a, s_a, b, grad(s_b.clone())), None), ((a, s_a, b, s_b), grad(fake((4, 128), F32)))):
        with pytest.raises(RuntimeError, match="gradient"):
            Q.mm_blockwise(*args, out=out)
        assert calls == []
        with torch.no_grad():
            Q.mm_blockwise(*args, out=out)
        assert calls.pop() == "mm_blockwise"


def test_writing_into_a_tensor_counts_as_a_new_version(calls):
    """What autograd saved and finds overwritten raises there; results that are written in place have to count."""
    a, s_a, b, s_b, c = fake((4, 256), U8), fake((4, 2), F32), fake((128, 256), U8), fake((1, 2), F32), fake((4, 128), F32)
    x, r = fake((128, 128), F32), fake((128, 128), F32)

    def versions(f, *tensors):
        before = [t._version for t in tensors]
        f()
        return [t._version > v for t, v in zip(tensors, before)]

    assert versions(lambda: Q.mm_blockwise(a, s_a, b, s_b, out=c, accumulate=True), c, a, s_a, b, s_b) == [True] + [False] * 4
    assert versions(lambda: Q.drop_add(x, 0.1, 0, residual=r, out=r), r, x) == [True, False]
    assert versions(lambda: Q.drop_add(x, 0.1, 0, residual=r, out=x), r, x) == [False, True]
    t = copies(128, 128)
    assert versions(lambda: Q.drop_q_blockwise(x, 0.1, 0, out=t), t.q_row, t.s_row, t.q_colT, t.s_colT, x) == [True] * 4 + [False]
    t = copies(128, 128, colwise=False)
    assert versions(lambda: Q.drop_q_blockwise(x, 0.1, 0, out=t), t.q_row, t.s_row) == [True] * 2
    w = torch.randn(128, 128, requires_grad=True)
    y = (w * 2).as_subclass(type(x))
    z = y.square()
    with torch.no_grad():
        Q.drop_add(y.detach(), 0.1, 0, out=y.detach())   # shares y's counter
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.sum().backward()


def test_casting_into_copies_counts_as_a_new_version(calls):
    """The linear layer saves the weight's copies for its backward pass: casting another weight into them has to be seen."""
    for tile in (Q.Q_T1x128, Q.Q_T128x128):
        t = copies(128, 128, tile)
        before = [c._version for c in (t.q_row, t.s_row, t.q_colT, t.s_colT)]
        Q.q_blockwise(fake((128, 128), F32), out=t)
        assert [c._version > v for c, v in zip((t.q_row, t.s_row, t.q_colT, t.s_colT), before)] == [True] * 4
