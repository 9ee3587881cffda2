"""The norm's entry points refuse bad arguments on the host, before any CUDA call, in the C ABI and in the
Python binding (no GPU needed)."""
import ctypes

import pytest
import torch

import nvfp4_quantization_current_gb300 as Q
from test_abi import A, MIS, status_of
from test_operators_abi import B2, L, fake  # noqa: F401 (L is a fixture)

C = ctypes.c_void_p(0x20000)
NORMS = ["norm_add", "norm_q_blockwise", "norm_grad"]


def add_args(x=A, dt=Q.Q_BF16, M=4, K=256, r=A, w=A, wt=Q.Q_F32, eps=1e-6, h=A, y=C, s=A, amax=None):
    return x, dt, M, K, r, w, wt, eps, h, y, s, amax, None, None


def cast_args(x=A, dt=Q.Q_BF16, M=128, K=256, r=A, w=A, wt=Q.Q_F32, eps=1e-6, h=A, s=A, q=A, sr=A, qc=A, sc=A):
    return x, dt, M, K, r, w, wt, eps, h, s, q, sr, qc, sc, None, None


def grad_args(dy=A, dt=Q.Q_F32, M=4, K=250, h=A, s=A, w=A, wt=Q.Q_F32, dh=A, dx=A, dw=A, work=A):
    return dy, dt, M, K, h, s, w, wt, dh, dx, dw, work, None, None


ARGS = {"norm_add": add_args, "norm_q_blockwise": cast_args, "norm_grad": grad_args}
FORWARD = [(dict(eps=-1.0), Q.Q_ERR_ARG, "eps"), (dict(eps=float("nan")), Q.Q_ERR_ARG, "eps"), (dict(eps=float("inf")), Q.Q_ERR_ARG, "eps"),
           (dict(x=None), Q.Q_ERR_ARG, "x is NULL"), (dict(x=MIS), Q.Q_ERR_ALIGN, "x is"), (dict(r=MIS), Q.Q_ERR_ALIGN, "residual"),
           (dict(h=None), Q.Q_ERR_ARG, "h is NULL"), (dict(h=MIS), Q.Q_ERR_ALIGN, "h is"), (dict(r=None), Q.Q_ERR_ARG, "without a residual"),
           (dict(s=None), Q.Q_ERR_ARG, "rstd"), (dict(s=B2), Q.Q_ERR_ALIGN, "rstd")]
EVERY = [(dict(M=-1), Q.Q_ERR_SHAPE, "negative"), (dict(M=1 << 31), Q.Q_ERR_SHAPE, "M = "), (dict(K=0), Q.Q_ERR_SHAPE, "K = 0"),
         (dict(K=1 << 31), Q.Q_ERR_SHAPE, "K = "), (dict(dt=2), Q.Q_ERR_DTYPE, "input dtype"), (dict(wt=2), Q.Q_ERR_DTYPE, "weight dtype"),
         (dict(w=None), Q.Q_ERR_ARG, "weight is NULL"), (dict(w=MIS), Q.Q_ERR_ALIGN, "weight")]
CASES = [(n, *c) for n in NORMS for c in EVERY] + [(n, *c) for n in NORMS[:2] for c in FORWARD] + [
    ("norm_add", dict(y=None), Q.Q_ERR_ARG, "y is NULL"), ("norm_add", dict(y=MIS), Q.Q_ERR_ALIGN, "y is"),
    ("norm_add", dict(y=A), Q.Q_ERR_ARG, "same buffer"), ("norm_add", dict(amax=B2), Q.Q_ERR_ALIGN, "amax"),
    ("norm_q_blockwise", dict(K=192), Q.Q_ERR_SHAPE, "K = 192"), ("norm_q_blockwise", dict(M=100), Q.Q_ERR_SHAPE, "q_colT"),
    ("norm_q_blockwise", dict(q=None, qc=None), Q.Q_ERR_ARG, "neither"), ("norm_q_blockwise", dict(sr=None), Q.Q_ERR_ARG, "s_row"),
    ("norm_q_blockwise", dict(q=MIS), Q.Q_ERR_ALIGN, "q_row"), ("norm_q_blockwise", dict(qc=MIS), Q.Q_ERR_ALIGN, "q_colT"),
    ("norm_q_blockwise", dict(sc=B2), Q.Q_ERR_ALIGN, "s_colT"),
    ("norm_grad", dict(dy=None), Q.Q_ERR_ARG, "dy"), ("norm_grad", dict(h=MIS), Q.Q_ERR_ALIGN, "h is"), ("norm_grad", dict(s=None), Q.Q_ERR_ARG, "rstd"),
    ("norm_grad", dict(dh=MIS), Q.Q_ERR_ALIGN, "dh"), ("norm_grad", dict(dx=None), Q.Q_ERR_ARG, "dx"), ("norm_grad", dict(work=None), Q.Q_ERR_ARG, "work"),
    ("norm_grad", dict(work=MIS), Q.Q_ERR_ALIGN, "work"), ("norm_grad", dict(dw=B2), Q.Q_ERR_ALIGN, "dw")]


@pytest.mark.parametrize("name,change,status,text", CASES)
def test_refusals(L, name, change, status, text):
    st, msg = status_of(L, name, *ARGS[name](**change))
    assert st == status and text in msg and name in msg


def test_injected_launch_failure_and_empty_calls(L):
    try:
        for name in NORMS:
            assert name in Q.__all__ and callable(getattr(Q, name))
            assert L.q_selftest_inject_launch_error(1) == Q.Q_OK
            st, msg = status_of(L, name, *ARGS[name]())
            assert st == Q.Q_ERR_CUDA and name in msg and "cudaErrorLaunchFailure" in msg
    finally:
        L.q_selftest_inject_launch_error(0)
    assert status_of(L, "norm_add", *add_args(M=0, x=None, r=None, w=None, h=None, y=None, s=None))[0] == Q.Q_OK
    assert status_of(L, "norm_q_blockwise", *cast_args(M=0, x=None, r=None, w=None, h=None, s=None, q=None, qc=None))[0] == Q.Q_OK
    assert status_of(L, "norm_grad", *grad_args(M=0, dy=None, h=None, s=None, w=None, dx=None, dw=None, work=None))[0] == Q.Q_OK


@pytest.mark.parametrize("dt", [Q.Q_BF16, Q.Q_F32])
def test_scratch_sizes(L, dt):
    """Whole rows of K floats, at least one, and bounded whatever M is."""
    for K in (1, 7, 64, 1111, 4096, 8192, 16384, 50000):
        sizes = [L.norm_grad_work(M, K, dt) for M in (1, 2, 100, 5000, 1 << 20, (1 << 31) - 1)]
        assert all(n > 0 and n % K == 0 for n in sizes) and sizes == sorted(sizes)
        assert sizes[-1] == sizes[-2] <= max(608 * 8 * K, 1 << 24)
    assert L.norm_grad_work(0, 4, dt) == L.norm_grad_work(4, 0, dt) == L.norm_grad_work(4, 4, 7) == 0


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(Q, "_call", lambda name, *args: made.append(name))
    monkeypatch.setattr(Q, "_stream", lambda dev: None)
    return made


def test_binding_refusals(calls):
    bf, f32 = torch.bfloat16, torch.float32
    x, w, s = fake((4, 256), bf), fake((256,), f32), fake((4,), f32)
    with pytest.raises(ValueError, match="CUDA"):
        Q.norm_add(torch.zeros(4, 256), w)
    for bad in (fake((4, 256), torch.float16), fake((256, 4), bf).t(), fake((), bf)):
        with pytest.raises(ValueError, match="x must be"):
            Q.norm_add(bad, w)
    for bad in (fake((255,), f32), fake((1, 256), f32), fake((256,), torch.float16), torch.zeros(256, device="meta"), fake((512,), f32)[::2]):
        with pytest.raises(ValueError, match="weight must"):
            Q.norm_add(x, bad)
    for r in (fake((4, 128), bf), fake((4, 256), f32)):
        with pytest.raises(ValueError, match="residual must"):
            Q.norm_add(x, w, residual=r)
    with pytest.raises(ValueError, match="h_out without"):
        Q.norm_add(x, w, h_out=x)
    for kw, text in ((dict(out=fake((4, 255), bf)), "out must"), (dict(residual=x, h_out=fake((4, 256), f32)), "h_out must"),
                     (dict(amax=fake((2,), f32)), "amax must"), (dict(amax=fake((1,), bf)), "amax must"), (dict(status=fake((1,), f32)), "status must")):
        with pytest.raises(ValueError, match=text):
            Q.norm_add(x, w, **kw)
    with pytest.raises(ValueError, match="2-D"):
        Q.norm_q_blockwise(fake((2, 4, 256), bf), w)
    with pytest.raises(ValueError, match="out.q_row"):
        Q.norm_q_blockwise(x, w, out=Q.BlockwiseTensor(fake((4, 128), torch.uint8), fake((4, 2), f32), None, None, Q.Q_T1x128))
    with pytest.raises(ValueError, match="h_out without"):
        Q.norm_q_blockwise(x, w, h_out=x)
    for kw, text in ((dict(h=fake((4, 255), bf)), "h must"), (dict(rstd=fake((5,), f32)), "rstd must"), (dict(dh=fake((4, 256), f32)), "dh must"),
                     (dict(out=fake((3, 256), bf)), "out must"), (dict(status=s), "status must")):
        with pytest.raises(ValueError, match=text):
            Q.norm_grad(**{**dict(dy=x, h=x, rstd=s, weight=w), **kw})
    assert calls == []


def test_gradients_are_not_lost(calls):
    bf, f32 = torch.bfloat16, torch.float32
    x, w, s = fake((4, 256), bf), fake((256,), f32), fake((4,), f32)
    grad = lambda t: t.detach().clone().requires_grad_()
    for args in (dict(x=grad(x), weight=w), dict(x=x, weight=grad(w)), dict(x=x, weight=w, residual=grad(x))):
        with pytest.raises(RuntimeError, match="gradient"):
            Q.norm_q_blockwise(**args)
        with pytest.raises(RuntimeError, match="gradient"):
            Q.norm_add(**args, out=x)
    for kw in (dict(dy=grad(x)), dict(h=grad(x)), dict(dh=grad(x)), dict(weight=grad(w)), dict(rstd=grad(s))):
        with pytest.raises(RuntimeError, match="gradient"):
            Q.norm_grad(**{**dict(dy=x, h=x, rstd=s, weight=w), **kw})
    assert calls == []
    with torch.no_grad():
        Q.norm_add(grad(x), w, out=fake((4, 256), bf))
    assert calls == ["norm_add"]


def test_writing_counts_as_a_new_version(calls):
    bf, f32 = torch.bfloat16, torch.float32
    x, r, w, s, top = fake((128, 256), bf), fake((128, 256), bf), fake((256,), f32), fake((128,), f32), fake((1,), f32)

    def versions(f, *tensors):
        before = [t._version for t in tensors]
        f()
        return [t._version > v for t, v in zip(tensors, before)]

    assert versions(lambda: Q.norm_add(x, w, residual=r, out=x, h_out=r, amax=top), x, r, top, w) == [True, True, True, False]
    assert versions(lambda: Q.norm_grad(x, r, s, w, out=x), x, r, s) == [True, False, False]
    t = Q.alloc_blockwise(128, 256, "cpu", "1x128", True, True)
    t = Q.BlockwiseTensor(*(fake(v.shape, v.dtype) for v in (t.q_row, t.s_row, t.q_colT, t.s_colT)), t.tile)
    assert versions(lambda: Q.norm_q_blockwise(x, w, residual=r, out=t, h_out=r), t.q_row, t.s_row, t.q_colT, t.s_colT, r, x) == [True] * 5 + [False]
