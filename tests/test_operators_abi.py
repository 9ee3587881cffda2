"""The operators on the blockwise copies refuse bad arguments on the host, before any CUDA call, in
the C ABI and in the Python binding (no GPU needed)."""
import ctypes
import re

import pytest
import torch

import nvfp4_quantization_current_gb300 as Q
from nvfp4_quantization_current_gb300 import build as B
from test_abi import A, HEADER, MIS, status_of

OPERATORS = ["mm_blockwise", "drop_add", "drop_q_blockwise"]
B2 = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def L():
    B.build()
    return Q.lib()


def test_declared_exported_and_public(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^q_status ((?:mm|drop)_\w+)\s*\(", text, flags=re.M))
    assert names == set(OPERATORS)
    for n in OPERATORS:
        assert hasattr(L, n) and n in Q.SIGNATURES and n in Q.__all__ and callable(getattr(Q, n))


def mm_args(a=A, s_a=A, ta=Q.Q_T1x128, b=A, s_b=A, tb=Q.Q_T128x128, M=4, N=128, K=256, c=A, out=Q.Q_BF16, acc=0):
    return a, s_a, ta, b, s_b, tb, M, N, K, c, out, acc, None, None


@pytest.mark.parametrize("change,status,text", [
    (dict(M=-1), Q.Q_ERR_SHAPE, "negative"), (dict(N=1 << 31), Q.Q_ERR_SHAPE, "2^31"), (dict(K=1 << 40), Q.Q_ERR_SHAPE, "2^31"),
    (dict(K=192), Q.Q_ERR_SHAPE, "K = 192"), (dict(N=130), Q.Q_ERR_SHAPE, "N (128x128"), (dict(ta=1), Q.Q_ERR_SHAPE, "M (128x128"),
    (dict(ta=2), Q.Q_ERR_ARG, "tile"), (dict(tb=-1), Q.Q_ERR_ARG, "tile"), (dict(out=2), Q.Q_ERR_DTYPE, "output dtype"),
    (dict(a=None), Q.Q_ERR_ARG, "a is NULL"), (dict(s_a=None), Q.Q_ERR_ARG, "s_a is NULL"), (dict(b=None), Q.Q_ERR_ARG, "b is NULL"),
    (dict(s_b=None), Q.Q_ERR_ARG, "s_b is NULL"), (dict(c=None), Q.Q_ERR_ARG, "c is NULL"), (dict(a=MIS), Q.Q_ERR_ALIGN, "a is"),
    (dict(b=MIS), Q.Q_ERR_ALIGN, "b is"), (dict(c=MIS), Q.Q_ERR_ALIGN, "c is"), (dict(s_a=B2), Q.Q_ERR_ALIGN, "s_a"),
    (dict(s_b=B2), Q.Q_ERR_ALIGN, "s_b"), (dict(K=0, c=None), Q.Q_ERR_ARG, "c is NULL"),
])
def test_mm_refusals(L, change, status, text):
    st, msg = status_of(L, "mm_blockwise", *mm_args(**change))
    assert st == status and text in msg and "mm_blockwise" in msg


def test_empty_calls_need_no_buffers(L):
    assert status_of(L, "mm_blockwise", *mm_args(M=0, a=None, s_a=None, c=None))[0] == Q.Q_OK
    assert status_of(L, "mm_blockwise", *mm_args(N=0, b=None, s_b=None, c=None))[0] == Q.Q_OK
    assert status_of(L, "mm_blockwise", *mm_args(K=0, a=None, b=None, acc=1))[0] == Q.Q_OK
    assert status_of(L, "drop_add", None, Q.Q_BF16, 0, None, 0.5, 0, 0, None, None)[0] == Q.Q_OK
    assert status_of(L, "drop_q_blockwise", None, Q.Q_BF16, 0, 128, 0.5, 0, 0, None, None, None, None, None, None)[0] == Q.Q_OK


def test_dropout_refusals(L):
    add = lambda x=A, dt=Q.Q_BF16, n=64, r=None, p=0.5, y=A: status_of(L, "drop_add", x, dt, n, r, p, 0, 0, y, None)
    for got, status, text in ((add(n=-1), Q.Q_ERR_SHAPE, "negative"), (add(dt=2), Q.Q_ERR_DTYPE, "dtype"), (add(x=None), Q.Q_ERR_ARG, "x is NULL"),
                              (add(y=None), Q.Q_ERR_ARG, "y is NULL"), (add(x=MIS), Q.Q_ERR_ALIGN, "x is"), (add(r=MIS), Q.Q_ERR_ALIGN, "residual"),
                              (add(y=MIS), Q.Q_ERR_ALIGN, "y is"), (add(p=-0.1), Q.Q_ERR_ARG, "outside [0, 1]"), (add(p=1.1), Q.Q_ERR_ARG, "outside"),
                              (add(p=float("nan")), Q.Q_ERR_ARG, "outside")):
        assert got[0] == status and text in got[1] and "drop_add" in got[1]
    cast = lambda x=A, M=128, K=128, p=0.5, q=A, s=A, qc=A, sc=A: status_of(L, "drop_q_blockwise", x, Q.Q_BF16, M, K, p, 0, 0, q, s, qc, sc, None, None)
    for got, status, text in ((cast(K=192), Q.Q_ERR_SHAPE, "K = 192"), (cast(M=100), Q.Q_ERR_SHAPE, "q_colT"), (cast(p=2.0), Q.Q_ERR_ARG, "outside"),
                              (cast(q=None, qc=None), Q.Q_ERR_ARG, "neither"), (cast(s=None), Q.Q_ERR_ARG, "s_row"), (cast(sc=B2), Q.Q_ERR_ALIGN, "s_colT"),
                              (cast(x=None), Q.Q_ERR_ARG, "x is NULL"), (cast(M=-1), Q.Q_ERR_SHAPE, "negative"), (cast(qc=MIS), Q.Q_ERR_ALIGN, "q_colT")):
        assert got[0] == status and text in got[1] and "drop_q_blockwise" in got[1]


def test_injected_launch_failure(L):
    calls = {"mm_blockwise": mm_args(), "drop_add": (A, Q.Q_F32, 64, A, 0.5, 1, 2, A, None),
             "drop_q_blockwise": (A, Q.Q_BF16, 128, 128, 0.5, 1, 2, A, A, A, A, None, None)}
    assert sorted(calls) == sorted(OPERATORS)
    try:
        for name, args in calls.items():
            assert L.q_selftest_inject_launch_error(1) == Q.Q_OK
            st, msg = status_of(L, name, *args)
            assert st == Q.Q_ERR_CUDA and name in msg and "cudaErrorLaunchFailure" in msg
    finally:
        L.q_selftest_inject_launch_error(0)


class _Cuda(torch.Tensor):
    """A CPU tensor that says it is a CUDA one, to reach the checks behind that question."""
    is_cuda = True


def fake(shape, dtype):
    return torch.zeros(shape, dtype=dtype).as_subclass(_Cuda)


def test_binding_refusals():
    u8, f32 = torch.uint8, torch.float32
    q, s, w, t = fake((4, 256), u8), fake((4, 2), f32), fake((128, 256), u8), fake((1, 2), f32)
    with pytest.raises(ValueError, match="CUDA"):
        Q.mm_blockwise(torch.zeros(4, 256, dtype=u8), torch.zeros(4, 2), w, t)
    with pytest.raises(ValueError, match="uint8"):
        Q.mm_blockwise(fake((4, 256), f32), s, w, t)
    with pytest.raises(ValueError, match="scales are"):
        Q.mm_blockwise(q, fake((4, 3), f32), w, t)
    with pytest.raises(ValueError, match="scales are"):
        Q.mm_blockwise(q, s, w, t, tile_b="1x128")
    with pytest.raises(ValueError, match="contiguous"):
        Q.mm_blockwise(fake((256, 4), u8).t(), s, w, t)
    with pytest.raises(ValueError, match="K = 256"):
        Q.mm_blockwise(q, s, fake((128, 384), u8), fake((1, 3), f32))
    with pytest.raises(ValueError, match="accumulate needs out"):
        Q.mm_blockwise(q, s, w, t, accumulate=True)
    with pytest.raises(ValueError, match="out must be"):
        Q.mm_blockwise(q, s, w, t, out=fake((4, 129), f32))
    with pytest.raises(KeyError):
        Q.mm_blockwise(q, s, w, t, tile_b="64x64")
    x = fake((4, 128), torch.bfloat16)
    with pytest.raises(ValueError, match="contiguous CUDA"):
        Q.drop_add(torch.zeros(4), 0.1, 0)
    with pytest.raises(ValueError, match="contiguous CUDA"):
        Q.drop_add(fake((4, 128), torch.float16), 0.1, 0)
    with pytest.raises(ValueError, match="residual must"):
        Q.drop_add(x, 0.1, 0, residual=fake((4, 127), torch.bfloat16))
    with pytest.raises(ValueError, match="out must"):
        Q.drop_add(x, 0.1, 0, out=fake((4, 128), f32))
    with pytest.raises(ValueError, match="CUDA"):
        Q.drop_q_blockwise(torch.zeros(128, 128), 0.1, 0)


def test_layer_refuses_odd_features():
    from nvfp4_quantization_current_gb300.linear import BlockwiseLinear
    with pytest.raises(ValueError, match="multiples of 128"):
        BlockwiseLinear(200, 128, device="cpu")
