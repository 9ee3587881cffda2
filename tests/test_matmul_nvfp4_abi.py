"""The NVFP4 product refuses bad arguments on the host, before any CUDA call, in the C ABI and in the Python
binding (no GPU needed)."""
import pytest
import torch

import nvfp4_quantization_current_gb300 as Q
from test_abi import A, MIS, status_of
from test_operators_abi import B2, L, fake  # noqa: F401 (L is a fixture)

U8, F32 = torch.uint8, torch.float32


def args(a=A, sb_a=MIS, s_a=A, ba=Q.Q_B1x16, b=A, sb_b=MIS, s_b=A, bb=Q.Q_B16x16, M=4, N=128, K=96, c=A, out=Q.Q_BF16, acc=0):
    return a, sb_a, s_a, ba, b, sb_b, s_b, bb, M, N, K, c, out, acc, None, None


@pytest.mark.parametrize("change,status,text", [
    (dict(M=-1), Q.Q_ERR_SHAPE, "negative"), (dict(N=1 << 31), Q.Q_ERR_SHAPE, "2^31"), (dict(K=1 << 40), Q.Q_ERR_SHAPE, "2^31"),
    (dict(K=48), Q.Q_ERR_SHAPE, "K = 48"), (dict(N=130), Q.Q_ERR_SHAPE, "N (16x16"), (dict(ba=1), Q.Q_ERR_SHAPE, "M (16x16"),
    (dict(ba=2), Q.Q_ERR_ARG, "blk"), (dict(bb=-1), Q.Q_ERR_ARG, "blk"), (dict(out=2), Q.Q_ERR_DTYPE, "output dtype"),
    (dict(a=None), Q.Q_ERR_ARG, "a is NULL"), (dict(sb_a=None), Q.Q_ERR_ARG, "sb_a is NULL"), (dict(s_a=None), Q.Q_ERR_ARG, "s_a is NULL"),
    (dict(b=None), Q.Q_ERR_ARG, "b is NULL"), (dict(sb_b=None), Q.Q_ERR_ARG, "sb_b is NULL"), (dict(s_b=None), Q.Q_ERR_ARG, "s_b is NULL"),
    (dict(c=None), Q.Q_ERR_ARG, "c is NULL"), (dict(a=MIS), Q.Q_ERR_ALIGN, "a is"), (dict(b=MIS), Q.Q_ERR_ALIGN, "b is"),
    (dict(c=MIS), Q.Q_ERR_ALIGN, "c is"), (dict(s_a=B2), Q.Q_ERR_ALIGN, "s_a"), (dict(s_b=B2), Q.Q_ERR_ALIGN, "s_b"),
    (dict(K=0, c=None), Q.Q_ERR_ARG, "c is NULL"),
])
def test_refusals(L, change, status, text):
    st, msg = status_of(L, "matmul_nvfp4", *args(**change))
    assert st == status and text in msg and "matmul_nvfp4" in msg


def test_empty_calls_and_injected_failures(L):
    assert "matmul_nvfp4" in Q.__all__
    assert status_of(L, "matmul_nvfp4", *args(M=0, a=None, sb_a=None, s_a=None, c=None))[0] == Q.Q_OK
    assert status_of(L, "matmul_nvfp4", *args(N=0, b=None, sb_b=None, s_b=None, c=None))[0] == Q.Q_OK
    assert status_of(L, "matmul_nvfp4", *args(K=0, a=None, b=None, acc=1))[0] == Q.Q_OK
    try:
        assert L.selftest_mm_give_up(1) == Q.Q_OK   # for the next call that launches
        assert status_of(L, "matmul_nvfp4", *args(K=48))[0] == Q.Q_ERR_SHAPE
        assert L.q_selftest_inject_launch_error(1) == Q.Q_OK
        st, msg = status_of(L, "matmul_nvfp4", *args())
        assert st == Q.Q_ERR_CUDA and "matmul_nvfp4" in msg and "cudaErrorLaunchFailure" in msg
    finally:
        L.q_selftest_inject_launch_error(0)
        L.selftest_mm_give_up(0)


def operands():
    return [fake((4, 48), U8), fake((4, 6), U8), fake((1,), F32), fake((128, 48), U8), fake((8, 6), U8), fake((1,), F32)]


def test_binding_refusals(monkeypatch):
    calls = []
    monkeypatch.setattr(Q, "_call", lambda name, *args: calls.append(name))
    monkeypatch.setattr(Q, "_stream", lambda dev: None)
    meta = lambda t: torch.empty(t.shape, dtype=t.dtype, device="meta").as_subclass(type(t))

    def refused(text, i=None, t=None, error=ValueError, **kw):
        ops = operands()
        if i is not None:
            ops[i] = t if t is not None else meta(ops[i])
        with pytest.raises(error, match=text):
            Q.matmul_nvfp4(*ops, **kw)
        assert calls == []

    refused("CUDA", 0, torch.zeros(4, 48, dtype=U8))
    for i in (1, 2, 3, 4, 5):
        refused("one device", i)
    refused("uint8", 0, fake((4, 48), F32))
    refused("uint8", 1, fake((4, 6), F32))
    refused("float32", 5, fake((1,), torch.float64))
    refused("contiguous", 0, fake((48, 4), U8).t())
    refused("contiguous", 4, fake((6, 8), U8).t())
    refused("block scales are", 1, fake((4, 5), U8))
    refused("block scales are", 2, fake((2,), F32))
    refused("block scales are", blk_b="1x16")
    refused("block scales are", blk_a="16x16")
    refused("accumulate needs out", accumulate=True)
    for out in (fake((4, 129), F32), fake((4, 128), torch.float16), fake((128, 4), F32).t()):
        refused("out must", out=out)
    refused("status must", status=fake((1,), F32))
    refused("32x32", blk_b="32x32", error=KeyError)
    ops = operands()
    ops[3], ops[4] = fake((128, 64), U8), fake((8, 8), U8)
    with pytest.raises(ValueError, match="K = 96, b has K = 128"):
        Q.matmul_nvfp4(*ops)
    for i in (2, 5):
        refused("gradient", i, fake((1,), F32).requires_grad_(), error=RuntimeError)
    refused("gradient", out=fake((4, 128), F32).requires_grad_(), error=RuntimeError)
    out = fake((4, 128), F32)
    before = out._version
    assert Q.matmul_nvfp4(*operands(), out=out, accumulate=True) is out and out._version > before and calls == ["matmul_nvfp4"]


def test_another_device_is_made_current(monkeypatch):
    """A launch goes to the current device: tensors on another one make theirs current for the call."""
    seen = []
    monkeypatch.setattr(Q, "_call", lambda name, *a: seen.append((name, current[-1])))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    current = [0]

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            current.append(self.dev.index)

        def __exit__(self, *_):
            current.pop()

    monkeypatch.setattr(torch.cuda, "device", Device)
    Q._call_on(torch.device("cuda", 0), "one")
    Q._call_on(torch.device("cuda", 3), "two")
    assert seen == [("one", 0), ("two", 3)] and current == [0]
