"""Forward-mode derivatives are refused, not dropped: with everything frozen no gradient is asked for, and a tangent would be
lost (no GPU needed)."""
import pytest
import torch
from torch.autograd import forward_ad

import nvfp4_quantization_current_gb300 as Q
import nvfp4_quantization_current_gb300.linear as linear
from test_operators_abi import L  # noqa: F401 (a fixture)

F32 = torch.float32
new = lambda *s: torch.randn(s)


@pytest.fixture(autouse=True)
def calls(L, monkeypatch):
    made = []
    monkeypatch.setattr(Q, "_call", lambda name, *args: made.append(name))
    monkeypatch.setattr(Q, "_stream", lambda dev: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    return made


def frozen(m):
    return m.requires_grad_(False)


def layers():
    kw = dict(device="cpu", dtype=F32)
    norm, first, fp4, plain = linear.RMSNorm(128, **kw), linear.NormBlockwiseLinear(128, 128, **kw), linear.NVFP4Linear(128, 128, **kw), \
        linear.BlockwiseLinear(128, 128, **kw)
    return dict(RMSNorm=frozen(norm), NormBlockwiseLinear=frozen(first), NVFP4Linear=lambda x: frozen(fp4)(x, offset=0), BlockwiseLinear=frozen(plain))


w = torch.ones(128)
one, codes, scales = torch.ones(1), torch.zeros(32, 64, dtype=torch.uint8), torch.zeros(32, 8, dtype=torch.uint8)
CALLS = {
    "norm_add": lambda d: Q.norm_add(d, w),
    "norm_add, weight": lambda d: Q.norm_add(new(32, 128), d[0]),
    "norm_add, residual": lambda d: Q.norm_add(new(32, 128), w, residual=d),
    "norm_add, out": lambda d: Q.norm_add(d, w, out=new(32, 128)),
    "norm_add, h_out": lambda d: Q.norm_add(new(32, 128), w, residual=new(32, 128), h_out=d),
    "norm_q_blockwise": lambda d: Q.norm_q_blockwise(d, w),
    "norm_grad": lambda d: Q.norm_grad(new(32, 128), d, torch.ones(32), w),
    "norm_grad, dh": lambda d: Q.norm_grad(new(32, 128), new(32, 128), torch.ones(32), w, dh=d),
    "drop_add": lambda d: Q.drop_add(d, 0.1, 0),
    "drop_add, residual": lambda d: Q.drop_add(new(32, 128), 0.1, 0, residual=d),
    "matmul_nvfp4": lambda d: Q.matmul_nvfp4(codes, scales, d[0, :1].clone(), codes, scales, one, blk_b="1x16"),
    "mm_blockwise": lambda d: Q.mm_blockwise(torch.zeros(32, 128, dtype=torch.uint8), d[:, :1].clone(), torch.zeros(128, 128, dtype=torch.uint8), torch.ones(1, 1)),
}


@pytest.mark.parametrize("name", list(CALLS) + list(layers()))
def test_a_tangent_is_refused(name, calls):
    f = CALLS.get(name) or layers()[name]
    with forward_ad.dual_level():
        d = forward_ad.make_dual(new(32, 128), new(32, 128))
        for mode in (torch.enable_grad, torch.no_grad):   # no_grad leaves forward mode on
            with mode(), pytest.raises((RuntimeError, NotImplementedError)):
                f(d)
        f(new(32, 128))   # a level alone changes nothing
    calls.clear()
    f(new(32, 128))
    assert calls
