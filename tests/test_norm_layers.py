"""What the layers on the norm and the NVFP4 product refuse and draw, on the CPU."""
import pytest
import torch

import nvfp4_quantization_current_gb300.linear as linear


def test_layers_refuse_what_their_kernels_do():
    for a, b in ((40, 32), (32, 40)):
        with pytest.raises(ValueError, match="multiples of 32"):
            linear.NVFP4Linear(a, b, device="cpu")
    for mask in (-1, 1 << 16):
        with pytest.raises(ValueError, match="16 bits"):
            linear.NVFP4Linear(32, 32, sign_mask=mask, device="cpu")
    with pytest.raises(ValueError, match="multiples of 128"):
        linear.NormBlockwiseLinear(200, 128, device="cpu")
    for eps in (0.0, -1.0, float("nan")):
        with pytest.raises(ValueError, match="positive"):
            linear.NormBlockwiseLinear(128, 128, eps=eps, device="cpu")


def test_parameters_and_seeds():
    torch.manual_seed(3)
    a, b = (linear.NVFP4Linear(64, 32, device="cpu") for _ in range(2))
    assert a.seed != b.seed and a.weight.shape == (32, 64) and [n for n, _ in a.named_parameters()] == ["weight"]
    torch.manual_seed(3)
    assert linear.NVFP4Linear(64, 32, device="cpu").seed == a.seed
    c = linear.NormBlockwiseLinear(128, 256, device="cpu")
    assert sorted(n for n, _ in c.named_parameters()) == ["norm_weight", "weight"] and c.norm_weight.shape == (128,)
    assert [n for n, _ in linear.RMSNorm(7, device="cpu").named_parameters()] == ["weight"]


def test_rows_are_padded_with_zeros():
    x = torch.ones(5, 3)
    assert linear._rows_to(x, 5) is x
    y = linear._rows_to(x, 4)
    assert y.shape == (8, 3) and bool((y[5:] == 0).all()) and bool((y[:5] == 1).all())
    assert linear._rows_to(x[:0], 16).shape == (0, 3)
