"""Types of C that the products do not know are refused with an error that says so (no GPU needed)."""
import pytest
import torch

import nvfp4_quantization_current_gb300 as Q
from test_operators_abi import fake

U8, F32 = torch.uint8, torch.float32


def test_unknown_types(monkeypatch):
    monkeypatch.setattr(Q, "_call", lambda name, *args: pytest.fail(name))
    f4 = fake((16, 64), U8), fake((16, 8), U8), fake((1,), F32)
    f8 = fake((128, 128), U8), fake((128, 1), F32)
    for dtype in (torch.float16, torch.int32, None):
        with pytest.raises(ValueError, match="bfloat16 or float32"):
            Q.matmul_nvfp4(*f4, *f4, blk_b="1x16", dtype=dtype)
        with pytest.raises(ValueError, match="bfloat16 or float32"):
            Q.mm_blockwise(*f8, *f8, tile_b="1x128", dtype=dtype)
    with pytest.raises(ValueError, match="out must"):
        Q.matmul_nvfp4(*f4, *f4, blk_b="1x16", out=fake((16, 16), torch.float16))
    with pytest.raises(ValueError, match="out must"):
        Q.mm_blockwise(*f8, *f8, tile_b="1x128", out=fake((128, 128), torch.float16))
