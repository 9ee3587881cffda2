"""Block and tile names and types that the products do not know are refused with an error that says so (no GPU needed)."""
import pytest
import torch

import nvfp4_quantization_current_gb300 as Q
from test_operators_abi import fake

U8, F32 = torch.uint8, torch.float32


def test_unknown_names_and_types(monkeypatch):
    monkeypatch.setattr(Q, "_call", lambda name, *args: pytest.fail(name))
    f4 = fake((16, 64), U8), fake((16, 8), U8), fake((1,), F32)
    f8 = fake((128, 128), U8), fake((128, 1), F32)
    for bad in ("1x32", None, 7):
        for kw in (dict(blk_a=bad), dict(blk_b=bad)):
            with pytest.raises(ValueError, match="1x16 or 16x16"):
                Q.matmul_nvfp4(*f4, *f4, **kw)
        for kw in (dict(tile_a=bad), dict(tile_b=bad)):
            with pytest.raises(ValueError, match="1x128 or 128x128"):
                Q.mm_blockwise(*f8, *f8, **kw)
    for dtype in (torch.float16, torch.int32, None):
        with pytest.raises(ValueError, match="bfloat16 or float32"):
            Q.matmul_nvfp4(*f4, *f4, blk_b="1x16", dtype=dtype)
        with pytest.raises(ValueError, match="bfloat16 or float32"):
            Q.mm_blockwise(*f8, *f8, tile_b="1x128", dtype=dtype)
    with pytest.raises(ValueError, match="out must"):
        Q.matmul_nvfp4(*f4, *f4, blk_b="1x16", out=fake((16, 16), torch.float16))
    with pytest.raises(ValueError, match="out must"):
        Q.mm_blockwise(*f8, *f8, tile_b="1x128", out=fake((128, 128), torch.float16))
