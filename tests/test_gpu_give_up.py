"""Products whose warp that issues the MMAs, or whose loads in one CTA of a pair, give up while operands are on their way into shared memory: their copies land
before that memory is put to other use, C stays as it is, and the next call is whole."""
import pytest
import torch

import nvfp4_quantization_current_gb300 as Q
from test_gpu_matmul_nvfp4 import operand as operand4
from test_gpu_operators import operand as operand8

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Q.lib()


def gives_up(call, out, times, how=2):
    """`times` calls that give up leave C as it is; one that does not writes what it should, the same every time."""
    fresh = out.clone()
    call(fresh, None)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = out.clone()
    for _ in range(times):
        assert Q.lib().selftest_mm_give_up(how) == Q.Q_OK
        try:
            call(out, status)
        finally:
            Q.lib().selftest_mm_give_up(0)
    assert status.item() == Q.Q_ST_TIMEOUT and torch.equal(out, before)
    status.zero_()
    call(out, status)
    assert status.item() == 0 and torch.equal(out, fresh)


# every width with splits of 1 to 8, few blocks for a CTA (all of them issued before anything is waited for) and many
SPLIT4 = [(1, 512, 256), (1, 512, 2048), (1, 4096, 4096), (16, 1024, 18432), (20, 4096, 1024), (20, 512, 8192), (64, 512, 4096), (60, 4096, 14336),
          (100, 1000, 4096), (128, 128, 2048), (190, 256, 8192), (190, 1024, 768)]


@pytest.mark.parametrize("M,N,K", SPLIT4)
@pytest.mark.parametrize("dtype,accumulate", [(BF16, False), (F32, True)])
def test_nvfp4_few_tokens(M, N, K, dtype, accumulate):
    a, b = operand4(M, K, "1x16", 1), operand4(N, K, "1x16", 2)
    c = torch.randn((M, N), device="cuda").to(dtype)
    gives_up(lambda out, status: Q.matmul_nvfp4(*a, *b, blk_b="1x16", out=out, accumulate=accumulate, status=status), c, 5)


SPLIT8 = [(1, 14336, 512), (1, 128, 128), (1, 128, 2048), (1, 4096, 4096), (20, 4096, 1024), (20, 2048, 2048), (40, 7168, 4096), (190, 1024, 8192), (300, 512, 8192)]


@pytest.mark.parametrize("M,N,K", SPLIT8)
@pytest.mark.parametrize("tile_b", ["128x128", "1x128"])
@pytest.mark.parametrize("dtype,accumulate", [(BF16, False), (F32, True)])
def test_blockwise_few_tokens(M, N, K, tile_b, dtype, accumulate):
    a, b = operand8(M, K, "1x128", 1), operand8(N, K, tile_b, 2)
    c = torch.randn((M, N), device="cuda").to(dtype)
    gives_up(lambda out, status: Q.mm_blockwise(*a, *b, tile_b=tile_b, out=out, accumulate=accumulate, status=status), c, 5)


# the CTA pairs' kernels: tiles of 256 and of 128 columns, C of any pitch and added to, fewer blocks than stages and more
@pytest.mark.parametrize("how", [2, 3, 4])
@pytest.mark.parametrize("M,N,K,dtype,accumulate", [(2560, 4096, 512, BF16, False), (333, 4096, 4096, BF16, False), (333, 4096, 4096, F32, False),
                                                    (2560, 2048, 2560, F32, True), (2500, 2047, 1024, BF16, True)])
def test_nvfp4_pairs(M, N, K, dtype, accumulate, how):
    a, b = operand4(M, K, "1x16", 1), operand4(N, K, "1x16", 2)
    c = torch.randn((M, N), device="cuda").to(dtype)
    gives_up(lambda out, status: Q.matmul_nvfp4(*a, *b, blk_b="1x16", out=out, accumulate=accumulate, status=status), c, 1, how)


@pytest.mark.parametrize("how", [2, 3, 4])
@pytest.mark.parametrize("M,N,K,tile_b,dtype,accumulate", [(2600, 2048, 256, "128x128", BF16, False), (2600, 2048, 2048, "1x128", F32, True)])
def test_blockwise_pairs(M, N, K, tile_b, dtype, accumulate, how):
    a, b = operand8(M, K, "1x128", 1), operand8(N, K, tile_b, 2)
    c = torch.randn((M, N), device="cuda").to(dtype)
    gives_up(lambda out, status: Q.mm_blockwise(*a, *b, tile_b=tile_b, out=out, accumulate=accumulate, status=status), c, 1, how)
