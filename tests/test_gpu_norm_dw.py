"""The weight's gradient of the norm with no row lost: factors of one and small whole numbers, whose products and sums are exact
in FP32 in any order (below 2^24), so that dw has to be equal."""
import pytest
import torch

pytestmark = pytest.mark.gpu

Q = pytest.importorskip("nvfp4_quantization_current_gb300")

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Q.lib()


# single rows, fewer rows than CTAs, one more than they share evenly, and rings that wrap many times; rows of every layout
SIZES = [(1, 1), (1, 4096), (2, 257), (151, 1111), (305, 7168), (609, 512), (3001, 100), (3001, 1111), (3001, 4096), (8192, 256), (8192, 264), (8192, 4096),
         (8191, 4097), (4865, 2048), (20000, 7), (20000, 300), (20000, 1000), (20000, 2304), (2433, 8200), (1217, 14336), (1500, 16384), (400, 18432), (307, 40001)]


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("dtype,wt", [(BF16, F32), (F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("with_dh", [False, True])
def test_every_row_counts_once(M, K, dtype, wt, with_dh):
    g = torch.Generator("cuda").manual_seed(M + K)
    new = lambda: torch.randint(-4, 5, (M, K), generator=g, device="cuda").to(dtype)   # 20000 products of at most 16: below 2^24
    h, dy = new(), new()
    h[h == 0], dy[dy == 0] = 3, -1   # no row goes by unseen
    w = torch.randn(K, generator=g, device="cuda").to(wt)
    dw = Q.norm_grad(dy, h, torch.ones(M, device="cuda"), w, new() if with_dh else None)[1]
    assert torch.equal(dw, (dy.double() * h.double()).sum(0).to(F32).to(wt))
