"""A row's norm is the same bits whatever call it is part of: few rows or many, stored or cast, with the residual's
addition or with the sum given, in rows of every layout."""
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


def make(M, K, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)
    return new(M, K), new(M, K), new(K)


# more rows than any ring's CTAs begin with; lengths that are no power of two among them, and rows that begin anywhere
@pytest.mark.parametrize("M,K", [(6000, 128), (6000, 250), (6000, 264), (6000, 301), (6000, 511), (6000, 513), (6000, 1111), (6000, 2304), (6000, 2056),
                                 (6000, 3333), (6000, 4096), (6000, 5001), (6000, 5120), (6000, 7168), (3000, 8191), (3000, 8192), (3000, 9001),
                                 (3000, 10240), (3000, 14336), (1500, 16383), (1500, 16384), (700, 18432), (300, 40001)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_do_not_depend_on_their_call(M, K, dtype):
    x, r, w = make(M, K, dtype, K)
    y, h, rstd = Q.norm_add(x, w, residual=r)
    for n in (1, 3, 77, 300, 1200):
        got = Q.norm_add(x[:n], w, residual=r[:n])
        assert all(torch.equal(a, b[:n]) for a, b in zip(got, (y, h, rstd))), n
    alone = Q.norm_add(h, w)   # the sum given
    assert torch.equal(alone[0], y) and torch.equal(alone[2], rstd)
    assert torch.equal(Q.norm_add(h[:5], w)[2], rstd[:5])


@pytest.mark.parametrize("M,K", [(6016, 256), (6016, 2304), (6016, 5120), (6016, 7168), (3200, 14336), (384, 18432)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_casts_do_not_depend_on_their_call(M, K, dtype):
    x, r, w = make(M, K, dtype, K)
    rstd = Q.norm_add(x, w, residual=r)[2]
    t, h, s = Q.norm_q_blockwise(x, w, residual=r, colwise=True)
    assert torch.equal(s, rstd)
    for n in (1, 77, 333):
        u, k, v = Q.norm_q_blockwise(x[:n], w, residual=r[:n])
        assert torch.equal(v, s[:n]) and torch.equal(k, h[:n]) and torch.equal(u.q_row, t.q_row[:n]) and torch.equal(u.s_row, t.s_row[:n])
    u, _, v = Q.norm_q_blockwise(x[:256], w, residual=r[:256], rowwise=False, colwise=True)
    assert torch.equal(v, s[:256]) and torch.equal(u.q_colT, t.q_colT[:, :256]) and torch.equal(u.s_colT, t.s_colT[:, :2])
    assert torch.equal(Q.norm_q_blockwise(h[:9], w)[2], s[:9])


@pytest.mark.parametrize("M,K", [(6000, 250), (6000, 1111), (6000, 5120), (6000, 7168), (3000, 9001), (700, 18432)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("with_dh", [False, True])
def test_a_rows_gradient_does_not_depend_on_its_call(M, K, dtype, with_dh):
    h, dy, w = make(M, K, dtype, K)
    dh = make(M, K, dtype, 1)[0] if with_dh else None
    rstd = Q.norm_add(h, w)[2]
    dx = Q.norm_grad(dy, h, rstd, w, dh)[0]
    for n in (1, 77, 1200):
        assert torch.equal(Q.norm_grad(dy[:n], h[:n], rstd[:n], w, None if dh is None else dh[:n])[0], dx[:n]), n
