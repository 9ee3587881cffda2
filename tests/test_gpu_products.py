"""mm_blockwise where it can go wrong beside its sums: waits that run out, and the kernel of many
tiles in all its forms.  Operands, references and tolerances are those of test_gpu_operators."""
import pytest
import torch

import nvfp4_quantization_current_gb300 as Q
from test_gpu_operators import mm_bound, mm_reference, operand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Q.lib()


def check(a, sa, ta, b, sb, tb, got, c=None):
    ref, tol = mm_bound(*mm_reference(a, sa, ta, b, sb, tb), a.shape[1] // 128, got.dtype, c)
    assert bool(((got.double() - ref).abs() <= tol).all())


# every width, splits of 1 to 8, and the kernel of many tiles with one and with several tiles for a CTA
@pytest.mark.parametrize("M,N,K,tb", [(1, 14336, 512, "128x128"), (1, 128, 512, "128x128"), (1, 128, 1024, "128x128"),
                                      (1, 128, 2048, "128x128"), (20, 4096, 1024, "128x128"), (20, 2048, 2048, "128x128"),
                                      (40, 14336, 2048, "128x128"), (40, 7168, 4096, "128x128"), (190, 1024, 8192, "128x128"),
                                      (300, 4096, 1024, "1x128"), (640, 512, 4096, "128x128"), (300, 512, 8192, "128x128"),
                                      (300, 4096, 2048, "1x128"), (640, 1024, 2048, "1x128"),
                                      (2600, 2048, 1024, "128x128"), (4999, 4991, 384, "1x128")])
@pytest.mark.parametrize("dtype,accumulate", [(torch.bfloat16, False), (torch.float32, True), (torch.bfloat16, True)])
def test_a_wait_that_runs_out_leaves_c_as_it_is(M, N, K, tb, dtype, accumulate):
    """One CTA of each cluster gives up: the others' sums have no use, and what lies in its shared memory is no sum."""
    a, sa = operand(M, K, "1x128", 1)
    b, sb = operand(N, K, tb, 2)
    c = torch.randn((M, N), device="cuda").to(dtype)
    out, status = c.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    assert Q.lib().selftest_mm_give_up(1) == Q.Q_OK
    try:
        Q.mm_blockwise(a, sa, b, sb, tile_b=tb, out=out, accumulate=accumulate, status=status)
    finally:
        Q.lib().selftest_mm_give_up(0)
    assert status.item() == Q.Q_ST_TIMEOUT
    assert torch.equal(out, c)
    status.zero_()
    Q.mm_blockwise(a, sa, b, sb, tile_b=tb, out=out, accumulate=accumulate, status=status)   # the next call is whole
    assert status.item() == 0
    check(a, sa, "1x128", b, sb, tb, out, c if accumulate else None)


@pytest.mark.parametrize("bits", [0xFFD5A5A5 - (1 << 32), 0x7FFFFFFF, 0x7F800001])
@pytest.mark.parametrize("K", [512, 2048])
def test_nan_scales_of_any_payload_reach_c(K, bits):
    """A NaN that is computed with is a result like another, whatever bits it came from."""
    a, sa = operand(5, K, "1x128", 1)
    b, sb = operand(256, K, "128x128", 2)
    clean = Q.mm_blockwise(a, sa, b, sb, dtype=torch.float32)
    sa.view(torch.int32)[2] = bits
    got = Q.mm_blockwise(a, sa, b, sb, dtype=torch.float32)
    rest = [0, 1, 3, 4]
    assert bool(got[2].isnan().all()) and torch.equal(got[rest], clean[rest])
    sb.view(torch.int32)[1] = bits
    got = Q.mm_blockwise(a, sa, b, sb, dtype=torch.float32)
    assert bool(got[:, 128:].isnan().all()) and torch.equal(got[rest][:, :128], clean[rest][:, :128])


# ---------------------------------------------------------------------------
# the kernel of many tiles (results of about 2000 x 2000 and more)
# ---------------------------------------------------------------------------

def product(M, N, K, ta, tb, dtype, accumulate, seed):
    a, sa = operand(M, K, ta, seed)
    b, sb = operand(N, K, tb, seed + 1)
    c = torch.randn((M, N), device="cuda").to(dtype) if accumulate else torch.full((M, N), torch.nan, device="cuda", dtype=dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = Q.mm_blockwise(a, sa, b, sb, ta, tb, out=c.clone(), accumulate=accumulate, status=status)
    assert status.item() == 0
    check(a, sa, ta, b, sb, tb, got, c if accumulate else None)


@pytest.mark.parametrize("ta,tb", [("1x128", "128x128"), ("128x128", "1x128"), ("128x128", "128x128"), ("1x128", "1x128")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("M,N,K", [(2560, 2048, 1024), (5120, 5120, 384)])
def test_many_tiles_in_every_form(M, N, K, ta, tb, dtype, accumulate):
    product(M, N, K, ta, tb, dtype, accumulate, 5)


# results that end inside a tile, with rows that a bulk store can take and rows that it cannot, and one block of K
@pytest.mark.parametrize("M,N,K,tb", [(3000, 3000, 256, "1x128"), (2600, 2500, 640, "1x128"), (2300, 3002, 512, "1x128"),
                                      (4999, 4991, 384, "1x128"), (4999, 5120, 128, "128x128"), (2305, 2561, 512, "1x128")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_many_tiles_of_odd_sizes(M, N, K, tb, dtype, accumulate):
    product(M, N, K, "1x128", tb, dtype, accumulate, M)


def test_many_tiles_in_a_row():
    """Calls that may begin before the one ahead has ended, each reading or adding to what that one wrote, against the same
    calls one at a time."""
    x0 = torch.randn((2560, 2048), generator=torch.Generator("cuda").manual_seed(1), device="cuda", dtype=torch.bfloat16)
    b, sb = operand(2048, 2048, "128x128", 2)
    sb /= 4096

    def chain(sync):
        x, c, outs = x0, torch.zeros((2560, 2048), device="cuda"), []
        for i in range(12):
            q = Q.q_blockwise(x, colwise=True)
            sync()
            y = Q.mm_blockwise(q.q_row, q.s_row, b, sb)
            sync()
            z = Q.mm_blockwise(q.q_row, q.s_row, b, sb, dtype=torch.float32)   # no kernel of another kind in between
            sync()
            for _ in range(2):
                Q.mm_blockwise(q.q_row, q.s_row, b, sb, out=c, accumulate=True)
                sync()
            d = Q.drop_q_blockwise(z, 0.25, i, colwise=True)
            sync()
            w = Q.mm_blockwise(d.q_colT, d.s_colT, q.q_colT, q.s_colT, tile_b="1x128", dtype=torch.float32)
            sync()
            few = Q.mm_blockwise(q.q_row[:16], q.s_row[:16], b, sb)
            sync()
            x = Q.drop_add(y, 0.25, i, residual=x)
            sync()
            outs += [y, z, w, few]
        torch.cuda.synchronize()
        return outs + [x, c]

    for a, r in zip(chain(lambda: None), chain(torch.cuda.synchronize)):
        assert bool(r.isfinite().all()) and torch.equal(a, r)


def test_many_tiles_in_a_graph_and_on_a_side_stream():
    a, sa = operand(2560, 1024, "1x128", 21)
    b, sb = operand(2048, 1024, "128x128", 22)
    want = Q.mm_blockwise(a, sa, b, sb, dtype=torch.float32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = Q.mm_blockwise(a, sa, b, sb, dtype=torch.float32)
    side.synchronize()
    assert torch.equal(got, want)
    out, total = torch.zeros_like(want), torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Q.mm_blockwise(a, sa, b, sb, out=out)
        Q.mm_blockwise(a, sa, b, sb, out=total, accumulate=True)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(total, want + want)
