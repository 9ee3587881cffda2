"""Rings of bulk copies whose wait runs out with copies in flight: the call reports it, writes nothing outside its outputs, and
the next call is whole."""
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


def guarded(shape, dtype):
    n = torch.Size(shape).numel() * dtype.itemsize
    buf = torch.full((n + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    return buf[512:512 + n].view(dtype).view(shape), lambda: bool((buf[:512] == 0xA5).all()) and bool((buf[512 + n:] == 0xA5).all())


def run(call, whole, waits):
    """A call that gives up, where the shape has waits, and one that does not."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(3):
        assert Q.lib().selftest_norm_give_up(1) == Q.Q_OK
        try:
            call(status)
        finally:
            Q.lib().selftest_norm_give_up(0)
    assert status.item() == (Q.Q_ST_TIMEOUT if waits else 0)
    if not waits:
        assert whole()
    status.zero_()
    call(status)
    assert status.item() == 0 and whole()


def make(M, K, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)
    return new(M, K), new(M, K), new(K)


# (rows, their length, whether a ring takes them): wide and narrow rows, rows that begin anywhere, one warp's, and too few for a ring
@pytest.mark.parametrize("M,K,dtype,ring", [(6000, 4096, BF16, True), (3000, 8192, BF16, True), (1500, 14336, BF16, True), (6000, 1111, F32, True),
                                            (6000, 301, BF16, True), (1500, 10001, F32, True), (100, 4096, BF16, False), (6000, 4096, F32, False)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_add(M, K, dtype, ring, residual):
    x, r, w = make(M, K, dtype, 1)
    r = r if residual else None
    want = Q.norm_add(x, w, residual=r)
    (out, out_ok), (h, h_ok), top = guarded((M, K), dtype), guarded((M, K), dtype), torch.zeros(1, device="cuda")
    got = {}

    def call(status):
        got["y"] = Q.norm_add(x, w, residual=r, out=out, h_out=h if residual else None, amax=top, status=status)

    run(call, lambda: all(torch.equal(a, b) for a, b in zip(got["y"], want)) and torch.equal(top, Q.q_amax(want[0])), ring)
    assert out_ok() and h_ok()


@pytest.mark.parametrize("M,K,ring", [(6016, 4096, True), (3200, 8192, True), (1536, 14336, True), (128, 4096, False)])
@pytest.mark.parametrize("rowwise,colwise", [(True, False), (True, True), (False, True)])
def test_norm_q_blockwise(M, K, ring, rowwise, colwise):
    x, r, w = make(M, K, BF16, 2)
    want = Q.norm_q_blockwise(x, w, residual=r, rowwise=rowwise, colwise=colwise)
    got = {}

    def call(status):
        got["t"] = Q.norm_q_blockwise(x, w, residual=r, rowwise=rowwise, colwise=colwise, status=status)

    def whole():
        a, b = got["t"], want
        return all(torch.equal(u, v) for u, v in zip((a[0].q_row, a[0].s_row, a[0].q_colT, a[0].s_colT, a[1], a[2]),
                                                     (b[0].q_row, b[0].s_row, b[0].q_colT, b[0].s_colT, b[1], b[2])) if u is not None)

    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert Q.lib().selftest_norm_give_up(1) == Q.Q_OK
    try:
        call(status)
    finally:
        Q.lib().selftest_norm_give_up(0)
    assert bool(status.item() & Q.Q_ST_TIMEOUT) == ring   # a transposed copy of what was left may report what is not finite there
    status.zero_()
    call(status)
    assert status.item() == 0 and whole()


@pytest.mark.parametrize("M,K,dtype,ring", [(6000, 4096, BF16, True), (10, 4096, BF16, True), (6000, 100, F32, True), (6000, 1111, F32, True),
                                            (1500, 16384, BF16, True), (50, 40000, F32, False)])
@pytest.mark.parametrize("with_dh", [False, True])
def test_norm_grad(M, K, dtype, ring, with_dh):
    h, dy, w = make(M, K, dtype, 3)
    dh = make(M, K, dtype, 4)[0] if with_dh else None
    rstd = Q.norm_add(h, w)[2]
    want = Q.norm_grad(dy, h, rstd, w, dh)
    out, ok = guarded((M, K), dtype)
    got = {}

    def call(status):
        got["g"] = Q.norm_grad(dy, h, rstd, w, dh, out=out, status=status)

    run(call, lambda: all(torch.equal(a, b) for a, b in zip(got["g"], want)), ring)
    assert ok()
