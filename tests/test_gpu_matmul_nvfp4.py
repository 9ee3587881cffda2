"""The product of NVFP4 copies against the products of what they decode to, in 64 bits.

Where every product and every sum is a small multiple of a power of two, FP32 is exact in any order and the result has to
be equal.  Otherwise: products of codes and block scales are exact; the tensor core adds 64 of them to the sum in one
instruction, and a term that is aligned to the largest loses at most 2^-23 of it, so that K terms lose at most K 2^-23 of
the sum of magnitudes, a split's sums 8 roundings, and the two tensors' scales one each; + 2^-24 of the result when it is
added to C, 2^-8 of it for bfloat16.
"""
import numpy as np
import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu

Q = pytest.importorskip("nvfp4_quantization_current_gb300")

BF16, F32 = torch.bfloat16, torch.float32
VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Q.lib()


def operand(rows, K, blk, seed, lossless=False):
    """Every code, with scales over eight binades (lossless: scales of 1/2, 1, 3/2 and 2, and a tensor scale of 1/4)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0, 256, (rows, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    shape = (rows // 16 if blk == "16x16" else rows, K // 16)
    if lossless:
        s = torch.randint(1, 5, shape, generator=g, device="cuda") / 2
        return q, s.to(torch.float8_e4m3fn).view(torch.uint8), torch.full((1,), 0.25, device="cuda")
    s = torch.exp2(torch.rand(shape, generator=g, device="cuda") * 8 - 4)
    return q, s.to(torch.float8_e4m3fn).view(torch.uint8), torch.rand(1, generator=g, device="cuda") * 2 + 0.1


def wide(q, sb, blk):
    v = torch.tensor(VALUES + [-v for v in VALUES], device=q.device, dtype=torch.float64)
    x = torch.stack((v[(q & 15).long()], v[(q >> 4).long()]), 2).flatten(1)
    s = sb.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
    return x * (s.repeat_interleave(16, 0) if blk == "16x16" else s)


def reference(a, sba, sa, ba, b, sbb, sb, bb):
    x, y = wide(a, sba, ba), wide(b, sbb, bb)
    s = sa.double() * sb.double()
    return x @ y.T * s, x.abs() @ y.abs().T * s


def check(M, N, K, ba="1x16", bb="16x16", dtype=BF16, accumulate=False, seed=1, lossless=False):
    A, B = operand(M, K, ba, seed, lossless), operand(N, K, bb, seed + 1, lossless)
    ref, mags = reference(*A, ba, *B, bb)
    c = None
    if accumulate:
        c = torch.randint(-64, 65, (M, N), device="cuda").to(dtype) if lossless else torch.randn((M, N), device="cuda").to(dtype)
    nb = M * N * dtype.itemsize
    buf = torch.full((nb + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    out = buf[512:512 + nb].view(dtype).view(M, N)
    if accumulate:
        out.copy_(c)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = Q.matmul_nvfp4(*A, *B, ba, bb, out=out, accumulate=accumulate, status=status)
    assert got is out and status.item() == 0
    assert bool((buf[:512] == 0xA5).all()) and bool((buf[512 + nb:] == 0xA5).all()), "written outside C"
    if lossless:   # 3600 terms at most, each a multiple of 1/16 up to 144: sums of 23 bits, and as many with C
        assert K <= 3600
        assert torch.equal(out, (ref + (0 if c is None else c.double())).float().to(dtype)), (out.double() - ref).abs().max()
        return
    tol = (K * 2.0 ** -23 + 11 * 2.0 ** -24) * mags
    if c is not None:
        ref = ref + c.double()
        tol = tol + 2.0 ** -24 * (ref.abs() + tol)
    tol = tol + (2.0 ** -8 * (ref.abs() + tol) if dtype == BF16 else 0.0)
    err = (out.double() - ref).abs() - tol
    assert bool((err <= 0).all()), f"{int((err > 0).sum())} of {M * N} outside, worst {float((err + tol).max())} for {float(tol.max())}"


ROWS = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 200, 255, 256, 257, 333, 640]


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows(M, dtype):
    check(M, 384, 1280, dtype=dtype, seed=M, lossless=True)
    check(M, 384, 1280, dtype=dtype, seed=M)


@pytest.mark.parametrize("M,N", [(1, 1), (1, 61), (3, 130), (128, 1), (130, 257), (257, 130), (64, 1000), (300, 515), (513, 2)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_odd_columns(M, N, dtype):
    check(M, N, 512, "1x16", "1x16", dtype, seed=M + N, lossless=True)


# whole and broken blocks of 256, scale rows that are multiples of 16, 4 and 2 bytes
@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 192, 224, 256, 288, 320, 480, 512, 544, 768, 992, 1024, 1056, 1280, 1536, 1600, 2080, 2304,
                               3584])
@pytest.mark.parametrize("M", [1, 20, 129, 300])
def test_reduction_lengths(K, M):
    check(M, 256, K, dtype=F32, seed=K, lossless=True)
    check(M, 136, K, bb="1x16", dtype=F32, seed=K + 3, lossless=True)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (20, 1000, 14336), (300, 512, 18432), (600, 640, 7168)])
def test_long_reductions(M, N, K):
    check(M, N, K, bb="1x16", dtype=F32, seed=K)


@pytest.mark.parametrize("ba,bb", [("1x16", "16x16"), ("16x16", "1x16"), ("16x16", "16x16"), ("1x16", "1x16")])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("M,N", [(16, 128), (144, 400), (384, 256), (256, 1152)])
def test_blocks_and_accumulate(M, N, ba, bb, dtype, accumulate):
    check(M, N, 768, ba, bb, dtype, accumulate, lossless=True)
    check(M, N, 768, ba, bb, dtype, accumulate)


# widths of 16 to 192 tokens with splits of 1 to 8, tiles that end inside them, and more tiles than the machine has
@pytest.mark.parametrize("M,N,K,bb", [(1, 4096, 3584, "16x16"), (16, 14336, 512, "16x16"), (17, 2048, 2048, "16x16"), (40, 4096, 3584, "16x16"),
                                      (64, 18432, 896, "16x16"), (100, 1000, 3584, "1x16"), (128, 7168, 2304, "16x16"), (200, 4096, 3584, "16x16"),
                                      (333, 4096, 2048, "16x16"), (350, 4000, 1152, "1x16"), (513, 700, 3584, "1x16"), (1024, 1024, 2560, "1x16"),
                                      (5000, 5120, 256, "16x16"), (5000, 5120, 256, "1x16"), (2600, 5120, 512, "1x16"), (4999, 4991, 768, "1x16"),
                                      (2305, 4608, 1792, "16x16"), (4600, 2300, 2304, "1x16"), (1000, 5120, 1056, "16x16"), (8192, 1280, 160, "16x16"),
                                      (3000, 2999, 96, "1x16"), (4, 7168, 2048, "16x16"), (130, 18432, 256, "16x16")])
@pytest.mark.parametrize("dtype,accumulate", [(BF16, False), (F32, True), (BF16, True)])
def test_plans(M, N, K, bb, dtype, accumulate):
    check(M, N, K, "1x16", bb, dtype, accumulate, seed=M, lossless=True)


# results whose tiles of 256 x 256 are too few for the machine, and take tiles of 256 x 128: ends inside them, one and two
# rounds, broken blocks of K, block scales at any address, columns of either CTA missing
NARROW = [(333, 4096, 2048, "16x16"), (257, 2816, 1280, "1x16"), (300, 2784, 768, "16x16"), (1769, 640, 512, "16x16"), (161, 2224, 1024, "16x16"),
          (380, 2312, 1280, "1x16"), (242, 4520, 256, "1x16"), (500, 4040, 1184, "1x16"), (2000, 600, 3584, "1x16"), (1790, 840, 288, "1x16")]


@pytest.mark.parametrize("M,N,K,bb", NARROW)
@pytest.mark.parametrize("dtype,accumulate", [(BF16, False), (F32, False), (F32, True), (BF16, True)])
def test_narrow_tiles(M, N, K, bb, dtype, accumulate):
    check(M, N, K, "1x16", bb, dtype, accumulate, seed=M + K, lossless=True)
    check(M, N, K, "1x16", bb, dtype, accumulate, seed=M)


# rows of C of 32, 16, 8, 4 and 2 bytes' pitch, added to and overwritten by the pair kernel
@pytest.mark.parametrize("N", [2304, 2312, 2308, 2310, 2311])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_pitches(N, dtype, accumulate):
    check(2601, N, 512, "1x16", "1x16", dtype, accumulate, seed=N, lossless=True)
    check(2601, N, 512, "1x16", "1x16", dtype, accumulate, seed=N)


def test_random_shapes():
    rng = np.random.default_rng(5)
    for i in range(60):
        M, K = int(np.exp(rng.uniform(0, 7.6))), 32 * int(rng.integers(1, 112))
        bb = ["1x16", "16x16"][i % 2]
        N = 16 * int(rng.integers(1, 120)) if bb == "16x16" else int(np.exp(rng.uniform(0, 7.6)))
        check(M, N, K, "1x16", bb, [BF16, F32][int(rng.integers(2))], bool(rng.integers(2)), seed=i, lossless=True)


def test_scales_at_odd_addresses():
    """Block scales have no alignment rule."""
    for K in (512, 1088, 96):
        A, B = operand(70, K, "1x16", 3, True), operand(128, K, "16x16", 4, True)
        want = Q.matmul_nvfp4(*A, *B, dtype=F32)
        for shift in (1, 2, 4, 8):
            moved = []
            for q, sb, s in (A, B):
                room = torch.zeros(sb.numel() + 32, dtype=torch.uint8, device="cuda")
                room[shift:shift + sb.numel()] = sb.flatten()
                moved += [q, room[shift:shift + sb.numel()].view(sb.shape), s]
            assert torch.equal(Q.matmul_nvfp4(*moved, dtype=F32), want)


@pytest.mark.parametrize("M,N", [(5, 256), (200, 256), (600, 640), (2300, 1536)])
def test_nan_inf_and_zero_stay_in_their_rows(M, N):
    K = 768
    A, B = operand(M, K, "1x16", 11), operand(N, K, "16x16", 12)
    clean = Q.matmul_nvfp4(*A, *B, dtype=F32)
    A[1][1, 20] = 0x7F      # a NaN scale: row 1
    B[1][N // 32, 3] = 0x7F   # and 16 columns
    got = Q.matmul_nvfp4(*A, *B, dtype=F32)
    cols = slice(N // 32 * 16, N // 32 * 16 + 16)
    assert bool(got[1].isnan().all()) and bool(got[:, cols].isnan().all())
    keep_r = torch.ones(M, dtype=torch.bool, device="cuda")
    keep_r[1] = False
    keep_c = torch.ones(N, dtype=torch.bool, device="cuda")
    keep_c[cols] = False
    assert torch.equal(got[keep_r][:, keep_c], clean[keep_r][:, keep_c])
    A, B = operand(M, K, "1x16", 11), operand(N, K, "16x16", 12)
    zero = lambda t: (torch.zeros_like(t[0]), *t[1:])
    assert bool((Q.matmul_nvfp4(*zero(A), *zero(B), dtype=F32) == 0).all())
    for s in (float("inf"), float("nan")):
        assert not bool(Q.matmul_nvfp4(A[0], A[1], torch.full((1,), s, device="cuda"), *B, dtype=F32).isfinite().any())
    # tensor scales whose product FP32 does not hold: powers of two change no bit of a normal result
    far = Q.matmul_nvfp4(A[0], A[1], A[2] * 2.0 ** -70, B[0], B[1], B[2] * 2.0 ** -62, dtype=F32)
    large = clean.abs() >= 2.0 ** 7
    assert bool(large.any()) and torch.equal((far.double() * 2.0 ** 132)[large], clean.double()[large])


def test_empty():
    B = operand(128, 256, "16x16", 1)
    A = operand(5, 256, "1x16", 1)
    assert Q.matmul_nvfp4(A[0][:0], A[1][:0], A[2], *B).shape == (0, 128)
    c = torch.ones((5, 128), device="cuda")
    A0 = (A[0][:, :0].contiguous(), A[1][:, :0].contiguous(), A[2])
    B0 = (B[0][:, :0].contiguous(), B[1][:, :0].contiguous(), B[2])
    assert torch.equal(Q.matmul_nvfp4(*A0, *B0, out=c, accumulate=True), torch.ones_like(c))
    assert torch.equal(Q.matmul_nvfp4(*A0, *B0, out=c), torch.zeros_like(c))


@pytest.mark.parametrize("M", [1, 40, 300, 2048])
def test_same_result_every_time(M):
    A, B = operand(M, 4096, "1x16", 8), operand(1024, 4096, "16x16", 9)
    first = Q.matmul_nvfp4(*A, *B, dtype=F32)
    for _ in range(5):
        assert torch.equal(first, Q.matmul_nvfp4(*A, *B, dtype=F32))


def test_streams_and_graphs():
    A, B, big = operand(33, 2048, "1x16", 21), operand(2048, 2048, "16x16", 22), operand(3000, 2048, "1x16", 23)
    want, many = Q.matmul_nvfp4(*A, *B), Q.matmul_nvfp4(*big, *B)
    torch.cuda.synchronize()
    s0, s1 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        with torch.cuda.stream(s0):
            x = Q.matmul_nvfp4(*A, *B)
        with torch.cuda.stream(s1):
            y = Q.matmul_nvfp4(*big, *B)
        got.append((x, y))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) and torch.equal(y, many) for x, y in got)
    out, wide_out = torch.zeros_like(want), torch.zeros_like(many)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            Q.matmul_nvfp4(*A, *B, out=out)
            Q.matmul_nvfp4(*big, *B, out=wide_out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(wide_out, many)


def test_calls_in_a_row():
    """Calls that may overlap their neighbours' ends: sums of equal terms are exact, a copy is made of the last result."""
    A, B, big = operand(24, 512, "1x16", 81, True), operand(512, 512, "16x16", 82, True), operand(700, 512, "1x16", 83, True)
    c, d = torch.zeros((24, 512), device="cuda"), torch.zeros((700, 512), device="cuda")
    one, two = Q.matmul_nvfp4(*A, *B, dtype=F32), Q.matmul_nvfp4(*big, *B, dtype=F32)
    torch.cuda.synchronize()
    for i in range(32):
        Q.matmul_nvfp4(*A, *B, out=c, accumulate=True)
        Q.matmul_nvfp4(*big, *B, out=d, accumulate=True)
        x = Q.matmul_nvfp4(*A, *B)
        q = Q.q_nvfp4(torch.cat((x, x))[:32].contiguous())
        y = Q.matmul_nvfp4(q.q_row, q.sb_row, q.s_global, *B)
    assert torch.equal(c, one * 32) and torch.equal(d, two * 32)
    torch.cuda.synchronize()
    q = Q.q_nvfp4(torch.cat((x, x))[:32].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(y, Q.matmul_nvfp4(q.q_row, q.sb_row, q.s_global, *B))


def test_output_past_32_bit_offsets():
    M, N = 40064, 57344 + 128   # 2.3e9 elements
    A, B = operand(M, 128, "1x16", 3, True), operand(N, 128, "16x16", 4, True)
    c = Q.matmul_nvfp4(*A, *B)
    for rows in (slice(0, 3), slice(20000, 20002), slice(M - 3, M)):
        ref, _ = reference(A[0][rows], A[1][rows], A[2], "1x16", *B, "16x16")
        assert torch.equal(c[rows], ref.float().to(BF16))


@pytest.mark.parametrize("kind", ["normal", "t3"])
def test_product_of_quantized_tensors(kind):
    """End to end from the recipe's copies: forward, input gradient and weight gradient are the products of what they decode to."""
    dev = lambda a: torch.from_numpy(a.view(np.int16).copy()).view(BF16).cuda()
    x, w, dy = dev(W.gen(kind, (256, 512), 31)), dev(W.gen("weight", (384, 512), 32)), dev(W.gen("grad", (256, 384), 33))
    wq = Q.q_nvfp4(w, "16x16", colwise=True)
    xr, xc = Q.q_nvfp4_recipe(x, 0xB4E1)
    dr, dc = Q.q_nvfp4_recipe(dy, 0xB4E1, "sr", seed=3)
    row, col = (lambda t: (t.q_row, t.sb_row, t.s_global)), (lambda t: (t.q_colT, t.sb_colT, t.s_global))
    for a, b, bb in ((row(xr), row(wq), "16x16"), (row(dr), col(wq), "16x16"), (col(dc), col(xc), "1x16")):
        got = Q.matmul_nvfp4(*a, *b, blk_b=bb, dtype=F32)
        ref, mags = reference(*a, "1x16", *b, bb)
        K = a[0].shape[1] * 2
        assert bool(((got.double() - ref).abs() <= (K * 2.0 ** -23 + 11 * 2.0 ** -24) * mags).all())
    # what they decode to is near the tensors: a code is off by at most half of its gap, a third of its value
    y = Q.matmul_nvfp4(*row(xr), *row(wq), dtype=F32)
    rel = float((y.double() - x.double() @ w.double().T).norm() / (x.double() @ w.double().T).norm())
    assert rel < 0.3


def test_a_wait_that_runs_out_leaves_c_as_it_is():
    L = Q.lib()
    for M, N, K in ((1, 512, 2048), (20, 4096, 1024), (100, 1000, 4096), (333, 4096, 4096), (2500, 4096, 512), (64, 128, 256)):
        A, B = operand(M, K, "1x16", 5), operand(N, K, "1x16", 6)
        want = Q.matmul_nvfp4(*A, *B, blk_b="1x16", dtype=F32)
        c = torch.full_like(want, 7.0)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert L.selftest_mm_give_up(1) == Q.Q_OK
        Q.matmul_nvfp4(*A, *B, blk_b="1x16", out=c, status=status)
        assert status.item() == Q.Q_ST_TIMEOUT and bool((c == 7.0).all())
        status.zero_()
        Q.matmul_nvfp4(*A, *B, blk_b="1x16", out=c, status=status)
        assert status.item() == 0 and torch.equal(c, want)
