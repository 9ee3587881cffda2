"""The operators on the blockwise copies against plain implementations in 64 bits: the block-scaled
product, dropout with the residual sum, the dropout cast, and the linear layer made of them.

Tolerances.  mm_blockwise: the products of E4M3 codes are exact in FP32, so an element's error is that
of FP32 sums of its terms t_k = s_a s_b a_k b_k.  Summing the 128 terms of a block loses at most 128
truncations of 2^-23 of the sum of magnitudes, the two scales and the sum over KB blocks at most
KB + 3 roundings of 2^-24: (2^-16 + (KB + 3) 2^-24) sum |t_k|, one rounding of 2^-24 of the result
more when it is added to C, and 2^-8 of the result for BF16.  The dropouts are compared bit for bit:
their steps are single IEEE operations that extended precision reproduces.
"""
import numpy as np
import pytest
import torch

import oracle as O
import workloads as W

pytestmark = pytest.mark.gpu

Q = pytest.importorskip("nvfp4_quantization_current_gb300")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Q.lib()


def dev(x):
    if x.dtype == np.uint16:
        return torch.from_numpy(x.view(np.int16).copy()).view(torch.bfloat16).cuda()
    return torch.from_numpy(x.copy()).cuda()


def host(t):
    if t.dtype == torch.bfloat16:
        return t.view(torch.int16).cpu().numpy().view(np.uint16)
    return t.cpu().numpy()


def same(a, b, what=""):
    a, b = np.asarray(a), np.asarray(b)
    assert a.shape == b.shape, (what, a.shape, b.shape)
    if a.dtype == np.float32:
        a, b = a.view(np.uint32), b.view(np.uint32)
    bad = np.argwhere(a != b)
    assert bad.size == 0, f"{what}: {len(bad)} differ, first at {bad[:3].tolist()}: {a[tuple(bad[0])]} for {b[tuple(bad[0])]}"


# ---------------------------------------------------------------------------
# mm_blockwise
# ---------------------------------------------------------------------------

def operand(rows, K, tile, seed, spread=True):
    """Codes over the whole E4M3 range but its NaNs, scales over six binades."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0, 256, (rows, K), generator=g, device="cuda", dtype=torch.uint8)
    q = torch.where((q & 0x7F) == 0x7F, 0, q)
    s = torch.exp2(torch.rand((rows // 128 if tile == "128x128" else rows, K // 128), generator=g, device="cuda") * 6 - 12)
    return q, s


def wide(q, s, tile):
    s = s.double().repeat_interleave(128, 1)
    if tile == "128x128":
        s = s.repeat_interleave(128, 0)
    return q.view(torch.float8_e4m3fn).double() * s


def mm_reference(a, sa, ta, b, sb, tb):
    x, y = wide(a, sa, ta), wide(b, sb, tb)
    return x @ y.T, x.abs() @ y.abs().T


def mm_bound(ref, mags, KB, dtype, c=None):
    tol = (2.0 ** -16 + (KB + 3) * 2.0 ** -24) * mags
    if c is not None:
        ref = ref + c.double()
        tol = tol + 2.0 ** -24 * (ref.abs() + tol)
    return ref, tol + (2.0 ** -8 * (ref.abs() + tol) if dtype == torch.bfloat16 else 0.0)


def check_mm(M, N, K, ta, tb, dtype, accumulate=False, seed=1):
    a, sa = operand(M, K, ta, seed)
    b, sb = operand(N, K, tb, seed + 1)
    c = torch.randn((M, N), device="cuda").to(dtype) if accumulate else None
    ref, tol = mm_bound(*mm_reference(a, sa, ta, b, sb, tb), K // 128, dtype, c)
    buf = torch.full((M * N * 4 + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    nb = M * N * (2 if dtype == torch.bfloat16 else 4)
    out = buf[512:512 + nb].view(dtype).view(M, N)
    if accumulate:
        out.copy_(c)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = Q.mm_blockwise(a, sa, b, sb, ta, tb, out=out, accumulate=accumulate, status=status)
    assert got is out and status.item() == 0
    err = (out.double() - ref).abs() - tol
    assert bool((err <= 0).all()), f"{int((err > 0).sum())} of {M * N} outside, worst {float((err + tol).max())} for {float(tol.max())}"
    assert bool((buf[:512] == 0xA5).all()) and bool((buf[512 + nb:] == 0xA5).all()), "written outside C"


ROWS = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 200, 255, 256, 257, 333, 640]


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_mm_rows(M, dtype):
    check_mm(M, 384, 640, "1x128", "128x128", dtype, seed=M)


@pytest.mark.parametrize("M,N", [(1, 1), (1, 61), (3, 130), (128, 1), (130, 257), (257, 130), (64, 1000), (300, 515), (513, 2)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_mm_odd_columns(M, N, dtype):
    check_mm(M, N, 256, "1x128", "1x128", dtype, seed=M + N)


@pytest.mark.parametrize("K", [128, 256, 384, 512, 896, 1024, 1152, 2176, 4096, 14336])
@pytest.mark.parametrize("M", [1, 20, 129])
def test_mm_reduction_lengths(K, M):
    check_mm(M, 256, K, "1x128", "128x128", torch.float32, seed=K)
    check_mm(M, 136, K, "1x128", "1x128", torch.float32, seed=K)


@pytest.mark.parametrize("ta,tb", [("1x128", "128x128"), ("128x128", "1x128"), ("128x128", "128x128"), ("1x128", "1x128")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("M,N", [(128, 128), (384, 256), (256, 1152)])
def test_mm_tiles_and_accumulate(M, N, ta, tb, dtype, accumulate):
    check_mm(M, N, 384, ta, tb, dtype, accumulate)


@pytest.mark.parametrize("M,N,K,tb", [(2048, 4096, 512, "128x128"), (1000, 5120, 1024, "128x128"), (4224, 2176, 384, "1x128"),
                                      (8192, 1280, 256, "128x128"), (130, 18432, 256, "128x128"), (5000, 384, 640, "1x128"),
                                      (40, 18432, 256, "128x128"), (4, 7168, 2048, "128x128")])
@pytest.mark.parametrize("dtype,accumulate", [(torch.bfloat16, False), (torch.float32, True), (torch.bfloat16, True)])
def test_mm_many_tiles(M, N, K, tb, dtype, accumulate):
    check_mm(M, N, K, "1x128", tb, dtype, accumulate)


# widths of 16 to 192 tokens with splits of 1 to 8, tiles that end inside them, and the pair kernel with reductions of
# 1, 2, 3, 7 and 9 blocks over more tiles than the machine has pairs
@pytest.mark.parametrize("M,N,K,tb", [(1, 4096, 4096, "128x128"), (16, 14336, 512, "128x128"), (17, 2048, 2048, "128x128"),
                                      (40, 4096, 4096, "128x128"), (64, 18432, 896, "128x128"), (100, 1000, 4096, "1x128"),
                                      (128, 7168, 2304, "128x128"), (200, 4096, 4096, "128x128"), (333, 4096, 4096, "128x128"),
                                      (350, 4000, 1152, "1x128"), (513, 700, 8192, "1x128"), (1024, 1024, 4096, "1x128"),
                                      (5000, 5120, 128, "128x128"), (5000, 5120, 128, "1x128"), (2600, 5120, 256, "1x128"),
                                      (4999, 4991, 384, "1x128"), (2305, 4608, 896, "128x128"), (4600, 2300, 1152, "1x128")])
@pytest.mark.parametrize("dtype,accumulate", [(torch.bfloat16, False), (torch.float32, True), (torch.bfloat16, True)])
def test_mm_plans(M, N, K, tb, dtype, accumulate):
    check_mm(M, N, K, "1x128", tb, dtype, accumulate, seed=M)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dropout_calls_in_a_row(dtype):
    """Calls that may overlap their neighbours' ends, each in place on the last one's result, against the same calls one at
    a time."""
    def chain(sync):
        x = torch.randn((4096, 2048), generator=torch.Generator("cuda").manual_seed(5), device="cuda").to(dtype)
        r, outs = x.clone(), []
        for i in range(24):
            Q.drop_add(x, 0.25, i, residual=r, out=r)
            sync()
            outs.append(Q.drop_q_blockwise(r, 0.25, i, colwise=True))
            sync()
            Q.drop_add(r, 0.5, 100 + i, out=x)
            sync()
        torch.cuda.synchronize()
        return [r, x] + [t for o in outs for t in (o.q_row, o.s_row, o.q_colT, o.s_colT)]

    for a, b in zip(chain(lambda: None), chain(torch.cuda.synchronize)):
        assert torch.equal(a, b)


# each width from its narrowest call on and each depth of split, results that end inside a tile and reductions that the
# split does not divide
@pytest.mark.parametrize("M,N,K,tb", [(3, 128, 768, "128x128"), (1, 198, 2816, "1x128"), (1, 128, 3456, "128x128"),
                                      (19, 10240, 1280, "128x128"), (17, 1933, 5120, "1x128"), (17, 2048, 4736, "128x128"),
                                      (642, 137, 1920, "1x128"), (81, 12939, 256, "1x128"), (36, 13131, 1536, "1x128"),
                                      (33, 6656, 2560, "128x128"), (1300, 154, 2432, "1x128"), (33, 3200, 7040, "128x128"),
                                      (132, 8290, 896, "1x128"), (649, 134, 6272, "1x128"), (163, 896, 5760, "128x128"),
                                      (524, 12895, 512, "1x128"), (555, 12928, 1024, "128x128"), (171, 6604, 1536, "1x128"),
                                      (1326, 411, 2432, "1x128"), (146, 3968, 3456, "128x128"), (1324, 155, 5760, "1x128"),
                                      (138, 1920, 8064, "128x128"), (100, 2048, 8192, "128x128"), (192, 2048, 8192, "1x128")])
@pytest.mark.parametrize("dtype,accumulate", [(torch.bfloat16, False), (torch.float32, True)])
def test_mm_widths_and_splits(M, N, K, tb, dtype, accumulate):
    check_mm(M, N, K, "1x128", tb, dtype, accumulate, seed=N)


def test_mm_calls_in_a_row():
    """Calls that may overlap their neighbours' ends (each result is the next one's input or accumulator)."""
    a, sa = operand(24, 512, "1x128", 81)
    b, sb = operand(512, 512, "128x128", 82)
    big, sbig = operand(700, 512, "1x128", 83)
    c = torch.zeros((24, 512), device="cuda")
    d = torch.zeros((700, 512), device="cuda")
    one, two = Q.mm_blockwise(a, sa, b, sb, dtype=torch.float32), Q.mm_blockwise(big, sbig, b, sb, dtype=torch.float32)
    torch.cuda.synchronize()
    for i in range(64):
        Q.mm_blockwise(a, sa, b, sb, out=c, accumulate=True)
        Q.mm_blockwise(big, sbig, b, sb, out=d, accumulate=True)
        x = Q.mm_blockwise(a, sa, b, sb)
        q = Q.q_blockwise(x)
        y = Q.mm_blockwise(q.q_row, q.s_row, b, sb)
    # the sums of 64 equal FP32 terms: each addition rounds once
    assert bool(((c.double() - 64 * one.double()).abs() <= 64 * 64 * 2.0 ** -24 * one.double().abs()).all())
    assert bool(((d.double() - 64 * two.double()).abs() <= 64 * 64 * 2.0 ** -24 * two.double().abs()).all())
    x1 = Q.mm_blockwise(a, sa, b, sb)
    torch.cuda.synchronize()
    q1 = Q.q_blockwise(x1)
    torch.cuda.synchronize()
    assert torch.equal(y, Q.mm_blockwise(q1.q_row, q1.s_row, b, sb))


def test_mm_on_two_streams():
    a, sa = operand(48, 2048, "1x128", 91)
    b, sb = operand(2048, 2048, "128x128", 92)
    big, sbig = operand(3000, 2048, "1x128", 93)
    want, wide = Q.mm_blockwise(a, sa, b, sb), Q.mm_blockwise(big, sbig, b, sb)
    torch.cuda.synchronize()
    s0, s1 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        with torch.cuda.stream(s0):
            x = Q.mm_blockwise(a, sa, b, sb)
        with torch.cuda.stream(s1):
            y = Q.mm_blockwise(big, sbig, b, sb)
        got.append((x, y))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) and torch.equal(y, wide) for x, y in got)


def test_mm_random_shapes():
    rng = np.random.default_rng(5)
    for i in range(40):
        M, K = int(np.exp(rng.uniform(0, 7.3))), 128 * int(rng.integers(1, 12))
        tb = ["1x128", "128x128"][i % 2]
        N = 128 * int(rng.integers(1, 12)) if tb == "128x128" else int(np.exp(rng.uniform(0, 7.3)))
        check_mm(M, N, K, "1x128", tb, [torch.bfloat16, torch.float32][int(rng.integers(2))], bool(rng.integers(2)), seed=i)


def test_mm_output_past_32_bit_offsets():
    M, N = 40064, 57344 + 128   # 2.3e9 elements
    a, sa = operand(M, 128, "1x128", 3)
    b, sb = operand(N, 128, "128x128", 4)
    c = Q.mm_blockwise(a, sa, b, sb)
    for rows in (slice(0, 3), slice(20000, 20002), slice(M - 3, M)):
        n = sb.shape[0] * 128
        ref, tol = mm_bound(*mm_reference(a[rows], sa[rows], "1x128", b, sb, "128x128"), 1, torch.bfloat16)
        assert bool(((c[rows].double() - ref).abs() <= tol).all()) and n == N


@pytest.mark.parametrize("M", [1, 40, 300, 2048])
def test_mm_same_result_every_time(M):
    a, sa = operand(M, 2048, "1x128", 8)
    b, sb = operand(1024, 2048, "128x128", 9)
    first = Q.mm_blockwise(a, sa, b, sb, dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(first, Q.mm_blockwise(a, sa, b, sb, dtype=torch.float32))


@pytest.mark.parametrize("M,N", [(5, 256), (200, 256), (600, 640), (2300, 1536)])
def test_mm_nan_inf_and_zero_stay_in_their_rows(M, N):
    a, sa = operand(M, 384, "1x128", 11)
    b, sb = operand(N, 384, "128x128", 12)
    clean = Q.mm_blockwise(a, sa, b, sb, dtype=torch.float32)
    a[1, 200] = 0x7F          # a NaN code: row 1
    b[130, 5] = 0xFF          # and column 130
    sa[3, 2] = float("inf")   # an infinite scale: row 3 (NaN or inf, by the sign of its block sum)
    got = Q.mm_blockwise(a, sa, b, sb, dtype=torch.float32)
    assert bool(got[1].isnan().all()) and bool(got[:, 130].isnan().all())
    assert not bool(got[3].isfinite().any())
    keep_r = torch.ones(M, dtype=torch.bool, device="cuda")
    keep_r[[1, 3]] = False
    keep_c = torch.ones(N, dtype=torch.bool, device="cuda")
    keep_c[130] = False
    assert torch.equal(got[keep_r][:, keep_c], clean[keep_r][:, keep_c])
    z = Q.mm_blockwise(torch.zeros_like(a), sa.clamp(max=1.0), torch.zeros_like(b), sb, dtype=torch.float32)
    assert bool((z == 0).all())


def test_mm_empty():
    a, sa = torch.empty((0, 256), dtype=torch.uint8, device="cuda"), torch.empty((0, 2), device="cuda")
    b, sb = operand(128, 256, "128x128", 1)
    assert Q.mm_blockwise(a, sa, b, sb).shape == (0, 128)
    a0, s0 = torch.empty((5, 0), dtype=torch.uint8, device="cuda"), torch.empty((5, 0), device="cuda")
    b0, t0 = torch.empty((128, 0), dtype=torch.uint8, device="cuda"), torch.empty((1, 0), device="cuda")
    c = torch.ones((5, 128), device="cuda")
    assert torch.equal(Q.mm_blockwise(a0, s0, b0, t0, out=c, accumulate=True), torch.ones_like(c))
    assert torch.equal(Q.mm_blockwise(a0, s0, b0, t0, out=c), torch.zeros_like(c))


def test_mm_on_a_side_stream_and_in_a_graph():
    a, sa = operand(33, 1024, "1x128", 21)
    b, sb = operand(512, 1024, "128x128", 22)
    want = Q.mm_blockwise(a, sa, b, sb)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = Q.mm_blockwise(a, sa, b, sb)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Q.mm_blockwise(a, sa, b, sb, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_mm_of_quantized_tensors_is_the_product():
    """End to end from q_blockwise: the product of the copies is the product of what they decode to."""
    x, w = dev(W.gen("normal", (256, 512), 31)), dev(W.gen("weight", (384, 512), 32))
    xq, wq = Q.q_blockwise(x, "1x128", colwise=True), Q.q_blockwise(w, "128x128", colwise=True)
    y = Q.mm_blockwise(xq.q_row, xq.s_row, wq.q_row, wq.s_row, dtype=torch.float32)
    X, Wd = xq.dequantize().double(), wq.dequantize().double()
    _, mags = X @ Wd.T, X.abs() @ Wd.abs().T
    # the decoded values are rounded FP32 products: one more rounding each
    assert bool(((y.double() - X @ Wd.T).abs() <= (2.0 ** -16 + 9 * 2.0 ** -24) * mags).all())


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------

M32 = np.uint64(0xFFFFFFFF)


def draws(n, seed, offset):
    """The 16-bit draws of n elements (numpy, unsigned 64-bit products)."""
    g = (np.arange((n + 7) // 8, dtype=np.uint64) + np.uint64(offset))
    c = [g & M32, g >> np.uint64(32), np.full_like(g, 2), np.zeros_like(g)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), q & M32, (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p & M32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    out = np.empty((len(g), 8), np.uint32)
    for i in range(4):
        out[:, 2 * i] = c[i] & np.uint64(0xFFFF)
        out[:, 2 * i + 1] = c[i] >> np.uint64(16)
    return out.reshape(-1)[:n]


def test_draws_are_the_oracles_philox():
    for seed, offset in ((0, 0), (0x123456789ABCDEF, 3), (2 ** 64 - 1, 2 ** 40 + 5)):
        d = draws(16, seed, offset)
        for b in range(2):
            g = offset + b
            w = O.philox4x32_10([g & 0xFFFFFFFF, g >> 32, 2, 0], [seed & 0xFFFFFFFF, seed >> 32])
            assert [int(v) for i in range(4) for v in (w[i] & 0xFFFF, w[i] >> 16)] == d[8 * b:8 * b + 8].tolist()


def as_f32(x):
    return W.bf16_bits_to_f32(x) if x.dtype == np.uint16 else x


def drop_reference(x, p, seed, offset, residual=None):
    """FP32 values before the output rounding, and the kept mask."""
    T = int(np.rint(p * 65536))
    keep = (draws(x.size, seed, offset) >= T).reshape(x.shape)
    c = np.float32(65536 / (65536 - T)) if T < 65536 else np.float32(0)
    with np.errstate(invalid="ignore", over="ignore"):
        v = as_f32(x).astype(np.longdouble) * np.longdouble(c)
        if residual is None:
            return np.where(keep, v, np.longdouble(0)).astype(np.float32), keep
        r = as_f32(residual).astype(np.longdouble)
        return np.where(keep, v + r, r).astype(np.float32), keep


def out_bits(v, like):
    return O.bf16_round(v) if like.dtype == np.uint16 else v


DROP_CASES = [((1, 1), 0.5), ((1, 7), 0.5), ((3, 3), 0.1), ((8, 8), 0.0), ((16, 33), 1.0), ((257, 129), 0.25), ((1, 2048), 0.9),
              ((100, 2049), 0.1), ((3001, 111), 0.3), ((64, 4096), 1e-6), ((64, 4096), 0.999995), ((5, 65536), 0.1)]


@pytest.mark.parametrize("shape,p", DROP_CASES)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("res", [False, True])
def test_drop_add(shape, p, bf16, res):
    x = W.gen("normal", shape, 41, bf16=bf16)
    r = W.gen("t3", shape, 42, bf16=bf16) if res else None
    seed, offset = 0xFEDCBA9876543210, (1 << 33) + 12345
    want, _ = drop_reference(x, p, seed, offset, r)
    n = x.size
    buf = torch.full((n * x.itemsize + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    out = buf[256:256 + n * x.itemsize].view(torch.bfloat16 if bf16 else torch.float32).view(shape)
    Q.drop_add(dev(x), p, seed, offset, None if r is None else dev(r), out=out)
    same(host(out), out_bits(want, x), f"{shape} p {p}")
    assert bool((buf[:256] == 0xA5).all()) and bool((buf[256 + n * x.itemsize:] == 0xA5).all())


def test_drop_add_in_place_matches_and_shards_draw_alike():
    x, r = W.gen("normal", (128, 1024), 43), W.gen("normal", (128, 1024), 44)
    want = Q.drop_add(dev(x), 0.2, 9, 100, dev(r))
    xi, ri = dev(x), dev(r)
    assert torch.equal(Q.drop_add(xi, 0.2, 9, 100, dev(r), out=xi), want)
    assert torch.equal(Q.drop_add(dev(x), 0.2, 9, 100, ri, out=ri), want)
    lower = Q.drop_add(dev(x[40:]), 0.2, 9, 100 + 40 * 1024 // 8, dev(r[40:]))
    assert torch.equal(lower, want[40:])


@pytest.mark.parametrize("bf16", [True, False])
def test_drop_add_masked_nan_and_inf(bf16):
    x = W.gen("normal", (64, 512), 45, bf16=False)
    keep = (draws(x.size, 77, 0) >= 32768).reshape(x.shape)
    x[~keep] = np.where(np.arange((~keep).sum()) % 2, np.float32(np.nan), np.float32(np.inf))
    x = W.to_bf16_bits(x) if bf16 else x
    y = Q.drop_add(dev(x), 0.5, 77)
    assert bool(y.isfinite().all()) and bool((y[torch.from_numpy(~keep).cuda()] == 0).all())
    r = dev(W.gen("normal", (64, 512), 46, bf16=bf16))
    z = Q.drop_add(dev(x), 0.5, 77, residual=r)
    assert torch.equal(z[torch.from_numpy(~keep).cuda()], r[torch.from_numpy(~keep).cuda()])


def test_drop_add_share_and_gradient():
    """The dropped share is T / 65536, kept elements keep the mean, and the
    backward call is the transpose of the (linear) forward call, also by
    differences: powers of two make every step exact."""
    n = 1 << 22
    y = Q.drop_add(torch.ones(n, device="cuda"), 0.25, 5)
    share = float((y == 0).double().mean())
    assert abs(share - 0.25) < 5 * (0.25 * 0.75 / n) ** 0.5
    x, d, g = (dev(W.gen("normal", (64, 512), 50 + i, bf16=False)).sign().mul(2.0 ** -i) for i in range(3))
    f = lambda v: Q.drop_add(v, 0.5, 6, 7)
    assert torch.equal(f(x + d) - f(x), f(d))
    assert float((f(d) * g).sum()) == float((d * f(g)).sum())


DROPQ_CASES = [("normal", (128, 128), True, 0.1), ("t3", (256, 640), True, 0.5), ("normal", (1, 128), False, 0.1),
               ("grad", (37, 256), False, 0.3), ("normal", (1000, 384), False, 0.1), ("outliers", (384, 896), True, 0.25),
               ("normal", (128, 256), True, 1.0), ("normal", (128, 256), True, 0.0), ("weight", (640, 128), True, 0.999995)]


@pytest.mark.parametrize("kind,shape,colwise,p", DROPQ_CASES)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("rowwise", [True, False])
def test_drop_q_blockwise(kind, shape, colwise, p, bf16, rowwise):
    if not (rowwise or colwise):
        return
    x = W.gen(kind, shape, 61, bf16=bf16)
    x[: shape[0] // 3] = 0
    y, _ = drop_reference(x, p, 0xABCDEF0123456789, 1 << 34)
    want = O.blockwise(y, O.T1x128, rowwise, colwise)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = Q.drop_q_blockwise(dev(x), p, 0xABCDEF0123456789, 1 << 34, rowwise, colwise, status=status)
    for f in ("q_row", "s_row", "q_colT", "s_colT"):
        if getattr(want, f) is None:
            assert getattr(got, f) is None
        else:
            same(host(getattr(got, f)), getattr(want, f), f)
    assert status.item() == 0


@pytest.mark.parametrize("shape", [(128, 128), (1024, 128), (128, 8064), (1152, 1152), (2944, 640)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.75])
@pytest.mark.parametrize("bf16", [True, False])
def test_drop_q_blockwise_rowwise_alone(shape, p, bf16):
    """The rowwise copy by itself is that of both directions, inf and NaN elements and empty blocks included."""
    x = dev(W.gen("outliers", shape, 63, bf16=bf16))
    x[5:40, :128] = 0
    x[41, 3], x[42, 5], x[43, 7], x[43, 8], x[44, -128:] = np.nan, np.inf, -np.inf, np.nan, 2.0 ** -133
    st = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2)]
    both = Q.drop_q_blockwise(x, p, 77, 3, colwise=True, status=st[0])
    alone = Q.drop_q_blockwise(x, p, 77, 3, status=st[1])
    assert torch.equal(both.q_row, alone.q_row) and st[0].item() == st[1].item()
    assert torch.equal(both.s_row.view(torch.int32), alone.s_row.view(torch.int32))


def test_drop_q_blockwise_drops_nan_and_reports_what_is_kept():
    x = W.gen("normal", (128, 256), 62, bf16=False)
    keep = (draws(x.size, 3, 0) >= 32768).reshape(x.shape)
    x[~keep] = np.nan
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, _ = drop_reference(x, 0.5, 3, 0)
    got = Q.drop_q_blockwise(dev(x), 0.5, 3, colwise=True, status=status)
    same(host(got.q_row), O.blockwise(y, O.T1x128).q_row)
    assert status.item() == 0
    x[tuple(np.argwhere(keep)[0])] = np.inf
    Q.drop_q_blockwise(dev(x), 0.5, 3, colwise=True, status=status)
    assert status.item() == Q.Q_ST_NONFINITE


# ---------------------------------------------------------------------------
# the layer
# ---------------------------------------------------------------------------

def lossless(shape, seed):
    """Integers of [-7, 7] with a 7 in every 1x128, 128x1 and 128x128 tile:
    alpha = 64 and every code is exact, so the layer computes with x itself."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-6, 7, shape, generator=g, device="cuda").float()
    i = torch.arange(shape[0], device="cuda")
    for k in range(0, shape[1], 128):
        x[i, k + i % 128] = 7.0
    return x


@pytest.mark.parametrize("M", [128, 200, 256])
@pytest.mark.parametrize("p", [0.0, 0.5])
def test_linear_layer_gradients(M, p):
    from nvfp4_quantization_current_gb300.linear import BlockwiseLinear
    layer = BlockwiseLinear(256, 128, p=p, seed=17, dtype=torch.float32)
    rows = -(-M // 128) * 128
    x = lossless((rows, 256), 1)[:M].contiguous().requires_grad_()
    with torch.no_grad():
        layer.weight.copy_(lossless((128, 256), 2))
    r = lossless((rows, 128), 3)[:M].contiguous().requires_grad_()
    y = layer(x, r, offset=40)
    keep = torch.from_numpy(draws(M * 128, 17, 40) >= int(p * 65536)).cuda().view(M, 128).double() / (1 - p)
    Y = x.double() @ layer.weight.double().T * keep + r.double()
    assert torch.equal(y.double(), Y)        # small integers: every sum is exact
    # a gradient that the dropout leaves lossless: its kept elements are integers of [-7, 7] doubled
    dy = lossless((rows, 128), 4)[:M].contiguous()
    y.backward(dy)
    g = dy.double() * keep
    # the tiles of the dropped gradient, and of ragged columns, need not be lossless: an E4M3 code is off by
    # at most 2^-4 of its value, a product of two by 2^-3 + 2^-8 (2^-12 for the FP32 steps)
    share = 2.0 ** -3 + 2.0 ** -8 + 2.0 ** -12
    for got, want, mags in ((x.grad, g @ layer.weight.double(), g.abs() @ layer.weight.double().abs()),
                            (layer.weight.grad, g.T @ x.double(), g.abs().T @ x.double().abs())):
        assert bool(((got.double() - want).abs() <= share * mags).all())
    assert torch.equal(r.grad, dy)
    # by differences: raising one weight raises the loss <dy, y> by its gradient, up to the same share
    with torch.no_grad():
        base = float((layer(x, r, offset=40).double() * dy.double()).sum())
        for n, k in ((0, 0), (5, 17), (127, 255)):
            if float(layer.weight[n, k]) < 7:
                layer.weight[n, k] += 1
                diff = float((layer(x, r, offset=40).double() * dy.double()).sum()) - base
                layer.weight[n, k] -= 1
                mags = float((g[:, n].abs() * x[:, k].double().abs()).sum())
                assert abs(diff - float(layer.weight.grad[n, k])) <= share * mags


def test_linear_layer_main_grad_and_serving():
    from nvfp4_quantization_current_gb300.linear import BlockwiseLinear
    torch.manual_seed(0)
    layer = BlockwiseLinear(256, 384, p=0.1, seed=3)
    x = torch.randn(2, 128, 256, device="cuda", dtype=torch.bfloat16)
    layer(x, offset=1).float().square().sum().backward()
    want = layer.weight.grad.float()
    layer.weight.grad = None
    layer.main_grad = torch.zeros(384, 256, device="cuda")
    for _ in range(2):
        layer(x, offset=1).float().square().sum().backward()
    assert layer.weight.grad is None
    assert torch.allclose(layer.main_grad, 2 * want, rtol=2.0 ** -7, atol=1e-6)
    layer.eval()
    with torch.no_grad():
        copies = layer.quantize_weight(colwise=False)
        one = layer(x[0, :1], copies=copies)
        t, w = Q.q_blockwise(x[0, :1].contiguous()), copies
        assert torch.equal(one, Q.mm_blockwise(t.q_row, t.s_row, w.q_row, w.s_row))


def test_first_call_of_a_host_thread():
    """A thread whose first CUDA call is the library's (an autograd thread can be one) has no current context yet."""
    import threading
    x = dev(W.gen("normal", (128, 256), 71))
    copies = Q.alloc_blockwise(128, 256, "cuda", "1x128", True, True)
    b, sb = operand(128, 256, "128x128", 72)
    c = torch.empty((128, 128), device="cuda")
    calls = [lambda: Q.drop_q_blockwise(x, 0.1, 1, out=copies), lambda: Q.mm_blockwise(copies.q_row, copies.s_row, b, sb, out=c),
             lambda: Q.q_blockwise(x, out=copies)]
    torch.cuda.synchronize()
    failed = []

    def run(f):
        try:
            f()
        except Exception as e:  # noqa: BLE001 (handed to the test's thread)
            failed.append(e)

    for f in calls:
        t = threading.Thread(target=run, args=(f,))
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
