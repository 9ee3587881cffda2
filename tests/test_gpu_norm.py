"""The norm ahead of a linear layer, its blockwise copies and its gradient against their formulas in 64 bits.

Tolerances.  A row's sum of squares is one of at most max(32, K / 1024) fused terms per thread and a tree of at most 10
additions, all positive, so it is off by at most n 2^-24 of itself with n = max(32, K / 1024) + 11, and rstd by half of
that and four roundings (the mean, + eps, the root, the quotient).  What follows from h and rstd alone is compared bit for
bit: y = (h rstd) w is two IEEE products and one rounding, its copies are the oracle's of that y.  The gradients: each FP32
product or sum below rounds by 2^-24, a sum of n terms by n 2^-24 of the sum of magnitudes, and the result by half a step
of its type (2^-8 for bfloat16).
"""
import numpy as np
import pytest
import torch

import oracle as O
import workloads as W

pytestmark = pytest.mark.gpu

Q = pytest.importorskip("nvfp4_quantization_current_gb300")

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
TINY = 1e-37   # below it results lose bits to underflow


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Q.lib()


def guarded(n, dtype):
    """(a tensor of n elements, a check that nothing was written around it)."""
    size = n * dtype.itemsize
    buf = torch.full((size + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    return buf[512:512 + size].view(dtype), lambda: bool((buf[:512] == 0xA5).all()) and bool((buf[512 + size:] == 0xA5).all())


def make(M, K, dtype, wt, residual, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = (new(M, K) * torch.exp(new(M, 1))).to(dtype)
    w = (1 + 0.2 * new(K)).to(wt)
    return x, w, new(M, K).to(dtype) if residual else None


def sum_terms(K):
    return max(32, -(-K // 1024)) + 11


def check_factor(h, rstd, eps, K):
    want = 1 / (h.double().square().mean(-1) + eps).sqrt()
    tol = (sum_terms(K) / 2 + 4) * U * want
    assert bool(((rstd.double() - want).abs() <= tol).all()), float(((rstd.double() - want).abs() / want).max() / U)


def y32(h, rstd, w):
    return (h.float() * rstd[:, None]) * w.float()


def check_norm(M, K, dtype, wt, residual, eps=1e-6, amax=True, seed=0):
    x, w, r = make(M, K, dtype, wt, residual, seed + K)
    out, out_ok = guarded(M * K, dtype)
    hb, h_ok = guarded(M * K, dtype)
    top = torch.full((1,), 7e30, device="cuda") if amax else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = x.clone()
    y, h, rstd = Q.norm_add(x, w, eps, r, amax=top, out=out.view(M, K), h_out=hb.view(M, K) if residual else None, status=status)
    assert torch.equal(x, before) and out_ok() and h_ok() and status.item() == 0
    assert torch.equal(h, x if r is None else (x.float() + r.float()).to(dtype))
    check_factor(h, rstd, eps, K)
    assert torch.equal(y, y32(h, rstd, w).to(dtype))
    if amax:
        assert float(top) == float(y.abs().max())
        assert torch.equal(top, Q.q_amax(y))


LENGTHS = [1, 2, 3, 5, 7, 8, 9, 31, 32, 33, 64, 100, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1000, 1024, 1111, 2040, 2047, 2048, 2049,
           4096, 4097, 4104, 7168, 8191, 8192, 8200, 14336, 16384, 16385, 16392, 18432, 32768, 32776, 40001, 65536]


@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("dtype,wt", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
def test_norm_row_lengths(K, dtype, wt):
    for M, residual in ((1, True), (3, False), (9, True)):
        check_norm(M, K, dtype, wt, residual)


@pytest.mark.parametrize("M,K", [(8192, 64), (3001, 1111), (1000, 4096), (257, 7168), (40, 18432), (700, 33)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_many_rows(M, K, dtype, residual):
    check_norm(M, K, dtype, dtype, residual, amax=False)
    check_norm(M, K, dtype, F32, residual, eps=0.5)


# rows of every layout the rings take, and one more row than their CTAs share evenly
MANY = [(5000, 2048), (2500, 4104), (4870, 4096), (2440, 8192), (1220, 14336), (1300, 16384), (3050, 513), (2000, 8191), (700, 10001), (400, 16383)]


@pytest.mark.parametrize("M,K", MANY)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_rings(M, K, dtype, residual):
    check_norm(M, K, dtype, F32, residual, amax=residual)
    check_norm(M, K, dtype, dtype, residual, amax=not residual)


@pytest.mark.parametrize("K", [257, 301, 385, 509, 511])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_rings_of_one_warp(K, dtype, residual):
    # behind rows of many warps, whose parts of large sums lie in shared memory
    x, w, r = make(3000, 8191, dtype, dtype, residual, 3)
    big = x * 1000
    for M in (2432, 5001):
        Q.norm_add(big, w, residual=r)
        check_norm(M, K, dtype, dtype, residual, amax=False)
        Q.norm_add(big, w, residual=r)
        check_norm(M, K, dtype, F32, residual)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("K", [2048, 2056, 1111])
def test_norm_rings_in_place(residual, K):
    x, w, r = make(5000, K, BF16, BF16, residual, 13)
    y, h, rstd = Q.norm_add(x, w, residual=r)
    a, b = x.clone(), None if r is None else r.clone()
    got = Q.norm_add(a, w, residual=b, out=b if residual else a, h_out=a if residual else None)
    assert torch.equal(got[0], y) and torch.equal(got[2], rstd) and (not residual or torch.equal(got[1], h))


def test_norm_in_place():
    x, w, r = make(37, 512, BF16, BF16, True, 1)
    y, h, rstd = Q.norm_add(x, w, residual=r)
    for swap in (False, True):
        a, b = x.clone(), r.clone()
        o = dict(out=a, h_out=b) if swap else dict(out=b, h_out=a)
        got = Q.norm_add(a, w, residual=b, **o)
        assert got[0] is o["out"] and got[1] is o["h_out"]
        assert torch.equal(got[0], y) and torch.equal(got[1], h) and torch.equal(got[2], rstd)
    for K in (512, 511, 50000):
        x, w, _ = make(5, K, F32, F32, False, 2)
        want = Q.norm_add(x, w)[0]
        assert torch.equal(Q.norm_add(x, w, out=x)[0], want)


@pytest.mark.parametrize("K", [64, 1000, 4096, 4097, 40000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_rows_keep_to_themselves(K, dtype):
    x, w, r = make(7, K, dtype, F32, True, 3)
    clean = Q.norm_add(x, w, residual=r)
    x[1, K // 2] = float("nan")
    x[2, 0] = float("inf")
    r[3, K - 1] = -float("inf")
    x[4], r[4] = 0, 0
    x[5] = 1e30   # squares past FP32's range
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    top = torch.empty(1, device="cuda")
    y, h, rstd = Q.norm_add(x, w, 1e-6, r, amax=top, status=status)
    for row in (0, 6):
        assert torch.equal(y[row], clean[0][row]) and torch.equal(rstd[row], clean[2][row])
    assert bool(y[1].isnan().all()) and bool(rstd[1].isnan())
    for row, col in ((2, 0), (3, K - 1)):   # inf times a factor of zero
        assert float(rstd[row]) == 0 and bool(y[row, col].isnan()) and int(y[row].isnan().sum()) == 1
    assert bool((y[4] == 0).all()) and abs(float(rstd[4]) - 1e3) < 1e-3
    assert float(rstd[5]) == 0 and bool((y[5] == 0).all())
    assert bool(top.isnan()) and status.item() == Q.Q_ST_NONFINITE


def test_norm_shapes_and_empty():
    x, w, _ = make(24, 256, BF16, BF16, False, 4)
    y, h, rstd = Q.norm_add(x.view(2, 3, 4, 256), w)
    assert y.shape == (2, 3, 4, 256) and rstd.shape == (2, 3, 4) and h.data_ptr() == x.data_ptr()
    one, _, s = Q.norm_add(x[0], w)
    assert one.shape == (256,) and s.shape == () and torch.equal(one, y.view(24, 256)[0])
    top = torch.ones(1, device="cuda")
    y, _, rstd = Q.norm_add(x[:0], w, amax=top)
    assert y.shape == (0, 256) and rstd.shape == (0,) and float(top) == 0
    dx, dw = Q.norm_grad(x[:0], x[:0], rstd, w)
    assert dx.shape == (0, 256) and bool((dw == 0).all())
    with pytest.raises(Q.QuantError, match="K = 0"):
        Q.norm_add(torch.empty((3, 0), device="cuda"), torch.empty(0, device="cuda"))


# ---------------------------------------------------------------------------
# the blockwise copies
# ---------------------------------------------------------------------------

def host(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16) if t.dtype == BF16 else t.cpu().numpy()


def check_cast(M, K, dtype, wt, residual, rowwise, colwise, seed=0):
    x, w, r = make(M, K, dtype, wt, residual, seed + M + K)
    x[: M // 5] = 0
    if residual:
        r[: M // 5] = 0
    bufs = {}
    for name, shape, t in (("q_row", (M, K), torch.uint8), ("s_row", (M, K // 128), F32), ("q_colT", (K, M), torch.uint8),
                           ("s_colT", (K, M // 128), F32)):
        bufs[name] = guarded(shape[0] * shape[1], t) if (rowwise if name.endswith("row") else colwise) else None
        if bufs[name]:
            bufs[name] = (bufs[name][0].view(shape), bufs[name][1])
    out = Q.BlockwiseTensor(*(b and b[0] for b in bufs.values()), Q.Q_T1x128)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, h, rstd = Q.norm_q_blockwise(x, w, 1e-6, r, rowwise, colwise, out=out, status=status)
    assert got is out and status.item() == 0 and all(b is None or b[1]() for b in bufs.values())
    assert torch.equal(h, x if r is None else (x.float() + r.float()).to(dtype))
    check_factor(h, rstd, 1e-6, K)
    want = O.blockwise(host(y32(h, rstd, w)), O.T1x128, rowwise, colwise)
    for name, b in bufs.items():
        if b:
            a, e = host(b[0]), getattr(want, name)
            assert np.array_equal(a.view(np.uint32) if a.dtype == np.float32 else a, e.view(np.uint32) if e.dtype == np.float32 else e), name


@pytest.mark.parametrize("M,K", [(1, 128), (2, 256), (37, 384), (333, 7168), (129, 4096), (8, 16384), (3, 32768), (2, 33024)])
@pytest.mark.parametrize("dtype,wt", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_cast_rows(M, K, dtype, wt, residual):
    check_cast(M, K, dtype, wt, residual, True, False)


@pytest.mark.parametrize("M,K", [(5000, 2048), (2500, 4096), (1300, 14336), (2440, 8192)])
@pytest.mark.parametrize("dtype,wt", [(BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_cast_rings(M, K, dtype, wt, residual):
    check_cast(M, K, dtype, wt, residual, True, False)


@pytest.mark.parametrize("M,K", [(128, 128), (256, 640), (1152, 384), (384, 8064), (128, 16512), (2944, 1152), (128, 33024), (2560, 4096), (4992, 2048)])
@pytest.mark.parametrize("dtype,wt", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("residual,rowwise", [(False, True), (True, True), (True, False)])
def test_norm_cast_both(M, K, dtype, wt, residual, rowwise):
    check_cast(M, K, dtype, wt, residual, rowwise, True)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_cast_reports_nonfinite(dtype):
    x, w, _ = make(128, 256, dtype, dtype, False, 5)
    x[77, 200] = float("inf")
    for kw in (dict(), dict(colwise=True), dict(rowwise=False, colwise=True)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        t, h, rstd = Q.norm_q_blockwise(x, w, status=status, **kw)
        assert status.item() == Q.Q_ST_NONFINITE
        want = O.blockwise(host(y32(h, rstd, w)), O.T1x128, True, True)
        if t.q_row is not None:
            assert np.array_equal(np.delete(host(t.q_row), 77, 0), np.delete(want.q_row, 77, 0))
        if t.q_colT is not None:
            assert np.array_equal(np.delete(host(t.q_colT), 200, 0), np.delete(want.q_colT, 200, 0))


# ---------------------------------------------------------------------------
# the gradient
# ---------------------------------------------------------------------------

def grad_reference(dy, h, rstd, w, dh):
    """(dx, dw) in 64 bits and bounds of what FP32 may lose before the last rounding."""
    M, K = h.shape
    s = rstd.double()[:, None]
    v, d = h.double() * s, dy.double()
    g = d * w.double()
    c = (g * v).mean(1, keepdim=True)
    dx = s * (g - v * c)
    # v, g and their product round once each, the sum over n terms; then the quotient, v c, the difference and the factor
    ec = (sum_terms(K) + 5) * U * (g * v).abs().mean(1, keepdim=True)
    edx = s.abs() * (3 * U * g.abs() + 4 * U * (v * c).abs() + v.abs() * ec)
    if dh is not None:
        dx = dx + dh.double()
        edx = edx + U * (dx.abs() + edx)
    # v rounds once; a thread adds M / (rows in flight) terms, a walk parts / 8, and then eight
    edw = (M + 16) * U * (d * v).abs().sum(0)
    return dx, edx, (d * v).sum(0), edw


def outside(got, want, err):
    tol = err + HALF_STEP[got.dtype] * (want.abs() + err) + TINY
    return int(((got.double() - want).abs() > tol).sum())


def check_grad(M, K, dtype, wt, with_dh, seed=0):
    h, w, dh = make(M, K, dtype, wt, with_dh, seed + M + K)
    dy = make(M, K, dtype, wt, False, seed + M + K + 1)[0]
    rstd = (h.float().square().mean(1) + 1e-6).rsqrt()
    out, ok = guarded(M * K, dtype)
    dx, dw = Q.norm_grad(dy, h, rstd, w, dh, out=out.view(M, K))
    assert ok() and dw.dtype == wt and dx.dtype == dtype
    wx, ex, ww, ew = grad_reference(dy, h, rstd, w, dh)
    assert outside(dx, wx, ex) == 0 and outside(dw, ww, ew) == 0
    again, none = Q.norm_grad(dy, h, rstd, w, dh, need_dw=False)
    assert none is None and torch.equal(again, dx)
    assert torch.equal(Q.norm_grad(dy, h, rstd, w, dh)[1], dw)   # the same sums every time


@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("dtype,wt", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
def test_grad_row_lengths(K, dtype, wt):
    for M, dh in ((1, True), (10, False)):
        check_grad(M, K, dtype, wt, dh)


@pytest.mark.parametrize("M,K", [(8192, 64), (3001, 1111), (1000, 4096), (2500, 7168), (700, 33), (400, 16392), (5000, 4097), (700, 14336), (305, 16384), (5000, 256),
                                 (20000, 7), (3000, 300), (1500, 8200)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dh", [False, True])
def test_grad_many_rows(M, K, dtype, dh):
    check_grad(M, K, dtype, dtype, dh)


def test_grad_in_place():
    for K in (512, 500, 511, 40000):
        h, w, dh = make(9, K, F32, F32, True, 6)
        dy = make(9, K, F32, F32, False, 7)[0]
        _, _, rstd = Q.norm_add(h, w)
        dx, dw = Q.norm_grad(dy, h, rstd, w, dh)
        for i in range(3):
            t = [dy.clone(), h.clone(), dh.clone()]
            got = Q.norm_grad(t[0], t[1], rstd, w, t[2], out=t[i])
            assert torch.equal(got[0], dx) and torch.equal(got[1], dw)


@pytest.mark.parametrize("residual", [False, True])
def test_autograd_and_differences(residual):
    """The module's gradients against 64-bit autograd of the formula, and against its differences."""
    x, w, r = make(33, 257, F32, F32, residual, 8)
    leaves = [t.clone().requires_grad_() for t in (x, w, r) if t is not None]
    y, h, _ = Q.norm_add(leaves[0], leaves[1], 1e-3, leaves[2] if residual else None)
    gy, gh = torch.randn(33, 257, device="cuda"), torch.randn(33, 257, device="cuda")
    ((y * gy).sum() + (h * gh).sum()).backward()

    def loss(x, w, r):
        h = x if r is None else x + r
        return (h / (h.square().mean(1, keepdim=True) + 1e-3).sqrt() * w * gy.double()).sum() + (h * gh.double()).sum()

    wide = [t.detach().double().requires_grad_() for t in leaves]
    loss(*wide, *([] if residual else [None])).backward()
    for a, b in zip(leaves, wide):
        assert float((a.grad.double() - b.grad).abs().max()) < 1e-4 * float(b.grad.abs().max())
    for i, t in enumerate(wide):
        d = torch.randn_like(t)
        p = [u.detach() for u in wide] + ([] if residual else [None])
        up, down = list(p), list(p)
        up[i], down[i] = p[i] + 1e-6 * d, p[i] - 1e-6 * d
        diff = float(loss(*up) - loss(*down)) / 2e-6
        assert abs(diff - float((leaves[i].grad.double() * d).sum())) < 1e-5 * float((leaves[i].grad.double().abs() * d.abs()).sum())


def test_second_derivative_raises():
    x, w, r = (t.requires_grad_() for t in make(4, 64, F32, F32, True, 9))
    y, h, _ = Q.norm_add(x, w, residual=r)
    (g,) = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivative"):
        g.sum().backward()


def test_streams_graphs_and_rows_of_calls():
    x, w, r = make(300, 1024, BF16, F32, True, 10)
    want = Q.norm_add(x, w, residual=r)
    cast = Q.norm_q_blockwise(x[:256], w, residual=r[:256], colwise=True)
    grad = Q.norm_grad(x, r, want[2], w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [Q.norm_add(x, w, residual=r) for _ in range(20)]
        gots = [Q.norm_grad(x, r, want[2], w) for _ in range(20)]
    here = [Q.norm_grad(x, r, want[2], w) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for y in got for a, b in zip(y, want))
    assert all(torch.equal(a, b) for y in gots + here for a, b in zip(y, grad))
    out, h = torch.zeros_like(x), torch.zeros_like(x)
    top = torch.zeros(1, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            Q.norm_add(x, w, residual=r, out=out, h_out=h, amax=top)
            c = Q.norm_q_blockwise(x[:256], w, residual=r[:256], colwise=True)
            d = Q.norm_grad(x, r, want[2], w)
    g.replay()
    out.zero_()
    top.fill_(9e9)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(h, want[1]) and torch.equal(top, Q.q_amax(want[0]))
    assert all(torch.equal(a, b) for a, b in zip(d, grad))
    for f in ("q_row", "s_row", "q_colT", "s_colT"):
        assert torch.equal(getattr(c[0], f), getattr(cast[0], f))


def test_offsets_past_32_bits():
    M, K = 300000, 8192   # 2.5e9 elements
    x = torch.empty((M, K), dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(11)
    rows = torch.tensor([0, 1, 131072, 262143, 262144, 299999], device="cuda")
    x.fill_(1.0)
    x[rows] = torch.randn((6, K), generator=g, device="cuda").to(BF16)
    w = torch.randn(K, generator=g, device="cuda").to(BF16)
    y, _, rstd = Q.norm_add(x, w)
    small = Q.norm_add(x[rows], w)
    assert torch.equal(y[rows], small[0]) and torch.equal(rstd[rows], small[2])
    dx, _ = Q.norm_grad(x, x, rstd, w, out=y, need_dw=False)
    assert torch.equal(dx[rows], Q.norm_grad(x[rows], x[rows], rstd[rows], w, need_dw=False)[0])
    del y, dx
    t, _, _ = Q.norm_q_blockwise(x[:299904], w, colwise=True)
    rows = rows[:5]
    small = Q.norm_q_blockwise(x[rows], w)[0]
    assert torch.equal(t.q_row[rows], small.q_row) and torch.equal(t.s_row[rows], small.s_row)
    last = Q.norm_q_blockwise(x[299776:299904], w, colwise=True)[0]
    assert torch.equal(t.q_colT[:, 299776:], last.q_colT) and torch.equal(t.s_colT[:, -1:], last.s_colT)


def test_inference_mode():
    x, w, r = make(9, 256, BF16, BF16, True, 14)
    want = Q.norm_add(x, w, residual=r)
    with torch.inference_mode():
        y, h, top = torch.empty_like(x), torch.empty_like(x), torch.zeros(1, device="cuda")
        got = Q.norm_add(x, w, residual=r, out=y, h_out=h, amax=top)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_first_call_of_a_host_thread():
    import threading
    x, w, _ = make(128, 256, BF16, BF16, False, 12)
    torch.cuda.synchronize()
    failed = []

    def run():
        try:
            Q.norm_q_blockwise(x, w, colwise=True)
        except Exception as e:  # noqa: BLE001 (handed to the test's thread)
            failed.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed, failed
