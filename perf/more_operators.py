"""The operators around a linear layer's input as cases to be timed and compared: the matrix product of
NVFP4 copies, the root-mean-square norm with the residual's addition, the same norm with its result as
blockwise FP8 copies, and the norm's gradient.

Each case runs in a plain form of elementary torch operations (``own`` false) or through the
library's entry points (``own`` true).  Sizes are those of the library's workloads (hidden 4096 with
FFN 14336 and sequence 8192; a 7168 / 18432 layer) plus single tokens, ragged and odd ones.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
FMAX = 448.0
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def mm(name, M, N, K, blk_b="16x16", out="bf16", accumulate=False):
    return {"name": name, "op": "mm", "M": M, "N": N, "K": K, "blk_b": blk_b, "out": out, "accumulate": accumulate}


def norm(name, op, M, K, dtype, residual, wt=None, colwise=False):
    return {"name": name, "op": op, "M": M, "K": K, "dtype": dtype, "residual": residual, "wt": wt or dtype, "colwise": colwise}


def listed():
    return [
        # one token through a 4096 x 4096 projection in four bits: the smallest product, latency
        mm("fp4 decode 1 token", 1, 4096, 4096),
        # a batch of sixteen sequences decoding through an FFN matrix: the weights' bytes
        mm("fp4 decode 16 tokens ffn", 16, 14336, 4096),
        # a ragged prompt chunk: rows that fill no tile, few tiles for the machine
        mm("fp4 prefill 333 tokens", 333, 4096, 4096),
        # forward of the FFN up-projection over a whole sequence
        mm("fp4 forward ffn", 8192, 14336, 4096),
        # weight gradient added into the FP32 main gradient; both operands with a scale per row and 16 elements
        mm("fp4 weight gradient ffn", 14336, 4096, 8192, "1x16", "f32", True),
        # sixteen sequences decoding: the norm's smallest call, latency
        norm("norm 16 rows", "norm", 16, 4096, "bf16", True),
        # the norm ahead of a layer over a whole sequence
        norm("norm add sequence", "norm", 8192, 4096, "bf16", True),
        # a first norm, without a residual, in FP32 on an odd shape
        norm("norm odd f32", "norm", 3001, 1111, "f32", False),
        # a ragged prompt chunk of the 7168 layer: the rowwise FP8 copy that the forward product reads
        norm("norm cast 333 rows", "normq", 333, 7168, "bf16", True),
        # a training step's sequence: both FP8 copies, for the forward product and the weight gradient
        norm("norm cast both", "normq", 8192, 4096, "bf16", True, colwise=True),
        # gradient of the norm over a whole sequence, with the residual stream's own gradient added
        norm("norm gradient sequence", "grad", 8192, 4096, "bf16", True),
        # an odd FP32 shape without a residual stream
        norm("norm gradient odd f32", "grad", 3001, 1111, "f32", False),
    ]


MOST_FLOPS = 2 * 8192 * 14336 * 4096


def draw(rng):
    def log_int(lo, hi, step=1):
        return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))) // step * step))

    op = rng.choice(["mm", "mm", "mm", "norm", "normq", "grad"])
    if op == "mm":
        kind = rng.choice(["decode", "forward", "forward", "weight"])
        while True:
            K = log_int(256, 18432, 32)
            if kind == "decode":
                M, N = log_int(1, 128), log_int(512, 18432, 16)
            else:
                M, N = log_int(129, 16384, 16 if kind == "weight" else 1), log_int(256, 18432, 16)
            if kind != "decode" and 2 * M * N * K < 1e9 or 2 * M * N * K > MOST_FLOPS:
                continue
            break
        c = mm("", M, N, K, "1x16" if kind == "weight" else "16x16", "f32" if kind == "weight" else rng.choice(["bf16", "bf16", "f32"]),
               kind == "weight" and rng.random() < 0.7)
    else:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        colwise = op == "normq" and rng.random() < 0.5
        M, K = log_int(128, 8192, 128) if colwise else log_int(1, 8192), log_int(128, 7168, 128) if op == "normq" else log_int(64, 7168)
        c = norm("", op, M, K, dtype, rng.random() < 0.6, rng.choice([dtype, "f32"]), colwise)
    del c["name"]
    return c


def work(case):
    c = case
    if c["op"] == "mm":
        M, N, K = c["M"], c["N"], c["K"]
        sb_b = N * (K // 16) // (16 if c["blk_b"] == "16x16" else 1)
        es = 2 if c["out"] == "bf16" else 4
        return {"bytes": (M + N) * K // 2 + M * (K // 16) + sb_b + 8 + M * N * es * (2 if c["accumulate"] else 1), "flops": 2 * M * N * K}
    n, es, ws = c["M"] * c["K"], 2 if c["dtype"] == "bf16" else 4, 2 if c["wt"] == "bf16" else 4
    if c["op"] == "grad":   # dy, h, dx, perhaps dh; the weight and its gradient; a row's factor
        return {"bytes": n * es * (4 if c["residual"] else 3) + 2 * ws * c["K"] + 4 * c["M"], "flops": 10 * n}
    read = n * es * (3 if c["residual"] else 1) + ws * c["K"] + 4 * c["M"]   # x, or x, the residual and their sum
    if c["op"] == "norm":
        return {"bytes": read + n * es, "flops": 5 * n}
    dirs = 2 if c["colwise"] else 1
    return {"bytes": read + dirs * (n + 4 * (n // BLOCK)), "flops": (5 + 2 * dirs) * n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)        # between neighbouring E2M1 magnitudes
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def fp4(x, blk):
    """NVFP4 copy of x: packed E2M1 codes (element 2j in the low half), E4M3 block scales (as bytes), the tensor's scale."""
    R, C = x.shape
    h = 16 if blk == "16x16" else 1
    s = x.abs().amax().clamp(min=1e-30) / (6 * FMAX)
    t = x.view(R // h, h, C // 16, 16) / s
    sb = (t.abs().amax(dim=(1, 3)) / 6).clamp(max=FMAX).to(torch.float8_e4m3fn)
    t = t / sb.float().clamp(min=2.0 ** -9)[:, None, :, None]
    codes = torch.bucketize(t.abs(), torch.tensor(BORDERS, device=x.device)).to(torch.uint8) + (t < 0).to(torch.uint8) * 8
    codes = codes.view(R, C // 2, 2)
    return (codes[..., 0] | codes[..., 1] << 4).contiguous(), sb.view(torch.uint8).contiguous(), s.reshape(1)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(shape, std):
        return torch.randn(shape, generator=g, device=DEV) * std

    M, K = c["M"], c["K"]
    # activations and gradients with row magnitudes that differ, weights of a common one
    rows = torch.exp(0.5 * normal((M, 1), 1.0))
    if c["op"] == "mm":
        N = c["N"]
        c["a"], c["sb_a"], c["s_a"] = fp4(normal((M, K), 1.0) * rows, "1x16")
        c["b"], c["sb_b"], c["s_b"] = fp4(normal((N, K), 0.02), c["blk_b"])
        c["type"] = TYPES[c["out"]]
        c["c"] = normal((M, N), 0.1).to(c["type"]) if c["accumulate"] else None
        return c
    c["type"] = TYPES[c["dtype"]]
    c["x"] = (normal((M, K), 1.0) * rows).to(c["type"])
    c["w"] = (1 + normal((K,), 0.1)).to(TYPES[c["wt"]])
    c["r"] = normal((M, K), 1.0).to(c["type"]) if c["residual"] else None
    if c["op"] == "grad":   # x is the sum that was normed, r the gradient of the residual stream behind it
        c["dy"] = normal((M, K), 1.0).to(c["type"])
        c["rstd"] = (c["x"].float().square().mean(1) + EPS).rsqrt()
    return c


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def wide4(q, sb, blk):
    """E2M1 value times block scale, FP32 (exact)."""
    values = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=q.device)
    v = torch.stack((values[(q & 15).long()], values[(q >> 4).long()]), 2).view(q.shape[0], -1)
    s = sb.view(torch.float8_e4m3fn).float()
    h = 16 if blk == "16x16" else 1
    return (v.view(s.shape[0], h, -1, 16) * s[:, None, :, None]).view(v.shape)


def blocks(y):
    """1x128 E4M3 values and FP32 scales of y."""
    t = y.view(y.shape[0], -1, BLOCK)
    b = t.abs().amax(2)
    alpha = torch.where(b == 0, 1.0, torch.full_like(b, FMAX) / b)
    q = (t * alpha[:, :, None]).clamp(-FMAX, FMAX).to(torch.float8_e4m3fn).view(y.shape)
    return q, 1.0 / alpha


def plain(c):
    if c["op"] == "mm":
        y = wide4(c["a"], c["sb_a"], "1x16") @ wide4(c["b"], c["sb_b"], c["blk_b"]).T * c["s_a"] * c["s_b"]
        return c["c"].add_(y) if c["accumulate"] else y.to(c["type"])
    w = c["w"].float()
    if c["op"] == "grad":
        v = c["x"].float() * c["rstd"][:, None]
        dy = c["dy"].float()
        g = dy * w
        dx = c["rstd"][:, None] * (g - v * (g * v).mean(1, keepdim=True))
        dx = dx if c["r"] is None else dx + c["r"].float()
        return dx.to(c["type"]), (dy * v).sum(0).to(c["w"].dtype)
    h = c["x"] if c["r"] is None else (c["x"].float() + c["r"].float()).to(c["type"])
    v = h.float()
    rstd = (v.square().mean(1) + EPS).rsqrt()
    y = v * rstd[:, None] * w
    sums = (rstd,) if c["r"] is None else (h, rstd)
    if c["op"] == "norm":
        return (y.to(c["type"]), *sums)
    return (*blocks(y), *(blocks(y.T.contiguous()) if c["colwise"] else ()), *sums)


# ---------------------------------------------------------------------------
# the library
# ---------------------------------------------------------------------------

def library(c):
    import nvfp4_quantization_current_gb300 as Q

    if c["op"] == "mm":
        return Q.matmul_nvfp4(c["a"], c["sb_a"], c["s_a"], c["b"], c["sb_b"], c["s_b"], "1x16", c["blk_b"], dtype=c["type"], out=c["c"],
                              accumulate=c["accumulate"])
    if c["op"] == "grad":
        return Q.norm_grad(c["dy"], c["x"], c["rstd"], c["w"], dh=c["r"])
    if c["op"] == "norm":
        y, h, rstd = Q.norm_add(c["x"], c["w"], EPS, residual=c["r"])
        return (y, rstd) if c["r"] is None else (y, h, rstd)
    t, h, rstd = Q.norm_q_blockwise(c["x"], c["w"], EPS, residual=c["r"], colwise=c["colwise"])
    out = (t.q_row.view(torch.float8_e4m3fn), t.s_row)
    if c["colwise"]:
        out += (t.q_colT.view(torch.float8_e4m3fn), t.s_colT)
    return (*out, rstd) if c["r"] is None else (*out, h, rstd)


def run(state):
    return library(state) if own else plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def to_e4m3(v):
    """Nearest E4M3 value, ties to even, of 64-bit v with |v| <= 448 (up to its own rounding)."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-FMAX, FMAX)


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "mm":
        def values(q, sb, rows):
            # magnitude of a 4-bit code from its fields: (1 + m/2) 2^(e - 1), or m/2 where the exponent field is zero
            n = torch.stack((q & 15, q >> 4), 2).flatten(1).double()
            sign = 1 - 2 * torch.floor(n / 8)
            e, m = torch.floor(n % 8 / 2), n % 2
            v = sign * torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e - 1))
            return v * sb.view(torch.float8_e4m3fn).double().repeat_interleave(rows, 0).repeat_interleave(16, 1)

        y = values(c["a"], c["sb_a"], 1) @ values(c["b"], c["sb_b"], 16 if c["blk_b"] == "16x16" else 1).T
        y = y * (c["s_a"].double() * c["s_b"].double())
        return y + c["c"].double() if c["accumulate"] else y
    x, w = c["x"].double(), c["w"].double()
    if c["op"] == "grad":
        # through the norm's Jacobian: d(x_j s)/dx_i = s d_ij - s^3 x_i x_j / K
        s = c["rstd"].double()[:, None]
        dy = c["dy"].double()
        g = dy * w
        dx = s * g - s ** 3 * x * ((g * x).sum(1, keepdim=True) / x.shape[1])
        return (dx if c["r"] is None else dx + c["r"].double()), torch.einsum("mk,mk->k", dy, x * s)
    h = x if c["r"] is None else (x + c["r"].double()).to(c["type"]).double()   # the sum as it is kept
    s = 1 / torch.sqrt((h * h).sum(1) / h.shape[1] + EPS)
    y = h * s[:, None] * w
    sums = (s,) if c["r"] is None else (h, s)
    if c["op"] == "norm":
        return (y, *sums)

    def cast(v):
        t = v.unflatten(1, (-1, BLOCK))
        sc = t.abs().amax(2) / FMAX
        sc = torch.where(sc == 0, 1.0, sc)
        return to_e4m3(t / sc[..., None]).flatten(1), sc

    return (*cast(y), *(cast(y.T) if c["colwise"] else ()), *sums)
