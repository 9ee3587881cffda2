"""The operators of a blockwise FP8 linear layer as cases to be timed and compared: the block-scaled
matrix product in its directions, dropout with the residual sum, and dropout fused into the blockwise
cast of a gradient.

Each case runs in a plain form of elementary torch operations (``own`` false) or through the
library's entry points (``own`` true).  Sizes are those of the library's workloads (hidden 4096 with
FFN 14336 and sequence 8192; a 7168 / 18432 layer) plus single tokens, ragged and odd ones.

Plain dropout draws the same numbers as the library: element i of the tensor takes 16 bits of
Philox4x32-10 block offset + i / 8 (key: the seed; third counter word 2), low half of a word first.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 128
FMAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def mm(name, M, N, K, tile_b="128x128", out="bf16", accumulate=False):
    return {"name": name, "op": "mm", "M": M, "N": N, "K": K, "tile_b": tile_b, "out": out, "accumulate": accumulate}


def drop(name, M, K, dtype, p, residual):
    return {"name": name, "op": "drop", "M": M, "K": K, "dtype": dtype, "p": p, "residual": residual}


def dropq(name, M, K, dtype, p, colwise):
    return {"name": name, "op": "dropq", "M": M, "K": K, "dtype": dtype, "p": p, "colwise": colwise}


def listed():
    return [
        # one token through a 4096 x 4096 projection: the smallest call, latency
        mm("decode 1 token", 1, 4096, 4096),
        # a batch of sixteen sequences decoding through an FFN matrix: the weights' bytes
        mm("decode 16 tokens ffn", 16, 14336, 4096),
        # a ragged prompt chunk: rows that fill no tile, few tiles for the machine
        mm("prefill 333 tokens", 333, 4096, 4096),
        # forward of the FFN up-projection over a whole sequence
        mm("forward ffn", 8192, 14336, 4096),
        # gradient of the input of that projection (long reduction)
        mm("input gradient ffn", 8192, 4096, 14336),
        # weight gradient added into the FP32 main gradient; both operands with 1x128 scales
        mm("weight gradient ffn", 14336, 4096, 8192, "1x128", "f32", True),
        # forward of the 7168 / 18432 layer over 16384 tokens: the largest
        mm("forward 7168 18432", 16384, 18432, 7168),
        # a short fine-tuning batch: dropout's smallest call
        drop("dropout 128 rows", 128, 4096, "bf16", 0.1, True),
        # residual dropout of a whole sequence
        drop("dropout add sequence", 8192, 4096, "bf16", 0.1, True),
        # backward of dropout in FP32 on an odd shape
        drop("dropout backward odd f32", 3001, 1111, "f32", 0.25, False),
        # output gradient of a sequence: dropout backward and both FP8 copies for dgrad and wgrad
        dropq("dropout cast both", 8192, 4096, "bf16", 0.1, True),
        # the rowwise copy alone of a ragged FP32 gradient
        dropq("dropout cast ragged f32", 1000, 4096, "f32", 0.1, False),
    ]


MOST_FLOPS = 2 * 16384 * 18432 * 7168


def draw(rng):
    def log_int(lo, hi, step=1):
        v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))) // step * step
        return max(lo, min(hi, v + step if v == 3 * 1024 else v))

    op = rng.choice(["mm", "mm", "mm", "drop", "dropq"])
    if op == "mm":
        kind = rng.choice(["decode", "forward", "forward", "weight"])
        while True:
            N, K = log_int(128, 18432, 128), log_int(128, 18432, 128)
            M = log_int(1, 128) if kind == "decode" else log_int(129, 16384) if kind == "forward" else log_int(128, 18432, 128)
            if kind != "decode" and 2 * M * N * K < 1e9 or 2 * M * N * K > MOST_FLOPS // 2:
                continue
            break
        c = mm("", M, N, K, "1x128" if kind == "weight" else "128x128", "f32" if kind == "weight" else rng.choice(["bf16", "bf16", "f32"]),
               kind == "weight" and rng.random() < 0.7)
    elif op == "drop":
        c = drop("", log_int(1, 16384), log_int(64, 7168), rng.choice(["bf16", "f32"]), round(rng.uniform(0.02, 0.6), 3), rng.random() < 0.6)
    else:
        both = rng.random() < 0.6
        c = dropq("", log_int(128, 16384, 128) if both else log_int(1, 16384), log_int(128, 7168, 128), rng.choice(["bf16", "f32"]),
                  round(rng.uniform(0.02, 0.6), 3), both)
    del c["name"]
    return c


def work(case):
    c = case
    if c["op"] == "mm":
        M, N, K = c["M"], c["N"], c["K"]
        s_b = N * (K // BLOCK) if c["tile_b"] == "1x128" else (N // BLOCK) * (K // BLOCK)
        es = 2 if c["out"] == "bf16" else 4
        return {"bytes": M * K + N * K + 4 * (M * (K // BLOCK) + s_b) + M * N * es * (2 if c["accumulate"] else 1), "flops": 2 * M * N * K}
    n, es = c["M"] * c["K"], 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "drop":
        return {"bytes": n * es * (3 if c["residual"] else 2), "flops": 2 * n}
    dirs = 2 if c["colwise"] else 1
    return {"bytes": n * es + dirs * (n + 4 * (n // BLOCK)), "flops": 3 * dirs * n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def quantized(x, tile):
    """E4M3 codes (uint8) and FP32 scales of x: one scale per 1x128 or 128x128 tile, largest magnitude to 448."""
    R, C = x.shape
    h = BLOCK if tile == "128x128" else 1
    t = x.view(R // h, h, C // BLOCK, BLOCK)
    s = t.abs().amax(dim=(1, 3)) / FMAX
    q = (t / s[:, None, :, None]).clamp(-FMAX, FMAX).to(torch.float8_e4m3fn)
    return q.view(R, C).view(torch.uint8), s.contiguous()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(shape, std):
        return torch.randn(shape, generator=g, device=DEV) * std

    if c["op"] == "mm":
        M, N, K = c["M"], c["N"], c["K"]
        # activations and gradients with row magnitudes that differ, weights of a common one
        rows = torch.exp(0.5 * normal((M, 1), 1.0))
        c["a"], c["s_a"] = quantized(normal((M, K), 1.0) * rows, "1x128")
        c["b"], c["s_b"] = quantized(normal((N, K), 0.02), c["tile_b"])
        c["type"] = torch.bfloat16 if c["out"] == "bf16" else torch.float32
        c["c"] = normal((M, N), 0.1).to(c["type"]) if c["accumulate"] else None
        return c
    M, K = c["M"], c["K"]
    c["type"] = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    c["x"] = normal((M, K), 1.0).to(c["type"])
    if c["op"] == "dropq":
        c["x"][: M // 64] = 0   # rows without a gradient (padding tokens)
    c["r"] = normal((M, K), 1.0).to(c["type"]) if c.get("residual") else None
    c["seed"] = int(seed) * 0x9E3779B97F4A7C15 % (1 << 63)
    c["offset"] = int(seed) % 1000003
    return c


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

MASK32 = 0xFFFFFFFF


def wide(m, x):
    """High and low halves of the 64-bit product of the constant m and 32-bit x (int64 tensors)."""
    low = m * (x & 0xFFFF)
    t = m * (x >> 16) + (low >> 16)
    return t >> 16, (t & 0xFFFF) << 16 | low & 0xFFFF


def philox(g, seed):
    """Philox4x32-10 of counters (g lo, g hi, 2, 0): an int64 tensor [len(g), 4] of 32-bit words."""
    c0, c1, c2, c3 = g & MASK32, g >> 32, torch.full_like(g, 2), torch.zeros_like(g)
    k0, k1 = seed & MASK32, seed >> 32
    for _ in range(10):
        h0, l0 = wide(0xD2511F53, c0)
        h1, l1 = wide(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & MASK32, (k1 + 0xBB67AE85) & MASK32
    return torch.stack((c0, c1, c2, c3), 1)


def dropped(c):
    """keep * x / (1 - p) in FP32, p to the nearest 1/65536."""
    n = c["x"].numel()
    words = philox(c["offset"] + torch.arange((n + 7) // 8, device=DEV), c["seed"])
    draws = torch.stack((words & 0xFFFF, words >> 16), 2).flatten()[:n].view_as(c["x"])
    T = round(c["p"] * 65536)
    return torch.where(draws >= T, c["x"].float() * (65536 / (65536 - T)), 0.0)


def blocks(y):
    """1x128 E4M3 values and FP32 scales of y."""
    t = y.view(y.shape[0], -1, BLOCK)
    b = t.abs().amax(2)
    alpha = torch.where(b == 0, 1.0, torch.full_like(b, FMAX) / b)
    q = (t * alpha[:, :, None]).clamp(-FMAX, FMAX).to(torch.float8_e4m3fn).view(y.shape)
    return q, 1.0 / alpha


def plain(c):
    if c["op"] == "mm":
        K, hb = c["K"], BLOCK if c["tile_b"] == "128x128" else 1
        a = c["a"].view(torch.float8_e4m3fn).float().view(c["M"], -1, BLOCK) * c["s_a"][:, :, None]
        b = c["b"].view(torch.float8_e4m3fn).float().view(c["N"] // hb, hb, -1, BLOCK) * c["s_b"][:, None, :, None]
        y = a.view(-1, K) @ b.view(-1, K).T
        if c["accumulate"]:
            return c["c"].add_(y)
        return y.to(c["type"])
    y = dropped(c)
    if c["op"] == "drop":
        return (y if c["r"] is None else y + c["r"].float()).to(c["type"])
    out = blocks(y)
    return (*out, *blocks(y.T.contiguous())) if c["colwise"] else out


# ---------------------------------------------------------------------------
# the library
# ---------------------------------------------------------------------------

def library(c):
    import nvfp4_quantization_current_gb300 as Q

    if c["op"] == "mm":
        return Q.mm_blockwise(c["a"], c["s_a"], c["b"], c["s_b"], "1x128", c["tile_b"], dtype=c["type"], out=c["c"], accumulate=c["accumulate"])
    if c["op"] == "drop":
        return Q.drop_add(c["x"], c["p"], c["seed"], c["offset"], residual=c["r"])
    t = Q.drop_q_blockwise(c["x"], c["p"], c["seed"], c["offset"], colwise=c["colwise"])
    out = (t.q_row.view(torch.float8_e4m3fn), t.s_row)
    return (*out, t.q_colT.view(torch.float8_e4m3fn), t.s_colT) if c["colwise"] else out


def run(state):
    return library(state) if own else plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def kept(n, offset, seed, T):
    """Truth values [n]: which elements the draws keep (numpy, unsigned 64-bit products)."""
    g = np.arange(offset, offset + -(-n // 8), dtype=np.uint64)
    low, half = np.uint64(MASK32), np.uint64(32)
    ctr = [g & low, g >> half, np.full_like(g, 2), np.zeros_like(g)]
    key = [seed % 2**32, seed // 2**32]
    for _ in range(10):
        p, q = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(q >> half) ^ ctr[1] ^ np.uint64(key[0]), q & low, (p >> half) ^ ctr[3] ^ np.uint64(key[1]), p & low]
        key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
    words = np.empty((len(g), 4), np.uint32)
    for i in range(4):
        words[:, i] = ctr[i]
    return torch.from_numpy((words.view("<u2").reshape(-1)[:n] >= T) if T < 65536 else np.zeros(n, bool))


def to_e4m3(v):
    """Nearest E4M3 value, ties to even, of 64-bit v with |v| <= 448 (up to its own rounding)."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-FMAX, FMAX)


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "mm":
        def values(q, s, rows):
            wide_s = s.double().repeat_interleave(rows, 0).repeat_interleave(BLOCK, 1)
            return wide_s.mul_(q.view(torch.float8_e4m3fn).double())

        y = values(c["a"], c["s_a"], 1) @ values(c["b"], c["s_b"], BLOCK if c["tile_b"] == "128x128" else 1).T
        return y + c["c"].double() if c["accumulate"] else y
    x, T = c["x"].double(), round(c["p"] * 65536)
    y = x * kept(x.numel(), c["offset"], c["seed"], T).to(DEV).view_as(x) * (65536 / (65536 - T))
    if c["op"] == "drop":
        return y if c["r"] is None else y + c["r"].double()

    def cast(v):
        t = v.unflatten(1, (-1, BLOCK))
        s = t.abs().amax(2) / FMAX
        s = torch.where(s == 0, 1.0, s)
        return to_e4m3(t / s[..., None]).flatten(1), s

    return (*cast(y), *cast(y.T)) if c["colwise"] else cast(y)
