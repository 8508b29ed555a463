"""Plain 64-bit forms of the 8-bit cache format and of softmax attention, with
the error bounds that the kernels' own roundings allow, for the tests of the
quantised cache and of the shared prefix. They share no code with the library."""
from __future__ import annotations

import math

import torch

D = 128
INT8, E4M3 = torch.int8, torch.float8_e4m3fn
DTYPES = [E4M3, INT8]
IDS = ["e4m3", "int8"]
FLOOR = 2.0 ** -100
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2
HALF_F16 = torch.finfo(torch.float16).eps / 2
HALF_F32 = torch.finfo(torch.float32).eps / 2


def e4m3_grid():
    """Every finite e4m3 value >= 0, ascending: index = code."""
    out = []
    for code in range(0x7f):
        e, m = code >> 3, code & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return torch.tensor(out, dtype=torch.float64)


def quantise(x, dtype):
    """(values of the codes, scales fp32) of bf16 rows, from the format's definition."""
    x = x.double()
    bad = ~torch.isfinite(x).all(-1)
    top = torch.where(bad, torch.ones_like(x[..., 0]), x.abs().amax(-1)).clamp_min(FLOOR)
    y0 = torch.where(bad[..., None], torch.zeros_like(x), x)
    if dtype == INT8:
        codes = torch.round(127 * y0 / top[..., None])  # fp64 holds every tie exactly
        scale = (top.float() / torch.tensor(127.0, device=x.device)).float()
    else:
        n = torch.ceil(torch.log2(top / 448))
        n = torch.where(top * torch.exp2(-n) > 448, n + 1, n)
        n = torch.where(top * torch.exp2(-n) <= 224, n - 1, n)
        y = y0 * torch.exp2(-n)[..., None]
        grid = e4m3_grid().to(x.device)
        a = y.abs().contiguous()
        hi = torch.searchsorted(grid, a).clamp_max(grid.numel() - 1)
        lo = (hi - 1).clamp_min(0)
        dl, dh = a - grid[lo], grid[hi] - a
        even = torch.where(lo % 2 == 0, lo, hi)
        pick = torch.where(dl < dh, lo, torch.where(dh < dl, hi, even))
        codes = grid[pick] * torch.sign(y)
        scale = torch.exp2(n).float()
    nan = torch.full_like(scale, math.nan)
    return codes, torch.where(bad, nan, scale)


def attention(q, k, v, n):
    """Softmax attention of rows q [r, d] over the first n rows of k, v (64 bits):
    (o [r, d], lse [r], a [r, d] = sum_j p_j |v_j|, delta [r] = bound of a logit's
    relative rounding: 130 fp32 roundings of sum_i |q_i k_i| / sqrt(d))."""
    q, k, v = q.double(), k[:n].double(), v[:n].double()
    if n == 0:
        z = torch.zeros_like(q)
        return z, torch.full(q.shape[:1], -math.inf, dtype=torch.float64, device=q.device), z, z[:, 0]
    s = q @ k.T / math.sqrt(D)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - top)
    tot = e.sum(-1, keepdim=True)
    p = e / tot
    delta = 130 * HALF_F32 * ((q.abs() @ k.abs().T) / math.sqrt(D)).amax(-1)
    return p @ v, (top + torch.log(tot))[:, 0], p @ v.abs(), delta


def join(parts):
    """Union of attention() results over disjoint position ranges."""
    lse = torch.stack([p[1] for p in parts])
    tot = torch.logsumexp(lse, 0)
    w = torch.where(torch.isinf(lse), torch.zeros_like(lse), torch.exp(lse - tot))[..., None]
    return (sum(wi * p[0] for wi, p in zip(w, parts)), tot, sum(wi * p[2] for wi, p in zip(w, parts)),
            torch.stack([p[3] for p in parts]).amax(0))


def bound(o, a, delta, weight_half_step, out_half_step, under=0.0):
    """Elementwise bound of |kernel - o|: the output's rounding, the weights'
    rounding (relative to a = sum p |v|), the logits' rounding on both the weights
    and the denominator (e^(2 delta) - 1), 2^-16 for exp2, the running rescales
    and the fp32 sums, and ``under`` for weights below the format's range."""
    rel = weight_half_step + torch.expm1(2 * delta)[:, None] + 2.0 ** -16
    return out_half_step * o.abs() + (1 + out_half_step) * (a * rel + under) + 1e-30


def lse_bound(lse, delta):
    """|kernel lse - lse|: the logits' rounding, 2^-16 relative in the sum, fp32's
    own rounding of the result."""
    return delta + 2.0 ** -16 + HALF_F32 * 4 * lse.abs()
