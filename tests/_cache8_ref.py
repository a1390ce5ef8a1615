"""Plain 64-bit forms of the 8-bit cache and of rotary positions, on the CPU,
and the error bounds that the tests hold the kernels to."""
from __future__ import annotations

import math

import torch

D, BLOCK = 128, 16
TOP = {"int8": 127.0, "e4m3": 448.0}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def half_step(dtype) -> float:
    """Relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def rope_rates(rd, base=10000.0, scaling="none", factor=1.0, orig_len=0, beta_fast=32.0, beta_slow=1.0):
    if scaling == "ntk":
        base = base * factor ** (rd / (rd - 2))
    f = [base ** (-2 * i / rd) for i in range(rd // 2)]
    gain = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "yarn":
        gain = 0.1 * math.log(factor) + 1
        keep = [min(1.0, max(0.0, (orig_len * x / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow))) for x in f]
        f = [x * (g + (1 - g) / factor) for x, g in zip(f, keep)]
    return torch.tensor(f, dtype=torch.float64), gain


def rope(x, positions, rates, gain, layout):
    """x [B, H, n, 128], positions [B, n] -> fp64, and |x1| + |x2| of each value's pair."""
    y = x.double().clone()
    size = torch.zeros_like(y)
    a = positions.double()[:, None, :, None] * rates
    c, s = a.cos() * gain, a.sin() * gain
    h = len(rates)
    one, two = (slice(0, h), slice(h, 2 * h)) if layout == "half" else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
    p, q = y[..., one].clone(), y[..., two].clone()
    y[..., one], y[..., two] = p * c - q * s, q * c + p * s
    size[..., one] = size[..., two] = (p.abs() + q.abs()) * gain
    return y, size


def e4m3(y):
    """The nearest e4m3 value, ties to the even code (fp64)."""
    a = y.abs()
    e = torch.frexp(a.clamp_min(2.0 ** -6))[1].double() - 1
    step = 2.0 ** (e - 3)
    return torch.copysign(torch.round(a / step) * step, y)


def quantise(x, fmt):
    """x [..., 16, 128] fp64 (finite) -> codes (as values, fp64) and fp32 scales [...]."""
    amax = x.abs().amax((-2, -1))
    y = x * TOP[fmt] / torch.where(amax > 0, amax, 1.0)[..., None, None]
    code = torch.round(y) if fmt == "int8" else e4m3(y)
    code = torch.where((amax > 0)[..., None, None], code, 0.0)  # not minus zero
    return code, amax.float() / torch.tensor(TOP[fmt], dtype=torch.float32)


def held(rows, fmt, dtype, capacity, lengths, garbage=None):
    """The cache's arrays for rows [B, H, n, 128] (values of dtype), of which
    lengths[b] are held; what lies behind a sequence is garbage (a Generator)
    or zero. Returns codes, scale, tail (CPU)."""
    b, h, n, _ = rows.shape
    code = torch.zeros(b, h, capacity, D, dtype=torch.int8)
    scale = torch.zeros(b, h, capacity // BLOCK)
    tail = torch.zeros(b, h, BLOCK, D, dtype=dtype)
    if garbage is not None:  # every byte, e4m3's NaNs among them; NaN scales and tails
        code = torch.randint(-128, 128, code.shape, generator=garbage, dtype=torch.int8)
        scale.fill_(float("nan"))
        tail.fill_(float("nan"))
    for s, length in enumerate(lengths):
        full = length // BLOCK
        if full:
            c, u = quantise(rows[s, :, :full * BLOCK].double().unflatten(1, (full, BLOCK)), fmt)
            code[s, :, :full * BLOCK] = c.flatten(1, 2).float().to(CODE[fmt]).view(torch.int8)
            scale[s, :, :full] = u
        if length:
            at = (length - 1) // BLOCK * BLOCK
            tail[s, :, :length - at] = rows[s, :, at:length].to(dtype)
    return code.view(CODE[fmt]), scale, tail


def values(code, scale, tail, length):
    """What one sequence's arrays [H, ...] stand for: [H, length, 128] fp64."""
    full = length // BLOCK * BLOCK
    x = code[:, :full].float().double() * scale[:, :full // BLOCK].double().repeat_interleave(BLOCK, 1)[..., None]
    return torch.cat((x, tail[:, :length - full].double()), 1)


def attend(q, k, v, count, scale, window, sinks):
    """q [H, n, 128], k, v [H_kv, length, 128] fp64 -> out [H, n, 128], and
    for the bounds: the largest sum |q_d k_d| |scale| and the largest |v|."""
    h, n, _ = q.shape
    hkv, length, _ = k.shape
    out = torch.zeros_like(q)
    if length == 0 or count == 0:
        return out, 0.0, 0.0
    g = h // hkv
    kk, vv = k.repeat_interleave(g, 0), v.repeat_interleave(g, 0)
    x = q[:, :count] @ kk.transpose(1, 2) * scale
    size = (q[:, :count].abs() @ kk.abs().transpose(1, 2)).max().item() * abs(scale)
    pos = length - count + torch.arange(count)[:, None]
    j = torch.arange(length)[None]
    see = j <= pos
    if window:
        see &= (j > pos - window) | (j < sinks)
    x = x.masked_fill(~see, float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top > float("-inf"), top, 0.0)).masked_fill(~see, 0.0)
    total = p.sum(-1, keepdim=True)
    out[:, :count] = (p @ vv) / torch.where(total > 0, total, 1.0)
    return out, size, vv.abs().max().item()


def attend_bound(want, dtype, size, vmax, length):
    """Largest error of an attention output.

    A score is a product of fp16 operands that hold the query to 2^-23 of its
    row's largest value and the codes exactly, summed in fp32 over 8 products
    of 16 terms (each sum off by at most 2^-22 of the magnitudes it holds:
    tensor-core sums may truncate) and scaled by three rounded factors: off by
    at most 2^-18 of sum |q k| |scale| =: size. An error d of the scores moves
    an average of values by at most 2 d vmax (both the weight and the total).
    exp2 and its rounded argument, the logarithm of a V scale in units of the
    largest one among it (magnitudes below 2 size + 16 for scales within 2^16
    of each other), add 2^-22 (2 size + 16) to each weight. Sums over the blocks: one fp32 rounding
    a block and merge, length / 16 + 40 of them, 2^-23 each. Weights in fp16
    (bf16 caches) are off by 2^-11 of themselves, and by 2^-31 of the largest
    weight where they are tiny; with remainders (fp32) by 2^-22. Then one
    rounding to dtype."""
    d = size * 2.0 ** -18 + (2 * size + 16) * 2.0 ** -22
    w = (2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -22) + length * 2.0 ** -30
    return vmax * (2 * d + 2 * w + (length / 16 + 40) * 2.0 ** -23) + want.abs() * half_step(dtype)
