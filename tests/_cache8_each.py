"""Attention over the 8-bit cache in 64 bits with a bound for every output by
itself, and inputs whose outputs say which tokens were counted."""
from __future__ import annotations

import torch

from tests import _cache8_ref as ref

D, BLOCK = 128, 16


def units(scale, tail, length):
    """The V unit of each token of one sequence [H, length]: its block's scale,
    or the power of two above the largest value of the partial block."""
    full = length // BLOCK * BLOCK
    u = scale[:, :full // BLOCK].double().repeat_interleave(BLOCK, 1)
    rest = tail[:, :length - full].double()
    if length > full:
        e = torch.frexp(rest.abs().amax((1, 2)))[1].double()
        u = torch.cat((u, (2.0 ** e)[:, None].expand(-1, length - full)), 1)
    return u


def attend(q, k, v, u, count, scale, window, sinks, dtype):
    """q [H, n, 128], k, v [H_kv, length, 128], u [H_kv, length], all fp64 ->
    the output [H, n, 128] and the largest error of each of its values.

    p the softmax, P = sum_j p_j |v_jd| the magnitudes that an output sums.
    - A score is off by at most d: 2^-18 of sum |q_d k_d| |scale| (its products'
      sums), 2^-24 of the row's largest |q_d| for each |k_d| and of the tail's
      largest |k_d| for each |q_d| (fp16 operands in units of those), and
      2^-22 (2 size + the binary orders between the V units + 16) (exp2, its
      rounded argument and the logarithm of a V scale). The weights and their
      total are then off by factors exp(+-d): expm1(2 d) P.
    - Weights in P V: bf16 caches hold them in fp16, 2^-11 of themselves or,
      where small, 2^-31 of the largest p_j u_j of the row, u_j the token's V
      unit, so the sum of |v_jd| / u_j times that; tails in fp16 as well, 2^-25
      of their unit. fp32 caches: 2^-23.
    - V units below 2^-90 of the largest (0 among them) may be taken for that:
      what they hold is below 2^-80 of the largest unit.
    - Sums over blocks, in fp32: (length / 16 + 40) 2^-23 of P and of the total.
    - One rounding to dtype."""
    h, n, _ = q.shape
    hkv, length, _ = k.shape
    out, lim = torch.zeros_like(q), torch.zeros_like(q)
    if length == 0 or count == 0:
        return out, lim
    g = h // hkv
    full = length // BLOCK * BLOCK
    kk, vv, uu = (t.repeat_interleave(g, 0) for t in (k, v, u))
    qq = q[:, :count]
    x = qq @ kk.transpose(1, 2) * scale
    size = qq.abs() @ kk.abs().transpose(1, 2) * abs(scale)
    size_of = size * 2.0 ** -18 + qq.abs().amax(-1, keepdim=True) * kk.abs().sum(-1)[:, None] * (abs(scale) * 2.0 ** -24)
    if length > full:
        size_of[..., full:] += kk[:, full:].abs().amax((1, 2))[:, None, None] * qq.abs().sum(-1, keepdim=True) * (abs(scale) * 2.0 ** -24)
    pos = length - count + torch.arange(count)[:, None]
    j = torch.arange(length)[None]
    see = j <= pos
    if window:
        see &= (j > pos - window) | (j < sinks)
    top = x.masked_fill(~see, float("-inf")).amax(-1, keepdim=True)
    p = torch.exp((x - torch.where(top > float("-inf"), top, 0.0)).masked_fill(~see, float("-inf")))
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-300)
    any_seen = see.any(-1).to(q.dtype)[None, :, None]
    out[:, :count] = p @ vv
    P = p @ vv.abs()
    umax = u.max().item()
    low = u[u > 0].min().item() if umax > 0 else 1.0
    span = float(torch.log2(torch.tensor(umax / low))) if umax > 0 else 0.0
    below = 2.0 ** -80 * umax if span > 90 or (u == 0).any() else 0.0
    most = (size * see).amax(-1, keepdim=True)
    d = (size_of * see).amax(-1, keepdim=True) + (2 * most + min(span, 90.0) + 16) * 2.0 ** -22
    e = torch.expm1(2 * d) * P + (length / 16 + 40) * 2.0 ** -23 * (P + out[:, :count].abs()) + below * any_seen
    if dtype == torch.bfloat16:
        code = torch.where(uu > 0, 1 / torch.where(uu > 0, uu, 1.0), 0.0)[..., None] * vv.abs()
        e += 2.0 ** -11 * P + 2.0 ** -31 * (p * uu[:, None]).amax(-1, keepdim=True) * (see.to(p.dtype) @ code)
        if length > full:
            e += 2.0 ** -25 * (p[..., full:].sum(-1, keepdim=True) * uu[:, full:].amax(-1)[:, None, None])
    else:
        e += 2.0 ** -23 * P
    e += (out[:, :count].abs() + e) * ref.half_step(dtype)
    lim[:, :count] = e + torch.finfo(dtype).tiny
    return out, lim


def one_hot(length, kind):
    """Values [length, 128] that tell the blocks apart: a block's channel (block
    * 37 % 128) holds its height, 1 to 7 by the block, in every token."""
    b = torch.arange(length) // BLOCK
    v = torch.zeros(length, D, dtype=kind)
    v[torch.arange(length), b * 37 % D] = (1 + b % 7).to(kind)
    return v


def one_hot_bound(want, dtype, length):
    """Equal scores: a weight is 2^(y - reference) with the same y for every
    token of a height, off by 2^-11 of itself (bf16: fp16 weights; none is
    small, the heights being within a factor of 7) or 2^-23, the logarithm,
    exp2 and reciprocal of the V scales by 2^-18 (magnitudes below 4), the
    heights' codes by half a step of the scale's rounding, 2^-24; sums as
    above. All terms of an output are positive, so each is a share of it."""
    w = 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -23
    share = w + 2.0 ** -18 + 2.0 ** -24 + 2 * (length / 16 + 40) * 2.0 ** -23
    return want.abs() * (share + ref.half_step(dtype) * (1 + share))
