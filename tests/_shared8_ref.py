"""Attention behind shared prefixes in 64 bits, with a bound for every output."""
from __future__ import annotations

import torch

from tests import _cache8_each as each
from tests import _cache8_ref as ref

BLOCK = ref.BLOCK


def sequence(k, v, b, length):
    """One sequence's keys, values, V units and which of its tokens are in the partial block, from arrays of ref.held."""
    kk, vv = (ref.values(a[0][b], a[1][b], a[2][b], length) for a in (k, v))
    return kk, vv, each.units(v[1][b], v[2][b], length), torch.arange(length) >= length // BLOCK * BLOCK


def attend(q, parts, count, scale, dtype):
    """q [H, n, 128] fp64, parts [(k, v, u, tail)] of the sequences that make up the tokens, in order -> the output and
    the largest error of each of its values.

    The bound is that of each.attend, term by term, with two partial blocks in place of one (a token's key, value and
    unit are those of its own), and with the parts that CTAs leave and that are joined: their sums round once a part as
    they do once a block, and a token's part is at least a block: twice length / 16 roundings, and 40 of merges."""
    h, n, _ = q.shape
    k, v = (torch.cat([p[i] for p in parts], 1) for i in (0, 1))
    u, tail = torch.cat([p[2] for p in parts], 1), torch.cat([p[3] for p in parts])
    length = k.shape[1]
    out, lim = torch.zeros_like(q), torch.zeros_like(q)
    if length == 0 or count == 0:
        return out, lim
    g = h // k.shape[0]
    kk, vv, uu = (t.repeat_interleave(g, 0) for t in (k, v, u))
    # the largest key value of a token's partial block, 0 for codes
    top_k = torch.cat([torch.where(p[3], (p[0] * p[3][None, :, None]).abs().amax((1, 2), keepdim=True)[..., 0], 0.0) if p[0].shape[1] else p[0][..., 0]
                       for p in parts], 1).repeat_interleave(g, 0)
    qq = q[:, :count]
    x = qq @ kk.transpose(1, 2) * scale
    size = qq.abs() @ kk.abs().transpose(1, 2) * abs(scale)
    size_of = size * 2.0 ** -18 + qq.abs().amax(-1, keepdim=True) * kk.abs().sum(-1)[:, None] * (abs(scale) * 2.0 ** -24)
    size_of = size_of + top_k[:, None] * qq.abs().sum(-1, keepdim=True) * (abs(scale) * 2.0 ** -24)
    see = torch.arange(length)[None] <= length - count + torch.arange(count)[:, None]
    top = x.masked_fill(~see, float("-inf")).amax(-1, keepdim=True)
    p = torch.exp((x - torch.where(top > float("-inf"), top, 0.0)).masked_fill(~see, float("-inf")))
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-300)
    out[:, :count] = p @ vv
    P = p @ vv.abs()
    umax = u.max().item()
    low = u[u > 0].min().item() if umax > 0 else 1.0
    span = float(torch.log2(torch.tensor(umax / low))) if umax > 0 else 0.0
    below = 2.0 ** -80 * umax if span > 90 or (u == 0).any() else 0.0
    most = (size * see).amax(-1, keepdim=True)
    d = (size_of * see).amax(-1, keepdim=True) + (2 * most + min(span, 90.0) + 16) * 2.0 ** -22
    e = torch.expm1(2 * d) * P + (length / 8 + 40) * 2.0 ** -23 * (P + out[:, :count].abs()) + below * see.any(-1)[None, :, None]
    if dtype == torch.bfloat16:
        code = torch.where(uu > 0, 1 / torch.where(uu > 0, uu, 1.0), 0.0)[..., None] * vv.abs()
        e += 2.0 ** -11 * P + 2.0 ** -31 * (p * uu[:, None]).amax(-1, keepdim=True) * (see.to(p.dtype) @ code)
        e += 2.0 ** -25 * (p * (uu * tail)[:, None]).sum(-1, keepdim=True)
    else:
        e += 2.0 ** -23 * P
    e += (out[:, :count].abs() + e) * ref.half_step(dtype)
    lim[:, :count] = e + torch.finfo(dtype).tiny
    return out, lim
