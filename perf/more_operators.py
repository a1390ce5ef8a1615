"""Operators for many samples of one prompt over the 8-bit cache, case by case: inputs, plain forms, the library's calls.

Layouts are head-major, as everywhere in the library: q [B, H, n, 128], a cache's codes [B, H_kv, capacity, 128] with a
scale for each 16 tokens of a (sequence, KV head) and the last block in full precision beside them.

  axes    rotary positions with several axes: pair i of a row's first `rd` values turns by the position on axis(i) times
          its frequency; positions [A, B, n].
  shared  causal softmax attention of the last n tokens of each sequence, which are those of a prefix that many sequences
          share, then the sequence's own.
  take    sequence b of a cache becomes the first lengths[b] tokens of sequence sequences[b] of another cache, or of its
          own; -1 leaves it as it is.
  keep    sequence b of a cache becomes counts[b] whole blocks of sequence b of another one, a list for each KV head, and
          then its last, partial block.
"""
import math

import torch

own = False

D = 128       # values of a head's row
BLOCK = 16    # tokens that share a scale
TOP = {"int8": 127.0, "e4m3": 448.0}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 32 sequences behind a video: latency of the smallest call
        dict(name="axes_step", op="axes", dtype="bf16", batch=32, heads=32, kv_heads=8, n=1, rd=128, layout="half", axes=3,
             spread="runs", apart=False, base=1000000.0),
        # a video prompt's queries and keys: time, height and width by turns
        dict(name="axes_video", op="axes", dtype="bf16", batch=1, heads=32, kv_heads=8, n=32768, rd=128, layout="half", axes=3,
             spread="turns", apart=False, base=5000000.0),
        # the patches of four images of odd size, rows and columns with frequencies of their own
        dict(name="axes_image", op="axes", dtype="fp32", batch=4, heads=16, kv_heads=16, n=1369, rd=128, layout="interleaved",
             axes=2, spread="runs", apart=True, base=10000.0),
        # the smallest shared attention: a few samples of one short prompt, one step
        dict(name="shared_small", op="shared", fmt="e4m3", dtype="bf16", batch=4, kv_heads=8, group=4, n=1, prefixes=1, shared=2048,
             lone=0, at=100, skew=13),
        # the decode step of 32 samples of a 32K prompt, some hundred tokens in
        dict(name="shared_step", op="shared", fmt="int8", dtype="bf16", batch=32, kv_heads=8, group=4, n=1, prefixes=1, shared=32768,
             lone=0, at=767, skew=11),
        # three prompts of unequal length, drafts of three tokens, and sequences of their own
        dict(name="shared_drafts", op="shared", fmt="e4m3", dtype="bf16", batch=27, kv_heads=4, group=8, n=3, prefixes=3, shared=12001,
             lone=3, at=1500, skew=41),
        # questions of 256 tokens behind a long document, prefilled together: products
        dict(name="shared_chunk", op="shared", fmt="int8", dtype="bf16", batch=8, kv_heads=8, group=4, n=256, prefixes=1, shared=16384,
             lone=0, at=256, skew=0),
        # the decode step of six samples in full precision
        dict(name="shared_fp32", op="shared", fmt="int8", dtype="fp32", batch=6, kv_heads=8, group=4, n=1, prefixes=1, shared=8191,
             lone=0, at=333, skew=29),
        # one prompt of 8K tokens becomes 16 samples, and is read back
        dict(name="take_fork", op="take", fmt="int8", dtype="bf16", batch=16, sources=1, kv_heads=8, at=8191, skew=0, cut=0, inside=False),
        # beams put in order within a cache, some of them cut back, and read back
        dict(name="take_beams", op="take", fmt="e4m3", dtype="fp32", batch=24, sources=24, kv_heads=8, at=517, skew=3, cut=5, inside=True),
        # every second block of eight sequences of 32K tokens stays
        dict(name="keep_half", op="keep", fmt="int8", dtype="bf16", batch=8, kv_heads=8, at=32768, skew=37, kept=0.5),
        # a few blocks of a few sequences in full precision
        dict(name="keep_few", op="keep", fmt="e4m3", dtype="fp32", batch=3, kv_heads=8, at=2500, skew=333, kept=0.21),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["axes", "shared", "shared", "take", "keep"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "axes":
        c.update(batch=_log(rng, 1, 32), kv_heads=rng.choice([1, 2, 4, 8]))
        c["heads"] = c["kv_heads"] * rng.choice([1, 2, 4, 8])
        c["n"] = 1 if rng.random() < 0.3 else _log(rng, 2, max(2, 16384 // (c["batch"] * (2 if c["dtype"] == "fp32" else 1))))
        c.update(rd=rng.choice([64, 96, 128]), layout=rng.choice(["half", "interleaved"]), axes=rng.choice([2, 3, 4]),
                 spread=rng.choice(["runs", "turns"]), base=rng.choice([10000.0, 500000.0, 1000000.0]))
        c["apart"] = c["spread"] == "runs" and rng.random() < 0.5
        return c
    c.update(fmt=rng.choice(["int8", "e4m3"]), kv_heads=rng.choice([1, 2, 4, 8]))
    if op == "shared":
        c["batch"], c["group"] = _log(rng, 1, 64), rng.choice([1, 2, 4, 8])
        c["n"] = rng.choice([1, 1, 1, 2, 5, _log(rng, 8, 256)])
        c["prefixes"] = rng.choice([1, 1, 2, max(1, c["batch"] // 4)])
        c["lone"] = rng.choice([0, 0, 1]) if c["batch"] > 1 else 0
        rows = c["batch"] * c["n"] * c["group"] * c["kv_heads"]
        most = max(64, min(32768, (1 << 30) // rows, (1 << 19) // (c["prefixes"] * c["kv_heads"])))
        c["shared"] = _log(rng, 16, most)
        c["at"] = c["n"] + _log(rng, 1, max(2, min(4096, (1 << 18) // (c["batch"] * c["kv_heads"]), (1 << 29) // rows)))
        c["skew"] = rng.randrange(0, 1 + c["at"] // c["batch"])
        return c
    if op == "take":
        c["batch"], c["inside"] = _log(rng, 1, 48), rng.random() < 0.5
        c["sources"] = c["batch"] if c["inside"] else _log(rng, 1, 8)
        c["at"] = _log(rng, 16, min(16384, (1 << 20) // (max(c["batch"], c["sources"]) * c["kv_heads"])))
        c["skew"], c["cut"] = rng.randrange(0, 1 + c["at"] // (2 * c["batch"])), rng.choice([0, 1, 7, 40])
        return c
    c["batch"] = _log(rng, 1, 32)
    c["at"] = _log(rng, 16, min(32768, (1 << 20) // (c["batch"] * c["kv_heads"])))
    c["skew"], c["kept"] = rng.randrange(0, 1 + c["at"] // (2 * c["batch"])), rng.choice([0.1, 0.3, 0.5, 0.9])
    return c


# What follows from a case alone: lengths, who belongs to whom, how much is kept.

def _lengths(c):
    """Tokens of each own sequence (shared, keep), or of each source (take)."""
    return [max(c.get("n", 1), c["at"] - b * c["skew"]) for b in range(c["sources"] if c["op"] == "take" else c["batch"])]


def _shared_lengths(c):
    return [max(1, c["shared"] - 1001 * g % (c["shared"] // 2 + 1)) for g in range(c["prefixes"])]


def _prefix_of(c):
    """Sequences take prefixes by turns, as slots are given out; the last `lone` have none."""
    return [b % c["prefixes"] if b < c["batch"] - c["lone"] else -1 for b in range(c["batch"])]


def _parents(c):
    """Whose tokens each sequence takes: within a cache, every third one stays and is taken by the next two."""
    return [b - b % 3 if c["inside"] else b % c["sources"] for b in range(c["batch"])]


def _taken(c):
    """Tokens that each sequence takes: of its parent's, up to `cut` times its place fewer, none below one."""
    have = _lengths(c)
    if c["inside"]:
        return [max(1, have[p] - (c["cut"] if p % 2 else 0)) for p in _parents(c)]
    return [max(1, have[p] - c["cut"] * (b // c["sources"])) for b, p in enumerate(_parents(c))]


def _kept(c):
    return [int(v // BLOCK * c["kept"]) for v in _lengths(c)]


def _axis_of(c):
    """The axis of each pair: runs of about equal length, or by turns."""
    pairs = c["rd"] // 2
    if c["spread"] == "turns":
        return [i % c["axes"] for i in range(pairs)]
    return [a for a, s in enumerate(_sections(c)) for _ in range(s)]


def _sections(c):
    """Pairs of each axis where they lie in runs: the first axis has fewer (16, 24, 24 of 64), as time has."""
    pairs, a = c["rd"] // 2, c["axes"]
    if c["apart"]:
        return [pairs // a + (1 if i < pairs % a else 0) for i in range(a)]
    rest = 3 * pairs // (4 * (a - 1))
    return [pairs - rest * (a - 1)] + [rest] * (a - 1)


def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "axes":
        x = c["batch"] * (c["heads"] + c["kv_heads"]) * c["n"]
        return {"bytes": 2 * es * x * D + 4 * c["axes"] * c["batch"] * c["n"], "flops": 3.0 * x * c["rd"]}
    row = 2 * (D + 4 / BLOCK)  # bytes of a token's codes and its share of the scales, K and V
    if c["op"] == "shared":
        heads, n = c["kv_heads"] * c["group"], c["n"]
        pre = _shared_lengths(c)
        used = {g for g in _prefix_of(c) if g >= 0}
        pairs = 0
        for g, v in zip(_prefix_of(c), _lengths(c)):
            pairs += n * ((pre[g] if g >= 0 else 0) + v - n) + n * (n + 1) // 2
        tokens = sum(pre[g] for g in used) + sum(_lengths(c))
        return {"bytes": row * tokens * c["kv_heads"] + 2 * es * c["batch"] * heads * n * D, "flops": 4.0 * D * pairs * heads}
    if c["op"] == "take":
        parents, taken = _parents(c), _taken(c)
        moved = [(p, t) for b, (p, t) in enumerate(zip(parents, taken)) if not (c["inside"] and p == b)]
        most = {}
        for p, t in moved:
            most[p] = max(most.get(p, 0), t)
        n = max(taken)
        codes = row * c["kv_heads"] * (sum(most.values()) + sum(t for _, t in moved))
        back = sum(taken) * c["kv_heads"]
        return {"bytes": codes + row * back + 2 * es * c["batch"] * c["kv_heads"] * n * D, "flops": 2.0 * back * D}
    held = sum(k * BLOCK + v % BLOCK for k, v in zip(_kept(c), _lengths(c))) * c["kv_heads"]
    n = max(1, *(k * BLOCK + v % BLOCK for k, v in zip(_kept(c), _lengths(c))))
    return {"bytes": 3 * row * held + 2 * es * c["batch"] * c["kv_heads"] * n * D, "flops": 2.0 * held * D}


# ---------------------------------------------------------------- inputs

def _cache(g, b, h, cap, fmt, dtype, lengths):
    """A filled cache's arrays: keys in a few groups around common means, as a head's are; what is past a length is zeros."""
    s = {"lengths": torch.tensor(lengths, dtype=torch.int32, device="cuda")}
    n = max(max(lengths), 1)
    live = torch.arange(n, device="cuda") < s["lengths"].view(b, 1)
    at = (s["lengths"].long() - 1).clamp_min(0) // BLOCK * BLOCK
    rows = at.view(b, 1, 1, 1) + torch.arange(BLOCK, device="cuda").view(1, 1, BLOCK, 1)
    for x in ("k", "v"):
        y = torch.randn(b, h, n, D, generator=g, device="cuda")
        if x == "k":
            mean = torch.randn(b * h * 32, D, generator=g, device="cuda")
            pick = torch.randint(0, 32, (b, h, n), generator=g, device="cuda") + 32 * torch.arange(b * h, device="cuda").view(b, h, 1)
            y = y.mul_(0.3).add_(mean[pick])
        y = (y * live.view(b, 1, n, 1)).to(dtype).float()
        y = torch.nn.functional.pad(y, (0, 0, 0, cap - n))
        blocks = y.view(b, h, cap // BLOCK, BLOCK * D)
        scale = blocks.abs().amax(-1) / TOP[fmt]
        z = (blocks / scale.clamp_min(1e-30).unsqueeze(-1)).view(b, h, cap, D)
        s[x + "_codes"] = (z.round() if fmt == "int8" else z.clamp(-448, 448)).to(CODE[fmt])
        s[x + "_scale"] = scale
        s[x + "_tail"] = y.gather(2, rows.expand(b, h, BLOCK, D)).to(dtype)
    return s


def _empty(b, h, cap, fmt, dtype):
    s = {"lengths": torch.zeros(b, dtype=torch.int32, device="cuda")}
    for x in ("k", "v"):
        s[x + "_codes"] = torch.zeros(b, h, cap, D, dtype=torch.int8, device="cuda").view(CODE[fmt])
        s[x + "_scale"] = torch.zeros(b, h, cap // BLOCK, device="cuda")
        s[x + "_tail"] = torch.zeros(b, h, BLOCK, D, dtype=dtype, device="cuda")
    return s


def _room(n):
    return (n + 2 * BLOCK - 1) // BLOCK * BLOCK


def _handle(s):
    import cluster_indexed_kv_gb300 as lkv
    return lkv.Cache8.from_tensors(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["k_tail"], s["v_tail"], s["lengths"])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, dtype, b = case, TYPE[case["dtype"]], case["batch"]
    i32 = dict(dtype=torch.int32, device="cuda")
    s = {"case": c}
    if c["op"] == "axes":
        s["q"] = torch.randn(b, c["heads"], c["n"], D, generator=g, device="cuda").to(dtype)
        s["k"] = torch.randn(b, c["kv_heads"], c["n"], D, generator=g, device="cuda").to(dtype)
        i = torch.arange(c["n"], device="cuda")
        first = torch.randint(0, 4096, (b, 1), generator=g, device="cuda")
        grid = [first + i // 900, first + i // 30 % 30, first + i % 30, first + i]  # frames of 30 x 30 patches; text goes on along all
        s["positions"] = torch.stack(grid[: c["axes"]]).to(torch.int32) if c["n"] > 1 else (first + 5000).expand(c["axes"], b, 1).to(torch.int32).contiguous()
        s["axis"], s["freq"] = torch.tensor(_axis_of(c), device="cuda"), _frequencies(c)
        if own:
            import cluster_indexed_kv_gb300 as lkv
            how = dict(axes=_axis_of(c)) if c["spread"] == "turns" else dict(sections=_sections(c), own_base=c["apart"])
            s["rope"] = lkv.Rope(rotary_dim=c["rd"], layout=c["layout"], base=c["base"], **how)
        return s
    h, fmt = c["kv_heads"], c["fmt"]
    if c["op"] == "shared":
        pre = _shared_lengths(c)
        s["prefix"] = _cache(g, c["prefixes"], h, _room(max(pre)), fmt, dtype, pre)
        s["cache"] = _cache(g, b, h, _room(max(_lengths(c))), fmt, dtype, _lengths(c))
        s["prefix_of"] = torch.tensor(_prefix_of(c), **i32)
        q = torch.randn(b, h, c["group"], c["n"], D, generator=g, device="cuda")
        # each query favours a few tokens of the prefix
        near = torch.randint(0, min(pre), (b, h, c["group"] * c["n"]), generator=g, device="cuda")
        to = s["prefix_of"].long().clamp_min(0)
        code = s["prefix"]["k_codes"].view(torch.int8)[to].gather(2, (near // BLOCK * BLOCK).unsqueeze(-1).expand(-1, -1, -1, D)).view(CODE[fmt])
        like = code.float() * s["prefix"]["k_scale"][to].gather(2, near // BLOCK).unsqueeze(-1)
        s["q"] = (q + 0.5 * like.view(q.shape)).view(b, h * c["group"], c["n"], D).to(dtype)
        if own:
            s["own"], s["own_prefix"] = _handle(s["cache"]), _handle(s["prefix"])
        return s
    if c["op"] == "take":
        s["source"] = _cache(g, c["sources"], h, _room(max(_lengths(c))), fmt, dtype, _lengths(c))
        s["cache"] = s["source"] if c["inside"] else _empty(b, h, _room(max(_taken(c))), fmt, dtype)
        s["sequences"], s["taken"] = torch.tensor(_parents(c), **i32), torch.tensor(_taken(c), **i32)
        s["n"] = max(_taken(c))
    else:
        s["source"] = _cache(g, b, h, _room(max(_lengths(c))), fmt, dtype, _lengths(c))
        most, have = max(max(_kept(c)), 1), torch.tensor([v // BLOCK for v in _lengths(c)], device="cuda")
        # the kept blocks, in order: the best `counts` of random marks
        mark = torch.rand(b, h, max(_lengths(c)) // BLOCK + 1, generator=g, device="cuda")
        mark = mark.masked_fill(torch.arange(mark.shape[2], device="cuda") >= have.view(b, 1, 1), -1.0)
        order = mark.argsort(-1, descending=True)[..., :most]
        s["counts"] = torch.tensor(_kept(c), **i32)
        order = order.masked_fill(torch.arange(most, device="cuda") >= s["counts"].view(b, 1, 1), 1 << 30)
        s["blocks"] = order.sort(-1).values.to(torch.int32).contiguous()
        s["n"] = max(1, *(k * BLOCK + v % BLOCK for k, v in zip(_kept(c), _lengths(c))))
        s["cache"] = _empty(b, h, _room(s["n"]), fmt, dtype)
    if own:
        s["own"] = _handle(s["cache"])
        s["own_source"] = s["own"] if s["source"] is s["cache"] else _handle(s["source"])
    return s


# ---------------------------------------------------------------- plain forms

def _frequencies(c):
    """Radians a position for each pair, in 64 bits: a program's table."""
    if c["apart"]:
        return torch.cat([c["base"] ** (-torch.arange(0, 2 * v, 2, dtype=torch.float64, device="cuda") / (2 * v)) for v in _sections(c)])
    return c["base"] ** (-torch.arange(0, c["rd"], 2, dtype=torch.float64, device="cuda") / c["rd"])


def _turned(x, cos, sin, rd, layout):
    y = x.float()
    if layout == "half":
        a, b = y[..., : rd // 2], y[..., rd // 2: rd]
        t = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = y[..., 0:rd:2], y[..., 1:rd:2]
        t = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((t, y[..., rd:]), -1).to(x.dtype)


def _plain_axes(s):
    c = s["case"]
    angle = s["positions"].double()[s["axis"]].permute(1, 2, 0) * s["freq"]  # 64 bits: far positions times small frequencies
    cos, sin = (f(angle).float().unsqueeze(1) for f in (torch.cos, torch.sin))
    return [_turned(s["q"], cos, sin, c["rd"], c["layout"]), _turned(s["k"], cos, sin, c["rd"], c["layout"])]


def _rows(s, x, n):
    """The first n rows of each sequence in fp32: a full block as code * scale, the last, partial one as it is, zeros behind."""
    codes, scale, tail = s[x + "_codes"], s[x + "_scale"], s[x + "_tail"]
    b, h = codes.shape[:2]
    pos = torch.arange(n, device=codes.device)
    length = s["lengths"].long().view(b, 1, 1, 1)
    v = codes[:, :, :n].float() * scale.repeat_interleave(BLOCK, 2)[:, :, :n].unsqueeze(-1)
    t = tail[:, :, pos % BLOCK].float()
    v = torch.where(pos.view(1, 1, n, 1) < length // BLOCK * BLOCK, v, t)
    return torch.where(pos.view(1, 1, n, 1) < length, v, 0.0)


def _plain_shared(s):
    c, q = s["case"], s["q"]
    b, hkv, g, n = c["batch"], c["kv_heads"], c["group"], c["n"]
    pre, mine = max(_shared_lengths(c)), max(_lengths(c))
    to = s["prefix_of"].long()
    has = to >= 0
    p_len = torch.where(has, s["prefix"]["lengths"].long()[to.clamp_min(0)], 0).view(b, 1, 1)
    length = s["cache"]["lengths"].long().view(b, 1, 1)
    i = torch.arange(n, device=q.device).view(1, n, 1)
    j = torch.arange(pre, device=q.device)
    see = torch.cat(((j < p_len) & (j <= p_len + length - n + i), torch.arange(mine, device=q.device) <= length - n + i), 2)
    x = q.float().view(b, hkv, g * n, D)
    # sequences of one prefix lie together in a product over its rows, so that these are unpacked once
    kp, vp = _rows(s["prefix"], "k", pre), _rows(s["prefix"], "v", pre)
    ko, vo = _rows(s["cache"], "k", mine), _rows(s["cache"], "v", mine)
    if c["prefixes"] == 1:
        far = (x.transpose(0, 1).reshape(hkv, -1, D) @ kp[0].transpose(-1, -2)).view(hkv, b, g * n, pre).transpose(0, 1)
    else:
        far = x @ kp[to.clamp_min(0)].transpose(-1, -2)
    y = torch.cat((far, x @ ko.transpose(-1, -2)), -1) * D ** -0.5
    y = y.reshape(b, hkv, g, n, -1).masked_fill(~see.view(b, 1, 1, n, -1), float("-inf"))
    top = y.amax(-1, keepdim=True)
    w = torch.exp(y - torch.where(top > float("-inf"), top, 0.0))
    total = w.sum(-1, keepdim=True)
    w = w.reshape(b, hkv, g * n, -1)
    if c["prefixes"] == 1:
        o = (w[..., :pre].transpose(0, 1).reshape(hkv, -1, pre) @ vp[0]).view(hkv, b, g * n, D).transpose(0, 1)
    else:
        o = w[..., :pre] @ vp[to.clamp_min(0)]
    o = (o + w[..., pre:] @ vo).reshape(b, hkv, g, n, D) / torch.where(total > 0, total, 1.0)
    return o.reshape(b, hkv * g, n, D).to(q.dtype)


def _last_rows(s, x, at):
    """Rows 16 * at[b, h] .. + 15 of each (sequence, KV head) as they would be read: what a tail takes over."""
    codes, scale, tail = s[x + "_codes"], s[x + "_scale"], s[x + "_tail"]
    b, h, cap, _ = codes.shape
    block = codes.view(torch.int8).view(b, h, cap // BLOCK, BLOCK * D).gather(2, at.view(b, h, 1, 1).expand(b, h, 1, BLOCK * D))
    v = block.view(codes.dtype).float() * scale.gather(2, at.unsqueeze(-1)).unsqueeze(-1)
    last = ((s["lengths"].long() - 1).clamp_min(0) // BLOCK).view(b, 1)
    return torch.where((at == last).view(b, h, 1, 1), tail, v.view(b, h, BLOCK, D).to(tail.dtype))


def _plain_take(s):
    c, src, dst = s["case"], s["source"], s["cache"]
    to, length = s["sequences"].long(), s["taken"]
    picked = {x: y[to] if y.dim() < 4 else y.view(torch.uint8)[to].view(y.dtype) for x, y in src.items()}
    last = ((length.long() - 1).clamp_min(0) // BLOCK).view(-1, 1).expand(-1, c["kv_heads"])
    full = length.long().view(-1, 1, 1) // BLOCK
    for x in ("k", "v"):
        tail = _last_rows(picked, x, last)
        nb = min(src[x + "_scale"].shape[2], dst[x + "_scale"].shape[2])
        new = torch.arange(nb, device="cuda") < full
        at = dst[x + "_codes"].view(torch.int8)[:, :, : nb * BLOCK].unflatten(2, (nb, BLOCK))
        at.copy_(torch.where(new[..., None, None], picked[x + "_codes"].view(torch.int8)[:, :, : nb * BLOCK].unflatten(2, (nb, BLOCK)), at))
        dst[x + "_scale"][:, :, :nb] = torch.where(new, picked[x + "_scale"][:, :, :nb], dst[x + "_scale"][:, :, :nb])
        dst[x + "_tail"].copy_(tail)
    dst["lengths"].copy_(length)
    return _back(s)


def _plain_keep(s):
    c, src, dst = s["case"], s["source"], s["cache"]
    b, h = c["batch"], c["kv_heads"]
    count, m = s["counts"].long().view(b, 1, 1), s["blocks"].shape[2]
    at = s["blocks"].long().clamp(0, src["k_scale"].shape[2] - 1)
    kept = torch.arange(m, device="cuda") < count
    part = src["lengths"].long() % BLOCK
    low = torch.where(kept, at, 0).amax(-1)
    last = torch.where(part.view(b, 1) > 0, (src["lengths"].long() // BLOCK).view(b, 1), low)
    for x in ("k", "v"):
        rows = src[x + "_codes"].view(torch.int8).view(b, h, -1, BLOCK * D).gather(2, at.unsqueeze(-1).expand(-1, -1, -1, BLOCK * D))
        to = dst[x + "_codes"].view(torch.int8).view(b, h, -1, BLOCK * D)[:, :, :m]
        to.copy_(torch.where(kept.unsqueeze(-1), rows, to))
        dst[x + "_scale"][:, :, :m] = torch.where(kept, src[x + "_scale"].gather(2, at), dst[x + "_scale"][:, :, :m])
        dst[x + "_tail"].copy_(_last_rows(src, x, last))
    dst["lengths"].copy_(s["counts"] * BLOCK + part.to(torch.int32))
    return _back(s)


def _back(s):
    """The cache's rows as values, and its lengths."""
    dtype = s["cache"]["k_tail"].dtype
    return [_rows(s["cache"], "k", s["n"]).to(dtype), _rows(s["cache"], "v", s["n"]).to(dtype), s["cache"]["lengths"]]


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if op == "axes":
        if own:
            return s["rope"].apply(s["q"], s["positions"], s["k"])
        return _plain_axes(s)
    if op == "shared":
        if own:
            return s["own"].attend_shared(s["q"], s["own_prefix"], s["prefix_of"], max_len=s["case"]["at"])
        return _plain_shared(s)
    if op == "take":
        if own:
            s["own"].take(s["own_source"], s["sequences"], s["taken"])
            return [*s["own"].read(s["n"]), s["own"].lengths]
        return _plain_take(s)
    if own:
        s["own"].keep(s["blocks"], s["counts"], s["own_source"])
        return [*s["own"].read(s["n"]), s["own"].lengths]
    return _plain_keep(s)


# ---------------------------------------------------------------- the definitions, in 64 bits

def _sequence(s, x, b):
    """A cache's sequence b as it stands, in 64 bits: [H, length, D]."""
    n = int(s["lengths"][b])
    full = n // BLOCK * BLOCK
    code = s[x + "_codes"][b, :, :full].float().double()
    scale = s[x + "_scale"][b, :, : full // BLOCK].double().repeat_interleave(BLOCK, 1)
    return torch.cat((code * scale.unsqueeze(-1), s[x + "_tail"][b, :, : n - full].double()), 1)


def _exact_axes(s):
    c, out = s["case"], []
    rd, rate = c["rd"], []
    for i, a in enumerate(_axis_of(c)):
        of = (_sections(c)[a], i - sum(_sections(c)[:a])) if c["apart"] else (rd // 2, i)
        rate.append(math.exp(-of[1] / of[0] * math.log(c["base"])))
    rate = torch.tensor(rate, dtype=torch.float64, device="cuda")
    where = torch.stack([s["positions"][a].double() for a in _axis_of(c)], -1)
    turn = torch.exp(1j * (where * rate)[:, None])
    for x in (s["q"], s["k"]):
        y = x.double()
        first, second = (y[..., : rd // 2], y[..., rd // 2: rd]) if c["layout"] == "half" else (y[..., 0:rd:2], y[..., 1:rd:2])
        z = torch.complex(first.contiguous(), second.contiguous()) * turn
        if c["layout"] == "half":
            y[..., : rd // 2], y[..., rd // 2: rd] = z.real, z.imag
        else:
            y[..., 0:rd:2], y[..., 1:rd:2] = z.real, z.imag
        out.append(y)
    return out


def _exact_shared(s):
    c = s["case"]
    out = torch.zeros(c["batch"], c["kv_heads"], c["group"], c["n"], D, dtype=torch.float64, device="cuda")
    q = s["q"].double().view(out.shape)
    for b, (g, length) in enumerate(zip(_prefix_of(c), _lengths(c))):
        k, v = _sequence(s["cache"], "k", b), _sequence(s["cache"], "v", b)
        if g >= 0:
            k = torch.cat((_sequence(s["prefix"], "k", g), k), 1)
            v = torch.cat((_sequence(s["prefix"], "v", g), v), 1)
        token = torch.arange(k.shape[1], device="cuda")
        hide = token > (k.shape[1] - c["n"] + torch.arange(c["n"], device="cuda")).unsqueeze(1)
        score = torch.einsum("hgnd,htd->hgnt", q[b], k) / math.sqrt(D)
        score.masked_fill_(hide, -math.inf)
        out[b] = torch.einsum("hgnt,htd->hgnd", torch.softmax(score, -1), v)
    return out.flatten(1, 2)


def _exact_moved(s, rows):
    """rows(x, b): [H, length, D] of sequence b after the call, in 64 bits."""
    c, out = s["case"], []
    for x in ("k", "v"):
        back = torch.zeros(c["batch"], c["kv_heads"], s["n"], D, dtype=torch.float64, device="cuda")
        for b in range(c["batch"]):
            y = rows(x, b)
            back[b, :, : y.shape[1]] = y
        out.append(back)
    return out + [None]


def _exact_take(s):
    parents, taken = _parents(s["case"]), _taken(s["case"])
    return _exact_moved(s, lambda x, b: _sequence(s["source"], x, parents[b])[:, : taken[b]])


def _exact_keep(s):
    c = s["case"]

    def rows(x, b):
        y = _sequence(s["source"], x, b)
        count, full = _kept(c)[b], _lengths(c)[b] // BLOCK
        z = y[:, : full * BLOCK].unflatten(1, (full, BLOCK)) if full else y.new_zeros(c["kv_heads"], 0, BLOCK, D)
        z = torch.stack([z[h, s["blocks"][b, h, :count].long()] for h in range(c["kv_heads"])])
        return torch.cat((z.flatten(1, 2), y[:, full * BLOCK:]), 1)

    return _exact_moved(s, rows)


def exact(case, seed):
    s = prepare(case, seed)
    return {"axes": _exact_axes, "shared": _exact_shared, "take": _exact_take, "keep": _exact_keep}[case["op"]](s)
