"""The 8-bit cache operators and rotary positions, case by case: inputs, plain forms, the library's calls.

Layouts are head-major, as the library's prefill keys: q [B, H, n, 128], k and v [B, H_kv, n, 128], H = H_kv * group.

  rope    pairs of the first `rd` of a row's 128 values are turned by position * frequency; q and k in one call.
  write   k and v rows go into a cache held in 8 bits, one scale for each 16 tokens of a (sequence, KV head), and are read
          back: a full block as code * scale, the last, partial block in full precision.
  read    the rows first[b] .. first[b] + n - 1 of a filled cache, zeros past a sequence's length.
  attend  causal softmax attention of the last n tokens of each sequence over such a cache; with a window, a token sees the
          `window` last tokens and the `sinks` first ones.
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
        # one decode step of eight sequences near 32K tokens: latency of the smallest call
        dict(name="rope_step", op="rope", dtype="bf16", batch=8, heads=32, kv_heads=8, n=1, at=32760, rd=128,
             layout="half", scaling="none", base=10000.0, factor=1.0),
        # a 32K prompt's queries and keys, half of each head rotated, positions stretched fourfold
        dict(name="rope_prompt", op="rope", dtype="bf16", batch=1, heads=32, kv_heads=8, n=32768, at=98304, rd=64,
             layout="interleaved", scaling="yarn", base=1000000.0, factor=4.0),
        # one decode step's rows of 32 sequences; every 16th sequence fills a block
        dict(name="write_step", op="write", fmt="int8", dtype="bf16", batch=32, kv_heads=8, n=1, at=8000, skew=7,
             capacity=8192),
        # the prompts of eight sequences of 32K tokens, written and read back
        dict(name="write_prompt", op="write", fmt="int8", dtype="bf16", batch=8, kv_heads=8, n=32768, at=0, skew=0,
             capacity=33280),
        # ragged chunks behind earlier ones, in fp32 and e4m3
        dict(name="write_ragged", op="write", fmt="e4m3", dtype="fp32", batch=3, kv_heads=8, n=2047, at=2048, skew=160,
             capacity=8192),
        # a whole 128K prompt for an index build
        dict(name="read_prompt", op="read", fmt="int8", dtype="bf16", batch=1, kv_heads=8, n=131072, at=131077, skew=0,
             capacity=131584),
        # the last tokens of a few sequences, past the end of the shorter ones
        dict(name="read_tail", op="read", fmt="e4m3", dtype="fp32", batch=2, kv_heads=8, n=777, at=2500, skew=333,
             capacity=4096),
        # the smallest attention: one sequence, one KV head, fp32
        dict(name="attend_tiny", op="attend", fmt="int8", dtype="fp32", batch=1, kv_heads=1, group=4, n=1, at=2048,
             skew=0, capacity=2112, window=0, sinks=0),
        # the decode step of eight sequences at 32K over everything
        dict(name="attend_b8_32k", op="attend", fmt="int8", dtype="bf16", batch=8, kv_heads=8, group=4, n=1, at=33001,
             skew=37, capacity=40960, window=0, sinks=0),
        # the decode step of 32 long sequences that see 1024 recent tokens and four first ones
        dict(name="attend_window", op="attend", fmt="e4m3", dtype="bf16", batch=32, kv_heads=8, group=4, n=1, at=33001,
             skew=101, capacity=33280, window=1024, sinks=4),
        # the decode step of one very long sequence: few rows, a long axis
        dict(name="attend_128k", op="attend", fmt="int8", dtype="bf16", batch=1, kv_heads=8, group=4, n=1, at=131579,
             skew=0, capacity=131584, window=0, sinks=0),
        # a prompt's last chunk over the cache of what came before it: products
        dict(name="attend_chunk", op="attend", fmt="int8", dtype="bf16", batch=1, kv_heads=8, group=4, n=2048, at=32768,
             skew=0, capacity=33280, window=0, sinks=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attend", "attend", "attend"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "rope":
        c.update(batch=_log(rng, 1, 32), kv_heads=rng.choice([1, 2, 4, 8]))
        c["heads"] = c["kv_heads"] * rng.choice([1, 2, 4, 8])
        c["n"] = 1 if rng.random() < 0.3 else _log(rng, 2, max(2, 16384 // (c["batch"] * (2 if c["dtype"] == "fp32" else 1))))
        c.update(at=_log(rng, 1, 1 << 20), rd=rng.choice([32, 64, 96, 128]), layout=rng.choice(["half", "interleaved"]),
                 scaling=rng.choice(["none", "linear", "ntk", "yarn"]), base=rng.choice([10000.0, 500000.0, 1000000.0]))
        c["factor"] = 1.0 if c["scaling"] == "none" else rng.choice([2.0, 4.0, 8.0])
        return c
    c.update(fmt=rng.choice(["int8", "e4m3"]), batch=_log(rng, 1, 32), kv_heads=rng.choice([1, 2, 4, 8]))
    rows = 1 << 20  # tokens of all slices, at most
    slices = c["batch"] * c["kv_heads"]
    if op == "write":
        c["n"] = 1 if rng.random() < 0.3 else _log(rng, 2, min(32768, rows // (2 * slices)))
        c["at"] = _log(rng, 16, 4096) if c["n"] == 1 else 16 * rng.randrange(0, 64)
        c["skew"] = rng.randrange(0, 1 + c["n"] // (4 * c["batch"])) if c["n"] > 1 else rng.randrange(0, 32)
    elif op == "read":
        c["n"] = _log(rng, 1, min(32768, rows // (2 * slices)))
        c["at"] = _log(rng, 1, 2 * c["n"])
        c["skew"] = rng.randrange(0, 64)
    else:
        c["group"] = rng.choice([1, 2, 4, 8])
        c["n"] = rng.choice([1, 1, 1, 2, 5, _log(rng, 8, 512)])
        most = min(131072, rows // slices)
        if c["n"] > 8:
            most = max(c["n"], min(most, (1 << 28) // (c["n"] * c["group"] * slices)))
        c["at"] = max(c["n"], _log(rng, 1, most))
        c["skew"] = rng.randrange(0, 1 + c["at"] // c["batch"])
        c["window"] = 0 if rng.random() < 0.5 else _log(rng, 1, 4096)
        c["sinks"] = 0 if c["window"] == 0 else rng.choice([0, 1, 4, 17])
    c["capacity"] = (c["at"] + c["n"] + 31) // BLOCK * BLOCK
    return c


def _lengths(c):
    """Tokens in each sequence before the call (write) or at the call (read, attend): they follow from the case alone."""
    low = c["n"] if c["op"] == "attend" else 0
    return [max(low, c["at"] - b * c["skew"]) for b in range(c["batch"])]


def _starts(c):
    if c["n"] == 1:
        return _lengths(c)
    return [v // BLOCK * BLOCK for v in _lengths(c)]


def _counts(c):
    """Tokens that each sequence writes: ragged where the case has a skew."""
    return [max(1, c["n"] - b * c["skew"]) if c["n"] > 1 else 1 for b in range(c["batch"])]


def _visible(c):
    """(tokens that some query of the sequence sees, pairs of a query and a token that it sees), over all sequences."""
    tokens = pairs = 0
    for length in _lengths(c):
        w, s, n = c["window"], c["sinks"], c["n"]
        first = length - n
        if w == 0:
            tokens += length
            pairs += n * first + n * (n + 1) // 2
        else:
            low = max(0, first - w + 1)
            tokens += length - low + min(s, low)
            for i in range(n):
                pos = first + i
                low = max(0, pos - w + 1)
                pairs += pos + 1 - low + min(s, low)
    return tokens, pairs


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        x = case["batch"] * (case["heads"] + case["kv_heads"]) * case["n"]
        return {"bytes": 2 * es * x * D + 4 * case["batch"] * case["n"], "flops": 3.0 * x * case["rd"]}
    if case["op"] == "write":
        rows = sum(_counts(case)) * case["kv_heads"]
        back = case["batch"] * case["kv_heads"] * (BLOCK if case["n"] == 1 else case["n"])
        return {"bytes": 2 * rows * (es * D + D + 4 / BLOCK) + 2 * es * back * D + 8 * case["batch"], "flops": 2.0 * rows * 4 * D}
    if case["op"] == "read":
        rows = case["batch"] * case["kv_heads"] * case["n"]
        held = sum(max(0, min(case["n"], v - f)) for v, f in zip(_lengths(case), _firsts(case))) * case["kv_heads"]
        return {"bytes": 2 * held * (D + 4 / BLOCK) + 2 * es * rows * D, "flops": 2.0 * held * D}
    tokens, pairs = _visible(case)
    heads = case["kv_heads"] * case["group"]
    return {"bytes": 2 * tokens * case["kv_heads"] * (D + 4 / BLOCK) + 2 * es * case["batch"] * heads * case["n"] * D,
            "flops": 4.0 * D * pairs * heads}


def _firsts(c):
    """The first row that a read asks for: the prompt from its start, shorter reads towards the end."""
    return [max(0, c["at"] - c["n"] - 5 * b) for b in range(c["batch"])]


# ---------------------------------------------------------------- inputs

def _keys(g, b, h, n):
    """Keys in a few groups around common means, as a head's keys are."""
    mean = torch.randn(b * h * 32, D, generator=g, device="cuda")
    pick = torch.randint(0, 32, (b, h, n), generator=g, device="cuda") + 32 * torch.arange(b * h, device="cuda").view(b, h, 1)
    x = torch.randn(b, h, n, D, generator=g, device="cuda").mul_(0.3)
    return x.add_(mean[pick])


def _values(g, b, h, n):
    return torch.randn(b, h, n, D, generator=g, device="cuda")


def _held(x, cap, fmt, dtype, lengths):
    """A cache's arrays for rows x [B, H, n, D] of which lengths[b] are there: codes, scales, the last block's rows."""
    b, h, n, _ = x.shape
    x = torch.nn.functional.pad(x, (0, 0, 0, cap - n))
    blocks = x.view(b, h, cap // BLOCK, BLOCK * D)
    scale = blocks.abs().amax(-1) / TOP[fmt]
    y = (blocks / scale.clamp_min(1e-30).unsqueeze(-1)).view(b, h, cap, D)
    codes = (y.round() if fmt == "int8" else y.clamp(-448, 448)).to(CODE[fmt])
    at = (lengths - 1).clamp_min(0) // BLOCK * BLOCK
    rows = at.view(b, 1, 1, 1) + torch.arange(BLOCK, device="cuda").view(1, 1, BLOCK, 1)
    tail = x.gather(2, rows.expand(b, h, BLOCK, D)).to(dtype)
    return codes, scale, tail


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, dtype, b = case, TYPE[case["dtype"]], case["batch"]
    i32 = dict(dtype=torch.int32, device="cuda")
    s = {"case": c}
    if c["op"] == "rope":
        s["q"] = torch.randn(b, c["heads"], c["n"], D, generator=g, device="cuda").to(dtype)
        s["k"] = torch.randn(b, c["kv_heads"], c["n"], D, generator=g, device="cuda").to(dtype)
        far = torch.randint(0, 64, (b, 1), generator=g, device="cuda")
        s["positions"] = (c["at"] + far + torch.arange(c["n"], device="cuda")).to(torch.int32)
        s["freq"], s["gain"] = _frequencies(c)
        if own:
            import cluster_indexed_kv_gb300 as lkv
            s["rope"] = lkv.Rope(rotary_dim=c["rd"], layout=c["layout"], base=c["base"], scaling=c["scaling"],
                                 factor=c["factor"], orig_len=ORIG_LEN)
        return s
    h, cap = c["kv_heads"], c["capacity"]
    lengths = torch.tensor(_starts(c) if c["op"] == "write" else _lengths(c), **i32)
    s["lengths"] = lengths
    if c["op"] == "write":
        s["k"], s["v"] = _keys(g, b, h, c["n"]).to(dtype), _values(g, b, h, c["n"]).to(dtype)
        s["start"], s["counts"] = lengths.clone(), torch.tensor(_counts(c), **i32)
        s["block"] = torch.div(lengths, BLOCK, rounding_mode="floor").to(torch.int32) * BLOCK if c["n"] == 1 else lengths.clone()
        for x, f in (("k", _keys), ("v", _values)):  # earlier tokens: their codes are not looked at here, but the tail is
            s[x + "_codes"] = torch.zeros(b, h, cap, D, dtype=torch.int8, device="cuda").view(CODE[c["fmt"]])
            s[x + "_scale"] = torch.zeros(b, h, cap // BLOCK, device="cuda")
            s[x + "_tail"] = f(g, b, h, BLOCK).to(dtype)
    else:
        n = max(_lengths(c))
        s["k_codes"], s["k_scale"], s["k_tail"] = _held(_keys(g, b, h, n).to(dtype).float(), cap, c["fmt"], dtype, lengths)
        s["v_codes"], s["v_scale"], s["v_tail"] = _held(_values(g, b, h, n).to(dtype).float(), cap, c["fmt"], dtype, lengths)
    if c["op"] == "read":
        s["first"] = torch.tensor(_firsts(c), **i32)
    if c["op"] == "attend":  # queries with a few keys each that they favour
        q = torch.randn(b, h, c["group"], c["n"], D, generator=g, device="cuda")
        near = torch.randint(0, 1 << 30, (b, h, c["group"], c["n"]), generator=g, device="cuda") % lengths.view(b, 1, 1, 1)
        like = _rows(s, "k", near.view(b, h, -1)).view(q.shape)
        s["q"] = (q + 0.5 * like).view(b, h * c["group"], c["n"], D).to(dtype)
    if own:
        import cluster_indexed_kv_gb300 as lkv
        s["cache"] = lkv.Cache8.from_tensors(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["k_tail"], s["v_tail"],
                                             s["lengths"])
    return s


# ---------------------------------------------------------------- plain forms

ORIG_LEN = 32768  # the context that stretched positions were made for


def _frequencies(c):
    """Radians a position for each pair, in 64 bits, and the gain that goes with stretched positions: a program's table."""
    rd, base, factor = c["rd"], c["base"], c["factor"]
    if c["scaling"] == "ntk":
        base = base * factor ** (rd / (rd - 2))
    f = base ** (-torch.arange(0, rd, 2, dtype=torch.float64, device="cuda") / rd)
    if c["scaling"] == "linear":
        f = f / factor
    if c["scaling"] == "yarn":
        keep = ((ORIG_LEN * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return f * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _turned(x, cos, sin, rd, layout):
    y = x.float()
    if layout == "half":
        a, b = y[..., : rd // 2], y[..., rd // 2: rd]
        t = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = y[..., 0:rd:2], y[..., 1:rd:2]
        t = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((t, y[..., rd:]), -1).to(x.dtype)


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].double().unsqueeze(-1) * s["freq"]  # 64 bits: far positions times small frequencies
    cos, sin = ((f(angle) * s["gain"]).float().unsqueeze(1) for f in (torch.cos, torch.sin))
    return [_turned(s["q"], cos, sin, c["rd"], c["layout"]), _turned(s["k"], cos, sin, c["rd"], c["layout"])]


def _codes(blocks, fmt):
    """blocks [..., 16 * D] fp32 -> (codes, scales). 64 bits: a value halfway between two codes is decided exactly."""
    top = blocks.abs().amax(-1, keepdim=True)
    y = blocks.double() * TOP[fmt] / torch.where(top > 0, top, 1.0).double()
    if fmt == "int8":
        code = y.round()
    else:
        step = torch.exp2(torch.frexp(y.abs().clamp_min(2.0 ** -6))[1].double() - 4)
        code = (y / step).round() * step
    return code.float().to(CODE[fmt]), (top / TOP[fmt]).squeeze(-1)


def _put(s, x):
    """Rows s[x] behind s["start"]: blocks that are full now become codes and a scale, the last block is kept as it is."""
    new, start, counts = s[x], s["start"].long(), s["counts"].long()
    b, h, n, _ = new.shape
    nb = (n + 2 * BLOCK - 2) // BLOCK
    base = start // BLOCK * BLOCK
    pos = base.view(b, 1) + torch.arange(nb * BLOCK, device=new.device)
    i = pos - start.view(b, 1)
    fresh = ((i >= 0) & (i < counts.view(b, 1))).view(b, 1, -1, 1)
    old = s[x + "_tail"].repeat(1, 1, nb, 1)
    rows = torch.where(fresh, new.gather(2, i.clamp(0, n - 1).view(b, 1, -1, 1).expand(b, h, -1, D)), old)
    codes, scale = _codes(rows.float().view(b, h, nb, BLOCK * D), s["case"]["fmt"])
    block = base.view(b, 1) // BLOCK + torch.arange(nb, device=new.device)
    end = start + counts
    full = (block + 1) * BLOCK <= end.view(b, 1)
    at = torch.nonzero(full, as_tuple=True)
    where = block[at]
    raw = s[x + "_codes"].view(torch.int8).view(b, h, -1, BLOCK * D)
    raw[at[0], :, where] = codes.view(torch.int8)[at[0], :, at[1]]
    s[x + "_scale"][at[0], :, where] = scale[at[0], :, at[1]]
    last = ((end - 1) // BLOCK * BLOCK - base).view(b, 1) + torch.arange(BLOCK, device=new.device)
    tail = rows.gather(2, last.view(b, 1, BLOCK, 1).expand(b, h, BLOCK, D))
    keep = (pos.gather(1, last) < end.view(b, 1)).view(b, 1, BLOCK, 1)
    s[x + "_tail"].copy_(torch.where(keep, tail, s[x + "_tail"]))
    return end


def _rows(s, x, pos):
    """The values at positions pos [B, n] or [B, H, n], in fp32; zeros past the length."""
    codes, scale, tail = s[x + "_codes"], s[x + "_scale"], s[x + "_tail"]
    b, h, cap, _ = codes.shape
    pos = (pos.unsqueeze(1) if pos.dim() == 2 else pos).long().expand(b, h, -1)
    length = s["lengths"].long().view(b, 1, 1)
    at = pos.clamp(0, cap - 1)
    code = codes.view(torch.int8).gather(2, at.unsqueeze(-1).expand(-1, -1, -1, D)).view(codes.dtype).float()
    v = code * scale.gather(2, at // BLOCK).unsqueeze(-1)
    t = tail.gather(2, (at % BLOCK).unsqueeze(-1).expand(-1, -1, -1, D)).float()
    v = torch.where((pos < length // BLOCK * BLOCK).unsqueeze(-1), v, t)
    return torch.where(((pos >= 0) & (pos < length)).unsqueeze(-1), v, 0.0)


def _plain_read(s, first, n):
    pos = first.long().view(-1, 1) + torch.arange(n, device=first.device)
    dtype = s["k_tail"].dtype
    return [_rows(s, "k", pos).to(dtype), _rows(s, "v", pos).to(dtype)]


def _plain_write(s):
    end = _put(s, "k")
    _put(s, "v")
    s["lengths"].copy_(end)
    return _plain_read(s, s["block"], BLOCK if s["case"]["n"] == 1 else s["case"]["n"]) + [s["lengths"]]


def _plain_attend(s):
    c, q = s["case"], s["q"]
    b, hkv, g, n, w, sinks = c["batch"], c["kv_heads"], c["group"], c["n"], c["window"], c["sinks"]
    length = s["lengths"].long().view(b, 1)
    if w == 0:  # the columns that some query sees
        cols = torch.arange(max(_lengths(c)), device=q.device).expand(b, -1)
    else:
        recent = length - n - w + 1 + torch.arange(w + n - 1, device=q.device)
        cols = torch.cat((torch.arange(sinks, device=q.device).expand(b, -1), torch.where(recent >= sinks, recent, -1)), 1)
    pos = length - n + torch.arange(n, device=q.device)
    j, i = cols.unsqueeze(1), pos.unsqueeze(2)
    see = (j >= 0) & (j <= i) & (j < length.unsqueeze(2))
    if w:
        see = see & ((j > i - w) | (j < sinks))
    k, v = _rows(s, "k", cols), _rows(s, "v", cols)
    x = q.float().view(b, hkv, g * n, D) @ k.transpose(-1, -2)
    x = (x * D ** -0.5).view(b, hkv, g, n, -1).masked_fill(~see.view(b, 1, 1, n, -1), float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top > float("-inf"), top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, hkv, g * n, -1) @ v).view(b, hkv, g, n, D) / torch.where(total > 0, total, 1.0)
    return o.view(b, hkv * g, n, D).to(q.dtype)


# ---------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    if c["op"] == "rope":
        if own:
            return s["rope"].apply(s["q"], s["positions"], s["k"])
        return _plain_rope(s)
    if c["op"] == "write":
        n = BLOCK if c["n"] == 1 else c["n"]
        if own:
            s["cache"].write(s["k"], s["v"], start=s["start"], counts=s["counts"])
            k, v = s["cache"].read(n, first=s["block"])
            return [k, v, s["cache"].lengths]
        return _plain_write(s)
    if c["op"] == "read":
        if own:
            return s["cache"].read(c["n"], first=s["first"])
        return _plain_read(s, s["first"], c["n"])
    if own:
        return s["cache"].attend(s["q"], window=c["window"], sinks=c["sinks"], max_len=c["at"])
    return _plain_attend(s)


# ---------------------------------------------------------------- the definitions, in 64 bits

def _e4m3(y):
    """The nearest value of four exponent and three fraction bits, ties to the even one."""
    a = y.abs()
    places = 3 - torch.floor(torch.log2(a.clamp_min(2.0 ** -6)))
    return torch.sign(y) * torch.round(a * 2.0 ** places) * 2.0 ** -places


def _sequence(s, x, b):
    """A cache's sequence b as it stands, in 64 bits: [H, length, D]."""
    n = int(s["lengths"][b])
    full = n // BLOCK * BLOCK
    code = s[x + "_codes"][b, :, :full].float().double()
    scale = s[x + "_scale"][b, :, : full // BLOCK].double().repeat_interleave(BLOCK, 1)
    return torch.cat((code * scale.unsqueeze(-1), s[x + "_tail"][b, :, : n - full].double()), 1)


def _exact_rope(s):
    c, out = s["case"], []
    rd, i = c["rd"], torch.arange(c["rd"] // 2, dtype=torch.float64, device="cuda")
    base = c["base"] * (c["factor"] ** (rd / (rd - 2.0)) if c["scaling"] == "ntk" else 1.0)
    rate, gain = torch.exp(-2.0 * i / rd * math.log(base)), 1.0
    if c["scaling"] == "linear":
        rate = rate / c["factor"]
    elif c["scaling"] == "yarn":
        turns = ORIG_LEN * rate / (2 * math.pi)
        part = torch.clamp((turns - 1.0) / 31.0, 0.0, 1.0)
        rate, gain = part * rate + (1.0 - part) * rate / c["factor"], 1.0 + 0.1 * math.log(c["factor"])
    turn = gain * torch.exp(1j * s["positions"].double()[:, None, :, None] * rate)
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


def _exact_write(s):
    c, out = s["case"], []
    starts, counts = _starts(c), _counts(c)
    n = BLOCK if c["n"] == 1 else c["n"]
    for x in ("k", "v"):
        back = torch.zeros(c["batch"], c["kv_heads"], n, D, dtype=torch.float64, device="cuda")
        for b, (start, count) in enumerate(zip(starts, counts)):
            low = start // BLOCK * BLOCK
            rows = torch.cat((s[x + "_tail"][b, :, : start - low], s[x][b, :, :count]), 1).double()
            full = (start + count - low) // BLOCK * BLOCK
            z = rows[:, :full].unflatten(1, (-1, BLOCK))
            unit = z.abs().amax((2, 3), keepdim=True) / TOP[c["fmt"]]
            y = z / torch.where(unit > 0, unit, 1.0)
            rows[:, :full] = ((torch.round(y) if c["fmt"] == "int8" else _e4m3(y)) * unit).flatten(1, 2)
            back[b, :, : rows.shape[1]] = rows[:, :n]
        out.append(back)
    return out + [None]


def _exact_read(s):
    c, out = s["case"], []
    for x in ("k", "v"):
        back = torch.zeros(c["batch"], c["kv_heads"], c["n"], D, dtype=torch.float64, device="cuda")
        for b, first in enumerate(_firsts(c)):
            rows = _sequence(s, x, b)[:, first: first + c["n"]]
            back[b, :, : rows.shape[1]] = rows
        out.append(back)
    return out


def _exact_attend(s):
    c = s["case"]
    out = torch.zeros(c["batch"], c["kv_heads"], c["group"], c["n"], D, dtype=torch.float64, device="cuda")
    q = s["q"].double().view(out.shape)
    for b, length in enumerate(_lengths(c)):
        k, v = _sequence(s, "k", b), _sequence(s, "v", b)
        token = torch.arange(length, device="cuda")
        for at in range(0, c["n"], 256):
            x = q[b, :, :, at: at + 256]
            pos = (length - c["n"] + at + torch.arange(x.shape[2], device="cuda")).unsqueeze(1)
            hide = token > pos
            if c["window"]:
                hide |= (token <= pos - c["window"]) & (token >= c["sinks"])
            score = torch.einsum("hgnd,htd->hgnt", x, k) / math.sqrt(D)
            score.masked_fill_(hide, -math.inf)
            out[b, :, :, at: at + 256] = torch.einsum("hgnt,htd->hgnd", torch.softmax(score, -1), v)
    return out.flatten(1, 2)


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "write": _exact_write, "read": _exact_read, "attend": _exact_attend}[case["op"]](s)
