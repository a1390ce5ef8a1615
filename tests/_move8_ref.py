"""Plain forms of taking and keeping tokens of an 8-bit cache, on the CPU."""
from __future__ import annotations

import torch

from tests import _cache8_ref as ref

BLOCK = ref.BLOCK


def filled(b, h, capacity, fmt, dtype, lengths, seed, big=1.0):
    """A cache's arrays on the CPU (codes, scale, tail of K and of V, lengths), garbage behind each length."""
    g = torch.Generator().manual_seed(seed)
    n = max(max(lengths), 1)
    arrays = []
    for _ in range(2):
        rows = (torch.randn(b, h, n, 128, generator=g) * big).to(dtype)
        arrays.append(ref.held(rows, fmt, dtype, capacity, lengths, garbage=g))
    return arrays, list(lengths)


def copy(cache):
    return [tuple(t.clone() for t in x) for x in cache[0]], list(cache[1])


def decoded(code, scale, tail, length, block):
    """The rows of a block as the tail holds them: the tail itself for the last block, else code * scale in fp32, rounded."""
    if block == (length - 1) // BLOCK:
        return tail
    rows = code[:, block * BLOCK:(block + 1) * BLOCK].float() * scale[:, block, None, None]
    return rows.to(tail.dtype)


def take(to, source, sequences, lengths):
    """(what the cache holds after, set of sequences that are refused): sequences and lengths are lists or None."""
    out, bad = copy(to), set()
    for b in range(len(to[1])):
        s = b if sequences is None else sequences[b]
        if s == -1:
            continue
        if not 0 <= s < len(source[1]):
            bad.add(b)
            continue
        have = source[1][s]
        n = have if lengths is None else lengths[b]
        if not 0 <= n <= have or n > to[0][0][0].shape[2]:
            bad.add(b)
            continue
        for x in range(2):
            code, scale, tail = (t[s] for t in source[0][x])
            full = n // BLOCK
            out[0][x][0].view(torch.int8)[b, :, :full * BLOCK] = code.view(torch.int8)[:, :full * BLOCK]
            out[0][x][1][b, :, :full] = scale[:, :full]
            if n:
                out[0][x][2][b] = decoded(code, scale, tail, have, (n - 1) // BLOCK)
        out[1][b] = n
    return out, bad


def keep(to, source, blocks, counts):
    """The same for keep: blocks [B][H_kv][m] and counts as lists."""
    out, bad = copy(to), set()
    for b, count in enumerate(counts):
        if count == -1:
            continue
        have = source[1][b]
        full, part = have // BLOCK, have % BLOCK
        lists = blocks[b]
        if not 0 <= count <= min(full, len(lists[0])) or count * BLOCK + part > to[0][0][0].shape[2] or any(
                x[j] >= full or x[j] <= (x[j - 1] if j else -1) for x in lists for j in range(count)):
            bad.add(b)
            continue
        for x in range(2):
            for h, kept in enumerate(lists):
                code, scale, tail = (t[b] for t in source[0][x])
                for j, k in enumerate(kept[:count]):
                    out[0][x][0].view(torch.int8)[b, h, j * BLOCK:(j + 1) * BLOCK] = code.view(torch.int8)[h, k * BLOCK:(k + 1) * BLOCK]
                    out[0][x][1][b, h, j] = scale[h, k]
                if part or count:
                    out[0][x][2][b, h] = decoded(code, scale, tail, have, full if part else kept[count - 1])[h]
        out[1][b] = count * BLOCK + part
    return out, bad


def same(got, want):
    """Every array equal to the last bit, but for the tail's rows behind a sequence's last token."""
    assert got[1] == want[1], (got[1], want[1])
    for x, y in zip(got[0], want[0]):
        a, e = x[0].view(torch.int8), y[0].view(torch.int8)
        assert torch.equal(a, e), f"codes differ in sequences {sorted(set((a != e).nonzero()[:, 0].tolist()))}"
        assert torch.equal(x[1].view(torch.int32), y[1].view(torch.int32)), "scales differ"
        bits = torch.int16 if x[2].dtype == torch.bfloat16 else torch.int32
        for b, n in enumerate(want[1]):
            rows = (n - 1) % BLOCK + 1 if n else 0
            assert torch.equal(x[2][b, :, :rows].contiguous().view(bits), y[2][b, :, :rows].contiguous().view(bits)), f"the tail of sequence {b} differs"
