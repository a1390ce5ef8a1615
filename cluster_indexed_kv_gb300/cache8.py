"""Rotary positions, and the key/value cache held in 8 bits (include/lkv.h:
lkv_rope_*, lkv_cache8_*). ``Rope`` holds one table, ``Cache8`` one cache's
tensors; the methods run on the current stream of the tensors' device, allocate
only the outputs they return (and an attention's workspace, where it needs
one), and can be captured into CUDA graphs. They have no backward pass: a tensor
that requires a gradient is refused where gradients are recorded.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib

_DTYPES = {torch.float32: _lib.LKV_DTYPE_FP32, torch.bfloat16: _lib.LKV_DTYPE_BF16}
_CODES = {torch.int8: _lib.LKV_CODE_INT8, torch.float8_e4m3fn: _lib.LKV_CODE_E4M3}
_FORMATS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
_D = 128
_BLOCK = _lib.LKV_CACHE8_BLOCK
_SCALE = _D ** -0.5
_INT32 = 2 ** 31 - 1
# torch's allocation on the current CUDA device without its dispatcher, where
# this build of torch has it: a small call costs less than its outputs did
# (from call to call, 16 rows read back 11.7 -> 7.1 us, an attention 11.3 -> 8.1)
_empty_here = getattr(getattr(torch._C, "_dynamo", None), "guards", None)
_empty_here = getattr(_empty_here, "_empty_strided_cuda", None)


def _empty(shape, dtype, index) -> torch.Tensor:
    """A new contiguous tensor of shape (a tuple) [B, H, n, 128] on CUDA device `index`."""
    if _empty_here is not None and torch._C._cuda_getDevice() == index:
        row = shape[2] * _D
        return _empty_here(shape, (shape[1] * row, row, _D, 1), dtype)
    return torch.empty(shape, dtype=dtype, device=f"cuda:{index}")


def _tensor(t, name, shape, dtype, index) -> int:
    """Data pointer of a contiguous tensor of this shape and type on CUDA device `index`."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.shape == shape
            and t.is_contiguous()):
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} requires a gradient, and this call has none to give: use torch.no_grad() or {name}.detach()")
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _range(**sizes) -> None:
    """Refuse sizes that do not fit the call's int32; smaller ones below 0 are the call's to refuse."""
    for name, value in sizes.items():
        if not -_INT32 <= value <= _INT32:
            raise ValueError(f"{name} must be in 0..2^31 - 1")


def _call(index, fn, *args) -> None:
    """fn(*args, stream) on the device's current stream, with the device current."""
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        _lib._check(status, None)


class Rope:
    """A table of rotary positions (lkv_rope_init): layout "half" pairs values
    (i, i + rotary_dim / 2), "interleaved" (2 i, 2 i + 1); scaling "none",
    "linear", "ntk" or "yarn" stretches the positions by ``factor`` (YaRN with
    the ramp over turns of its formula; checkpoints may want one over pair
    indexes). ``table`` is what the calls read: for frequencies f_i of one's own,
    ``table.turn[i] = round(f_i / (2 * math.pi) * 2 ** 64)`` for each pair, and
    ``table.gain``.

    Positions on several axes (time, height, width; at most 4): ``sections``
    gives each axis a run of that many pairs, in order, which fill rotary_dim /
    2; or ``axes`` names the axis of each pair. With own_base the frequencies
    begin anew in each section, as if it were a rotation of 2 * section values."""

    def __init__(self, *, rotary_dim: int = _D, layout: str = "half", base: float = 10000.0,
                 scaling: str = "none", factor: float = 1.0, orig_len: int = 0,
                 beta_fast: float = 32.0, beta_slow: float = 1.0, sections=None, axes=None,
                 own_base: bool = False):
        if not 0 <= rotary_dim <= _INT32 or not 0 <= orig_len <= _INT32:
            raise ValueError("rotary_dim and orig_len must be in 0..2^31 - 1")
        lay = {"half": _lib.LKV_ROPE_HALF, "interleaved": _lib.LKV_ROPE_INTERLEAVED}[layout]
        how = {"none": _lib.LKV_ROPE_NONE, "linear": _lib.LKV_ROPE_LINEAR, "ntk": _lib.LKV_ROPE_NTK,
               "yarn": _lib.LKV_ROPE_YARN}[scaling]
        rest = (lay, how, orig_len, base, factor, beta_fast, beta_slow)
        self.table = _lib.lkv_rope_init(rotary_dim, *rest)
        self.n_axes = 0  # 0: positions are [B, n]
        if sections is not None:
            if axes is not None:
                raise ValueError("sections or axes, not both")
            sections = [int(s) for s in sections]
            if any(s < 1 for s in sections) or sum(sections) != rotary_dim // 2:
                raise ValueError(f"sections must be at least 1 each and {rotary_dim // 2} together, got {sections}")
            axes = [a for a, s in enumerate(sections) for _ in range(s)]
        elif own_base:
            raise ValueError("own_base without sections")
        if axes is not None:
            axes = [int(a) for a in axes]
            if len(axes) != rotary_dim // 2 or not all(0 <= a < _lib.LKV_ROPE_AXES for a in axes):
                raise ValueError(f"axes must name one of at most {_lib.LKV_ROPE_AXES} axes for each of {rotary_dim // 2} pairs")
            self.n_axes = max(axes) + 1
            self._axis = (C.c_uint8 * len(axes))(*axes)
        if own_base:
            at = 0
            for s in sections:
                t = _lib.lkv_rope_init(2 * s, *rest)
                self.table.turn[at:at + s] = t.turn[:s]
                at += s
        self._at = C.addressof(self.table)
        self._apply, self._apply_axes = _lib.load().lkv_rope_apply, _lib.load().lkv_rope_apply_axes

    def apply(self, q: torch.Tensor, positions: torch.Tensor, k: torch.Tensor | None = None, *,
              q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None):
        """Rotate q [B, H, n, 128] and, if given, k [B, H_kv, n, 128] by
        positions int32 [B, n], or [A, B, n] where the table has A axes.
        Returns q_out, or (q_out, k_out) with k; the outputs may be q and k
        themselves (in place), and are new tensors by default."""
        if not isinstance(q, torch.Tensor) or not q.is_cuda:
            raise ValueError("q must be a CUDA tensor")
        dt, dev, q_shape = q.dtype, q.get_device(), q.shape
        if dt not in _DTYPES:
            raise TypeError("q must be float32 or bfloat16")
        if len(q_shape) != 4 or q_shape[3] != _D:
            raise ValueError(f"q must have shape [B, H, n, {_D}], got {tuple(q_shape)}")
        batch, heads, n, _ = q_shape
        qp = _tensor(q, "q", q_shape, dt, dev)
        axes = self.n_axes
        pp = _tensor(positions, "positions", (axes, batch, n) if axes else (batch, n), torch.int32, dev)
        if q_out is None:
            q_out = _empty((batch, heads, n, _D), dt, dev)
            qo = q_out.data_ptr()
        else:
            qo = _tensor(q_out, "q_out", q_shape, dt, dev)
        kp = ko = None
        kv_heads = 0
        if k is not None:
            if not isinstance(k, torch.Tensor) or k.dim() != 4:
                raise ValueError(f"k must be a tensor of shape [B, H_kv, n, {_D}]")
            kv_heads = k.shape[1]
            shape = (batch, kv_heads, n, _D)
            kp = _tensor(k, "k", shape, dt, dev)
            if k_out is None:
                k_out = _empty(shape, dt, dev)
                ko = k_out.data_ptr()
            else:
                ko = _tensor(k_out, "k_out", shape, dt, dev)
        elif k_out is not None:
            raise ValueError("k_out without k")
        if axes:
            _call(dev, self._apply_axes, self._at, self._axis, axes, _DTYPES[dt], batch, heads, kv_heads, n, qp, kp,
                  pp, qo, ko)
        else:
            _call(dev, self._apply, self._at, _DTYPES[dt], batch, heads, kv_heads, n, qp, kp, pp,
                  qo, ko)
        return q_out if k is None else (q_out, k_out)


class Cache8:
    """A key/value cache held in 8 bits (lkv_cache8): ``k_codes``, ``v_codes``
    [B, H_kv, capacity, 128] (int8 or float8_e4m3fn), ``k_scale``, ``v_scale``
    fp32 [B, H_kv, capacity / 16], ``k_tail``, ``v_tail`` [B, H_kv, 16, 128]
    (the last block in full precision) and ``lengths`` int32 [B], all on the
    device and the caller's to read. Methods that write must not overlap, on
    the GPU, with others on the same cache."""

    def __init__(self, *, batch: int, n_kv_heads: int, capacity: int, dtype: torch.dtype,
                 fmt: str = "int8", device: torch.device | str = "cuda"):
        if fmt not in _FORMATS:
            raise ValueError('fmt must be "int8" or "e4m3"')
        if capacity < 1 or capacity % _BLOCK:
            raise ValueError(f"capacity must be a multiple of {_BLOCK}")
        slices = (batch, n_kv_heads)
        z = dict(device=device)
        codes = [torch.zeros(*slices, capacity, _D, dtype=torch.int8, **z).view(_FORMATS[fmt])
                 for _ in range(2)]
        scale = [torch.zeros(*slices, capacity // _BLOCK, dtype=torch.float32, **z) for _ in range(2)]
        tail = [torch.zeros(*slices, _BLOCK, _D, dtype=dtype, **z) for _ in range(2)]
        self._bind(*codes, *scale, *tail, torch.zeros(batch, dtype=torch.int32, **z))

    @classmethod
    def from_tensors(cls, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scale: torch.Tensor,
                     v_scale: torch.Tensor, k_tail: torch.Tensor, v_tail: torch.Tensor,
                     lengths: torch.Tensor) -> "Cache8":
        """A cache on tensors that already hold one (they are not copied)."""
        self = cls.__new__(cls)
        self._bind(k_codes, v_codes, k_scale, v_scale, k_tail, v_tail, lengths)
        return self

    def _bind(self, k_codes, v_codes, k_scale, v_scale, k_tail, v_tail, lengths):
        if not isinstance(k_codes, torch.Tensor) or not k_codes.is_cuda:
            raise ValueError("k_codes must be a CUDA tensor")
        if k_codes.dtype not in _CODES:
            raise TypeError("k_codes must be int8 or float8_e4m3fn")
        if k_codes.dim() != 4 or k_codes.shape[3] != _D or k_codes.shape[2] % _BLOCK:
            raise ValueError(f"k_codes must have shape [B, H_kv, capacity (a multiple of {_BLOCK}), {_D}]")
        if not isinstance(k_tail, torch.Tensor) or k_tail.dtype not in _DTYPES:
            raise TypeError("k_tail must be a float32 or bfloat16 tensor")
        self.batch, self.n_kv_heads, self.capacity, _ = k_codes.shape
        self.device, self.dtype = k_codes.device, k_tail.dtype
        slices, dev = (self.batch, self.n_kv_heads), k_codes.get_device()
        self._index = dev
        blocks, tails = (*slices, self.capacity // _BLOCK), (*slices, _BLOCK, _D)
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.k_tail, self.v_tail, self.lengths = k_tail, v_tail, lengths
        self._ticket = torch.zeros(self.batch + 1, dtype=torch.int32, device=self.device)
        self._view = _lib.lkv_cache8(
            self.batch, self.n_kv_heads, self.capacity, _DTYPES[self.dtype], _CODES[k_codes.dtype], 0,
            _tensor(k_codes, "k_codes", k_codes.shape, k_codes.dtype, dev),
            _tensor(v_codes, "v_codes", k_codes.shape, k_codes.dtype, dev),
            _tensor(k_scale, "k_scale", blocks, torch.float32, dev),
            _tensor(v_scale, "v_scale", blocks, torch.float32, dev),
            _tensor(k_tail, "k_tail", tails, self.dtype, dev),
            _tensor(v_tail, "v_tail", tails, self.dtype, dev),
            _tensor(lengths, "lengths", (self.batch,), torch.int32, dev),
            self._ticket.data_ptr())
        self._at = C.addressof(self._view)
        self._ws_bytes = {}  # workspace of an attention, by its sizes
        lib = _lib.load()
        self._write, self._read = lib.lkv_cache8_write, lib.lkv_cache8_read
        self._attend, self._status = lib.lkv_cache8_attend, lib.lkv_cache8_status
        self._attend_shared = lib.lkv_cache8_attend_shared
        self._take, self._keep = lib.lkv_cache8_take, lib.lkv_cache8_keep

    def write(self, k: torch.Tensor, v: torch.Tensor, *, start: torch.Tensor | None = None,
              counts: torch.Tensor | None = None) -> None:
        """Append k, v [B, H_kv, n, 128]: sequence b takes its first counts[b]
        rows (default: all n) at positions start[b].. (default: its length),
        and its length becomes start[b] + counts[b]. start may take back
        tokens of the last block, or down to a multiple of 16."""
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError(f"k must be a tensor of shape [B, H_kv, n, {_D}]")
        dev, dt, batch = self._index, self.dtype, self.batch
        shape = (batch, self.n_kv_heads, k.shape[2], _D)
        kp, vp = _tensor(k, "k", shape, dt, dev), _tensor(v, "v", shape, dt, dev)
        sp = None if start is None else _tensor(start, "start", (batch,), torch.int32, dev)
        cp = None if counts is None else _tensor(counts, "counts", (batch,), torch.int32, dev)
        _call(dev, self._write, self._at, kp, vp, shape[2], sp, cp)

    def read(self, n: int, *, first: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
             v_out: torch.Tensor | None = None):
        """Rows first[b] .. first[b] + n - 1 (default: from 0) of every
        sequence as (k, v) [B, H_kv, n, 128] of the cache's dtype; zeros
        outside a sequence. The layout is the one Context.build_index takes."""
        dev, dt = self._index, self.dtype
        if not 0 <= n <= _INT32:
            raise ValueError("n must be in 0..2^31 - 1")
        shape = (self.batch, self.n_kv_heads, n, _D)
        if k_out is None:
            k_out = _empty(shape, dt, dev)
        if v_out is None:
            v_out = _empty(shape, dt, dev)
        kp, vp = _tensor(k_out, "k_out", shape, dt, dev), _tensor(v_out, "v_out", shape, dt, dev)
        fp = None if first is None else _tensor(first, "first", (self.batch,), torch.int32, dev)
        _call(dev, self._read, self._at, fp, n, kp, vp)
        return k_out, v_out

    def _source(self, source) -> int:
        """Address of the cache that a take or keep reads."""
        if source is None:
            return self._at
        if not isinstance(source, Cache8):
            raise TypeError("source must be a Cache8")
        if source._index != self._index:
            raise ValueError(f"source must be on cuda:{self._index}, got cuda:{source._index}")
        return source._at

    def take(self, source: Cache8 | None = None, sequences: torch.Tensor | None = None,
             lengths: torch.Tensor | None = None) -> None:
        """Sequence b becomes the first lengths[b] tokens (default: all) of
        sequence sequences[b] (default: b; -1 leaves b as it is) of source, or
        of this cache itself, whose sequences then take what the others held
        before the call: samples of one prompt, beams put in order, sequences
        moved together, cut back at any token, freed (length 0). sequences and
        lengths are int32 [B]. Other batches and capacities of source fit."""
        dev, batch = self._index, self.batch
        at = self._source(source)
        sp = None if sequences is None else _tensor(sequences, "sequences", (batch,), torch.int32, dev)
        lp = None if lengths is None else _tensor(lengths, "lengths", (batch,), torch.int32, dev)
        ws_bytes = _lib.lkv_cache8_take_workspace(self._at, at)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=self.device) if ws_bytes else None
        _call(dev, self._take, self._at, at, sp, lp, ws.data_ptr() if ws_bytes else None, ws_bytes)

    def keep(self, blocks: torch.Tensor, counts: torch.Tensor, source: Cache8 | None = None) -> None:
        """Whole blocks of 16 tokens stay, or come from source (of the same
        batch), chosen for each KV head: block j < counts[b] of (b, h) becomes
        block blocks[b, h, j], and the partial block follows. blocks int32
        [B, H_kv, m], each list strictly ascending in its first counts[b]
        entries; counts int32 [B], -1 to leave a sequence as it is."""
        dev = self._index
        at = self._source(source)
        if not isinstance(blocks, torch.Tensor) or blocks.dim() != 3:
            raise ValueError("blocks must be a tensor of shape [B, H_kv, m]")
        m = blocks.shape[2]
        bp = _tensor(blocks, "blocks", (self.batch, self.n_kv_heads, m), torch.int32, dev)
        cp = _tensor(counts, "counts", (self.batch,), torch.int32, dev)
        _call(dev, self._keep, self._at, at, bp, m, cp)

    def attend(self, q: torch.Tensor, *, counts: torch.Tensor | None = None, scale: float | None = None,
               window: int = 0, sinks: int = 0, max_len: int = 0,
               out: torch.Tensor | None = None) -> torch.Tensor:
        """Causal attention of each sequence's last n tokens, whose keys and
        values the cache holds: q [B, H, n, 128], H a multiple of H_kv. With
        counts, the first counts[b] rows of sequence b are its last tokens and
        its other rows are padding (zero in the output). scale defaults to
        1 / sqrt(128). window > 0: a token sees the `window` last ones up to
        itself and the `sinks` first ones. max_len: a bound of the lengths
        known to the caller (0: none); it only steers the split of the work."""
        dev = self._index
        group, n, qp, cp, out, op = self._queries(q, counts, out)
        if not (0 <= window <= _INT32 and 0 <= sinks <= _INT32 and 0 <= max_len <= _INT32):
            _range(window=window, sinks=sinks, max_len=max_len)
        max_len = self._bound(max_len)
        sizes = (group, n, window, sinks, max_len)
        ws_bytes = self._ws_bytes.get(sizes)
        if ws_bytes is None:
            with torch.cuda.device(dev):
                ws_bytes = _lib.lkv_cache8_attend_workspace(self._at, *sizes)
            if len(self._ws_bytes) > 1000:
                self._ws_bytes.clear()
            self._ws_bytes[sizes] = ws_bytes
        # a new workspace for each call: calls on several streams do not share one
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=self.device) if ws_bytes else None
        _call(dev, self._attend, self._at, qp, group, n, cp, _SCALE if scale is None else scale, window,
              sinks, max_len, op, ws.data_ptr() if ws_bytes else None, ws_bytes)
        return out

    def attend_shared(self, q: torch.Tensor, prefix: Cache8, prefix_of: torch.Tensor | None = None, *,
                      counts: torch.Tensor | None = None, scale: float | None = None, max_len: int = 0,
                      out: torch.Tensor | None = None) -> torch.Tensor:
        """Causal attention of sequences behind shared prefixes: sequence b's
        tokens are those of sequence prefix_of[b] of the cache ``prefix`` (int32
        [B]; default 0 for all; -1: none), then its own here. q, counts, scale
        and out are attend's; q's rows are the sequence's last tokens. Each
        prefix is read once for all sequences behind it. max_len bounds this
        cache's lengths."""
        dev = self._index
        if not isinstance(prefix, Cache8):
            raise TypeError("prefix must be a Cache8")
        if prefix._index != dev:
            raise ValueError(f"prefix must be on cuda:{dev}, got cuda:{prefix._index}")
        group, n, qp, cp, out, op = self._queries(q, counts, out)
        pp = None if prefix_of is None else _tensor(prefix_of, "prefix_of", (self.batch,), torch.int32, dev)
        if not 0 <= max_len <= _INT32:
            raise ValueError("max_len must be in 0..2^31 - 1")
        max_len = self._bound(max_len)
        sizes = (prefix.batch, group, n, max_len)
        ws_bytes = self._ws_bytes.get(sizes)
        if ws_bytes is None:
            with torch.cuda.device(dev):
                ws_bytes = _lib.lkv_cache8_attend_shared_workspace(self._at, prefix._at, group, n, max_len)
            if len(self._ws_bytes) > 1000:
                self._ws_bytes.clear()
            self._ws_bytes[sizes] = ws_bytes
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=self.device) if ws_bytes else None
        _call(dev, self._attend_shared, self._at, prefix._at, pp, qp, group, n, cp, _SCALE if scale is None else scale,
              max_len, op, ws.data_ptr() if ws_bytes else None, ws_bytes)
        return out

    def _queries(self, q, counts, out):
        """Of an attention: group, n, addresses of q and counts, and the output with its address."""
        if not isinstance(q, torch.Tensor) or q.dim() != 4:
            raise ValueError(f"q must be a tensor of shape [B, H, n, {_D}]")
        dev, dt = self._index, self.dtype
        _, heads, n, _ = q.shape
        group = heads // self.n_kv_heads
        if group * self.n_kv_heads != heads or heads == 0:
            raise ValueError(f"q's {heads} heads are not a multiple of the cache's {self.n_kv_heads}")
        shape = (self.batch, heads, n, _D)
        qp = _tensor(q, "q", shape, dt, dev)
        cp = None if counts is None else _tensor(counts, "counts", (self.batch,), torch.int32, dev)
        if out is None:
            out = _empty(shape, dt, dev)
            return group, n, qp, cp, out, out.data_ptr()
        return group, n, qp, cp, out, _tensor(out, "out", shape, dt, dev)

    def _bound(self, max_len: int) -> int:
        """max_len in steps of a 64th to a 128th of itself (a server's bound that
        grows with every token does not ask for the workspace each time), 0 from
        the capacity on."""
        if max_len:
            step = (1 << max(4, max_len.bit_length() - 7)) - 1
            max_len = (max_len + step) & ~step
        return 0 if max_len >= self.capacity else max_len

    def check(self) -> None:
        """Wait for the current stream; raise LKVError if, since the last
        check, an attention, take or keep gave up waiting for its copies (what
        it made is not complete), a write, take or keep did not fit, or a write
        held a value that is not finite.
        Everything is reported once, in one error: the first of these that
        there is."""
        _call(self._index, self._status, self._at)
