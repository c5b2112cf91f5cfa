"""Binding of the key/value cache in 8 bits and the attention over it (see
include/qkv_cte.h): writing, reading back, attention from one query on.

Argument marshalling only, with the rules of block_ops.py.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .block_ops import _DTYPE, _fits, _launch, _tensor, _vector
from .qkv_cte import (QKV_CTE_ERR_UNSUPPORTED, QkvCteError, _check, _cleared, _empty, _handle, _raw_stream, _side,
                      _used_on, _written, load, qkv_cte_status)

_QUERY = (torch.bfloat16, torch.float16)
_I32 = (torch.int32,)
_increment_version = torch.autograd.graph.increment_version
_NONE = (None, 0, 0, 0)


class qkv_cte_cache_desc(ctypes.Structure):
    _fields_ = [
        ("pages", ctypes.c_int64),
        ("n_kv_heads", ctypes.c_int32),
        ("d_head", ctypes.c_int32),
        ("block_tokens", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
    ]


class qkv_cte_cache_pages(ctypes.Structure):
    _fields_ = [
        ("k_codes", ctypes.c_void_p),
        ("k_sf", ctypes.c_void_p),
        ("v_codes", ctypes.c_void_p),
        ("v_sf", ctypes.c_void_p),
        ("table", ctypes.c_void_p),
        ("table_stride", ctypes.c_int64),
        ("max_blocks", ctypes.c_int32),
    ]


_bound = None


def _lib() -> ctypes.CDLL:
    """The library with the argument types of these entry points set."""
    global _bound
    if _bound is not None:
        return _bound
    lib = load()
    P, I64, I32, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    SIZE = ctypes.c_size_t
    PAGES = ctypes.POINTER(qkv_cte_cache_pages)
    lib.qkv_cte_cache_plan.argtypes = [ctypes.POINTER(P), ctypes.POINTER(qkv_cte_cache_desc), ctypes.POINTER(SIZE),
                                       ctypes.POINTER(SIZE)]
    lib.qkv_cte_cache_destroy.argtypes = [P]
    lib.qkv_cte_cache_destroy.restype = None
    lib.qkv_cte_cache_write.argtypes = [P, PAGES] + [P, I64, I64, I64] * 2 + [I64, I64, P, P, I32, P]
    lib.qkv_cte_cache_read.argtypes = [P, PAGES] + [P, I64, I64, I64] * 2 + [I64, I64, P, P, I32, P]
    lib.qkv_cte_cache_attention.argtypes = ([P, PAGES] + [P, I64, I64, I64] * 2
                                            + [P, I64, I64, I32, P, P, I64, F, I32, I32, I32, P, SIZE, P, P])
    lib.qkv_cte_cache_attention_workspace.argtypes = [P, I64, I64, I32, I64, ctypes.POINTER(SIZE)]
    for name in ("plan", "write", "read", "attention", "attention_workspace"):
        getattr(lib, "qkv_cte_cache_" + name).restype = ctypes.c_int
    _bound = lib
    return lib


def _heads(name: str, t, dtypes, device, heads, d, shape=None):
    """(address, batch, row and head stride), batch and seq of [B, S, heads, d] or [S, heads, d].
    What is right is tested first, with as few calls into torch as will do."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.device == device:
        s = t.shape
        if len(s) == 4 and s[3] == d and (heads is None or s[2] == heads) and (shape is None or s == shape):
            b, r, h, one = t.stride()
            if one == 1:
                return (t.data_ptr(), b, r, h), s[0], s[1]
    _tensor(name, t, dtypes, device)
    s, st = t.shape, t.stride()
    if len(s) not in (3, 4) or s[-1] != d or (heads is not None and s[-2] != heads):
        n = "heads" if heads is None else heads
        raise ValueError(f"{name}: expected [B, S, {n}, {d}] or [S, {n}, {d}], got {tuple(s)}")
    if shape is not None and s != shape:
        raise ValueError(f"{name}: shape {tuple(s)} is not {tuple(shape)}")
    if st[-1] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return (t.data_ptr(), 0, st[0], st[1]), 1, s[0]


class QkvCteCache:
    """Keys and values of attention in 8 bits: a pool of pages on one device.

    >>> cache = QkvCteCache(pages, n_kv_heads, d_head, block_tokens=64)
    >>> cache.write(k, v, starts, table=table)                    # out of the projection's output
    >>> out, _ = cache.attention(q, lengths, table=table, causal=True)
    >>> k, v = cache.read(starts, n, lengths, table=table)

    k, v: [B, S, n_kv_heads, d_head] or [S, n_kv_heads, d_head] of bf16, fp16 or fp32; q the
    same with its own number of heads, bf16 or fp16; any strides with contiguous lanes.
    starts, counts, lengths: int32 [B]. table: int32 [B, max_blocks] (or [max_blocks]: one for
    every sequence), the pages of each sequence in order; without one, sequence b owns
    pages // B pages from page b * (pages // B) on.

    The pool is allocated here, or given: k and v uint8 [pages, n_kv_heads, block_tokens,
    d_head] with k_sf and v_sf uint8 [pages, n_kv_heads]. Calls that write and calls that
    read the same pages must not overlap on the GPU; attention and read calls may run on
    any number of streams. The object may go while its calls are pending; a stream given as a
    raw handle has to outlive the object, and the object the graphs that captured its calls.
    The constructor waits for the stream that is current.
    """

    def __init__(self, pages: int, n_kv_heads: int, d_head: int, block_tokens: int = 64, device=None, k=None,
                 k_sf=None, v=None, v_sf=None, flags: int = 0):
        self.plan = None
        _fits("pages", pages, 63)
        for name, n in (("n_kv_heads", n_kv_heads), ("d_head", d_head), ("block_tokens", block_tokens),
                        ("flags", flags)):
            _fits(name, n)
        desc = qkv_cte_cache_desc(pages, n_kv_heads, d_head, block_tokens, flags)
        plan = ctypes.c_void_p()
        _check(_lib().qkv_cte_cache_plan(ctypes.byref(plan), ctypes.byref(desc), None, None))
        self.plan = plan
        self.pages, self.n_kv_heads, self.d_head, self.block_tokens = pages, n_kv_heads, d_head, block_tokens
        given = next((t for t in (k, k_sf, v, v_sf) if t is not None), None)
        if device is not None:
            dev = torch.device(device)
        elif isinstance(given, torch.Tensor):
            dev = given.device
        else:
            dev = torch.device("cuda", torch.cuda.current_device())
        if dev.type != "cuda":
            raise ValueError(f"device: {dev} is not a CUDA device")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        codes, scales = (pages, n_kv_heads, block_tokens, d_head), (pages, n_kv_heads)
        self._streams, self._own = {_raw_stream(dev.index)}, []  # streams the allocator knows to use what is ours

        def part(name, t, shape):
            if t is None:
                t = _cleared(shape, dev)
                self._own.append(t)
            elif not isinstance(t, torch.Tensor) or t.dim() != len(shape):
                raise ValueError(f"{name}: expected a tensor of shape {shape}")
            _vector(name, t, (torch.uint8,), dev, math.prod(shape))
            if tuple(t.shape) != shape:
                raise ValueError(f"{name}: shape {tuple(t.shape)} is not {shape}")
            return t

        self.k, self.v = part("k", k, codes), part("v", v, codes)
        self.k_sf, self.v_sf = part("k_sf", k_sf, scales), part("v_sf", v_sf, scales)
        self._status = _cleared(256, dev)
        self._own.append(self._status)
        self._base = (self.k.data_ptr(), self.k_sf.data_ptr(), self.v.data_ptr(), self.v_sf.data_ptr())
        self._needs = {}  # workspace bytes by sizes
        self._status_at = self._status.data_ptr()
        # version counters (inference tensors have none)
        self._k_counted, self._v_counted = ([t for t in pair if not t.is_inference()]
                                            for pair in ((self.k, self.k_sf), (self.v, self.v_sf)))

    def _pages(self, table, batch):
        """The table as the library takes it, and its positions per sequence."""
        if table is None:
            p, stride, blocks = None, 0, self.pages // batch if batch else 1
        elif (isinstance(table, torch.Tensor) and table.dtype is torch.int32 and table.device == self.device
              and len(table.shape) == 2 and table.shape[0] == batch > 1 and table.stride(1) == 1 and table.stride(0)):
            p, stride, blocks = table.data_ptr(), table.stride(0), table.shape[1]
        else:
            _tensor("table", table, _I32, self.device)
            if table.dim() not in (1, 2) or (table.dim() == 2 and table.shape[0] != batch):
                raise ValueError(f"table: expected [{batch}, blocks] or [blocks], got {tuple(table.shape)}")
            blocks = table.shape[-1]
            if blocks > 1 and table.stride(-1) != 1:
                raise ValueError("table: the last dimension must be contiguous")
            p, stride = table.data_ptr(), table.stride(0) if table.dim() == 2 and batch > 1 else 0
            if table.dim() == 2 and batch > 1 and stride == 0:
                raise ValueError("table: rows must not be expanded; give one row as [blocks]")
        if blocks >> 31:
            _fits("table", blocks)
        return qkv_cte_cache_pages(*self._base, p, stride, blocks), blocks * self.block_tokens

    def _index(self, name, t, batch):
        return _vector(name, t, _I32, self.device, batch)

    def _stream(self, stream):
        handle = _raw_stream(self.device.index) if stream is None else _handle(stream)
        if handle not in self._streams:
            for t in self._own:
                _used_on(t, set(), handle)
            self._streams.add(handle)
        return handle

    def write(self, k, v, starts, counts=None, table=None, stream=None):
        """Quantise k and v (one of them may be None) into the cache: row s < counts[b] (all
        rows without counts) becomes token starts[b] + s of sequence b."""
        first = k if k is not None else v
        if not isinstance(first, torch.Tensor):
            raise TypeError("k, v: expected a torch.Tensor")
        dt, n, d = first.dtype, self.n_kv_heads, self.d_head
        ak, batch, seq = _heads("k" if k is not None else "v", first, _DTYPE, self.device, n, d)
        if k is None:
            ak, av = _NONE, ak
        else:
            av = _heads("v", v, (dt,), self.device, n, d, first.shape)[0] if v is not None else _NONE
        pages, _ = self._pages(table, batch)
        ps, pc = self._index("starts", starts, batch), self._index("counts", counts, batch)
        _launch(_lib().qkv_cte_cache_write, self.device, self._stream(stream), self.plan, ctypes.byref(pages), *ak, *av,
                batch, seq, ps, pc, _DTYPE[dt])
        _increment_version((self._k_counted if k is not None else []) + (self._v_counted if v is not None else []))

    def read(self, starts, seq: int, lengths, table=None, dtype=torch.bfloat16, k=None, v=None, stream=None):
        """(k, v) [B, seq, n_kv_heads, d_head]: tokens starts[b] + s; zeros from lengths[b] on.
        Both are allocated here when neither is given; a given one alone is read alone."""
        _tensor("starts", starts, _I32, self.device)
        if starts.dim() != 1:
            raise ValueError(f"starts: expected one dimension, got {tuple(starts.shape)}")
        batch, n, d = starts.shape[0], self.n_kv_heads, self.d_head
        if seq < 0 or seq >> 31:
            raise QkvCteError(QKV_CTE_ERR_UNSUPPORTED, f"seq {seq} is not within 0 to 2^31 - 1")
        side = None if stream is None else _side(stream, self.device)
        given = None
        if k is None and v is None:
            if dtype not in _DTYPE:
                raise TypeError(f"dtype: {dtype} not in {tuple(_DTYPE)}")
            k, v = (_empty(side, (batch, seq, n, d), dtype, self.device) for _ in range(2))
            ak, av = ((t.data_ptr(), seq * n * d, n * d, d) for t in (k, v))
        else:
            given = k, v
            dtype = (k if k is not None else v).dtype
            args = []
            for name, t in (("k", k), ("v", v)):
                if t is None:
                    args.append(_NONE)
                    continue
                at, b, rows = _heads(name, t, (dtype,) if dtype in _DTYPE else _DTYPE, self.device, n, d)
                if (b, rows) != (batch, seq):
                    raise ValueError(f"{name}: shape {tuple(t.shape)} is not {(batch, seq, n, d)}")
                args.append(at)
            ak, av = args
        pages, _ = self._pages(table, batch)
        ps, pl = self._index("starts", starts, batch), self._index("lengths", lengths, batch)
        _launch(_lib().qkv_cte_cache_read, self.device, self._stream(stream), self.plan, ctypes.byref(pages), *ak, *av,
                batch, seq, ps, pl, _DTYPE[dtype])
        if given is not None:
            _written(*given)
        return k, v

    def attention_workspace(self, batch: int, seq: int, heads: int, max_length: int) -> int:
        """Workspace bytes of an attention call (a function of the sizes alone)."""
        key = batch, seq, heads, max_length
        need = self._needs.get(key)
        if need is None:
            _fits("heads", heads)
            for name, v in (("batch", batch), ("seq", seq), ("max_length", max_length)):
                _fits(name, v, 63)
            n = ctypes.c_size_t()
            _check(_lib().qkv_cte_cache_attention_workspace(self.plan, *key, ctypes.byref(n)))
            if len(self._needs) >= 256:
                self._needs.clear()
            self._needs[key] = need = n.value
        return need

    def attention(self, q, lengths, counts=None, table=None, causal: bool = False, window: int = 0, scale=None,
                  out=None, lse=None, stats: bool = False, max_length=None, workspace=None, stream=None):
        """(out, lse): attention of q [B, S, heads, d_head] or [S, heads, d_head] over the
        sequences' lengths[b] tokens. The queries are the last tokens of their sequence: row s
        < counts[b] (all rows without counts) stands at lengths[b] - counts[b] + s, which
        matters with `causal`; then `window` > 0 leaves each row the last `window` tokens. Rows
        that see nothing, and those from counts[b] on, are zeros. `scale`: 1 / sqrt(d_head) by
        default. The fp32 log-sum lse [..., heads] is written when given or asked for with
        `stats`, else None. `max_length`: a length that no sequence is expected to pass (by
        default what the table holds); only speed depends on it. Many rows of q and out want to
        start on 32-byte boundaries (see the header)."""
        dev, d = self.device, self.d_head
        aq, batch, seq = _heads("q", q, _QUERY, dev, None, d)
        heads, dt, shape = q.shape[-2], q.dtype, q.shape
        pages, capacity = self._pages(table, batch)
        pl, pc = self._index("lengths", lengths, batch), self._index("counts", counts, batch)
        if max_length is None:
            max_length = capacity
        if window >> 31:
            _fits("window", window)
        side = None if stream is None else _side(stream, dev)
        given = None if out is None and lse is None else (out, lse)
        if out is None:
            out = torch.empty(shape, dtype=dt, device=dev) if side is None else _empty(side, shape, dt, dev)
            ao = (out.data_ptr(), seq * heads * d, heads * d, d)
        else:
            ao = _heads("out", out, (dt,), dev, heads, d, shape)[0]
        if stats and lse is None:
            lse = _empty(side, shape[:-1], torch.float32, dev)
        pe = None
        if lse is not None:
            pe = _vector("lse", lse, (torch.float32,), dev, batch * seq * heads)
            if lse.dim() > 1 and lse.shape != shape[:-1]:
                raise ValueError(f"lse: shape {tuple(lse.shape)} is neither {tuple(shape[:-1])} nor flat")
        need, pw = self.attention_workspace(batch, seq, heads, max_length), None
        if need:
            if workspace is None:
                workspace = _empty(side, (need,), torch.uint8, dev)
            need = workspace.numel()
            pw = _vector("workspace", workspace, (torch.uint8,), dev, need)
        _launch(_lib().qkv_cte_cache_attention, dev, self._stream(stream), self.plan, ctypes.byref(pages), *aq, *ao, pe,
                batch, seq, heads, pl, pc, max_length, d ** -0.5 if scale is None else scale, 1 if causal else 0, window,
                _DTYPE[dt], pw, need, self._status_at)
        if given:
            _written(*given)
        return out, lse

    def status(self, stream=None) -> int:
        """Synchronise and raise QkvCteError if a bounded device wait of an attention call
        since the last call ran out."""
        with torch.cuda.device(self.device):
            return qkv_cte_status(self._status, stream)

    def close(self):
        if self.plan is not None:
            _lib().qkv_cte_cache_destroy(self.plan)
            self.plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
