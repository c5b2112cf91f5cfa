"""Bindings of the operators around the projection (see include/qkv_cte.h): layer norm
with its backward pass, rotary positions with several axes and the product with bias,
activation, gate and residual.

Argument marshalling only, as in qkv_cte.py: every computation runs in the library's
kernels. Tensors live on one CUDA device, which need not be the current one; a call
runs on `stream` (default: that device's current stream) and does not synchronise.
Results carry no autograd graph; tensors given for them count as modified in place.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence

import torch

from .qkv_cte import (QKV_CTE_ERR_UNSUPPORTED, QKV_CTE_INPUT_BF16, QKV_CTE_INPUT_PACKED,
                      QKV_CTE_INPUT_ROW_FP8, QkvCteError, _check, _cleared, _current_device, _empty, _raw_stream,
                      _handle, _side, _used_on, _written, load, qkv_cte_status)

QKV_CTE_DTYPE_BF16 = 0
QKV_CTE_DTYPE_FP16 = 1
QKV_CTE_DTYPE_FP32 = 2
QKV_CTE_ROPE_PER_AXIS = 0
QKV_CTE_ROPE_SHARED = 1
QKV_CTE_ROPE_ROTATE_HALF = 0
QKV_CTE_ROPE_INTERLEAVED = 1
QKV_CTE_ACT_NONE = 0
QKV_CTE_ACT_GELU_TANH = 1
QKV_CTE_ACT_GELU_ERF = 2
QKV_CTE_ACT_SILU = 3

_DTYPE = {torch.bfloat16: QKV_CTE_DTYPE_BF16, torch.float16: QKV_CTE_DTYPE_FP16, torch.float32: QKV_CTE_DTYPE_FP32}


class qkv_cte_rope_desc(ctypes.Structure):
    _fields_ = [
        ("d_head", ctypes.c_int32),
        ("n_axes", ctypes.c_int32),
        ("axis_dims", ctypes.c_int32 * 4),
        ("spectrum", ctypes.c_int32),
        ("pairing", ctypes.c_int32),
        ("theta", ctypes.c_double),
    ]


class qkv_cte_linear_desc(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int64),
        ("in_features", ctypes.c_int32),
        ("out_features", ctypes.c_int32),
        ("act", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("input_layout", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
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
    lib.qkv_cte_layer_norm.argtypes = [P, I64, P, P, P, I64, P, P, I64, I32, F, I32, I32, P]
    lib.qkv_cte_layer_norm_backward.argtypes = [P, I64, P, I64, P, P, P, P, I64, P, P, I64, I32, I32, I32, P, SIZE, P]
    lib.qkv_cte_layer_norm_backward_workspace.argtypes = [I64, I32, ctypes.POINTER(SIZE)]
    lib.qkv_cte_rope_plan.argtypes = [ctypes.POINTER(P), ctypes.POINTER(qkv_cte_rope_desc)]
    lib.qkv_cte_rope_destroy.argtypes = [P]
    lib.qkv_cte_rope_tables.argtypes = [P, I64, I64, P, I64, P, P, P, P]
    lib.qkv_cte_rope_apply.argtypes = [P, P, I64, I64, I64, P, I64, I64, I64, I64, I64, I32, P, I64, P, I32, I32, P]
    lib.qkv_cte_linear_plan.argtypes = [ctypes.POINTER(P), ctypes.POINTER(qkv_cte_linear_desc), ctypes.POINTER(SIZE)]
    lib.qkv_cte_linear_destroy.argtypes = [P]
    lib.qkv_cte_linear_run.argtypes = [P] * 9 + [I64, P, I64, P, SIZE, P]
    for name in ("layer_norm", "layer_norm_backward", "layer_norm_backward_workspace", "rope_plan", "rope_tables",
                 "rope_apply", "linear_plan", "linear_run"):
        getattr(lib, "qkv_cte_" + name).restype = ctypes.c_int
    lib.qkv_cte_rope_destroy.restype = None
    lib.qkv_cte_linear_destroy.restype = None
    _bound = lib
    return lib


def _fits(name: str, v, bits: int = 31):
    """v, refused where ctypes would cut it down to the C type's width without a word."""
    if not -1 << bits <= v < 1 << bits:
        raise QkvCteError(QKV_CTE_ERR_UNSUPPORTED, f"{name} {v} does not fit {bits + 1} bits")
    return v


def _launch(fn, device, stream, *args):
    """fn(*args, stream) with `device` current."""
    if stream is None:
        handle = _raw_stream(device.index)
    else:
        handle = stream if type(stream) is int else _handle(stream)
    if device.index == _current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, handle)
    if rc:
        _check(rc)


def _tensor(name: str, t, dtypes, device=None):
    """t, checked to be a CUDA tensor of one of `dtypes` (on `device`)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {tuple(dtypes)}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, not on {device}")
    return t


# The checks below test what is right first, with as few calls into torch as will do (a
# small kernel's call is bound by the host), and look for what is wrong afterwards.

def _vector(name: str, t, dtypes, device, n: int, last: int = 1) -> Optional[int]:
    """Address of a contiguous tensor of n elements, or None. `last`: the length of the last
    dimension of a tensor that is not flat (unless its order cannot matter)."""
    if t is None:
        return None
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.device == device and t.numel() == n
            and t.is_contiguous() and (last == 1 or n == last or t.dim() == 1 or t.shape[-1] == last)):
        return t.data_ptr()
    _tensor(name, t, dtypes, device)
    rows = f" in rows of {last}" if last != 1 else ""
    raise ValueError(f"{name}: must be contiguous with {n} elements{rows}, got shape {tuple(t.shape)}")


def _statistic(name: str, t, device, shape, rows: int) -> int:
    """Address of an fp32 value per row of a tensor of `shape`. Where that has several
    leading dimensions, t's have to be the same (those of one element aside) unless flat."""
    p = _vector(name, t, (torch.float32,), device, rows)
    if len(shape) > 2 and t.dim() > 1 and [v for v in t.shape if v != 1] != [v for v in shape[:-1] if v != 1]:
        raise ValueError(f"{name}: shape {tuple(t.shape)} is neither {tuple(shape[:-1])} nor flat")
    return p


def _rows(name: str, t, dtypes, device=None, shape=None):
    """(address, row stride) of [..., cols] as rows; the elements of a row are contiguous."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and (t.is_cuda if device is None else t.device == device):
        strides = t.stride()
        if len(strides) == 2 and strides[1] == 1 and (shape is None or t.shape == shape):
            return t.data_ptr(), strides[0]
    _tensor(name, t, dtypes, device)
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} is not {tuple(shape)}")
    if not strides:
        raise ValueError(f"{name}: needs at least one dimension")
    if t.shape[-1] > 1 and strides[-1] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if len(strides) == 1:
        return t.data_ptr(), t.shape[0]
    if len(strides) > 2:
        try:
            t = t.view(-1, t.shape[-1]) if t.numel() else t.reshape(-1, max(t.shape[-1], 1))
        except RuntimeError:
            raise ValueError(f"{name}: its rows must be evenly spaced") from None
    return t.data_ptr(), t.stride(0)


def qkv_cte_layer_norm(x, weight=None, bias=None, eps=1e-6, out=None, mean=None, rstd=None, stats=False, stream=None):
    """Layer norm over the last dimension of x [..., cols] (bf16, fp16 or fp32; rows may be
    strided). weight, bias: [cols] of x's type or fp32, or None. Returns (y, mean, rstd);
    the fp32 statistics [...] are written when given or asked for with `stats`, else None.
    `out` may be x."""
    px, ldx = _rows("x", x, _DTYPE)
    dev, shape, dt = x.device, x.shape, x.dtype
    cols = shape[-1]
    if cols >> 31:
        _fits("cols", cols)
    rows = x.numel() // cols if cols else 0
    param = weight if weight is not None else bias
    pdt = param.dtype if isinstance(param, torch.Tensor) else dt
    if pdt is not dt and pdt is not torch.float32:
        raise TypeError(f"weight and bias: dtype {pdt} is neither {dt} nor torch.float32")
    pw = _vector("weight", weight, (pdt,), dev, cols)
    pb = _vector("bias", bias, (pdt,), dev, cols)
    given = None if out is None and mean is None and rstd is None else (out, mean, rstd)
    side = None if stream is None else _side(stream, dev)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=dev) if side is None else _empty(side, shape, dt, dev)
        py, ldy = out.data_ptr(), cols
    else:
        py, ldy = _rows("out", out, (dt,), dev, shape)
    if stats:
        if mean is None:
            mean = _empty(side, shape[:-1], torch.float32, dev)
        if rstd is None:
            rstd = _empty(side, shape[:-1], torch.float32, dev)
    pm = None if mean is None else _statistic("mean", mean, dev, shape, rows)
    pr = None if rstd is None else _statistic("rstd", rstd, dev, shape, rows)
    _launch(_lib().qkv_cte_layer_norm, dev, stream, px, ldx, pw, pb, py, ldy, pm, pr, rows, cols, eps, _DTYPE[dt],
            _DTYPE[pdt])
    if given:
        _written(*given)
    return out, mean, rstd


@functools.lru_cache(maxsize=64)
def qkv_cte_layer_norm_backward_workspace(rows: int, cols: int) -> int:
    """Workspace bytes of qkv_cte_layer_norm_backward (a function of the sizes alone)."""
    n = ctypes.c_size_t()
    _check(_lib().qkv_cte_layer_norm_backward_workspace(_fits("rows", rows, 63), _fits("cols", cols), ctypes.byref(n)))
    return n.value


def qkv_cte_layer_norm_backward(dy, x, mean, rstd, weight=None, dx=None, dweight=None, dbias=None, workspace=None,
                                stream=None):
    """Gradients of qkv_cte_layer_norm: (dx, dweight, dbias), the outputs given, or, with
    none given, all three allocated here (dweight and dbias of weight's type, fp32 without
    a weight). mean, rstd: the forward pass's statistics. dx may be dy or x."""
    px, ldx = _rows("x", x, _DTYPE)
    dev, cols = x.device, x.shape[-1]
    if cols >> 31:
        _fits("cols", cols)
    rows = x.numel() // cols if cols else 0
    pg, ldg = _rows("dy", dy, (x.dtype,), dev, x.shape)
    param = weight if weight is not None else dweight if dweight is not None else dbias
    pdt = param.dtype if isinstance(param, torch.Tensor) else torch.float32
    if pdt not in (x.dtype, torch.float32):
        raise TypeError(f"weight, dweight and dbias: dtype {pdt} is neither {x.dtype} nor torch.float32")
    side = None if stream is None else _side(stream, dev)
    given = None
    if dx is None and dweight is None and dbias is None:
        if side is None:
            dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
            dweight = torch.empty(cols, dtype=pdt, device=dev)
            dbias = torch.empty(cols, dtype=pdt, device=dev)
        else:
            dx = _empty(side, x.shape, x.dtype, dev)
            dweight = _empty(side, (cols,), pdt, dev)
            dbias = _empty(side, (cols,), pdt, dev)
        pd, ldd, pdw, pdb = dx.data_ptr(), cols, dweight.data_ptr(), dbias.data_ptr()
    else:
        pd, ldd = _rows("dx", dx, (x.dtype,), dev, x.shape) if dx is not None else (None, 0)
        pdw = _vector("dweight", dweight, (pdt,), dev, cols)
        pdb = _vector("dbias", dbias, (pdt,), dev, cols)
        given = dx, dweight, dbias
    pw = _vector("weight", weight, (pdt,), dev, cols)
    pm = None if mean is None else _statistic("mean", mean, dev, x.shape, rows)
    pr = None if rstd is None else _statistic("rstd", rstd, dev, x.shape, rows)
    ws_bytes, pws = 0, None
    if (dweight is not None or dbias is not None) and rows:
        if workspace is None:
            workspace = _empty(side, (qkv_cte_layer_norm_backward_workspace(rows, cols),), torch.uint8, dev)
        ws_bytes = workspace.numel()
        pws = _vector("workspace", workspace, (torch.uint8,), dev, ws_bytes)
    _launch(_lib().qkv_cte_layer_norm_backward, dev, stream, pg, ldg, px, ldx, pw, pm, pr, pd, ldd, pdw, pdb, rows,
            cols, _DTYPE[x.dtype], _DTYPE[pdt], pws, ws_bytes)
    if given:
        _written(*given)
    return dx, dweight, dbias


class QkvCteRopeAxes:
    """Rotary positions with several axes: a plan for heads of `d_head` lanes of which
    axis i turns `axis_dims[i]`.

    >>> rope = QkvCteRopeAxes(128, (44, 42, 42))
    >>> cos, sin = rope.tables(1, 32760, grids=grids)      # what QkvCte takes
    >>> k = rope(k, positions=positions)                   # a tensor of its own

    A row stands either at positions[s] (int32 [S, axes], or [B, S, axes]) or at the s-th
    point of its batch's grid (grids: int32 [B, axes], last axis fastest; rows behind the
    grid's end are padding and not rotated). Flat tensors in that order are taken too.
    """

    def __init__(self, d_head: int, axis_dims: Sequence[int], theta: float = 10000.0,
                 spectrum: int = QKV_CTE_ROPE_PER_AXIS, pairing: int = QKV_CTE_ROPE_ROTATE_HALF):
        self.plan = None
        dims = [_fits("axis_dims", int(v)) for v in axis_dims]
        for name, v in (("d_head", d_head), ("spectrum", spectrum), ("pairing", pairing)):
            _fits(name, v)
        desc = qkv_cte_rope_desc(d_head, len(dims), (ctypes.c_int32 * 4)(*dims[:4]), spectrum, pairing, theta)
        plan = ctypes.c_void_p()
        _check(_lib().qkv_cte_rope_plan(ctypes.byref(plan), ctypes.byref(desc)))
        self.plan = plan
        self.d_head, self.n_axes = d_head, len(dims)

    def _where(self, batch, seq, positions, grids, device):
        if (positions is None) == (grids is None):
            raise ValueError("give positions or grids (one of them)")
        if grids is not None:
            return None, 0, _vector("grids", grids, (torch.int32,), device, batch * self.n_axes, self.n_axes)
        one = seq * self.n_axes
        per_batch = isinstance(positions, torch.Tensor) and positions.dim() == 3
        if per_batch and positions.shape[:2] != (batch, seq):
            raise ValueError(f"positions: shape {tuple(positions.shape)} is not {(batch, seq, self.n_axes)}")
        p = _vector("positions", positions, (torch.int32,), device, one * batch if per_batch else one, self.n_axes)
        return p, one if per_batch else 0, None

    def tables(self, batch: int, seq: int, positions=None, grids=None, cos=None, sin=None, stream=None):
        """(cos, sin): fp32 [batch * seq, d_head], allocated here when not given."""
        where = grids if grids is not None else positions
        if not isinstance(where, torch.Tensor):
            raise ValueError("give positions or grids (one of them)")
        dev = where.device
        if not where.is_cuda:
            raise ValueError("positions and grids: must be CUDA tensors")
        p, stride, g = self._where(batch, seq, positions, grids, dev)
        given = None if cos is None and sin is None else (cos, sin)
        n, d, f32 = batch * seq, self.d_head, (torch.float32,)
        side = None if stream is None else _side(stream, dev)
        if cos is None:
            cos = _empty(side, (n, d), torch.float32, dev)
        if sin is None:
            sin = _empty(side, (n, d), torch.float32, dev)
        if given is None:
            pc, ps = cos.data_ptr(), sin.data_ptr()
        else:
            pc, ps = _vector("cos", cos, f32, dev, n * d, d), _vector("sin", sin, f32, dev, n * d, d)
        _launch(_lib().qkv_cte_rope_tables, dev, stream, self.plan, batch, seq, p, stride, g, pc, ps)
        if given:
            _written(*given)
        return cos, sin

    def __call__(self, x, positions=None, grids=None, out=None, inverse=False, stream=None):
        """x [B, S, heads, d_head] or [S, heads, d_head] rotated (turned back with
        `inverse`: the rotation's gradient); any strides with contiguous lanes. `out` may be x."""
        _tensor("x", x, _DTYPE)
        dev, shape, dt, sx = x.device, x.shape, x.dtype, x.stride()
        if len(shape) not in (3, 4) or shape[-1] != self.d_head:
            raise ValueError(f"x: expected [B, S, heads, {self.d_head}] or [S, heads, {self.d_head}], "
                             f"got {tuple(shape)}")
        if sx[-1] != 1:
            raise ValueError("x: the last dimension must be contiguous")
        given = out
        if out is None:
            side = None if stream is None else _side(stream, dev)
            out = torch.empty(shape, dtype=dt, device=dev) if side is None else _empty(side, shape, dt, dev)
        else:
            _tensor("out", out, (dt,), dev)
            if out.shape != shape:
                raise ValueError(f"out: shape {tuple(out.shape)} is not {tuple(shape)}")
        sy = out.stride()
        if sy[-1] != 1:
            raise ValueError("out: the last dimension must be contiguous")
        batch, bx, by = (shape[0], sx[0], sy[0]) if len(shape) == 4 else (1, 0, 0)
        seq, heads = shape[-3], shape[-2]
        if heads >> 31:
            _fits("heads", heads)
        p, stride, g = self._where(batch, seq, positions, grids, dev)
        _launch(_lib().qkv_cte_rope_apply, dev, stream, self.plan, x.data_ptr(), bx, sx[-3], sx[-2], out.data_ptr(),
                by, sy[-3], sy[-2], batch, seq, heads, p, stride, g, _DTYPE[dt], 1 if inverse else 0)
        if given is not None:
            _written(given)
        return out

    def close(self):
        if self.plan is not None:
            _lib().qkv_cte_rope_destroy(self.plan)
            self.plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_BF16_BITS = (torch.bfloat16, torch.int16, torch.uint16)


class QkvCteLinear:
    """The product with bias, activation, gate and residual: a plan plus its workspace on
    one device.

    >>> op = QkvCteLinear(tokens, 5120, 20480, act=QKV_CTE_ACT_GELU_TANH, input_layout=QKV_CTE_INPUT_BF16)
    >>> h = op(x, None, W, w_sf, bias=b)
    >>> x = out_proj(A, a_scale, W, w_sf, bias=b, gate=g, residual=x, out=x)

    A [T, K], a_scale [T], W [N, K] and w_sf [N, K/32] are the operands of QkvCte (flat, or
    with more leading dimensions: the last one counts); `residual` and `out` are [T, N] of
    `out_dtype` with contiguous rows (strided rows are fine, and `out` may be `residual`).
    Calls that overlap on the GPU need an object each: they would share the workspace. The
    first call may run on any stream, and the object may go while its calls are pending; a
    stream given as a raw handle has to outlive the object, and the object the graphs that
    captured its calls. The constructor waits for the stream that is current.
    """

    def __init__(self, tokens: int, in_features: int, out_features: int, act: int = QKV_CTE_ACT_NONE,
                 out_dtype=torch.bfloat16, input_layout: int = QKV_CTE_INPUT_ROW_FP8, device=None, flags: int = 0):
        self.plan = None
        if out_dtype not in _DTYPE:
            raise TypeError(f"out_dtype: {out_dtype} not in {tuple(_DTYPE)}")
        _fits("tokens", tokens, 63)
        for name, v in (("in_features", in_features), ("out_features", out_features), ("act", act),
                        ("input_layout", input_layout), ("flags", flags)):
            _fits(name, v)
        desc = qkv_cte_linear_desc(tokens, in_features, out_features, act, _DTYPE[out_dtype], input_layout, flags)
        plan, n = ctypes.c_void_p(), ctypes.c_size_t()
        _check(_lib().qkv_cte_linear_plan(ctypes.byref(plan), ctypes.byref(desc), ctypes.byref(n)))
        self.plan, self.workspace_bytes = plan, n.value
        self.shape, self.in_features, self.out_dtype, self.input_layout = (
            (tokens, out_features), in_features, out_dtype, input_layout)
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        if dev.type != "cuda":
            raise ValueError(f"device: {dev} is not a CUDA device")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self.workspace = _cleared(max(self.workspace_bytes, 256), dev)
        self._streams = {_raw_stream(dev.index)}  # those the allocator knows to use the workspace

    def __call__(self, A, a_scale, W, w_sf, bias=None, gate=None, residual=None, out=None, w_col_scale=None,
                 stream=None):
        (T, N), K, dev = self.shape, self.in_features, self.device
        layout = self.input_layout
        row = K + 4 if layout == QKV_CTE_INPUT_PACKED else K
        pa = _vector("A", A, _BF16_BITS if layout == QKV_CTE_INPUT_BF16 else (torch.uint8,), dev, T * row, row)
        ps = _vector("a_scale", a_scale, (torch.float32,), dev, T)
        pw = _vector("W", W, (torch.uint8,), dev, N * K, K)
        pf = _vector("w_sf", w_sf, (torch.uint8,), dev, N * (K // 32), K // 32)
        pc = _vector("w_col_scale", w_col_scale, (torch.float32,), dev, N)
        pb = _vector("bias", bias, _BF16_BITS, dev, N)
        pg = _vector("gate", gate, _BF16_BITS, dev, N)
        pr, ldr = _rows("residual", residual, (self.out_dtype,), dev, (T, N)) if residual is not None else (None, 0)
        given = out
        if out is None:
            side = None if stream is None else _side(stream, dev)
            out = (torch.empty(self.shape, dtype=self.out_dtype, device=dev) if side is None
                   else _empty(side, self.shape, self.out_dtype, dev))
        po, ldo = _rows("out", out, (self.out_dtype,), dev, (T, N))
        handle = _raw_stream(dev.index) if stream is None else _handle(stream)
        if handle not in self._streams:
            _used_on(self.workspace, self._streams, handle)
        _launch(_lib().qkv_cte_linear_run, dev, handle, self.plan, pa, ps, pw, pf, pc, pb, pg, pr, ldr, po, ldo,
                self.workspace.data_ptr(), self.workspace.numel())
        if given is not None:
            _written(given)
        return out

    def status(self, stream=None) -> int:
        """Synchronise and raise QkvCteError if a bounded device wait of a run since the
        last call ran out."""
        with torch.cuda.device(self.device):
            return qkv_cte_status(self.workspace, stream)

    def close(self):
        if self.plan is not None:
            _lib().qkv_cte_linear_destroy(self.plan)
            self.plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
