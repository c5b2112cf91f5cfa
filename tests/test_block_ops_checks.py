"""CPU checks of the block operators' entry points: every refusal comes before any
launch, with its documented code (no GPU, the addresses are never read)."""
import ctypes

import pytest
import torch

import rope_tcgen05_mxfp8_gb300 as pkg
from rope_tcgen05_mxfp8_gb300 import block_ops as bo
from rope_tcgen05_mxfp8_gb300 import build as b
from rope_tcgen05_mxfp8_gb300 import qkv_cte as q

MB = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _built():
    b.build()


# --- layer norm ---------------------------------------------------------------------

LN = dict(x=16 * MB, ldx=64, w=1 * MB, b=2 * MB, y=32 * MB, ldy=64, mean=3 * MB, rstd=4 * MB, rows=8, cols=64,
          eps=1e-6, dtype=0, pdtype=0)


def _ln(**kw):
    a = dict(LN, **kw)
    return bo._lib().qkv_cte_layer_norm(a["x"], a["ldx"], a["w"], a["b"], a["y"], a["ldy"], a["mean"], a["rstd"],
                                        a["rows"], a["cols"], a["eps"], a["dtype"], a["pdtype"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(y=None), -1),
    (dict(rows=-1), -1), (dict(rows=0), 0), (dict(rows=0, x=None, y=None), 0), (dict(rows=2 ** 31), -2),
    (dict(cols=0), -1), (dict(cols=-5), -1), (dict(cols=2 ** 28 + 1, ldx=2 ** 29, ldy=2 ** 29), -2),
    (dict(eps=-1e-6), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1),
    (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(pdtype=1), -1), (dict(dtype=2, pdtype=0), -1),
    (dict(ldx=63), -1), (dict(ldy=63), -1), (dict(ldy=0), -1), (dict(ldx=-64), -1),
    (dict(ldx=2 ** 61), -2),
    (dict(x=16 * MB + 1), -2), (dict(y=32 * MB + 1), -2), (dict(mean=3 * MB + 2), -2), (dict(w=MB + 1), -2),
    (dict(pdtype=2, w=MB + 2), -2),
    (dict(y=16 * MB + 2), -1),                      # shifted by one element: neither the same nor disjoint
    (dict(y=16 * MB, ldy=128, ldx=64), -1),         # the same start, another stride
    (dict(mean=16 * MB), -1), (dict(rstd=32 * MB), -1), (dict(mean=4 * MB), -1), (dict(w=32 * MB), -1),
    (dict(w=3 * MB), -1),
    (dict(x=16 * MB, y=16 * MB + 100, ldx=128, ldy=128), -1),   # column ranges that share columns
])
def test_layer_norm_refusals(kw, code):
    assert _ln(**kw) == code
    if code:
        assert "qkv_cte_layer_norm" in q.qkv_cte_last_error()


LNB = dict(dy=16 * MB, lddy=64, x=32 * MB, ldx=64, w=1 * MB, mean=3 * MB, rstd=4 * MB, dx=48 * MB, lddx=64,
           dw=5 * MB, db=6 * MB, rows=8, cols=64, dtype=0, pdtype=0, ws=64 * MB, wsn=8 * 2 * 64 * 4)


def _lnb(**kw):
    a = dict(LNB, **kw)
    return bo._lib().qkv_cte_layer_norm_backward(
        a["dy"], a["lddy"], a["x"], a["ldx"], a["w"], a["mean"], a["rstd"], a["dx"], a["lddx"], a["dw"], a["db"],
        a["rows"], a["cols"], a["dtype"], a["pdtype"], a["ws"], a["wsn"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), -1), (dict(x=None), -1), (dict(mean=None), -1), (dict(rstd=None), -1),
    (dict(dx=None, dw=None, db=None), -1),
    (dict(rows=-1), -1), (dict(rows=2 ** 31), -2), (dict(cols=0), -1), (dict(rows=0, dw=None, db=None), 0),
    (dict(dtype=9), -1), (dict(pdtype=1), -1),
    (dict(lddy=32), -1), (dict(ldx=1), -1), (dict(lddx=0), -1),
    (dict(ws=None), -1), (dict(ws=64 * MB + 16), -2), (dict(wsn=8 * 2 * 64 * 4 - 1), -1), (dict(wsn=0), -1),
    (dict(ws=48 * MB), -1), (dict(ws=16 * MB), -1), (dict(ws=5 * MB), -1),
    (dict(dx=16 * MB + 2), -1), (dict(dx=32 * MB, lddx=128), -1), (dict(dx=1 * MB), -1),
    (dict(dw=6 * MB), -1), (dict(dw=1 * MB), -1), (dict(db=3 * MB), -1), (dict(dw=48 * MB), -1),
    (dict(dw=5 * MB + 1), -2), (dict(x=32 * MB + 1), -2),
])
def test_layer_norm_backward_refusals(kw, code):
    assert _lnb(**kw) == code


def test_layer_norm_backward_workspace_is_bounded():
    assert pkg.qkv_cte_layer_norm_backward_workspace(0, 64) == 0
    assert pkg.qkv_cte_layer_norm_backward_workspace(3, 64) == 3 * 2 * 64 * 4
    big = pkg.qkv_cte_layer_norm_backward_workspace(10 ** 6, 5120)
    assert big == pkg.qkv_cte_layer_norm_backward_workspace(10 ** 9, 5120) and big < 64 * MB
    for rows, cols, code in ((-1, 64, -1), (1, 0, -1), (2 ** 31, 64, -2)):
        with pytest.raises(pkg.QkvCteError) as ei:
            pkg.qkv_cte_layer_norm_backward_workspace(rows, cols)
        assert ei.value.code == code


# --- rotary positions -----------------------------------------------------------------

@pytest.mark.parametrize("d,dims,kw,code", [
    (128, (44, 42, 42), {}, 0), (128, (128,), {}, 0), (2, (2,), {}, 0), (512, (128,) * 4, {}, 0),
    (514, (514,), {}, -2), (127, (127,), {}, -1), (0, (0,), {}, -1), (128, (64, 62), {}, -1), (128, (64, 66), {}, -1),
    (128, (43, 43, 42), {}, -1), (128, (), {}, -1), (128, (128, 0), {}, -1), (10, (2,) * 5, {}, -1),
    (128, (128,), dict(theta=0.5), -1), (128, (128,), dict(theta=float("nan")), -1),
    (128, (128,), dict(theta=float("inf")), -1),
    (128, (128,), dict(spectrum=2), -1), (128, (128,), dict(pairing=-1), -1),
])
def test_rope_plan_validation(d, dims, kw, code):
    try:
        pkg.QkvCteRopeAxes(d, dims, **kw).close()
        got = 0
    except pkg.QkvCteError as e:
        got = e.code
    assert got == code


ROPE = dict(x=16 * MB, xb=0, xs=512, xh=128, y=32 * MB, yb=0, ys=512, yh=128, batch=1, seq=8, heads=4, pos=1 * MB,
            pstride=0, grids=None, dtype=0, inverse=0)


def _rope(plan, **kw):
    a = dict(ROPE, **kw)
    return bo._lib().qkv_cte_rope_apply(plan, a["x"], a["xb"], a["xs"], a["xh"], a["y"], a["yb"], a["ys"], a["yh"],
                                        a["batch"], a["seq"], a["heads"], a["pos"], a["pstride"], a["grids"],
                                        a["dtype"], a["inverse"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(y=None), -1), (dict(pos=None), -1), (dict(grids=2 * MB), -1),
    (dict(seq=0, x=None, y=None, pos=None), 0), (dict(heads=0), 0), (dict(batch=0), 0),
    (dict(seq=-1), -1), (dict(batch=-1), -1), (dict(heads=-1), -1), (dict(heads=2 ** 20), -2),
    (dict(batch=2 ** 20, seq=2 ** 20), -2), (dict(seq=2 ** 31), -2),
    (dict(dtype=3), -1), (dict(inverse=2), -1),
    (dict(x=16 * MB + 1), -2), (dict(pos=MB + 2), -2),
    (dict(ys=384), -1),                              # rows of 4 heads of 128 overlap
    (dict(yh=64), -1), (dict(ys=0), -1), (dict(batch=2, yb=0), -1), (dict(xs=-512), -1),
    (dict(xs=2 ** 62), -2),
    (dict(y=16 * MB + 2), -1), (dict(y=16 * MB, ys=1024), -1),
    (dict(xs=1024, ys=1024, y=16 * MB + 2 * 500), -1),  # column ranges that share columns
    (dict(y=1 * MB), -1),                            # the positions
    (dict(batch=2, xb=4096, yb=4096, pstride=16), -1),
])
def test_rope_refusals(kw, code):
    rope = pkg.QkvCteRopeAxes(128, (44, 42, 42))
    assert _rope(rope.plan, **kw) == code
    assert _rope(None, **kw) == -1


def test_rope_tables_refusals():
    rope = pkg.QkvCteRopeAxes(128, (44, 42, 42))
    f = bo._lib().qkv_cte_rope_tables
    ok = (rope.plan, 1, 8, MB, 0, None, 16 * MB, 32 * MB, None)
    for i, v, code in ((0, None, -1), (1, -1, -1), (2, -1, -1), (2, 0, 0), (3, None, -1), (5, 2 * MB, -1),
                       (6, None, -1), (7, None, -1), (6, 16 * MB + 4, -2), (7, 16 * MB, -1), (6, MB, -1),
                       (2, 2 ** 31, -2)):
        args = list(ok)
        args[i] = v
        assert f(*args) == code, (i, v)


# --- the binding's own checks ---------------------------------------------------------

def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.qkv_cte_layer_norm(x)
    with pytest.raises(TypeError):
        pkg.qkv_cte_layer_norm(x.double())
    with pytest.raises(TypeError):
        pkg.qkv_cte_layer_norm([1.0])
    rope = pkg.QkvCteRopeAxes(8, (8,))
    with pytest.raises(ValueError, match="CUDA"):
        rope(torch.zeros(2, 3, 8), positions=torch.zeros(2, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="positions or grids"):
        rope.tables(1, 4)


def test_new_entry_points_are_exported():
    lib = ctypes.CDLL(pkg.library_path())
    for name in ("qkv_cte_layer_norm", "qkv_cte_layer_norm_backward", "qkv_cte_layer_norm_backward_workspace",
                 "qkv_cte_rope_plan", "qkv_cte_rope_destroy", "qkv_cte_rope_tables", "qkv_cte_rope_apply"):
        assert hasattr(lib, name)


# --- the product ----------------------------------------------------------------------

@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(tokens=0), 0), (dict(tokens=1), 0), (dict(tokens=-1), -1), (dict(tokens=2 ** 31), -2),
    (dict(tokens=2 ** 31 - 1), -2), (dict(in_features=2 ** 30 + 32), -2),
    (dict(in_features=0), -1), (dict(in_features=48), -2), (dict(in_features=32), 0), (dict(in_features=-32), -1),
    (dict(out_features=0), -1), (dict(out_features=1), 0), (dict(out_features=2 ** 31 - 1), -2),
    (dict(act=4), -1), (dict(act=-1), -1), (dict(act=3), 0), (dict(out_dtype=3), -1), (dict(out_dtype=2), 0),
    (dict(input_layout=3), -1), (dict(flags=2), -1), (dict(flags=1), 0),
])
def test_linear_plan_validation(kw, code):
    a = dict(tokens=300, in_features=256, out_features=500, act=0, out_dtype=0, input_layout=0, flags=0)
    a.update(kw)
    plan, n = ctypes.c_void_p(), ctypes.c_size_t()
    lib = bo._lib()
    desc = bo.qkv_cte_linear_desc(*[a[k] for k, _ in bo.qkv_cte_linear_desc._fields_])
    assert lib.qkv_cte_linear_plan(ctypes.byref(plan), ctypes.byref(desc), ctypes.byref(n)) == code
    assert (plan.value is not None) == (code == 0)
    lib.qkv_cte_linear_destroy(plan)
    assert lib.qkv_cte_linear_plan(None, ctypes.byref(desc), ctypes.byref(n)) == -1


LIN = dict(A=16 * MB, a_scale=1 * MB, W=32 * MB, w_sf=48 * MB, col=2 * MB, bias=3 * MB, gate=4 * MB, res=64 * MB,
           ldr=512, O=80 * MB, ldo=512, ws=128 * MB, wsn=None)


@pytest.mark.parametrize("tokens", [3, 300])
@pytest.mark.parametrize("kw,code", [
    (dict(A=None), -1), (dict(W=None), -1), (dict(w_sf=None), -1), (dict(O=None), -1), (dict(ws=None), -1),
    (dict(a_scale=None), -1), (dict(wsn=255), -1),
    (dict(ldo=511), -1), (dict(ldr=511), -1), (dict(ldr=-1), -1), (dict(ldo=2 ** 61), -2),
    (dict(A=16 * MB + 8), -2), (dict(W=32 * MB + 8), -2), (dict(w_sf=48 * MB + 2), -2), (dict(O=80 * MB + 1), -2),
    (dict(res=64 * MB + 1), -2), (dict(bias=3 * MB + 8), -2), (dict(gate=4 * MB + 2), -2), (dict(col=2 * MB + 4), -2),
    (dict(a_scale=MB + 2), -2), (dict(ws=128 * MB + 128), -2),
    (dict(O=16 * MB), -1), (dict(O=32 * MB), -1), (dict(O=3 * MB), -1), (dict(O=128 * MB), -1), (dict(ws=16 * MB), -1),
    (dict(ws=64 * MB), -1), (dict(O=64 * MB + 2), -1), (dict(O=64 * MB, ldo=1024), -1),
    (dict(O=64 * MB + 1000, ldo=1024, ldr=1024), -1),
])
def test_linear_run_refusals(tokens, kw, code):
    plan, n = ctypes.c_void_p(), ctypes.c_size_t()
    lib = bo._lib()
    desc = bo.qkv_cte_linear_desc(tokens, 256, 512, 0, 0, 0, 0)
    assert lib.qkv_cte_linear_plan(ctypes.byref(plan), ctypes.byref(desc), ctypes.byref(n)) == 0
    a = dict(LIN, wsn=n.value)
    a.update(kw)
    got = lib.qkv_cte_linear_run(plan, a["A"], a["a_scale"], a["W"], a["w_sf"], a["col"], a["bias"], a["gate"], a["res"],
                                 a["ldr"], a["O"], a["ldo"], a["ws"], a["wsn"], None)
    lib.qkv_cte_linear_destroy(plan)
    assert got == code
    assert lib.qkv_cte_linear_run(None, *[None] * 8, 0, None, 0, None, 0, None) == -1


def test_linear_produced_inputs_take_no_scale():
    lib = bo._lib()
    for layout in (1, 2):
        plan, n = ctypes.c_void_p(), ctypes.c_size_t()
        desc = bo.qkv_cte_linear_desc(3, 256, 512, 0, 0, layout, 0)
        assert lib.qkv_cte_linear_plan(ctypes.byref(plan), ctypes.byref(desc), ctypes.byref(n)) == 0
        a = dict(LIN, wsn=n.value)
        got = lib.qkv_cte_linear_run(plan, a["A"], a["a_scale"], a["W"], a["w_sf"], None, None, None, None, 0, a["O"],
                                     512, a["ws"], a["wsn"], None)
        lib.qkv_cte_linear_destroy(plan)
        assert got == -1
