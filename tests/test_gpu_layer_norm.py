"""Layer norm and its gradients against a plain implementation in 64 bits.

Tolerances. u = 2^-24 (half an fp32 step), h = eps(type)/2 (half a step of the output's
type). A thread adds at most 64 elements of a row one after the other and the group
joins its threads in at most 11 levels, so a row sum is off by at most 80 u times the
sum of its terms' magnitudes, whatever their order within that scheme."""
import pytest
import torch

import rope_tcgen05_mxfp8_gb300 as lib

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
K = 80
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _half_step(dt):
    return torch.finfo(dt).eps / 2, torch.finfo(dt).tiny * torch.finfo(dt).eps / 2  # relative, subnormal


def _inputs(rows, cols, dt, pt, seed, offset=0.3):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device=DEV) + offset * torch.randn(rows, 1, generator=g, device=DEV)
    w = 1 + 0.3 * torch.randn(cols, generator=g, device=DEV)
    b = 0.3 * torch.randn(cols, generator=g, device=DEV)
    dy = torch.randn(rows, cols, generator=g, device=DEV)
    return x.to(dt), w.to(pt), b.to(pt), dy.to(dt)


def _reference(x, w, b, eps):
    x = x.double()
    mean = x.mean(-1)
    var = ((x - mean[..., None]) ** 2).mean(-1)
    rstd = (var + eps) ** -0.5
    xh = (x - mean[..., None]) * rstd[..., None]
    y = xh * (1 if w is None else w.double()) + (0 if b is None else b.double())
    return y, mean, rstd, xh


def _check_forward(x, w, b, eps, y, mean, rstd):
    ry, rm, rr, xh = _reference(x, w, b, eps)
    big = x.double().abs().amax(-1)
    # mean: the sum's error and one rounding each of the sum's scaling and 1/cols
    em = (K + 2) * U * big
    # rstd: the variance is a mean of squares about the computed mean (an error of em in
    # it adds em^2 to the variance, and em times the mean residual, which is at most em
    # again); each square is off by 3 u and by 2 em |x - mean|
    dev = (x.double() - rm[..., None]).abs()
    ev = (K + 6) * U * (dev ** 2).mean(-1) + 2 * em * dev.mean(-1) * 2 * U + 2 * em ** 2 + 2 * U * dev.mean(-1) * big
    er = 0.5 * rr ** 3 * ev + 4 * U * rr
    if mean is not None:
        assert bool(((mean.double() - rm).abs() <= em + U * rm.abs()).all())
        assert bool(((rstd.double() - rr).abs() <= 1.1 * er).all())
    h, sub = _half_step(y.dtype)
    wv = torch.ones_like(xh[0]) if w is None else w.double().abs()
    exh = (em + U * big)[..., None] * rr[..., None] + 1.1 * dev * er[..., None] + 2 * U * xh.abs()
    tol = h * ry.abs() + sub + 1.01 * (wv * exh) + U * (ry.abs() + wv * xh.abs())
    err = (y.double() - ry).abs()
    assert bool((err <= tol).all()), f"worst excess {(err - tol).max().item():.3e}"


SHAPES = [(1, 1), (3, 1), (2, 2), (5, 7), (1, 64), (33, 128), (7, 1000), (4, 1024), (9, 1283), (6, 5120), (2, 8191),
          (3, 16384), (2, 20480), (1, 40000), (700, 264)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("x,p", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
def test_forward(rows, cols, x, p):
    xt, w, b, _ = _inputs(rows, cols, TYPES[x], TYPES[p], rows * 31 + cols)
    y, mean, rstd = lib.qkv_cte_layer_norm(xt, w, b, eps=1e-5, stats=True)
    assert y.dtype == xt.dtype and mean.shape == (rows,)
    _check_forward(xt, w, b, 1e-5, y, mean, rstd)


@pytest.mark.parametrize("w,b", [(False, False), (True, False), (False, True)])
def test_forward_without_parameters(w, b):
    xt, wt, bt, _ = _inputs(5, 5120, torch.bfloat16, torch.float32, 3)
    wt, bt = wt if w else None, bt if b else None
    y, mean, rstd = lib.qkv_cte_layer_norm(xt, wt, bt, eps=1e-6)
    assert mean is None and rstd is None
    _check_forward(xt, wt, bt, 1e-6, y, None, None)


def test_forward_far_mean_keeps_the_variance():
    """A row offset a thousand times its spread: the variance is taken about the mean."""
    xt, w, b, _ = _inputs(8, 4096, torch.float32, torch.float32, 5)
    xt = xt + 1000.0
    y, mean, rstd = lib.qkv_cte_layer_norm(xt, w, b, stats=True)
    _check_forward(xt, w, b, 1e-6, y, mean, rstd)


def test_forward_constant_rows_and_non_finite_rows():
    x = torch.full((4, 640), 3.0, device=DEV, dtype=torch.bfloat16)
    x[1, 5], x[2, 6] = float("inf"), float("nan")
    w, b = torch.ones(640, device=DEV), torch.full((640,), 0.25, device=DEV)
    y, mean, rstd = lib.qkv_cte_layer_norm(x, w, b, eps=1e-6, stats=True)
    assert bool((y[0] == 0.25).all()) and bool((y[3] == 0.25).all())       # no deviation: the bias
    assert abs(rstd[0].item() - 1000.0) < 1e-3
    assert bool(y[1].isnan().all()) and bool(y[2].isnan().all())           # only their own rows
    y0 = lib.qkv_cte_layer_norm(x, w, b, eps=0.0)[0]
    assert bool(y0[0].isnan().all())                                       # 0 / 0, as the formula says


@pytest.mark.parametrize("cols,pad,shift", [(640, 8, 0), (640, 3, 1), (77, 5, 0), (5120, 64, 4)])
def test_forward_strided_shifted_and_in_place(cols, pad, shift):
    rows = 13
    wide = torch.full((rows, cols + pad + shift), 7.0, dtype=torch.bfloat16, device=DEV)
    xt, w, b, _ = _inputs(rows, cols, torch.bfloat16, torch.bfloat16, cols)
    view = wide[:, shift: shift + cols]
    view.copy_(xt)
    out = torch.full_like(wide, 9.0)
    y, _, _ = lib.qkv_cte_layer_norm(view, w, b, out=out[:, shift: shift + cols])
    _check_forward(xt, w, b, 1e-6, y, None, None)
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[:, shift: shift + cols] = False
    assert bool((out[keep] == 9.0).all())                                  # nothing between the rows
    lib.qkv_cte_layer_norm(view, w, b, out=view)
    assert torch.equal(view, y) and bool((wide[keep] == 7.0).all())


def test_forward_broadcast_row_and_leading_dimensions():
    xt, w, b, _ = _inputs(1, 256, torch.float32, torch.float32, 9)
    y, _, _ = lib.qkv_cte_layer_norm(xt.expand(6, 256), w, b)
    assert y.shape == (6, 256) and bool((y == y[0]).all())
    x3 = xt.expand(6, 256).reshape(2, 3, 256).contiguous()
    y3, mean, _ = lib.qkv_cte_layer_norm(x3, w, b, stats=True)
    assert y3.shape == (2, 3, 256) and mean.shape == (2, 3) and torch.equal(y3.reshape(6, 256), y)


def test_empty():
    x = torch.empty(0, 64, device=DEV)
    y, mean, rstd = lib.qkv_cte_layer_norm(x, stats=True)
    assert y.shape == (0, 64) and mean.numel() == 0
    dx, dw, db = lib.qkv_cte_layer_norm_backward(x, x, mean, rstd, torch.ones(64, device=DEV))
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())


def _check_backward(dy, x, mean, rstd, w, dx, dw, db):
    d, r = dy.double(), rstd.double()[..., None]
    xh = (x.double() - mean.double()[..., None]) * r
    g = d * (1 if w is None else w.double())
    n = x.shape[-1]
    c1, c2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    if dx is not None:
        ref = r * (g - c1 - xh * c2)
        e1 = (K + 3) * U * g.abs().mean(-1, keepdim=True)
        e2 = (K + 7) * U * (g * xh).abs().mean(-1, keepdim=True)
        each = 3 * U * g.abs() + 2 * U * c1.abs() + 6 * U * (xh * c2).abs() + e1 + xh.abs() * e2
        h, sub = _half_step(dx.dtype)
        tol = h * ref.abs() + sub + 1.01 * (r.abs() * each + 2 * U * ref.abs())
        err = (dx.double() - ref).abs()
        assert bool((err <= tol).all()), f"dx: worst excess {(err - tol).max().item():.3e}"
    rows = d.reshape(-1, n).shape[0]
    for got, terms, name in ((dw, d * xh, "dweight"), (db, d, "dbias")):
        if got is None:
            continue
        terms = terms.reshape(-1, n)
        ref, mag = terms.sum(0), terms.abs().sum(0)
        h, sub = _half_step(got.dtype)
        # any order of adding `rows` terms, each off by 4 u
        tol = h * ref.abs() + sub + 1.01 * (rows + 4) * U * mag
        err = (got.double() - ref).abs()
        assert bool((err <= tol).all()), f"{name}: worst excess {(err - tol).max().item():.3e}"


def _saved(x, eps=1e-5):
    _, m, r, _ = _reference(x, None, None, eps)
    return m.float(), r.float()


@pytest.mark.parametrize("rows,cols", SHAPES + [(2000, 96), (5000, 8)])
@pytest.mark.parametrize("x,p", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
def test_backward(rows, cols, x, p):
    xt, w, _, dy = _inputs(rows, cols, TYPES[x], TYPES[p], rows * 17 + cols)
    mean, rstd = _saved(xt)
    dx, dw, db = lib.qkv_cte_layer_norm_backward(dy, xt, mean, rstd, w)
    assert dw.dtype == w.dtype and dx.dtype == xt.dtype
    _check_backward(dy, xt, mean, rstd, w, dx, dw, db)
    again = lib.qkv_cte_layer_norm_backward(dy, xt, mean, rstd, w)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), again))     # a fixed order of sums


@pytest.mark.parametrize("which", [("dx",), ("dweight",), ("dbias",), ("dx", "dbias")])
@pytest.mark.parametrize("cols", [640, 77, 30000])
def test_backward_single_outputs_and_no_weight(which, cols):
    xt, _, _, dy = _inputs(11, cols, torch.bfloat16, torch.float32, 4)
    mean, rstd = _saved(xt)
    outs = {n: torch.full((cols,), 5.0, device=DEV) for n in which if n != "dx"}
    if "dx" in which:
        outs["dx"] = torch.empty_like(xt)
    dx, dw, db = lib.qkv_cte_layer_norm_backward(dy, xt, mean, rstd, None, **outs)
    assert (dx is not None, dw is not None, db is not None) == tuple(n in which for n in ("dx", "dweight", "dbias"))
    _check_backward(dy, xt, mean, rstd, None, dx, dw, db)


@pytest.mark.parametrize("cols", [640, 333])
def test_backward_strided_and_in_place(cols):
    xt, w, _, dy = _inputs(9, cols, torch.bfloat16, torch.bfloat16, 6)
    mean, rstd = _saved(xt)
    wide = torch.zeros(9, 2 * cols + 3, dtype=torch.bfloat16, device=DEV)
    xv, gv = wide[:, :cols], wide[:, cols + 1: 2 * cols + 1]
    xv.copy_(xt)
    gv.copy_(dy)
    ref = lib.qkv_cte_layer_norm_backward(dy, xt, mean, rstd, w)
    got = lib.qkv_cte_layer_norm_backward(gv, xv, mean, rstd, w)
    _check_backward(dy, xt, mean, rstd, w, *got)
    dw, db = torch.empty_like(w), torch.empty_like(w)
    dx, _, _ = lib.qkv_cte_layer_norm_backward(gv, xv, mean, rstd, w, dx=gv, dweight=dw, dbias=db)
    assert dx is gv and torch.equal(gv, got[0]) and torch.equal(xv, xt)
    _check_backward(dy, xt, mean, rstd, w, ref[0], dw, db)


def test_gradient_against_differences():
    """The gradients against central differences of the forward pass's definition, in 64 bits."""
    xt, w, b, dy = _inputs(3, 24, torch.float32, torch.float32, 8)
    y, mean, rstd = lib.qkv_cte_layer_norm(xt, w, b, eps=1e-5, stats=True)
    dx, dw, db = lib.qkv_cte_layer_norm_backward(dy, xt, mean, rstd, w)
    loss = lambda x, w, b: (_reference(x, w, b, 1e-5)[0] * dy.double()).sum()  # noqa: E731
    step = 2.0 ** -17
    for t, grad, i in ((xt, dx, 0), (w, dw, 1), (b, db, 2)):
        for j in range(0, t.numel(), 5):
            args = [xt.double(), w.double(), b.double()]
            lo, hi = args[i].clone(), args[i].clone()
            lo.view(-1)[j] -= step
            hi.view(-1)[j] += step
            args[i] = hi
            up = loss(*args)
            args[i] = lo
            diff = (up - loss(*args)) / (2 * step)
            # the difference's own error: third derivatives (of order 100 at this spread)
            # times step^2 / 6, about 1e-9; the fp32 gradient: as in _check_backward
            assert abs(diff.item() - grad.view(-1)[j].item()) <= 1e-4


def test_other_stream_and_captured_graph():
    xt, w, b, dy = _inputs(300, 1024, torch.bfloat16, torch.float32, 12)
    ref, mean, rstd = lib.qkv_cte_layer_norm(xt, w, b, stats=True)
    gref = lib.qkv_cte_layer_norm_backward(dy, xt, mean, rstd, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y, m2, r2 = lib.qkv_cte_layer_norm(xt, w, b, stats=True, stream=s)
    got = lib.qkv_cte_layer_norm_backward(dy, xt, m2, r2, w, stream=s)
    s.synchronize()
    assert torch.equal(y, ref) and all(torch.equal(a, b) for a, b in zip(got, gref))
    out = torch.zeros_like(xt)
    grads = [torch.zeros_like(xt), torch.zeros_like(w), torch.zeros_like(w)]
    ws = torch.empty(lib.qkv_cte_layer_norm_backward_workspace(300, 1024), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.qkv_cte_layer_norm(xt, w, b, out=out, mean=m2, rstd=r2)
        lib.qkv_cte_layer_norm_backward(dy, xt, m2, r2, w, *grads, workspace=ws)
    for _ in range(2):
        out.zero_()
        for t in grads:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and all(torch.equal(a, b) for a, b in zip(grads, gref))


def test_binding_refusals():
    x = torch.zeros(4, 64, device=DEV, dtype=torch.bfloat16)
    w = torch.ones(64, device=DEV)
    for bad in (dict(weight=w[:32]), dict(weight=w, bias=w.bfloat16()), dict(weight=w.half()), dict(weight=w.cpu()),
                dict(out=torch.zeros(4, 32, device=DEV, dtype=torch.bfloat16)), dict(out=torch.zeros(4, 64, device=DEV))):
        with pytest.raises((ValueError, TypeError)):
            lib.qkv_cte_layer_norm(x, **bad)
    with pytest.raises(ValueError, match="contiguous"):
        lib.qkv_cte_layer_norm(torch.zeros(64, 4, device=DEV).t())
    with pytest.raises(lib.QkvCteError):
        lib.qkv_cte_layer_norm(x, out=x[:1].expand(4, 64))


@pytest.mark.parametrize("rows,cols", [(5, 640), (7, 333), (5, 12288), (6, 30000), (4, 9001)])
@pytest.mark.parametrize("into", ["dy", "x"])
def test_backward_in_place_at_every_width(rows, cols, into):
    """dx over dy or over x: the column sums still see what was there."""
    xt, w, _, dy = _inputs(rows, cols, torch.bfloat16, torch.float32, cols)
    mean, rstd = _saved(xt)
    x2, dy2 = xt.clone(), dy.clone()
    dw, db = torch.empty_like(w), torch.empty_like(w)
    dx, _, _ = lib.qkv_cte_layer_norm_backward(dy2, x2, mean, rstd, w, dx=dy2 if into == "dy" else x2, dweight=dw,
                                               dbias=db)
    _check_backward(dy, xt, mean, rstd, w, dx, dw, db)
    assert torch.equal(x2 if into == "dy" else dy2, xt if into == "dy" else dy)


@pytest.mark.parametrize("cols", [7, 77, 333, 1283, 5121])
def test_forward_in_place_off_16_byte_boundaries(cols):
    """Many rows whose 16-byte pieces they share with their neighbours."""
    xt, w, b, _ = _inputs(3000, cols, torch.bfloat16, torch.float32, cols)
    y, _, _ = lib.qkv_cte_layer_norm(xt, w, b)
    _check_forward(xt, w, b, 1e-6, y, None, None)
    z = xt.clone()
    lib.qkv_cte_layer_norm(z, w, b, out=z)
    assert torch.equal(z, y)
