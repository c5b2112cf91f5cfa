"""The block operators in a run together, as a transformer block uses them around the
projection: norm -> quantise -> fused QKV with the tables of a video grid -> output
product with gate and residual (in place) -> norm -> product with GELU -> product with
gate and residual; and the way back through the rotation and the norm. Every step is
checked against 64 bits on its own actual inputs, with the tolerances of its own tests."""
import math

import pytest
import torch

import rope_tcgen05_mxfp8_gb300 as lib
import workloads as wl
from gpu_harness import check_outputs
from test_gpu_layer_norm import _check_forward
from test_gpu_linear import Case
from test_gpu_rope_axes import _angles, _rotate

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
GRID = (5, 8, 8)
T, H, HEADS, D, F = 5 * 8 * 8, 512, 4, 128, 1100  # F: an odd feed-forward width


class Block:
    """Weights, plans and buffers of one block."""

    def __init__(self):
        g = torch.Generator(device=DEV).manual_seed(0)
        self.call = wl.custom_call(tokens=T, hidden=H, n_q_heads=HEADS, n_kv_heads=HEADS, d_head=D, norm=0, rope=1,
                                   rope_grid=GRID, seed=7)
        self.inp = wl.make_inputs(self.call)
        self.w = {k: v.to(DEV) for k, v in self.inp.items() if v is not None}
        self.x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
        self.scale1, self.shift1, self.scale2, self.shift2 = (
            0.2 * torch.randn(H, generator=g, device=DEV) for _ in range(4))
        self.gate1, self.gate2 = (torch.randn(H, generator=g, device=DEV).bfloat16() for _ in range(2))
        # the in_features of the last product: F padded to whole blocks of 32 with zero weights
        self.Fp = (F + 31) // 32 * 32
        self.out = Case(T, H, H, seed=1)
        self.up = Case(T, H, self.Fp, "gelu_tanh", seed=2)
        self.up.W[F:] = 0
        self.up.bias[F:] = 0
        self.down = Case(T, self.Fp, H, seed=3)
        self.rope = lib.QkvCteRopeAxes(D, (44, 42, 42))
        self.grid = torch.tensor([GRID], dtype=torch.int32, device=DEV)
        self.qkv = lib.QkvCte(T, H, HEADS, HEADS, D, norm=0, rope=1)
        bf16 = lib.QKV_CTE_INPUT_BF16
        self.op_out = lib.QkvCteLinear(T, H, H, input_layout=bf16)
        self.op_up = lib.QkvCteLinear(T, H, self.Fp, act=lib.QKV_CTE_ACT_GELU_TANH, input_layout=bf16)
        self.op_down = lib.QkvCteLinear(T, self.Fp, H, input_layout=bf16)

    def forward(self, x):
        """All of it on the current stream; every intermediate is returned."""
        r = {}
        r["n1"], _, _ = lib.qkv_cte_layer_norm(x, 1 + self.scale1, self.shift1)
        r["codes"], r["row_scale"], _ = lib.qkv_cte_row_quantize(r["n1"])
        r["cos"], r["sin"] = self.rope.tables(1, T, grids=self.grid)
        r["qkv"] = self.qkv(r["codes"], r["row_scale"], self.w["W"], self.w["w_sf"], self.w["bias"], None, None,
                            r["cos"], r["sin"])
        # no attention here: the rotated queries stand for its output
        r["attn"] = r["qkv"][:, : H].contiguous()
        r["x1"] = x.clone()
        self.op_out(r["attn"], None, self.out.W, self.out.sf, bias=self.out.bias, gate=self.gate1, residual=r["x1"],
                    out=r["x1"])
        r["n2"], _, _ = lib.qkv_cte_layer_norm(r["x1"], 1 + self.scale2, self.shift2)
        r["h"] = self.op_up(r["n2"], None, self.up.W, self.up.sf, bias=self.up.bias)
        r["y"] = self.op_down(r["h"], None, self.down.W, self.down.sf, bias=self.down.bias, gate=self.gate2,
                              residual=r["x1"])
        return r


def _product(case, a_bf16, out, gate=None, residual=None):
    codes, scale = wl.row_quantise(a_bf16.cpu())
    case.A, case.s, case.gate, case.res = codes.to(DEV), scale.to(DEV), gate, residual
    case.check(out)


def test_block_forward_step_by_step():
    b = Block()
    r = b.forward(b.x)
    _check_forward(b.x, 1 + b.scale1, b.shift1, 1e-6, r["n1"], None, None)
    codes, scale = wl.row_quantise(r["n1"].cpu())
    assert torch.equal(r["codes"].cpu(), codes) and torch.equal(r["row_scale"].cpu(), scale)
    inp = dict(b.inp, A=codes, a_scale=scale, cos=r["cos"].cpu(), sin=r["sin"].cpu())
    check_outputs(b.call, inp, r["qkv"], None, None, name="block")
    assert (r["cos"].cpu() - b.inp["cos"]).abs().max().item() <= 8 * U  # the workload's own tables
    _product(b.out, r["attn"], r["x1"], b.gate1, b.x)
    _check_forward(r["x1"], 1 + b.scale2, b.shift2, 1e-6, r["n2"], None, None)
    _product(b.up, r["n2"], r["h"])
    assert bool((r["h"][:, F:] == 0).all())                             # GELU(0) in the padding
    _product(b.down, r["h"], r["y"], b.gate2, r["x1"])
    for op in (b.op_out, b.op_up, b.op_down, b.qkv):
        assert op.status() == 0


def test_block_captured_and_on_another_stream():
    b = Block()
    want = b.forward(b.x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = b.forward(b.x)
    s.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    x = torch.zeros_like(b.x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.forward(x)
    x.copy_(b.x)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)


def test_two_blocks_on_two_streams():
    a, b = Block(), Block()
    want = a.forward(a.x)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            ga = a.forward(a.x)
        with torch.cuda.stream(t):
            gb = b.forward(b.x)
        s.synchronize()
        t.synchronize()
        assert all(torch.equal(ga[k], want[k]) and torch.equal(gb[k], want[k]) for k in want)


def test_gradient_through_rotation_and_norm():
    """x -> norm -> heads -> rotation, and back: against autograd in 64 bits."""
    g = torch.Generator(device=DEV).manual_seed(5)
    n, d, dims = 6, 96, (32, 32, 32)
    x = torch.randn(40, n * d, generator=g, device=DEV)
    w = 1 + 0.2 * torch.randn(n * d, generator=g, device=DEV)
    bias = 0.2 * torch.randn(n * d, generator=g, device=DEV)
    dq = torch.randn(40, n, d, generator=g, device=DEV)
    pos = torch.randint(0, 1000, (40, 3), generator=g, device=DEV, dtype=torch.int32)
    rope = lib.QkvCteRopeAxes(d, dims, pairing=lib.QKV_CTE_ROPE_INTERLEAVED)
    y, mean, rstd = lib.qkv_cte_layer_norm(x, w, bias, eps=1e-5, stats=True)
    q = rope(y.view(40, n, d), positions=pos)
    dy = rope(dq, positions=pos, inverse=True)
    dx, dw, db = lib.qkv_cte_layer_norm_backward(dy.view(40, n * d), x, mean, rstd, w)
    xr, wr, br = (t.double().requires_grad_() for t in (x, w, bias))
    mu = xr.mean(-1, keepdim=True)
    xh = (xr - mu) * (((xr - mu) ** 2).mean(-1, keepdim=True) + 1e-5) ** -0.5
    yr = xh * wr + br
    qr, _ = _rotate(yr.view(40, n, d), _angles(d, dims, 0, 10000.0, pos), 1)
    (qr * dq.double()).sum().backward()
    # dy is off by 9 u of its pair (test_gpu_rope_axes), the statistics and sums by 90 u;
    # dx is linear in dy with gain at most rstd max|w| (2 + max|xh|^2), dw and db add 40 rows
    big = float(xh.abs().max())
    e = (18 + 2 * 90) * U * float(dq.abs().max()) * 2 * float(w.abs().max())
    gain = float(rstd.max()) * (2 + big ** 2)
    assert (q.double() - qr).abs().max().item() <= 200 * U * float(yr.abs().max()) * 2
    assert (dx.double() - xr.grad).abs().max().item() <= e * gain
    assert (dw.double() - wr.grad).abs().max().item() <= 40 * e * big
    assert (db.double() - br.grad).abs().max().item() <= 40 * e
    assert math.isfinite(float(dx.abs().max()))
