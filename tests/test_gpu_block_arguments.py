"""Calls of the block operators that must be refused, or that an earlier failed call must
not make fail."""
import subprocess
import sys

import pytest
import torch

import rope_tcgen05_mxfp8_gb300 as lib
from test_gpu_linear import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_transposed_positions_and_grids_are_refused():
    rope = lib.QkvCteRopeAxes(24, (8, 8, 8))
    x = torch.randn(2, 10, 4, 24, device=DEV)
    pos = torch.randint(0, 50, (10, 3), device=DEV, dtype=torch.int32)
    both = torch.stack([pos, pos + 1])
    want = rope(x, positions=pos)
    assert torch.equal(rope(x, positions=pos.reshape(-1)), want)             # flat
    assert not torch.equal(rope(x, positions=both), want)
    grid = torch.tensor([[2, 5, 1], [3, 2, 1]], dtype=torch.int32, device=DEV)
    assert torch.equal(rope(x, grids=grid.reshape(-1)), rope(x, grids=grid))
    for bad in (dict(positions=pos.t().contiguous()), dict(positions=both.transpose(0, 1).contiguous()),
                dict(positions=both.transpose(1, 2).contiguous()), dict(positions=pos.reshape(1, 30)),
                dict(grids=grid.t().contiguous())):
        with pytest.raises(ValueError):
            rope(x, **bad)
        with pytest.raises(ValueError):
            rope.tables(2, 10, **bad)
    n = (20, 24)
    for bad in (torch.empty(24, 20, device=DEV), torch.empty(10, 48, device=DEV)):
        with pytest.raises(ValueError):
            rope.tables(2, 10, positions=pos, cos=bad, sin=torch.empty(n, device=DEV))
        with pytest.raises(ValueError):
            rope.tables(2, 10, positions=pos, cos=torch.empty(n, device=DEV), sin=bad)


def test_transposed_operands_of_the_product_are_refused():
    c = Case(6, 64, 96)
    op = c.op()
    want = c.run(op)
    lead = op(c.A.view(2, 3, 64), c.s.view(2, 3), c.W.view(4, 24, 64), c.sf.view(4, 24, 2), bias=c.bias)
    assert torch.equal(lead, want)                                            # leading dimensions
    assert torch.equal(op(c.A.reshape(-1), c.s, c.W.reshape(-1), c.sf.reshape(-1), bias=c.bias), want)
    for kw in (dict(A=c.A.t().contiguous()), dict(W=c.W.t().contiguous()), dict(w_sf=c.sf.t().contiguous())):
        a = dict(dict(A=c.A, W=c.W, w_sf=c.sf), **kw)
        with pytest.raises(ValueError):
            op(a["A"], c.s, a["W"], a["w_sf"], bias=c.bias)
    packed = torch.cat([c.A, c.s.view(torch.uint8).view(6, 4)], dim=1).contiguous()
    pop = c.op(input_layout=lib.QKV_CTE_INPUT_PACKED)
    assert torch.equal(pop(packed, None, c.W, c.sf, bias=c.bias), want)
    with pytest.raises(ValueError):
        pop(packed.t().contiguous(), None, c.W, c.sf, bias=c.bias)


def test_reordered_statistics_are_refused():
    x = torch.randn(2, 3, 64, device=DEV)
    y, mean, rstd = lib.qkv_cte_layer_norm(x, stats=True)
    want = lib.qkv_cte_layer_norm_backward(y, x, mean, rstd)
    for m, r in ((mean.reshape(-1), rstd.reshape(-1)), (mean[..., None], rstd[..., None])):
        assert all(torch.equal(a, b) for a, b in zip(lib.qkv_cte_layer_norm_backward(y, x, m, r), want))
    flat = lib.qkv_cte_layer_norm_backward(y.view(6, 64), x.view(6, 64), mean, rstd)
    assert torch.equal(flat[0].view(2, 3, 64), want[0])
    bad = torch.empty(3, 2, device=DEV)
    with pytest.raises(ValueError):
        lib.qkv_cte_layer_norm(x, mean=bad, rstd=rstd)
    with pytest.raises(ValueError):
        lib.qkv_cte_layer_norm(x, mean=mean, rstd=bad)
    with pytest.raises(ValueError):
        lib.qkv_cte_layer_norm_backward(y, x, bad, rstd)
    with pytest.raises(ValueError):
        lib.qkv_cte_layer_norm_backward(y, x, mean, bad)


def test_host_positions_and_devices_are_refused():
    rope = lib.QkvCteRopeAxes(24, (8, 8, 8))
    pos = torch.zeros(10, 3, dtype=torch.int32)
    for stream in (None, torch.cuda.Stream()):
        with pytest.raises(ValueError, match="CUDA"):
            rope.tables(1, 10, positions=pos, stream=stream)
        with pytest.raises(ValueError, match="CUDA"):
            rope.tables(1, 10, grids=pos[:1], stream=stream)
    with pytest.raises(ValueError, match="CUDA"):
        lib.QkvCteLinear(4, 64, 32, device="cpu")


def test_more_columns_than_32_bits_are_refused():
    """2^32 + 64 columns are not 64."""
    x = torch.zeros(1, 2 ** 32 + 64, device=DEV, dtype=torch.bfloat16)
    with pytest.raises((ValueError, lib.QkvCteError)):
        lib.qkv_cte_layer_norm(x, out=x)
    with pytest.raises((ValueError, lib.QkvCteError)):
        lib.qkv_cte_layer_norm_backward(x, x, torch.zeros(1, device=DEV), torch.ones(1, device=DEV), dx=x)


def test_in_place_results_count_as_changes():
    """autograd sees that a tensor it saved was overwritten."""
    rope = lib.QkvCteRopeAxes(64, (64,))
    pos = torch.arange(6, device=DEV, dtype=torch.int32)[:, None]
    c = Case(6, 64, 64, residual=True, out="fp32")
    op = c.op()

    def norm(t):
        lib.qkv_cte_layer_norm(t, out=t)

    def norm_backward(t):
        lib.qkv_cte_layer_norm_backward(t, t, torch.zeros(6, device=DEV), torch.ones(6, device=DEV), dx=t)

    def turn(t):
        rope(t.view(6, 1, 64), positions=pos, out=t.view(6, 1, 64))

    def product(t):
        c.run(op, residual=t, out=t)

    for write in (norm, norm_backward, turn, product):
        leaf = torch.randn(6, 64, device=DEV, requires_grad=True)
        z = leaf * 1.0
        loss = (z * z).sum()                       # saves z
        with torch.no_grad():
            write(z.detach())
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    with torch.inference_mode():                   # tensors without a version counter
        t = torch.randn(6, 64, device=DEV)
        for write in (norm, norm_backward, turn, product):
            write(t)


STALE = r"""
import os
import sys

import torch
import rope_tcgen05_mxfp8_gb300 as lib
rope = lib.QkvCteRopeAxes(64, (64,))
x = torch.randn(6, 2, 64, device="cuda")
pos = torch.arange(6, device="cuda", dtype=torch.int32)[:, None]
want = rope(x, positions=pos)
op = lib.QkvCteLinear(2, 64, 32)
A = torch.zeros(2, 64, dtype=torch.uint8, device="cuda")
s = torch.ones(2, device="cuda")
W = torch.zeros(32, 64, dtype=torch.uint8, device="cuda")
sf = torch.full((32, 2), 127, dtype=torch.uint8, device="cuda")
out = op(A, s, W, sf)
y = torch.empty_like(x)
torch.cuda.synchronize()
side = torch.cuda.Stream()
graph = torch.cuda.CUDAGraph()
with torch.cuda.stream(side):
    graph.capture_begin()
    try:
        side.synchronize()                    # not allowed here: the capture is lost
    except Exception as e:
        print("lost:", type(e).__name__)
    try:
        op(A, s, W, sf, out=out)
        raise SystemExit("the call into a lost capture went through")
    except lib.QkvCteError as e:
        print("refused:", e)
    try:
        graph.capture_end()
    except Exception as e:
        print("ended:", type(e).__name__)
rope(x, positions=pos, out=y)                 # a call of its own: nothing is wrong with it
torch.cuda.synchronize()
assert torch.equal(y, want)
print("fine")
sys.stdout.flush()
os._exit(0)                                   # without tearing the graph down
"""


def test_a_failed_launch_is_not_reported_again():
    """A launch that CUDA refuses is reported by its own call only. (In a process of its
    own: it ends a graph capture half way.)"""
    r = subprocess.run([sys.executable, "-c", STALE], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "refused" in r.stdout and "fine" in r.stdout, r.stdout + r.stderr
