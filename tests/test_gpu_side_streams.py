"""Calls on another stream than the current one, without a synchronisation in between:
the current stream is busy (a spinning kernel of some milliseconds) with work that ends
in memory the allocator has already taken back."""
import pytest
import torch

import rope_tcgen05_mxfp8_gb300 as lib
from test_gpu_linear import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"
SPIN = 100_000_000  # clock cycles: 50 ms or more


def _norm():
    x = torch.randn(300, 1024, device=DEV).bfloat16()
    w = torch.rand(1024, device=DEV)
    return lambda **kw: lib.qkv_cte_layer_norm(x, w, w, stats=True, **kw)


def _norm_backward():
    x, dy = (torch.randn(300, 1024, device=DEV).bfloat16() for _ in range(2))
    w = torch.rand(1024, device=DEV)
    _, mean, rstd = lib.qkv_cte_layer_norm(x, w, stats=True)
    return lambda **kw: lib.qkv_cte_layer_norm_backward(dy, x, mean, rstd, w, **kw)


def _rope():
    rope = lib.QkvCteRopeAxes(128, (44, 42, 42))
    x = torch.randn(500, 8, 128, device=DEV).bfloat16()
    grid = torch.tensor([[5, 10, 10]], dtype=torch.int32, device=DEV)
    return lambda **kw: (rope(x, grids=grid, **kw), *rope.tables(1, 500, grids=grid, **kw))


def _linear():
    c = Case(40, 640, 512, "gelu_tanh", "bf16", gate=True, residual=True)
    op = c.op(input_layout=lib.QKV_CTE_INPUT_BF16)
    return lambda **kw: (c.run(op, A=c.x, **kw),)


BLOCK_OPS = [_norm, _norm_backward, _rope, _linear]


def _results_survive(make, as_handle):
    """The results do not lie in memory that the current stream has yet to write."""
    f = make()
    want = [t.clone() for t in f()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(SPIN)
    # what the allocator would hand out for the results: written after the spin, already freed
    late = [torch.full((n,), 7, dtype=torch.uint8, device=DEV)
            for t in want for n in [t.numel() * t.element_size()] * 3]
    late += [torch.full((1 << 19,), 7, dtype=torch.uint8, device=DEV) for _ in range(8)]
    del late
    got = f(stream=s.cuda_stream if as_handle else s)
    s.synchronize()
    assert all(torch.equal(g, w) for g, w in zip([g.clone() for g in got], want))
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("make", BLOCK_OPS)
def test_results_on_another_stream(make, as_handle):
    _results_survive(make, as_handle)


@pytest.mark.parametrize("make", BLOCK_OPS)
def test_results_used_on_the_current_stream_are_kept_for_it(make):
    """A result of another stream's call, dropped while the current stream still reads it:
    its memory goes to no later call on that other stream before the reading is done."""
    f = make()
    want = [t.clone() for t in f()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = f(stream=s)
    s.synchronize()
    torch.cuda._sleep(SPIN)
    copies = [g.clone() for g in got]
    del got
    with torch.cuda.stream(s):
        late = [torch.full((t.numel() * t.element_size(),), 7, dtype=torch.uint8, device=DEV) for t in want * 3]
    torch.cuda.synchronize()
    assert all(torch.equal(c, w) for c, w in zip(copies, want)) and late
