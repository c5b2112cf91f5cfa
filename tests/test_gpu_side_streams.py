"""Calls on another stream than the current one, without a synchronisation in between:
the current stream is busy (a spinning kernel of some milliseconds) with work that ends
in memory the allocator has already taken back."""
import pytest
import torch

import rope_tcgen05_mxfp8_gb300 as lib
import workloads as wl
from rope_tcgen05_mxfp8_gb300 import qkv_cte as q
from gpu_harness import assert_same_to_rounding
from test_gpu_linear import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"
SPIN = 100_000_000  # clock cycles: 50 ms or more
TINY = wl.workload("tiny")[0]  # the projection's


def _same(a, b):
    """Equal bits; the projection's Q and K, whose sums of squares are added in a
    run-dependent order, to rounding."""
    if a.shape == (TINY.tokens, TINY.n_q_heads * TINY.d_head * 3):
        assert_same_to_rounding(TINY, a, b)
        return True
    return torch.equal(a, b)


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


def _projection():
    call = TINY
    t = {k: v.to(DEV) if v is not None else None for k, v in wl.make_inputs(call).items()}
    op = lib.QkvCte(call.tokens, call.hidden, call.n_q_heads, call.n_kv_heads, call.d_head)
    return lambda **kw: (op(t["A"], t["a_scale"], t["W"], t["w_sf"], t["bias"], t["gamma_q"], t["gamma_k"], t["cos"],
                            t["sin"], **kw),)


def _producer():
    x = torch.randn(300, 1024, device=DEV).bfloat16()
    packed = torch.randint(0, 100, (300, 1028), device=DEV, dtype=torch.uint8)
    return lambda **kw: (*lib.qkv_cte_row_quantize(x, **kw)[:2], *lib.qkv_cte_unpack_rows(packed, **kw))


def _permute():
    x = torch.randn(4 * 64, 96, device=DEV)
    return lambda **kw: (lib.qkv_cte_interleaved_to_rotate_half(x, 2, 1, 64, **kw),)


BLOCK_OPS = [_norm, _norm_backward, _rope, _linear]
PROJECTION = [_projection, _producer, _permute]


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
    assert all(_same(g, w) for g, w in zip([g.clone() for g in got], want))
    torch.cuda.synchronize()
    assert all(_same(g, w) for g, w in zip(got, want))


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


def _dirty(n):
    """Leave n bytes of ones with the allocator."""
    t = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    del t


def _run_linear(T):
    c = Case(T, 640, 512, "silu", "bf16")
    size = c.op(input_layout=lib.QKV_CTE_INPUT_BF16).workspace.numel()
    make = lambda: c.op(input_layout=lib.QKV_CTE_INPUT_BF16)  # noqa: E731
    return make, lambda op, s: c.run(op, A=c.x, stream=s), size, c.run(make(), A=c.x)


def _run_projection(_):
    call = TINY
    t = {k: v.to(DEV) if v is not None else None for k, v in wl.make_inputs(call).items()}
    make = lambda: lib.QkvCte(call.tokens, call.hidden, call.n_q_heads, call.n_kv_heads, call.d_head)  # noqa: E731
    run = lambda op, s: op(t["A"], t["a_scale"], t["W"], t["w_sf"], t["bias"], t["gamma_q"], t["gamma_k"],  # noqa: E731
                           t["cos"], t["sin"], stream=s)
    return make, run, make().workspace.numel(), run(make(), None)


def _workspace_is_ready(make, run, size, want):
    """An object made while the constructor's stream is busy, used at once on another
    stream: its workspace already holds what the first run needs."""
    _dirty(size)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(SPIN // 4)
    op = make()
    with torch.cuda.stream(s):
        left = op.workspace.count_nonzero()
    got = run(op, s)
    s.synchronize()
    assert left.item() == 0
    assert op.status(s) == 0
    assert _same(got, want)
    torch.cuda.synchronize()
    assert _same(run(op, None), want) and op.status() == 0


def _workspace_outlives_its_object(make, run, size, want, current):
    """An object dropped while its call is pending: no later tensor gets the workspace
    before the call has run."""
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    op = make()
    with torch.cuda.stream(s):
        torch.cuda._sleep(SPIN)
        got = run(op, None) if current else None
    if not current:
        got = run(op, s)
    del op
    late = [torch.full((size,), 255, dtype=torch.uint8, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    assert _same(got, want)
    assert all(bool((t == 255).all()) for t in late)


@pytest.mark.parametrize("T", [3, 40, 700])
def test_linear_workspace_is_ready_for_any_stream(T):
    _workspace_is_ready(*_run_linear(T))


@pytest.mark.parametrize("current", [False, True])
@pytest.mark.parametrize("T", [3, 40, 700])
def test_linear_workspace_outlives_its_object(T, current):
    _workspace_outlives_its_object(*_run_linear(T), current)


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("make", PROJECTION)
def test_projection_results_on_another_stream(make, as_handle):
    _results_survive(make, as_handle)


def test_projection_workspace_is_ready_for_any_stream():
    _workspace_is_ready(*_run_projection(0))


@pytest.mark.parametrize("current", [False, True])
def test_projection_workspace_outlives_its_object(current):
    _workspace_outlives_its_object(*_run_projection(0), current)


@pytest.mark.parametrize("T", [3, 700])
def test_object_made_within_a_capture(T):
    """The workspace's fill is then part of the graph, before the run that needs it."""
    make, run, size, want = _run_linear(T)
    _dirty(size)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op = make()
        got = run(op, None)
    for _ in range(2):
        op.workspace.fill_(255)
        got.zero_()
        graph.replay()
        assert op.status() == 0 and torch.equal(got, want)


@pytest.mark.parametrize("stream", [0, "default"])
@pytest.mark.parametrize("make", BLOCK_OPS + PROJECTION)
def test_results_on_the_default_stream_from_another(make, stream):
    """The default stream, by its handle 0 or as an object, while another one is current."""
    with torch.cuda.stream(torch.cuda.Stream()):
        f = make()
        want = [t.clone() for t in f()]
        torch.cuda.synchronize()
        torch.cuda._sleep(SPIN)
        late = [torch.full((n,), 7, dtype=torch.uint8, device=DEV)
                for t in want for n in [t.numel() * t.element_size()] * 3]
        late += [torch.full((1 << 19,), 7, dtype=torch.uint8, device=DEV) for _ in range(8)]
        del late
        got = f(stream=torch.cuda.default_stream() if stream else 0)
        torch.cuda.synchronize()
        assert all(_same(g, w) for g, w in zip(got, want))
        # as memory of that stream, not of some other that a handle of 0 might name
        assert q._side(torch.cuda.default_stream() if stream else 0, got[0].device).cuda_stream == 0


@pytest.mark.parametrize("case", [lambda: _run_linear(3), lambda: _run_linear(700), lambda: _run_projection(0)])
def test_workspace_of_another_stream_outlives_a_call_on_the_default_one(case):
    make, run, size, want = case()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        op = make()
    torch.cuda._sleep(SPIN)
    got = run(op, None)
    del op
    with torch.cuda.stream(s):
        late = [torch.full((size,), 255, dtype=torch.uint8, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    assert _same(got, want)
    assert all(bool((t == 255).all()) for t in late)
