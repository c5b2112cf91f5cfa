"""The product with bias, activation, gate and residual against a plain implementation in
64 bits, on the codes and scales themselves.

Tolerances. u = 2^-24, h = eps(type)/2. The products of two e4m3 codes are exact; the
tensor core adds 32 of them to an fp32 accumulator per step, and a step is taken to lose
at most 2^-22 of the magnitudes added so far: (K/32 + 4) 2^-22 sum |a w|, which also
covers joining partial sums. Scale and bias: 4 u of their magnitudes. An activation's
slope is at most 1.13 and its own error 2^-20 |z| (linear_epilogue.cuh)."""
import math

import pytest
import torch

import rope_tcgen05_mxfp8_gb300 as lib

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = {"none": lib.QKV_CTE_ACT_NONE, "gelu_tanh": lib.QKV_CTE_ACT_GELU_TANH, "gelu_erf": lib.QKV_CTE_ACT_GELU_ERF,
        "silu": lib.QKV_CTE_ACT_SILU}


def _codes(shape, gen):
    """Finite e4m3 codes of every magnitude."""
    c = torch.randint(0, 256, shape, generator=gen, device=DEV, dtype=torch.int32)
    c = torch.where((c & 0x7F) == 0x7F, c - 1, c)
    return c.to(torch.uint8)


class Case:
    def __init__(self, T, K, N, act="none", out="bf16", gate=False, residual=False, col=False, bias=True, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed + 7 * T + K + 3 * N)
        self.T, self.K, self.N, self.act, self.dt = T, K, N, act, TYPES[out]
        # normal activations quantised per row, so that the sums look like a projection's
        x = torch.randn(T, K, generator=g, device=DEV).bfloat16()
        self.x = x
        amax = x.float().abs().amax(1)
        self.s = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
        self.A = (x.float() / self.s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        self.W = _codes((N, K), g)
        self.sf = torch.randint(108, 118, (N, K // 32), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
        self.bias = torch.randn(N, generator=g, device=DEV).bfloat16() if bias else None
        self.gate = torch.randn(N, generator=g, device=DEV).bfloat16() if gate else None
        self.col = 0.5 + torch.rand(N, generator=g, device=DEV) if col else None
        self.res = torch.randn(T, N, generator=g, device=DEV).to(self.dt) if residual else None

    def op(self, **kw):
        return lib.QkvCteLinear(self.T, self.K, self.N, act=ACTS[self.act], out_dtype=self.dt, **kw)

    def run(self, op=None, A=None, s=None, **kw):
        op = op or self.op()
        kw = dict(dict(bias=self.bias, gate=self.gate, residual=self.res, w_col_scale=self.col), **kw)
        return op(self.A if A is None else A, self.s if A is None else s, self.W, self.sf, **kw)

    def reference(self, res="own"):
        """(value, tolerance) in 64 bits."""
        res = self.res if isinstance(res, str) else res
        a = self.A.view(torch.float8_e4m3fn).double()
        w = self.W.view(torch.float8_e4m3fn).double() * torch.exp2(
            self.sf.double() - 127).repeat_interleave(32, dim=1)
        scale = self.s.double()[:, None] * (self.col.double() if self.col is not None else 1.0)
        b = self.bias.double() if self.bias is not None else torch.zeros(self.N, device=DEV).double()
        z = (a @ w.t()) * scale + b
        ez = (self.K / 32 + 4) * 2.0 ** -22 * (a.abs() @ w.abs().t()) * scale + 4 * U * (z.abs() + b.abs())
        v = {"none": lambda z: z, "silu": lambda z: z * torch.sigmoid(z),
             "gelu_tanh": lambda z: z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)),
             "gelu_erf": lambda z: 0.5 * z * torch.erfc(-z / math.sqrt(2))}[self.act](z)
        ev = 1.13 * ez + (0 if self.act == "none" else 2.0 ** -20 * z.abs())
        if self.gate is not None:
            v, ev = v * self.gate.double(), ev * self.gate.double().abs() + U * (v * self.gate.double()).abs()
        if res is not None:
            v, ev = v + res.double(), ev + U * (v.abs() + res.double().abs())
        h = torch.finfo(self.dt).eps / 2
        sub = torch.finfo(self.dt).tiny * torch.finfo(self.dt).eps / 2
        return v, h * v.abs() + sub + 1.01 * ev

    def check(self, out, res="own", rows=slice(None)):
        ref, tol = self.reference(res)
        err = (out.double() - ref).abs()[rows]
        bad = ~(err <= tol[rows])
        assert not bool(bad.any()), (f"{int(bad.sum())} of {bad.numel()} outside, worst excess "
                                     f"{(err - tol[rows]).max().item():.3e}, first at {bad.nonzero()[0].tolist()}")


SIZES = [(1, 32, 1), (1, 128, 16), (1, 512, 5120), (1, 5120, 240), (2, 64, 7), (3, 96, 333), (7, 160, 128), (8, 2048, 256),
         (15, 1024, 129), (16, 128, 512), (17, 256, 100), (33, 5120, 64), (64, 1056, 241), (65, 32, 300), (100, 224, 128),
         (127, 384, 128), (128, 640, 255), (129, 640, 480), (200, 128, 8), (255, 1024, 240), (256, 5120, 256),
         (257, 416, 1000), (300, 2560, 17), (513, 1056, 333), (777, 96, 2000), (1000, 1056, 333), (2100, 288, 720)]


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_sizes(T, K, N, out):
    c = Case(T, K, N, "gelu_tanh" if T % 2 else "none", out, gate=T % 3 == 0, residual=N % 2 == 0, col=K % 64 == 0)
    op = c.op()
    c.check(c.run(op))
    assert op.status() == 0


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "gelu_erf", "silu"])
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,N", [(5, 96), (300, 500)])
@pytest.mark.parametrize("parts", ["plain", "bias", "all"])
def test_epilogues(act, out, T, N, parts):
    c = Case(T, 256, N, act, out, gate=parts == "all", residual=parts == "all", col=parts == "all",
             bias=parts != "plain")
    c.check(c.run())


@pytest.mark.parametrize("T,K,N", [(1, 512, 640), (40, 1056, 333), (400, 640, 500)])
def test_bf16_and_packed_inputs_give_the_fp8_result(T, K, N):
    c = Case(T, K, N, "silu", "bf16", gate=True, residual=True)
    want = c.run()
    c.check(want)
    got = c.run(c.op(input_layout=lib.QKV_CTE_INPUT_BF16), A=c.x)
    assert torch.equal(got, want)
    packed = torch.cat([c.A, c.s.view(torch.uint8).view(T, 4)], dim=1).contiguous()
    assert torch.equal(c.run(c.op(input_layout=lib.QKV_CTE_INPUT_PACKED), A=packed), want)


@pytest.mark.parametrize("T", [3, 70, 300])
@pytest.mark.parametrize("N,pad,shift", [(256, 16, 0), (256, 3, 0), (250, 6, 1), (96, 0, 0), (33, 1, 5)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_strided_rows_and_in_place(T, N, pad, shift, out):
    c = Case(T, 160, N, "none", out, gate=True, residual=True)
    wide = torch.full((T, N + pad + shift), 3.0, dtype=c.dt, device=DEV)
    view = wide[:, shift: shift + N]
    y = c.run(out=view)
    assert y is view
    c.check(view)
    between = torch.ones_like(wide, dtype=torch.bool)
    between[:, shift: shift + N] = False
    assert bool((wide[between] == 3.0).all())
    res = torch.empty_like(wide)[:, shift: shift + N]
    res.copy_(c.res)
    assert torch.equal(c.run(residual=res), view)
    assert torch.equal(c.run(residual=res, out=res), view)                  # in place
    row = c.res[:1].expand(T, N)
    c.check(c.run(residual=row), res=row)                                   # one row for all


def test_padding_rows_and_empty():
    """Rows that hold zeros give act(bias); no tokens launch nothing."""
    c = Case(130, 256, 64, "gelu_erf", "fp32")
    c.A[100:] = 0
    c.s[100:] = 1.0
    c.check(c.run())
    e = Case(2, 64, 32)
    op = lib.QkvCteLinear(0, 64, 32)
    assert op(e.A[:0], e.s[:0], e.W, e.sf).shape == (0, 32)


def test_non_finite_stays_in_its_row_and_column():
    for T in (4, 300):
        c = Case(T, 256, 96, "none", "fp32", residual=True)
        c.s[1] = float("inf")
        c.bias[5] = float("nan")
        c.A[2, 3] = 0x7F                                                     # an e4m3 NaN
        out = c.run()
        ok = torch.ones(T, 96, dtype=torch.bool, device=DEV)
        ok[1:3] = False
        ok[:, 5] = False
        assert bool(out[2].isnan().all()) and bool(out[:, 5].isnan().all()) and not bool(out[1].isfinite().any())
        ref, tol = c.reference()
        assert bool(((out.double() - ref).abs() <= tol)[ok].all())


def test_repeat_runs_are_identical_and_share_a_workspace_in_turn():
    for T in (2, 50, 1300):
        c, d = Case(T, 1056, 500, "gelu_tanh", seed=1), Case(T, 1056, 500, "gelu_tanh", seed=2)
        op = c.op()
        a = c.run(op)
        b = d.run(op)
        assert torch.equal(c.run(op), a) and torch.equal(d.run(op), b)
        c.check(a)
        d.check(b)


@pytest.mark.parametrize("T", [1, 60, 700])
def test_other_stream_and_captured_graph(T):
    c = Case(T, 640, 512, "gelu_tanh", "bf16", gate=True, residual=True)
    op = c.op(input_layout=lib.QKV_CTE_INPUT_BF16)
    want = c.run(op, A=c.x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = c.run(op, A=c.x, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(op, A=c.x, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert op.status() == 0


@pytest.mark.parametrize("T", [3, 300])
def test_bounded_waits_report_and_the_next_run_is_right(T):
    c = Case(T, 256, 128)
    op = c.op(flags=lib.QKV_CTE_FLAG_TEST_STALL)
    c.run(op)
    with pytest.raises(lib.QkvCteError) as ei:
        op.status()
    assert ei.value.code == lib.QKV_CTE_ERR_DEVICE_TIMEOUT
    assert op.status() == 0
    c.check(c.run())


def test_binding_refusals():
    c = Case(4, 64, 32, residual=True)
    op = c.op()
    for kw in (dict(bias=c.bias[:16]), dict(bias=c.bias.float()), dict(gate=c.bias.cpu()), dict(residual=c.res[:2]),
               dict(residual=c.res.float()), dict(out=torch.zeros(4, 31, dtype=c.dt, device=DEV)),
               dict(w_col_scale=c.bias)):
        with pytest.raises((ValueError, TypeError)):
            c.run(op, **kw)
    with pytest.raises((ValueError, TypeError)):
        op(c.x, c.s, c.W, c.sf)
    with pytest.raises(lib.QkvCteError):
        op(c.A, None, c.W, c.sf)
    with pytest.raises(lib.QkvCteError):
        c.run(op, out=c.res[:1].expand(4, 32))


def test_large_offsets():
    """Row offsets past 2^32 bytes: the last rows of a 5 GB output."""
    T, K, N = 160000, 64, 16384
    c = Case(64, K, N, "none", "bf16")
    op = lib.QkvCteLinear(T, K, N)
    A = c.A.repeat(T // 64, 1)
    s = c.s.repeat(T // 64)
    out = op(A, s, c.W, c.sf, bias=c.bias)
    ref, tol = c.reference()
    for t0 in (0, T // 2 // 64 * 64, T - 64):
        assert bool(((out[t0: t0 + 64].double() - ref).abs() <= tol).all())


# K1's form of the product (more than 512 tokens, rows on 32-byte boundaries), one size for
# each of its tile widths
WIDE = [(700, 64, 720), (2560, 96, 1008), (4096, 64, 960)]


@pytest.mark.parametrize("T,K,N", WIDE)
@pytest.mark.parametrize("act", ["none", "gelu_tanh", "gelu_erf", "silu"])
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("parts", ["plain", "bias", "residual", "all"])
def test_wide_rows_epilogues(T, K, N, act, out, parts):
    c = Case(T, K, N, act, out, gate=parts == "all", residual=parts in ("residual", "all"), col=parts == "all",
             bias=parts != "plain")
    op = c.op()
    c.check(c.run(op))
    assert op.status() == 0


@pytest.mark.parametrize("T", [513, 768, 769, 897, 1025])
@pytest.mark.parametrize("K", [32, 288, 416])
@pytest.mark.parametrize("N", [16, 128, 240, 256, 496])
def test_wide_rows_tile_edges(T, K, N):
    c = Case(T, K, N, "none", "bf16", gate=True, residual=True)
    c.check(c.run())


@pytest.mark.parametrize("N", [1, 15, 17, 250, 255, 333])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_ragged_columns_in_padded_rows(N, out):
    """Rows on 32-byte boundaries whose last 16 columns are not whole."""
    c = Case(600, 160, N, "silu", out, gate=True, residual=True, col=True)
    wide = torch.full((600, 352), 3.0, dtype=c.dt, device=DEV)
    res = torch.empty_like(wide)[:, :N]
    res.copy_(c.res)
    y = c.run(out=wide[:, :N], residual=res)
    c.check(y)
    assert bool((wide[:, N:] == 3.0).all())
    assert torch.equal(c.run(out=res, residual=res), y)


def test_wide_rows_strided_in_place_and_broadcast_residual():
    c = Case(900, 160, 512, "gelu_tanh", "bf16", gate=True, residual=True)
    want = c.run()
    c.check(want)
    wide = torch.full((900, 640), 3.0, dtype=c.dt, device=DEV)
    y = c.run(out=wide[:, 64: 576])
    assert torch.equal(y, want) and bool((wide[:, :64] == 3.0).all()) and bool((wide[:, 576:] == 3.0).all())
    z = c.res.clone()
    assert torch.equal(c.run(out=z, residual=z), want)
    row = c.res[:1].expand(900, 512)
    c.check(c.run(residual=row), res=row)


def test_wide_rows_bounded_waits_report():
    c = Case(700, 256, 128)
    op = c.op(flags=lib.QKV_CTE_FLAG_TEST_STALL)
    c.run(op)
    with pytest.raises(lib.QkvCteError) as ei:
        op.status()
    assert ei.value.code == lib.QKV_CTE_ERR_DEVICE_TIMEOUT
    c.check(c.run())


@pytest.mark.parametrize("T,K,N", [(700, 4128, 97), (2048, 64, 1281), (5000, 160, 333), (3000, 32, 1)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_many_tokens_off_32_byte_rows(T, K, N, out):
    c = Case(T, K, N, "gelu_tanh", out, gate=True, residual=True)
    c.check(c.run())


def test_identity_weights_give_the_codes_back():
    """W = 1 on the diagonal and scales of 2^0: every output is one code times its row scale."""
    for T in (9, 600):
        K = 256
        c = Case(T, K, K, "none", "fp32", bias=False)
        c.W = torch.zeros(K, K, dtype=torch.uint8, device=DEV)
        c.W[torch.arange(K), torch.arange(K)] = 0x38  # 1.0
        c.sf.fill_(127)
        want = c.A.view(torch.float8_e4m3fn).float() * c.s[:, None]
        assert torch.equal(c.run(), want)
