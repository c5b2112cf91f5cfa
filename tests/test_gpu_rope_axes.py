"""Rotary positions with several axes against a plain implementation in 64 bits.

Tolerances. u = 2^-24. A table value: the angle's remainder of at most pi/4 is rounded to
fp32 (u pi/4), sincospif is within 2 steps (4 u, of values up to 1), and a position p
makes the step's few 2^-53 (and the 64-bit reference's own product error) worth at most
p 2^-50: 6 u + p 2^-50. A rotated value adds two products and a sum, each rounded (fp32):
3 u (|lo| + |hi|), and the rounding to the output's type."""
import math

import pytest
import torch

import rope_tcgen05_mxfp8_gb300 as lib
import workloads as wl

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _angles(d, dims, spectrum, theta, pos):
    """pos [..., axes] -> angles [..., d/2] in 64 bits."""
    cols, pair = [], 0
    for a, dim in enumerate(dims):
        for j in range(dim // 2):
            e = 2 * j / dim if spectrum == 0 else 2 * pair / d
            cols.append(pos[..., a].double() * theta ** -e)
            pair += 1
    return torch.stack(cols, dim=-1)


def _grid_positions(grids, seq):
    """(positions [B, S, axes], live [B, S])."""
    pos, live = [], []
    for size in grids.tolist():
        n = min(seq, math.prod(max(v, 0) for v in size))
        s = torch.arange(seq)
        left, cols = s, []
        for v in reversed(size):
            cols.append(left % max(v, 1))
            left = left // max(v, 1)
        pos.append(torch.stack(cols[::-1], dim=1))
        live.append(s < n)
    return torch.stack(pos), torch.stack(live)


def _rotate(x, ang, pairing, inverse=False):
    """x [..., heads, d], ang [..., d/2]."""
    c, s = ang.cos()[..., None, :], ang.sin()[..., None, :]
    s = -s if inverse else s
    h = x.shape[-1] // 2
    x = x.double()
    lo, hi = (x[..., :h], x[..., h:]) if pairing == 0 else (x[..., 0::2], x[..., 1::2])
    a, b = lo * c - hi * s, hi * c + lo * s
    mag = lo.abs() + hi.abs()
    if pairing == 0:
        return torch.cat([a, b], -1), torch.cat([mag, mag], -1)
    return torch.stack([a, b], -1).flatten(-2), torch.stack([mag, mag], -1).flatten(-2)


def _check(y, ref, mag, far):
    h = torch.finfo(y.dtype).eps / 2
    sub = torch.finfo(y.dtype).tiny * torch.finfo(y.dtype).eps / 2
    tol = h * ref.abs() + sub + 1.01 * (9 * U + far * 2.0 ** -50) * mag
    err = (y.double() - ref).abs()
    assert bool((err <= tol).all()), f"worst excess {(err - tol).max().item():.3e}"


HEADS = [(128, (44, 42, 42)), (64, (64,)), (96, (32, 32, 32)), (2, (2,)), (6, (2, 4)), (10, (10,)), (84, (72, 4, 8)),
         (40, (10, 10, 10, 10)), (512, (128, 128, 256)), (24, (8, 8, 8))]


@pytest.mark.parametrize("d,dims", HEADS)
@pytest.mark.parametrize("pairing", [0, 1])
@pytest.mark.parametrize("spectrum", [0, 1])
@pytest.mark.parametrize("x", ["bf16", "fp16", "fp32"])
def test_apply_positions(d, dims, pairing, spectrum, x):
    rope = lib.QkvCteRopeAxes(d, dims, pairing=pairing, spectrum=spectrum)
    g = torch.Generator(device=DEV).manual_seed(d)
    xt = torch.randn(2, 19, 9, d, generator=g, device=DEV).to(TYPES[x])
    pos = torch.randint(-500, 500, (19, len(dims)), generator=g, device=DEV, dtype=torch.int32)
    for inverse in (False, True):
        y = rope(xt, positions=pos, inverse=inverse)
        ref, mag = _rotate(xt, _angles(d, dims, spectrum, 10000.0, pos), pairing, inverse)
        _check(y, ref, mag, 500)


@pytest.mark.parametrize("d,dims", HEADS)
@pytest.mark.parametrize("pairing", [0, 1])
def test_tables(d, dims, pairing):
    rope = lib.QkvCteRopeAxes(d, dims, pairing=pairing)
    g = torch.Generator().manual_seed(d + 1)
    for far in (0, 1000, 10 ** 6, 2 ** 31 - 200):
        pos = torch.randint(0, 100, (2, 33, len(dims)), generator=g) + far
        pos[0, 0] = -pos[0, 0]
        cos, sin = rope.tables(2, 33, positions=pos.to(torch.int32).to(DEV))
        ang = _angles(d, dims, 0, 10000.0, pos).reshape(66, d // 2)
        for got, ref in ((cos, ang.cos()), (sin, ang.sin())):
            ref = torch.cat([ref, ref], 1) if pairing == 0 else ref.repeat_interleave(2, 1)
            assert got.shape == (66, d)
            assert (got.cpu().double() - ref).abs().max().item() <= 6 * U + (far + 100) * 2.0 ** -50


def test_small_angles_keep_relative_accuracy():
    """The slowest pairs of near positions turn by 1e-4: their sine keeps fp32 digits."""
    rope = lib.QkvCteRopeAxes(128, (128,))
    pos = torch.arange(1, 65, dtype=torch.int32, device=DEV)[:, None]
    _, sin = rope.tables(1, 64, positions=pos)
    ref = _angles(128, (128,), 0, 10000.0, pos).sin()
    rel = ((sin[:, :64].double() - ref) / ref).abs()
    assert rel[ref < 0.5].max().item() <= 8 * U


def test_grid_tables_match_the_projection_workload():
    """The 480p grid gives the tables that the projection's workload supplies (fp32 there)."""
    call = wl.workload("short")[0]
    inp = wl.make_inputs(call)
    rope = lib.QkvCteRopeAxes(128, (44, 42, 42))
    grid = torch.tensor([list(call.rope_grid)], dtype=torch.int32, device=DEV)
    cos, sin = rope.tables(1, call.tokens, grids=grid)
    n = min(call.tokens, math.prod(call.rope_grid))
    # the workload rounds a 64-bit cosine to fp32 (u)
    assert (cos[:n].cpu() - inp["cos"][:n]).abs().max().item() <= 8 * U
    assert (sin[:n].cpu() - inp["sin"][:n]).abs().max().item() <= 8 * U


@pytest.mark.parametrize("pairing", [0, 1])
@pytest.mark.parametrize("grids", [[[3, 4, 5], [2, 3, 7]], [[60, 1, 1], [1, 1, 1]], [[0, 4, 5], [3, -1, 2]],
                                   [[100, 100, 100], [2147483647, 2147483647, 2147483647]]])
def test_grids_and_padding_rows(grids, pairing):
    rope = lib.QkvCteRopeAxes(24, (8, 8, 8), pairing=pairing)
    g = torch.tensor(grids, dtype=torch.int32)
    xt = torch.randn(2, 66, 3, 24, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    pos, live = _grid_positions(g, 66)
    xt[~live.to(DEV)] = float("inf")                     # padding may hold anything
    y = rope(xt, grids=g.to(DEV))
    ref, mag = _rotate(xt, _angles(24, (8, 8, 8), 0, 10000.0, pos).to(DEV), pairing)
    on = live.to(DEV)
    _check(y[on], ref[on], mag[on], 100)
    assert torch.equal(y[~on], xt[~on])
    z = xt.clone()
    rope(z, grids=g.to(DEV), out=z)
    assert torch.equal(z, y)
    cos, sin = rope.tables(2, 66, grids=g.to(DEV))
    off = ~on.reshape(-1)
    assert bool((cos[off] == 1).all()) and bool((sin[off] == 0).all())


def test_strided_layouts_and_side_by_side_columns():
    rope = lib.QkvCteRopeAxes(128, (44, 42, 42))
    gen = torch.Generator(device=DEV).manual_seed(2)
    pos = torch.randint(0, 50, (10, 3), generator=gen, device=DEV, dtype=torch.int32)
    ang = _angles(128, (44, 42, 42), 0, 10000.0, pos)
    wide = torch.randn(2, 10, 3 * 5 * 128, generator=gen, device=DEV).bfloat16()
    heads = wide.unflatten(2, (15, 128))
    q, k = heads[:, :, :5], heads[:, :, 5:10]
    v0 = heads[:, :, 10:].clone()
    ref, mag = _rotate(q, ang, 0)
    y = rope(q, positions=pos)
    _check(y, ref, mag, 50)
    q0 = q.clone()
    rope(q, positions=pos, out=k)                        # into the neighbouring columns
    assert torch.equal(k, y) and torch.equal(q, q0) and torch.equal(heads[:, :, 10:], v0)
    rope(q, positions=pos, out=q)
    assert torch.equal(q, y)
    bnsd = q0.transpose(1, 2).contiguous()               # [B, n, S, d]
    z = rope(bnsd.transpose(1, 2), positions=pos, out=torch.empty_like(bnsd).transpose(1, 2))
    assert torch.equal(z, y)
    odd = torch.zeros(2 * 10 * 5 * 128 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(2, 10, 5, 128)
    odd.copy_(q0)                                        # 2-byte aligned only
    assert torch.equal(rope(odd, positions=pos), y)
    one = q0[:, :1].expand(2, 10, 5, 128)                # one row for every position
    ref, mag = _rotate(one, ang, 0)
    _check(rope(one, positions=pos), ref, mag, 50)
    flat = rope(q0[0], positions=pos)
    assert torch.equal(flat, y[0])


def test_inverse_is_the_gradient():
    """<R x, z> = <x, R' z> for every x and z; R' R x = x."""
    rope = lib.QkvCteRopeAxes(96, (32, 32, 32), pairing=1, spectrum=1)
    gen = torch.Generator(device=DEV).manual_seed(3)
    pos = torch.randint(0, 10 ** 6, (17, 3), generator=gen, device=DEV, dtype=torch.int32)
    x, z = (torch.randn(17, 4, 96, generator=gen, device=DEV) for _ in range(2))
    y = rope(x, positions=pos)
    dx = rope(z, positions=pos, inverse=True)
    # each of the 17*4*96 products is off by 9 u of its pair's magnitudes
    bound = 2 * 9 * U * (y.abs().double() * 2 * z.abs().double()).sum().item() * 2
    assert abs((y.double() * z.double()).sum().item() - (x.double() * dx.double()).sum().item()) <= bound
    back = rope(y, positions=pos, inverse=True)
    pairs = x.view(17, 4, 48, 2).abs().sum(-1, keepdim=True).expand(-1, -1, -1, 2).reshape_as(x)
    assert bool(((back - x).abs() <= 40 * U * pairs).all())


@pytest.mark.parametrize("heads", [1, 7, 8, 9, 41])
def test_head_counts_single_row_and_empty(heads):
    rope = lib.QkvCteRopeAxes(64, (32, 32))
    x = torch.randn(1, heads, 64, generator=torch.Generator(device=DEV).manual_seed(heads), device=DEV)
    pos = torch.tensor([[3, 9]], dtype=torch.int32, device=DEV)
    ref, mag = _rotate(x, _angles(64, (32, 32), 0, 10000.0, pos), 0)
    _check(rope(x, positions=pos), ref, mag, 9)
    empty = rope(x[:0], positions=pos[:0])
    assert empty.shape == (0, heads, 64)


def test_other_stream_and_captured_graph():
    rope = lib.QkvCteRopeAxes(128, (44, 42, 42))
    x = torch.randn(500, 8, 128, device=DEV).bfloat16()
    grid = torch.tensor([[5, 10, 10]], dtype=torch.int32, device=DEV)
    ref = rope(x, grids=grid)
    cos, sin = rope.tables(1, 500, grids=grid)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = rope(x, grids=grid, stream=s)
    s.synchronize()
    assert torch.equal(y, ref)
    out, c2, s2 = torch.zeros_like(x), torch.zeros_like(cos), torch.zeros_like(sin)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rope(x, grids=grid, out=out)
        rope.tables(1, 500, grids=grid, cos=c2, sin=s2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(c2, cos) and torch.equal(s2, sin)
