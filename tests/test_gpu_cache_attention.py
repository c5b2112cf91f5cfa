"""Attention over the 8-bit cache against 64 bits, at the lengths, masks and layouts where it
can go wrong.

Tolerance, from the arithmetic. Codes and queries are exact; a score is off by its fp32 sum
and product (d + 8 roundings, each at most 2^-23 of sum |q k| c, tensor cores may truncate),
so a weight is off by e = (d + 8) 2^-23 Z + 2^-20 relative, Z the row's largest sum |q k| c
(2^-20: the exponential and the maxima's factors). Weights are rounded to fp16 (2^-11), or
by 2^-25 of the largest where they are tiny. The output's sum of n terms adds n 2^-24. All of
these are relative to M = sum p |v| / sum p, twice e for numerator and denominator; then one
rounding to the output's type."""
import math

import pytest
import torch

import rope_tcgen05_mxfp8_gb300 as lib
from kv_cache_reference import Cache, attention

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Case:
    """Sequences of `lengths` tokens in shuffled pages of a pool whose every unused slot and
    page is NaN."""

    def __init__(self, lengths, S=1, nq=4, nkv=2, d=128, bt=64, dt="bf16", counts=None, causal=False, window=0,
                 scale=None, seed=0, spread=3, holes=(), shared=False, table=True, gain=1.0, extra=0):
        g = torch.Generator().manual_seed(seed)
        B = len(lengths)
        self.lengths, self.counts, self.S, self.nq, self.d, self.dt = lengths, counts, S, nq, d, dt
        self.causal, self.window, self.scale = causal, window, d ** -0.5 if scale is None else scale
        blocks = max(1, -(-max([1] + lengths) // bt)) + extra
        pages = (1 if shared else B) * blocks + (2 if table else 0)
        order = torch.randperm(pages, generator=g) if table else torch.arange(pages)
        self.table = order[: (1 if shared else B) * blocks].view(-1, blocks).tolist()
        if shared:
            self.table = self.table * B
        self.shared, self.with_table = shared, table
        x = torch.randn(2, pages, nkv, bt, d, generator=g)
        codes = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        sf = (127 - 7 + torch.randint(-spread, spread + 1, (2, pages, nkv), generator=g)).to(torch.uint8)
        live = torch.zeros(pages, bt, dtype=torch.bool)
        for b, n in enumerate(lengths):
            for t in range(min(n, blocks * bt)):
                live[self.table[b][t // bt], t % bt] = True
        codes[:, ~live[:, None, :, None].expand(pages, nkv, bt, d)] = 0x7F
        sf[:, ~live.any(dim=1)] = 255
        for b, j in holes:
            self.table[b][j] = (-1, pages, 2 ** 31 - 1, -2 ** 31)[(b + j) % 4]
        self.codes, self.sf = codes, sf
        self.q = (gain * torch.randn(B, S, nq, d, generator=g)).to(TYPES[dt])
        self.bt, self.nkv, self.pages = bt, nkv, pages
        self.upload()

    def upload(self):
        self.cache = lib.QkvCteCache(self.pages, self.nkv, self.d, block_tokens=self.bt, k=self.codes[0].to(DEV),
                                     v=self.codes[1].to(DEV), k_sf=self.sf[0].to(DEV), v_sf=self.sf[1].to(DEV))
        if not self.with_table:
            self.dev_table = None
        else:
            self.dev_table = _i32(self.table[0] if self.shared else self.table)

    def run(self, q=None, **kw):
        kw.setdefault("stats", True)
        return self.cache.attention(self.q.to(DEV) if q is None else q, _i32(self.lengths),
                                    counts=None if self.counts is None else _i32(self.counts), table=self.dev_table,
                                    causal=self.causal, window=self.window, scale=self.scale, **kw)

    def reference(self):
        counts = [self.S] * len(self.lengths) if self.counts is None else self.counts
        return attention(self.q, Cache(self.codes[0], self.sf[0]), Cache(self.codes[1], self.sf[1]), self.lengths,
                         counts, self.table, self.scale, self.causal, self.window, DEV)

    def check(self, out, lse):
        ref, ref_lse, mag, big = self.reference()
        e = (self.d + 8) * 2.0 ** -23 * big + 2.0 ** -20
        n = max([1] + self.lengths)
        half = torch.finfo(TYPES[self.dt]).eps / 2
        tiny = torch.finfo(TYPES[self.dt]).tiny * torch.finfo(TYPES[self.dt]).eps / 2  # half the least step
        tol = (2.0 ** -11 + n * 2.0 ** -24 + 2 * e[..., None]) * mag
        tol = tol + half * (ref.abs() + tol) + tiny + 2.0 ** -24 * mag
        got = out.double()
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        bad = ((got - ref).abs() > tol) & ~torch.isnan(ref)
        worst = torch.nan_to_num((got - ref).abs() / tol.clamp(min=1e-300)).max().item()
        assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} out of tolerance, worst {worst:.2f} of it"
        if lse is not None:
            assert torch.equal(torch.isinf(lse), torch.isinf(ref_lse)) and torch.equal(torch.isnan(lse), torch.isnan(ref_lse))
            d = torch.nan_to_num(lse.double() - ref_lse, nan=0.0, posinf=0.0, neginf=0.0).abs()
            lim = e + n * 2.0 ** -24 + 2.0 ** -22 * (1 + torch.nan_to_num(ref_lse, neginf=0.0).abs())
            assert bool((d <= torch.nan_to_num(lim, nan=1.0)).all())

    def run_and_check(self):
        self.check(*self.run())


@pytest.mark.parametrize("S", [1, 2, 7, 8, 9, 40, 130, 300])
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(S, causal):
    """From no token to several tiles, lengths on every side of the tiles' edges (causal rows
    of short sequences see nothing)."""
    Case([0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 515], S=S, causal=causal).run_and_check()


@pytest.mark.parametrize("S,nq", [(8, 2), (9, 2), (16, 2), (17, 2), (32, 2), (33, 2), (63, 1), (64, 1), (65, 1), (128, 1),
                                  (129, 1), (255, 1), (256, 1), (257, 1), (511, 1), (512, 1), (513, 1), (1030, 1)])
def test_rows_at_the_edges_of_tiles_and_forms(S, nq):
    Case([1100, 140], S=S, nq=nq, nkv=1, d=64, bt=32, causal=True).run_and_check()


@pytest.mark.parametrize("bt", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("S", [3, 50])
def test_heads_and_pages(bt, d, S):
    Case([300, 77, 131], S=S, d=d, bt=bt, causal=True, dt="fp16" if d % 32 else "bf16", seed=d + bt).run_and_check()


@pytest.mark.parametrize("nq,nkv", [(1, 1), (3, 1), (5, 5), (12, 4), (16, 1), (17, 1), (40, 8), (48, 2), (130, 1)])
@pytest.mark.parametrize("S", [1, 5, 33])
def test_shared_heads(nq, nkv, S):
    Case([200, 65], S=S, nq=nq, nkv=nkv, d=64, causal=True, dt="fp16").run_and_check()


@pytest.mark.parametrize("window", [1, 2, 16, 63, 100, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("S", [1, 4, 200])
def test_window(window, S):
    Case([400, 201, 64, 3], S=S, causal=True, window=window, bt=32).run_and_check()


@pytest.mark.parametrize("S,counts", [(6, [6, 0, 3, -2, 100]), (150, [150, 0, 1, 129, 77])])
@pytest.mark.parametrize("causal", [False, True])
def test_padded_queries(S, counts, causal):
    c = Case([200, 100, 150, 20, 90], S=S, counts=counts, causal=causal, d=96)
    c.counts = counts
    out, lse = c.run()
    c.counts = [max(0, min(v, S)) for v in counts]
    c.check(out, lse)
    for b, n in enumerate(c.counts):
        assert bool((out[b, n:] == 0).all()) and bool((lse[b, n:] == -math.inf).all())


@pytest.mark.parametrize("S", [2, 140])
def test_holes(S):
    """Blocks without a page are not attended; rows that see only those are empty."""
    c = Case([300, 130, 64], S=S, bt=64, causal=True, holes=((0, 0), (0, 2), (1, 1), (2, 0)))
    c.run_and_check()
    c = Case([300, 130], S=S, bt=16, holes=tuple((0, j) for j in range(19)) + ((1, 3),))
    out, lse = c.run()
    c.check(out, lse)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())


@pytest.mark.parametrize("S", [3, 200])
@pytest.mark.parametrize("which", [0, 1])
def test_nan_where_it_is_seen(S, which):
    """A page whose scale is NaN: rows that see one of its keys are NaN, the others are not
    touched, in the same tile as well."""
    c = Case([400, 230], S=S, bt=16, causal=True, window=30)
    page = c.table[0][23], c.table[1][12]
    for p in page:
        c.sf[which, p, 1] = 255
    c.upload()
    c.run_and_check()


@pytest.mark.parametrize("S", [1, 20, 300])
def test_unlike_scales(S):
    """Value scales 2^40 apart, a zero page with the least scale, and weights that leave the
    large scale next to nothing."""
    c = Case([512], S=S, nq=2, nkv=2, d=64, bt=64, spread=0)
    for j, e in enumerate((107, 147, 107, 1, 120, 127, 135, 110)):
        c.sf[1, c.table[0][j]] = e
    c.codes[1, c.table[0][3]] = 0
    # the keys of the page of large values point away from every query
    c.q = c.q.abs() + 0.5
    kc = c.codes[0, c.table[0][1]]
    c.codes[0, c.table[0][1]] = kc | 0x80
    c.upload()
    c.run_and_check()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("S", [2, 150])
def test_peaks_and_far_queries(dt, S):
    """Large scores (one key takes all), and queries of extreme size."""
    Case([300], S=S, dt=dt, gain=12.0).run_and_check()
    c = Case([300], S=S, dt=dt, scale=2.0 ** -30 * 0.1)
    c.q = (c.q.float() * (2.0 ** 30 if dt == "bf16" else 1000.0)).to(c.q.dtype)
    c.run_and_check()
    c = Case([300], S=S, dt=dt)
    c.q[:, :, 0] = 0
    c.q[:, :, 1] = (c.q[:, :, 1].float() * 1e-6).to(c.q.dtype)
    c.run_and_check()


def test_queries_that_are_not_finite():
    for S in (3, 140):
        c = Case([200], S=S, causal=True)
        want, _ = c.run()
        c.q[0, 1, 1, 5] = math.nan
        c.q[0, 2, 3, 0] = math.inf
        out, _ = c.run()
        assert bool(torch.isnan(out[0, 1, 1]).all()) and bool(torch.isnan(out[0, 2, 3]).all())
        keep = torch.ones(S, 4, dtype=torch.bool, device=DEV)
        keep[1, 1] = keep[2, 3] = False
        assert torch.equal(out[0][keep], want[0][keep])


@pytest.mark.parametrize("S", [1, 3, 90])
def test_layouts(S):
    """Queries out of a wider row, unaligned ones, transposed heads; results into views."""
    c = Case([150, 260], S=S, nq=6, nkv=3, d=64, causal=True)
    want, lse = c.run()
    c.check(want, lse)
    q = c.q.to(DEV)
    wide = torch.full((2, S, 12, 64), math.nan, dtype=torch.bfloat16, device=DEV)
    wide[:, :, :6] = q
    assert torch.equal(c.run(wide[:, :, :6])[0], want)
    got = c.run(wide[:, :, :6], out=wide[:, :, 6:], stats=False)[0]     # beside the queries
    assert torch.equal(got, want)
    odd = torch.empty(2 * S * 6 * 65 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(2, S, 6, 65)[..., :64]
    odd.copy_(q)
    assert torch.equal(c.run(odd)[0], want)
    heads_first = q.transpose(1, 2).contiguous().transpose(1, 2)
    out = torch.empty(2, 6, S, 64, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    flat = torch.empty(2 * S * 6, device=DEV)
    version = out._version
    got, gl = c.run(heads_first, out=out, lse=flat)
    assert torch.equal(got, want) and torch.equal(gl.view(2, S, 6), lse) and got is out and out._version > version
    odd_out = torch.empty(2 * S * 6 * 65 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(2, S, 6, 65)[..., :64]
    assert torch.equal(c.run(q, out=odd_out)[0], want)
    c3 = c.cache.attention(q[1], _i32(c.lengths[1:]), table=c.dev_table[1], causal=True)[0]
    assert c3.shape == q[1].shape
    c.check(torch.stack([want[0], c3]), None)


@pytest.mark.parametrize("S", [1, 60])
def test_tables(S):
    """No table, one row for all sequences, a table wider than the sequences, a page twice."""
    Case([150, 100], S=S, table=False).run_and_check()
    Case([150, 100, 1], S=S, shared=True).run_and_check()
    Case([150, 100], S=S, extra=40).run_and_check()
    c = Case([256, 100], S=S)
    c.table[0][3] = c.table[0][0]
    c.table[1][0] = c.table[0][1]
    c.upload()
    c.run_and_check()


@pytest.mark.parametrize("S", [1, 5, 64])
def test_long(S):
    """Keys divided among many blocks, with uneven lengths."""
    c = Case([20011, 3, 9000], S=S, nq=2, nkv=1, d=64, bt=128, causal=True)
    out, lse = c.run()
    c.check(out, lse)
    few = c.run(max_length=1)
    c.check(*few)                        # as one part
    again = c.run()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("S", [1, 200])
def test_far_pages(S):
    """Codes past 2^32 bytes of the pool give what the same codes near its start give."""
    n, d, bt, T = 40, 128, 64, 1900
    pages = (1 << 32) // (n * d * bt) + 40
    far = lib.QkvCteCache(pages, n, d, block_tokens=bt, k=torch.empty(pages, n, bt, d, dtype=torch.uint8, device=DEV),
                          v=torch.empty(pages, n, bt, d, dtype=torch.uint8, device=DEV))
    near = lib.QkvCteCache(30, n, d, block_tokens=bt)
    table = torch.arange(pages - 1, pages - 31, -1, dtype=torch.int32, device=DEV)[None]
    k, v = torch.randn(2, 1, T, n, d, device=DEV).bfloat16()
    q = torch.randn(1, S, n, d, device=DEV).bfloat16()
    far.write(k, v, _i32([0]), table=table)
    near.write(k, v, _i32([0]))
    a = far.attention(q, _i32([T]), table=table, causal=True, max_length=T)[0]
    b = near.attention(q, _i32([T]), causal=True, max_length=T)[0]
    assert torch.equal(a, b)


def test_lengths_beyond_the_table():
    c = Case([128, 128], S=2, bt=64)
    want, _ = c.run()
    c.lengths = [1000, 2 ** 31 - 1]
    got, _ = c.run()
    assert torch.equal(got, want)
    c.lengths = [-1, -2 ** 31]
    got, lse = c.run()
    assert bool((got == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("S", [1, 200])
def test_captured_and_replayed_with_other_lengths(S):
    c = Case([700, 300], S=S, causal=True)
    q, table = torch.zeros_like(c.q).to(DEV), c.dev_table
    lengths = _i32([1, 1])
    c.run(q)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):                    # two graphs of one object
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = c.cache.attention(q, lengths, table=table, causal=True, stats=True)
        graphs.append((g, r))
    q.copy_(c.q)
    for lens in ([700, 300], [64, 299], [700, 1]):
        lengths.copy_(_i32(lens))
        for g, r in graphs:
            g.replay()
        torch.cuda.synchronize()
        c.lengths = lens
        for g, r in graphs:
            c.check(*r)


@pytest.mark.parametrize("S", [1, 200])
def test_streams(S):
    """Another stream than the current one, and two at once."""
    c = Case([700, 300], S=S, causal=True)
    want = c.run()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    q, lengths = c.q.to(DEV), _i32(c.lengths)
    torch.cuda.synchronize()
    rs = []
    for _ in range(4):
        rs += [c.cache.attention(q, lengths, table=c.dev_table, causal=True, stats=True, stream=s) for s in (a, b)]
    torch.cuda.synchronize()
    assert all(torch.equal(r[0], want[0]) and torch.equal(r[1], want[1]) for r in rs)
    assert c.cache.status() == 0


def test_empty_calls():
    c = Case([100], S=1)
    out, lse = c.cache.attention(c.q.to(DEV)[:, :0], _i32([100]), table=c.dev_table, stats=True)
    assert out.shape == (1, 0, 4, 128) and lse.shape == (1, 0, 4)
    out, _ = c.cache.attention(c.q.to(DEV)[:0], _i32([]), table=c.dev_table[:0])
    assert out.shape == (0, 1, 4, 128)
