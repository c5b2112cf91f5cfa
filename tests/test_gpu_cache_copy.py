"""Writing keys and values to the 8-bit cache and reading them back, bit for bit against 64
bits (a code rounds once, so there is one right answer)."""
import math

import pytest
import torch

import rope_tcgen05_mxfp8_gb300 as lib
from kv_cache_reference import Cache

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Case:
    """A pool of garbage, shuffled pages and a batch of rows."""

    def __init__(self, starts, counts, S, n, d, bt, dt, blocks, seed=0, fused=False, shift=0, holes=(), table=True):
        g = torch.Generator().manual_seed(seed)
        B = len(starts)
        self.starts, self.counts, self.S = starts, counts, S
        pages = B * blocks + 3
        self.table = torch.randperm(pages, generator=g)[: B * blocks].view(B, blocks).tolist()
        if not table:
            pages = B * blocks
            self.table = [[b * blocks + j for j in range(blocks)] for b in range(B)]
        for b, j in holes:
            self.table[b][j] = (-1, pages, 2 ** 31 - 1, -2 ** 31)[(b + j) % 4]
        self.with_table = table
        codes = torch.randint(0, 256, (2, pages, n, bt, d), generator=g, dtype=torch.uint8)
        codes[(codes & 127) == 127] = 3
        sf = torch.randint(100, 140, (2, pages, n), generator=g, dtype=torch.uint8)
        self.cache = lib.QkvCteCache(pages, n, d, block_tokens=bt, k=codes[0].to(DEV), v=codes[1].to(DEV),
                                     k_sf=sf[0].to(DEV), v_sf=sf[1].to(DEV))
        self.ref = [Cache(codes[0], sf[0]), Cache(codes[1], sf[1])]
        wide = 3 if fused else 1
        x = torch.randn(2, B, S, wide * n, d + shift, generator=g) * torch.exp2(
            torch.randint(-9, 9, (2, B, S, wide * n, 1), generator=g).float())
        self.x = [x[i].to(TYPES[dt]).to(DEV)[:, :, (wide - 1) * n:, shift:] for i in range(2)]

    def args(self):
        return dict(counts=None if self.counts is None else _i32(self.counts),
                    table=_i32(self.table) if self.with_table else None)

    def write(self, which=(0, 1)):
        k, v = (self.x[i] if i in which else None for i in range(2))
        self.cache.write(k, v, _i32(self.starts), **self.args())
        counts = [self.S] * len(self.starts) if self.counts is None else [max(0, min(c, self.S)) for c in self.counts]
        for i in which:
            self.ref[i].write(self.x[i], self.starts, counts, self.table)

    def check(self):
        for ref, codes, sf in ((self.ref[0], self.cache.k, self.cache.k_sf), (self.ref[1], self.cache.v, self.cache.v_sf)):
            assert torch.equal(sf.cpu().int(), ref.sf)
            assert torch.equal(codes.cpu().view(torch.float8_e4m3fn).double(), ref.val)  # untouched slots too


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("d,bt", [(128, 64), (128, 128), (128, 16), (16, 16), (16, 128), (80, 32), (48, 64), (112, 128)])
def test_write_ragged(dt, d, bt):
    c = Case([0, 5, bt, 2 * bt - 1], [70, 0, 1, 33], 70, 3, d, bt, dt, 70 // bt + 4, seed=d + bt)
    c.write()
    c.check()


@pytest.mark.parametrize("starts,counts,S", [
    ([0], None, 1), ([63], None, 1), ([64], None, 1), ([0], None, 64), ([1], None, 63), ([63], None, 2),
    ([0, 0], [1, 64], 64), ([10, 20], [-5, 1000], 30),   # counts outside 0 to S count as the nearest
    ([-3, -40], None, 30),                               # tokens before 0 are dropped
    ([250, 256], None, 20),                              # and those past the table
    ([2 ** 31 - 1, -2 ** 31], None, 20)])
def test_write_edges(starts, counts, S):
    c = Case(starts, counts, S, 2, 64, 64, "bf16", 4)
    c.write()
    c.check()


@pytest.mark.parametrize("kw", [dict(fused=True), dict(shift=1), dict(shift=8), dict(shift=1, fused=True),
                                dict(holes=((0, 1), (1, 0), (1, 2))), dict(table=False)])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_write_layouts(kw, dt):
    c = Case([3, 40], [100, 60], 100, 2, 96, 32, dt, 6, **kw)
    c.write()
    c.check()


def test_write_k_or_v_alone():
    c = Case([3, 40], None, 50, 2, 64, 32, "fp16", 4)
    c.write(which=(1,))
    c.check()
    c.write(which=(0,))
    c.check()


def test_token_by_token():
    """Growing scales move the codes that are there; one write of all gives the same scales."""
    c = Case([0], None, 150, 2, 32, 64, "bf16", 3)
    x = [t.clone() for t in c.x]
    grow = torch.exp2(torch.arange(150, device=DEV).float() / 8 - 9).bfloat16()[None, :, None, None]
    x = [t * grow for t in x]
    for s in range(150):
        c.starts, c.S, c.x = [s], 1, [t[:, s: s + 1] for t in x]
        c.write()
    c.check()
    k_sf = c.cache.k_sf.clone()
    c.starts, c.S, c.x = [0], 150, x
    c.write()
    c.check()
    used = [c.table[0][j] for j in range(3)]
    assert torch.equal(k_sf[used], c.cache.k_sf[used])


@pytest.mark.parametrize("dt,value", [("fp32", 1e-45), ("fp32", 1.1754944e-38), ("fp32", 3.4e38), ("fp32", 448.0),
                                      ("fp32", 448.00003), ("bf16", 0.0), ("bf16", 9.2e-41), ("bf16", 3.38e38),
                                      ("fp16", 6e-8), ("fp16", 65504.0), ("bf16", math.inf), ("bf16", math.nan),
                                      ("fp16", -math.inf), ("fp16", math.nan), ("fp32", math.nan), ("fp32", -math.inf)])
def test_write_extreme_values(dt, value):
    c = Case([5], None, 40, 2, 32, 32, dt, 3)
    for x in c.x:
        x[0, :, 0] *= 0
        x[0, 11, 0, 7] = value
        x[0, 12, 0, 8] = -value
    c.cache.k_sf[c.table[0][0]] = 1      # (the earlier tokens' scale)
    c.ref[0].sf[c.table[0][0]] = 1
    c.write()
    c.check()
    c.starts, c.S, c.x = [45], 2, [x[:, :2] for x in c.x]   # and on: a NaN stays
    c.write()
    c.check()


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("d,bt", [(128, 64), (128, 128), (16, 16), (80, 32), (48, 16)])
def test_read(dt, d, bt):
    c = Case([0, 5, -7, 3 * bt - 2], None, 3 * bt + 9, 3, d, bt, dt, 4, holes=((1, 1), (3, 3)), seed=d + bt)
    c.cache.k_sf[c.table[0][1], 1] = 255
    c.ref[0].sf[c.table[0][1], 1] = 255
    lengths = [3 * bt + 1, 2 * bt, 10 * bt, 0]
    k, v = c.cache.read(_i32(c.starts), c.S, _i32(lengths), table=_i32(c.table), dtype=TYPES[dt])
    for ref, got in ((c.ref[0], k), (c.ref[1], v)):
        want = torch.zeros(4, c.S, 3, d, dtype=torch.float64)
        for b in range(4):
            n = min(max(lengths[b], 0), 4 * bt)
            x, _ = ref.tokens(b, n, c.table)
            for s in range(c.S):
                if 0 <= c.starts[b] + s < n:
                    want[b, s] = x[c.starts[b] + s]
        want = want.to(TYPES[dt])        # every value fits fp32, so this rounds once
        assert torch.equal(torch.nan_to_num(got.cpu().float(), nan=-1e30), torch.nan_to_num(want.float(), nan=-1e30))


def test_read_into_views_and_alone():
    c = Case([1, 2], None, 40, 2, 48, 32, "bf16", 3)
    c.write()
    lengths, starts, table = _i32([41, 42]), _i32([0, 0]), _i32(c.table)
    k, v = c.cache.read(starts, 45, lengths, table=table)
    for shift in (0, 1, 8):
        wide = torch.full((2, 45, 5, 48 + 8), 7.0, dtype=torch.bfloat16, device=DEV)
        view = wide[:, :, 1:3, shift: shift + 48]
        version = wide._version
        got = c.cache.read(starts, 45, lengths, table=table, v=view)
        assert got[0] is None and got[1] is view and wide._version > version
        assert torch.equal(view, v)
        wide[:, :, 1:3, shift: shift + 48] = 7
        assert bool((wide == 7).all())
    one = c.cache.read(starts[:1], 45, lengths[:1], table=table[0], k=torch.empty(45, 2, 48, dtype=torch.bfloat16, device=DEV))
    assert torch.equal(one[0], k[0])


def test_round_trip_is_within_half_a_step():
    c = Case([0], None, 200, 2, 64, 64, "fp32", 4)
    c.write()
    k, _ = c.cache.read(_i32([0]), 200, _i32([200]), table=_i32(c.table), dtype=torch.float32)
    x = c.x[0]
    top = x.abs().amax(dim=3, keepdim=True)
    pad = torch.nn.functional.pad(top, (0, 0, 0, 0, 0, 56)).unflatten(1, (4, 64)).amax(dim=2)
    page_top = pad.repeat_interleave(64, dim=1)[:, :200]
    # half a step: 2^-4 of the value; below 2^-6 of the scale, 2^-10 of it, which is at most
    # 2^-18 * 2 of the page's largest element (that lies above 224 scales)
    assert bool(((k - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 * page_top / 224).all())


def test_many_rows_and_far_pages():
    """Codes past 2^32 bytes of the pool; one row of pages for all sequences in a read."""
    n, d, bt = 40, 128, 64
    pages = (1 << 32) // (n * d * bt) + 40
    cache = lib.QkvCteCache(pages, n, d, block_tokens=bt, k=torch.empty(pages, n, bt, d, dtype=torch.uint8, device=DEV),
                            v=torch.empty(pages, n, bt, d, dtype=torch.uint8, device=DEV))
    table = torch.arange(pages - 1, pages - 31, -1, dtype=torch.int32, device=DEV)
    x = torch.randn(1, 1900, n, d, device=DEV).bfloat16()
    cache.write(x, x, _i32([20]), table=table[None])
    k, v = cache.read(_i32([20, 20]), 1900, _i32([1920, 1920]), table=table)
    assert torch.equal(k[0], v[1]) and torch.equal(k[0], k[1])
    assert bool(((k[0].float() - x[0].float()).abs() <= 2.0 ** -4 * x[0].float().abs() + 2.0 ** -9 * 8 / 224).all())
    assert bool((cache.k_sf[: pages - 30] == 0).all())


def test_nothing_to_do():
    c = Case([0], None, 4, 1, 32, 16, "bf16", 2)
    c.cache.write(c.x[0][:, :0], c.x[1][:, :0], _i32([0]), table=_i32(c.table))
    c.cache.write(c.x[0][:0], c.x[1][:0], _i32([]), table=torch.empty(0, 2, dtype=torch.int32, device=DEV))
    c.check()
    k, v = c.cache.read(_i32([0]), 0, _i32([0]), table=_i32(c.table))
    assert k.shape == (1, 0, 1, 32) and v.shape == k.shape
