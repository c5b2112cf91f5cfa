"""Attention over the 8-bit cache where value scales are small or lie far apart: what a row does
not see, or sees with next to no weight, takes nothing from the rest. Tolerances as derived in
test_gpu_cache_attention; forms: up to 64 query rows per key head, and beyond."""
import math

import pytest
import torch

from kv_cache_reference import Cache
from test_gpu_cache_attention import DEV, Case

pytestmark = pytest.mark.gpu
BOTH_FORMS = pytest.mark.parametrize("S", [1, 20, 65, 300])


class Apart(Case):
    """A weight is rounded to fp16 times its page's value scale, relative to the row's largest such
    product, which is held as 2^6 at least, in the form for few rows as 2: by 2^-11 of itself, or, where
    that is less, by half of fp16's least step, 2^-25, which is 2^-31 or 2^-26 of the largest. Each key's
    code can be off by that much."""

    def check(self, out, lse):
        counts = [self.S] * len(self.lengths) if self.counts is None else self.counts
        k, v = Cache(self.codes[0], self.sf[0]), Cache(self.codes[1], self.sf[1])
        ref, ref_lse, mag, big = self.reference()
        # the largest p 2^(sf - 127) and the sum of |code| are the same attention over other values
        top, total = torch.zeros_like(ref), torch.zeros_like(ref)
        n, G = self.lengths[0], self.nq // self.nkv
        kv, _ = k.tokens(0, n, self.table)
        codes = torch.cat([v.val[p] for p in self.table[0]], dim=1)[:, :n].to(DEV)
        sf = torch.cat([v.sf[p, :, None].expand(-1, self.bt) for p in self.table[0]], dim=1)[:, :n].double().to(DEV)
        t, pos = torch.arange(n, device=DEV), n - self.S + torch.arange(self.S, device=DEV)
        seen = torch.ones(self.S, n, dtype=torch.bool, device=DEV)
        if self.causal:
            seen = t[None] <= pos[:, None]
            if self.window:
                seen &= t[None] > pos[:, None] - self.window
        for h in range(self.nq):
            z = self.scale * (self.q[0, :, h].to(DEV).double() @ kv[:, h // G].to(DEV).t()) - ref_lse[0, :, h, None]
            w = torch.where(seen, z / math.log(2) + sf[h // G] - 127, torch.full_like(z, -math.inf)).amax(dim=1)
            top[0, :, h] = torch.exp2(w)[:, None]
            total[0, :, h] = seen.double() @ codes[h // G].abs()
        e = (self.d + 8) * 2.0 ** -23 * big + 2.0 ** -20
        half, tiny = 2.0 ** -8, 2.0 ** -134          # of bf16: half a step, half the least step
        tol = (2.0 ** -11 + n * 2.0 ** -24 + 2 * e[..., None]) * mag + 2.0 ** (-26 if self.S * G <= 64 else -31) * top * total
        tol = tol + half * (ref.abs() + tol) + tiny
        miss = (out.double() - ref).abs()
        assert bool((miss <= tol).all()), f"{int((~(miss <= tol)).sum())} of {miss.numel()}, worst {(miss / tol).max().item():.3g} of it"
        lim = e + n * 2.0 ** -24 + 2.0 ** -22 * (1 + ref_lse.abs())
        assert bool(((lse.double() - ref_lse).abs() <= lim).all())


def _case(scales, S, **kw):
    """One sequence, a value scale per page."""
    kw = dict(dict(nq=2, nkv=2, d=64, bt=16, spread=0), **kw)
    c = Apart([kw.pop("length", len(scales) * kw["bt"])], S=S, **kw)
    for j, e in enumerate(scales):
        c.sf[1, c.table[0][j]] = e
    return c


def _towards(c, page, exponent):
    """The page's keys along all queries (which become positive), or against them for a negative
    exponent: scores of about +-2^|exponent|."""
    c.q = c.q.abs() + 0.5
    p = c.table[0][page]
    k = c.codes[0, p]
    c.codes[0, p] = torch.where((k & 127) == 127, k, (k & 127) | (0x80 if exponent < 0 else 0))
    # |code| about 80 and d lanes of about 1.3: the sum is about 104 d
    c.sf[0, p] = 127 + round(abs(exponent) - math.log2(104 * c.d * c.scale))


@pytest.mark.parametrize("scales", [range(1, 11), [1] * 10, [6] * 10, [7] * 10, [3, 8] * 5, [4, 20, 1, 9]])
@BOTH_FORMS
def test_least_scales(S, scales):
    """Values near the least normal numbers of fp32 and bf16."""
    c = _case(list(scales), S)
    c.upload()
    out, lse = c.run()
    c.check(out, lse)
    assert bool((out != 0).any())


@pytest.mark.parametrize("above", [24, 34, 45, 60, 110])
@BOTH_FORMS
def test_hidden_page_of_large_values(S, above):
    """A page 2^above larger behind the causal edge of the earlier rows, and one before every row's
    window, in the tiles of keys that the rows walk."""
    scales = [120 + j % 3 for j in range(30)]
    c = _case(scales, S, causal=True, length=470)
    c.sf[1, c.table[0][29]] = 121 + above        # seen by the last rows alone (or by all there are)
    c.upload()
    c.run_and_check()
    n = min(S, 120)                              # rows from position 470 - n on, which see 33 keys back
    c = _case(scales, n, causal=True, window=33, length=470)
    before = (470 - n - 33) // 16 - 1
    for j in range(before - 3, before + 1):
        c.sf[1, c.table[0][j]] = 121 + above
    c.upload()
    out, lse = c.run()
    c.check(out, lse)
    c.sf[1, :] = c.sf[1, :].clamp(max=122)       # the hidden pages like the rest: nothing changes
    c.upload()
    like, like_lse = c.run()
    c.check(like, like_lse)
    assert torch.allclose(out.float(), like.float(), rtol=2.0 ** -7, atol=2.0 ** -9 * float(like.abs().max()))


@pytest.mark.parametrize("above,score", [(30, 6), (34, 7), (45, 7), (60, 8), (110, 8), (126, 9)])
@pytest.mark.parametrize("page", [0, 3, 11])
@BOTH_FORMS
def test_large_values_of_negligible_weight(S, above, score, page):
    """The page of large values stands 2^score away from the queries: its weight times its values is
    next to nothing, and the other pages' values come out."""
    c = _case([119 + j % 2 for j in range(12)], S)
    _towards(c, page, -score)
    c.sf[1, c.table[0][page]] = 120 + above
    c.upload()
    ref, _, _, _ = c.reference()
    with_small = float(ref.abs().max())
    assert with_small < 2.0 ** 6                 # (the large page's share is below that)
    c.run_and_check()


@pytest.mark.parametrize("least", [1, 30, 70, 100])
@pytest.mark.parametrize("score", [4, 5, 6, 7])
@pytest.mark.parametrize("page", [0, 5, 9])
@BOTH_FORMS
def test_least_values_of_nearly_all_weight(S, page, score, least):
    """The other way round: a page of small values (of zeros, at the least scale) takes nearly all
    of the weight, and what is left of the others is the answer."""
    c = _case([150 + j % 3 for j in range(10)], S)
    _towards(c, page, score)
    p = c.table[0][page]
    c.sf[1, p] = least
    if least == 1:
        k = c.codes[1, p]
        c.codes[1, p] = torch.where((k & 127) == 127, k, torch.zeros_like(k))
    c.upload()
    c.run_and_check()


@pytest.mark.parametrize("page", [0, 3, 11])
@BOTH_FORMS
def test_zeros_of_all_the_weight(S, page):
    """A page of zeros 2^300 above the rest in weight: nothing of the rest is left."""
    c = _case([127] * 12, S)
    _towards(c, page, 8)
    k = c.codes[1, c.table[0][page]]
    c.codes[1, c.table[0][page]] = torch.where((k & 127) == 127, k, torch.zeros_like(k))
    c.upload()
    for longest in (None, 1, 10 ** 6):
        out, lse = c.run(max_length=longest)
        c.check(out, lse)
        assert bool((out == 0).all())


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("spread", [0, 4])
@BOTH_FORMS
def test_a_single_key_comes_out_as_it_is(S, spread, dt):
    """The value of the only key that a row sees is a code times a power of two: no rounding at all."""
    c = Case([700], S=S, nq=4, nkv=2, d=64, bt=16, dt=dt, causal=True, window=1, spread=spread, gain=3.0)
    for longest in (None, 1, 10 ** 6):
        out, lse = c.run(max_length=longest)
        ref, _, _, _ = c.reference()
        assert torch.equal(out.double(), ref)
    c.check(out, lse)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 50)])
@BOTH_FORMS
def test_scales_of_the_whole_range(S, seed, causal, window):
    g = torch.Generator().manual_seed(seed)
    least, most = ((1, 230), (100, 160), (60, 200), (1, 60), (180, 230), (1, 230))[seed]
    c = _case([120] * 30, S, causal=causal, window=window, length=470, seed=seed, gain=(1.0, 8.0)[seed & 1])
    c.sf[1][c.sf[1] != 255] = torch.randint(least, most + 1, (int((c.sf[1] != 255).sum()),), generator=g, dtype=torch.uint8)
    if seed == 5:                                # a page of zeros now and then
        for j in range(0, 30, 4):
            p = c.table[0][j]
            k = c.codes[1, p]
            c.codes[1, p] = torch.where((k & 127) == 127, k, torch.zeros_like(k))
            c.sf[1, p] = 1
    c.upload()
    c.run_and_check()


@BOTH_FORMS
@pytest.mark.parametrize("nan_pages", [8, 9, 29, 30])
def test_nan_pages_before_any_other(S, nan_pages):
    """Pages of NaN values first: the rows that see one are NaN, their log-sums are not."""
    c = _case([150] * 30, S, causal=True, window=200, length=470)
    for j in range(nan_pages):
        c.sf[1, c.table[0][j]] = 255
    c.upload()
    Case.check(c, *c.run())


@pytest.mark.parametrize("lead", [4, 6, 7])
@pytest.mark.parametrize("S", [1, 70])
def test_scales_far_apart_over_parts(S, lead):
    """Keys divided among blocks: one part holds zeros that take nearly all the weight, another the
    large values, joined from parts that are far apart in both."""
    c = _case([127 + 100 if j > 30 else 127 for j in range(64)], S, nq=1, nkv=1, bt=128)
    p = c.table[0][2]
    _towards(c, 2, lead)
    c.sf[1, p] = 1
    c.codes[1, p] = 0
    c.upload()
    out, lse = c.run()
    c.check(out, lse)
    c.check(*c.run(max_length=1))


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@BOTH_FORMS
def test_queries_that_are_not_finite(S, dt, value):
    """Where every score is an infinity of one sign, too; rows that see nothing stay empty."""
    c = Case([40, 40], S=S, nq=2, nkv=2, d=32, bt=16, dt=dt, causal=True)
    live = (c.codes[0] & 127) != 127
    c.codes[0] = torch.where(live, (c.codes[0] & 0x7F).clamp(min=8), c.codes[0])   # positive, not zero
    c.upload()
    want, want_lse = c.run()
    c.check(want, want_lse)
    c.q[0, S // 2, 1, 7] = value
    out, lse = c.run()
    sees = S - 1 - S // 2 < 40
    bad = torch.zeros(2, S, 2, dtype=torch.bool, device=DEV)
    bad[0, S // 2, 1] = sees
    assert torch.equal(torch.isnan(out), bad[..., None].expand_as(out)) and torch.equal(torch.isnan(lse), bad)
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], want_lse[~bad])
