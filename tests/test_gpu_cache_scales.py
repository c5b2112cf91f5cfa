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
    product, which is held as 2^6 at least: by 2^-11 of itself, or, where that is less, by half of
    fp16's least step, 2^-25, which is 2^-31 of the largest. Each key's code can be off by that much."""

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
        tol = (2.0 ** -11 + n * 2.0 ** -24 + 2 * e[..., None]) * mag + 2.0 ** -31 * top * total
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


@pytest.mark.parametrize("scales", [range(1, 11), [1] * 10, [6] * 10, [7] * 10, [3, 8] * 5, [4, 20, 1, 9]])
@BOTH_FORMS
def test_least_scales(S, scales):
    """Values near the least normal numbers of fp32 and bf16."""
    c = _case(list(scales), S)
    c.upload()
    out, lse = c.run()
    c.check(out, lse)
    assert bool((out != 0).any())
