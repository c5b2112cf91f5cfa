"""The 8-bit key/value cache in 64 bits, token by token: what the tests compare with."""
import math

import torch

F8 = torch.float8_e4m3fn
E4M3_MAX = 448.0


def least_exponent(amax: float) -> int:
    """Biased exponent of the least power of two (from 2^-126) that brings amax to at most 448."""
    if not math.isfinite(amax):
        return 255
    e = -126
    while e < 127 and amax > math.ldexp(E4M3_MAX, e):
        e += 1
    return e + 127


def grid(y):
    """To the e4m3 grid, ties to even, saturating."""
    ulp = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / ulp) * ulp).clamp(-E4M3_MAX, E4M3_MAX)


class Cache:
    """K or V: code values [pages, heads, bt, d] (64 bits) and exponents [pages, heads]."""

    def __init__(self, codes, sf):
        self.val, self.sf = codes.cpu().view(F8).double(), sf.cpu().int()

    def write(self, x, starts, counts, table):
        x = x.cpu().double()
        pages, heads, bt, _ = self.val.shape
        for b in range(x.shape[0]):
            first, n = starts[b], counts[b]
            for blk in range(max(0, first // bt), -(-(first + n) // bt)):
                if blk >= len(table[b]) or not 0 <= table[b][blk] < pages:
                    continue
                page = table[b][blk]
                lo, hi = max(first, blk * bt), min(first + n, blk * bt + bt)
                if hi <= lo:
                    continue
                at = lo - blk * bt
                for h in range(heads):
                    new = x[b, lo - first: hi - first, h]
                    e = least_exponent(new.abs().max().item() if bool(torch.isfinite(new).all()) else math.inf)
                    if at:
                        old = int(self.sf[page, h])
                        e = max(e, old)
                        if e != 255 and e != old:
                            self.val[page, h, :at] = grid(self.val[page, h, :at] * 2.0 ** (old - e))
                    self.sf[page, h] = e
                    self.val[page, h, at: at + hi - lo] = 0 if e == 255 else grid(new * 2.0 ** (127 - e))

    def tokens(self, b, n, table):
        """(values [n, heads, d], present [n]): holes are absent."""
        pages, heads, bt, d = self.val.shape
        out, there = torch.zeros(n, heads, d, dtype=torch.float64), torch.zeros(n, dtype=torch.bool)
        for blk in range(-(-n // bt)):
            if blk < len(table[b]) and 0 <= table[b][blk] < pages:
                page = table[b][blk]
                m = min(bt, n - blk * bt)
                e = self.sf[page].double()
                scale = torch.where(e == 255, torch.full_like(e, math.nan), torch.exp2(e - 127))
                out[blk * bt: blk * bt + m] = (self.val[page, :, :m] * scale[:, None, None]).transpose(0, 1)
                there[blk * bt: blk * bt + m] = True
        return out, there


def attention(q, k, v, lengths, counts, table, scale, causal, window, device="cpu"):
    """64-bit (out, lse, mean |v| under the weights, largest sum of |q k| * scale per row)."""
    B, S, nq, d = q.shape
    G = nq // k.val.shape[1]
    out = torch.zeros(B, S, nq, d, dtype=torch.float64, device=device)
    mag = torch.zeros_like(out)
    lse = torch.full((B, S, nq), -math.inf, dtype=torch.float64, device=device)
    big = torch.zeros(B, S, nq, dtype=torch.float64, device=device)
    bt = k.val.shape[2]
    for b in range(B):
        n = max(0, min(lengths[b], len(table[b]) * bt))
        c = max(0, min(counts[b], S))
        if n == 0 or c == 0:
            continue
        (kv, there), (vv, _) = k.tokens(b, n, table), v.tokens(b, n, table)
        kv, vv, there = kv.to(device), vv.to(device), there.to(device)
        pos = n - c + torch.arange(c, device=device)
        t = torch.arange(n, device=device)
        seen = there[None, :].expand(c, n)
        if causal:
            seen = seen & (t[None] <= pos[:, None])
            if window:
                seen = seen & (t[None] > pos[:, None] - window)
        for h in range(nq):
            qq = q[b, :c, h].to(device).double()
            kk = kv[:, h // G]
            z = torch.where(seen, scale * (qq @ kk.t()), torch.full((c, n), -math.inf, dtype=torch.float64, device=device))
            w = torch.logsumexp(z, dim=1)
            dead = ~seen.any(dim=1)
            p = torch.where(seen, torch.exp(z - torch.where(dead, torch.zeros_like(w), w)[:, None]), torch.zeros_like(z))
            vh = vv[:, h // G]
            # a key that a row does not see adds nothing, whatever it holds
            vz = torch.nan_to_num(vh, nan=0.0)
            o = p @ vz
            bad = (seen.double() @ torch.isnan(vh).double()) > 0
            out[b, :c, h] = torch.where(bad, torch.full_like(o, math.nan), o)
            mag[b, :c, h] = p @ vz.abs()
            lse[b, :c, h] = w
            big[b, :c, h] = (scale * (qq.abs() @ torch.nan_to_num(kk).abs().t()) * seen).amax(dim=1)
    return out, lse, mag, big
