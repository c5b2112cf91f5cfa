"""Attention over the 8-bit cache: every head size over many tiles of keys, with one and with two
tiles of rows (tolerance as derived in test_gpu_cache_attention)."""
import pytest

from test_gpu_cache_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("S,causal,window", [(130, False, 0), (130, True, 300), (700, True, 0), (70, False, 0)])
def test_many_tiles_of_keys(d, S, causal, window):
    c = Case([2309, 1537], S=S, nq=2, nkv=1 if S == 70 else 2, d=d, bt=32, causal=causal, window=window, seed=d)
    out, lse = c.run()
    c.check(out, lse)
    c.check(*c.run(max_length=1))        # the keys in one part
