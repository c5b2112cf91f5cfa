"""CPU checks of the key/value cache's entry points: every refusal comes before any launch,
with its documented code (no GPU, the addresses are never read)."""
import ctypes

import pytest
import torch

import rope_tcgen05_mxfp8_gb300 as pkg
from rope_tcgen05_mxfp8_gb300 import build as b
from rope_tcgen05_mxfp8_gb300 import kv_cache as kc
from rope_tcgen05_mxfp8_gb300 import qkv_cte as q

MB = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _built():
    b.build()


DESC = dict(pages=8, n_kv_heads=2, d_head=64, block_tokens=32, flags=0)


def _plan(**kw):
    d = dict(DESC, **kw)
    plan, codes, scales = ctypes.c_void_p(), ctypes.c_size_t(), ctypes.c_size_t()
    desc = kc.qkv_cte_cache_desc(*(d[k] for k in ("pages", "n_kv_heads", "d_head", "block_tokens", "flags")))
    rc = kc._lib().qkv_cte_cache_plan(ctypes.byref(plan), ctypes.byref(desc), ctypes.byref(codes), ctypes.byref(scales))
    return rc, plan, codes.value, scales.value


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(pages=0), -1), (dict(pages=-1), -1), (dict(n_kv_heads=0), -1), (dict(d_head=0), -1),
    (dict(d_head=8), -2), (dict(d_head=72), -2), (dict(d_head=144), -2), (dict(d_head=128), 0), (dict(d_head=16), 0),
    (dict(block_tokens=16), 0), (dict(block_tokens=128), 0), (dict(block_tokens=0), -2), (dict(block_tokens=48), -2),
    (dict(block_tokens=256), -2), (dict(block_tokens=8), -2), (dict(flags=2), -1), (dict(flags=1), 0),
    (dict(pages=2 ** 31), -2), (dict(pages=2 ** 31 - 1), 0), (dict(n_kv_heads=65536), -2)])
def test_plan(kw, code):
    rc, plan, codes, scales = _plan(**kw)
    assert rc == code
    if code == 0:
        d = dict(DESC, **kw)
        assert scales == d["pages"] * d["n_kv_heads"] and codes == scales * d["block_tokens"] * d["d_head"]
        kc._lib().qkv_cte_cache_destroy(plan)
    else:
        assert not plan.value and "qkv_cte_cache_plan" in q.qkv_cte_last_error()


def test_null_plans():
    lib = kc._lib()
    desc = kc.qkv_cte_cache_desc(8, 2, 64, 32, 0)
    assert lib.qkv_cte_cache_plan(None, ctypes.byref(desc), None, None) == -1
    assert lib.qkv_cte_cache_plan(ctypes.byref(ctypes.c_void_p()), None, None, None) == -1
    lib.qkv_cte_cache_destroy(None)
    n = ctypes.c_size_t()
    assert lib.qkv_cte_cache_attention_workspace(None, 1, 1, 2, 8, ctypes.byref(n)) == -1


# codes 32 KB each, scales 16 bytes each
POOL = dict(kc=64 * MB, ks=65 * MB, vc=66 * MB, vs=67 * MB, table=68 * MB, stride=4, blocks=4)
COPY = dict(k=1 * MB, kb=1280, ks_=128, kh=64, v=2 * MB, vb=1280, vs_=128, vh=64, batch=2, seq=10, starts=70 * MB,
            second=71 * MB, dtype=0, read=False)


def _pages(a):
    return kc.qkv_cte_cache_pages(a["kc"], a["ks"], a["vc"], a["vs"], a["table"], a["stride"], a["blocks"])


def _copy(**kw):
    a = dict(POOL, **COPY)
    a.update(kw)
    _, plan, _, _ = _plan()
    fn = kc._lib().qkv_cte_cache_read if a["read"] else kc._lib().qkv_cte_cache_write
    rc = fn(plan if a.get("plan", True) else None, ctypes.byref(_pages(a)) if a.get("pages", True) else None, a["k"],
            a["kb"], a["ks_"], a["kh"], a["v"], a["vb"], a["vs_"], a["vh"], a["batch"], a["seq"], a["starts"],
            a["second"], a["dtype"], None)
    kc._lib().qkv_cte_cache_destroy(plan)
    return rc


COMMON = [
    (dict(plan=False), -1), (dict(pages=False), -1), (dict(kc=None), -1), (dict(vs=None), -1),
    (dict(kc=64 * MB + 8), -2), (dict(table=68 * MB + 2), -2), (dict(blocks=0), -1), (dict(blocks=-3), -1),
    (dict(blocks=2 ** 26, stride=2 ** 26), -2), (dict(stride=3), -1), (dict(stride=-4), -1),
    (dict(stride=2 ** 62), -2), (dict(table=None, blocks=5), -1),
    (dict(vc=64 * MB + 16 * 1024), -1), (dict(ks=66 * MB + 64), -1), (dict(table=64 * MB), -1),
    (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(batch=-1), -1), (dict(seq=-1), -1),
    (dict(batch=0), 0), (dict(seq=0), 0), (dict(seq=2 ** 31), -2), (dict(batch=2 ** 20, seq=2 ** 11, table=68 * MB, stride=0), -2),
    (dict(k=None, v=None), -1), (dict(starts=None), -1), (dict(starts=70 * MB + 1), -2), (dict(second=71 * MB + 2), -2),
    (dict(k=1 * MB + 1), -2), (dict(kb=-1280), -1), (dict(ks_=2 ** 60), -2),
    (dict(k=64 * MB), -1), (dict(v=67 * MB - 64), -1),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(stride=0), -1),                                  # one row of pages, two writers
    (dict(starts=64 * MB), -1), (dict(second=67 * MB), -1),
])
def test_write_refusals(kw, code):
    assert _copy(**kw) == code
    if code:
        assert "qkv_cte_cache_write" in q.qkv_cte_last_error()


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(second=None), -1), (dict(kh=0), -1), (dict(ks_=64), -1), (dict(kb=0), -1),   # results must be distinct
    (dict(v=1 * MB + 64), -1), (dict(k=70 * MB - 64), -1), (dict(v=71 * MB), -1),
])
def test_read_refusals(kw, code):
    assert _copy(read=True, **kw) == code
    if code:
        assert "qkv_cte_cache_read" in q.qkv_cte_last_error()


ATT = dict(q=1 * MB, qb=2560, qs=256, qh=64, o=2 * MB, ob=2560, os=256, oh=64, lse=3 * MB, batch=2, seq=10, heads=4,
           lengths=70 * MB, counts=71 * MB, longest=128, scale=0.125, causal=0, window=0, dtype=0, ws=80 * MB,
           wsn=None, status=72 * MB)


def _workspace(plan, a):
    n = ctypes.c_size_t()
    rc = kc._lib().qkv_cte_cache_attention_workspace(plan, a["batch"], a["seq"], a["heads"], a["longest"], ctypes.byref(n))
    return rc, n.value


def _att(**kw):
    a = dict(POOL, **ATT)
    a.update(kw)
    _, plan, _, _ = _plan()
    wsn = a["wsn"] if a["wsn"] is not None else _workspace(plan, a)[1]
    rc = kc._lib().qkv_cte_cache_attention(
        plan, ctypes.byref(_pages(a)), a["q"], a["qb"], a["qs"], a["qh"], a["o"], a["ob"], a["os"], a["oh"], a["lse"],
        a["batch"], a["seq"], a["heads"], a["lengths"], a["counts"], a["longest"], a["scale"], a["causal"], a["window"],
        a["dtype"], a["ws"], wsn, a["status"], None)
    kc._lib().qkv_cte_cache_destroy(plan)
    return rc


LONG = dict(table=68 * MB, stride=4096, blocks=4096, longest=131072, batch=1, seq=1)   # keys in parts


@pytest.mark.parametrize("kw,code", [
    (dict(kc=None), -1), (dict(vc=64 * MB + 1), -2), (dict(blocks=0), -1), (dict(table=None, blocks=5), -1),
    (dict(heads=0), -1), (dict(heads=3), -1), (dict(heads=-2), -1), (dict(longest=-1), -1),
    (dict(batch=-1), -1), (dict(seq=-1), -1), (dict(batch=0), 0), (dict(seq=0), 0),
    (dict(seq=2 ** 31 - 1), -2), (dict(heads=2 ** 30), -2), (dict(batch=1, seq=(2 ** 31 - 1024) // 4), -2),
    (dict(dtype=2), -2), (dict(dtype=3), -1),
    (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(causal=2), -1), (dict(window=-1), -1), (dict(window=5), -1),
    (dict(lengths=None), -1), (dict(lengths=70 * MB + 1), -2), (dict(counts=71 * MB + 2), -2),
    (dict(status=None), -1), (dict(status=72 * MB + 2), -2), (dict(lse=3 * MB + 2), -2),
    (dict(q=None), -1), (dict(q=MB + 1), -2), (dict(qs=-256), -1), (dict(o=None), -1), (dict(o=2 * MB + 1), -2),
    (dict(os=64), -1), (dict(oh=0), -1), (dict(ob=0), -1), (dict(ob=2 ** 61), -2),
    (dict(o=MB), -1), (dict(o=MB + 64), -1),                          # over the queries
    (dict(o=64 * MB), -1), (dict(o=68 * MB), -1), (dict(o=70 * MB - 64), -1), (dict(lse=2 * MB), -1), (dict(lse=MB), -1),
    (dict(lse=66 * MB), -1), (dict(lse=70 * MB), -1), (dict(status=2 * MB), -1), (dict(status=65 * MB), -1),
    (dict(status=3 * MB), -1), (dict(status=MB + 4), -1),
    (dict(LONG, ws=None), -1), (dict(LONG, ws=80 * MB + 16), -2), (dict(LONG, wsn=16), -1), (dict(LONG, ws=64 * MB), -1),
    (dict(LONG, ws=2 * MB), -1), (dict(LONG, ws=72 * MB), -1), (dict(LONG, ws=MB), -1), (dict(LONG, ws=70 * MB), -1),
])
def test_attention_refusals(kw, code):
    assert _att(**kw) == code
    if code:
        assert "qkv_cte_cache_attention" in q.qkv_cte_last_error()


def test_workspace():
    """Nothing for keys in one part; grows with the rows otherwise; refusals."""
    _, plan, _, _ = _plan()
    base = dict(batch=1, seq=1, heads=4, longest=64)
    assert _workspace(plan, base) == (0, 0)
    one, two = (_workspace(plan, dict(base, longest=10 ** 6, seq=s)) for s in (1, 2))
    assert one[0] == two[0] == 0 and two[1] >= one[1] > 0
    assert _workspace(plan, dict(base, heads=3))[0] == -1
    assert _workspace(plan, dict(base, longest=-1))[0] == -1
    assert _workspace(plan, dict(base, seq=2 ** 31))[0] == -2
    assert _workspace(plan, dict(base, longest=2 ** 62))[0] == 0
    assert kc._lib().qkv_cte_cache_attention_workspace(plan, 1, 1, 4, 8, None) == -1
    kc._lib().qkv_cte_cache_destroy(plan)


def test_binding_refuses_numbers_beyond_the_c_types():
    big = 2 ** 32
    for kw in (dict(n_kv_heads=big + 2), dict(d_head=big + 64), dict(block_tokens=big + 64), dict(flags=big), dict(pages=2 ** 64)):
        with pytest.raises(pkg.QkvCteError) as ei:
            pkg.QkvCteCache(**dict(dict(pages=8, n_kv_heads=2, d_head=64), **kw))
        assert ei.value.code == pkg.QKV_CTE_ERR_UNSUPPORTED


def test_binding_refuses_other_devices():
    with pytest.raises(ValueError, match="CUDA"):
        pkg.QkvCteCache(8, 2, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        pkg.QkvCteCache(8, 2, 64, k=torch.zeros(8, 2, 64, 64, dtype=torch.uint8))


