"""The cache and its attention in a run with their neighbours: fused projection (norm, rotation)
-> keys and values into the cache -> attention of its query columns -> output product; chunk by
chunk, captured, on two threads; refusals of the binding; a wait that runs out."""
import threading

import pytest
import torch

import rope_tcgen05_mxfp8_gb300 as lib
import workloads as wl
from kv_cache_reference import Cache, attention
from test_gpu_linear import Case as Product

pytestmark = pytest.mark.gpu
DEV = "cuda"
T, H, HEADS, KV, D, BT = 5 * 8 * 8, 512, 8, 2, 64, 32


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _check_attention(out, ref, mag, big, n):
    """As derived in test_gpu_cache_attention."""
    e = (D + 8) * 2.0 ** -23 * big + 2.0 ** -20
    tol = (2.0 ** -11 + n * 2.0 ** -24 + 2 * e[..., None]) * mag
    tol = tol + 2.0 ** -8 * (ref.abs() + tol) + 2.0 ** -24 * mag
    assert bool(((out.double() - ref).abs() <= tol).all())


class Block:
    """One block's projection, cache and output product."""

    def __init__(self, seed=3):
        self.call = wl.custom_call(tokens=T, hidden=H, n_q_heads=HEADS, n_kv_heads=KV, d_head=D, norm=2, rope=1,
                                   rope_grid=(5, 8, 8), seed=seed)
        self.w = {k: v.to(DEV) for k, v in wl.make_inputs(self.call).items() if v is not None}
        self.qkv = lib.QkvCte(T, H, HEADS, KV, D, norm=2, rope=1)
        blocks = -(-T // BT)
        self.cache = lib.QkvCteCache(blocks + 2, KV, D, block_tokens=BT)
        self.table = torch.randperm(blocks + 2, generator=torch.Generator().manual_seed(seed))[:blocks].tolist()
        self.dev_table = _i32(self.table)
        self.product = Product(T, HEADS * D, H, seed=4)
        self.out = lib.QkvCteLinear(T, HEADS * D, H, input_layout=lib.QKV_CTE_INPUT_BF16)
        self.zero, self.full = _i32([0]), _i32([T])

    def project(self):
        w = self.w
        fused = self.qkv(w["A"], w["a_scale"], w["W"], w["w_sf"], w["bias"], w["gamma_q"], w["gamma_k"], w["cos"], w["sin"])
        heads = fused.view(1, T, HEADS + 2 * KV, D)
        return heads[:, :, :HEADS], heads[:, :, HEADS: HEADS + KV], heads[:, :, HEADS + KV:]

    def run(self):
        q, k, v = self.project()
        self.cache.write(k, v, self.zero, table=self.dev_table)
        o, lse = self.cache.attention(q, self.full, table=self.dev_table, causal=True, stats=True)
        y = self.out(o.view(T, HEADS * D), None, self.product.W, self.product.sf, bias=self.product.bias)
        return q, k, v, o, lse, y

    def reference(self, q, k, v):
        shape = self.cache.k.shape
        refs = []
        for x in (k, v):
            c = Cache(torch.zeros(shape, dtype=torch.uint8), torch.zeros(shape[:2], dtype=torch.uint8))
            c.write(x, [0], [T], [self.table])
            refs.append(c)
        return refs


def test_block_step_by_step():
    b = Block()
    q, k, v, o, lse, y = b.run()
    kr, vr = b.reference(q, k, v)
    for ref, codes, sf in ((kr, b.cache.k, b.cache.k_sf), (vr, b.cache.v, b.cache.v_sf)):
        used = sorted(b.table)
        assert torch.equal(sf.cpu().int()[used], ref.sf[used])
        assert torch.equal(codes.cpu().view(torch.float8_e4m3fn).double()[used], ref.val[used])
    ref, _, mag, big = attention(q.cpu(), kr, vr, [T], [T], [b.table], D ** -0.5, True, 0, DEV)
    _check_attention(o, ref, mag, big, T)
    codes, scale = wl.row_quantise(o.view(T, HEADS * D).cpu())
    b.product.A, b.product.s, b.product.gate, b.product.res = codes.to(DEV), scale.to(DEV), None, None
    b.product.check(y)
    for op in (b.qkv, b.cache, b.out):
        assert op.status() == 0


def test_chunk_by_chunk():
    """Uneven chunks, down to single tokens: each attends to what has been written, and the scales
    at the end are those of one write."""
    b = Block()
    q, k, v = b.project()
    b.cache.write(k, v, b.zero, table=b.dev_table)
    whole = b.cache.k_sf.clone(), b.cache.v_sf.clone()
    shape = b.cache.k.shape
    refs = [Cache(b.cache.k, b.cache.k_sf), Cache(b.cache.v, b.cache.v_sf)]
    at = 0
    for n in (1, 1, 5, 60, 1, 130, 2, 120):
        part = slice(at, at + n)
        b.cache.write(k[:, part], v[:, part], _i32([at]), table=b.dev_table)
        for r, x in zip(refs, (k, v)):
            r.write(x[:, part], [at], [n], [b.table])
        at += n
        o, _ = b.cache.attention(q[:, part], _i32([at]), table=b.dev_table, causal=True)
        ref, _, mag, big = attention(q[:, part].cpu(), *refs, [at], [n], [b.table], D ** -0.5, True, 0, DEV)
        _check_attention(o, ref, mag, big, at)
    assert at == T and torch.equal(whole[0], b.cache.k_sf) and torch.equal(whole[1], b.cache.v_sf)
    assert b.cache.k.shape == shape


def test_captured_and_on_another_stream():
    b = Block()
    want = b.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = b.run()
    s.synchronize()
    keep = [t.clone() for t in want]
    assert all(torch.equal(g, w) for g, w in zip(got[3:], keep[3:]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.run()
    for _ in range(2):
        b.cache.k.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got[3:], keep[3:]))


def test_two_threads():
    b = Block()
    q, k, v = (t.clone() for t in b.project())
    b.cache.write(k, v, b.zero, table=b.dev_table)
    want = b.cache.attention(q, b.full, table=b.dev_table, causal=True)[0]
    one = b.cache.attention(q[:, -1:], b.full, table=b.dev_table, causal=True)[0]
    torch.cuda.synchronize()
    bad = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(30):
                x = b.cache.attention(q, b.full, table=b.dev_table, causal=True)[0]
                y = b.cache.attention(q[:, -1:], b.full, table=b.dev_table, causal=True, max_length=100000)[0]
                torch.cuda.current_stream().synchronize()
                if not (torch.equal(x, want) and torch.allclose(y.float(), one.float(), rtol=2 ** -7, atol=2 ** -7)):
                    bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad and b.cache.status() == 0


def test_bounded_waits_report_and_the_context_survives():
    """With the test hook nothing is handed to the tensor cores: every wait runs out, the call
    ends, the status says so, and the next call is right."""
    b = Block()
    q, k, v = b.project()
    b.cache.write(k, v, b.zero, table=b.dev_table)
    want = b.cache.attention(q, b.full, table=b.dev_table)[0]
    c = b.cache
    stalled = lib.QkvCteCache(c.pages, KV, D, block_tokens=BT, k=c.k, v=c.v, k_sf=c.k_sf, v_sf=c.v_sf,
                              flags=lib.QKV_CTE_FLAG_TEST_STALL)
    stalled.attention(q[:, :130], b.full, table=b.dev_table)
    with pytest.raises(lib.QkvCteError) as ei:
        stalled.status()
    assert ei.value.code == lib.QKV_CTE_ERR_DEVICE_TIMEOUT
    assert stalled.status() == 0
    assert torch.equal(c.attention(q, b.full, table=b.dev_table)[0], want) and c.status() == 0


def test_binding_refusals():
    b = Block()
    q, k, v = b.project()
    c, t, n = b.cache, b.dev_table, b.full
    bad = [
        lambda: c.write(k.float().double(), v, b.zero), lambda: c.write(k, v.float(), b.zero, table=t),
        lambda: c.write(k[..., :32], v, b.zero, table=t), lambda: c.write(k, v[:, :10], b.zero, table=t),
        lambda: c.write(k.cpu(), v, b.zero, table=t), lambda: c.write(k.transpose(2, 3).contiguous().transpose(2, 3), v, b.zero, table=t),
        lambda: c.write(None, None, b.zero, table=t), lambda: c.write(k, v, n.long(), table=t),
        lambda: c.write(k, v, _i32([0, 0]), table=t), lambda: c.write(k, v, b.zero, counts=_i32([1, 2]), table=t),
        lambda: c.write(k, v, b.zero, table=t.long()), lambda: c.write(k, v, b.zero, table=t.cpu()),
        lambda: c.write(k, v, b.zero, table=t.view(1, 1, -1)), lambda: c.write(k, v, b.zero, table=t.expand(3, -1)),
        lambda: c.write(torch.cat([k, k]), torch.cat([v, v]), _i32([0, 0]), table=t.expand(2, -1)),
        lambda: c.write(torch.cat([k, k]), torch.cat([v, v]), _i32([0, 0]), table=t),
        lambda: c.read(b.zero, -1, n, table=t), lambda: c.read(b.zero, 2 ** 31, n, table=t),
        lambda: c.read(b.zero, T, n, table=t, dtype=torch.float64), lambda: c.read(b.zero, T, n.cpu(), table=t),
        lambda: c.read(b.zero.view(1, 1), T, n, table=t), lambda: c.read(b.zero, 10, n, table=t, k=k),
        lambda: c.read(b.zero, T, n, table=t, k=torch.empty_like(k), v=torch.empty(1, T, KV, D, device=DEV)),
        lambda: c.attention(q.float(), n, table=t), lambda: c.attention(q[..., :32], n, table=t),
        lambda: c.attention(q[:, :, :7], n, table=t), lambda: c.attention(q, n, table=t, window=3),
        lambda: c.attention(q, n, table=t, scale=0.0), lambda: c.attention(q, n, table=t, scale=float("nan")),
        lambda: c.attention(q, n, table=t, out=q), lambda: c.attention(q, n, table=t, out=q.float()),
        lambda: c.attention(q, n, table=t, out=torch.empty_like(q)[:, 1:]), lambda: c.attention(q, n[:0], table=t),
        lambda: c.attention(q, n, table=t, lse=torch.empty(1, HEADS, T, device=DEV)), lambda: c.attention(q, n, table=t, window=2 ** 32 + 5, causal=True),
        lambda: c.attention(q, n, table=t, max_length=-1),
        lambda: lib.QkvCteCache(4, KV, D, k=c.k), lambda: lib.QkvCteCache(c.pages, KV, D, block_tokens=BT, k=c.k.float()),
        lambda: lib.QkvCteCache(c.pages, KV, D, block_tokens=BT, k=c.k, v=c.k),
    ]
    before = c.k.clone()
    for i, call in enumerate(bad[:-1]):
        with pytest.raises((ValueError, TypeError, lib.QkvCteError)):
            call()
            pytest.fail(f"call {i} was taken")
    both = bad[-1]()                                    # one pool for K and V: refused when it is used
    with pytest.raises(lib.QkvCteError):
        both.write(k, v, b.zero, table=t)
    with pytest.raises(lib.QkvCteError):
        both.attention(q, n, table=t)
    torch.cuda.synchronize()
    assert torch.equal(before, c.k)


def test_writes_count_as_modification_in_place():
    b = Block()
    _, k, v = b.project()
    versions = [t._version for t in (b.cache.k, b.cache.k_sf, b.cache.v, b.cache.v_sf)]
    b.cache.write(k, None, b.zero, table=b.dev_table)
    after = [t._version for t in (b.cache.k, b.cache.k_sf, b.cache.v, b.cache.v_sf)]
    assert all(a > o for a, o in zip(after[:2], versions[:2])) and after[2:] == versions[2:]
    with torch.inference_mode():
        c = lib.QkvCteCache(4, KV, D, block_tokens=BT)
        c.write(k[:, :10], v[:, :10], b.zero)
        c.attention(k[:, :10].repeat_interleave(2, dim=2), _i32([10]))
    torch.cuda.synchronize()
