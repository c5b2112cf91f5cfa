"""The block operators beside the fused QKV projection, as measured workloads.

Four operators: the matrix product with bias, activation, gate and residual in its
epilogue (row-scaled e4m3 activations, MXFP8 weights), layer norm, its backward pass,
and rotary positions with several axes. Each case can be computed two ways: in plain
torch operations (``own`` false), or by the library's kernels (``own`` true).
"""
import math

import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one time-step embedding entering a block: a single row, latency counts
        dict(name="linear_one_row", op="linear", T=1, K=512, N=5120, act="silu", inp="bf16", gate=False,
             residual=False, col=False, out="bf16"),
        # a short prompt's or context's tokens through an embedding layer
        dict(name="linear_context", op="linear", T=512, K=4096, N=5120, act="gelu_tanh", inp="fp8", gate=False,
             residual=False, col=False, out="bf16"),
        # attention's output projection at 480p: gate and residual in the epilogue
        dict(name="linear_out_proj", op="linear", T=32760, K=5120, N=5120, act="none", inp="fp8", gate=True,
             residual=True, col=False, out="bf16"),
        # the feed-forward block's first layer on a short clip, fed by a bf16 norm
        dict(name="linear_ffn_up", op="linear", T=4096, K=5120, N=20480, act="gelu_tanh", inp="bf16", gate=False,
             residual=False, col=False, out="bf16"),
        # ragged in every direction: an adapter of odd width on an fp32 residual stream
        dict(name="linear_ragged", op="linear", T=1000, K=1056, N=333, act="gelu_erf", inp="fp8", gate=True,
             residual=True, col=True, out="fp32"),
        # the norm of one token
        dict(name="norm_one_row", op="norm", rows=1, cols=5120, x="bf16", p="bf16", stats=False),
        # the modulated norm before the projection at 480p, fp32 scale and shift
        dict(name="norm_480p", op="norm", rows=32760, cols=5120, x="bf16", p="fp32", stats=True),
        # training of the norms at a short clip
        dict(name="norm_backward_short", op="norm_backward", rows=4096, cols=5120, x="bf16", p="fp32"),
        # an odd width in fp32, few rows
        dict(name="norm_backward_ragged", op="norm_backward", rows=333, cols=1283, x="fp32", p="fp32"),
        # tables for the projection at 480p, the patches of a packed sequence in any order
        dict(name="rope_tables_480p", op="rope_tables", B=1, S=32760, d=128, dims="44,42,42", pairing="half",
             spectrum="axis", source="positions", far=0),
        # the queries inside a fused [T, I] projection output, rotated out of place
        dict(name="rope_queries_480p", op="rope", B=1, S=32760, heads=40, d=128, dims="44,42,42", pairing="half",
             spectrum="axis", source="grid", x="bf16", fused=True, inverse=False, far=0),
        # a padded batch's gradient: interleaved pairs, explicit far positions, fp16
        dict(name="rope_gradient_far", op="rope", B=2, S=777, heads=12, d=96, dims="32,32,32", pairing="inter",
             spectrum="shared", source="positions", x="fp16", fused=False, inverse=True, far=1000000),
    ]


def _dims(case):
    return tuple(int(v) for v in case["dims"].split(","))


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "norm", "norm_backward", "rope", "rope_tables"])
    if op == "linear":
        T, K, N = _log(rng, 1, 32760), 32 * _log(rng, 2, 160), _log(rng, 1, 20480)
        while T * N * K > 32760 * 5120 * 5120:
            T = max(1, T // 2)
        return dict(op=op, T=T, K=K, N=N, act=rng.choice(["none", "gelu_tanh", "gelu_erf", "silu"]),
                    inp=rng.choice(["fp8", "bf16"]), gate=rng.random() < 0.5, residual=rng.random() < 0.5,
                    col=rng.random() < 0.3, out=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op in ("norm", "norm_backward"):
        rows, cols = _log(rng, 1, 32760), _log(rng, 1, 20480)
        while rows * cols > 32760 * 5120 // (2 if op == "norm_backward" else 1):
            rows = max(1, rows // 2)
        x = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        case = dict(op=op, rows=rows, cols=cols, x=x, p=rng.choice([x, "fp32"]))
        if op == "norm":
            case["stats"] = rng.random() < 0.5
        return case
    axes = rng.choice([1, 2, 3])
    pairs = [_log(rng, 1, 64) for _ in range(axes)]
    d = 2 * sum(pairs)
    case = dict(op=op, B=rng.choice([1, 2, 3]), S=_log(rng, 1, 10920), d=d, dims=",".join(str(2 * p) for p in pairs),
                pairing=rng.choice(["half", "inter"]), spectrum=rng.choice(["axis", "shared"]),
                source=rng.choice(["grid", "positions"]), far=rng.choice([0, 1000, 1000000]))
    if op == "rope":
        heads = _log(rng, 1, 40)
        while case["B"] * case["S"] * heads * d > 32760 * 5120:
            case["S"] = max(1, case["S"] // 2)
        case.update(heads=heads, x=rng.choice(["bf16", "fp16", "fp32"]), fused=rng.random() < 0.3,
                    inverse=rng.random() < 0.5)
    else:  # tables of explicit positions (a grid's tables would not depend on the inputs' seed)
        case["source"] = "positions"
        while case["B"] * case["S"] * d > 32760 * 128:
            case["S"] = max(1, case["S"] // 2)
    return case


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _grid_of(S, axes, g):
    """A latent grid of `axes` sizes whose volume is S where S factors so (the 480p
    grid does), and at most S otherwise (the rows behind it are padding)."""
    if (S, axes) == (32760, 3):
        return [21, 30, 52]
    if axes == 1:
        return [max(1, S - int(torch.randint(0, 1 + S // 8, (1,), generator=g)))]
    sizes, left = [], S
    for a in range(axes - 1):
        sizes.append(max(1, int(round(left ** (1.0 / (axes - a))))))
        left //= sizes[-1]
    return sizes + [max(1, left)]


def _hidden(rows, cols, gen, dev):
    """Hidden states: normal, with a few channels far larger than the rest and an
    offset per row, as residual streams have them."""
    x = torch.randn(rows, cols, generator=gen, device=dev)
    chan = torch.rand(cols, generator=gen, device=dev)
    x = x * torch.where(chan > 0.995, 20.0, 1.0)
    return x + 0.3 * torch.randn(rows, 1, generator=gen, device=dev)


def _quantise_rows(x):
    """bf16 rows -> e4m3 codes and one fp32 scale each: s = amax / 448 (1 for a row of
    zeros), code = e4m3(x / s), both quotients IEEE fp32 divisions."""
    x = x.float()
    amax = x.abs().amax(dim=1)
    s = torch.where(amax > 0, amax / torch.full_like(amax, E4M3_MAX), torch.ones_like(amax))
    q = (x / s[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return q.to(torch.float8_e4m3fn).view(torch.uint8), s


def _mx_weights(N, K, gen, dev):
    """MXFP8 weights: e4m3 codes and a power-of-two scale per 32 elements along K."""
    w = 0.02 * torch.randn(N, K, generator=gen, device=dev)
    blocks = w.reshape(N, K // 32, 32)
    amax = blocks.abs().amax(dim=2)
    e = torch.ceil(torch.log2(amax.double() / E4M3_MAX)).clamp(-126, 127)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    q = (blocks / torch.exp2(e).float()[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return q.reshape(N, K).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        x = _hidden(T, K, gen, dev).to(torch.bfloat16)
        if case["inp"] == "bf16":
            st["A"], st["a_scale"] = x, None
        else:
            st["A"], st["a_scale"] = _quantise_rows(x)
        st["W"], st["w_sf"] = _mx_weights(N, K, gen, dev)
        st["bias"] = (0.02 * torch.randn(N, generator=gen, device=dev)).to(torch.bfloat16)
        dt = DTYPES[case["out"]]
        st["gate"] = (0.5 * torch.randn(N, generator=gen, device=dev)).to(torch.bfloat16) if case["gate"] else None
        st["col"] = (1.0 + 0.1 * torch.randn(N, generator=gen, device=dev)) if case["col"] else None
        st["residual"] = torch.randn(T, N, generator=gen, device=dev).to(dt) if case["residual"] else None
        if own:
            import rope_tcgen05_mxfp8_gb300 as lib
            acts = {"none": lib.QKV_CTE_ACT_NONE, "gelu_tanh": lib.QKV_CTE_ACT_GELU_TANH,
                    "gelu_erf": lib.QKV_CTE_ACT_GELU_ERF, "silu": lib.QKV_CTE_ACT_SILU}
            st["plan"] = lib.QkvCteLinear(
                T, K, N, act=acts[case["act"]], out_dtype=dt, device=dev,
                input_layout=lib.QKV_CTE_INPUT_BF16 if case["inp"] == "bf16" else lib.QKV_CTE_INPUT_ROW_FP8)
    elif op in ("norm", "norm_backward"):
        R, C = case["rows"], case["cols"]
        dt, pt = DTYPES[case["x"]], DTYPES[case["p"]]
        st["x"] = _hidden(R, C, gen, dev).to(dt)
        st["weight"] = (1.0 + 0.2 * torch.randn(C, generator=gen, device=dev)).to(pt)
        st["bias"] = (0.2 * torch.randn(C, generator=gen, device=dev)).to(pt)
        st["eps"] = 1e-6
        if op == "norm_backward":
            st["dy"] = torch.randn(R, C, generator=gen, device=dev).to(dt)
            x = st["x"].double()  # the statistics that the forward pass left
            mean = x.mean(dim=1)
            var = (x - mean[:, None]).square().mean(dim=1)
            st["mean"], st["rstd"] = mean.float(), torch.rsqrt(var + st["eps"]).float()
    else:
        B, S, d, dims = case["B"], case["S"], case["d"], _dims(case)
        axes = len(dims)
        host = torch.Generator()
        host.manual_seed(seed)
        st["positions"], st["grids"] = None, None
        if case["source"] == "grid":
            rows = []
            for b in range(B):
                size = _grid_of(S if b == 0 else max(1, S - S // 5), axes, host)
                rows.append(size)
            st["grids"] = torch.tensor(rows, dtype=torch.int32).to(dev)
        else:
            p = torch.randint(0, max(2, S), (S, axes), generator=host) + case["far"]
            st["positions"] = p.to(torch.int32).to(dev)
        if op == "rope":
            n, dt = case["heads"], DTYPES[case["x"]]
            if case["fused"]:  # the first heads of a wider row, as in a fused projection's output
                wide = torch.randn(B, S, 3 * n * d, generator=gen, device=dev).to(dt)
                st["x"] = wide[:, :, : n * d].unflatten(2, (n, d))
            else:
                st["x"] = torch.randn(B, S, n, d, generator=gen, device=dev).to(dt)
        if own:
            import rope_tcgen05_mxfp8_gb300 as lib
            st["rope"] = lib.QkvCteRopeAxes(
                d, dims, theta=10000.0,
                pairing=lib.QKV_CTE_ROPE_ROTATE_HALF if case["pairing"] == "half" else lib.QKV_CTE_ROPE_INTERLEAVED,
                spectrum=lib.QKV_CTE_ROPE_PER_AXIS if case["spectrum"] == "axis" else lib.QKV_CTE_ROPE_SHARED)
    return st


# ----------------------------------------------------------------------------
# the operators
# ----------------------------------------------------------------------------

def run(st):
    case = st["case"]
    return (_run_own if own else _run_plain)(case["op"], case, st)


def _run_own(op, case, st):
    import rope_tcgen05_mxfp8_gb300 as lib
    if op == "linear":
        return st["plan"](st["A"], st["a_scale"], st["W"], st["w_sf"], bias=st["bias"], gate=st["gate"],
                          residual=st["residual"], w_col_scale=st["col"])
    if op == "norm":
        y, mean, rstd = lib.qkv_cte_layer_norm(st["x"], st["weight"], st["bias"], eps=st["eps"],
                                               stats=case["stats"])
        return (y, mean, rstd) if case["stats"] else y
    if op == "norm_backward":
        return lib.qkv_cte_layer_norm_backward(st["dy"], st["x"], st["mean"], st["rstd"], st["weight"])
    if op == "rope_tables":
        return st["rope"].tables(case["B"], case["S"], positions=st["positions"], grids=st["grids"])
    return st["rope"](st["x"], positions=st["positions"], grids=st["grids"], inverse=case["inverse"])


def _run_plain(op, case, st):
    if op == "linear":
        if case["inp"] == "bf16":
            codes, scale = _quantise_rows(st["A"])
        else:
            codes, scale = st["A"], st["a_scale"]
        a = codes.view(torch.float8_e4m3fn).float()
        w = st["W"].view(torch.float8_e4m3fn).float()
        w = w * torch.exp2(st["w_sf"].float() - 127.0).repeat_interleave(32, dim=1)
        z = torch.matmul(a, w.t()) * scale[:, None]
        if st["col"] is not None:
            z = z * st["col"]
        z = z + st["bias"].float()
        if case["act"] == "gelu_tanh":
            z = 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
        elif case["act"] == "gelu_erf":
            z = 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
        elif case["act"] == "silu":
            z = z / (1.0 + torch.exp(-z))
        if st["gate"] is not None:
            z = z * st["gate"].float()
        if st["residual"] is not None:
            z = z + st["residual"].float()
        return z.to(DTYPES[case["out"]])
    if op == "norm":
        x = st["x"].float()
        mean = x.mean(dim=1)
        xc = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((xc * xc).mean(dim=1) + st["eps"])
        y = (xc * rstd[:, None] * st["weight"].float() + st["bias"].float()).to(st["x"].dtype)
        return (y, mean, rstd) if case["stats"] else y
    if op == "norm_backward":
        dy, rstd = st["dy"].float(), st["rstd"][:, None]
        xh = (st["x"].float() - st["mean"][:, None]) * rstd
        g = dy * st["weight"].float()
        dx = rstd * (g - g.mean(dim=1, keepdim=True) - xh * (g * xh).mean(dim=1, keepdim=True))
        pt = st["weight"].dtype
        return dx.to(st["x"].dtype), (dy * xh).sum(dim=0).to(pt), dy.sum(dim=0).to(pt)
    cos, sin = _plain_cos_sin(case, st)  # [B, S, d/2], 64 bits
    if op == "rope_tables":
        if case["pairing"] == "half":
            cos, sin = torch.cat([cos, cos], dim=2), torch.cat([sin, sin], dim=2)
        else:
            cos, sin = cos.repeat_interleave(2, dim=2), sin.repeat_interleave(2, dim=2)
        return cos.float().flatten(0, 1), sin.float().flatten(0, 1)
    c, s = cos.float()[:, :, None, :], sin.float()[:, :, None, :]
    if case["inverse"]:
        s = -s
    x, h = st["x"].float(), case["d"] // 2
    if case["pairing"] == "half":
        lo, hi = x[..., :h], x[..., h:]
        y = torch.cat([lo * c - hi * s, hi * c + lo * s], dim=3)
    else:
        lo, hi = x[..., 0::2], x[..., 1::2]
        y = torch.stack([lo * c - hi * s, hi * c + lo * s], dim=4).flatten(3)
    return y.to(st["x"].dtype)


def _plain_cos_sin(case, st):
    """Angles in 64 bits (far positions), position by position; rows behind a grid's
    end turn by nothing."""
    B, S, d, dims = case["B"], case["S"], case["d"], _dims(case)
    if st["grids"] is not None:
        g = st["grids"].long()
        dev = g.device
        s = torch.arange(S, device=dev)[None, :]
        coords, live = [None] * len(dims), s < g.prod(dim=1)[:, None]
        left = s.expand(B, S)
        for a in reversed(range(len(dims))):
            coords[a] = left % g[:, a : a + 1]
            left = left // g[:, a : a + 1]
        pos = torch.stack(coords, dim=2) * live[:, :, None]
    else:
        pos = st["positions"].long()[None].expand(B, -1, -1)
        dev = pos.device
    parts, first = [], 0
    for a, dim in enumerate(dims):
        j = torch.arange(dim // 2, device=dev, dtype=torch.float64)
        e = 2.0 * j / dim if case["spectrum"] == "axis" else 2.0 * (j + first) / d
        parts.append(pos[:, :, a : a + 1].double() * torch.pow(10000.0, -e))
        first += dim // 2
    ang = torch.cat(parts, dim=2)
    return torch.cos(ang), torch.sin(ang)


def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    op = case["op"]
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        o = T * N * size[case["out"]]
        b = T * K * 2 if case["inp"] == "bf16" else T * K + 4 * T
        b += N * K + N * K // 32 + 2 * N + (2 * N if case["gate"] else 0) + (4 * N if case["col"] else 0)
        return {"bytes": b + o * (2 if case["residual"] else 1), "flops": 2 * T * N * K}
    if op == "norm":
        R, C = case["rows"], case["cols"]
        return {"bytes": 2 * R * C * size[case["x"]] + 2 * C * size[case["p"]] + (8 * R if case["stats"] else 0),
                "flops": 8 * R * C}
    if op == "norm_backward":
        R, C = case["rows"], case["cols"]
        return {"bytes": 3 * R * C * size[case["x"]] + 3 * C * size[case["p"]] + 8 * R, "flops": 14 * R * C}
    rows = case["B"] * case["S"]
    pos = (case["B"] if case["source"] == "grid" else case["S"]) * len(_dims(case)) * 4
    if op == "rope_tables":
        return {"bytes": 2 * rows * case["d"] * 4 + pos, "flops": rows * case["d"]}
    n = rows * case["heads"] * case["d"]
    return {"bytes": 2 * n * size[case["x"]] + pos, "flops": 3 * n}


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        if case["inp"] == "bf16":
            x = st["A"].double()
            top = x.abs().amax(dim=1)
            scale = torch.where(top > 0, (top / E4M3_MAX).float().double(), torch.ones_like(top))
            a = (x / scale[:, None]).float().clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).double()
        else:
            a, scale = st["A"].view(torch.float8_e4m3fn).double(), st["a_scale"].double()
        N, K = st["W"].shape
        out = []
        for n0 in range(0, N, 4096):
            n1 = min(N, n0 + 4096)
            w = st["W"][n0:n1].view(torch.float8_e4m3fn).double().reshape(n1 - n0, K // 32, 32)
            w = torch.ldexp(w, st["w_sf"][n0:n1].int()[:, :, None] - 127).reshape(n1 - n0, K)
            z = (a @ w.t()) * scale[:, None]
            if st["col"] is not None:
                z = z * st["col"][n0:n1].double()
            z = z + st["bias"][n0:n1].double()
            if case["act"] == "gelu_tanh":
                u = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z.pow(3))
                z = z * torch.sigmoid(2.0 * u)
            elif case["act"] == "gelu_erf":
                z = 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
            elif case["act"] == "silu":
                z = z * torch.sigmoid(z)
            if st["gate"] is not None:
                z = z * st["gate"][n0:n1].double()
            if st["residual"] is not None:
                z = z + st["residual"][:, n0:n1].double()
            out.append(z)
        return torch.cat(out, dim=1)
    if op == "norm":
        x = st["x"].double()
        n = x.shape[1]
        mean = x.sum(dim=1) / n
        var = (x - mean[:, None]).pow(2).sum(dim=1) / n
        rstd = (var + st["eps"]).pow(-0.5)
        y = torch.addcmul(st["bias"].double(), (x - mean[:, None]) * rstd[:, None], st["weight"].double())
        return (y, mean, rstd) if case["stats"] else y
    if op == "norm_backward":
        x, dy, w = st["x"].double(), st["dy"].double(), st["weight"].double()
        r = st["rstd"].double()[:, None]
        n = x.shape[1]
        xh = (x - st["mean"].double()[:, None]) * r
        s1 = (dy @ w)[:, None] / n
        s2 = ((dy * xh) @ w)[:, None] / n
        return r * (dy * w - s1 - xh * s2), torch.einsum("rc,rc->c", dy, xh), dy.sum(dim=0)
    # rotary positions: complex turns, axis by axis
    B, S, d, dims = case["B"], case["S"], case["d"], _dims(case)
    turns = []
    for b in range(B):
        if st["grids"] is not None:
            size = [int(v) for v in st["grids"][b]]
            axes = torch.meshgrid(*[torch.arange(v, dtype=torch.float64) for v in size], indexing="ij")
            pos = torch.stack([a.reshape(-1) for a in axes], dim=1)[:S]
            pos = torch.cat([pos, torch.zeros(S - len(pos), len(dims), dtype=torch.float64)])
        else:
            pos = st["positions"].cpu().double()
        cols, pair = [], 0
        for a, dim in enumerate(dims):
            for j in range(dim // 2):
                e = j / (dim // 2) if case["spectrum"] == "axis" else pair / (d // 2)
                cols.append(pos[:, a] * math.exp(-e * math.log(10000.0)))
                pair += 1
        turns.append(torch.stack(cols, dim=1))
    turn = torch.stack(turns)
    turn = torch.polar(torch.ones_like(turn), turn)
    if op == "rope_tables":
        half = case["pairing"] == "half"
        wide = torch.cat([turn, turn], dim=2) if half else torch.stack([turn, turn], dim=3).flatten(2)
        return wide.real.reshape(B * S, d).contiguous(), wide.imag.reshape(B * S, d).contiguous()
    turn = turn.to(st["x"].device)[:, :, None, :]
    if case["inverse"]:
        turn = turn.conj()
    x = st["x"].double()
    if case["pairing"] == "half":
        y = torch.complex(x[..., : d // 2], x[..., d // 2 :]) * turn
        return torch.cat([y.real, y.imag], dim=3)
    y = torch.complex(x[..., 0::2].contiguous(), x[..., 1::2].contiguous()) * turn
    return torch.view_as_real(y).flatten(3)
