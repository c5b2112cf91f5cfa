"""The product's activations over [-12, 12] and beyond, relative to the result: with
identity-like weights z is the row's scale, exactly.

Tolerances, u = 2^-24. The activation's own relative error: 2^-20, and u |argument| for
each rounding of the exponential's argument. GELU (tanh) forms its argument with six (two
constants, four operations) for any output. For 16-bit outputs, GELU (erf) squares and
scales with three and the fast exponential multiplies by log2 e with two more. The
output's rounding adds half a step of its type (or half its smallest subnormal). Values
below 2^-119 may be taken as zero: there the exponential leaves fp32's range."""
import math

import pytest
import torch

import rope_tcgen05_mxfp8_gb300 as lib
from test_gpu_linear import ACTS, DEV, TYPES

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _exact(act, z):
    """(value, |argument of the exponential|) in 64 bits."""
    if act == "gelu_tanh":
        u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        return z * torch.special.expit(u), u.abs()
    if act == "gelu_erf":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2)), 0.5 * z * z
    if act == "silu":
        return z * torch.special.expit(z), z.abs()
    return z, torch.zeros_like(z)


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "gelu_erf", "silu"])
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,pad", [(60, 0), (2400, 0), (2400, 1)])
def test_values_relative_to_the_result(act, out, T, pad):
    """T = 60: the channel-major form; 2400: K1; with odd rows: the channel-major form."""
    N, K = 32, 32
    dt = TYPES[out]
    mag = torch.cat([torch.linspace(0, 12, T - T // 3, device=DEV),
                     torch.logspace(-6, 1.9, T // 3, device=DEV)]).float()
    A = torch.zeros(T, K, dtype=torch.uint8, device=DEV)
    A[:, 0] = 0x38                                                   # 1.0
    W = torch.zeros(N, K, dtype=torch.uint8, device=DEV)
    W[0::2, 0], W[1::2, 0] = 0x38, 0xB8                              # 1.0 and -1.0
    sf = torch.full((N, K // 32), 127, dtype=torch.uint8, device=DEV)
    op = lib.QkvCteLinear(T, K, N, act=ACTS[act], out_dtype=dt)
    wide = torch.zeros(T, N + pad, dtype=dt, device=DEV)
    got = op(A, mag, W, sf, out=wide[:, :N]).double()
    z = torch.stack([mag, -mag], 1).repeat(1, N // 2).double()
    ref, arg = _exact(act, z)
    e = 2.0 ** -20 if act != "none" else 0.0
    roundings = {"gelu_tanh": 6}.get(act, 0)
    if out != "fp32":
        roundings += {"gelu_erf": 5, "none": 0}.get(act, 2)
    e = e + roundings * U * arg
    fi = torch.finfo(dt)
    tol = ref.abs() * (fi.eps / 2) + 1.01 * ref.abs() * e + fi.tiny * fi.eps / 2
    tol = torch.where(ref.abs() < 2.0 ** -119, torch.full_like(tol, 2.0 ** -119), tol)
    over = ref.abs() > fi.max
    err = torch.where(over, torch.zeros_like(ref), (got - ref).abs())
    worst = (err / tol).max().item()
    at = (err / tol).argmax().item()
    assert worst <= 1.0, f"{worst:.3g} tolerances at z = {z.flatten()[at].item():.6g}"
