"""GELU, SILU and their slopes at every bf16 pre-activation of up to 128, far
tails included, against 64 bits.  A row an expert, so that the bias' gradient
is a slope and, with one column of dy set, the row weight's an activation, both
in fp32; the product's z is one weight, so y is an activation rounded.

Bounds, from the formulas the kernels use (u = 2^-24; the hardware's 2^x is
good to 4 u and 1/x to 2 u of the result, subnormals as zero):
  sigmoid  s = 1 / (1 + 2^(-log2(e) z)).  The exponent takes the constant's and
    the product's rounding, |z| 2 u of 2^x; with the sum and the reciprocal s is
    good to r = (2 |z| + 8) u of itself, and where 2^x overflows s is 0 (below
    2^-126).  silu = z s: r + u.  Slope s (1 + z (1 - s)): s's error times the
    factor, then the factor's: |z| times s's and the subtraction's, and three
    roundings.
  Phi by Abramowitz and Stegun 7.1.26, 1 - Phi(|z|) = e p(t) / 2 with e =
    exp(-z^2 / 2), t = 1 / (1 + 0.3275911 |z| / sqrt 2), p of degree 5 without a
    constant: the method's own error is computed in 64 bits from its formula.
    e: an exponent of three roundings, 1.5 z^2 u, and 4 u; t: 6 u, which a term
    of degree i takes i times, 30 u at most of the sum of the terms' sizes, and
    10 u for the roundings of the chain.  gelu = z Phi; slope Phi + z e / sqrt(2 pi).
"""
import math

import pytest
import torch

from experts_reference import ACTS, U, act64, bf16_bound, slope64
from test_gpu_experts import status

pytestmark = pytest.mark.gpu

COLUMNS = 64
LEAST = 2.0 ** -126


def values():
    """Every bf16 of size up to 128, filled up with zeros to rows of COLUMNS."""
    v = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    v = v[v.float().abs() <= 128.0]
    return torch.cat([v, v.new_zeros(-v.numel() % COLUMNS)]).view(-1, COLUMNS).contiguous()


def bounds(z, act):
    """Bounds of act(z) and its slope in fp32."""
    a, size = act64(z, act), z.abs()
    if act == "silu":
        s = torch.sigmoid(z)
        r = (2 * size + 8) * U
        ds = s * r + LEAST
        slope = ds * (1 + z * (1 - s)).abs() + s * size * (ds + U) + 3 * U * s * (1 + size * (1 - s))
        return a.abs() * (r + U) + size * LEAST + LEAST, slope + size * LEAST + LEAST
    t = 1.0 / (1.0 + 0.3275911 * size / math.sqrt(2.0))
    c = (0.254829592, -0.284496736, 1.421413741, -1.453152027, 1.061405429)
    e = torch.exp(-z * z / 2)
    p = sum(k * t ** (i + 1) for i, k in enumerate(c))
    terms = sum(abs(k) * t ** (i + 1) for i, k in enumerate(c))
    method = (e * p / 2 - torch.erfc(size / math.sqrt(2.0)) / 2).abs()
    de = e * (1.5 * z * z + 5) * U + LEAST
    dphi = method + 0.5 * (de * p.abs() + (e + de) * terms * 40 * U) + 2 * U * 0.5 * torch.erfc(-z / math.sqrt(2.0)) + LEAST
    density = 1.0 / math.sqrt(2.0 * math.pi)
    return size * dphi + U * a.abs() + LEAST, dphi + size * density * (de + 3 * U * e) + 2 * U * slope64(z, act).abs() + LEAST


def check(got, want, bound, z, what):
    off = (got.double() - want).abs()
    worst = int((off / bound).argmax())
    assert bool((off <= bound).all()), "%s: %.3g of the bound at z = %g" % (
        what, float((off / bound).flatten()[worst]), float(z.flatten()[worst]))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_every_pre_activation(act):
    from gpu_path import B
    z = values()
    E, N = z.shape
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    cnt = torch.ones(E, dtype=torch.int32, device="cuda")
    st = status()
    z64 = z.double()
    da, ds = bounds(z64, act)
    ws = torch.empty(B.ep_expert_gemm_backward_workspace_bytes(E, N, E, ACTS[act]), dtype=torch.uint8, device="cuda")
    dy, slope = torch.ones_like(z), torch.empty((E, N), device="cuda")
    B.ep_expert_gemm_backward(dy, None, None, z, off, cnt, ws, st, dbias=slope, activation=ACTS[act])
    check(slope, slope64(z64, act), ds, z64, "slope")
    a, column = torch.empty((E, N), device="cuda"), torch.empty(E, device="cuda")
    for n in range(N):
        dy.zero_()
        dy[:, n] = 1.0
        B.ep_expert_gemm_backward(dy, None, None, z, off, cnt, ws, st, d_row_weight=column, activation=ACTS[act])
        a[:, n] = column
    check(a, act64(z64, act), da, z64, "activation")
    # the product: one weight a feature, one row of ones in the first term
    x = torch.zeros((E, 8), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.0
    w = torch.zeros((E, N, 8), dtype=torch.bfloat16, device="cuda")
    w[:, :, 0] = z
    y, saved = torch.empty_like(z), torch.empty_like(z)
    B.ep_expert_gemm(x, w, off, cnt, y, st, activation=ACTS[act], z=saved)
    normal = z.abs() >= LEAST       # (the tensor cores take the subnormals their way)
    assert bool((saved == z)[normal].all())
    check(y[normal], act64(z64, act)[normal], bf16_bound(act64(z64, act), da)[normal], z64[normal], "y")
    assert int(st.item()) == 0
