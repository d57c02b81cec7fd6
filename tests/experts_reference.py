"""The experts' operators from their definitions in 64 bits, expert by expert,
and elementwise error bounds of a computation that accumulates in fp32.

Bounds.  u = 2^-24.  A sum of n products of bf16 (or scaled E4M3) values in
fp32, in any order, each addition rounded or truncated, is off by at most
2 n u sum |a b| to first order; (n + 16) * 2^-23 is taken, which leaves room for the
bias and the scales.  An error dz of a pre-activation moves relu by at most
dz and gelu and silu by at most 1.13 dz (their largest slopes are 1.129 and
1.0998); their second derivatives are at most 0.8 (gelu 0.798, silu 0.5).
The functions themselves (exp, erf, a division) are good to 16 u of their
result plus, where 1 + erf cancels, 4 u of z.  bf16 keeps 8
significant bits: a rounding to nearest is off by at most half a unit of the
last, 2^-8 of the value, or half the least subnormal, 2^-134.
"""
import math

import torch

U = 2.0 ** -24
BF = 2.0 ** -8
TINY = 2.0 ** -134
ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3, "swiglu": 4}
SLOPE = 1.13


def act64(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    return torch.ones_like(z)


def act_error(z, dz, act):
    """Bound of the activation's error where z is off by dz."""
    if act in ("none", "relu"):
        return dz
    return SLOPE * dz + 16 * U * act64(z, act).abs() + 4 * U * z.abs()


def activate(z, dz, act):
    """(a, bound) from the pre-activation and its bound; swiglu takes both halves."""
    if act != "swiglu":
        return act64(z, act), act_error(z, dz, act)
    n = z.shape[-1] // 2
    g, up, dg, du = z[..., :n], z[..., n:], dz[..., :n], dz[..., n:]
    s, ds = act64(g, "silu"), act_error(g, dg, "silu")
    return s * up, ds * up.abs() + s.abs() * du + ds * du + 2 * U * (s * up).abs()


def bf16_bound(v, dv):
    """Bound after rounding a value v known to dv."""
    return dv + BF * (v.abs() + dv) + TINY


def product_rows(x, w, bias, act, rw, res):
    """One expert's rows (64-bit x [m, K], w [Nw, K]): y, z and their bounds, rounded to bf16."""
    z = x @ w.T
    dz = (x.shape[1] + 16) * 2 * U * (x.abs() @ w.abs().T)
    if bias is not None:
        z = z + bias
        dz = dz + 2 * U * z.abs()
    a, da = activate(z, dz, act)
    if rw is not None:
        a, da = a * rw[:, None], da * rw.abs()[:, None] + U * (a * rw[:, None]).abs()
    if res is not None:
        a = a + res
        da = da + 2 * U * (a.abs() + res.abs())
    return a, bf16_bound(a, da), z, bf16_bound(z, dz)


def backward_rows(dy, x, w, z, act, rw):
    """One expert's gradients and bounds: dict of (value, bound)."""
    m, n = dy.shape
    da = dy if rw is None else dy * rw[:, None]
    if act == "swiglu":
        g, up = z[:, :n], z[:, n:]
        a = act64(g, "silu") * up
        dz = torch.cat([da * up * slope64(g, "silu"), da * act64(g, "silu")], 1)
        # the slope is a sum of two terms that may cancel: 32 u of their sizes
        big = torch.cat([(da * up).abs() * (1 + g.abs()), (da * act64(g, "silu")).abs()], 1)
    elif z is None:
        a, dz, big = None, da, da.abs()
    else:
        a = act64(z, act)
        dz = da * slope64(z, act)
        big = da.abs() if act in ("none", "relu") else da.abs() * (1 + z.abs())
    e_dz = 32 * U * big
    r_dz = bf16_bound(dz, e_dz)          # rounded for the products
    nw = dz.shape[1]
    out = {}
    dx = dz @ w
    out["dx"] = (dx, bf16_bound(dx, (r_dz + (nw + 16) * 2 * U * (dz.abs() + r_dz)) @ w.abs()))
    dw = dz.T @ x
    out["dw"] = (dw, bf16_bound(dw, (r_dz + (m + 16) * 2 * U * (dz.abs() + r_dz)).T @ x.abs()))
    out["dbias"] = (dz.sum(0), (e_dz + (m + 16) * 2 * U * dz.abs()).sum(0))
    if a is not None:
        big_a = (dy * a).abs() + dy.abs() * (z if act != "swiglu" else z[:, :n] * z[:, n:]).abs()
        out["d_row_weight"] = ((dy * a).sum(1), ((n + 48) * 2 * U * big_a).sum(1))
    return out


def few_tokens(x, idx, tw, w_up, b_up, act, w_down, b_down, res):
    """The whole layer for the given tensors: out and its bound."""
    T, K = idx.shape
    H = x.shape[1]
    out = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    err = torch.zeros_like(out)
    big = torch.zeros_like(out)
    for e in torch.unique(idx).tolist():
        if e < 0 or e >= w_up.shape[0]:
            continue
        t, k = torch.nonzero(idx == e, as_tuple=True)
        xe, wu, wd = x[t].double(), w_up[e].double(), w_down[e].double()
        h, dh, _, _ = product_rows(xe, wu, None if b_up is None else b_up[e].double(), act, None, None)
        p = h @ wd.T
        dp = dh @ wd.abs().T + (wd.shape[1] + 16) * 2 * U * ((h.abs() + dh) @ wd.abs().T)
        if b_down is not None:
            p = p + b_down[e].double()
            dp = dp + 2 * U * p.abs()
        c = tw[t, k].double()[:, None]
        out.index_add_(0, t, c * p)
        err.index_add_(0, t, c.abs() * dp)
        big.index_add_(0, t, (c * p).abs() + c.abs() * dp)
    if res is not None:
        out = out + res.double()
        big = big + res.double().abs()
    return out, bf16_bound(out, err + (K + 2) * 2 * U * big)


def check(got, want, bound, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), what + ": not finite"
    off = (got - want).abs()
    bad = off > bound
    assert not bool(bad.any()), "%s: %d beyond the bound, one by %.3g times" % (
        what, int(bad.sum()), float((off / bound)[bad].max()))
