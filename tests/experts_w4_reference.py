"""4-bit weights: how tests make them, what they stand for in 64 bits, and the
error bounds of the products with them (experts_reference's, with other weights).

The products of a group may be summed as (16 + u) x, with (16 + zero) times the
sum of x taken off afterwards, in fp32: a sum's error is then bounded with
(16 + u + 16 + |zero|) |scale| |x| in the place of |w x|.  FP4 codes are summed
as they are, or as multiples of a power of two.
"""
import torch

import experts_reference as plain

FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def make(g, E, rows, depth, group, form="int", zero=False, scales=torch.bfloat16, std=None):
    """Codes [E, rows, depth / 2], scales and zero points (or None) [E, depth / group, rows]."""
    codes = torch.randint(0, 256, (E, rows, depth // 2), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
    size = (std or depth ** -0.5) / (4.6 if form == "int" else 2.8)
    sf = ((torch.rand((E, depth // group, rows), generator=g, device="cuda") + 0.5) * size).to(scales)
    # scales of either sign, and zero points with a fraction
    sf = torch.where(torch.rand(sf.shape, generator=g, device="cuda") < 0.1, -sf, sf)
    z = (torch.rand(sf.shape, generator=g, device="cuda") * 15).to(scales) if zero else None
    return codes, sf, z


def values(codes, sf, zero, form):
    """(weights, bound weights) of one expert in 64 bits, [rows, depth]."""
    rows, half = codes.shape
    u = torch.stack([codes & 15, codes >> 4], -1).reshape(rows, 2 * half).long()
    group = 2 * half // sf.shape[0]
    s = sf.double().repeat_interleave(group, 0).T
    if form == "fp4":
        v = torch.tensor(FP4 + tuple(-a for a in FP4), dtype=torch.float64, device=codes.device)[u]
        return v * s, v.abs() * s.abs()
    z = 8.0 if zero is None else zero.double().repeat_interleave(group, 0).T
    return (u - z) * s, (32.0 + u + (z if zero is None else z.abs())) * s.abs()


def product_rows(x, w, big, bias, act, rw, res):
    """experts_reference.product_rows with the sum's error by `big`."""
    z = x @ w.T
    dz = (x.shape[1] + 16) * 2 * plain.U * (x.abs() @ big.T)
    if bias is not None:
        z = z + bias
        dz = dz + 2 * plain.U * z.abs()
    a, da = plain.activate(z, dz, act)
    if rw is not None:
        a, da = a * rw[:, None], da * rw.abs()[:, None] + plain.U * (a * rw[:, None]).abs()
    if res is not None:
        a = a + res
        da = da + 2 * plain.U * (a.abs() + res.abs())
    return a, plain.bf16_bound(a, da)


def few_tokens(x, idx, tw, up, b_up, act, down, b_down, res, form):
    """The whole layer: out and its bound; up and down are (codes, scales, zero points)."""
    T, K = idx.shape
    H = x.shape[1]
    out = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    err, big_out = torch.zeros_like(out), torch.zeros_like(out)

    def of(w, e):
        return values(w[0][e], w[1][e], None if w[2] is None else w[2][e], form)

    for e in torch.unique(idx).tolist():
        if e < 0 or e >= up[0].shape[0]:
            continue
        t, k = torch.nonzero(idx == e, as_tuple=True)
        w, big = of(up, e)
        h, dh = product_rows(x[t].double(), w, big, None if b_up is None else b_up[e].double(), act, None, None)
        w, big = of(down, e)
        p = h @ w.T
        dp = dh @ w.abs().T + (w.shape[1] + 16) * 2 * plain.U * ((h.abs() + dh) @ big.T)
        if b_down is not None:
            p = p + b_down[e].double()
            dp = dp + 2 * plain.U * p.abs()
        c = tw[t, k].double()[:, None]
        out.index_add_(0, t, c * p)
        err.index_add_(0, t, c.abs() * dp)
        big_out.index_add_(0, t, (c * p).abs() + c.abs() * dp)
    if res is not None:
        out = out + res.double()
        big_out = big_out + res.double().abs()
    return out, plain.bf16_bound(out, err + (K + 2) * 2 * plain.U * big_out)
