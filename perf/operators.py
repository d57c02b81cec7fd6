"""Cases that measure the experts' operators: what stands between dispatch and combine.

Three operators, each in a plain form of elementary torch operations and, where
``own`` is true, as a user of the library calls it:

* ``product``: the experts' matrix product over the expanded receive rows
  (expert e's rows are ``expert_offset[e] .. + num_tokens_per_expert[e]``)
  with bias, activation, row weight and residual in its epilogue, bf16 or FP8;
* ``backward``: its gradients for the rows, the weights, the bias and the row
  weights;
* ``few``: the whole mixture-of-experts layer (up product, activation, down
  product, weighted sum over each token's experts, residual) for a few tokens.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "silu", "swiglu")


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _product(name, T, E, K, H, N, act, fp8=False, bias=False, weight=False, residual=False, save=False,
             align=1, zipf=0.0, mask=0.0):
    return dict(name=name, op="product", T=T, E=E, K=K, H=H, N=N, act=act, fp8=fp8, bias=bias, weight=weight,
                residual=residual, save=save, align=align, zipf=zipf, mask=mask)


def _backward(name, T, E, K, H, N, act, bias=False, weight=False, align=1, zipf=0.0, mask=0.0):
    return dict(name=name, op="backward", T=T, E=E, K=K, H=H, N=N, act=act, bias=bias, weight=weight, align=align,
                zipf=zipf, mask=mask)


def _few(name, T, E, K, H, N, act, bias=False, residual=False, zipf=0.0, mask=0.0):
    return dict(name=name, op="few", T=T, E=E, K=K, H=H, N=N, act=act, bias=bias, residual=residual, zipf=zipf,
                mask=mask)


def listed():
    return [
        # the small parity workload's rows through one expert layer, everything in the epilogue: a call's latency
        _product("product_tiny", 128, 16, 4, 256, 512, "silu", bias=True, weight=True, residual=True),
        # the up product of a DeepSeek-V3-shaped prefill step: about 128 rows for each of 256 experts
        _product("product_up_prefill", 4096, 256, 8, 7168, 2048, "swiglu"),
        # the same rows kept for the backward pass, fewer and fuller experts: bound by the tensor cores
        _product("product_up_train", 4096, 32, 8, 7168, 2048, "swiglu", save=True, align=128),
        # a shared expert or an output projection: one group of rows, with bias, activation and residual
        _product("product_dense", 8192, 1, 1, 7168, 7168, "gelu", bias=True, residual=True),
        # FP8 rows as the dispatch leaves them, FP8 weights: the up product of fuller experts
        _product("product_fp8_up", 4096, 64, 8, 7168, 2048, "swiglu", fp8=True),
        # FP8 rows of a short step, down product with the top-k weight applied to each row
        _product("product_fp8_down", 512, 128, 8, 2048, 7168, "none", fp8=True, weight=True, align=16),
        # gradients on the small workload
        _backward("backward_tiny", 128, 16, 4, 256, 512, "silu", bias=True, weight=True),
        # a training step's gated up product, about 1024 rows for each expert
        _backward("backward_up_train", 4096, 32, 8, 7168, 2048, "swiglu", align=128),
        # odd widths, popular and empty experts, masked entries
        _backward("backward_skewed", 1001, 40, 5, 1000, 1352, "gelu", bias=True, weight=True, zipf=0.8, mask=0.05),
        # one token through the whole layer: only its eight experts' weights are read
        _few("few_one_token", 1, 256, 8, 7168, 2048, "swiglu"),
        # a small decode batch with odd routing: popular experts, masked entries, bias and residual
        _few("few_batch", 17, 256, 8, 7168, 2048, "swiglu", bias=True, residual=True, zipf=0.8, mask=0.05),
        # the decode workload: 128 tokens reach nearly every expert
        _few("few_decode", 128, 256, 8, 7168, 2048, "swiglu", residual=True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    while True:
        op = rng.choice(("product", "product", "backward", "few"))
        act = rng.choice(ACTS)
        fp8 = op == "product" and rng.random() < 0.35
        step = 128 if fp8 else 8
        E = _log_int(rng, 1, 256)
        K = rng.randint(1, min(8, E))
        T = _log_int(rng, 1, 256 if op == "few" else 8192)
        H = _log_int(rng, 128, 7168, step)
        N = _log_int(rng, 128, 7168, step)
        zipf = rng.choice((0.0, 0.0, 0.5, 0.8))
        mask = rng.choice((0.0, 0.05, 0.3))
        Nw = 2 * N if act == "swiglu" else N
        # no dearer than the largest listed ones: operations with the plain form's padding, weights, rows
        popular = 1.0 if zipf == 0.0 else min(8.0, E / 4.0 + 1.0)
        if T * K * H * Nw * popular > 9.0e11 or E * H * Nw > 4.0e9 or T * K * max(H, Nw) > 5.0e8:
            continue
        c = dict(op=op, T=T, E=E, K=K, H=H, N=N, act=act, zipf=zipf, mask=mask, bias=rng.random() < 0.5)
        if op == "few":
            c.update(residual=rng.random() < 0.5)
        else:
            c.update(weight=rng.random() < 0.5, align=rng.choice((1, 1, 16, 128)))
        if op == "product":
            c.update(fp8=fp8, residual=rng.random() < 0.4, save=rng.random() < 0.3)
        return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _route(c, gen):
    """Top-k experts of every token: distinct, uniform or by popularity ~ i^-zipf, some masked."""
    T, E, K = c["T"], c["E"], c["K"]
    dev = "cuda"
    keys = -torch.log(-torch.log(torch.rand((T, E), generator=gen, device=dev).clamp(1e-20, 1 - 1e-7)))
    if c["zipf"] > 0:
        order = torch.randperm(E, generator=gen, device=dev)
        keys = keys - c["zipf"] * torch.log(order.float() + 1.0)
    idx = torch.argsort(keys, dim=1, descending=True, stable=True)[:, :K].contiguous()
    if c["mask"] > 0:
        idx[torch.rand((T, K), generator=gen, device=dev) < c["mask"]] = -1
    weights = torch.softmax(torch.randn((T, K), generator=gen, device=dev), dim=1)
    return idx, weights


def _to_fp8(a, rows, cols):
    """Codes and fp32 scales of blocks of rows x cols, the largest of a block at 448."""
    lead, (n, k) = a.shape[:-2], a.shape[-2:]
    b = a.float().reshape(*lead, n // rows, rows, k // cols, cols)
    amax = b.abs().amax(dim=(-3, -1), keepdim=True).clamp_min(1e-12)
    codes = (b * (448.0 / amax)).to(torch.float8_e4m3fn).reshape(a.shape)
    return codes, (amax / 448.0).reshape(*lead, n // rows, k // cols).contiguous()


def _weights(gen, shape, fan_in, fp8):
    """bf16 weights N(0, 1/fan_in), or their FP8 codes with one scale for each 128 x 128 block."""
    if not fp8:
        w = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, fan_in ** -0.5, generator=gen)
        return w, None
    w = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    sf = torch.empty((shape[0], shape[1] // 128, shape[2] // 128), device="cuda")
    for e in range(shape[0]):
        one = torch.empty(shape[1:], device="cuda").normal_(0.0, fan_in ** -0.5, generator=gen)
        w[e], sf[e] = _to_fp8(one, 128, 128)
    return w, sf


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    E, H, N = c["E"], c["H"], c["N"]
    Nw = 2 * N if c["act"] == "swiglu" else N

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)

    idx, topw = _route(c, gen)
    s = dict(case=c, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if c["op"] == "few":
        s.update(x=normal(c["T"], H), topk_idx=idx, topk_weights=topw,
                 w_up=_weights(gen, (E, Nw, H), H, False)[0], w_down=_weights(gen, (E, H, N), N, False)[0],
                 bias_up=normal(E, Nw, dtype=torch.float32, std=0.1) if c["bias"] else None,
                 bias_down=normal(E, H, dtype=torch.float32, std=0.1) if c["bias"] else None,
                 residual=normal(c["T"], H) if c["residual"] else None,
                 out=torch.empty((c["T"], H), dtype=torch.bfloat16, device="cuda"))
        return s
    # the expanded receive rows: expert by expert, each block padded to the alignment
    flat = idx.reshape(-1)
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    align = c["align"]
    padded = (counts + align - 1) // align * align
    ends = torch.cumsum(padded, 0)
    starts = ends - padded
    rows = c["T"] * c["K"] + E * (align - 1)
    # plain form's view: row of every (expert, position), `rows` (a row of zeros) where there is none
    longest = max(1, int(counts.max()))
    pos = torch.arange(longest, device="cuda")
    table = torch.where(pos[None, :] < counts[:, None], starts[:, None] + pos[None, :], rows)
    s.update(rows=rows, table=table, num_tokens_per_expert=counts.to(torch.int32),
             expert_offset=torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), ends]).to(torch.int32))
    # rows of no expert hold what an earlier step left there
    x = normal(rows, H)
    s["row_weight"] = torch.rand(rows, generator=gen, device="cuda") if c["weight"] else None
    s["bias"] = normal(E, Nw, dtype=torch.float32, std=0.1) if c["bias"] else None
    if c["op"] == "product":
        s["w"], s["w_sf"] = _weights(gen, (E, Nw, H), H, c["fp8"])
        s["x"], s["x_sf"] = _to_fp8(x, 1, 128) if c["fp8"] else (x, None)
        s["residual"] = normal(rows, N) if c["residual"] else None
        # zero rows where no expert's row is: they are not written
        s["y"] = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
        s["z"] = torch.zeros((rows, Nw), dtype=torch.bfloat16, device="cuda") if c["save"] else None
        return s
    s["x"], (s["w"], _) = x, _weights(gen, (E, Nw, H), H, False)
    s["dy"], s["z"] = normal(rows, N), normal(rows, Nw)
    s["dx"] = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
    s["dw"] = torch.empty((E, Nw, H), dtype=torch.bfloat16, device="cuda")
    s["dbias"] = torch.empty((E, Nw), device="cuda") if c["bias"] else None
    s["d_row_weight"] = torch.zeros(rows, device="cuda") if c["weight"] else None
    return s


# --------------------------------------------------------------------------
# plain forms: 32 bits throughout, rounded once at the end
# --------------------------------------------------------------------------

def _act(z, act):
    if act == "relu":
        return torch.clamp_min(z, 0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "swiglu":
        gate, up = z.chunk(2, dim=-1)
        return gate / (1.0 + torch.exp(-gate)) * up
    return z


def _act_back(da, z, act):
    """Gradient of the pre-activation from the activation's."""
    if act == "relu":
        return da * (z > 0)
    if act == "gelu":
        return da * (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
                     + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-z))
        return da * sig * (1.0 + z * (1.0 - sig))
    if act == "swiglu":
        gate, up = z.chunk(2, dim=-1)
        sig = 1.0 / (1.0 + torch.exp(-gate))
        return torch.cat([da * up * sig * (1.0 + gate * (1.0 - sig)), da * gate * sig], dim=-1)
    return da


def _padded(a, s):
    """[E, longest, ...]: the rows of every expert, rows of zeros after its last."""
    return torch.cat([a.float(), torch.zeros_like(a[:1], dtype=torch.float32)])[s["table"]]


def _rows(a, s):
    """Back to the expanded rows; zeros where no expert's row is."""
    out = torch.zeros((s["rows"] + 1,) + a.shape[2:], device="cuda")
    out[s["table"].reshape(-1)] = a.reshape((-1,) + a.shape[2:])
    return out[:-1]


def _plain_product(s):
    c = s["case"]
    x, w = s["x"].float(), s["w"].float()
    if c["fp8"]:
        x = (x.reshape(s["rows"], -1, 128) * s["x_sf"][:, :, None]).reshape(s["rows"], -1)
        E, Nw, H = w.shape
        w = (w.reshape(E, Nw // 128, 128, H // 128, 128) * s["w_sf"][:, :, None, :, None]).reshape(E, Nw, H)
    z = torch.bmm(_padded(x, s), w.transpose(1, 2))
    if c["bias"]:
        z = z + s["bias"][:, None, :]
    y = _act(z, c["act"])
    if c["weight"]:
        y = y * _padded(s["row_weight"][:, None], s)
    if c["residual"]:
        y = y + _padded(s["residual"], s)
    out = {"y": _rows(y, s).to(torch.bfloat16)}
    if c["save"]:
        out["z"] = _rows(z, s).to(torch.bfloat16)
    return out


def _plain_backward(s):
    c = s["case"]
    dy, z, x = _padded(s["dy"], s), _padded(s["z"], s), _padded(s["x"], s)
    out = {}
    da = dy
    if c["weight"]:
        out["d_row_weight"] = _rows((dy * _act(z, c["act"])).sum(-1), s)
        da = dy * _padded(s["row_weight"][:, None], s)
    dz = _act_back(da, z, c["act"])
    out["dx"] = _rows(torch.bmm(dz, s["w"].float()), s).to(torch.bfloat16)
    out["dw"] = torch.bmm(dz.transpose(1, 2), x).to(torch.bfloat16)
    if c["bias"]:
        out["dbias"] = dz.sum(1)
    return out


def _plain_few(s):
    c = s["case"]
    T, K = s["topk_idx"].shape
    flat = s["topk_idx"].reshape(-1)
    entry = torch.nonzero(flat >= 0).reshape(-1)
    out = torch.zeros((T * K + 1, c["H"]), device="cuda")
    # entries in the order of their experts; each expert's in a row of a padded table
    active, group, counts = torch.unique(flat[entry], return_inverse=True, return_counts=True)
    if active.numel() > 0:
        order = torch.argsort(group, stable=True)
        entry, group = entry[order], group[order]
        place = torch.arange(entry.numel(), device="cuda") - (torch.cumsum(counts, 0) - counts)[group]
        table = torch.full((active.numel(), int(counts.max())), T * K, device="cuda", dtype=torch.int64)
        table[group, place] = entry
        xs = torch.cat([s["x"].float(), torch.zeros((1, c["H"]), device="cuda")])[
            torch.where(table < T * K, table // K, T)]
        z = torch.bmm(xs, s["w_up"][active].float().transpose(1, 2))
        if c["bias"]:
            z = z + s["bias_up"][active][:, None, :]
        p = torch.bmm(_act(z, c["act"]), s["w_down"][active].float().transpose(1, 2))
        if c["bias"]:
            p = p + s["bias_down"][active][:, None, :]
        out[table.reshape(-1)] = p.reshape(-1, c["H"])
    y = (out[:-1].reshape(T, K, -1) * s["topk_weights"][:, :, None] * (s["topk_idx"] >= 0)[:, :, None]).sum(1)
    if c["residual"]:
        y = y + s["residual"].float()
    return {"out": y.to(torch.bfloat16)}


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------

def _own(s):
    import combine_ep_get_gb300 as ep
    c = s["case"]
    act = {"none": ep.EP_ACT_NONE, "relu": ep.EP_ACT_RELU, "gelu": ep.EP_ACT_GELU, "silu": ep.EP_ACT_SILU,
           "swiglu": ep.EP_ACT_SWIGLU}[c["act"]]
    if c["op"] == "product":
        ep.ep_expert_gemm(s["x"], s["w"], s["expert_offset"], s["num_tokens_per_expert"], s["y"], s["status"],
                          bias=s["bias"], activation=act, row_weight=s["row_weight"], residual=s["residual"],
                          z=s["z"], x_sf=s["x_sf"], w_sf=s["w_sf"])
        return {"y": s["y"], "z": s["z"]} if c["save"] else {"y": s["y"]}
    if c["op"] == "backward":
        if "workspace" not in s:
            s["workspace"] = torch.empty(ep.ep_expert_gemm_backward_workspace_bytes(s["rows"], c["N"], c["E"], act),
                                         dtype=torch.uint8, device="cuda")
        ep.ep_expert_gemm_backward(s["dy"], s["x"], s["w"], s["z"], s["expert_offset"], s["num_tokens_per_expert"],
                                   s["workspace"], s["status"], dx=s["dx"], dw=s["dw"], dbias=s["dbias"],
                                   d_row_weight=s["d_row_weight"], activation=act, row_weight=s["row_weight"])
        out = {"dx": s["dx"], "dw": s["dw"]}
        if c["weight"]:
            out["d_row_weight"] = s["d_row_weight"]
        if c["bias"]:
            out["dbias"] = s["dbias"]
        return out
    if "workspace" not in s:
        s["workspace"] = torch.empty(ep.ep_moe_few_tokens_workspace_bytes(c["T"], c["K"], c["H"], c["N"], c["E"]),
                                     dtype=torch.uint8, device="cuda")
    ep.ep_moe_few_tokens(s["x"], s["topk_idx"], s["topk_weights"], s["w_up"], s["w_down"], s["workspace"], s["out"],
                         s["status"], bias_up=s["bias_up"], bias_down=s["bias_down"], residual=s["residual"],
                         activation=act)
    return {"out": s["out"]}


def run(state):
    if own:
        return _own(state)
    return {"product": _plain_product, "backward": _plain_backward, "few": _plain_few}[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c = case
    T, E, K, H, N = c["T"], c["E"], c["K"], c["H"], c["N"]
    Nw = 2 * N if c["act"] == "swiglu" else N
    rows = T * K * (1.0 - c["mask"])
    # experts that some token names, as if uniform (popularity leaves a few more out)
    active = E * (1.0 - (1.0 - rows / T / E) ** T)
    if c["op"] == "few":
        size = 2.0 * active * (Nw * H + H * N) + 2.0 * T * H * (3 if c["residual"] else 2) + T * K * 12.0
        if c["bias"]:
            size += 4.0 * active * (Nw + H)
        return {"bytes": size, "flops": 2.0 * rows * (Nw * H + H * N)}
    if c["op"] == "product":
        item = 1 if c["fp8"] else 2
        size = item * (rows * H + active * Nw * H) + 2.0 * rows * N
        if c["fp8"]:
            size += 4.0 * (rows * (H // 128) + active * (Nw // 128) * (H // 128))
        size += 2.0 * rows * N * c["residual"] + 2.0 * rows * Nw * c["save"]
        size += 4.0 * rows * c["weight"] + 4.0 * active * Nw * c["bias"]
        return {"bytes": size, "flops": 2.0 * rows * Nw * H}
    size = 2.0 * (2 * rows * H + rows * N + rows * Nw + active * Nw * H + E * Nw * H)
    size += 8.0 * rows * c["weight"] + 4.0 * E * Nw * c["bias"]
    return {"bytes": size, "flops": 4.0 * rows * Nw * H}


# --------------------------------------------------------------------------
# the definitions in 64 bits, expert by expert
# --------------------------------------------------------------------------

def _act64(z, act):
    """The activation and its derivative (two of them for the gated one: by the gate and by the other half)."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z)), (z > 0).double()
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    if act == "silu":
        sig = torch.sigmoid(z)
        return z * sig, sig + z * sig * (1.0 - sig)
    half = z.shape[-1] // 2
    gate, up = z[..., :half], z[..., half:]
    sig = torch.sigmoid(gate)
    return gate * sig * up, torch.cat([up * (sig + gate * sig * (1.0 - sig)), gate * sig], -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "few":
        out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
        for e in torch.unique(s["topk_idx"]).tolist():
            if e < 0:
                continue
            t, k = torch.nonzero(s["topk_idx"] == e, as_tuple=True)
            z = s["x"][t].double() @ s["w_up"][e].double().T
            if c["bias"]:
                z = z + s["bias_up"][e].double()
            p = _act64(z, c["act"])[0] @ s["w_down"][e].double().T
            if c["bias"]:
                p = p + s["bias_down"][e].double()
            out.index_add_(0, t, p * s["topk_weights"][t, k].double()[:, None])
        if c["residual"]:
            out += s["residual"].double()
        return {"out": out}
    first, count = s["expert_offset"].tolist(), s["num_tokens_per_expert"].tolist()
    rows, E, H, N = s["rows"], c["E"], c["H"], c["N"]
    Nw = s["w"].shape[1]

    def empty(*shape):
        return torch.zeros(shape, dtype=torch.float64, device="cuda")

    if c["op"] == "product":
        out = {"y": empty(rows, N)}
        if c["save"]:
            out["z"] = empty(rows, Nw)
        for e in range(E):
            r = slice(first[e], first[e] + count[e])
            x, w = s["x"][r].double(), s["w"][e].double()
            if c["fp8"]:
                x = x * s["x_sf"][r].double().repeat_interleave(128, 1)
                w = w * s["w_sf"][e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
            z = x @ w.T
            if c["bias"]:
                z = z + s["bias"][e].double()
            y = _act64(z, c["act"])[0]
            if c["weight"]:
                y = y * s["row_weight"][r].double()[:, None]
            if c["residual"]:
                y = y + s["residual"][r].double()
            out["y"][r] = y
            if c["save"]:
                out["z"][r] = z
        return out
    out = {"dx": empty(rows, H), "dw": empty(E, Nw, H)}
    if c["weight"]:
        out["d_row_weight"] = empty(rows)
    if c["bias"]:
        out["dbias"] = empty(E, Nw)
    for e in range(E):
        r = slice(first[e], first[e] + count[e])
        a, slope = _act64(s["z"][r].double(), c["act"])
        da = dy = s["dy"][r].double()
        if c["weight"]:
            out["d_row_weight"][r] = (dy * a).sum(1)
            da = dy * s["row_weight"][r].double()[:, None]
        dz = slope * (torch.cat([da, da], 1) if c["act"] == "swiglu" else da)
        out["dx"][r] = dz @ s["w"][e].double()
        out["dw"][e] = dz.T @ s["x"][r].double()
        if c["bias"]:
            out["dbias"][e] = dz.sum(0)
    return out
