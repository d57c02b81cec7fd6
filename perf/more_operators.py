"""Cases that measure the operators around the experts' products: the router and
its balance loss, with their gradients, and the experts with 4-bit weights.

Five operators, each in a plain form of elementary torch operations and, where
``own`` is true, as a user of the library calls it:

* ``route``: each token's top-k experts and their weights from the router's
  logits (softmax or sigmoid scores, selection bias, group-limited choice);
* ``balance``: the balance loss of each sequence, per-expert counts and the
  loss's derivative by the scores;
* ``route_backward``: the gradient of the logits, through the weights of the
  chosen experts and through the balance loss;
* ``product4``: the experts' matrix product over the expanded receive rows with
  4-bit weights and group scales (one expert of one row is a matrix-vector
  product);
* ``few4``: the whole mixture-of-experts layer for a few tokens with 4-bit
  weights.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "silu", "swiglu")
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _route(name, T, E, K, score, dtype="fp32", bias=False, groups=1, topk_groups=1, normalize=True, scale=1.0, pad=0,
           mask=0.0):
    return dict(name=name, op="route", T=T, E=E, K=K, score=score, dtype=dtype, bias=bias, groups=groups,
                topk_groups=topk_groups, normalize=normalize, scale=scale, pad=pad, mask=mask)


def _balance(name, T, E, K, score, dtype="fp32", sequences=1, pad=0, mask=0.0):
    return dict(name=name, op="balance", T=T, E=E, K=K, score=score, dtype=dtype, sequences=sequences, pad=pad, mask=mask)


def _backward(name, T, E, K, score, dtype="fp32", sequences=1, normalize=True, scale=1.0, parts="both", pad=0, mask=0.0):
    return dict(name=name, op="route_backward", T=T, E=E, K=K, score=score, dtype=dtype, sequences=sequences,
                normalize=normalize, scale=scale, parts=parts, pad=pad, mask=mask)


def _product4(name, T, E, K, H, N, act, form="int", zero=False, group=128, scales="bf16", bias=False, weight=False,
              residual=False, align=1, zipf=0.0, mask=0.0):
    return dict(name=name, op="product4", T=T, E=E, K=K, H=H, N=N, act=act, form=form, zero=zero, group=group,
                scales=scales, bias=bias, weight=weight, residual=residual, align=align, zipf=zipf, mask=mask)


def _few4(name, T, E, K, H, N, act, form="int", zero=False, group=128, scales="bf16", bias=False, residual=False,
          zipf=0.0, mask=0.0):
    return dict(name=name, op="few4", T=T, E=E, K=K, H=H, N=N, act=act, form=form, zero=zero, group=group,
                scales=scales, bias=bias, residual=residual, zipf=zipf, mask=mask)


def listed():
    return [
        # the decode workload's router: 128 tokens, sigmoid scores with the bias of loss-free balancing, 4 of 8 groups
        _route("route_decode", 128, 256, 8, "sigmoid", bias=True, groups=8, topk_groups=4, scale=2.5),
        # the large workload's router, softmax over 256 experts
        _route("route_large", 32768, 256, 8, "softmax"),
        # a training step's loss, sequence by sequence, over ragged sequences with padding tokens
        _balance("balance_sequences", 4096, 256, 8, "sigmoid", sequences=5, mask=0.05),
        # the large workload's loss over the whole batch
        _balance("balance_large", 32768, 256, 8, "softmax", dtype="bf16"),
        # the same training step's gradient, through the weights and the loss
        _backward("route_backward_sequences", 4096, 256, 8, "sigmoid", sequences=5, scale=2.5, mask=0.05),
        # the large workload's gradient, an odd row of logits
        _backward("route_backward_large", 32768, 256, 8, "softmax", pad=1),
        # one token through an output projection or a shared expert: a plain matrix-vector product
        _product4("product4_vector", 1, 1, 1, 7168, 7168, "none", bias=True, residual=True),
        # the up product of a decode step after the dispatch: about four rows for each of 256 experts
        _product4("product4_up_decode", 128, 256, 8, 7168, 2048, "swiglu"),
        # the down product of the same step in the FP4 type with small groups, row weights applied
        _product4("product4_down_fp4", 128, 256, 8, 2048, 7168, "none", form="fp4", group=32, weight=True, align=16),
        # one token through the whole layer: its eight experts' weights are read
        _few4("few4_one_token", 1, 256, 8, 7168, 2048, "swiglu"),
        # a small decode batch with odd routing, zero points, fp32 scales of small groups, bias and residual
        _few4("few4_batch", 17, 256, 8, 7168, 2048, "swiglu", zero=True, group=64, scales="fp32", bias=True,
              residual=True, zipf=0.8, mask=0.05),
        # the decode workload: 128 tokens reach nearly every expert
        _few4("few4_decode", 128, 256, 8, 7168, 2048, "swiglu", residual=True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    while True:
        op = rng.choice(("route", "balance", "route_backward", "product4", "few4"))
        if op in ("route", "balance", "route_backward"):
            E = _log_int(rng, 2, 1024)
            K = rng.randint(1, min(16, E))
            T = _log_int(rng, 1, 32768)
            if T * E > 32768 * 256:
                continue
            c = dict(op=op, T=T, E=E, K=K, score=rng.choice(("softmax", "sigmoid")), dtype=rng.choice(tuple(TYPES)),
                     pad=rng.choice((0, 0, 1, 8)), mask=rng.choice((0.0, 0.05, 0.3)))
            if op == "route":
                groups = rng.choice([g for g in (1, 1, 2, 4, 8, 16) if E % g == 0])
                least = -(-K // (E // groups))
                c.update(bias=rng.random() < 0.5, groups=groups, topk_groups=rng.randint(least, groups))
            else:
                c.update(sequences=_log_int(rng, 1, min(64, T)))
            if op != "balance":
                c.update(normalize=rng.random() < 0.6, scale=rng.choice((1.0, 2.5)))
            if op == "route_backward":
                c.update(parts=rng.choice(("both", "both", "weights", "loss")))
            return c
        act, form = rng.choice(ACTS), rng.choice(("int", "int", "fp4"))
        group = rng.choice((32, 64, 128, 128))
        E = _log_int(rng, 1, 256)
        K = rng.randint(1, min(8, E))
        T = _log_int(rng, 1, 256)
        H = _log_int(rng, 128, 7168, group)
        N = _log_int(rng, 128, 7168, group if op == "few4" else 8)
        zipf, mask = rng.choice((0.0, 0.0, 0.5, 0.8)), rng.choice((0.0, 0.05, 0.3))
        Nw = 2 * N if act == "swiglu" else N
        # no dearer than the largest listed one: weights, operations with the plain form's padding
        popular = 1.0 if zipf == 0.0 else min(8.0, E / 4.0 + 1.0)
        if E * H * Nw > 4.0e9 or T * K * H * Nw * popular > 1.0e11:
            continue
        c = dict(op=op, T=T, E=E, K=K, H=H, N=N, act=act, form=form, zero=form == "int" and rng.random() < 0.4,
                 group=group, scales=rng.choice(("bf16", "fp32")), bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                 zipf=zipf, mask=mask)
        if op == "product4":
            c.update(weight=rng.random() < 0.5, align=rng.choice((1, 1, 16)))
        return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # by the low three bits; the fourth is the sign


def _choose(idx_keys, K):
    """Indices of the K largest keys of each row, equal ones by the lower index."""
    return torch.sort(idx_keys, dim=1, descending=True, stable=True).indices[:, :K].contiguous()


def _experts_of(c, gen):
    """Top-k experts of every token: distinct, uniform or by popularity ~ i^-zipf, some masked."""
    T, E, K = c["T"], c["E"], c["K"]
    keys = -torch.log(-torch.log(torch.rand((T, E), generator=gen, device="cuda").clamp(1e-20, 1 - 1e-7)))
    if c["zipf"] > 0:
        order = torch.randperm(E, generator=gen, device="cuda")
        keys = keys - c["zipf"] * torch.log(order.float() + 1.0)
    idx = _choose(keys, K)
    if c["mask"] > 0:
        idx[torch.rand((T, K), generator=gen, device="cuda") < c["mask"]] = -1
    return idx, torch.softmax(torch.randn((T, K), generator=gen, device="cuda"), dim=1)


def _quantized(c, gen, E, rows, depth):
    """4-bit codes [E, rows, depth / 2] of weights N(0, 1 / depth), two to a byte, the earlier in the low half; scales
    (and zero points) [E, depth / group, rows]."""
    g, dt = c["group"], TYPES[c["scales"]]
    codes = torch.empty((E, rows, depth // 2), dtype=torch.uint8, device="cuda")
    sf = torch.empty((E, depth // g, rows), dtype=dt, device="cuda")
    zero = torch.empty_like(sf) if c["zero"] else None
    middle = torch.tensor([(a + b) / 2 for a, b in zip(FP4, FP4[1:])], device="cuda")
    for e in range(E):
        w = torch.empty((rows, depth // g, g), device="cuda").normal_(0.0, depth ** -0.5, generator=gen)
        if c["form"] == "fp4":
            s = (w.abs().amax(-1) / 6.0).clamp_min(1e-8).to(dt)
            v = w / s.float()[..., None]
            u = torch.bucketize(v.abs(), middle) + 8 * (v < 0)
        elif c["zero"]:
            lo, hi = w.amin(-1), w.amax(-1)
            s = ((hi - lo) / 15.0).clamp_min(1e-8).to(dt)
            z = torch.round(-lo / s.float()).clamp(0, 15).to(dt)
            u = (torch.round(w / s.float()[..., None]) + z.float()[..., None]).clamp(0, 15)
            zero[e] = z.T
        else:
            s = (w.abs().amax(-1) / 7.0).clamp_min(1e-8).to(dt)
            u = (torch.round(w / s.float()[..., None]) + 8).clamp(0, 15)
        sf[e] = s.T
        u = u.to(torch.uint8).reshape(rows, depth // 2, 2)
        codes[e] = u[..., 0] | (u[..., 1] << 4)
    return codes, sf, zero


def _sequences(c, rng):
    """Offsets of ragged sequences, an empty one among several; some tokens behind the last."""
    T, S = c["T"], c["sequences"]
    if S == 1:
        return None
    cuts = torch.rand(S - 1, generator=rng, device="cuda").sort().values
    ends = torch.cat([(cuts * T).to(torch.int32), torch.tensor([T - T // 50], dtype=torch.int32, device="cuda")])
    if S > 2:
        ends[S // 2] = ends[S // 2 - 1]
    ends = torch.cummax(ends.clamp(max=T - T // 50), 0).values.to(torch.int32)
    return torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), ends])


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)

    s = dict(case=c, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if c["op"] in ("route", "balance", "route_backward"):
        T, E, K = c["T"], c["E"], c["K"]
        # some experts are liked by every token; the logits are columns of a wider matrix where pad > 0
        logits = normal(T, E + c["pad"], dtype=torch.float32, std=1.2) + normal(E + c["pad"], dtype=torch.float32, std=0.6)
        s["logits"] = logits.to(TYPES[c["dtype"]])[:, :E]
        s["token_mask"] = (torch.rand(T, generator=gen, device="cuda") >= c["mask"]) if c["mask"] > 0 else None
        if c["op"] == "route":
            # steps of 0.001 up or down, as loss-free balancing makes them
            s["bias"] = torch.round(normal(E, dtype=torch.float32, std=40.0)) * 0.001 if c["bias"] else None
            s["topk_idx"] = torch.empty((T, K), dtype=torch.int64, device="cuda")
            s["topk_weights"] = torch.empty((T, K), device="cuda")
            return s
        s["topk_idx"] = _choose(s["logits"].float(), K)
        if s["token_mask"] is not None:
            s["topk_idx"][~s["token_mask"]] = -1
        s["seq_offset"] = _sequences(c, gen)
        S = c["sequences"]
        if c["op"] == "balance":
            s.update(loss=torch.empty(1, device="cuda"), load=torch.empty((S, E), device="cuda"),
                     counts=torch.empty((S, E), dtype=torch.int32, device="cuda"))
            return s
        # the derivative of the loss by the scores as the forward call leaves it: positive, about coeff / tokens
        s["load"] = torch.rand((S, E), generator=gen, device="cuda") * (2.0 / T) if c["parts"] != "weights" else None
        s["d_loss"] = torch.rand(1, generator=gen, device="cuda") + 0.5 if c["parts"] != "weights" else None
        s["d_topk_weights"] = normal(T, K, dtype=torch.float32, std=1.0 / T) if c["parts"] != "loss" else None
        s["d_logits"] = torch.empty((T, E), dtype=s["logits"].dtype, device="cuda")
        return s
    E, H, N = c["E"], c["H"], c["N"]
    Nw = 2 * N if c["act"] == "swiglu" else N
    idx, topw = _experts_of(c, gen)
    if c["op"] == "few4":
        s["w_up"], s["up_sf"], s["up_zero"] = _quantized(c, gen, E, Nw, H)
        s["w_down"], s["down_sf"], s["down_zero"] = _quantized(c, gen, E, H, N)
        s.update(x=normal(c["T"], H), topk_idx=idx, topk_weights=topw,
                 bias_up=normal(E, Nw, dtype=torch.float32, std=0.1) if c["bias"] else None,
                 bias_down=normal(E, H, dtype=torch.float32, std=0.1) if c["bias"] else None,
                 residual=normal(c["T"], H) if c["residual"] else None,
                 out=torch.empty((c["T"], H), dtype=torch.bfloat16, device="cuda"))
        return s
    # the expanded receive rows: expert by expert, each block padded to the alignment
    flat = idx.reshape(-1)
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    padded = (counts + c["align"] - 1) // c["align"] * c["align"]
    ends = torch.cumsum(padded, 0)
    starts = ends - padded
    rows = c["T"] * c["K"] + E * (c["align"] - 1)
    pos = torch.arange(max(1, int(counts.max())), device="cuda")
    # plain form's view: row of every (expert, position), `rows` (a row of zeros) where there is none
    table = torch.where(pos[None, :] < counts[:, None], starts[:, None] + pos[None, :], rows)
    s["w"], s["w_sf"], s["w_zero"] = _quantized(c, gen, E, Nw, H)
    s.update(rows=rows, table=table, num_tokens_per_expert=counts.to(torch.int32),
             expert_offset=torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), ends]).to(torch.int32),
             x=normal(rows, H), bias=normal(E, Nw, dtype=torch.float32, std=0.1) if c["bias"] else None,
             row_weight=torch.rand(rows, generator=gen, device="cuda") if c["weight"] else None,
             residual=normal(rows, N) if c["residual"] else None,
             # zero rows where no expert's row is: they are not written
             y=torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda"))
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _scores(l, score):
    """Scores and their normalised form (the same for softmax)."""
    if score == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
        return p, p
    s = 1.0 / (1.0 + torch.exp(-l))
    return s, s / s.sum(1, keepdim=True)


def _plain_route(s):
    c = s["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    l = s["logits"].float()
    score = _scores(l, c["score"])[0]
    if s["bias"] is None and G == 1:
        key = l                     # scores rise with logits
    else:                           # in 64 bits: choices next to a border
        key = _scores(l.double(), c["score"])[0]
        if s["bias"] is not None:
            key = key + s["bias"].double()
    if c["topk_groups"] < G:
        best = torch.sort(key.reshape(T, G, E // G), dim=2, descending=True).values[:, :, :2].sum(2)
        keep = torch.zeros((T, G), dtype=torch.bool, device="cuda")
        keep.scatter_(1, _choose(best, c["topk_groups"]), True)
        key = torch.where(keep.repeat_interleave(E // G, 1), key, -math.inf)
    idx = _choose(key, K)
    w = score.gather(1, idx)
    if c["normalize"]:
        w = w / w.sum(1, keepdim=True)
    w = w * c["scale"]
    if s["token_mask"] is not None:
        idx = torch.where(s["token_mask"][:, None], idx, -1)
        w = torch.where(s["token_mask"][:, None], w, 0.0)
    return {"topk_idx": idx, "topk_weights": w}


def _sequence_of(s):
    """Sequence of every token, S for those behind the last one or masked."""
    c = s["case"]
    if s["seq_offset"] is None:
        q = torch.zeros(c["T"], dtype=torch.int64, device="cuda")
    else:
        at = torch.arange(c["T"], device="cuda")
        q = (at[:, None] >= s["seq_offset"][None, 1:]).sum(1)
    if s["token_mask"] is not None:
        q = torch.where(s["token_mask"], q, c["sequences"])
    return q


def _plain_balance(s):
    c = s["case"]
    E, K, S = c["E"], c["K"], c["sequences"]
    q = _sequence_of(s)
    p = _scores(s["logits"].float(), c["score"])[1]
    # sums over up to 32768 tokens in 64 bits
    total = torch.zeros((S + 1, E), dtype=torch.float64, device="cuda").index_add_(0, q, p.double())[:S]
    n = torch.zeros(S + 1, dtype=torch.int64, device="cuda").index_add_(0, q, torch.ones_like(q))[:S]
    counts = torch.zeros((S + 1) * (E + 1), dtype=torch.int64, device="cuda")
    at = q[:, None] * (E + 1) + torch.where(s["topk_idx"] >= 0, s["topk_idx"], E)
    counts.index_add_(0, at.reshape(-1), torch.ones_like(at).reshape(-1))
    counts = counts.reshape(S + 1, E + 1)[:S, :E]
    n = n.clamp_min(1).double()[:, None]
    load = counts.double() * (COEFF * E / (S * K)) / (n * n)
    return {"loss": (load * total).sum().float().reshape(1), "load": load.float(),
            "num_tokens_per_expert": counts.to(torch.int32)}


COEFF = 0.01


def _plain_backward(s):
    c = s["case"]
    T, E, K = c["T"], c["E"], c["K"]
    l = s["logits"].float()
    score, p = _scores(l, c["score"])
    through = torch.zeros((T, E + 1), device="cuda")     # derivative by the scores, from the weights
    if s["d_topk_weights"] is not None:
        there = s["topk_idx"] >= 0
        g = torch.where(there, s["d_topk_weights"], 0.0) * c["scale"]
        if c["normalize"]:
            chosen = torch.where(there, score.gather(1, s["topk_idx"].clamp_min(0)), 0.0)
            d = chosen.sum(1, keepdim=True).clamp_min(1e-30)
            g = torch.where(there, (g - (g * chosen).sum(1, keepdim=True) / d) / d, 0.0)
        through.scatter_add_(1, torch.where(there, s["topk_idx"], E), g)
    through = through[:, :E]
    share = torch.zeros((T, E), device="cuda")           # derivative by the normalised scores, from the loss
    if s["load"] is not None:
        rows = torch.cat([s["load"], torch.zeros((1, E), device="cuda")])
        share = rows[_sequence_of(s)] * s["d_loss"]
    if c["score"] == "softmax":
        a = through + share
        d = p * (a - (a * p).sum(1, keepdim=True))
    else:
        d = (1.0 - score) * (score * through + p * (share - (share * p).sum(1, keepdim=True)))
    if s["token_mask"] is not None:
        d = torch.where(s["token_mask"][:, None], d, 0.0)
    return {"d_logits": d.to(s["logits"].dtype)}


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


def _weights(c, codes, sf, zero, dtype=torch.float32):
    """Weights [.., rows, depth] from codes, scales and zero points."""
    u = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], codes.shape[-1] * 2)
    u = u.reshape(*u.shape[:-1], -1, c["group"])
    if c["form"] == "fp4":
        v = torch.tensor(FP4 + tuple(-a for a in FP4), dtype=dtype, device="cuda")[u.int()]
    elif zero is not None:
        v = u.to(dtype) - zero.transpose(-1, -2).to(dtype)[..., None]
    else:
        v = u.to(dtype) - 8.0
    v = v * sf.transpose(-1, -2).to(dtype)[..., None]
    return v.reshape(*v.shape[:-2], -1)


AT_ONCE = 16     # experts whose weights the plain forms hold in 32 bits at a time


def _plain_product4(s):
    c = s["case"]
    x = torch.cat([s["x"].float(), torch.zeros((1, c["H"]), device="cuda")])
    out = torch.zeros((s["rows"] + 1, c["N"]), device="cuda")
    weight = torch.cat([s["row_weight"], torch.zeros(1, device="cuda")]) if c["weight"] else None
    residual = torch.cat([s["residual"].float(), torch.zeros((1, c["N"]), device="cuda")]) if c["residual"] else None
    for e in range(0, c["E"], AT_ONCE):
        part = slice(e, e + AT_ONCE)
        table = s["table"][part]
        w = _weights(c, s["w"][part], s["w_sf"][part], s["w_zero"][part] if c["zero"] else None)
        z = torch.bmm(x[table], w.transpose(1, 2))
        if c["bias"]:
            z = z + s["bias"][part][:, None, :]
        y = _act(z, c["act"])
        if weight is not None:
            y = y * weight[table][..., None]
        if residual is not None:
            y = y + residual[table]
        out[table.reshape(-1)] = y.reshape(-1, c["N"])
    out[-1] = 0.0
    return {"y": out[:-1].to(torch.bfloat16)}


def _plain_few4(s):
    c = s["case"]
    T, K, H = c["T"], c["K"], c["H"]
    flat = s["topk_idx"].reshape(-1)
    entry = torch.nonzero(flat >= 0).reshape(-1)
    out = torch.zeros((T * K + 1, H), device="cuda")
    # entries in the order of their experts; each expert's in a row of a padded table
    active, group, counts = torch.unique(flat[entry], return_inverse=True, return_counts=True)
    if active.numel() > 0:
        order = torch.argsort(group, stable=True)
        entry, group = entry[order], group[order]
        place = torch.arange(entry.numel(), device="cuda") - (torch.cumsum(counts, 0) - counts)[group]
        table = torch.full((active.numel(), int(counts.max())), T * K, device="cuda", dtype=torch.int64)
        table[group, place] = entry
        x = torch.cat([s["x"].float(), torch.zeros((1, H), device="cuda")])
        for a in range(0, active.numel(), AT_ONCE):
            some, rows = active[a:a + AT_ONCE], table[a:a + AT_ONCE]
            z = torch.bmm(x[torch.where(rows < T * K, rows // K, T)],
                          _weights(c, s["w_up"][some], s["up_sf"][some], s["up_zero"][some] if c["zero"] else None)
                          .transpose(1, 2))
            if c["bias"]:
                z = z + s["bias_up"][some][:, None, :]
            p = torch.bmm(_act(z, c["act"]),
                          _weights(c, s["w_down"][some], s["down_sf"][some], s["down_zero"][some] if c["zero"] else None)
                          .transpose(1, 2))
            if c["bias"]:
                p = p + s["bias_down"][some][:, None, :]
            out[rows.reshape(-1)] = p.reshape(-1, H)
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
    if c["op"] in ("route", "balance", "route_backward"):
        score = ep.EP_SCORE_SOFTMAX if c["score"] == "softmax" else ep.EP_SCORE_SIGMOID
        if c["op"] == "route":
            ep.ep_route(s["logits"], s["topk_idx"], s["topk_weights"], s["status"], score=score, bias=s["bias"],
                        token_mask=s["token_mask"], num_groups=c["groups"], topk_groups=c["topk_groups"],
                        normalize=c["normalize"], scale=c["scale"])
            return {"topk_idx": s["topk_idx"], "topk_weights": s["topk_weights"]}
        if c["op"] == "balance":
            if "workspace" not in s:
                s["workspace"] = torch.empty(ep.ep_balance_loss_workspace_bytes(c["T"], c["E"], c["sequences"]),
                                             dtype=torch.uint8, device="cuda")
            ep.ep_balance_loss(s["logits"], s["topk_idx"], s["workspace"], s["loss"], s["load"], s["status"], score=score,
                               token_mask=s["token_mask"], seq_offset=s["seq_offset"], coeff=COEFF,
                               num_tokens_per_expert=s["counts"])
            return {"loss": s["loss"], "load": s["load"], "num_tokens_per_expert": s["counts"]}
        ep.ep_route_backward(s["logits"], s["topk_idx"], s["d_logits"], s["status"], d_topk_weights=s["d_topk_weights"],
                             load=s["load"], d_loss=s["d_loss"], score=score, token_mask=s["token_mask"],
                             seq_offset=s["seq_offset"], normalize=c["normalize"], scale=c["scale"])
        return {"d_logits": s["d_logits"]}
    act = {"none": ep.EP_ACT_NONE, "relu": ep.EP_ACT_RELU, "gelu": ep.EP_ACT_GELU, "silu": ep.EP_ACT_SILU,
           "swiglu": ep.EP_ACT_SWIGLU}[c["act"]]
    form = ep.EP_W4_FP if c["form"] == "fp4" else ep.EP_W4_INT
    if c["op"] == "product4":
        ep.ep_expert_gemm_w4(s["x"], s["w"], s["w_sf"], s["expert_offset"], s["num_tokens_per_expert"], s["y"],
                             s["status"], w_zero=s["w_zero"], w_format=form, bias=s["bias"], activation=act,
                             row_weight=s["row_weight"], residual=s["residual"])
        return {"y": s["y"]}
    if "workspace" not in s:
        s["workspace"] = torch.empty(ep.ep_moe_few_tokens_w4_workspace_bytes(c["T"], c["K"], c["H"], c["N"], c["E"]),
                                     dtype=torch.uint8, device="cuda")
    ep.ep_moe_few_tokens_w4(s["x"], s["topk_idx"], s["topk_weights"], s["w_up"], s["up_sf"], s["w_down"], s["down_sf"],
                            s["workspace"], s["out"], s["status"], up_zero=s["up_zero"], down_zero=s["down_zero"],
                            w_format=form, bias_up=s["bias_up"], bias_down=s["bias_down"], residual=s["residual"],
                            activation=act)
    return {"out": s["out"]}


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "balance": _plain_balance, "route_backward": _plain_backward,
            "product4": _plain_product4, "few4": _plain_few4}[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c = case
    T, E, K = c["T"], c["E"], c["K"]
    if c["op"] in ("route", "balance", "route_backward"):
        live = T * (1.0 - c["mask"])
        item = 4 if c["dtype"] == "fp32" else 2
        size = live * E * item + (T if c["mask"] > 0 else 0)
        # an exponential, a division and a few additions a logit
        if c["op"] == "route":
            return {"bytes": size + T * K * 12.0, "flops": 12.0 * live * E}
        if c["op"] == "balance":
            return {"bytes": size + live * K * 8.0 + c["sequences"] * E * 8.0, "flops": 10.0 * live * E}
        size += T * E * item + live * K * 8.0
        if c["parts"] != "loss":
            size += live * K * 4.0
        if c["parts"] != "weights":
            size += c["sequences"] * E * 4.0
        return {"bytes": size, "flops": 16.0 * live * E}
    H, N = c["H"], c["N"]
    Nw = 2 * N if c["act"] == "swiglu" else N
    rows = T * K * (1.0 - c["mask"])
    # experts that some token names, as if uniform (popularity leaves a few more out)
    active = E * (1.0 - (1.0 - rows / T / E) ** T)
    # half a byte, and a scale and perhaps a zero point for each group
    weight = 0.5 + (2 if c["scales"] == "bf16" else 4) * (2 if c["zero"] else 1) / c["group"]
    if c["op"] == "few4":
        size = weight * active * (Nw * H + H * N) + 2.0 * T * H * (3 if c["residual"] else 2) + T * K * 12.0
        size += 4.0 * active * (Nw + H) * c["bias"]
        return {"bytes": size, "flops": 2.0 * rows * (Nw * H + H * N)}
    size = weight * active * Nw * H + 2.0 * rows * (H + N) + 2.0 * rows * N * c["residual"]
    size += 4.0 * rows * c["weight"] + 4.0 * active * Nw * c["bias"]
    return {"bytes": size, "flops": 2.0 * rows * Nw * H}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _act64(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if act == "silu":
        return z * torch.sigmoid(z)
    gate, up = z.chunk(2, dim=-1)
    return gate * torch.sigmoid(gate) * up


def _expert64(c, codes, sf, zero):
    """One expert's weights [rows, depth] in 64 bits."""
    rows, half = codes.shape
    u = torch.empty((rows, half, 2), dtype=torch.int64, device="cuda")
    u[..., 0], u[..., 1] = codes % 16, codes // 16
    u = u.reshape(rows, 2 * half)
    if c["form"] == "fp4":
        # sign, two bits of exponent, one of fraction
        e, m = (u // 2) % 4, (u % 2).double()
        v = torch.where(e == 0, m * 0.5, torch.exp2((e - 1).double()) * (1.0 + 0.5 * m)) * (1.0 - 2.0 * (u // 8).double())
    else:
        v = u.double() - (8.0 if zero is None else zero.double().repeat_interleave(c["group"], 0).T)
    return v * sf.double().repeat_interleave(c["group"], 0).T


def _sequence_list(s):
    """Token numbers of every sequence, masked ones left out."""
    c = s["case"]
    at = [0, c["T"]] if s["seq_offset"] is None else s["seq_offset"].tolist()
    live = torch.ones(c["T"], dtype=torch.bool, device="cuda") if s["token_mask"] is None else s["token_mask"]
    return [torch.nonzero(live[a:b]).reshape(-1) + a for a, b in zip(at, at[1:])]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    T, E, K = c["T"], c["E"], c["K"]
    if c["op"] == "route":
        l = s["logits"].double()
        score = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
        key = l if s["bias"] is None and c["groups"] == 1 else score
        if s["bias"] is not None:
            key = key + s["bias"].double()
        if c["topk_groups"] < c["groups"]:
            G = c["groups"]
            best = key.view(T, G, -1).topk(min(2, E // G), dim=2).values.sum(2)
            _, order = torch.sort(-best, dim=1, stable=True)
            closed = torch.ones((T, G), dtype=torch.bool, device="cuda").scatter_(1, order[:, :c["topk_groups"]], False)
            key = key.masked_fill(closed.repeat_interleave(E // G, 1), -math.inf)
        _, order = torch.sort(-key, dim=1, stable=True)
        idx = order[:, :K].contiguous()
        w = torch.gather(score, 1, idx)
        if c["normalize"]:
            w /= w.sum(1, keepdim=True)
        w *= c["scale"]
        if s["token_mask"] is not None:
            idx[~s["token_mask"]] = -1
            w[~s["token_mask"]] = 0.0
        return {"topk_idx": idx, "topk_weights": w}
    if c["op"] in ("balance", "route_backward"):
        l = s["logits"].double().requires_grad_(c["op"] == "route_backward")
        score = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
        p = score / score.sum(1, keepdim=True)
        S = c["sequences"]
        if c["op"] == "balance":
            loss, load, counts = torch.zeros((), dtype=torch.float64, device="cuda"), [], []
            for tokens in _sequence_list(s):
                named = s["topk_idx"][tokens].reshape(-1)
                count, n = torch.bincount(named[named >= 0], minlength=E), max(1, tokens.numel())
                f = count.double() * E / (K * n)
                loss = loss + COEFF / S * (f * p[tokens].sum(0) / n).sum()
                load.append(COEFF / S * f / n)
                counts.append(count.to(torch.int32))
            return {"loss": loss.reshape(1), "load": torch.stack(load), "num_tokens_per_expert": torch.stack(counts)}
        # the gradient of a scalar whose derivatives by weights and scores are the given ones
        total = (l * 0.0).sum()
        there = s["topk_idx"] >= 0
        if s["d_topk_weights"] is not None:
            w = torch.where(there, score.gather(1, s["topk_idx"].clamp_min(0)), 0.0)
            if c["normalize"]:
                w = w / torch.where(there.any(1), w.sum(1), 1.0)[:, None]
            total = total + (w * c["scale"] * s["d_topk_weights"].double()).sum()
        if s["load"] is not None:
            for q, tokens in enumerate(_sequence_list(s)):
                total = total + s["d_loss"].double()[0] * (p[tokens] * s["load"][q].double()).sum()
        d, = torch.autograd.grad(total, l)
        if s["token_mask"] is not None:
            d = d * s["token_mask"][:, None]
        return {"d_logits": d}
    if c["op"] == "few4":
        out = torch.zeros((T, c["H"]), dtype=torch.float64, device="cuda")
        for e in torch.unique(s["topk_idx"]).tolist():
            if e < 0:
                continue
            t, k = torch.nonzero(s["topk_idx"] == e, as_tuple=True)
            z = s["x"][t].double() @ _expert64(c, s["w_up"][e], s["up_sf"][e], s["up_zero"][e] if c["zero"] else None).T
            if c["bias"]:
                z = z + s["bias_up"][e].double()
            w = _expert64(c, s["w_down"][e], s["down_sf"][e], s["down_zero"][e] if c["zero"] else None)
            p = _act64(z, c["act"]) @ w.T
            if c["bias"]:
                p = p + s["bias_down"][e].double()
            out.index_add_(0, t, p * s["topk_weights"][t, k].double()[:, None])
        if c["residual"]:
            out += s["residual"].double()
        return {"out": out}
    y = torch.zeros((s["rows"], c["N"]), dtype=torch.float64, device="cuda")
    first, count = s["expert_offset"].tolist(), s["num_tokens_per_expert"].tolist()
    for e in range(E):
        if count[e] == 0:
            continue
        r = slice(first[e], first[e] + count[e])
        z = s["x"][r].double() @ _expert64(c, s["w"][e], s["w_sf"][e], s["w_zero"][e] if c["zero"] else None).T
        if c["bias"]:
            z = z + s["bias"][e].double()
        a = _act64(z, c["act"])
        if c["weight"]:
            a = a * s["row_weight"][r].double()[:, None]
        if c["residual"]:
            a = a + s["residual"][r].double()
        y[r] = a
    return {"y": y}
