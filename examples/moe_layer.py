"""A mixture-of-experts layer on the library: one call for a few tokens, the
rows path (layout, expanded dispatch, two experts' products, expanded combine)
for many, and the rows path's backward pass.

    python examples/moe_layer.py [--tokens 4096] [--hidden 2048] [--inner 1024] [--experts 32] [--topk 4]

Every tensor lives on the GPU; nothing here waits for it but the timing.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_ep_get_gb300 as ep  # noqa: E402

ALIGNMENT = 16      # rows of an expert's block start at a multiple of this


class MoeLayer:
    """Weights of E experts: w_up [E, 2 inner, H] (gate rows first), w_down [E, H, inner], bf16.
    A layer keeps its workspaces from call to call: its calls go to one stream at a time."""

    def __init__(self, w_up, w_down, ranks=1):
        self.w_up, self.w_down, self.ranks = w_up, w_down, ranks
        self.experts, self.hidden, self.inner = w_down.shape
        self.status = torch.zeros(1, dtype=torch.int32, device=w_up.device)
        self._workspace = {}

    def _scratch(self, what, nbytes):
        """One workspace for each use, grown when a call needs more."""
        ws = self._workspace.get(what)
        if ws is None or ws.numel() < nbytes:
            ws = self._workspace[what] = torch.empty(nbytes, dtype=torch.uint8, device=self.w_up.device)
        return ws

    def few_tokens(self, x, topk_idx, topk_weights, residual=None):
        """The whole layer in one call, at most EP_FEW_MAX_TOKENS tokens."""
        T, K = topk_idx.shape
        out = torch.empty_like(x)
        ws = self._scratch("few", ep.ep_moe_few_tokens_workspace_bytes(T, K, self.hidden, self.inner, self.experts))
        ep.ep_moe_few_tokens(x, topk_idx, topk_weights, self.w_up, self.w_down, ws, out, self.status,
                             residual=residual, activation=ep.EP_ACT_SWIGLU)
        return out

    def rows(self, x, topk_idx, topk_weights, train=False):
        """The layer over expanded rows; with train, what backward() needs is kept."""
        T, K = topk_idx.shape
        E, R, H = self.experts, self.ranks, self.hidden
        bf, dev = torch.bfloat16, x.device
        layout = ep.alloc_layout(T, E, R, K=K, device=dev)
        ws = self._scratch("layout", ep.ep_layout_workspace_bytes(T, K, E, R))
        ep.ep_get_layout(topk_idx, E, R, layout, ws, self.status, expert_alignment=ALIGNMENT)
        n = ep.ep_expanded_capacity_bound(T, K, E, ALIGNMENT)   # no need to know how many rows there are
        recv_x = torch.empty((n, H), dtype=bf, device=dev)
        recv_src = torch.empty(n, dtype=torch.int32, device=dev)
        recv_w = torch.empty(n, dtype=torch.float32, device=dev)
        ep.ep_dispatch_expanded(x, topk_idx, topk_weights, E, R, layout, recv_x, recv_src, recv_w, self.status)
        first, count = layout.expert_offset, layout.num_tokens_per_expert
        h = torch.empty((n, self.inner), dtype=bf, device=dev)
        y = torch.empty((n, H), dtype=bf, device=dev)
        z_up = torch.empty((n, 2 * self.inner), dtype=bf, device=dev) if train else None
        z_down = torch.empty((n, H), dtype=bf, device=dev) if train else None
        ep.ep_expert_gemm(recv_x, self.w_up, first, count, h, self.status, activation=ep.EP_ACT_SWIGLU, z=z_up)
        ep.ep_expert_gemm(h, self.w_down, first, count, y, self.status, row_weight=recv_w, z=z_down)
        out = torch.empty((T, H), dtype=bf, device=dev)
        ep.ep_combine_expanded(y, None, K, E, R, layout, out, self.status)
        saved = (topk_idx, layout, recv_x, recv_w, h, z_up, z_down) if train else None
        return (out, saved) if train else out

    def backward(self, d_out, saved):
        """Gradients of x, topk_weights, w_up and w_down.  The combine's
        gradient is a dispatch, the dispatch's a combine."""
        topk_idx, layout, recv_x, recv_w, h, z_up, z_down = saved
        T, K = topk_idx.shape
        E, R, n = self.experts, self.ranks, recv_x.shape[0]
        dev = d_out.device
        first, count = layout.expert_offset, layout.num_tokens_per_expert
        d_y = torch.empty_like(recv_x)
        ep.ep_dispatch_expanded(d_out, topk_idx, None, E, R, layout, d_y, None, None, self.status)
        d_h, d_down, d_row = torch.empty_like(h), torch.empty_like(self.w_down), torch.empty(n, device=dev)
        ws = self._scratch("backward", max(
            ep.ep_expert_gemm_backward_workspace_bytes(n, self.hidden, E, ep.EP_ACT_NONE),
            ep.ep_expert_gemm_backward_workspace_bytes(n, self.inner, E, ep.EP_ACT_SWIGLU)))
        ep.ep_expert_gemm_backward(d_y, h, self.w_down, z_down, first, count, ws, self.status, dx=d_h, dw=d_down,
                                   d_row_weight=d_row, row_weight=recv_w)
        d_recv, d_up = torch.empty_like(recv_x), torch.empty_like(self.w_up)
        ep.ep_expert_gemm_backward(d_h, recv_x, self.w_up, z_up, first, count, ws, self.status, dx=d_recv, dw=d_up,
                                   activation=ep.EP_ACT_SWIGLU)
        d_x = torch.empty_like(d_out)
        ep.ep_combine_expanded(d_recv, None, K, E, R, layout, d_x, self.status)
        row = layout.expanded_row
        d_topk = torch.where(row >= 0, d_row[row.clamp_min(0).long()], torch.zeros((), device=dev))
        return d_x, d_topk, d_up, d_down

    def __call__(self, x, topk_idx, topk_weights):
        if x.shape[0] <= ep.EP_FEW_MAX_TOKENS and topk_idx.shape[1] <= ep.EP_FEW_MAX_TOPK:
            return self.few_tokens(x, topk_idx, topk_weights)
        return self.rows(x, topk_idx, topk_weights)


def inputs(tokens, hidden, inner, experts, topk, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)

    idx = torch.argsort(torch.rand((tokens, experts), generator=g, device="cuda"), dim=1)[:, :topk].contiguous()
    weights = torch.softmax(torch.randn((tokens, topk), generator=g, device="cuda"), dim=1)
    return (normal(tokens, hidden), idx, weights, normal(experts, 2 * inner, hidden, std=hidden ** -0.5),
            normal(experts, hidden, inner, std=inner ** -0.5))


def timed(what, f, n=20):
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        f()
    b.record()
    torch.cuda.synchronize()
    print("%-28s %9.1f us" % (what, a.elapsed_time(b) / n * 1e3))


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("tokens", 4096), ("hidden", 2048), ("inner", 1024), ("experts", 32), ("topk", 4)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    x, idx, weights, w_up, w_down = inputs(a.tokens, a.hidden, a.inner, a.experts, a.topk)
    layer = MoeLayer(w_up, w_down)
    few = min(a.tokens, 16)
    one, many = layer.few_tokens(x[:few], idx[:few], weights[:few]), layer.rows(x, idx, weights)
    print("few-token call against the rows path, largest difference: %.4f of %.4f"
          % (float((one - many[:few]).abs().max()), float(many[:few].abs().max())))
    timed("few tokens (%d)" % few, lambda: layer.few_tokens(x[:few], idx[:few], weights[:few]))
    timed("rows path (%d)" % a.tokens, lambda: layer.rows(x, idx, weights))
    d_out = torch.randn(x.shape, device="cuda").to(torch.bfloat16)
    _, saved = layer.rows(x, idx, weights, train=True)
    timed("rows path, backward", lambda: layer.backward(d_out, saved))
    status = int(layer.status.item())
    print("status:", ep.ep_status_string(status))
    return status


if __name__ == "__main__":
    sys.exit(main())
