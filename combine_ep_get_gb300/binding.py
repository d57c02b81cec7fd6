"""ctypes binding of libep_get.so with the C ABI's entry-point names.

Argument marshalling only: tensors become device pointers, the current torch
CUDA stream becomes the cudaStream_t, and a non-zero host status raises.  All
computation happens in the library's CUDA kernels.  Importing this module
fails when the library has not been built (there is no CPU fallback).
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# EP_GET_LIBRARY names another build of the same library to load instead:
# the bounds-checked copy that the tests build (ep_bounds_checked() says which
# one is loaded).  Unset, the product library.
LIB_PATH = os.environ.get("EP_GET_LIBRARY") or os.path.join(_HERE, "libep_get.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("%s is not built; run `python -c \"import __graft_entry__ as g; "
                      "g.build()\"` or `python combine_ep_get_gb300/build.py`" % LIB_PATH)

_lib = ctypes.CDLL(LIB_PATH)

EP_OK = 0
EP_ERR_INVALID_ARG = 1
EP_ERR_UNSUPPORTED = 2
EP_ERR_INVALID_INDEX = 4
EP_ERR_CAPACITY = 8
EP_ERR_TIMEOUT = 16
EP_ERR_CUDA = 32
EP_ERR_OUT_OF_BOUNDS = 64
EP_BF16 = 0
EP_FP8_E4M3 = 1
EP_FP16 = 2
EP_FP32 = 3
EP_ACT_NONE = 0
EP_ACT_RELU = 1
EP_ACT_GELU = 2
EP_ACT_SILU = 3
EP_ACT_SWIGLU = 4
EP_FEW_MAX_TOKENS = 256
EP_FEW_MAX_TOPK = 16
EP_SCORE_SOFTMAX = 0
EP_SCORE_SIGMOID = 1
EP_W4_INT = 0
EP_W4_FP = 1

_vp = ctypes.c_void_p
_i = ctypes.c_int
_i64 = ctypes.c_int64


class ep_layout_t(ctypes.Structure):
    _fields_ = [("num_tokens_per_rank", _vp), ("num_tokens_per_node", _vp),
                ("num_tokens_per_expert", _vp), ("is_token_in_rank", _vp), ("rank_offset", _vp),
                ("expert_offset", _vp), ("dst_row", _vp), ("src_dst_count", _vp),
                ("token_offset", _vp), ("expanded_row", _vp), ("node_offset", _vp), ("node_row", _vp)]


_lib.ep_layout_workspace_bytes.restype = ctypes.c_size_t
_lib.ep_layout_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
_lib.ep_recv_capacity_bound.restype = _i64
_lib.ep_recv_capacity_bound.argtypes = [_i, _i, _i]
_lib.ep_get_layout.restype = ctypes.c_int32
_lib.ep_get_layout.argtypes = [_vp, _i, _i, _i, _i, _i, _i, ctypes.POINTER(ep_layout_t), _vp,
                               ctypes.c_size_t, _vp, _vp]
_lib.ep_get_layout_static_scratch.restype = ctypes.c_int32
_lib.ep_get_layout_static_scratch.argtypes = [_vp, _i, _i, _i, _i, _i, _i, ctypes.POINTER(ep_layout_t),
                                              _vp, _vp]
_lib.ep_dispatch.restype = ctypes.c_int32
_lib.ep_dispatch.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.POINTER(ep_layout_t), _i,
                             _i64, _vp, _vp, _i, _vp, _vp, _vp, _i, _vp, _vp]
_lib.ep_layout_and_dispatch.restype = ctypes.c_int32
_lib.ep_layout_and_dispatch.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, ctypes.POINTER(ep_layout_t), _vp,
                                        ctypes.c_size_t, _i, _i64, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp]
_lib.ep_combine.restype = ctypes.c_int32
_lib.ep_combine.argtypes = [_vp, _i64, _vp, _vp, _i, _i, _i, _i, _i, ctypes.POINTER(ep_layout_t),
                            _vp, _i, _vp, _vp]
_lib.ep_expanded_capacity_bound.restype = _i64
_lib.ep_expanded_capacity_bound.argtypes = [_i, _i, _i, _i]
_lib.ep_dispatch_expanded.restype = ctypes.c_int32
_lib.ep_dispatch_expanded.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.POINTER(ep_layout_t), _i,
                                      _i64, _vp, _vp, _i, _vp, _vp, _i, _vp, _vp]
_lib.ep_combine_expanded.restype = ctypes.c_int32
_lib.ep_combine_expanded.argtypes = [_vp, _i64, _vp, _i, _i, _i, _i, _i, ctypes.POINTER(ep_layout_t), _vp,
                                     _i, _vp, _vp]
_lib.ep_combine_topk_weights.restype = ctypes.c_int32
_lib.ep_combine_topk_weights.argtypes = [_vp, _i64, _i, _i, _i, _i, ctypes.POINTER(ep_layout_t), _vp, _vp,
                                         _vp]
_lib.ep_accumulate_expert_stats.restype = ctypes.c_int32
_lib.ep_accumulate_expert_stats.argtypes = [ctypes.POINTER(ep_layout_t), _i, _vp, _vp]
_lib.ep_status_string.restype = ctypes.c_char_p
_lib.ep_status_string.argtypes = [ctypes.c_int32]
_lib.ep_abi_version.restype = _i
_lib.ep_abi_version.argtypes = []
_lib.ep_bounds_checked.restype = _i
_lib.ep_bounds_checked.argtypes = []
_lib.ep_dispatch_hierarchical.restype = ctypes.c_int32
_lib.ep_dispatch_hierarchical.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, ctypes.POINTER(ep_layout_t), _i,
                                          _i64, _vp, _vp, _vp, _i64, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp]
_lib.ep_combine_hierarchical.restype = ctypes.c_int32
_lib.ep_combine_hierarchical.argtypes = [_vp, _i64, _vp, _vp, _i, _i, _i, _i, _i, _i, ctypes.POINTER(ep_layout_t),
                                         _i64, _vp, _vp, _vp, _vp]
_lib.ep_theoretical_num_sms.restype = _i
_lib.ep_theoretical_num_sms.argtypes = [_i, _i, _i, _i, _i, _i, ctypes.c_double, ctypes.c_double,
                                        ctypes.c_double, _i, _i]
_lib.ep_expert_gemm.restype = ctypes.c_int32
_lib.ep_expert_gemm.argtypes = [_vp, _vp, _i, _vp, _vp, _i, _vp, _i, _vp, _vp, _i64, _i, _i, _i, _vp, _vp, _vp, _vp,
                                _vp, _vp]
_lib.ep_expert_gemm_backward_workspace_bytes.restype = ctypes.c_size_t
_lib.ep_expert_gemm_backward_workspace_bytes.argtypes = [_i64, _i, _i, _i]
_lib.ep_expert_gemm_backward.restype = ctypes.c_int32
_lib.ep_expert_gemm_backward.argtypes = [_vp, _vp, _vp, _vp, _i, _vp, _i64, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp,
                                         _vp, ctypes.c_size_t, _vp, _vp]
_lib.ep_moe_few_tokens_workspace_bytes.restype = ctypes.c_size_t
_lib.ep_moe_few_tokens_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
_lib.ep_moe_few_tokens.restype = ctypes.c_int32
_lib.ep_moe_few_tokens.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp,
                                   ctypes.c_size_t, _vp, _vp, _vp]
_f = ctypes.c_float
_sz = ctypes.c_size_t
_lib.ep_route.restype = ctypes.c_int32
_lib.ep_route.argtypes = [_vp, _i, _i64, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp, _vp]
_lib.ep_balance_loss_workspace_bytes.restype = _sz
_lib.ep_balance_loss_workspace_bytes.argtypes = [_i, _i, _i]
_lib.ep_balance_loss.restype = ctypes.c_int32
_lib.ep_balance_loss.argtypes = [_vp, _i, _i64, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp, _vp, _sz, _vp, _vp]
_lib.ep_route_backward.restype = ctypes.c_int32
_lib.ep_route_backward.argtypes = [_vp, _i, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _i64,
                                   _vp, _vp]
_lib.ep_expert_gemm_w4.restype = ctypes.c_int32
_lib.ep_expert_gemm_w4.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _vp, _i, _vp, _vp, _i64, _i, _i, _i, _vp, _vp, _vp,
                                   _vp, _vp]
_lib.ep_moe_few_tokens_w4_workspace_bytes.restype = _sz
_lib.ep_moe_few_tokens_w4_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
_lib.ep_moe_few_tokens_w4.restype = ctypes.c_int32
_lib.ep_moe_few_tokens_w4.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _i, _vp, _i, _i, _vp, _i,
                                      _i, _i, _i, _i, _vp, _sz, _vp, _vp, _vp]


def library():
    """The loaded ctypes library (for callers that marshal raw pointers)."""
    return _lib


def ep_bounds_checked() -> bool:
    """True when the loaded library is the bounds-checked build."""
    return bool(_lib.ep_bounds_checked())


def _ptr(t):
    if t is None:
        return None
    return t.data_ptr()


# The current stream's handle without a Stream object around it, which costs a
# call more than all of its checks; torch.cuda.current_stream() where a torch
# has no such shortcut.  The device without torch.cuda's check that CUDA is up:
# a call has tensors on it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and _current_device is not None:
        return _raw_stream(_current_device())
    return torch.cuda.current_stream().cuda_stream


def _check(code, what):
    if code != EP_OK:
        raise RuntimeError("%s failed: %s" % (what, ep_status_string(code)))
    return code


def ep_status_string(status) -> str:
    return _lib.ep_status_string(int(status)).decode()


def ep_layout_workspace_bytes(num_tokens, num_topk, num_experts, num_ranks, ranks_per_node=0) -> int:
    return int(_lib.ep_layout_workspace_bytes(num_tokens, num_topk, num_experts, num_ranks,
                                              ranks_per_node))


def ep_recv_capacity_bound(num_tokens, num_topk, num_ranks) -> int:
    return int(_lib.ep_recv_capacity_bound(num_tokens, num_topk, num_ranks))


def ep_theoretical_num_sms(hidden, num_topk, num_experts, num_ranks, hbm_gbs, out_dtype=EP_BF16,
                           is_combine=False, sm_read_gbs=200.0, sm_write_gbs=50.0,
                           prefer_overlap_with_compute=True, device_sms=None) -> int:
    """SM count for the SM-limited mode; device_sms defaults to the current
    device's SM count.  Raises ValueError for arguments the library rejects."""
    if device_sms is None:
        device_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    n = int(_lib.ep_theoretical_num_sms(hidden, num_topk, num_experts, num_ranks, out_dtype, int(is_combine),
                                        float(hbm_gbs), float(sm_read_gbs), float(sm_write_gbs),
                                        int(prefer_overlap_with_compute), int(device_sms)))
    if n == 0:
        raise ValueError("ep_theoretical_num_sms: invalid arguments")
    return n


class Layout:
    """Device tensors of one routing layout plus their ep_layout_t view."""

    def __init__(self, T, E, R, ranks_per_node=0, with_src_dst=True, device="cuda", K=None, node_rows=False):
        i32 = dict(dtype=torch.int32, device=device)
        nodes = R // ranks_per_node if ranks_per_node > 0 else 0
        self.T, self.E, self.R, self.ranks_per_node = T, E, R, ranks_per_node
        self.num_tokens_per_rank = torch.empty(R, **i32)
        self.num_tokens_per_node = torch.empty(nodes, **i32) if nodes else None
        self.num_tokens_per_expert = torch.empty(E, **i32)
        self.is_token_in_rank = torch.empty((T, R), dtype=torch.uint8, device=device)
        self.rank_offset = torch.empty(R + 1, **i32)
        self.expert_offset = torch.empty(E + 1, **i32)
        self.dst_row = torch.empty((T, R), **i32)
        self.src_dst_count = torch.empty((R, R), **i32) if (with_src_dst and T % R == 0) else None
        self.token_offset = torch.empty(T + 1, **i32)
        # expanded (per-expert) rows are produced when K is given
        self.expanded_row = torch.empty((T, K), **i32) if K is not None else None
        # per-node scale-out rows (hierarchical path) when node_rows is set
        self.node_offset = torch.empty(nodes + 1, **i32) if (node_rows and nodes) else None
        self.node_row = torch.empty((T, nodes), **i32) if (node_rows and nodes) else None
        self.c = ep_layout_t(*[_ptr(getattr(self, f)) for f, _ in ep_layout_t._fields_])

    @property
    def num_recv(self) -> int:
        """N = rank_offset[R] (one device-to-host read)."""
        return int(self.rank_offset[-1].item())


def alloc_layout(T, E, R, ranks_per_node=0, with_src_dst=True, device="cuda", K=None, node_rows=False) -> Layout:
    """Device arrays of a layout; pass K to also get the expanded rows, and
    node_rows=True (with ranks_per_node > 0) for the hierarchical path's node rows."""
    return Layout(T, E, R, ranks_per_node, with_src_dst, device, K, node_rows)


def ep_expanded_capacity_bound(num_tokens, num_topk, num_experts, expert_alignment=1) -> int:
    return int(_lib.ep_expanded_capacity_bound(num_tokens, num_topk, num_experts, expert_alignment))


def ep_get_layout(topk_idx, num_experts, num_ranks, layout, workspace, d_status, ranks_per_node=0,
                  expert_alignment=1, stream=None):
    T, K = topk_idx.shape
    assert topk_idx.dtype == torch.int64 and topk_idx.is_contiguous()
    code = _lib.ep_get_layout(_ptr(topk_idx), T, K, num_experts, num_ranks, ranks_per_node,
                              expert_alignment, ctypes.byref(layout.c), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _ptr(d_status),
                              _stream(stream))
    return _check(code, "ep_get_layout")


def ep_get_layout_static_scratch(topk_idx, num_experts, num_ranks, layout, d_status, ranks_per_node=0,
                                 expert_alignment=1, stream=None):
    """ep_get_layout using the library's built-in scratch instead of a caller
    workspace, for callers that cannot allocate device memory (see the C
    header for the size limit and the ordering rule)."""
    T, K = topk_idx.shape
    assert topk_idx.dtype == torch.int64 and topk_idx.is_contiguous()
    code = _lib.ep_get_layout_static_scratch(_ptr(topk_idx), T, K, num_experts, num_ranks,
                                             ranks_per_node, expert_alignment, ctypes.byref(layout.c),
                                             _ptr(d_status), _stream(stream))
    return _check(code, "ep_get_layout_static_scratch")


def ep_dispatch(x, topk_idx, topk_weights, num_experts, num_ranks, layout, recv_x, recv_topk_idx,
                recv_topk_weights, recv_src_idx, d_status, recv_sf=None, out_dtype=EP_BF16,
                sf_col_major=False, num_sms=0, stream=None):
    T, H = x.shape
    K = topk_idx.shape[1]
    assert x.element_size() == 2 and x.is_contiguous() and recv_x.is_contiguous()
    capacity = recv_x.shape[0]
    code = _lib.ep_dispatch(_ptr(x), _ptr(topk_idx), _ptr(topk_weights), T, H, K, num_experts,
                            num_ranks, ctypes.byref(layout.c), out_dtype, capacity, _ptr(recv_x),
                            _ptr(recv_sf), 1 if sf_col_major else 0, _ptr(recv_topk_idx),
                            _ptr(recv_topk_weights), _ptr(recv_src_idx), num_sms, _ptr(d_status),
                            _stream(stream))
    return _check(code, "ep_dispatch")


def ep_dispatch_expanded(x, topk_idx, topk_weights, num_experts, num_ranks, layout, recv_x, recv_src_idx,
                         recv_weight, d_status, recv_sf=None, out_dtype=EP_BF16, sf_col_major=False,
                         num_sms=0, stream=None):
    T, H = x.shape
    K = topk_idx.shape[1]
    assert x.element_size() == 2 and x.is_contiguous() and recv_x.is_contiguous()
    code = _lib.ep_dispatch_expanded(_ptr(x), _ptr(topk_idx), _ptr(topk_weights), T, H, K, num_experts,
                                     num_ranks, ctypes.byref(layout.c), out_dtype, recv_x.shape[0],
                                     _ptr(recv_x), _ptr(recv_sf), 1 if sf_col_major else 0,
                                     _ptr(recv_src_idx), _ptr(recv_weight), num_sms, _ptr(d_status),
                                     _stream(stream))
    return _check(code, "ep_dispatch_expanded")


def ep_combine_expanded(y, topk_weights, num_topk, num_experts, num_ranks, layout, out, d_status,
                        num_sms=0, stream=None):
    T, H = out.shape
    assert y.element_size() == 2 and y.is_contiguous() and out.is_contiguous()
    code = _lib.ep_combine_expanded(_ptr(y), y.shape[0], _ptr(topk_weights), T, H, num_topk, num_experts,
                                    num_ranks, ctypes.byref(layout.c), _ptr(out), num_sms, _ptr(d_status),
                                    _stream(stream))
    return _check(code, "ep_combine_expanded")


def ep_combine_topk_weights(recv_topk_weights, num_experts, num_ranks, layout, combined, d_status,
                            stream=None):
    T, K = combined.shape
    assert recv_topk_weights.is_contiguous() and combined.is_contiguous()
    code = _lib.ep_combine_topk_weights(_ptr(recv_topk_weights), recv_topk_weights.shape[0], T, K,
                                        num_experts, num_ranks, ctypes.byref(layout.c), _ptr(combined),
                                        _ptr(d_status), _stream(stream))
    return _check(code, "ep_combine_topk_weights")


def ep_accumulate_expert_stats(layout, num_experts, stats, stream=None):
    assert stats.dtype == torch.int64 and stats.is_contiguous()
    code = _lib.ep_accumulate_expert_stats(ctypes.byref(layout.c), num_experts, _ptr(stats), _stream(stream))
    return _check(code, "ep_accumulate_expert_stats")


def ep_layout_and_dispatch(x, topk_idx, topk_weights, num_experts, num_ranks, layout, workspace, recv_x,
                           recv_topk_idx, recv_topk_weights, recv_src_idx, d_status, recv_sf=None,
                           out_dtype=EP_BF16, sf_col_major=False, ranks_per_node=0, expert_alignment=1,
                           stream=None):
    """ep_get_layout and ep_dispatch in one call (see the C header): one kernel
    for few tokens, else the layout kernel and the dispatch, whose first wave
    starts on the layout's rows-ready signal in `workspace`.  Size `workspace`
    with ep_layout_workspace_bytes and the receive arrays with
    ep_recv_capacity_bound; the workspace belongs to the call until the
    dispatch completes."""
    T, H = x.shape
    K = topk_idx.shape[1]
    assert x.element_size() == 2 and x.is_contiguous() and recv_x.is_contiguous()
    assert topk_idx.dtype == torch.int64 and topk_idx.is_contiguous()
    code = _lib.ep_layout_and_dispatch(_ptr(x), _ptr(topk_idx), _ptr(topk_weights), T, H, K, num_experts, num_ranks,
                                       ranks_per_node, expert_alignment, ctypes.byref(layout.c), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), out_dtype, recv_x.shape[0],
                                       _ptr(recv_x), _ptr(recv_sf), 1 if sf_col_major else 0, _ptr(recv_topk_idx),
                                       _ptr(recv_topk_weights), _ptr(recv_src_idx), _ptr(d_status), _stream(stream))
    return _check(code, "ep_layout_and_dispatch")


def ep_combine(y, topk_idx, topk_weights, num_experts, num_ranks, layout, out, d_status, num_sms=0,
               stream=None):
    T, H = out.shape
    K = topk_idx.shape[1]
    assert y.element_size() == 2 and y.is_contiguous() and out.is_contiguous()
    code = _lib.ep_combine(_ptr(y), y.shape[0], _ptr(topk_idx), _ptr(topk_weights), T, H, K,
                           num_experts, num_ranks, ctypes.byref(layout.c), _ptr(out), num_sms,
                           _ptr(d_status), _stream(stream))
    return _check(code, "ep_combine")


def ep_dispatch_hierarchical(x, topk_idx, topk_weights, num_experts, num_ranks, ranks_per_node, layout, node_x,
                             recv_x, d_status, node_sf=None, node_src_idx=None, recv_sf=None, recv_topk_idx=None,
                             recv_topk_weights=None, recv_src_idx=None, out_dtype=EP_BF16, sf_col_major=False,
                             stream=None):
    """Two-stage dispatch: node_x / node_sf / node_src_idx are the per-node
    scale-out buffers (node_capacity = node_x.shape[0]); recv_* as ep_dispatch."""
    T, H = x.shape
    K = topk_idx.shape[1]
    assert x.element_size() == 2 and x.is_contiguous() and recv_x.is_contiguous() and node_x.is_contiguous()
    code = _lib.ep_dispatch_hierarchical(_ptr(x), _ptr(topk_idx), _ptr(topk_weights), T, H, K, num_experts,
                                         num_ranks, ranks_per_node, ctypes.byref(layout.c), out_dtype,
                                         node_x.shape[0], _ptr(node_x), _ptr(node_sf), _ptr(node_src_idx),
                                         recv_x.shape[0], _ptr(recv_x), _ptr(recv_sf), int(sf_col_major),
                                         _ptr(recv_topk_idx), _ptr(recv_topk_weights), _ptr(recv_src_idx),
                                         _ptr(d_status), _stream(stream))
    return _check(code, "ep_dispatch_hierarchical")


def ep_combine_hierarchical(y, topk_idx, topk_weights, num_experts, num_ranks, ranks_per_node, layout, node_y,
                            out, d_status, stream=None):
    """Two-stage combine: node_y (bf16 [node_capacity, H]) receives the
    per-(token, node) partials; out the combined rows."""
    T, K = topk_idx.shape
    H = out.shape[1]
    assert y.element_size() == 2 and out.element_size() == 2 and node_y.element_size() == 2
    code = _lib.ep_combine_hierarchical(_ptr(y), y.shape[0], _ptr(topk_idx), _ptr(topk_weights), T, H, K,
                                        num_experts, num_ranks, ranks_per_node, ctypes.byref(layout.c),
                                        node_y.shape[0], _ptr(node_y), _ptr(out), _ptr(d_status), _stream(stream))
    return _check(code, "ep_combine_hierarchical")


def _here(t, name):
    """Device of a call's first tensor, for the others' checks: a call's kernels run on the current device, and its
    tensors have to be there (pinned ones are on none, -1)."""
    at = t.get_device()
    assert at < 0 or at == _now(), "%s: on another than the current device" % name
    return at


def _now():
    return _current_device() if _current_device is not None else torch.cuda.current_device()


def _reached(t, here):
    """Whether kernels reach a tensor: on the GPU or pinned; with `here`, from _here, on that GPU (the current one where
    the first tensor is pinned)."""
    if here is None:
        return t.is_cuda or t.is_pinned()
    at = t.get_device()
    return at == (here if here >= 0 else _now()) if at >= 0 else t.is_cuda or t.is_pinned()


def _take(t, dtype, shape, name, here=None):
    """Address of a contiguous tensor of this type and shape (the library
    takes no strides) on the GPU (or pinned, which kernels reach too); None
    stays None."""
    if t is None:
        return None
    assert t.dtype is dtype and t.shape == shape and t.is_contiguous() and (
        (t.is_cuda if here is None else t.get_device() == here >= 0) or _reached(t, here)), \
        "%s: a contiguous %s tensor of shape %s on the current GPU is wanted" % (name, dtype, tuple(shape))
    return t.data_ptr()


def _take_any(t, name, here=None):
    """Address of a contiguous tensor of any shape on the GPU."""
    assert t.is_contiguous() and (
        (t.is_cuda if here is None else t.get_device() == here >= 0) or _reached(t, here)), \
        "%s: a contiguous tensor on the current GPU is wanted" % name
    return t.data_ptr()


def _word(d_status, here=None):
    """Address of the status word; None stays None (the library answers invalid_arg)."""
    if d_status is None:
        return None
    assert d_status.dtype is torch.int32 and (
        (d_status.is_cuda if here is None else d_status.get_device() == here >= 0) or _reached(d_status, here)), \
        "d_status: an int32 word on the current GPU is wanted"
    return d_status.data_ptr()


def _blocks(expert_offset, num_tokens_per_expert, E, here=None):
    """Addresses of the experts' blocks (offsets may go on past the last expert's)."""
    assert expert_offset.dtype is torch.int32 and expert_offset.numel() >= E
    return (_take_any(expert_offset, "expert_offset", here),
            _take(num_tokens_per_expert, torch.int32, (E,), "num_tokens_per_expert", here))


def ep_expert_gemm(x, w, expert_offset, num_tokens_per_expert, y, d_status, bias=None, activation=EP_ACT_NONE,
                   row_weight=None, residual=None, z=None, x_sf=None, w_sf=None, sf_col_major=False, stream=None):
    """Experts' matrix product over the expanded receive rows, with bias,
    activation, row weight and residual in its epilogue (see the C header).
    x [rows, k] and w [E, n_w, k] are bf16, or both float8_e4m3fn (or uint8
    codes) with x_sf and w_sf; a layout's expert_offset and
    num_tokens_per_expert say which rows are whose.  y [rows, n] (and z
    [rows, n_w], the pre-activation for the backward call) are written at the
    experts' rows."""
    bf16, f32 = torch.bfloat16, torch.float32
    rows, k_dim = x.shape
    E, n_w, _ = w.shape
    gated = activation == EP_ACT_SWIGLU
    assert not gated or n_w % 2 == 0
    n_dim = n_w // 2 if gated else n_w
    fp8 = x.element_size() == 1
    kind = x.dtype if fp8 else bf16
    scales = scale_weights = None
    if fp8:
        assert kind in (torch.float8_e4m3fn, torch.uint8)
        stride = (rows + 3) // 4 * 4 if sf_col_major else rows
        assert x_sf.dtype is f32 and x_sf.numel() >= stride * (k_dim // 128)
        scales, scale_weights = _take_any(x_sf, "x_sf"), _take(w_sf, f32, (E, n_w // 128, k_dim // 128), "w_sf")
    first, count = _blocks(expert_offset, num_tokens_per_expert, E)
    code = _lib.ep_expert_gemm(_take(x, kind, (rows, k_dim), "x"), scales, 1 if sf_col_major else 0,
                               _take(w, kind, (E, n_w, k_dim), "w"), scale_weights, EP_FP8_E4M3 if fp8 else EP_BF16,
                               _take(bias, f32, (E, n_w), "bias"), activation,
                               _take(row_weight, f32, (rows,), "row_weight"),
                               _take(residual, bf16, (rows, n_dim), "residual"), rows, k_dim, n_dim, E, first, count,
                               _take(y, bf16, (rows, n_dim), "y"), _take(z, bf16, (rows, n_w), "z"), _word(d_status),
                               _stream(stream))
    return _check(code, "ep_expert_gemm")


def ep_expert_gemm_backward_workspace_bytes(num_rows, n_dim, num_experts, activation=EP_ACT_NONE) -> int:
    return int(_lib.ep_expert_gemm_backward_workspace_bytes(num_rows, n_dim, num_experts, activation))


def ep_expert_gemm_backward(dy, x, w, z, expert_offset, num_tokens_per_expert, workspace, d_status, dx=None, dw=None,
                            dbias=None, d_row_weight=None, activation=EP_ACT_NONE, row_weight=None, stream=None):
    """Gradients of ep_expert_gemm (bf16) for its rows, weights, bias and row
    weights, each where its output is given (see the C header).  x may be None
    without dw, w without dx, z without an activation and d_row_weight.  The
    residual's gradient is dy itself."""
    bf16, f32 = torch.bfloat16, torch.float32
    rows, n_dim = dy.shape
    like_w = w if w is not None else dw
    if like_w is not None:
        E, n_w, k_dim = like_w.shape
    else:   # no product can be wanted: x and w are not read, k_dim is any width
        E, n_w = num_tokens_per_expert.numel(), 2 * n_dim if activation == EP_ACT_SWIGLU else n_dim
        like_x = x if x is not None else dx
        k_dim = like_x.shape[1] if like_x is not None else 8
    assert n_w == (2 * n_dim if activation == EP_ACT_SWIGLU else n_dim)
    first, count = _blocks(expert_offset, num_tokens_per_expert, E)
    code = _lib.ep_expert_gemm_backward(
        _take(dy, bf16, (rows, n_dim), "dy"), _take(x, bf16, (rows, k_dim), "x"), _take(w, bf16, (E, n_w, k_dim), "w"),
        _take(z, bf16, (rows, n_w), "z"), activation, _take(row_weight, f32, (rows,), "row_weight"), rows, k_dim, n_dim,
        E, first, count, _take(dx, bf16, (rows, k_dim), "dx"), _take(dw, bf16, (E, n_w, k_dim), "dw"),
        _take(dbias, f32, (E, n_w), "dbias"), _take(d_row_weight, f32, (rows,), "d_row_weight"),
        _take_any(workspace, "workspace"), workspace.nbytes, _word(d_status), _stream(stream))
    return _check(code, "ep_expert_gemm_backward")


def ep_moe_few_tokens_workspace_bytes(num_tokens, num_topk, hidden, inner, num_experts) -> int:
    return int(_lib.ep_moe_few_tokens_workspace_bytes(num_tokens, num_topk, hidden, inner, num_experts))


def ep_moe_few_tokens(x, topk_idx, topk_weights, w_up, w_down, workspace, out, d_status, bias_up=None, bias_down=None,
                      residual=None, activation=EP_ACT_SWIGLU, stream=None):
    """A whole mixture-of-experts layer for at most EP_FEW_MAX_TOKENS tokens,
    in two kernels (see the C header): x and out [T, H], w_up [E, n_w, H],
    w_down [E, H, inner], bf16."""
    bf16, f32 = torch.bfloat16, torch.float32
    T, H = x.shape
    K = topk_idx.shape[1]
    E, n_w, _ = w_up.shape
    inner = w_down.shape[2]
    assert n_w == (2 * inner if activation == EP_ACT_SWIGLU else inner)
    code = _lib.ep_moe_few_tokens(
        _take(x, bf16, (T, H), "x"), _take(topk_idx, torch.int64, (T, K), "topk_idx"),
        _take(topk_weights, f32, (T, K), "topk_weights"), _take(w_up, bf16, (E, n_w, H), "w_up"),
        _take(bias_up, f32, (E, n_w), "bias_up"), activation, _take(w_down, bf16, (E, H, inner), "w_down"),
        _take(bias_down, f32, (E, H), "bias_down"), _take(residual, bf16, (T, H), "residual"), T, H, inner, K, E,
        _take_any(workspace, "workspace"), workspace.nbytes, _take(out, bf16, (T, H), "out"), _word(d_status),
        _stream(stream))
    return _check(code, "ep_moe_few_tokens")


_ROW_TYPES = {torch.bfloat16: EP_BF16, torch.float16: EP_FP16, torch.float32: EP_FP32}


def _rows_of(t, shape, name):
    """Address, type, row stride and device of a matrix whose rows are contiguous (columns of a wider one will do)."""
    assert t.dtype in _ROW_TYPES and t.shape == shape and (t.is_cuda or t.is_pinned()), \
        "%s: a %s tensor of bf16, fp16 or fp32 on the GPU is wanted" % (name, tuple(shape))
    here = _here(t, name)
    rows, cols = shape
    assert cols <= 1 or rows == 0 or t.stride(1) == 1, "%s: rows must be contiguous" % name
    stride = t.stride(0) if rows > 1 else cols
    assert stride >= cols, "%s: rows must not overlap" % name
    return t.data_ptr(), _ROW_TYPES[t.dtype], stride, here


def _mask(token_mask, T, here):
    """Address of a token mask: bool or uint8, one byte a token."""
    if token_mask is None:
        return None
    assert token_mask.dtype in (torch.bool, torch.uint8), "token_mask: bool or uint8 is wanted"
    return _take(token_mask, token_mask.dtype, (T,), "token_mask", here)


def _sequences(seq_offset, here):
    """Address of sequences' offsets and how many sequences there are; None: one of all tokens."""
    if seq_offset is None:
        return None, 1
    return _take(seq_offset, torch.int32, (seq_offset.numel(),), "seq_offset", here), seq_offset.numel() - 1


def ep_route(logits, topk_idx, topk_weights, d_status, score=EP_SCORE_SOFTMAX, bias=None, token_mask=None, num_groups=1,
             topk_groups=None, normalize=True, scale=1.0, stream=None):
    """Each token's top-k experts and their weights from the router's logits
    (see the C header): logits [T, E] bf16, fp16 or fp32, its rows contiguous;
    topk_idx int64 and topk_weights fp32 [T, K] are written.  What
    ep_get_layout, the dispatch and the few-token layers take."""
    T, E = logits.shape
    K = topk_idx.shape[1]
    address, kind, stride, here = _rows_of(logits, (T, E), "logits")
    code = _lib.ep_route(address, kind, stride, _take(bias, torch.float32, (E,), "bias", here),
                         _mask(token_mask, T, here), T, E, K, score, num_groups,
                         num_groups if topk_groups is None else topk_groups, 1 if normalize else 0, scale,
                         _take(topk_idx, torch.int64, (T, K), "topk_idx", here),
                         _take(topk_weights, torch.float32, (T, K), "topk_weights", here), _word(d_status, here),
                         _stream(stream))
    return _check(code, "ep_route")


def ep_balance_loss_workspace_bytes(num_tokens, num_experts, num_sequences=1) -> int:
    return int(_lib.ep_balance_loss_workspace_bytes(num_tokens, num_experts, num_sequences))


def ep_balance_loss(logits, topk_idx, workspace, loss, load, d_status, score=EP_SCORE_SOFTMAX, token_mask=None,
                    seq_offset=None, coeff=1.0, num_tokens_per_expert=None, stream=None):
    """Balance loss of the router (see the C header), over all tokens or the
    mean over the sequences that seq_offset (int32 [S + 1]) cuts: loss fp32 [1],
    load fp32 [S, E] (its derivative by the normalised scores, for
    ep_route_backward) and num_tokens_per_expert int32 [S, E] are written."""
    f32 = torch.float32
    T, E = logits.shape
    K = topk_idx.shape[1]
    address, kind, stride, here = _rows_of(logits, (T, E), "logits")
    offsets, S = _sequences(seq_offset, here)
    code = _lib.ep_balance_loss(address, kind, stride, _take(topk_idx, torch.int64, (T, K), "topk_idx", here),
                                _mask(token_mask, T, here), offsets, T, E, K, S, score, coeff,
                                _take(loss, f32, (1,), "loss", here), _take(load, f32, (S, E), "load", here),
                                _take(num_tokens_per_expert, torch.int32, (S, E), "num_tokens_per_expert", here),
                                _take_any(workspace, "workspace", here), workspace.nbytes,
                                _word(d_status, here), _stream(stream))
    return _check(code, "ep_balance_loss")


def ep_route_backward(logits, topk_idx, d_logits, d_status, d_topk_weights=None, load=None, d_loss=None,
                      score=EP_SCORE_SOFTMAX, token_mask=None, seq_offset=None, normalize=True, scale=1.0, stream=None):
    """Gradient of the router's logits through the top-k weights
    (d_topk_weights fp32 [T, K]) and through the balance loss (load from
    ep_balance_loss, d_loss fp32 [1]), each where it is given (see the C
    header).  d_logits [T, E] of the logits' type is written."""
    f32 = torch.float32
    T, E = logits.shape
    K = topk_idx.shape[1]
    address, kind, stride, here = _rows_of(logits, (T, E), "logits")
    out, out_kind, out_stride, _ = _rows_of(d_logits, (T, E), "d_logits")
    assert out_kind == kind, "d_logits: the logits' type is wanted"
    offsets, S = _sequences(seq_offset, here)
    code = _lib.ep_route_backward(address, kind, stride, _take(topk_idx, torch.int64, (T, K), "topk_idx", here),
                                  _mask(token_mask, T, here), _take(d_topk_weights, f32, (T, K), "d_topk_weights", here),
                                  _take(load, f32, (S, E), "load", here), _take(d_loss, f32, (1,), "d_loss", here), offsets,
                                  T, E, K, S, score, 1 if normalize else 0, scale, out, out_stride,
                                  _word(d_status, here), _stream(stream))
    return _check(code, "ep_route_backward")


def _weights4(w, sf, zero, depth, name, here):
    """Addresses of 4-bit weights, their scales and zero points, the scales' type and the group."""
    E, n_w, half = w.shape
    assert half * 2 == depth and sf.dtype in (torch.bfloat16, torch.float32), "%s: codes [E, n_w, k / 2] are wanted" % name
    groups = sf.shape[1]
    assert groups > 0 and depth % groups == 0, "%s: scales [E, k / group, n_w] are wanted" % name
    shape = (E, groups, n_w)
    return (_take(w, torch.uint8, (E, n_w, half), name, here), _take(sf, sf.dtype, shape, name + "'s scales", here),
            _take(zero, sf.dtype, shape, name + "'s zero points", here), EP_FP32 if sf.dtype is torch.float32 else EP_BF16,
            depth // groups)


def ep_expert_gemm_w4(x, w, w_sf, expert_offset, num_tokens_per_expert, y, d_status, w_zero=None, w_format=EP_W4_INT,
                      bias=None, activation=EP_ACT_NONE, row_weight=None, residual=None, stream=None):
    """ep_expert_gemm with 4-bit weights for the rows of a decode step (see the C
    header): x [rows, k] bf16, w uint8 [E, n_w, k / 2] (two codes a byte, the
    even k's in the low half), w_sf and w_zero [E, k / group, n_w] bf16 or
    fp32, group 32, 64 or 128."""
    bf16, f32 = torch.bfloat16, torch.float32
    rows, k_dim = x.shape
    E, n_w, _ = w.shape
    gated = activation == EP_ACT_SWIGLU
    assert not gated or n_w % 2 == 0
    n_dim = n_w // 2 if gated else n_w
    here = _here(x, "x")
    codes, sf, zero, sf_kind, group = _weights4(w, w_sf, w_zero, k_dim, "w", here)
    first, count = _blocks(expert_offset, num_tokens_per_expert, E, here)
    code = _lib.ep_expert_gemm_w4(_take(x, bf16, (rows, k_dim), "x", here), codes, sf, zero, sf_kind, w_format, group,
                                  _take(bias, f32, (E, n_w), "bias", here), activation,
                                  _take(row_weight, f32, (rows,), "row_weight", here),
                                  _take(residual, bf16, (rows, n_dim), "residual", here), rows, k_dim, n_dim, E, first,
                                  count, _take(y, bf16, (rows, n_dim), "y", here), _word(d_status, here),
                                  _stream(stream))
    return _check(code, "ep_expert_gemm_w4")


def ep_moe_few_tokens_w4_workspace_bytes(num_tokens, num_topk, hidden, inner, num_experts) -> int:
    return int(_lib.ep_moe_few_tokens_w4_workspace_bytes(num_tokens, num_topk, hidden, inner, num_experts))


def ep_moe_few_tokens_w4(x, topk_idx, topk_weights, w_up, up_sf, w_down, down_sf, workspace, out, d_status, up_zero=None,
                         down_zero=None, w_format=EP_W4_INT, bias_up=None, bias_down=None, residual=None,
                         activation=EP_ACT_SWIGLU, stream=None):
    """ep_moe_few_tokens with 4-bit weights (see the C header): w_up uint8
    [E, n_w, H / 2], w_down uint8 [E, H, inner / 2], scales and zero points
    [E, H / group, n_w] and [E, inner / group, H], bf16 or fp32."""
    bf16, f32 = torch.bfloat16, torch.float32
    T, H = x.shape
    K = topk_idx.shape[1]
    E, n_w, _ = w_up.shape
    inner = w_down.shape[2] * 2
    assert n_w == (2 * inner if activation == EP_ACT_SWIGLU else inner) and w_down.shape[:2] == (E, H)
    assert up_sf.dtype is down_sf.dtype, "both scales are of one type"
    here = _here(x, "x")
    up, sf_up, zero_up, sf_kind, up_group = _weights4(w_up, up_sf, up_zero, H, "w_up", here)
    down, sf_down, zero_down, _, down_group = _weights4(w_down, down_sf, down_zero, inner, "w_down", here)
    code = _lib.ep_moe_few_tokens_w4(
        _take(x, bf16, (T, H), "x", here), _take(topk_idx, torch.int64, (T, K), "topk_idx", here),
        _take(topk_weights, f32, (T, K), "topk_weights", here), up, sf_up, zero_up, up_group,
        _take(bias_up, f32, (E, n_w), "bias_up", here), activation, down, sf_down, zero_down, down_group,
        _take(bias_down, f32, (E, H), "bias_down", here), sf_kind, w_format,
        _take(residual, bf16, (T, H), "residual", here), T, H, inner, K, E, _take_any(workspace, "workspace", here),
        workspace.nbytes, _take(out, bf16, (T, H), "out", here), _word(d_status, here), _stream(stream))
    return _check(code, "ep_moe_few_tokens_w4")
