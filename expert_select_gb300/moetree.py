"""Thin ctypes binding of libmoetree (include/moetree.h).

Argument marshalling only: every function takes torch tensors that already live
where the C ABI wants them (device or host), passes their data pointers, the
current CUDA stream and plain integers to the C entry point of the same name, and
raises MoeError on a non-zero status. All computation runs in the library's
kernels. The library is loaded from this package directory; if it is missing the
import of any entry point fails loudly (there is no fallback).
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional, Sequence

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoetree.so")

MOE_OK, MOE_ERR_ARG, MOE_ERR_CUDA, MOE_ERR_NOSLOT, MOE_ERR_TIMEOUT = 0, -1, -2, -3, -4
MOE_ERR_DEVICE_CHECK, MOE_ERR_UNSUPPORTED = -5, -6
MOE_DTYPE_F32, MOE_DTYPE_BF16 = 0, 1
MOE_ROUTE_NATURAL, MOE_ROUTE_ACCEPT, MOE_ROUTE_FIXED_B = 0, 1, 2
MOE_FFN_AUTO, MOE_FFN_SIMT, MOE_FFN_TCGEN05 = 0, 1, 2
MOE_MAX_DEPTHS = 16
MOE_INFO_FIELDS = 5

# Every function declared in include/moetree.h.
EXPORTS = (
    "moe_status_str", "moe_abi_version", "moe_workspace_bytes", "moe_router_logits",
    "moe_tree_select", "moe_expert_permute", "moe_expert_forward", "moe_tree_forward",
    "moe_workspace_check", "moe_residency_create", "moe_residency_destroy",
    "moe_residency_query", "moe_residency_plan", "moe_residency_publish", "moe_expert_upload",
    "moe_event_wait", "moe_tree_forward_noalloc", "moe_offload_forward", "moe_draft_select",
    "moe_tree_route", "moe_tree_block_stats", "moe_noalloc_check", "moe_offload_upload_wait",
    "moe_rms_norm", "moe_attention_workspace_bytes", "moe_tree_attention", "moe_kv_append",
    "moe_kv_commit", "moe_block_norm", "moe_few_workspace_bytes", "moe_few_forward", "moe_sample",
    "moe_tree_accept", "moe_pages_workspace_bytes", "moe_kv_reserve", "moe_kv_free", "moe_kv_fork",
    "moe_kv_compact", "moe_kv_copy_pages",
)


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_str(status)} ({status})")
        self.status = status


class LayerDesc(C.Structure):
    _fields_ = [("d", C.c_int), ("E", C.c_int), ("k", C.c_int), ("f", C.c_int), ("dtype", C.c_int),
                ("slots", C.c_int)]


class SelectParams(C.Structure):
    _fields_ = [("mode", C.c_int), ("n_c", C.c_int), ("c_by_depth", C.c_double * MOE_MAX_DEPTHS),
                ("pool_all", C.c_int), ("anchor", C.c_int), ("prune", C.c_int),
                ("reroute_budget", C.c_int), ("min_set", C.c_int), ("fixed_B", C.c_int)]


class TreeOutputs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in
                ("logits", "topk_idx", "gates", "eligible", "info", "counts", "offsets", "perm")]


class OffloadStats(C.Structure):
    _fields_ = [("needed", C.c_int), ("hits", C.c_int), ("uploads", C.c_int),
                ("passes", C.c_int), ("h2d_bytes", C.c_longlong)]


class TreeStats(C.Structure):
    _fields_ = [("trees", C.c_int), ("assignments", C.c_int), ("union_experts", C.c_int),
                ("max_per_expert", C.c_int), ("reuse", C.c_double),
                ("union_nat_mean", C.c_double), ("union_sel_mean", C.c_double),
                ("m_mean", C.c_double), ("pruned_mean", C.c_double), ("exact_trees", C.c_int)]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class RunOpts(C.Structure):
    _fields_ = [("ffn_path", C.c_int), ("ffn_begin", C.c_void_p), ("ffn_end", C.c_void_p),
                ("residual", C.c_int), ("select_begin", C.c_void_p), ("norm_input", C.c_int),
                ("ffn_max_ctas", C.c_int)]


class CacheDesc(C.Structure):
    _fields_ = [("H", C.c_int), ("H_kv", C.c_int), ("dh", C.c_int), ("dtype", C.c_int),
                ("page_size", C.c_int), ("n_pages", C.c_int), ("max_pages", C.c_int),
                ("stride_page", C.c_longlong), ("stride_tok", C.c_longlong),
                ("stride_head", C.c_longlong), ("window", C.c_int), ("sink_tokens", C.c_int),
                ("scale", C.c_float)]


class RopeParams(C.Structure):
    _fields_ = [("q_weight", C.c_void_p), ("k_weight", C.c_void_p), ("eps", C.c_float),
                ("inv_freq", C.c_void_p), ("rot_dim", C.c_int), ("rope_scale", C.c_float)]


class SampleParams(C.Structure):
    _fields_ = [("V", C.c_int), ("dtype", C.c_int), ("param_rows", C.c_int),
                ("temperature", C.c_void_p), ("top_k", C.c_void_p), ("top_p", C.c_void_p),
                ("min_p", C.c_void_p)]


class PageBook(C.Structure):
    _fields_ = [("page_table", C.c_void_p), ("held", C.c_void_p), ("cache_len", C.c_void_p),
                ("ref", C.c_void_p), ("B", C.c_int), ("max_pages", C.c_int), ("n_pages", C.c_int),
                ("page_size", C.c_int)]


_lib = None


def lib() -> C.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run __graft_entry__.build() "
                               "(the CUDA library is required; there is no fallback)")
        L = C.CDLL(LIB_PATH)
        P, I, S = C.c_void_p, C.c_int, C.c_size_t
        sig = {
            "moe_status_str": ([I], C.c_char_p),
            "moe_abi_version": ([], I),
            "moe_workspace_bytes": ([P, I, I], S),
            "moe_router_logits": ([P, P, P, I, P, P], I),
            "moe_rms_norm": ([P, P, I, P, P], I),
            "moe_tree_select": ([P, P, P, P, I, I, P, P, P, P, P, P], I),
            "moe_expert_permute": ([P, P, I, P, P, P, P, P], I),
            "moe_expert_forward": ([P, P, P, P, P, P, P, P, I, P, P, P, P], I),
            "moe_tree_forward": ([P, P, P, P, P, P, P, P, P, I, I, P, P, P, P, P, P], I),
            "moe_workspace_check": ([P, P, P], I),
            "moe_residency_create": ([I, I, I, P], I),
            "moe_residency_destroy": ([P], I),
            "moe_residency_query": ([P, I, P, P], I),
            "moe_residency_plan": ([P, I, P, I, P, P, P, P], I),
            "moe_residency_publish": ([P, I, P, P, P], I),
            "moe_expert_upload": ([P, P, P, P, P, P, P, P, P, I, P, P], I),
            "moe_event_wait": ([P, C.c_double], I),
            "moe_tree_forward_noalloc": ([P, P, P, P, P, P, P, P, P, I, I, P, P, P, P, P], I),
            "moe_offload_forward": ([P, P, P, P, P, P, P, P, P, P, P, I, P, I, I, P, P, P, P, P,
                                     P, P], I),
            "moe_draft_select": ([P, I, P, P, P, P, C.c_float, I, P, P, P, P, P, P, P], I),
            "moe_tree_route": ([P, P, P, P, P, I, I, P, P, P, P, P, P, P], I),
            "moe_tree_block_stats": ([P, I, I, P, P, P, P, P], I),
            "moe_noalloc_check": ([P, P], I),
            "moe_offload_upload_wait": ([P, I, C.c_double, P, P], I),
            "moe_attention_workspace_bytes": ([P, I, I], S),
            "moe_tree_attention": ([P, P, C.c_longlong, P, P, P, P, P, P, P, I, I, I, P, P, P, P],
                                   I),
            "moe_kv_append": ([P, P, P, C.c_longlong, P, C.c_longlong, P, C.c_longlong, P, P, P, P,
                               P, P, I, I, I, P, P, P], I),
            "moe_kv_commit": ([P, P, P, P, P, P, P, I, I, P, P, P], I),
            "moe_block_norm": ([P, P, P, P, P, I, C.c_float, P, C.c_float, I, P, P, P], I),
            "moe_few_workspace_bytes": ([P, I], S),
            "moe_few_forward": ([P, P, P, P, P, P, P, I, P, P, P, P, P, P, P], I),
            "moe_sample": ([P, P, C.c_longlong, P, I, P, P, P], I),
            "moe_tree_accept": ([P, P, P, P, I, I, I, I, P, P, P, P], I),
            "moe_pages_workspace_bytes": ([P], S),
            "moe_kv_reserve": ([P, I, P, P, P], I),
            "moe_kv_free": ([P, P, P, I, P, P], I),
            "moe_kv_fork": ([P, P, P, I, P, P, P], I),
            "moe_kv_compact": ([P, P, P, P, P, P, P], I),
            "moe_kv_copy_pages": ([P, P, P, P, I, P, P, P], I),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def status_str(status: int) -> str:
    return lib().moe_status_str(status).decode()


def _check(fn: str, status: int) -> int:
    if status != MOE_OK:
        raise MoeError(fn, status)
    return status


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def layer_desc(d: int, E: int, k: int, f: int, dtype, slots: int = 0) -> LayerDesc:
    """slots: expert slots in the weight pools (0 = E, one slot per expert)."""
    code = MOE_DTYPE_BF16 if dtype in (torch.bfloat16, "bf16") else MOE_DTYPE_F32
    return LayerDesc(d, E, k, f, code, slots)


def select_params(mode: int = MOE_ROUTE_ACCEPT, c: Sequence[float] = (1.0,), pool_all=False,
                  anchor=True, prune=False, reroute_budget=8, min_set=16, fixed_B=0) -> SelectParams:
    p = SelectParams()
    p.mode = mode
    p.n_c = len(c)
    for i, v in enumerate(c):
        p.c_by_depth[i] = float(v)
    p.pool_all, p.anchor, p.prune = int(pool_all), int(anchor), int(prune)
    p.reroute_budget, p.min_set, p.fixed_B = reroute_budget, min_set, fixed_B
    return p


def moe_workspace_bytes(L: LayerDesc, B: int, N: int) -> int:
    return int(lib().moe_workspace_bytes(C.byref(L), B, N))


def workspace(L: LayerDesc, B: int, N: int, device="cuda") -> torch.Tensor:
    """A device byte buffer of moe_workspace_bytes (torch allocations are 256-B aligned)."""
    n = moe_workspace_bytes(L, B, N)
    if n == 0:
        raise MoeError("moe_workspace_bytes", MOE_ERR_ARG)
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_router_logits(L, x, W_r, logits, stream=None):
    return _check("moe_router_logits", lib().moe_router_logits(
        C.byref(L), _ptr(x), _ptr(W_r), x.shape[0], _ptr(logits), _stream(stream)))


def moe_rms_norm(L, x, xn, stream=None):
    return _check("moe_rms_norm", lib().moe_rms_norm(
        C.byref(L), _ptr(x), x.shape[0], _ptr(xn), _stream(stream)))


def moe_tree_select(L, P, logits, depth, B, N, resident, topk_idx, gates, eligible=None,
                    info=None, stream=None):
    return _check("moe_tree_select", lib().moe_tree_select(
        C.byref(L), C.byref(P), _ptr(logits), _ptr(depth), B, N, _ptr(resident), _ptr(topk_idx),
        _ptr(gates), _ptr(eligible), _ptr(info), _stream(stream)))


def moe_tree_route(L, P, x, W_r, depth, B, N, resident, logits, topk_idx, gates, eligible=None,
                   info=None, stream=None):
    return _check("moe_tree_route", lib().moe_tree_route(
        C.byref(L), C.byref(P), _ptr(x), _ptr(W_r), _ptr(depth), B, N, _ptr(resident),
        _ptr(logits), _ptr(topk_idx), _ptr(gates), _ptr(eligible), _ptr(info), _stream(stream)))


def moe_tree_block_stats(L, B, N, info=None, counts=None, ws=None, stream=None) -> TreeStats:
    """Counters of the last block (union, reuse, per-tree set sizes); waits for the stream."""
    st = TreeStats()
    _check("moe_tree_block_stats", lib().moe_tree_block_stats(
        C.byref(L), B, N, _ptr(info), _ptr(counts), _ptr(ws), C.byref(st), _stream(stream)))
    return st


def moe_expert_permute(L, topk_idx, counts, offsets, perm, ws, stream=None):
    return _check("moe_expert_permute", lib().moe_expert_permute(
        C.byref(L), _ptr(topk_idx), topk_idx.shape[0], _ptr(counts), _ptr(offsets), _ptr(perm),
        _ptr(ws), _stream(stream)))


def _event(ev):
    if ev is None:
        return None
    if not ev.cuda_event:
        raise ValueError("torch.cuda.Event has no CUDA event yet: record it once first")
    return C.c_void_p(ev.cuda_event)


def run_opts(ffn_path: int = MOE_FFN_AUTO, begin=None, end=None, residual=False,
             select_begin=None, norm_input=False, ffn_max_ctas: int = 0) -> RunOpts:
    """Options for the forward entry points. `begin`/`end` are torch.cuda.Event
    objects recorded around the grouped-expert kernel, `select_begin` one recorded before
    the selection launch; `residual` returns x + MoE(x); `norm_input` routes and computes
    the experts on the RMS pre-norm of x (the residual still adds x); `ffn_max_ctas` caps
    the tensor-core expert kernel's CTAs (0: one per SM)."""
    return RunOpts(ffn_path, _event(begin), _event(end), int(residual), _event(select_begin),
                   int(norm_input), int(ffn_max_ctas))


def moe_expert_forward(L, x, W_gate, W_up, W_down, slot_of_expert, topk_idx, gates, y, ws,
                       opts: Optional[RunOpts] = None, stream=None):
    return _check("moe_expert_forward", lib().moe_expert_forward(
        C.byref(L), _ptr(x), _ptr(W_gate), _ptr(W_up), _ptr(W_down), _ptr(slot_of_expert),
        _ptr(topk_idx), _ptr(gates), x.shape[0], _ptr(y), _ptr(ws),
        None if opts is None else C.byref(opts), _stream(stream)))


def tree_outputs(**tensors) -> TreeOutputs:
    o = TreeOutputs()
    for k, v in tensors.items():
        setattr(o, k, None if v is None else v.data_ptr())
    return o


def moe_tree_forward(L, P, x, W_r, W_gate, W_up, W_down, slot_of_expert, depth, B, N, resident,
                     y, ws, out: Optional[TreeOutputs] = None, opts: Optional[RunOpts] = None,
                     stream=None):
    return _check("moe_tree_forward", lib().moe_tree_forward(
        C.byref(L), C.byref(P), _ptr(x), _ptr(W_r), _ptr(W_gate), _ptr(W_up), _ptr(W_down),
        _ptr(slot_of_expert), _ptr(depth), B, N, _ptr(resident), _ptr(y),
        None if out is None else C.byref(out), _ptr(ws),
        None if opts is None else C.byref(opts), _stream(stream)))


def moe_tree_forward_noalloc(L, P, x, W_r, W_gate, W_up, W_down, slot_of_expert, depth, B, N,
                             resident, y, out: Optional[TreeOutputs] = None,
                             opts: Optional[RunOpts] = None, stream=None):
    """moe_tree_forward with the library's built-in 16 MiB scratch instead of a
    caller-allocated workspace (for callers that cannot allocate device memory)."""
    return _check("moe_tree_forward_noalloc", lib().moe_tree_forward_noalloc(
        C.byref(L), C.byref(P), _ptr(x), _ptr(W_r), _ptr(W_gate), _ptr(W_up), _ptr(W_down),
        _ptr(slot_of_expert), _ptr(depth), B, N, _ptr(resident), _ptr(y),
        None if out is None else C.byref(out), None if opts is None else C.byref(opts),
        _stream(stream)))


def moe_workspace_check(ws, stream=None) -> int:
    flags = C.c_int(0)
    st = lib().moe_workspace_check(_ptr(ws), C.byref(flags), _stream(stream))
    if st not in (MOE_OK, MOE_ERR_DEVICE_CHECK):
        raise MoeError("moe_workspace_check", st)
    return flags.value


def moe_noalloc_check(stream=None) -> int:
    """Reads and clears the check word of moe_tree_forward_noalloc's built-in scratch."""
    flags = C.c_int(0)
    st = lib().moe_noalloc_check(C.byref(flags), _stream(stream))
    if st not in (MOE_OK, MOE_ERR_DEVICE_CHECK):
        raise MoeError("moe_noalloc_check", st)
    return flags.value


class Residency:
    """Owner of a moe_residency table (host metadata of the expert slots)."""

    def __init__(self, n_layers: int, E: int, slots: int):
        self.E, self.slots = E, slots
        h = C.c_void_p()
        _check("moe_residency_create", lib().moe_residency_create(n_layers, E, slots, C.byref(h)))
        self.h = h

    def close(self):
        if self.h:
            lib().moe_residency_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def query(self, layer: int):
        import numpy as np
        slot = np.empty(self.E, dtype=np.int32)
        res = np.empty(self.E, dtype=np.uint8)
        _check("moe_residency_query", lib().moe_residency_query(
            self.h, layer, slot.ctypes.data_as(C.c_void_p), res.ctypes.data_as(C.c_void_p)))
        return slot, res

    def plan(self, layer: int, needed):
        import numpy as np
        nd = np.ascontiguousarray(np.asarray(needed, dtype=np.int32))
        ue = np.empty(max(1, len(nd)), dtype=np.int32)
        us = np.empty(max(1, len(nd)), dtype=np.int32)
        n_up, hits = C.c_int(0), C.c_int(0)
        _check("moe_residency_plan", lib().moe_residency_plan(
            self.h, layer, nd.ctypes.data_as(C.c_void_p), len(nd), ue.ctypes.data_as(C.c_void_p),
            us.ctypes.data_as(C.c_void_p), C.byref(n_up), C.byref(hits)))
        return ue[:n_up.value].copy(), us[:n_up.value].copy(), hits.value

    def upload_wait(self, layer: int, timeout_s: float = 10.0):
        """(ms the compute stream waited for uploads, number of waits) in the last
        moe_offload_forward call on `layer`."""
        ms, n = C.c_double(0), C.c_int(0)
        _check("moe_offload_upload_wait", lib().moe_offload_upload_wait(
            self.h, layer, float(timeout_s), C.byref(ms), C.byref(n)))
        return ms.value, n.value

    def publish(self, layer: int, slot_dev=None, res_dev=None, stream=None):
        _check("moe_residency_publish", lib().moe_residency_publish(
            self.h, layer, _ptr(slot_dev), _ptr(res_dev), _stream(stream)))


def moe_expert_upload(L, host_gate, host_up, host_down, slot_gate, slot_up, slot_down,
                      up_expert, up_slot, side_stream, done_event=None):
    import numpy as np
    ue = np.ascontiguousarray(np.asarray(up_expert, dtype=np.int32))
    us = np.ascontiguousarray(np.asarray(up_slot, dtype=np.int32))
    return _check("moe_expert_upload", lib().moe_expert_upload(
        C.byref(L), _ptr(host_gate), _ptr(host_up), _ptr(host_down), _ptr(slot_gate),
        _ptr(slot_up), _ptr(slot_down), ue.ctypes.data_as(C.c_void_p),
        us.ctypes.data_as(C.c_void_p), len(ue), C.c_void_p(side_stream.cuda_stream),
        _event(done_event)))


def moe_offload_forward(L, P, x, W_r, host_gate, host_up, host_down, slot_gate, slot_up,
                        slot_down, table: "Residency", layer: int, depth, B, N, y, ws,
                        out: Optional[TreeOutputs] = None, opts: Optional[RunOpts] = None,
                        stream=None, side_stream=None) -> OffloadStats:
    """The layer with offloaded experts; returns the call's OffloadStats."""
    st = OffloadStats()
    side = side_stream if side_stream is not None else torch.cuda.current_stream()
    _check("moe_offload_forward", lib().moe_offload_forward(
        C.byref(L), C.byref(P), _ptr(x), _ptr(W_r), _ptr(host_gate), _ptr(host_up),
        _ptr(host_down), _ptr(slot_gate), _ptr(slot_up), _ptr(slot_down), table.h, layer,
        _ptr(depth), B, N, _ptr(y), None if out is None else C.byref(out), C.byref(st), _ptr(ws),
        None if opts is None else C.byref(opts), _stream(stream), C.c_void_p(side.cuda_stream)))
    return st


def moe_draft_select(L, parent, depth, logp, footprint, lam: float, gamma: int, selected,
                     sel_parent, sel_depth, x=None, x_sel=None, n_union=None, stream=None):
    """Cost-aware choice of the draft tree to verify (see include/moetree.h)."""
    return _check("moe_draft_select", lib().moe_draft_select(
        C.byref(L), parent.shape[0], _ptr(parent), _ptr(depth), _ptr(logp), _ptr(footprint),
        float(lam), gamma, _ptr(x), _ptr(selected), _ptr(sel_parent), _ptr(sel_depth),
        _ptr(x_sel), _ptr(n_union), _stream(stream)))


# ------------------------------------------------------------- attention half of the block

_CODE = {torch.float32: MOE_DTYPE_F32, torch.bfloat16: MOE_DTYPE_BF16}
_TORCH = {v: k for k, v in _CODE.items()}


def _refuse(fn: str, name: str, t: torch.Tensor, dtype, shape, index, dense=True):
    """Says why a tensor is not what its pointer would be taken for."""
    if t.dtype != dtype:
        raise ValueError(f"{fn}: {name} is {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != index:
        raise ValueError(f"{fn}: {name} is on {t.device}, the first tensor on device {index}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be contiguous")


def _dense(fn, name, t, dtype, shape, index):
    """Refuses a tensor (None passes) of another type, shape, device or layout. One expression, as
    it runs for every argument of every call."""
    if t is not None and not (t.dtype is dtype and t.shape == shape and t.get_device() == index and
                              t.is_contiguous()):
        _refuse(fn, name, t, dtype, shape, index)


def _rows(fn, name, t, dtype, shape, index) -> int:
    """A [rows, heads, dh] tensor whose rows may be a part of wider ones; its row stride."""
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == index):
        _refuse(fn, name, t, dtype, shape, index, dense=False)
    ld, head, one = t.stride()
    n, heads, dh = shape
    if n == 0:
        return heads * dh
    if one != 1 or (heads > 1 and head != dh):
        raise ValueError(f"{fn}: the heads of {name}'s rows must lie side by side")
    return ld if n > 1 else heads * dh  # (a single row has no stride to speak of)


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else None
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_entry = {}  # entry points by name, looked up once


def _run(fn: str, index: int, stream, *args) -> int:
    """Calls entry point `fn` on device `index`, on `stream` or the device's current one."""
    call = _entry.get(fn)
    if call is None:
        call = _entry[fn] = getattr(lib(), fn)
    if index < 0:
        raise ValueError(f"{fn}: the tensors must be on a CUDA device")
    if _device() == index:
        st = call(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(index):
            st = call(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    if st != MOE_OK:
        raise MoeError(fn, st)
    return st


def cache_desc(pages: torch.Tensor, H: int, max_pages: int, window: int = 0, sink_tokens: int = 0,
               scale: Optional[float] = None) -> CacheDesc:
    """The cache of one layer whose K pool is `pages`, [n_pages, page_size, H_kv, dh] or a view
    with those dimensions (a head-major pool is one, permuted); the V pool has the same shape
    and strides. H: query heads; max_pages: entries of a page-table row; window, sink_tokens:
    see moe_cache_desc; scale: of q.k, 1 / sqrt(dh) if not given."""
    n, page, h_kv, dh = pages.shape
    if pages.dtype not in _CODE:
        raise ValueError(f"cache_desc: pages are {pages.dtype}, expected float32 or bfloat16")
    if dh > 1 and pages.stride(3) != 1:
        raise ValueError("cache_desc: a head's elements must lie side by side")
    st = [pages.stride(i) if pages.shape[i] > 1 else max(pages.stride(i), dh) for i in range(3)]
    st = [v if pages.shape[i] > 1 else (v + 7) // 8 * 8 for i, v in enumerate(st)]
    return CacheDesc(H, h_kv, dh, _CODE[pages.dtype], page, n, max_pages, *st, window, sink_tokens,
                     dh ** -0.5 if scale is None else scale)


def _like_cache(fn, C_, k_pages, v_pages, index, dt):
    """Refuses pools that are not what the cache's description says."""
    shape = (C_.n_pages, C_.page_size, C_.H_kv, C_.dh)
    st = (C_.stride_page, C_.stride_tok, C_.stride_head, 1)
    if not (k_pages.dtype is dt and k_pages.shape == shape and k_pages.stride() == st and
            v_pages.dtype is dt and v_pages.shape == shape and v_pages.stride() == st and
            v_pages.get_device() == index):
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            _refuse(fn, name, t, dt, shape, index, dense=False)
            # (a dimension of one element has no stride to speak of)
            if any(n > 1 and x != y for n, x, y in zip(shape, t.stride(), st)):
                raise ValueError(f"{fn}: {name} has other strides than the cache description")


def _pools(fn, C_, k_pages, v_pages, page_table, cache_len, B, row_start):
    """Checks the cache's tensors against its description; the device index and type."""
    index, dt = k_pages.get_device(), _TORCH[C_.dtype]
    _like_cache(fn, C_, k_pages, v_pages, index, dt)
    i32 = torch.int32
    _dense(fn, "page_table", page_table, i32, (B, C_.max_pages), index)
    _dense(fn, "cache_len", cache_len, i32, (B,), index)
    if row_start is not None:
        _dense(fn, "row_start", row_start, i32, (B + 1,), index)
    return index, dt


def _scratch(fn, ws, index, need):
    if ws is not None and not (ws.dtype is torch.uint8 and ws.get_device() == index and
                               ws.is_contiguous() and ws.numel() >= need):
        _refuse(fn, "workspace", ws, torch.uint8, None, index)
        raise ValueError(f"{fn}: the workspace has {ws.numel()} bytes, expected {need} or more")


def moe_attention_workspace_bytes(C_: CacheDesc, B: int, N: int) -> int:
    return int(lib().moe_attention_workspace_bytes(C.byref(C_), B, N))


def attention_workspace(C_: CacheDesc, B: int, N: int, device="cuda") -> torch.Tensor:
    """A device byte buffer of moe_attention_workspace_bytes whose head is zeroed."""
    n = moe_attention_workspace_bytes(C_, B, N)
    if n == 0:
        raise MoeError("moe_attention_workspace_bytes", MOE_ERR_ARG)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:4096].zero_()
    return ws


def moe_tree_attention(C_, q, k_pages, v_pages, page_table, cache_len, B, N, out, ws, parent=None,
                       row_start=None, sink_logit=None, lse=None, stream=None):
    """Attention of a block's nodes over the paged cache (see include/moetree.h). q, out
    [R, H, dh]; pools as given to cache_desc."""
    fn, R, H = "moe_tree_attention", q.shape[0], C_.H
    index, dt = _pools(fn, C_, k_pages, v_pages, page_table, cache_len, B, row_start)
    shape = (R, H, C_.dh)
    ldq = _rows(fn, "q", q, dt, shape, index)
    _dense(fn, "out", out, dt, shape, index)
    if parent is not None:
        _dense(fn, "parent", parent, torch.int32, (R,), index)
    if sink_logit is not None:
        _dense(fn, "sink_logit", sink_logit, torch.float32, (H,), index)
    if lse is not None:
        _dense(fn, "lse", lse, torch.float32, (R, H), index)
    desc = C.byref(C_)
    if B > 0 and N > 0:
        if ws is None:
            raise ValueError(f"{fn}: it needs a workspace")
        _scratch(fn, ws, index, _lib.moe_attention_workspace_bytes(desc, B, N) if _lib else
                 moe_attention_workspace_bytes(C_, B, N))
    return _run(fn, index, stream, desc, q.data_ptr(), ldq, k_pages.data_ptr(),
                v_pages.data_ptr(), page_table.data_ptr(), cache_len.data_ptr(), _at(row_start),
                _at(parent), _at(sink_logit), B, N, R, out.data_ptr(), _at(lse), _at(ws))


def moe_kv_append(C_, q, k, v, k_pages, v_pages, page_table, cache_len, B, N, q_out, ws=None,
                  depth=None, row_start=None, inv_freq=None, rope_scale=1.0, q_weight=None,
                  k_weight=None, eps=1e-6, stream=None):
    """Writes a block's k and v to the cache and rotates its q (see include/moetree.h). q, k, v
    [R, heads, dh] may be parts of one projection's rows; q and q_out may both be None."""
    fn, R, dh = "moe_kv_append", k.shape[0], C_.dh
    index, dt = _pools(fn, C_, k_pages, v_pages, page_table, cache_len, B, row_start)
    ldq = 0
    if q is not None:
        ldq = _rows(fn, "q", q, dt, (R, C_.H, dh), index)
        _dense(fn, "q_out", q_out, dt, (R, C_.H, dh), index)
    kv = (R, C_.H_kv, dh)
    ldk, ldv = _rows(fn, "k", k, dt, kv, index), _rows(fn, "v", v, dt, kv, index)
    if depth is not None:
        _dense(fn, "depth", depth, torch.int32, (R,), index)
    rot = 0
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        _dense(fn, "inv_freq", inv_freq, torch.float32, inv_freq.shape, index)
    if q_weight is not None:
        _dense(fn, "q_weight", q_weight, dt, (dh,), index)
    if k_weight is not None:
        _dense(fn, "k_weight", k_weight, dt, (dh,), index)
    _scratch(fn, ws, index, 4096)
    P = RopeParams(_at(q_weight), _at(k_weight), eps, _at(inv_freq), rot, rope_scale)
    return _run(fn, index, stream, C.byref(C_), C.byref(P), _at(q), ldq, k.data_ptr(), ldk,
                v.data_ptr(), ldv, k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
                cache_len.data_ptr(), _at(row_start), _at(depth), B, N, R, _at(q_out), _at(ws))


def moe_kv_commit(C_, k_pages, v_pages, page_table, cache_len, path, n_accept, new_len, ws=None,
                  stream=None):
    """Moves each sequence's accepted path to the front of its block (see include/moetree.h).
    path [B, P], n_accept [B], new_len [B] (may be cache_len), all int32 on the device."""
    fn = "moe_kv_commit"
    B, P = path.shape
    index, _ = _pools(fn, C_, k_pages, v_pages, page_table, cache_len, B, None)
    _dense(fn, "path", path, torch.int32, (B, P), index)
    _dense(fn, "n_accept", n_accept, torch.int32, (B,), index)
    _dense(fn, "new_len", new_len, torch.int32, (B,), index)
    _scratch(fn, ws, index, 4096)
    return _run(fn, index, stream, C.byref(C_), k_pages.data_ptr(), v_pages.data_ptr(),
                page_table.data_ptr(), cache_len.data_ptr(), path.data_ptr(), n_accept.data_ptr(),
                B, P, new_len.data_ptr(), _at(ws))


def moe_block_norm(L, x, branch=None, h=None, hn=None, w_post=None, gate=None, gate_rows=0,
                   scale=1.0, w_pre=None, eps=1e-6, stream=None):
    """The norms and the residual between the halves of a block (see include/moetree.h):
    h = x + scale * gate * norm(branch), hn = norm(h), both [R, d]."""
    fn, d, dt, index = "moe_block_norm", L.d, _TORCH[L.dtype], x.get_device()
    R = x.shape[0]
    shape = (R, d)
    _dense(fn, "x", x, dt, shape, index)
    _dense(fn, "branch", branch, dt, shape, index)
    _dense(fn, "h", h, dt, shape, index)
    _dense(fn, "hn", hn, dt, shape, index)
    _dense(fn, "w_post", w_post, dt, (d,), index)
    _dense(fn, "w_pre", w_pre, dt, (d,), index)
    if gate is not None:
        if gate_rows < 1:
            raise ValueError(f"{fn}: gate_rows is {gate_rows}, expected the rows of a gate row")
        _dense(fn, "gate", gate, dt, (-(-R // gate_rows), d), index)
    return _run(fn, index, stream, C.byref(L), x.data_ptr(), _at(branch), _at(w_post), _at(gate),
                gate_rows, scale, _at(w_pre), eps, R, _at(h), _at(hn))


# ------------------------------------------------------------- a decoding round's other calls

MOE_FEW_HEAD_BYTES = 36864


def _zeroed(n: int, device, head: int = 4096) -> torch.Tensor:
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:head].zero_()
    return ws


def moe_few_workspace_bytes(L: LayerDesc, R: int) -> int:
    return int(lib().moe_few_workspace_bytes(C.byref(L), R))


def few_workspace(L: LayerDesc, R: int, device="cuda") -> torch.Tensor:
    """A device byte buffer of moe_few_workspace_bytes whose head is zeroed."""
    n = moe_few_workspace_bytes(L, R)
    if n == 0:
        raise MoeError("moe_few_workspace_bytes", MOE_ERR_ARG)
    return _zeroed(n, device, MOE_FEW_HEAD_BYTES)


def moe_few_forward(L, x, W_r, W_gate, W_up, W_down, slot_of_expert, y, ws, logits=None,
                    topk_idx=None, gates=None, opts: Optional[RunOpts] = None, stream=None):
    """The whole layer for up to 16 tokens in one launch (see include/moetree.h). x, y [R, d]; ws
    from few_workspace."""
    fn, R, d, f, dt = "moe_few_forward", x.shape[0], L.d, L.f, _TORCH[L.dtype]
    index, S = x.get_device(), L.slots if L.slots > 0 else L.E
    _dense(fn, "x", x, dt, (R, d), index)
    _dense(fn, "y", y, dt, (R, d), index)
    _dense(fn, "W_r", W_r, dt, (L.E, d), index)
    _dense(fn, "W_gate", W_gate, dt, (S, f, d), index)
    _dense(fn, "W_up", W_up, dt, (S, f, d), index)
    _dense(fn, "W_down", W_down, dt, (S, d, f), index)
    _dense(fn, "slot_of_expert", slot_of_expert, torch.int32, (L.E,), index)
    _dense(fn, "logits", logits, torch.float32, (R, L.E), index)
    _dense(fn, "topk_idx", topk_idx, torch.int32, (R, L.k), index)
    _dense(fn, "gates", gates, torch.float32, (R, L.k), index)
    desc = C.byref(L)
    if 0 < R <= 16:
        if ws is None:
            raise ValueError(f"{fn}: it needs a workspace")
        _scratch(fn, ws, index, lib().moe_few_workspace_bytes(desc, R))
    return _run(fn, index, stream, desc, x.data_ptr(), W_r.data_ptr(), W_gate.data_ptr(),
                W_up.data_ptr(), W_down.data_ptr(), _at(slot_of_expert), R, y.data_ptr(),
                _at(logits), _at(topk_idx), _at(gates), _at(ws),
                None if opts is None else C.byref(opts))


def moe_sample(logits, u, token, temperature=None, top_k=None, top_p=None, min_p=None,
               param_rows: int = 1, logprob=None, stream=None):
    """Samples a token from each row of logits [R, V] (rows may be a part of wider ones) at the
    random numbers u [R] (see include/moetree.h). temperature, top_k (int32), top_p, min_p
    [ceil(R / param_rows)] on the device, or None."""
    fn, index = "moe_sample", logits.get_device()
    R, V = logits.shape
    code = _CODE.get(logits.dtype)
    if code is None:
        raise ValueError(f"{fn}: logits are {logits.dtype}, expected float32 or bfloat16")
    if V > 1 and logits.stride(1) != 1:
        raise ValueError(f"{fn}: a row's logits must lie side by side")
    if param_rows < 1:
        raise ValueError(f"{fn}: param_rows is {param_rows}, expected the rows of an entry")
    ld = logits.stride(0) if R > 1 else V
    f32, n = torch.float32, (-(-R // param_rows),)
    _dense(fn, "u", u, f32, (R,), index)
    _dense(fn, "token", token, torch.int32, (R,), index)
    _dense(fn, "logprob", logprob, f32, (R,), index)
    _dense(fn, "temperature", temperature, f32, n, index)
    _dense(fn, "top_k", top_k, torch.int32, n, index)
    _dense(fn, "top_p", top_p, f32, n, index)
    _dense(fn, "min_p", min_p, f32, n, index)
    P = SampleParams(V, code, param_rows, _at(temperature), _at(top_k), _at(top_p), _at(min_p))
    return _run(fn, index, stream, C.byref(P), logits.data_ptr(), ld, u.data_ptr(), R,
                token.data_ptr(), _at(logprob))


def moe_tree_accept(token, parent, sampled, B, N, path, n_accept, emitted=None, row_start=None,
                    stream=None):
    """Follows the sampled tokens through B draft trees (see include/moetree.h). token, parent (or
    None: chains), sampled [R]; path, emitted [B, P]; n_accept [B]; all int32."""
    fn, i32, R, index = "moe_tree_accept", torch.int32, token.shape[0], path.get_device()
    P = path.shape[1]
    _dense(fn, "token", token, i32, (R,), index)
    _dense(fn, "parent", parent, i32, (R,), index)
    _dense(fn, "sampled", sampled, i32, (R,), index)
    _dense(fn, "row_start", row_start, i32, (B + 1,), index)
    _dense(fn, "path", path, i32, (B, P), index)
    _dense(fn, "n_accept", n_accept, i32, (B,), index)
    _dense(fn, "emitted", emitted, i32, (B, P), index)
    return _run(fn, index, stream, token.data_ptr(), _at(parent), sampled.data_ptr(),
                _at(row_start), B, N, R, P, path.data_ptr(), n_accept.data_ptr(), _at(emitted))


def page_book(page_table, held, cache_len, ref, page_size: int) -> PageBook:
    """The book of a cache's pages (see moe_page_book): page_table [B, max_pages], held [B],
    cache_len [B], ref [n_pages], int32 on one device. It keeps the tensors alive."""
    fn, i32, index = "page_book", torch.int32, page_table.get_device()
    B, width = page_table.shape
    _dense(fn, "page_table", page_table, i32, (B, width), index)
    _dense(fn, "held", held, i32, (B,), index)
    _dense(fn, "cache_len", cache_len, i32, (B,), index)
    _dense(fn, "ref", ref, i32, (ref.numel(),), index)
    K = PageBook(page_table.data_ptr(), held.data_ptr(), cache_len.data_ptr(), ref.data_ptr(), B,
                 width, ref.numel(), page_size)
    K.tensors, K.index, K.desc = (page_table, held, cache_len, ref), index, C.byref(K)
    K.need = None  # bytes of workspace, asked for once
    return K


def moe_pages_workspace_bytes(K: PageBook) -> int:
    return int(lib().moe_pages_workspace_bytes(C.byref(K)))


def pages_workspace(K: PageBook, device=None) -> torch.Tensor:
    """A device byte buffer of moe_pages_workspace_bytes whose head is zeroed."""
    n = moe_pages_workspace_bytes(K)
    if n == 0:
        raise MoeError("moe_pages_workspace_bytes", MOE_ERR_ARG)
    return _zeroed(n, K.tensors[0].device if device is None else device)


def _pages_scratch(fn, K, ws):
    if ws is None:
        raise ValueError(f"{fn}: it needs a workspace")
    if K.need is None:
        K.need = moe_pages_workspace_bytes(K)
    _scratch(fn, ws, K.index, K.need)
    return K.desc, ws.data_ptr()


def moe_kv_reserve(K, N, ws, n_new=None, stream=None):
    """Room for N (n_new [B]: for each sequence its own) more tokens (see include/moetree.h)."""
    fn = "moe_kv_reserve"
    _dense(fn, "n_new", n_new, torch.int32, (K.B,), K.index)
    desc, at = _pages_scratch(fn, K, ws)
    return _run(fn, K.index, stream, desc, N, _at(n_new), at)


def moe_kv_free(K, seqs, ws, keep=None, stream=None):
    """Gives back the pages of the sequences seqs [n] behind their first keep [n] tokens (None:
    all)."""
    fn, shape = "moe_kv_free", (seqs.numel(),)
    _dense(fn, "seqs", seqs, torch.int32, shape, K.index)
    _dense(fn, "keep", keep, torch.int32, shape, K.index)
    desc, at = _pages_scratch(fn, K, ws)
    return _run(fn, K.index, stream, desc, seqs.data_ptr(), _at(keep), shape[0], at)


def moe_kv_fork(K, src, dst, moves, ws, stream=None):
    """Sequences dst [n] become forks of src [n]; moves [n, 3] is for moe_kv_copy_pages."""
    fn, n = "moe_kv_fork", src.numel()
    _dense(fn, "src", src, torch.int32, (n,), K.index)
    _dense(fn, "dst", dst, torch.int32, (n,), K.index)
    _dense(fn, "moves", moves, torch.int32, (n, 3), K.index)
    desc, at = _pages_scratch(fn, K, ws)
    return _run(fn, K.index, stream, desc, src.data_ptr(), dst.data_ptr(), n, moves.data_ptr(), at)


def moe_kv_compact(K, table_out, ref_out, moves, counts, ws, stream=None):
    """Plans a dense pool: table_out, ref_out (may be the book's own), moves [n_pages // 2, 3],
    counts [2] (moves, pages in use)."""
    fn, i32 = "moe_kv_compact", torch.int32
    _dense(fn, "table_out", table_out, i32, (K.B, K.max_pages), K.index)
    _dense(fn, "ref_out", ref_out, i32, (K.n_pages,), K.index)
    _dense(fn, "moves", moves, i32, (K.n_pages // 2, 3), K.index)
    _dense(fn, "counts", counts, i32, (2,), K.index)
    desc, at = _pages_scratch(fn, K, ws)
    return _run(fn, K.index, stream, desc, table_out.data_ptr(), ref_out.data_ptr(),
                moves.data_ptr(), counts.data_ptr(), at)


def moe_kv_copy_pages(C_, k_pages, v_pages, moves, count=None, ws=None, stream=None):
    """Copies the tokens of moves [n, 3] (page, new page, tokens) between a layer's pages; count: a
    device int32 tensor whose first element says how many of them, None: all."""
    fn, n = "moe_kv_copy_pages", moves.shape[0]
    index, dt = k_pages.get_device(), _TORCH[C_.dtype]
    _like_cache(fn, C_, k_pages, v_pages, index, dt)
    _dense(fn, "moves", moves, torch.int32, (n, 3), index)
    if count is not None:
        _dense(fn, "count", count, torch.int32, count.shape, index)
        if count.numel() < 1:
            raise ValueError(f"{fn}: count has no element")
    _scratch(fn, ws, index, 4096)
    return _run(fn, index, stream, C.byref(C_), k_pages.data_ptr(), v_pages.data_ptr(),
                moves.data_ptr(), n, _at(count), _at(ws))


def moe_event_wait(event, timeout_s: float) -> None:
    _check("moe_event_wait", lib().moe_event_wait(_event(event), float(timeout_s)))
