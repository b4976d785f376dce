"""ctypes binding of libkvc.so (the C ABI declared in include/kvc.h).

Argument marshalling only: every step of the correction path runs in the CUDA
library.  Each function has the name of the C entry point it calls, takes
torch tensors (or raw integer device addresses, or None for NULL), passes
their data pointers / element strides and the current CUDA stream, and raises
``KvcError`` when the library returns a non-OK status (``check=False``
returns the status code instead).

The library must have been built in-tree (``__graft_entry__.build()``); a
missing library raises at import time -- there is no other implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence, Union

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvc.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libkvc.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
lib = ctypes.CDLL(LIB_PATH)

# ----------------------------------------------------------------- constants
KVC_OK = 0
KVC_ERR_INVALID_ARGUMENT = 1
KVC_ERR_SHAPE = 2
KVC_ERR_DTYPE = 3
KVC_ERR_ALIGNMENT = 4
KVC_ERR_ALIAS = 5
KVC_ERR_WORKSPACE = 6
KVC_ERR_UNSUPPORTED = 7
KVC_ERR_CUDA = 8
KVC_ERR_DEVICE_TIMEOUT = 9
KVC_ERR_NUMERICAL = 10

KVC_BF16 = 0
KVC_F32 = 1
KVC_E4M3 = 2

EXPORTS = ("kvc_version", "kvc_status_string", "kvc_last_error",
           "kvc_build_states_workspace", "kvc_build_states", "kvc_match_anchors",
           "kvc_apply_correction", "kvc_chain_edge_workspace", "kvc_chain_edge",
           "kvc_selftest_bounded_wait", "kvc_chain_edge_noalloc", "kvc_pool_insert",
           "kvc_build_representation", "kvc_match_representation",
           "kvc_page_plan", "kvc_page_write", "kvc_paged_attention_workspace",
           "kvc_paged_attention", "kvc_rotate_heads", "kvc_rotary_turns", "kvc_page_write_scaled",
           "kvc_paged_attention_scaled_workspace", "kvc_paged_attention_scaled")

KVC_NOALLOC_MAX_UNITS = 262144

KVC_PLAN_OK = 0
KVC_PLAN_NO_PAGES = 1
KVC_PLAN_ROW_FULL = 2
KVC_PLAN_INVALID = 3
KVC_PLAN_TOKENS = 4

KVC_ROTARY_PLAIN = 0
KVC_ROTARY_LINEAR = 1
KVC_ROTARY_BANDS = 2
KVC_ROTARY_RAMP = 3


class KvcError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        self.message = lib.kvc_last_error().decode()
        super().__init__("%s: %s: %s" % (where, lib.kvc_status_string(status).decode(), self.message))


# ------------------------------------------------------------------- structs
class kvc_cache_view(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("s_req", ctypes.c_int64),
                ("s_layer", ctypes.c_int64), ("s_head", ctypes.c_int64),
                ("s_tok", ctypes.c_int64)]


class kvc_segments(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int32), ("T", ctypes.c_int32), ("L", ctypes.c_int32),
                ("H", ctypes.c_int32), ("d", ctypes.c_int32), ("S", ctypes.c_int32),
                ("max_seg_len", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("seg_request", ctypes.POINTER(ctypes.c_int32)),
                ("seg_start", ctypes.POINTER(ctypes.c_int32)),
                ("seg_len", ctypes.POINTER(ctypes.c_int32))]


class kvc_params(ctypes.Structure):
    _fields_ = [("rank", ctypes.c_int32), ("oversample", ctypes.c_int32),
                ("power_iters", ctypes.c_int32), ("n_anchors", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("energy_frac", ctypes.c_float),
                ("temperature", ctypes.c_float), ("tau", ctypes.c_float),
                ("select_mode", ctypes.c_int32), ("reuse_ratio", ctypes.c_float),
                ("summary_mode", ctypes.c_int32), ("rank_c", ctypes.c_int32),
                ("omega_c", ctypes.c_void_p)]


class kvc_paged(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("L", ctypes.c_int32),
                ("H", ctypes.c_int32), ("d", ctypes.c_int32), ("R", ctypes.c_int32),
                ("max_blocks", ctypes.c_int32), ("dtype", ctypes.c_int)]


class kvc_attn_params(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int32), ("n_tokens", ctypes.c_int32),
                ("layer", ctypes.c_int32), ("causal", ctypes.c_int32), ("window", ctypes.c_int32),
                ("scale", ctypes.c_float), ("q_s_tok", ctypes.c_int64),
                ("q_s_head", ctypes.c_int64), ("out_s_tok", ctypes.c_int64),
                ("out_s_head", ctypes.c_int64)]


class kvc_scales(ctypes.Structure):
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("s_page", ctypes.c_int64),
                ("s_layer", ctypes.c_int64), ("s_head", ctypes.c_int64), ("block", ctypes.c_int32)]


class kvc_rotary_params(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("n_tokens", "n_q_heads", "n_kv_heads", "d", "rot_dim",
                                               "interleaved", "norm")]
                + [("eps", ctypes.c_float), ("amplitude", ctypes.c_float), ("dtype", ctypes.c_int)]
                + [(n, ctypes.c_int64) for n in ("q_s_tok", "q_s_head", "k_s_tok", "k_s_head",
                                                 "q_out_s_tok", "q_out_s_head", "k_out_s_tok",
                                                 "k_out_s_head")])


class kvc_rotary_scaling(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("factor", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("original", ctypes.c_double)]


_VIEW = kvc_cache_view
_PG_P = ctypes.POINTER(kvc_paged)
_ATT_P = ctypes.POINTER(kvc_attn_params)
_SEG_P = ctypes.POINTER(kvc_segments)
_PRM_P = ctypes.POINTER(kvc_params)
_VP = ctypes.c_void_p
_ST = ctypes.c_int

lib.kvc_version.restype = ctypes.c_char_p
lib.kvc_status_string.restype = ctypes.c_char_p
lib.kvc_status_string.argtypes = [_ST]
lib.kvc_last_error.restype = ctypes.c_char_p
lib.kvc_build_states_workspace.restype = ctypes.c_size_t
lib.kvc_build_states_workspace.argtypes = [_SEG_P, _PRM_P]
lib.kvc_build_states.restype = _ST
lib.kvc_build_states.argtypes = [_SEG_P, _PRM_P, _VIEW, _VIEW, _VIEW, _VIEW, _VP, ctypes.c_int32,
                                 _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP, _VP]
lib.kvc_pool_insert.restype = _ST
lib.kvc_pool_insert.argtypes = [_SEG_P, _PRM_P, _VIEW, _VIEW, _VIEW, _VIEW, _VP, _VP, _VP, _VP, _VP,
                                _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP, _VP]
lib.kvc_match_anchors.restype = _ST
lib.kvc_match_anchors.argtypes = [_SEG_P, _PRM_P, _VIEW, _VP, _VP, _VP, _VP, _VP, _VP]
lib.kvc_apply_correction.restype = _ST
lib.kvc_apply_correction.argtypes = [_SEG_P, _PRM_P, _VIEW, _VIEW, _VP, _VP, _VP, _VP, _VP,
                                     _VIEW, _VIEW, _VP, _VP, _VP, _VP, _VP, _VP]
lib.kvc_chain_edge_workspace.restype = ctypes.c_size_t
lib.kvc_chain_edge_workspace.argtypes = [_SEG_P, _PRM_P]
lib.kvc_chain_edge.restype = _ST
lib.kvc_chain_edge.argtypes = [ctypes.c_int32, _SEG_P, _PRM_P, _VIEW, _VIEW, _VP, _VP, _VP, _VP,
                               _VP, _VIEW, _VIEW, _VIEW, _VIEW, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                               ctypes.c_size_t, _VP, _VP]
lib.kvc_chain_edge_noalloc.restype = _ST
lib.kvc_chain_edge_noalloc.argtypes = [ctypes.c_int32, _SEG_P, _PRM_P, _VIEW, _VIEW, _VP, _VP, _VP,
                                       _VP, _VP, _VIEW, _VIEW, _VIEW, _VIEW, _VP, _VP, _VP, _VP,
                                       _VP, _VP, _VP, _VP]
lib.kvc_build_representation.restype = _ST
lib.kvc_build_representation.argtypes = [_SEG_P, _PRM_P, _VIEW, _VP, _VP, _VP, _VP, _VP]
lib.kvc_match_representation.restype = _ST
lib.kvc_match_representation.argtypes = [_SEG_P, _PRM_P, _VP, _VP, _VP, _VP, _VP, _VP]
lib.kvc_selftest_bounded_wait.restype = _ST
lib.kvc_selftest_bounded_wait.argtypes = [ctypes.c_int32, _VP, _VP]

lib.kvc_page_plan.restype = _ST
lib.kvc_page_plan.argtypes = [_PG_P, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_int32, _VP, _VP, _VP,
                              _VP, _VP]
lib.kvc_page_write.restype = _ST
lib.kvc_page_write.argtypes = [_PG_P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                               _VIEW, _VIEW, _VP, _VIEW, _VIEW, _VP]
lib.kvc_paged_attention_workspace.restype = ctypes.c_size_t
lib.kvc_paged_attention_workspace.argtypes = [_PG_P, _ATT_P]
lib.kvc_paged_attention.restype = _ST
lib.kvc_paged_attention.argtypes = [_PG_P, _ATT_P, _VP, _VIEW, _VIEW, _VP, _VP, _VP, _VP, _VP, _VP,
                                    ctypes.c_size_t, _VP, _VP]

lib.kvc_page_write_scaled.restype = _ST
lib.kvc_page_write_scaled.argtypes = [_PG_P, ctypes.POINTER(kvc_scales), ctypes.c_int32,
                                      ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _VIEW, _VIEW,
                                      _VP, _VIEW, _VIEW, ctypes.c_int32, _VP]
lib.kvc_paged_attention_scaled_workspace.restype = ctypes.c_size_t
lib.kvc_paged_attention_scaled_workspace.argtypes = [_PG_P, _ATT_P, ctypes.POINTER(kvc_scales)]
lib.kvc_paged_attention_scaled.restype = _ST
lib.kvc_paged_attention_scaled.argtypes = [_PG_P, _ATT_P, ctypes.POINTER(kvc_scales), _VP, _VIEW,
                                           _VIEW, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t,
                                           _VP, _VP]
lib.kvc_rotate_heads.restype = _ST
lib.kvc_rotate_heads.argtypes = [ctypes.POINTER(kvc_rotary_params), _VP, _VP, _VP, _VP, _VP, _VP,
                                 _VP, _VP, _VP]
lib.kvc_rotary_turns.restype = _ST
lib.kvc_rotary_turns.argtypes = [ctypes.POINTER(kvc_rotary_scaling), ctypes.c_double, ctypes.c_int32,
                                 _VP, ctypes.POINTER(ctypes.c_float)]


# ------------------------------------------------------------------- helpers
Ptr = Union[None, int, "torch.Tensor"]  # noqa: F821


def _addr(x: Ptr) -> Optional[int]:
    return x if x is None or isinstance(x, int) else x.data_ptr()


_raw_stream = None      # (device of the thread, its current stream) getters, once CUDA is up


def _stream(stream) -> Optional[int]:
    """The handle of a stream, or of torch's current one.  A small call spends most
    of its time on the host: building a torch Stream object would cost 3 us of it."""
    global _raw_stream
    if stream is None:
        if _raw_stream is not None:
            device, current = _raw_stream
            return current(device())
        import torch
        if not torch.cuda.is_available():
            return None
        handle = int(torch.cuda.current_stream().cuda_stream)
        if hasattr(torch._C, "_cuda_getCurrentRawStream") and hasattr(torch._C, "_cuda_getDevice"):
            _raw_stream = (torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
        return handle
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def cache_view(t: Ptr, strides: Optional[Sequence[int]] = None) -> kvc_cache_view:
    """View of a [R, L, H, T, d] cache tensor (d contiguous), or a NULL view.

    ``t`` may be a raw integer address, in which case ``strides`` =
    (s_req, s_layer, s_head, s_tok) in elements must be given."""
    if t is None:
        return kvc_cache_view(None, 0, 0, 0, 0)
    if isinstance(t, int):
        s = tuple(int(v) for v in strides)
        return kvc_cache_view(t, *s)
    st = t.stride()
    if len(st) != 5 or st[4] != 1:
        raise ValueError("cache tensors are [R, L, H, T, d] with a contiguous last dimension")
    return kvc_cache_view(t.data_ptr(), st[0], st[1], st[2], st[3])


class Segments:
    """kvc_segments plus the host arrays it points to (kept alive here)."""

    def __init__(self, R: int, T: int, L: int, H: int, d: int, dtype: str,
                 seg_request: Sequence[int], seg_start: Sequence[int], seg_len: Sequence[int],
                 max_seg_len: Optional[int] = None):
        self.req = np.ascontiguousarray(np.asarray(seg_request, dtype=np.int32))
        self.start = np.ascontiguousarray(np.asarray(seg_start, dtype=np.int32))
        self.len = np.ascontiguousarray(np.asarray(seg_len, dtype=np.int32))
        S = int(self.len.size)
        mx = int(max_seg_len) if max_seg_len is not None else (int(self.len.max()) if S else 1)
        ip = ctypes.POINTER(ctypes.c_int32)
        self.c = kvc_segments(
            R, T, L, H, d, S, mx, KVC_BF16 if dtype in ("bf16", KVC_BF16) else
            (KVC_F32 if dtype in ("f32", KVC_F32) else int(dtype)),
            self.req.ctypes.data_as(ip) if S else None,
            self.start.ctypes.data_as(ip) if S else None,
            self.len.ctypes.data_as(ip) if S else None)

    @classmethod
    def from_workload(cls, wl) -> "Segments":
        return cls(wl.R, wl.T, wl.L, wl.H, wl.d, wl.dtype, wl.seg_request, wl.seg_start,
                   wl.seg_len, wl.max_seg_len)

    @property
    def ref(self):
        return ctypes.byref(self.c)


def params(rank: int = 32, oversample: int = 8, power_iters: int = 2, n_anchors: int = 8,
           top_k: int = 0, energy_frac: float = 0.9, temperature: float = 0.1,
           tau: float = 0.32, reuse_ratio: Optional[float] = None,
           rank_c: Optional[int] = None, omega_c: Ptr = None) -> kvc_params:
    """Method parameters; ``reuse_ratio`` switches to the reuse-ratio mode,
    ``rank_c`` (with the device test matrix ``omega_c`` [d, rank_c +
    oversample]) to rank-r_C anchor representations.  The returned struct
    holds omega_c's raw address: keep the tensor alive while it is used."""
    return kvc_params(rank, oversample, power_iters, n_anchors,
                      top_k if top_k > 0 else n_anchors, energy_frac, temperature, tau,
                      0 if reuse_ratio is None else 1,
                      0.0 if reuse_ratio is None else float(reuse_ratio),
                      0 if rank_c is None else 1, 0 if rank_c is None else int(rank_c),
                      _addr(omega_c))


def params_from_workload(wl, omega_c: Ptr = None, **over) -> kvc_params:
    """Parameters of a synthetic workload; rank-mode workloads need their
    omega_c tensor (``WorkloadInputs.omega_c``)."""
    kw = dict(rank=wl.r, oversample=wl.oversample, power_iters=wl.power_iters, n_anchors=wl.A,
              top_k=wl.k_top, energy_frac=wl.energy_frac, temperature=wl.temperature, tau=wl.tau)
    if getattr(wl, "summary_mode", "mean") == "rank":
        kw.update(rank_c=wl.rank_c, omega_c=omega_c)
    kw.update(over)
    return params(**kw)


def _done(st: int, where: str, check: bool) -> int:
    if check and st != KVC_OK:
        raise KvcError(st, where)
    return st


def _nbytes(t: Ptr) -> int:
    if t is None or isinstance(t, int):
        return 0
    return t.numel() * t.element_size()


# --------------------------------------------------------------- entry points
def kvc_version() -> str:
    return lib.kvc_version().decode()


def kvc_build_states_workspace(seg: Segments, prm: kvc_params) -> int:
    return int(lib.kvc_build_states_workspace(seg.ref, ctypes.byref(prm)))


def kvc_chain_edge_workspace(seg: Segments, prm: kvc_params) -> int:
    return int(lib.kvc_chain_edge_workspace(seg.ref, ctypes.byref(prm)))


def kvc_build_states(seg: Segments, prm: kvc_params, exact_K, exact_V, ref_K, ref_V, omega: Ptr,
                     slot: int, U_K: Ptr, W_K: Ptr, U_V: Ptr, W_V: Ptr, sigma: Ptr,
                     eff_rank: Ptr, workspace: Ptr, dev_status: Ptr, stream=None,
                     workspace_bytes: Optional[int] = None, check: bool = True) -> int:
    ws_bytes = _nbytes(workspace) if workspace_bytes is None else int(workspace_bytes)
    st = lib.kvc_build_states(seg.ref, ctypes.byref(prm), _v(exact_K), _v(exact_V), _v(ref_K),
                              _v(ref_V), _addr(omega), int(slot), _addr(U_K), _addr(W_K),
                              _addr(U_V), _addr(W_V), _addr(sigma), _addr(eff_rank),
                              _addr(workspace), ws_bytes, _addr(dev_status), _stream(stream))
    return _done(st, "kvc_build_states", check)


def kvc_pool_insert(seg: Segments, prm: kvc_params, dense_K, dense_V, held_K, held_V,
                    omega: Ptr, fallback: Ptr, pool_next: Ptr, U_K: Ptr, W_K: Ptr, U_V: Ptr,
                    W_V: Ptr, summaries: Ptr, sigma: Ptr, eff_rank: Ptr, workspace: Ptr,
                    dev_status: Ptr, stream=None, workspace_bytes: Optional[int] = None,
                    check: bool = True) -> int:
    ws_bytes = _nbytes(workspace) if workspace_bytes is None else int(workspace_bytes)
    st = lib.kvc_pool_insert(seg.ref, ctypes.byref(prm), _v(dense_K), _v(dense_V), _v(held_K),
                             _v(held_V), _addr(omega), _addr(fallback), _addr(pool_next),
                             _addr(U_K), _addr(W_K), _addr(U_V), _addr(W_V), _addr(summaries),
                             _addr(sigma), _addr(eff_rank), _addr(workspace), ws_bytes,
                             _addr(dev_status), _stream(stream))
    return _done(st, "kvc_pool_insert", check)


def kvc_match_anchors(seg: Segments, prm: kvc_params, ref_K, summaries: Ptr, weights: Ptr,
                      best: Ptr, query: Ptr = None, dev_status: Ptr = None, stream=None,
                      check: bool = True) -> int:
    st = lib.kvc_match_anchors(seg.ref, ctypes.byref(prm), _v(ref_K), _addr(summaries),
                               _addr(weights), _addr(best), _addr(query), _addr(dev_status),
                               _stream(stream))
    return _done(st, "kvc_match_anchors", check)


def kvc_build_representation(seg: Segments, prm: kvc_params, cache_K, rep: Ptr,
                             rep_sigma: Ptr = None, rep_eff_rank: Ptr = None,
                             dev_status: Ptr = None, stream=None, check: bool = True) -> int:
    st = lib.kvc_build_representation(seg.ref, ctypes.byref(prm), _v(cache_K), _addr(rep),
                                      _addr(rep_sigma), _addr(rep_eff_rank), _addr(dev_status),
                                      _stream(stream))
    return _done(st, "kvc_build_representation", check)


def kvc_match_representation(seg: Segments, prm: kvc_params, query_rep: Ptr, anchor_reps: Ptr,
                             weights: Ptr, best: Ptr, dev_status: Ptr = None, stream=None,
                             check: bool = True) -> int:
    st = lib.kvc_match_representation(seg.ref, ctypes.byref(prm), _addr(query_rep),
                                      _addr(anchor_reps), _addr(weights), _addr(best),
                                      _addr(dev_status), _stream(stream))
    return _done(st, "kvc_match_representation", check)


def kvc_apply_correction(seg: Segments, prm: kvc_params, ref_K, ref_V, U_K: Ptr, W_K: Ptr,
                         U_V: Ptr, W_V: Ptr, weights: Ptr, out_K, out_V, partial: Ptr,
                         score: Ptr, fallback: Ptr, dev_status: Ptr, stream=None,
                         check: bool = True, ksum_out: Ptr = None) -> int:
    st = lib.kvc_apply_correction(seg.ref, ctypes.byref(prm), _v(ref_K), _v(ref_V), _addr(U_K),
                                  _addr(W_K), _addr(U_V), _addr(W_V), _addr(weights), _v(out_K),
                                  _v(out_V), _addr(partial), _addr(score), _addr(fallback),
                                  _addr(ksum_out), _addr(dev_status), _stream(stream))
    return _done(st, "kvc_apply_correction", check)


def kvc_chain_edge(edge: int, seg: Segments, prm: kvc_params, ref_K, ref_V, summaries: Ptr,
                   U_K: Ptr, W_K: Ptr, U_V: Ptr, W_V: Ptr, dense_K, dense_V, out_K, out_V,
                   weights: Ptr, best: Ptr, score: Ptr, fallback: Ptr, workspace: Ptr,
                   dev_status: Ptr, stream=None, workspace_bytes: Optional[int] = None,
                   check: bool = True, ksum_in: Ptr = None, ksum_out: Ptr = None) -> int:
    """``ksum_out`` [S, L, H, 4, d] receives the column sums of the held keys
    this edge leaves; passing it as the next edge's ``ksum_in`` spares that
    edge's match the pass over the key rows."""
    ws_bytes = _nbytes(workspace) if workspace_bytes is None else int(workspace_bytes)
    st = lib.kvc_chain_edge(int(edge), seg.ref, ctypes.byref(prm), _v(ref_K), _v(ref_V),
                            _addr(summaries), _addr(U_K), _addr(W_K), _addr(U_V), _addr(W_V),
                            _v(dense_K), _v(dense_V), _v(out_K), _v(out_V), _addr(weights),
                            _addr(best), _addr(score), _addr(fallback), _addr(ksum_in),
                            _addr(ksum_out), _addr(workspace), ws_bytes, _addr(dev_status),
                            _stream(stream))
    return _done(st, "kvc_chain_edge", check)


def kvc_chain_edge_noalloc(edge: int, seg: Segments, prm: kvc_params, ref_K, ref_V,
                           summaries: Ptr, U_K: Ptr, W_K: Ptr, U_V: Ptr, W_V: Ptr, dense_K,
                           dense_V, out_K, out_V, weights: Ptr, best: Ptr, score: Ptr,
                           fallback: Ptr, dev_status: Ptr, stream=None, check: bool = True,
                           ksum_in: Ptr = None, ksum_out: Ptr = None) -> int:
    """kvc_chain_edge without a workspace argument, for callers that cannot
    allocate device memory (the library's own device scratch array is used;
    include/kvc.h states its size limit and the rule that overlapping calls
    on one device race)."""
    st = lib.kvc_chain_edge_noalloc(int(edge), seg.ref, ctypes.byref(prm), _v(ref_K), _v(ref_V),
                                    _addr(summaries), _addr(U_K), _addr(W_K), _addr(U_V),
                                    _addr(W_V), _v(dense_K), _v(dense_V), _v(out_K), _v(out_V),
                                    _addr(weights), _addr(best), _addr(score), _addr(fallback),
                                    _addr(ksum_in), _addr(ksum_out), _addr(dev_status),
                                    _stream(stream))
    return _done(st, "kvc_chain_edge_noalloc", check)


def kvc_selftest_bounded_wait(max_polls: int, dev_status: Ptr, stream=None,
                              check: bool = True) -> int:
    st = lib.kvc_selftest_bounded_wait(int(max_polls), _addr(dev_status), _stream(stream))
    return _done(st, "kvc_selftest_bounded_wait", check)


def _v(x) -> kvc_cache_view:
    return x if type(x) is kvc_cache_view else cache_view(x)


# ---------------------------------------------------------------- paged caches
def paged(n_pages: int, page_size: int, L: int, H: int, d: int, dtype: str, R: int,
          max_blocks: int) -> kvc_paged:
    """Descriptor of page pools [n_pages, L, H, page_size, d] and of block
    tables [R, max_blocks]; ``dtype`` is "bf16", "f32" or, for scaled pools, "e4m3"."""
    code = {"bf16": KVC_BF16, "f32": KVC_F32, "e4m3": KVC_E4M3}.get(dtype)
    return kvc_paged(n_pages, page_size, L, H, d, R, max_blocks, int(dtype) if code is None else code)


def attn_params(q, out, layer: int = 0, scale: float = 0.0, causal: bool = True,
                window: int = 0) -> kvc_attn_params:
    """Attention parameters for query and output tensors [N, Hq, d] (any token
    and head strides, d contiguous); ``scale`` 0 means 1 / sqrt(d)."""
    for t in (q, out):
        if t.dim() != 3 or (t.stride(-1) != 1 and t.shape[-1] > 1) or t.shape != q.shape:
            raise ValueError("q and out are [N, Hq, d] with a contiguous last dimension")
    N, Hq, d = q.shape
    return kvc_attn_params(Hq, N, layer, int(causal), window, scale if scale else d ** -0.5,
                           q.stride(0), q.stride(1), out.stride(0), out.stride(1))


def kvc_page_plan(pg: kvc_paged, new_lens: Ptr, kv_lens: Ptr, kv_lens_out: Ptr, block_table: Ptr,
                  free_pages: Ptr, n_free: Ptr, n_free_out: Ptr, q_start: Ptr, slot_map: Ptr,
                  positions: Ptr, plan_status: Ptr, stream=None,
                  max_tokens: Optional[int] = None, check: bool = True) -> int:
    """Block tables, slots and positions of a step's new tokens.
    ``max_tokens`` is the length of ``slot_map`` and ``positions`` (taken from
    the tensor if not given)."""
    if max_tokens is None:
        max_tokens = slot_map.numel()
    st = lib.kvc_page_plan(ctypes.byref(pg), _addr(new_lens), _addr(kv_lens), _addr(kv_lens_out),
                           _addr(block_table), _addr(free_pages), _addr(n_free), _addr(n_free_out),
                           max_tokens, _addr(q_start), _addr(slot_map), _addr(positions),
                           _addr(plan_status), _stream(stream))
    return _done(st, "kvc_page_plan", check)


def kvc_page_write(pg: kvc_paged, src_K, src_V, slot_map: Ptr, pool_K, pool_V, layer: int = 0,
                   stream=None, shape: Optional[Sequence[int]] = None, check: bool = True) -> int:
    """Rows of ``src_K`` / ``src_V`` [n_src, n_layers, H, T, d] into the slots
    ``slot_map`` [n_src, T] of layers ``layer`` .. of the pools.  Raw views
    need ``shape`` = (n_src, n_layers, T)."""
    if shape is not None:
        n, nl, T = shape
    else:
        n, nl, _, T, _ = src_K.shape
    st = lib.kvc_page_write(ctypes.byref(pg), n, T, layer, nl, _v(src_K), _v(src_V),
                            _addr(slot_map), _v(pool_K), _v(pool_V), _stream(stream))
    return _done(st, "kvc_page_write", check)


def kvc_paged_attention_workspace(pg: kvc_paged, at: kvc_attn_params) -> int:
    return int(lib.kvc_paged_attention_workspace(ctypes.byref(pg), ctypes.byref(at)))


def kvc_paged_attention(pg: kvc_paged, at: kvc_attn_params, q: Ptr, pool_K, pool_V,
                        block_table: Ptr, q_start: Ptr, kv_lens: Ptr, out: Ptr, workspace: Ptr,
                        dev_status: Ptr, lse: Ptr = None, stream=None,
                        workspace_bytes: Optional[int] = None, check: bool = True) -> int:
    """Attention of every request's new tokens over its pages.  The first
    8,192 bytes of ``workspace`` must be zero before its first use."""
    ws_bytes = _nbytes(workspace) if workspace_bytes is None else int(workspace_bytes)
    st = lib.kvc_paged_attention(ctypes.byref(pg), ctypes.byref(at), _addr(q), _v(pool_K),
                                 _v(pool_V), _addr(block_table), _addr(q_start), _addr(kv_lens),
                                 _addr(out), _addr(lse), _addr(workspace), ws_bytes,
                                 _addr(dev_status), _stream(stream))
    return _done(st, "kvc_paged_attention", check)


# ---------------------------------------------------------------- scaled pools
def scales(K, V, block: int) -> kvc_scales:
    """Exponent bytes of scaled pools, uint8 tensors [n_pages, L, H, ceil(page_size /
    block)] of K's and V's blocks of ``block`` rows, with the blocks of a page side by side.
    The struct holds their raw addresses: keep the tensors alive while it is used."""
    import torch
    for t in (K, V):
        if (t.dim() != 4 or t.dtype != torch.uint8 or t.shape != K.shape or t.stride() != K.stride()
                or (t.stride(3) != 1 and t.shape[3] > 1)):
            raise ValueError("exponents are [n_pages, L, H, blocks] uint8 with a contiguous last "
                             "dimension, alike for K and V")
    return kvc_scales(K.data_ptr(), V.data_ptr(), K.stride(0), K.stride(1), K.stride(2), block)


def kvc_page_write_scaled(pg: kvc_paged, sc: kvc_scales, src_K, src_V, slot_map: Ptr, pool_K, pool_V,
                          layer: int = 0, keep: bool = False, stream=None,
                          shape: Optional[Sequence[int]] = None, check: bool = True) -> int:
    """bf16 rows of ``src_K`` / ``src_V`` [n_src, n_layers, H, T, d] into the slots
    ``slot_map`` [n_src, T] of layers ``layer`` .. of scaled pools.  ``keep``: blocks of
    which some rows are overwritten keep the others.  Raw views need ``shape`` =
    (n_src, n_layers, T)."""
    if shape is not None:
        n, nl, T = shape
    else:
        n, nl, _, T, _ = src_K.shape
    st = lib.kvc_page_write_scaled(ctypes.byref(pg), ctypes.byref(sc), n, T, layer, nl, _v(src_K),
                                   _v(src_V), _addr(slot_map), _v(pool_K), _v(pool_V), int(keep),
                                   _stream(stream))
    return _done(st, "kvc_page_write_scaled", check)


def kvc_paged_attention_scaled_workspace(pg: kvc_paged, at: kvc_attn_params, sc: kvc_scales) -> int:
    return int(lib.kvc_paged_attention_scaled_workspace(ctypes.byref(pg), ctypes.byref(at),
                                                        ctypes.byref(sc)))


def kvc_paged_attention_scaled(pg: kvc_paged, at: kvc_attn_params, sc: kvc_scales, q: Ptr, pool_K,
                               pool_V, block_table: Ptr, q_start: Ptr, kv_lens: Ptr, out: Ptr,
                               workspace: Ptr, dev_status: Ptr, lse: Ptr = None, stream=None,
                               workspace_bytes: Optional[int] = None, check: bool = True) -> int:
    """kvc_paged_attention over scaled pools; q and out are bf16."""
    ws_bytes = _nbytes(workspace) if workspace_bytes is None else int(workspace_bytes)
    st = lib.kvc_paged_attention_scaled(ctypes.byref(pg), ctypes.byref(at), ctypes.byref(sc),
                                        _addr(q), _v(pool_K), _v(pool_V), _addr(block_table),
                                        _addr(q_start), _addr(kv_lens), _addr(out), _addr(lse),
                                        _addr(workspace), ws_bytes, _addr(dev_status),
                                        _stream(stream))
    return _done(st, "kvc_paged_attention_scaled", check)


# ------------------------------------------------------- positions of the heads
_MODES = {"none": KVC_ROTARY_PLAIN, "linear": KVC_ROTARY_LINEAR, "bands": KVC_ROTARY_BANDS,
          "ramp": KVC_ROTARY_RAMP}


def rotary_turns(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                 low: float = 1.0, high: float = 4.0, original: float = 8192.0):
    """(turns, amplitude): the pairs' frequencies base^(-2 i / rot_dim) as turns per
    position in units of 2^-64, a host int64 tensor [rot_dim / 2] (``.cuda()`` it once),
    and the rotation's amplitude.  ``scaling`` for long contexts: "none", "linear" (all
    divided by ``factor``), "bands" (model configurations say "llama3": those that make at least ``high`` turns within
    ``original`` positions stay, those of at most ``low`` are divided, the share kept
    between is linear in the turns) or "ramp" ("yarn": it is linear in the pair's number, and the
    amplitude grows with the factor)."""
    import torch
    if scaling not in _MODES:
        raise ValueError("scaling is one of " + ", ".join(_MODES))
    turns = torch.zeros(max(rot_dim, 0) // 2, dtype=torch.int64)
    sc, amplitude = kvc_rotary_scaling(_MODES[scaling], factor, low, high, original), ctypes.c_float()
    _done(lib.kvc_rotary_turns(ctypes.byref(sc), base, rot_dim, turns.data_ptr(),
                               ctypes.byref(amplitude)), "kvc_rotary_turns", True)
    return turns, float(amplitude.value)


def rotary_params(q, k, q_out, k_out, rot_dim: int, interleaved: bool = False, norm: bool = False,
                  eps: float = 1e-6, amplitude: float = 1.0) -> kvc_rotary_params:
    """Descriptor of a rotation of ``q`` [N, Hq, d] and ``k`` [N, H, d] (either may be None)
    into ``q_out`` and ``k_out``, which may be they themselves."""
    import torch
    heads, strides, like = [], [], None
    for x, y in ((q, q_out), (k, k_out)):
        if (x is None) != (y is None):
            raise ValueError("an output goes with each of q and k that is given")
        if x is None:
            heads.append(0)
            strides.append((0, 0, 0, 0))
            continue
        like = x if like is None else like
        for t in (x, y):
            if (t.dim() != 3 or (t.stride(-1) != 1 and t.shape[-1] > 1) or t.shape != x.shape
                    or t.dtype != like.dtype or t.device != like.device):
                raise ValueError("q, k and outputs are [N, heads, d] of one type on one device, "
                                 "with a contiguous last dimension")
        if x.shape[0] != like.shape[0] or x.shape[2] != like.shape[2]:
            raise ValueError("q and k have the same tokens and head dim")
        heads.append(x.shape[1])
        strides.append((x.stride(0), x.stride(1), y.stride(0), y.stride(1)))
    if like is None:
        raise ValueError("neither q nor k is given")
    dtype = {torch.bfloat16: KVC_BF16, torch.float32: KVC_F32}.get(like.dtype)
    if dtype is None:
        raise ValueError("q and k are bfloat16 or float32")
    (a, b, e, f), (c, d, g, h) = strides
    return kvc_rotary_params(like.shape[0], heads[0], heads[1], like.shape[2], rot_dim,
                             int(interleaved), int(norm), eps, amplitude, dtype,
                             a, b, c, d, e, f, g, h)


def kvc_rotate_heads(rp: kvc_rotary_params, q: Ptr, k: Ptr, positions: Ptr, turns: Ptr, q_out: Ptr,
                     k_out: Ptr, w_q: Ptr = None, w_k: Ptr = None, stream=None,
                     check: bool = True) -> int:
    """Norms of the query and key heads and their rotation by position.  ``turns`` is the
    device copy of ``rotary_turns``' table."""
    st = lib.kvc_rotate_heads(ctypes.byref(rp), _addr(q), _addr(k), _addr(w_q), _addr(w_k),
                              _addr(positions), _addr(turns), _addr(q_out), _addr(k_out),
                              _stream(stream))
    return _done(st, "kvc_rotate_heads", check)
