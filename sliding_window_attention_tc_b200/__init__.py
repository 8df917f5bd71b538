"""Python binding of libtc, the Tensor Cache layer for B200 (sm_100a).

This module only marshals arguments: it checks that tensors are contiguous
and of the right dtype, allocates outputs and workspace with PyTorch when the
caller does not pass them, and calls the C-ABI entry points declared in
``include/tc.h`` through ctypes.  Every step of the layer runs in the CUDA
kernels of ``libtc.so``; there is no CPU or PyTorch fallback.  Importing this
package fails if ``libtc.so`` has not been built
(``python sliding_window_attention_tc_b200/build.py``).

The layer ("Tensor Cache: Eviction-conditioned Associative Memory for
Transformers", §3.1-§3.2): per head, exact softmax attention over the last W
keys (L1) plus a d_k x d_v matrix A written only by pairs evicted from the
window, A <- lambda A + eta k v^T, read as m = q A (L2), fused as
y = y_local + sigmoid(g) m.  Within a step the eviction is written before the
read.

Around it: rotate and rotate_backward (rotary positions of q and k), and
PagedCache with cache_append, cache_attend, cache_evict and cache_step, the
streaming state for rows of different lengths and grouped heads, in which the
least attended pair leaves into A instead of the oldest.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtc.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libtc.so not found at {LIB_PATH}; build it with "
                      "`python sliding_window_attention_tc_b200/build.py`")

_lib = ctypes.CDLL(LIB_PATH)

TC_OK = 0
STATUS_NAMES = {0: "TC_OK", 1: "TC_ERR_INVALID_ARG", 2: "TC_ERR_UNSUPPORTED",
                3: "TC_ERR_NO_DEVICE", 4: "TC_ERR_CUDA", 5: "TC_ERR_DEVICE_BOUNDS",
                6: "TC_ERR_DEVICE_TIMEOUT", 7: "TC_ERR_WORKSPACE"}
TC_F32, TC_BF16 = 0, 1
TC_PREFILL_L1_ONLY = 1
TC_PREFILL_STATE_ONLY = 2
TC_PREFILL_DELTA_RULE = 4
TC_PREFILL_CHUNK_MEAN = 8
TC_WRITE_OUTER, TC_WRITE_DELTA = 0, 1
TC_PATH_AUTO, TC_PATH_FUSED, TC_PATH_GENERAL = 0, 1, 2

# Exported C symbols declared in include/tc.h.
EXPORTED = ("tc_prefill_workspace_size", "tc_prefill", "tc_prefill_launch_count", "tc_prefill_host_workspace_size",
            "tc_prefill_host", "tc_decode_step", "tc_decode_step_host_workspace_size",
            "tc_decode_step_host", "tc_get_device_status", "tc_status_string", "tc_version",
            "tc_prefill_no_alloc", "tc_prefill_from_state", "tc_prefill_from_state_workspace_size",
            "tc_state_fold", "tc_decode_step_ragged", "tc_backward", "tc_backward_workspace_size",
            "tc_set_wait_limit_ns", "tc_prefill_varlen", "tc_prefill_varlen_workspace_size",
            "tc_backward_launch_count", "tc_set_prefill_path", "tc_get_prefill_path",
            "tc_prefill_path_for", "tc_rotate", "tc_cache_append", "tc_cache_attend",
            "tc_cache_attend_workspace_size", "tc_cache_evict", "tc_cache_evict_workspace_size",
            "tc_cache_step", "tc_cache_step_workspace_size")
TC_ROTATE_BACKWARD = 1
TC_CACHE_ACCUMULATE = 1


class PrefillDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("H", ctypes.c_int64), ("T", ctypes.c_int64),
                ("dk", ctypes.c_int64), ("dv", ctypes.c_int64), ("W", ctypes.c_int64),
                ("C", ctypes.c_int64), ("dtype", ctypes.c_int), ("flags", ctypes.c_uint32)]


class DecodeStateC(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("H", ctypes.c_int64), ("dk", ctypes.c_int64),
                ("dv", ctypes.c_int64), ("W", ctypes.c_int64), ("t", ctypes.c_int64),
                ("kv_dtype", ctypes.c_int), ("ring_k", ctypes.c_void_p),
                ("ring_v", ctypes.c_void_p), ("A", ctypes.c_void_p),
                ("lam", ctypes.c_void_p), ("eta", ctypes.c_void_p), ("g", ctypes.c_void_p),
                ("write_rule", ctypes.c_int)]


class RotaryC(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int64), ("interleaved", ctypes.c_int64), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double),
                ("train_len", ctypes.c_double), ("gain", ctypes.c_double)]


_I3 = ctypes.c_int64 * 3


class RotateDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("Hq", ctypes.c_int64), ("H", ctypes.c_int64),
                ("T", ctypes.c_int64), ("d", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("flags", ctypes.c_uint32), ("q_stride", _I3), ("k_stride", _I3),
                ("q_out_stride", _I3), ("k_out_stride", _I3)]


class PagedCacheC(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("H", ctypes.c_int64), ("d", ctypes.c_int64),
                ("page", ctypes.c_int64), ("n_pages", ctypes.c_int64), ("max_pages", ctypes.c_int64),
                ("dtype", ctypes.c_int), ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("mass", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("len", ctypes.c_void_p), ("clock", ctypes.c_void_p), ("A", ctypes.c_void_p),
                ("lam", ctypes.c_void_p), ("eta", ctypes.c_void_p)]


class AppendArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("Hq", ctypes.c_int64), ("q", ctypes.c_void_p),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q_stride", _I3),
                ("k_stride", _I3), ("v_stride", _I3), ("counts", ctypes.c_void_p),
                ("mass_in", ctypes.c_void_p), ("q_out", ctypes.c_void_p)]


_I2 = ctypes.c_int64 * 2


class StepArgs(ctypes.Structure):
    _fields_ = [("Hq", ctypes.c_int64), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("q_stride", _I2), ("k_stride", _I2), ("v_stride", _I2),
                ("g", ctypes.c_void_p), ("y", ctypes.c_void_p), ("budget", ctypes.c_int64),
                ("recent", ctypes.c_int64), ("flags", ctypes.c_uint32)]


_vp, _sz, _int = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
_PD = ctypes.POINTER(PrefillDesc)
_DS = ctypes.POINTER(DecodeStateC)
_lib.tc_prefill_workspace_size.argtypes = [_PD]
_lib.tc_prefill_workspace_size.restype = _sz
_lib.tc_prefill.argtypes = [_PD] + [_vp] * 9 + [_sz, _vp]
_lib.tc_prefill.restype = _int
_lib.tc_backward_launch_count.argtypes = [_PD, ctypes.POINTER(_int)]
_lib.tc_backward_launch_count.restype = _int
_lib.tc_prefill_launch_count.argtypes = [_PD]
_lib.tc_prefill_launch_count.restype = _int
_lib.tc_prefill_host_workspace_size.argtypes = [_PD]
_lib.tc_prefill_host_workspace_size.restype = _sz
_lib.tc_prefill_host.argtypes = [_PD] + [_vp] * 9 + [_sz, _vp]
_lib.tc_prefill_host.restype = _int
_lib.tc_prefill_no_alloc.argtypes = [_PD] + [_vp] * 8 + [_vp]
_lib.tc_prefill_no_alloc.restype = _int
_lib.tc_prefill_from_state_workspace_size.argtypes = [_PD, ctypes.c_int64]
_lib.tc_prefill_from_state_workspace_size.restype = _sz
_lib.tc_prefill_from_state.argtypes = [_PD, ctypes.c_int64] + [_vp] * 12 + [_sz, _vp]
_lib.tc_prefill_from_state.restype = _int
_lib.tc_prefill_varlen_workspace_size.argtypes = [_PD]
_lib.tc_prefill_varlen_workspace_size.restype = _sz
_lib.tc_prefill_varlen.argtypes = [_PD, _vp, ctypes.c_int64] + [_vp] * 9 + [_sz, _vp]
_lib.tc_prefill_varlen.restype = _int
_lib.tc_backward_workspace_size.argtypes = [_PD]
_lib.tc_backward_workspace_size.restype = _sz
_lib.tc_backward.argtypes = [_PD] + [_vp] * 14 + [_sz, _vp]
_lib.tc_backward.restype = _int
_lib.tc_state_fold.argtypes = [ctypes.c_int64] * 5 + [_vp] * 4 + [_vp]
_lib.tc_state_fold.restype = _int
_lib.tc_decode_step.argtypes = [_DS] + [_vp] * 4 + [_vp]
_lib.tc_decode_step.restype = _int
_lib.tc_decode_step_ragged.argtypes = [_DS] + [_vp] * 5 + [_vp]
_lib.tc_decode_step_ragged.restype = _int
_lib.tc_decode_step_host_workspace_size.argtypes = [_DS]
_lib.tc_decode_step_host_workspace_size.restype = _sz
_lib.tc_decode_step_host.argtypes = [_DS] + [_vp] * 5 + [_sz, _vp]
_lib.tc_decode_step_host.restype = _int
_lib.tc_get_device_status.argtypes = [_vp]
_lib.tc_get_device_status.restype = _int
_lib.tc_status_string.argtypes = [_int]
_lib.tc_status_string.restype = ctypes.c_char_p
_lib.tc_version.argtypes = []
_lib.tc_version.restype = ctypes.c_char_p
_lib.tc_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
_lib.tc_set_wait_limit_ns.restype = None
_lib.tc_set_prefill_path.argtypes = [_int]
_lib.tc_set_prefill_path.restype = _int
_lib.tc_get_prefill_path.argtypes = []
_lib.tc_get_prefill_path.restype = _int
_lib.tc_prefill_path_for.argtypes = [_PD, ctypes.c_int64]
_lib.tc_prefill_path_for.restype = _int

_PC, _PR = ctypes.POINTER(PagedCacheC), ctypes.POINTER(RotaryC)
# the small per-call structures go as packed bytes (or by reference): see _PACK_*
_lib.tc_rotate.argtypes = [_vp, _PR, _vp, ctypes.c_int64] + [_vp] * 4 + [_vp]
_lib.tc_rotate.restype = _int
_lib.tc_cache_append.argtypes = [_PC, _PR, _vp, _vp]
_lib.tc_cache_append.restype = _int
_lib.tc_cache_attend_workspace_size.argtypes = [_PC, ctypes.c_int64, ctypes.c_uint32]
_lib.tc_cache_attend_workspace_size.restype = _sz
_lib.tc_cache_attend.argtypes = [_PC, ctypes.c_int64, _vp, _vp, _vp, ctypes.c_uint32, _vp, _sz, _vp]
_lib.tc_cache_attend.restype = _int
_lib.tc_cache_evict_workspace_size.argtypes = [_PC]
_lib.tc_cache_evict_workspace_size.restype = _sz
_lib.tc_cache_evict.argtypes = [_PC, ctypes.c_int64, ctypes.c_int64, _vp, _sz, _vp]
_lib.tc_cache_evict.restype = _int
_lib.tc_cache_step_workspace_size.argtypes = [_PC, ctypes.c_int64, ctypes.c_uint32]
_lib.tc_cache_step_workspace_size.restype = _sz
_lib.tc_cache_step.argtypes = [_PC, _PR, _vp, _vp, _sz, _vp]
_lib.tc_cache_step.restype = _int

SIZE_ERROR = ctypes.c_size_t(-1).value


class TCError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {STATUS_NAMES.get(self.status, self.status)} "
                         f"({status_string(self.status)})")


def status_string(status: int) -> str:
    return _lib.tc_status_string(int(status)).decode()


def version() -> str:
    return _lib.tc_version().decode()


def lib_handle() -> ctypes.CDLL:
    """The loaded libtc (for tests that call the C-ABI directly)."""
    return _lib


def _check(st: int, where: str):
    if st != TC_OK:
        raise TCError(st, where)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return TC_F32
    if t.dtype == torch.bfloat16:
        return TC_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _on_device(current: int, *ts):
    """Every CUDA tensor must live on the current device `current`: the
    kernels run there, and another GPU's buffer would be read over the peer
    link (or fault without peer access).  The library refuses such pointers
    too; checking here gives a clear Python error first."""
    for t in ts:
        if t is not None and t.device.type == "cuda" and t.device.index != current:
            raise ValueError(f"tensor on {t.device} but the current CUDA device is cuda:{current}; "
                             "call under torch.cuda.device(...) of the tensors' device")


def _dev_check(*ts):
    if any(t is not None and t.device.type == "cuda" for t in ts):
        _on_device(torch.cuda.current_device(), *ts)


# The C-ABI sees only addresses, so a tensor of the wrong size or element type
# would have a kernel read or write past its end: shapes and dtypes are
# checked here, before any call.
def _expect(t: Optional[torch.Tensor], name: str, shape, dtype):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}; expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")


def _expect_layer(B, H, T, dk, dv, dt, q, k, v, lam, eta, g, y=None, A_final=None):
    """q, k [B,H,T,dk], v (and y) [B,H,T,dv] in dt; lam, eta, g [H] float32;
    A_final [B,H,dk,dv] float32 (None entries are not checked)."""
    _expect(q, "q", (B, H, T, dk), dt)
    _expect(k, "k", (B, H, T, dk), dt)
    _expect(v, "v", (B, H, T, dv), dt)
    for name, t in (("lam", lam), ("eta", eta), ("g", g)):
        if t is None:
            raise ValueError(f"{name} is required")
        _expect(t, name, (H,), torch.float32)
    _expect(y, "y", (B, H, T, dv), dt)
    _expect(A_final, "A_final", (B, H, dk, dv), torch.float32)


def make_prefill_desc(B, H, T, dk, dv, W, C, dtype: int, l1_only: bool = False,
                      state_only: bool = False, delta_rule: bool = False,
                      chunk_mean: bool = False) -> PrefillDesc:
    flags = ((TC_PREFILL_L1_ONLY if l1_only else 0) | (TC_PREFILL_STATE_ONLY if state_only else 0)
             | (TC_PREFILL_DELTA_RULE if delta_rule else 0)
             | (TC_PREFILL_CHUNK_MEAN if chunk_mean else 0))
    return PrefillDesc(int(B), int(H), int(T), int(dk), int(dv), int(W), int(C), int(dtype),
                       flags)


def prefill_workspace_size(desc: PrefillDesc) -> int:
    n = _lib.tc_prefill_workspace_size(ctypes.byref(desc))
    if n == SIZE_ERROR:
        raise TCError(1, "tc_prefill_workspace_size")
    return int(n)


def _desc_of(q, v, W, C, l1_only, delta_rule=False):
    B, H, T, dk = q.shape
    return make_prefill_desc(B, H, T, dk, v.shape[-1], W, C, _dtype_code(q), l1_only,
                             delta_rule=delta_rule)


def prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor,
            eta: torch.Tensor, g: torch.Tensor, W: int, C: int, *, l1_only: bool = False,
            delta_rule: bool = False, y: Optional[torch.Tensor] = None,
            A_final: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
            stream=None):
    """tc_prefill on device tensors q, k [B,H,T,dk], v [B,H,T,dv] (float32 or
    bfloat16), lam, eta, g [H] float32.  Returns (y, A_final); A_final is
    None with l1_only.  delta_rule selects the delta-rule write."""
    desc = _desc_of(q, v, W, C, l1_only, delta_rule)
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    _expect_layer(B, H, T, dk, dv, q.dtype, q, k, v, lam, eta, g, y, A_final)
    if y is None:
        y = torch.empty((B, H, T, dv), dtype=q.dtype, device=q.device)
    if A_final is None and not l1_only:
        A_final = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    need = prefill_workspace_size(desc)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _contig(q, k, v, lam, eta, g, y, A_final, workspace)
    _dev_check(q, k, v, lam, eta, g, y, A_final, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = _lib.tc_prefill(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(eta),
                         _ptr(g), _ptr(y), _ptr(A_final), _ptr(workspace), ws_bytes,
                         _stream(stream))
    _check(st, "tc_prefill")
    return y, A_final


def prefill_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                   max_seqlen: int, lam: torch.Tensor, eta: torch.Tensor, g: torch.Tensor,
                   W: int, C: int, *, l1_only: bool = False, y: Optional[torch.Tensor] = None,
                   A_final: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """tc_prefill_varlen: len(cu_seqlens) - 1 sequences packed token-major,
    q, k [total,H,dk], v [total,H,dv] bfloat16; sequence b is rows
    cu_seqlens[b] .. cu_seqlens[b+1]-1 (cu_seqlens int64 on the device),
    max_seqlen its longest length.  Each sequence starts from an empty
    state.  Returns (y [total,H,dv], A_final [B,H,dk,dv] float32 or None with
    l1_only)."""
    total, H, dk = k.shape
    dv = v.shape[-1]
    B = cu_seqlens.numel() - 1
    if B < 1:
        raise ValueError("cu_seqlens needs at least two entries")
    _expect(cu_seqlens, "cu_seqlens", (B + 1,), torch.int64)
    _expect(q, "q", (total, H, dk), k.dtype)
    _expect(v, "v", (total, H, dv), k.dtype)
    for name, t in (("lam", lam), ("eta", eta), ("g", g)):
        _expect(t, name, (H,), torch.float32)
    _expect(y, "y", (total, H, dv), k.dtype)
    _expect(A_final, "A_final", (B, H, dk, dv), torch.float32)
    desc = make_prefill_desc(B, H, int(max_seqlen), dk, dv, W, C, _dtype_code(k), l1_only)
    if y is None:
        y = torch.empty((total, H, dv), dtype=k.dtype, device=k.device)
    if A_final is None and not l1_only:
        A_final = torch.empty((B, H, dk, dv), dtype=torch.float32, device=k.device)
    need = _lib.tc_prefill_varlen_workspace_size(ctypes.byref(desc))
    if need == SIZE_ERROR:
        raise TCError(2, "tc_prefill_varlen_workspace_size")
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=k.device)
    _contig(q, k, v, cu_seqlens, lam, eta, g, y, A_final, workspace)
    _dev_check(q, k, v, cu_seqlens, lam, eta, g, y, A_final, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = _lib.tc_prefill_varlen(ctypes.byref(desc), _ptr(cu_seqlens), int(total), _ptr(q),
                                _ptr(k), _ptr(v), _ptr(lam), _ptr(eta), _ptr(g), _ptr(y),
                                _ptr(A_final), _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "tc_prefill_varlen")
    return y, A_final


def write_pairs(k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor, eta: torch.Tensor,
                A: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A after writing the pairs k [B,H,n,dk], v [B,H,n,dv] in order into an
    empty state with the layer's write, A <- lam A + eta k v^T per pair:
    tc_prefill_from_state, state only, over the n pairs plus one token with
    W = 1, so that exactly the n pairs are evicted (one chunk of n)."""
    B, H, n, dk = k.shape
    dv = v.shape[-1]
    pad_k = torch.zeros((B, H, 1, dk), dtype=k.dtype, device=k.device)
    pad_v = torch.zeros((B, H, 1, dv), dtype=v.dtype, device=v.device)
    ks = torch.cat([k, pad_k], dim=2).contiguous()
    vs = torch.cat([v, pad_v], dim=2).contiguous()
    g = torch.zeros(H, dtype=torch.float32, device=k.device)
    _, A = prefill_from_state(None, ks, vs, lam, eta, g, 1, max(n, 1), 0, state_only=True,
                              A_final=A)
    return A


def prefill_from_state(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                       lam: torch.Tensor, eta: torch.Tensor, g: torch.Tensor, W: int, C: int,
                       t0: int, halo_k: Optional[torch.Tensor] = None,
                       halo_v: Optional[torch.Tensor] = None, A_init: Optional[torch.Tensor] = None,
                       *, state_only: bool = False, l1_only: bool = False,
                       delta_rule: bool = False, chunk_mean: bool = False,
                       y: Optional[torch.Tensor] = None,
                       A_final: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None):
    """tc_prefill_from_state: the layer over the new tokens k, v [B,H,T,d]
    (queries q, unless state_only) starting at global position t0, given the
    halo (keys / values of tokens t0 - min(t0, W) .. t0 - 1, oldest first) and
    A_init (A after the evictions before t0; None = zero).  Returns
    (y, A_final); y is None with state_only."""
    B, H, T, dk = k.shape
    dv = v.shape[-1]
    desc = make_prefill_desc(B, H, T, dk, dv, W, C, _dtype_code(k), l1_only, state_only,
                             delta_rule, chunk_mean)
    _expect_layer(B, H, T, dk, dv, k.dtype, q, k, v, lam, eta, g, y, A_final)
    n_halo = min(int(t0), int(W))
    _expect(halo_k, "halo_k", (B, H, n_halo, dk), k.dtype)
    _expect(halo_v, "halo_v", (B, H, n_halo, dv), k.dtype)
    _expect(A_init, "A_init", (B, H, dk, dv), torch.float32)
    if y is None and not state_only:
        y = torch.empty((B, H, T, dv), dtype=k.dtype, device=k.device)
    if A_final is None and not l1_only:
        A_final = torch.empty((B, H, dk, dv), dtype=torch.float32, device=k.device)
    need = _lib.tc_prefill_from_state_workspace_size(ctypes.byref(desc), int(t0))
    if need == SIZE_ERROR:
        raise TCError(1, "tc_prefill_from_state_workspace_size")
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=k.device)
    _contig(q, k, v, lam, eta, g, y, A_final, workspace, halo_k, halo_v, A_init)
    _dev_check(q, k, v, lam, eta, g, y, A_final, workspace, halo_k, halo_v, A_init)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = _lib.tc_prefill_from_state(ctypes.byref(desc), int(t0), _ptr(halo_k), _ptr(halo_v),
                                    _ptr(A_init), _ptr(q), _ptr(k), _ptr(v), _ptr(lam),
                                    _ptr(eta), _ptr(g), _ptr(y), _ptr(A_final), _ptr(workspace),
                                    ws_bytes, _stream(stream))
    _check(st, "tc_prefill_from_state")
    return y, A_final


def state_fold(dA: torch.Tensor, E: torch.Tensor, lam: torch.Tensor,
               A_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """tc_state_fold: dA [n_parts,B,H,dk,dv] float32, E [n_parts] int64,
    lam [H] float32 (all on the device).  Returns the state before piece
    n_parts."""
    n, B, H, dk, dv = dA.shape
    if A_out is None:
        A_out = torch.empty((B, H, dk, dv), dtype=torch.float32, device=lam.device)
    _contig(dA, E, lam, A_out)
    _dev_check(dA, E, lam, A_out)
    if dA.dtype != torch.float32 or E.dtype != torch.int64:
        raise TypeError("dA must be float32 and E int64")
    _expect(E, "E", (n,), torch.int64)
    _expect(lam, "lam", (H,), torch.float32)
    _expect(A_out, "A_out", (B, H, dk, dv), torch.float32)
    st = _lib.tc_state_fold(B, H, dk, dv, n, _ptr(dA) if n else None, _ptr(E) if n else None,
                            _ptr(lam), _ptr(A_out), _stream(stream))
    _check(st, "tc_state_fold")
    return A_out


def backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor,
             eta: torch.Tensor, g: torch.Tensor, W: int, dy: torch.Tensor, *,
             workspace: Optional[torch.Tensor] = None, stream=None):
    """tc_backward: gradients of L = sum <dy, y> for the layer over q, k, v
    [B,H,T,d] (from an empty state, outer-product write).  Returns
    (dq, dk, dv [float32, input layout], dlam, deta, dg [H] float32)."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    desc = make_prefill_desc(B, H, T, dk, dv, W, 1, _dtype_code(q))
    _expect_layer(B, H, T, dk, dv, q.dtype, q, k, v, lam, eta, g)
    _expect(dy, "dy", (B, H, T, dv), q.dtype)
    f = dict(dtype=torch.float32, device=q.device)
    dq, dkk, dvv = torch.empty(B, H, T, dk, **f), torch.empty(B, H, T, dk, **f), torch.empty(B, H, T, dv, **f)
    dl, de, dg_ = torch.empty(H, **f), torch.empty(H, **f), torch.empty(H, **f)
    need = _lib.tc_backward_workspace_size(ctypes.byref(desc))
    if need == SIZE_ERROR:
        raise TCError(1, "tc_backward_workspace_size")
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _contig(q, k, v, lam, eta, g, dy, workspace)
    _dev_check(q, k, v, lam, eta, g, dy, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = _lib.tc_backward(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(eta),
                          _ptr(g), _ptr(dy), _ptr(dq), _ptr(dkk), _ptr(dvv), _ptr(dl), _ptr(de),
                          _ptr(dg_), _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "tc_backward")
    return dq, dkk, dvv, dl, de, dg_


def backward_launch_count(q: torch.Tensor, W: int, v: Optional[torch.Tensor] = None):
    """(launches, tensor_cores) of one tc_backward call on tensors shaped like
    q [B,H,T,d_k] (and v [B,H,T,d_v], default q's shape) with window W."""
    B, H, T, dk = q.shape
    dv = dk if v is None else v.shape[-1]
    desc = make_prefill_desc(B, H, T, dk, dv, W, 1, _dtype_code(q))
    tcf = _int(0)
    n = _lib.tc_backward_launch_count(ctypes.byref(desc), ctypes.byref(tcf))
    if n < 0:
        raise TCError(1, "tc_backward_launch_count")
    return int(n), bool(tcf.value)


def prefill_launch_count(desc: PrefillDesc) -> int:
    """Kernel launches one tc_prefill call enqueues for desc."""
    n = _lib.tc_prefill_launch_count(ctypes.byref(desc))
    if n < 0:
        raise TCError(1, "tc_prefill_launch_count")
    return int(n)


_PATHS = {"auto": TC_PATH_AUTO, "fused": TC_PATH_FUSED, "general": TC_PATH_GENERAL}


def set_prefill_path(path) -> None:
    """tc_set_prefill_path: "auto" (default), "fused" or "general" (or the
    TC_PATH_* value), for calls both tensor-core paths can take.  Process-wide."""
    code = _PATHS.get(path, path) if isinstance(path, str) else int(path)
    if not isinstance(code, int):
        raise TCError(1, "tc_set_prefill_path")
    _check(_lib.tc_set_prefill_path(code), "tc_set_prefill_path")


def get_prefill_path() -> str:
    """The current tc_set_prefill_path setting, by name."""
    code = int(_lib.tc_get_prefill_path())
    return {v: k for k, v in _PATHS.items()}[code]


class prefill_path:
    """Context manager: tc_set_prefill_path(path) inside, the previous setting after."""

    def __init__(self, path):
        self.path = path

    def __enter__(self):
        self.prev = get_prefill_path()
        set_prefill_path(self.path)
        return self

    def __exit__(self, *exc):
        set_prefill_path(self.prev)
        return False


def prefill_path_for(desc: PrefillDesc, t0: int = 0):
    """tc_prefill_path_for: "fused" or "general", the tensor-core path a call
    described by desc (continuing at t0) would take now; None when neither takes it."""
    code = int(_lib.tc_prefill_path_for(ctypes.byref(desc), ctypes.c_int64(int(t0))))
    return None if code < 0 else {TC_PATH_FUSED: "fused", TC_PATH_GENERAL: "general"}[code]


NO_ALLOC_SCRATCH_BYTES = 16 << 20


def prefill_no_alloc(q, k, v, lam, eta, g, W, C, *, l1_only=False, y=None, A_final=None,
                     stream=None):
    """tc_prefill_no_alloc: tc_prefill using the library's built-in scratch
    array (no workspace argument) for callers that cannot allocate device
    memory.  y / A_final are allocated here by PyTorch only when not given."""
    desc = _desc_of(q, v, W, C, l1_only)
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    _expect_layer(B, H, T, dk, dv, q.dtype, q, k, v, lam, eta, g, y, A_final)
    if y is None:
        y = torch.empty((B, H, T, dv), dtype=q.dtype, device=q.device)
    if A_final is None and not l1_only:
        A_final = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    _contig(q, k, v, lam, eta, g, y, A_final)
    _dev_check(q, k, v, lam, eta, g, y, A_final)
    st = _lib.tc_prefill_no_alloc(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(lam),
                                  _ptr(eta), _ptr(g), _ptr(y), _ptr(A_final), _stream(stream))
    _check(st, "tc_prefill_no_alloc")
    return y, A_final


def prefill_host_workspace_size(desc: PrefillDesc) -> int:
    n = _lib.tc_prefill_host_workspace_size(ctypes.byref(desc))
    if n == SIZE_ERROR:
        raise TCError(1, "tc_prefill_host_workspace_size")
    return int(n)


def prefill_host(q, k, v, lam, eta, g, W, C, y, A_final=None, *, workspace, l1_only=False,
                 stream=None):
    """tc_prefill_host: q, k, v, lam, eta, g, y (and A_final) are HOST tensors
    (pinned for asynchronous copies); workspace is a device byte tensor of
    prefill_host_workspace_size bytes.  Enqueued on stream; synchronize
    before reading y."""
    desc = _desc_of(q, v, W, C, l1_only)
    B, H, T, dk = q.shape
    _expect_layer(B, H, T, dk, v.shape[-1], q.dtype, q, k, v, lam, eta, g, y, A_final)
    if y is None:
        raise ValueError("y (a host tensor) is required")
    _contig(q, k, v, lam, eta, g, y, A_final, workspace)
    _dev_check(workspace)
    st = _lib.tc_prefill_host(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(lam),
                              _ptr(eta), _ptr(g), _ptr(y), _ptr(A_final), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "tc_prefill_host")
    return y, A_final


@dataclass
class DecodeState:
    """Streaming state (caller-owned device tensors, updated in place):
    ring_k [B,H,W,dk], ring_v [B,H,W,dv], A [B,H,dk,dv] float32, lam/eta/g
    [H] float32, the clock t (tokens consumed so far) and the write rule
    (TC_WRITE_OUTER, the paper's layer, or TC_WRITE_DELTA)."""
    ring_k: torch.Tensor
    ring_v: torch.Tensor
    A: torch.Tensor
    lam: torch.Tensor
    eta: torch.Tensor
    g: torch.Tensor
    t: int
    write_rule: int = 0

    def c_struct(self) -> DecodeStateC:
        B, H, W, dk = self.ring_k.shape
        dv = self.ring_v.shape[-1]
        _dtype_code(self.ring_k)
        _expect(self.ring_v, "ring_v", (B, H, W, dv), self.ring_k.dtype)
        _expect(self.A, "A", (B, H, dk, dv), torch.float32)
        for name, t in (("lam", self.lam), ("eta", self.eta), ("g", self.g)):
            _expect(t, name, (H,), torch.float32)
        _contig(self.ring_k, self.ring_v, self.A, self.lam, self.eta, self.g)
        _dev_check(self.ring_k, self.ring_v, self.A, self.lam, self.eta, self.g)
        return DecodeStateC(B, H, dk, dv, W, int(self.t), _dtype_code(self.ring_k),
                            self.ring_k.data_ptr(), self.ring_v.data_ptr(), self.A.data_ptr(),
                            self.lam.data_ptr(), self.eta.data_ptr(), self.g.data_ptr(),
                            int(self.write_rule))

    @staticmethod
    def empty(B, H, W, dk, dv, lam, eta, g, dtype=torch.bfloat16, device="cuda"):
        return DecodeState(torch.zeros((B, H, W, dk), dtype=dtype, device=device),
                           torch.zeros((B, H, W, dv), dtype=dtype, device=device),
                           torch.zeros((B, H, dk, dv), dtype=torch.float32, device=device),
                           lam, eta, g, 0)


def _expect_step(state: DecodeState, q, k, v, y):
    """q, k [B,H,dk], v and y [B,H,dv] in the ring's dtype."""
    B, H, _, dk = state.ring_k.shape
    dv = state.ring_v.shape[-1]
    dt = state.ring_k.dtype
    _expect(q, "q", (B, H, dk), dt)
    _expect(k, "k", (B, H, dk), dt)
    _expect(v, "v", (B, H, dv), dt)
    _expect(y, "y", (B, H, dv), dt)


def decode_step(state: DecodeState, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """tc_decode_step: q, k [B,H,dk], v [B,H,dv] device tensors in the ring's
    dtype.  Updates the ring and A in place, advances state.t, returns y."""
    cs = state.c_struct()
    _expect_step(state, q, k, v, y)
    if y is None:
        y = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    _contig(q, k, v, y)
    _dev_check(q, k, v, y)
    st = _lib.tc_decode_step(ctypes.byref(cs), _ptr(q), _ptr(k), _ptr(v), _ptr(y),
                             _stream(stream))
    _check(st, "tc_decode_step")
    state.t = int(cs.t)
    return y


def decode_step_ragged(state: DecodeState, t_rows: torch.Tensor, q: torch.Tensor,
                       k: torch.Tensor, v: torch.Tensor, y: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """tc_decode_step_ragged: one step for every batch row b at its own clock
    t_rows[b] (device int64 [B]; negative = empty row, left untouched).  The
    library advances the non-negative clocks on the device; state.t is not
    used."""
    cs = state.c_struct()
    _expect_step(state, q, k, v, y)
    _expect(t_rows, "t_rows", (state.ring_k.shape[0],), torch.int64)
    if y is None:
        y = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    _contig(q, k, v, y, t_rows)
    _dev_check(q, k, v, y, t_rows)
    st = _lib.tc_decode_step_ragged(ctypes.byref(cs), _ptr(t_rows), _ptr(q), _ptr(k), _ptr(v),
                                    _ptr(y), _stream(stream))
    _check(st, "tc_decode_step_ragged")
    return y


def decode_step_host_workspace_size(state: DecodeState) -> int:
    cs = state.c_struct()
    n = _lib.tc_decode_step_host_workspace_size(ctypes.byref(cs))
    if n == SIZE_ERROR:
        raise TCError(1, "tc_decode_step_host_workspace_size")
    return int(n)


def decode_step_host(state: DecodeState, q, k, v, y, *, workspace, stream=None):
    """tc_decode_step_host: q, k, v, y are HOST tensors (pinned); the state
    stays on the device.  Enqueued on stream; synchronize before reading y."""
    cs = state.c_struct()
    _expect_step(state, q, k, v, y)
    _contig(q, k, v, y, workspace)
    _dev_check(workspace)
    st = _lib.tc_decode_step_host(ctypes.byref(cs), _ptr(q), _ptr(k), _ptr(v), _ptr(y),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream(stream))
    _check(st, "tc_decode_step_host")
    state.t = int(cs.t)
    return y


# ---- rotary positions and the paged cache --------------------------------------

class Rotary:
    """Rotary positions (tc_rotary): the head's leading `rot` dimensions are
    turned by position * frequency.  `interleaved` pairs neighbours instead of
    halves; factor, low, high and train_len extend the context (factor alone:
    linear interpolation; with low < high: by parts); gain multiplies the
    rotated part.  Immutable; make it once and pass it to every call."""

    __slots__ = ("c", "ref")

    def __init__(self, rot: int, base: float = 10000.0, *, interleaved: bool = False,
                 factor: float = 1.0, low: float = 0.0, high: float = 0.0, train_len: float = 0.0,
                 gain: float = 1.0):
        if rot < 0 or rot % 2:
            raise ValueError("rot must be even and not negative")
        object.__setattr__(self, "c", RotaryC(int(rot), int(bool(interleaved)), float(base),
                                              float(factor), float(low), float(high),
                                              float(train_len), float(gain)))
        object.__setattr__(self, "ref", ctypes.pointer(self.c))

    def __setattr__(self, name, value):
        raise AttributeError("Rotary is immutable")


# tc_rotate_desc, tc_append_args and tc_step_args as struct formats: packing them
# takes a tenth of the time that filling a ctypes structure does, and a call of a
# few microseconds feels it.
_PACK_ROTATE = struct.Struct("=5qiI12q")
_PACK_APPEND = struct.Struct("=2q3Q9q3Q")
_PACK_STEP = struct.Struct("=q3Q6q2Q2qI4x")
assert (_PACK_ROTATE.size, _PACK_APPEND.size, _PACK_STEP.size) == tuple(
    ctypes.sizeof(s) for s in (RotateDesc, AppendArgs, StepArgs))


_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _addr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _raw_stream(dev: int, *ts, stream=None, used=(), made=False):
    """The stream to launch on, for tensors that must all be on CUDA device
    `dev`, the current one.  `used`: what the call may have allocated itself,
    on the current stream; the allocator learns that a given stream uses it.
    `made`: it did allocate: the memory may be a block that work queued on the
    current stream still writes, so a given stream waits for that work first."""
    for t in ts:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensor on {t.device}; the call's other tensors are on "
                             f"{'the CPU' if dev < 0 else f'cuda:{dev}'}")
    if dev < 0:
        raise ValueError("the tensors must be on a CUDA device")
    if _current_device() != dev:
        raise ValueError(f"tensors on cuda:{dev} but the current CUDA device is cuda:{_current_device()}; "
                         "call under torch.cuda.device(...) of the tensors' device")
    if stream is None:
        return _current_stream(dev)
    if made and stream.cuda_stream != _current_stream(dev):
        stream.wait_stream(torch.cuda.current_stream(dev))
    for t in used:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream


def _rows(t: torch.Tensor, name: str, shape, dtype):
    """Rows [..., d] with a contiguous head dimension; returns the strides."""
    if t.shape != shape or t.dtype is not dtype:
        _expect(t, name, shape, dtype)
    s = t.stride()
    if s[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the head dimension must be contiguous")
    return s


def _rotate(q, k, rotary, positions, t0, q_out, k_out, flags, stream):
    qn, dtype = q.shape, q.dtype
    if len(qn) != 4:
        raise ValueError("q must be [B,Hq,T,d]")
    B, Hq, T, d = qn
    made = q_out is None or (k is not None and k_out is None)
    if q_out is None:
        q_out = torch.empty(qn, dtype=dtype, device=q.device)
    a, c = _rows(q, "q", qn, dtype), _rows(q_out, "q_out", qn, dtype)
    if k is None:
        if k_out is not None:
            raise ValueError("k_out without k")
        H, b, e, kp, kop = 0, _NO_STRIDE, _NO_STRIDE, 0, 0
    else:
        kn = k.shape
        if len(kn) != 4 or kn[0] != B or kn[2] != T or kn[3] != d:
            raise ValueError(f"k has shape {tuple(kn)}; expected [{B},H,{T},{d}]")
        H = kn[1]
        if k_out is None:
            k_out = torch.empty(kn, dtype=dtype, device=q.device)
        b, e = _rows(k, "k", kn, dtype), _rows(k_out, "k_out", kn, dtype)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    pp = 0
    if positions is not None:
        _expect(positions, "positions", (B, T), torch.int64)
        _contig(positions)
        pp = positions.data_ptr()
    desc = _PACK_ROTATE.pack(B, Hq, H, T, d, _dtype_code(q), flags, a[0], a[1], a[2], b[0], b[1], b[2], c[0], c[1], c[2],
                             e[0], e[1], e[2])
    s = _raw_stream(q.get_device(), k, q_out, k_out, positions, stream=stream, used=(q_out, k_out), made=made)
    st = _lib.tc_rotate(desc, rotary.ref, pp, t0, q.data_ptr(), kp, q_out.data_ptr(), kop, s)
    if st:
        raise TCError(st, "tc_rotate")
    return q_out, k_out


_NO_STRIDE = (0, 0, 0)


def rotate(q: torch.Tensor, k: Optional[torch.Tensor], rotary: Rotary, *,
           positions: Optional[torch.Tensor] = None, t0: int = 0, q_out: Optional[torch.Tensor] = None,
           k_out: Optional[torch.Tensor] = None, stream=None):
    """tc_rotate: q [B,Hq,T,d] and k [B,H,T,d] (or None) turned by their
    positions: positions [B,T] int64, or t0, t0 + 1, ...  Any strides with a
    contiguous head dimension (slices of a fused projection, transposed
    views); the outputs are contiguous [B,heads,T,d] unless given, and may be
    the inputs.  Returns (q_out, k_out)."""
    return _rotate(q, k, rotary, positions, t0, q_out, k_out, 0, stream)


def rotate_backward(dq: torch.Tensor, dk: Optional[torch.Tensor], rotary: Rotary, *,
                    positions: Optional[torch.Tensor] = None, t0: int = 0,
                    dq_out: Optional[torch.Tensor] = None, dk_out: Optional[torch.Tensor] = None,
                    stream=None):
    """tc_rotate with TC_ROTATE_BACKWARD: gradients of rotate's inputs from
    gradients of its outputs (those that backward returns, for instance)."""
    return _rotate(dq, dk, rotary, positions, t0, dq_out, dk_out, TC_ROTATE_BACKWARD, stream)


class PagedCache:
    """Paged streaming state (tc_paged_cache): caller-owned device tensors,
    updated in place by the cache_* calls.

    k_pages, v_pages [n_pages,H,page,d] (float32 or bfloat16), table
    [B,max_pages] int32, lens and clocks [B] int64 (pairs held; tokens consumed;
    a negative length is an empty row); mass float32 and pos int32
    [n_pages,H,page] for accumulation and eviction; A [B,H,d,d] float32 with
    lam, eta [H] for the memory.  The tensors are checked here, once, and
    cannot be exchanged afterwards (their contents can)."""

    __slots__ = ("k_pages", "v_pages", "table", "lens", "clocks", "mass", "pos", "A", "lam", "eta",
                 "c", "ref", "B", "H", "d", "dtype", "device", "dev")

    def __init__(self, k_pages, v_pages, table, lens, clocks, *, mass=None, pos=None, A=None, lam=None,
                 eta=None):
        if k_pages.dim() != 4 or table.dim() != 2:
            raise ValueError("k_pages must be [n_pages,H,page,d] and table [B,max_pages]")
        n_pages, H, page, d = k_pages.shape
        B, max_pages = table.shape
        dt = _dtype_code(k_pages)
        _expect(v_pages, "v_pages", k_pages.shape, k_pages.dtype)
        _expect(table, "table", (B, max_pages), torch.int32)
        _expect(lens, "lens", (B,), torch.int64)
        _expect(clocks, "clocks", (B,), torch.int64)
        _expect(mass, "mass", (n_pages, H, page), torch.float32)
        _expect(pos, "pos", (n_pages, H, page), torch.int32)
        if (mass is None) != (pos is None):
            raise ValueError("mass and pos go together")
        _expect(A, "A", (B, H, d, d), torch.float32)
        if A is not None:
            if lam is None or eta is None:
                raise ValueError("A needs lam and eta")
            _expect(lam, "lam", (H,), torch.float32)
            _expect(eta, "eta", (H,), torch.float32)
        ts = (k_pages, v_pages, table, lens, clocks, mass, pos, A, lam, eta)
        _contig(*ts)
        if any(t is not None and t.device != k_pages.device for t in ts):
            raise ValueError("the cache's tensors must be on one device")
        p = [None if t is None else t.data_ptr() for t in ts]
        c = PagedCacheC(B, H, d, page, n_pages, max_pages, dt, p[0], p[1], p[5], p[6], p[2], p[3], p[4],
                        p[7], p[8] if A is not None else None, p[9] if A is not None else None)
        for name, x in zip(self.__slots__, ts + (c, ctypes.pointer(c), B, H, d, k_pages.dtype, k_pages.device,
                                               k_pages.get_device())):
            object.__setattr__(self, name, x)

    def __setattr__(self, name, value):
        raise AttributeError("a PagedCache's tensors are fixed; make another one")

    @staticmethod
    def empty(B, H, d, page, n_pages, max_pages, *, lam=None, eta=None, dtype=torch.bfloat16,
              device="cuda"):
        """An empty cache: rows hold nothing (lens 0), no page is dealt (table
        -1: the caller's allocator fills it), with a memory when lam and eta
        are given."""
        f = dict(dtype=torch.float32, device=device)
        return PagedCache(torch.zeros((n_pages, H, page, d), dtype=dtype, device=device),
                          torch.zeros((n_pages, H, page, d), dtype=dtype, device=device),
                          torch.full((B, max_pages), -1, dtype=torch.int32, device=device),
                          torch.zeros(B, dtype=torch.int64, device=device),
                          torch.zeros(B, dtype=torch.int64, device=device),
                          mass=torch.zeros((n_pages, H, page), **f),
                          pos=torch.zeros((n_pages, H, page), dtype=torch.int32, device=device),
                          A=None if lam is None else torch.zeros((B, H, d, d), **f), lam=lam, eta=eta)


def _workspace(size: int, where: str, workspace, device):
    if size == SIZE_ERROR:
        raise TCError(1, where)
    if workspace is None:
        workspace = torch.empty(max(size, 1), dtype=torch.uint8, device=device)
    elif not workspace.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return workspace, workspace.nbytes


def _new_workspace(size: int, where: str, cache):
    return _workspace(size, where, None, cache.device)[0]


def cache_append(cache: PagedCache, k: torch.Tensor, v: torch.Tensor, *, rotary: Optional[Rotary] = None,
                 q: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                 mass: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None, stream=None):
    """tc_cache_append: tokens k, v [B,H,T,d] enter their rows' pages, k rotated
    by the row's clock (rotary None: as it is); of row b the first counts[b]
    (int64 [B]; None: all T).  mass [B,H,T] float32: the weights they start
    with (None: 0).  q [B,Hq,T,d], the same tokens' queries, is rotated into
    q_out, which is returned (None without q).  k, v and q may have any strides
    with a contiguous head dimension."""
    if k.dim() != 4:
        raise ValueError("k must be [B,H,T,d]")
    B, H, d, T = cache.B, cache.H, cache.d, k.shape[2]
    kn = (B, H, T, d)
    ks, vs = _rows(k, "k", kn, cache.dtype), _rows(v, "v", kn, cache.dtype)
    qs, Hq = _NO_STRIDE, 0
    made = q is not None and q_out is None
    if q is not None:
        if q.dim() != 4:
            raise ValueError("q must be [B,Hq,T,d]")
        Hq = q.shape[1]
        qn = (B, Hq, T, d)
        qs = _rows(q, "q", qn, cache.dtype)
        if q_out is None:
            q_out = torch.empty(qn, dtype=q.dtype, device=q.device)
        elif q_out.shape != qn or q_out.dtype is not cache.dtype:
            _expect(q_out, "q_out", qn, cache.dtype)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if counts is not None:
        _expect(counts, "counts", (B,), torch.int64)
    if mass is not None:
        _expect(mass, "mass", (B, H, T), torch.float32)
    _contig(counts, mass, q_out)
    s = _raw_stream(cache.dev, k, v, q, q_out, counts, mass, stream=stream, used=(q_out,), made=made)
    a = _PACK_APPEND.pack(T, Hq, _addr(q), k.data_ptr(), v.data_ptr(), *qs[:3], *ks[:3], *vs[:3], _addr(counts),
                          _addr(mass), _addr(q_out))
    st = _lib.tc_cache_append(cache.ref, None if rotary is None else rotary.ref, a, s)
    if st:
        raise TCError(st, "tc_cache_append")
    return q_out


def cache_attend_workspace(cache: PagedCache, Hq: int, *, accumulate: bool = False) -> torch.Tensor:
    """A workspace for cache_attend on this cache (one per concurrent stream)."""
    n = _lib.tc_cache_attend_workspace_size(cache.ref, int(Hq), TC_CACHE_ACCUMULATE if accumulate else 0)
    return _new_workspace(n, "tc_cache_attend_workspace_size", cache)


def cache_attend(cache: PagedCache, q: torch.Tensor, *, g: Optional[torch.Tensor] = None,
                 accumulate: bool = False, y: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """tc_cache_attend: attention of one token per row, q [B,Hq,d] (rotated),
    over the row's pairs, plus sigmoid(g) q A when g [Hq] float32 is given.
    accumulate adds each pair's weight to the cache's mass.  Returns y
    [B,Hq,d]; rows that are empty (negative length) are not written."""
    Hq = _query_heads(cache, q)
    if g is not None:
        _expect(g, "g", (Hq,), torch.float32)
        if cache.A is None:
            raise ValueError("g reads the memory, but the cache has none")
    if accumulate and cache.mass is None:
        raise ValueError("accumulate needs a cache with mass")
    made = y is None or workspace is None
    if y is None:
        y = torch.empty_like(q)
    elif y.shape != q.shape or y.dtype is not cache.dtype:
        _expect(y, "y", q.shape, cache.dtype)
    flags = TC_CACHE_ACCUMULATE if accumulate else 0
    n = 0 if workspace is not None else _lib.tc_cache_attend_workspace_size(cache.ref, Hq, flags)
    workspace, room = _workspace(n, "tc_cache_attend_workspace_size", workspace, cache.device)
    _contig(q, g, y)
    s = _raw_stream(cache.dev, q, g, y, workspace, stream=stream, used=(y, workspace), made=made)
    st = _lib.tc_cache_attend(cache.ref, Hq, q.data_ptr(), _addr(g), y.data_ptr(), flags, workspace.data_ptr(), room, s)
    if st:
        raise TCError(st, "tc_cache_attend")
    return y


def _query_heads(cache: PagedCache, q: torch.Tensor) -> int:
    if q.dim() != 3:
        raise ValueError("q must be [B,Hq,d]")
    Hq = q.shape[1]
    _rows(q, "q", (cache.B, Hq, cache.d), cache.dtype)
    if Hq < 1 or Hq % cache.H:
        raise ValueError(f"{Hq} query heads over {cache.H} key/value heads")
    return Hq


def cache_evict_workspace(cache: PagedCache) -> torch.Tensor:
    """A workspace for cache_evict on this cache (one per concurrent stream)."""
    return _new_workspace(_lib.tc_cache_evict_workspace_size(cache.ref), "tc_cache_evict_workspace_size", cache)


def cache_evict(cache: PagedCache, budget: int, *, recent: int = 1,
                workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """tc_cache_evict: every row that holds more than budget pairs loses its
    least attended ones (per head), which are written into the memory A; the
    pairs of the last `recent` positions go last."""
    if cache.mass is None:
        raise ValueError("eviction needs a cache with mass and pos")
    made = workspace is None
    n = _lib.tc_cache_evict_workspace_size(cache.ref) if made else 0
    workspace, room = _workspace(n, "tc_cache_evict_workspace_size", workspace, cache.device)
    s = _raw_stream(cache.dev, workspace, stream=stream, used=(workspace,), made=made)
    _check(_lib.tc_cache_evict(cache.ref, int(budget), int(recent), workspace.data_ptr(), room, s), "tc_cache_evict")


def cache_step_workspace(cache: PagedCache, Hq: int, *, accumulate: bool = True) -> torch.Tensor:
    """A workspace for cache_step on this cache (one per concurrent stream)."""
    n = _lib.tc_cache_step_workspace_size(cache.ref, int(Hq), TC_CACHE_ACCUMULATE if accumulate else 0)
    return _new_workspace(n, "tc_cache_step_workspace_size", cache)


def cache_step(cache: PagedCache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, budget: int, *,
               rotary: Optional[Rotary] = None, recent: int = 1, g: Optional[torch.Tensor] = None,
               accumulate: bool = True, y: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """tc_cache_step: one serving step of every row, in the layer's order: the
    token's pair k, v [B,H,d] enters (rotated), the least attended pair beyond
    budget leaves into the memory, and q [B,Hq,d] (rotated here) reads both.
    q, k and v may have any strides with a contiguous head dimension.  Returns
    y [B,Hq,d]."""
    Hq = _query_heads(cache, q)
    kn = (cache.B, cache.H, cache.d)
    qs, ks, vs = _rows(q, "q", (cache.B, Hq, cache.d), cache.dtype), _rows(k, "k", kn, cache.dtype), _rows(v, "v", kn, cache.dtype)
    if g is not None:
        _expect(g, "g", (Hq,), torch.float32)
        if cache.A is None:
            raise ValueError("g reads the memory, but the cache has none")
    if cache.mass is None:
        raise ValueError("a step needs a cache with mass and pos")
    made = y is None or workspace is None
    if y is None:
        y = torch.empty((cache.B, Hq, cache.d), dtype=cache.dtype, device=q.device)
    elif y.shape != q.shape or y.dtype is not cache.dtype:
        _expect(y, "y", q.shape, cache.dtype)
    flags = TC_CACHE_ACCUMULATE if accumulate else 0
    n = 0 if workspace is not None else _lib.tc_cache_step_workspace_size(cache.ref, Hq, flags)
    workspace, room = _workspace(n, "tc_cache_step_workspace_size", workspace, cache.device)
    _contig(g, y)
    s = _raw_stream(cache.dev, q, k, v, g, y, workspace, stream=stream, used=(y, workspace), made=made)
    a = _PACK_STEP.pack(Hq, q.data_ptr(), k.data_ptr(), v.data_ptr(), *qs[:2], *ks[:2], *vs[:2], _addr(g), y.data_ptr(),
                        int(budget), int(recent), flags)
    st = _lib.tc_cache_step(cache.ref, None if rotary is None else rotary.ref, a, workspace.data_ptr(), room, s)
    if st:
        raise TCError(st, "tc_cache_step")
    return y


def set_wait_limit_ns(ns: int) -> None:
    """tc_set_wait_limit_ns: limit of the tensor-core kernels' bounded waits
    (0 restores the 2 s default).  Process-wide; meant for tests of the
    timeout path."""
    _lib.tc_set_wait_limit_ns(int(ns))


def device_status(stream=None) -> int:
    """tc_get_device_status: synchronizes stream, returns and clears the
    device status word."""
    return int(_lib.tc_get_device_status(_stream(stream)))
