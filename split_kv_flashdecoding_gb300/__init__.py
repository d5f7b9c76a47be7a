"""split_kv_flashdecoding_gb300 -- split-KV decode attention for GB300 (sm_103a).

A thin Python binding over the C ABI of libfd (include/fd.h).  Every step of
the computation runs in libfd's CUDA kernels; this module only marshals
pointers, sizes and the stream.  PyTorch supplies device memory and streams.

Entry points (same names as the C ABI, minus the ``fd_`` prefix):
  plan(...)          -> PlanInfo        host planner (chunk length, grid size)
  plan_work_items()  -> int32 [n, 5]    the plan's CTAs (b, kv_head, split, t0, t1)
  decode_split(...)                     stage 1: partial (O_i, LSE_i) per split
  merge(...)                            stage 2: LSE merge into O, LSE
  decode(...)        -> (O, LSE)        plan + stage 1 + stage 2
  decode_static_workspace(...)          the same for callers that cannot allocate
                                        (scratch in a fixed array in the library)
  plan_paged(...), decode_paged(...)    the same over a paged KV cache (page tables)
  decode_fp8(...), decode_paged_fp8()   FP8 (E4M3) K/V, one scale per KV head
  decode_int4(...), decode_paged_int4() INT4 K/V, one scale per key row and KV head
  decode_paged_int8(...)                INT8 K/V in pages, one scale per page and KV head
  plan_graph(...), decode_graph(...)    graph-capturable decode (device-side plan)
  merge_states(...)                     merge attention states (sequence shards)
  plan_shared(...), decode_shared(...)  decode over prefixes that requests share
  plan_shared_paged(), decode_shared_paged()  (each prefix attended once), ragged and paged;
  decode_shared_fp8(), decode_shared_paged_fp8()  FP8 (E4M3) K/V
  plan_prefill_paged(...),              attention of one to many tokens a request over an
  prefill_paged_int8(...)               INT8 cache: causal, or over all keys
  plan_rope(...), append_paged(...)     rotary positions and the write of new keys and
  append_paged_fp8(), append_paged_int4(), values into a paged cache
  append_paged_int8()
  fork_pages(...), compact_pages(...)   next page tables on the device, and the page
  copy_pages(...)                       copies they need
  get_device_status(workspace)          read and clear the kernels' error word

There is no CPU fallback: if libfd.so cannot be loaded, importing the library
functions raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np

try:
    import torch
except ImportError:  # pragma: no cover  (host planning works without it)
    torch = None

from ._build_lib import LIB as _LIB_PATH, build

TILE_TOKENS = 32
WORKSPACE_HEADER_BYTES = 256
DEFAULT_TIMEOUT_NS = 1_000_000_000

FD_OK = 0
STATUS_NAMES = {
    0: "FD_OK", -1: "FD_ERR_INVALID_ARG", -2: "FD_ERR_UNSUPPORTED", -3: "FD_ERR_WORKSPACE",
    -4: "FD_ERR_CUDA", -5: "FD_ERR_TIMEOUT", -6: "FD_ERR_DEVICE_BOUNDS", -7: "FD_ERR_NO_PAGES",
}


class FdError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)} ({code})")
        self.code = code


class PlanInfo(ctypes.Structure):
    """Mirror of fd_plan_info (include/fd.h)."""
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_qo_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("group_size", ctypes.c_int32),
        ("chunk", ctypes.c_int32),
        ("total_splits", ctypes.c_int32),
        ("max_splits", ctypes.c_int32),
        ("num_work", ctypes.c_int32),
        ("num_partial_rows", ctypes.c_int32),
        ("num_sms", ctypes.c_int32),
        ("ctas_per_sm", ctypes.c_int32),
        ("total_tokens", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_int64),
        ("timeout_ns", ctypes.c_int64),
    ]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class SharedPlan(ctypes.Structure):
    """Mirror of fd_shared_plan (include/fd.h)."""
    _fields_ = [
        ("suffix", PlanInfo),
        ("num_prefixes", ctypes.c_int32),
        ("chunk", ctypes.c_int32),
        ("num_items", ctypes.c_int32),
        ("num_partial_rows", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("prefix_rows", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_int64),
        ("timeout_ns", ctypes.c_int64),
    ]


class PrefillPlan(ctypes.Structure):
    """Mirror of fd_prefill_plan (include/fd.h)."""
    _fields_ = [(name, ctypes.c_int32) for name in (
        "batch", "num_tokens", "num_qo_heads", "num_kv_heads", "head_dim", "page_size", "causal", "chunk",
        "num_items", "num_partial_rows", "num_merged_rows", "num_page_entries")] + [
        ("workspace_bytes", ctypes.c_int64), ("timeout_ns", ctypes.c_int64)]


class RopeInfo(ctypes.Structure):
    """Mirror of fd_rope_info (include/fd.h)."""
    _fields_ = [
        ("head_dim", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("gain", ctypes.c_float),
        ("step", ctypes.c_uint64 * 64),
    ]


class RopeConfig(ctypes.Structure):
    """Mirror of fd_rope_config (include/fd.h)."""
    _fields_ = [
        ("base", ctypes.c_double),
        ("factor", ctypes.c_double),
        ("trained_len", ctypes.c_double),
        ("low", ctypes.c_double),
        ("high", ctypes.c_double),
        ("scaling", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
    ]


ROPE_SCALINGS = {"linear": 1, "bands": 2, "yarn": 3}

_lock = threading.Lock()
_lib = None

# Every symbol include/fd.h declares, with its ctypes signature.
_P, _I, _I64, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
_PI = ctypes.POINTER(PlanInfo)
_PS = ctypes.POINTER(SharedPlan)
_PP = ctypes.POINTER(PrefillPlan)
_APPEND = [_I, _I, _I, _I, _I, _I, _I, _P, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _I, _P, _P,
           _I64, _P, _P]
SIGNATURES = {
    "fd_status_string": ([_I], ctypes.c_char_p),
    "fd_version": ([], _I),
    "fd_num_sms": ([_I, ctypes.POINTER(ctypes.c_int)], _I),
    "fd_plan": ([_I, _I, _I, _I, _P, _I, _I, _I, _PI], _I),
    "fd_plan_work_items": ([_PI, _P, _P, _I64], _I),
    "fd_decode_split": ([_PI, _P, _P, _P, _P, _F, _P, _P, _P, _I64, _P], _I),
    "fd_merge": ([_PI, _P, _P, _P, _P, _P, _P, _I64, _P], _I),
    "fd_decode": ([_I, _I, _I, _I, _P, _P, _P, _P, _P, _F, _P, _P, _P, _I64, _P], _I),
    "fd_get_device_status": ([_P, _P], _I),
    "fd_decode_static_workspace": ([_I, _I, _I, _I, _P, _P, _P, _P, _P, _F, _P, _P, _P], _I),
    "fd_plan_paged": ([_I, _I, _I, _I, _I, _P, _P, _I, _I, _I, _PI], _I),
    "fd_decode_paged": ([_I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P,
                         _P, _I64, _P], _I),
    "fd_decode_fp8": ([_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _P, _I64, _P], _I),
    "fd_plan_graph": ([_I, _I, _I, _I, _I64, _I, _I, _PI], _I),
    "fd_merge_states": ([_I, _I, _I, _P, _P, _P, _P, _P], _I),
    "fd_decode_graph": ([_PI, _P, _P, _P, _P, _F, _P, _P, _P, _I64, _P], _I),
    "fd_decode_paged_fp8": ([_I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _F,
                             _P, _P, _P, _I64, _P], _I),
    "fd_decode_int4": ([_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _P, _I64, _P], _I),
    "fd_decode_paged_int4": ([_I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _F,
                              _P, _P, _P, _I64, _P], _I),
    "fd_decode_paged_int8": ([_I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _F,
                              _P, _P, _P, _I64, _P], _I),
    "fd_plan_shared": ([_I, _I, _I, _I, _I, _P, _P, _I64, _I, _I, _PS], _I),
    "fd_plan_shared_paged": ([_I, _I, _I, _I, _I, _I, _P, _P, _P, _I64, _I, _I, _PS], _I),
    "fd_decode_shared": ([_PS, _P, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _P, _I64, _P], _I),
    "fd_decode_shared_paged": ([_PS, _I, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _F, _P, _P, _P,
                                _I64, _P], _I),
    "fd_decode_shared_fp8": ([_PS, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _P, _I64, _P], _I),
    "fd_decode_shared_paged_fp8": ([_PS, _I, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _F, _P,
                                    _P, _P, _I64, _P], _I),
    "fd_plan_prefill_paged": ([_I, _I, _I, _I, _I, _P, _P, _P, _I, _I, _I, _PP], _I),
    "fd_prefill_paged_int8": ([_PP, _I, _P, _P, _P, _P, _P, _I64, _P, _P, _P, _P, _F, _P, _P, _P, _I64, _P], _I),
    "fd_plan_rope": ([_I, _I, ctypes.POINTER(RopeConfig), ctypes.POINTER(RopeInfo)], _I),
    "fd_append_paged": (_APPEND + [_P, _I64, _P], _I),
    "fd_append_paged_fp8": (_APPEND + [_P, _P, _P, _I64, _P], _I),
    "fd_append_paged_int4": (_APPEND + [_P, _P, _P, _I64, _P], _I),
    "fd_append_paged_int8": (_APPEND + [_P, _P, _P, _I64, _P], _I),
    "fd_pages_workspace_bytes": ([_I, _I, ctypes.POINTER(ctypes.c_int64)], _I),
    "fd_fork_pages": ([_I, _I, _I, _I, _P, _P, _P, _P, _I, _P, _I, _P, _P, _P, _P, _P, _P, _I64, _P], _I),
    "fd_compact_pages": ([_I, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _I64, _P], _I),
    "fd_copy_pages": ([_I, _P, _P, _I, _I, _P, _P, _P, _I64, _P], _I),
}


def lib(auto_build: bool = True):
    """Load libfd.so (building it first if it is missing or stale)."""
    global _lib
    with _lock:
        if _lib is None:
            path = build() if auto_build else _LIB_PATH
            if not os.path.exists(path):
                raise FdError(-4, f"libfd.so missing at {path}")
            handle = ctypes.CDLL(path)
            for name, (args, res) in SIGNATURES.items():
                fn = getattr(handle, name)
                fn.argtypes = args
                fn.restype = res
            _lib = handle
    return _lib


def _check(rc: int, what: str):
    if rc != FD_OK:
        raise FdError(rc, what)


def _host_indptr(kv_indptr) -> np.ndarray:
    if type(kv_indptr) is np.ndarray and kv_indptr.dtype == np.int32 and kv_indptr.ndim == 1 and \
            kv_indptr.flags.c_contiguous:
        return kv_indptr
    try:
        import torch
        if isinstance(kv_indptr, torch.Tensor):
            kv_indptr = kv_indptr.detach().cpu().numpy()
    except ImportError:  # pragma: no cover
        pass
    a = np.ascontiguousarray(np.asarray(kv_indptr, dtype=np.int32).reshape(-1))
    return a


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream):
    if stream is None:   # the current stream's handle, without building a Stream object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def status_string(code: int) -> str:
    return lib().fd_status_string(code).decode()


def num_sms(device: int = -1) -> int:
    out = ctypes.c_int(0)
    _check(lib().fd_num_sms(device, ctypes.byref(out)), "fd_num_sms")
    return out.value


def plan(batch: int, num_qo_heads: int, num_kv_heads: int, head_dim: int, kv_indptr_host,
         *, num_sms: int = 0, ctas_per_sm: int = 0, chunk: int = 0,
         timeout_ns: int | None = None) -> PlanInfo:
    """fd_plan: choose the chunk length and size the split grid (host only)."""
    ip = _host_indptr(kv_indptr_host)
    if ip.size != batch + 1:
        raise FdError(-1, "kv_indptr must have batch+1 entries")
    info = PlanInfo()
    _check(lib().fd_plan(batch, num_qo_heads, num_kv_heads, head_dim,
                         ip.ctypes.data_as(ctypes.c_void_p), num_sms, ctas_per_sm, chunk,
                         ctypes.byref(info)), "fd_plan")
    if timeout_ns is not None:
        info.timeout_ns = timeout_ns
    return info


def plan_work_items(info: PlanInfo, kv_indptr_host) -> np.ndarray:
    """fd_plan_work_items: int32 [num_work, 5] = (b, kv_head, split, t0, t1)."""
    ip = _host_indptr(kv_indptr_host)
    items = np.zeros((max(info.num_work, 1), 5), dtype=np.int32)
    _check(lib().fd_plan_work_items(ctypes.byref(info), ip.ctypes.data_as(ctypes.c_void_p),
                                    items.ctypes.data_as(ctypes.c_void_p), info.num_work),
           "fd_plan_work_items")
    return items[: info.num_work]


def decode_split(info: PlanInfo, q, k, v, kv_indptr_dev, scale: float, partial_o, partial_lse,
                 workspace, stream=None):
    """fd_decode_split on torch CUDA tensors (stage 1; writes partial_o/partial_lse)."""
    _check(lib().fd_decode_split(ctypes.byref(info), _ptr(q), _ptr(k), _ptr(v),
                                 _ptr(kv_indptr_dev), float(scale), _ptr(partial_o),
                                 _ptr(partial_lse), _ptr(workspace), workspace.numel() *
                                 workspace.element_size(), _stream(stream)), "fd_decode_split")


def merge(info: PlanInfo, kv_indptr_dev, partial_o, partial_lse, o, lse, workspace, stream=None):
    """fd_merge on torch CUDA tensors (stage 2; writes o/lse)."""
    _check(lib().fd_merge(ctypes.byref(info), _ptr(kv_indptr_dev), _ptr(partial_o),
                          _ptr(partial_lse), _ptr(o), _ptr(lse), _ptr(workspace),
                          workspace.numel() * workspace.element_size(), _stream(stream)),
           "fd_merge")


def workspace_bytes(batch, num_qo_heads, num_kv_heads, head_dim, kv_indptr_host) -> int:
    """Workspace fd_decode needs for these arguments on the current device."""
    return plan(batch, num_qo_heads, num_kv_heads, head_dim, kv_indptr_host).workspace_bytes


def decode(q, k, v, kv_indptr_host, kv_indptr_dev, scale: float, *, o=None, lse=None,
           workspace=None, stream=None):
    """fd_decode: q [B,Hq,D], k/v [T,Hkv,D] bf16 CUDA tensors -> (O fp32, LSE fp32).

    kv_indptr_host: int32 [B+1] on the host (numpy or CPU tensor);
    kv_indptr_dev: the same values as an int32 CUDA tensor.
    """
    import torch
    B, Hq, D = q.shape
    Hkv = k.shape[1]
    ip = _host_indptr(kv_indptr_host)
    if o is None:
        o = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        need = plan(B, Hq, Hkv, D, ip).workspace_bytes
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    _check(lib().fd_decode(B, Hq, Hkv, D, ip.ctypes.data_as(ctypes.c_void_p), _ptr(kv_indptr_dev),
                           _ptr(q), _ptr(k), _ptr(v), float(scale), _ptr(o), _ptr(lse),
                           _ptr(workspace), workspace.numel() * workspace.element_size(),
                           _stream(stream)), "fd_decode")
    return o, lse


def decode_static_workspace(q, k, v, kv_indptr_host, kv_indptr_dev, scale: float, *, o=None,
                            lse=None, stream=None):
    """fd_decode_static_workspace: fd_decode for callers that cannot allocate.

    The library keeps the scratch in a fixed device array (16 MiB per GPU), so
    only inputs and outputs are passed; o/lse are allocated here only when not
    given.  Calls that can overlap on the GPU race (they share the array).
    """
    import torch
    B, Hq, D = q.shape
    Hkv = k.shape[1]
    ip = _host_indptr(kv_indptr_host)
    if o is None:
        o = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    _check(lib().fd_decode_static_workspace(B, Hq, Hkv, D, ip.ctypes.data_as(ctypes.c_void_p),
                                            _ptr(kv_indptr_dev), _ptr(q), _ptr(k), _ptr(v),
                                            float(scale), _ptr(o), _ptr(lse), _stream(stream)),
           "fd_decode_static_workspace")
    return o, lse


def plan_paged(batch: int, num_qo_heads: int, num_kv_heads: int, head_dim: int, page_size: int,
               kv_page_indptr_host, kv_last_page_len_host, *, num_sms: int = 0,
               ctas_per_sm: int = 0, chunk: int = 0) -> PlanInfo:
    """fd_plan_paged: the plan of a paged layout (host only)."""
    ip = _host_indptr(kv_page_indptr_host)
    ll = _host_indptr(kv_last_page_len_host)
    if ip.size != batch + 1 or ll.size != batch:
        raise FdError(-1, "kv_page_indptr must have batch+1 and kv_last_page_len batch entries")
    info = PlanInfo()
    _check(lib().fd_plan_paged(batch, num_qo_heads, num_kv_heads, head_dim, page_size,
                               ip.ctypes.data_as(ctypes.c_void_p), ll.ctypes.data_as(ctypes.c_void_p),
                               num_sms, ctas_per_sm, chunk, ctypes.byref(info)), "fd_plan_paged")
    return info


def decode_paged(q, k_pages, v_pages, kv_page_indptr_host, kv_last_page_len_host,
                 kv_page_indptr_dev, kv_last_page_len_dev, kv_page_indices_dev, scale: float, *,
                 o=None, lse=None, workspace=None, stream=None):
    """fd_decode_paged: q [B,Hq,D], page pools k/v [num_pages, page_size, Hkv, D] bf16.

    Page tables as in include/fd.h (host copies of indptr and last-page
    lengths for the plan, device copies plus the page indices for the kernels).
    """
    import torch
    B, Hq, D = q.shape
    num_pages, page_size, Hkv = k_pages.shape[0], k_pages.shape[1], k_pages.shape[2]
    ip = _host_indptr(kv_page_indptr_host)
    ll = _host_indptr(kv_last_page_len_host)
    if o is None:
        o = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        need = plan_paged(B, Hq, Hkv, D, page_size, ip, ll).workspace_bytes
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    _check(lib().fd_decode_paged(B, Hq, Hkv, D, page_size, num_pages,
                                 ip.ctypes.data_as(ctypes.c_void_p),
                                 ll.ctypes.data_as(ctypes.c_void_p), _ptr(kv_page_indptr_dev),
                                 _ptr(kv_last_page_len_dev), _ptr(kv_page_indices_dev), _ptr(q),
                                 _ptr(k_pages), _ptr(v_pages), float(scale), _ptr(o), _ptr(lse),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream)), "fd_decode_paged")
    return o, lse


def _fp8_bytes(x):
    """An FP8 K/V tensor as torch gives it (float8_e4m3fn) or as raw uint8."""
    import torch
    if x.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise FdError(-1, "FP8 K/V must be uint8 or float8_e4m3fn")
    return x


def decode_fp8(q, k_fp8, v_fp8, k_scale, v_scale, kv_indptr_host, kv_indptr_dev, scale: float, *,
               o=None, lse=None, workspace=None, stream=None):
    """fd_decode_fp8: q [B,Hq,D] bf16, k/v [T,Hkv,D] E4M3 bytes (uint8 or
    float8_e4m3fn), k_scale / v_scale fp32 [Hkv] CUDA tensors -> (O, LSE) fp32."""
    import torch
    B, Hq, D = q.shape
    Hkv = k_fp8.shape[1]
    ip = _host_indptr(kv_indptr_host)
    if o is None:
        o = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        need = plan(B, Hq, Hkv, D, ip).workspace_bytes
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    _check(lib().fd_decode_fp8(B, Hq, Hkv, D, ip.ctypes.data_as(ctypes.c_void_p), _ptr(kv_indptr_dev),
                               _ptr(q), _ptr(_fp8_bytes(k_fp8)), _ptr(_fp8_bytes(v_fp8)),
                               _ptr(k_scale), _ptr(v_scale), float(scale), _ptr(o), _ptr(lse),
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream(stream)), "fd_decode_fp8")
    return o, lse


def decode_paged_fp8(q, k_pages_fp8, v_pages_fp8, k_scale, v_scale, kv_page_indptr_host,
                     kv_last_page_len_host, kv_page_indptr_dev, kv_last_page_len_dev,
                     kv_page_indices_dev, scale: float, *, o=None, lse=None, workspace=None,
                     stream=None):
    """fd_decode_paged_fp8: fd_decode_paged over E4M3 page pools with
    per-KV-head fp32 scales."""
    import torch
    B, Hq, D = q.shape
    num_pages, page_size, Hkv = k_pages_fp8.shape[0], k_pages_fp8.shape[1], k_pages_fp8.shape[2]
    ip = _host_indptr(kv_page_indptr_host)
    ll = _host_indptr(kv_last_page_len_host)
    if o is None:
        o = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        need = plan_paged(B, Hq, Hkv, D, page_size, ip, ll).workspace_bytes
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    _check(lib().fd_decode_paged_fp8(B, Hq, Hkv, D, page_size, num_pages,
                                     ip.ctypes.data_as(ctypes.c_void_p),
                                     ll.ctypes.data_as(ctypes.c_void_p), _ptr(kv_page_indptr_dev),
                                     _ptr(kv_last_page_len_dev), _ptr(kv_page_indices_dev), _ptr(q),
                                     _ptr(_fp8_bytes(k_pages_fp8)), _ptr(_fp8_bytes(v_pages_fp8)),
                                     _ptr(k_scale), _ptr(v_scale), float(scale), _ptr(o), _ptr(lse),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _stream(stream)), "fd_decode_paged_fp8")
    return o, lse


def _int4_bytes(x, D: int):
    """Packed INT4 K/V: uint8 with D / 2 bytes per (row, KV head)."""
    import torch
    if x.dtype != torch.uint8 or x.shape[-1] != D // 2:
        raise FdError(-1, "INT4 K/V must be uint8 [..., Hkv, head_dim / 2]")
    return x


def decode_int4(q, k_int4, v_int4, k_scale, v_scale, kv_indptr_host, kv_indptr_dev, scale: float, *,
                o=None, lse=None, workspace=None, stream=None):
    """fd_decode_int4: q [B,Hq,D] bf16, k/v [T,Hkv,D/2] packed four-bit codes
    (uint8), k_scale / v_scale fp32 [Hkv, T] CUDA tensors -> (O, LSE) fp32."""
    import torch
    B, Hq, D = q.shape
    Hkv = k_int4.shape[1]
    ip = _host_indptr(kv_indptr_host)
    if o is None:
        o = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        need = plan(B, Hq, Hkv, D, ip).workspace_bytes
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    _check(lib().fd_decode_int4(B, Hq, Hkv, D, ip.ctypes.data_as(ctypes.c_void_p),
                                _ptr(kv_indptr_dev), _ptr(q), _ptr(_int4_bytes(k_int4, D)),
                                _ptr(_int4_bytes(v_int4, D)), _ptr(k_scale), _ptr(v_scale),
                                float(scale), _ptr(o), _ptr(lse), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(stream)),
           "fd_decode_int4")
    return o, lse


def decode_paged_int4(q, k_pages_int4, v_pages_int4, k_scale, v_scale, kv_page_indptr_host,
                      kv_last_page_len_host, kv_page_indptr_dev, kv_last_page_len_dev,
                      kv_page_indices_dev, scale: float, *, o=None, lse=None, workspace=None,
                      stream=None):
    """fd_decode_paged_int4: fd_decode_paged over packed INT4 page pools
    [num_pages, page_size, Hkv, D/2] with fp32 scales [Hkv, num_pages * page_size]."""
    import torch
    B, Hq, D = q.shape
    num_pages, page_size, Hkv = k_pages_int4.shape[0], k_pages_int4.shape[1], k_pages_int4.shape[2]
    ip = _host_indptr(kv_page_indptr_host)
    ll = _host_indptr(kv_last_page_len_host)
    if o is None:
        o = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        need = plan_paged(B, Hq, Hkv, D, page_size, ip, ll).workspace_bytes
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    _check(lib().fd_decode_paged_int4(B, Hq, Hkv, D, page_size, num_pages,
                                      ip.ctypes.data_as(ctypes.c_void_p),
                                      ll.ctypes.data_as(ctypes.c_void_p), _ptr(kv_page_indptr_dev),
                                      _ptr(kv_last_page_len_dev), _ptr(kv_page_indices_dev), _ptr(q),
                                      _ptr(_int4_bytes(k_pages_int4, D)),
                                      _ptr(_int4_bytes(v_pages_int4, D)), _ptr(k_scale),
                                      _ptr(v_scale), float(scale), _ptr(o), _ptr(lse),
                                      _ptr(workspace), workspace.numel() * workspace.element_size(),
                                      _stream(stream)), "fd_decode_paged_int4")
    return o, lse


def plan_graph(batch: int, num_qo_heads: int, num_kv_heads: int, head_dim: int,
               max_total_tokens: int, *, num_sms: int = 0, chunk: int = 0) -> PlanInfo:
    """fd_plan_graph: a plan for any kv_indptr of at most max_total_tokens keys
    (host only; fixes the chunk, sizes the workspace)."""
    info = PlanInfo()
    _check(lib().fd_plan_graph(batch, num_qo_heads, num_kv_heads, head_dim, int(max_total_tokens),
                               num_sms, chunk, ctypes.byref(info)), "fd_plan_graph")
    return info


def decode_graph(info: PlanInfo, q, k, v, kv_indptr_dev, scale: float, o, lse, workspace,
                 stream=None):
    """fd_decode_graph: device data only (capturable in a CUDA graph); o, lse
    and the workspace (info.workspace_bytes, zero-filled once) are given."""
    _check(lib().fd_decode_graph(ctypes.byref(info), _ptr(kv_indptr_dev), _ptr(q), _ptr(k), _ptr(v),
                                 float(scale), _ptr(o), _ptr(lse), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream)),
           "fd_decode_graph")


def merge_states(o_states, lse_states, *, o=None, lse=None, stream=None):
    """fd_merge_states: o_states fp32 [S, ..., D] and lse_states fp32 [S, ...]
    (S attention states over disjoint parts of the keys) -> merged (O, LSE)."""
    import torch
    S, D = o_states.shape[0], o_states.shape[-1]
    rows = lse_states[0].numel()
    if o is None:
        o = torch.empty(o_states.shape[1:], dtype=torch.float32, device=o_states.device)
    if lse is None:
        lse = torch.empty(lse_states.shape[1:], dtype=torch.float32, device=lse_states.device)
    _check(lib().fd_merge_states(S, rows, D, _ptr(o_states), _ptr(lse_states), _ptr(o), _ptr(lse),
                                 _stream(stream)), "fd_merge_states")
    return o, lse


class _Same:
    """No change of the current device."""

    def __enter__(self):
        pass

    def __exit__(self, *exc):
        return False


_SAME = _Same()


def _on(tensor, stream=None):
    """The tensor's device and the call's stream, made current for the call: its
    launches go there, and what it allocates belongs to that stream."""
    if not tensor.is_cuda:
        raise FdError(-1, "the inputs must be CUDA tensors")
    if stream is not None:
        if stream.device != tensor.device:
            raise FdError(-1, "the stream belongs to another device than the inputs")
        return torch.cuda.stream(stream)
    return _SAME if tensor.get_device() == torch.cuda.current_device() else torch.cuda.device(tensor.device)


def _need(what: str, t, dtype, dev: int) -> int:
    """Address of t, a contiguous tensor of this type on CUDA device `dev`."""
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    raise FdError(-1, f"{what} must be a contiguous {dtype} CUDA tensor on the inputs' device")


def _ws(workspace, dev: int):
    """(address, bytes) of a workspace on the inputs' device."""
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise FdError(-3, "workspace must be a contiguous CUDA tensor on the inputs' device")
    return workspace.data_ptr(), workspace.nbytes


def scale_heads(num_kv_heads: int) -> int:
    """Entries of a page's row of INT8 scales: num_kv_heads rounded up to a multiple of 4."""
    return -(-num_kv_heads // 4) * 4


def _int8_cache(name, k_pages, v_pages, k_scale, v_scale, num_kv_heads, head_dim, dev):
    """Addresses of an INT8 cache's pools and scales, checked against one another."""
    shape = k_pages.shape
    if len(shape) != 4 or v_pages.shape != shape or shape[2] != num_kv_heads or shape[3] != head_dim:
        raise FdError(-1, f"{name}: pools of another shape")
    rows = (shape[0], scale_heads(num_kv_heads))
    if k_scale.shape != rows or v_scale.shape != rows:
        raise FdError(-1, f"{name}: scales must be [num_pages, num_kv_heads rounded up to a multiple of 4]")
    return (_need("k_pages", k_pages, torch.int8, dev), _need("v_pages", v_pages, torch.int8, dev),
            _need("k_scale", k_scale, torch.float32, dev), _need("v_scale", v_scale, torch.float32, dev))


def decode_paged_int8(q, k_pages_int8, v_pages_int8, k_scale, v_scale, kv_page_indptr_host,
                      kv_last_page_len_host, kv_page_indptr_dev, kv_last_page_len_dev,
                      kv_page_indices_dev, scale: float, *, o=None, lse=None, workspace=None,
                      stream=None):
    """fd_decode_paged_int8: fd_decode_paged over int8 page pools
    [num_pages, page_size, Hkv, D] with fp32 scales [num_pages, scale_heads(Hkv)]."""
    shape, pool = q.shape, k_pages_int8.shape
    if len(shape) != 3 or len(pool) != 4:
        raise FdError(-1, "fd_decode_paged_int8: q must be [batch, num_qo_heads, head_dim], pools of four dimensions")
    (B, Hq, D), (num_pages, page_size, Hkv, _) = shape, pool
    ip, ll = _host_indptr(kv_page_indptr_host), _host_indptr(kv_last_page_len_host)
    if ip.size != B + 1 or ll.size != B or kv_page_indptr_dev.numel() != B + 1 or \
            kv_last_page_len_dev.numel() < B or kv_page_indices_dev.numel() < ip[B]:
        raise FdError(-1, "fd_decode_paged_int8: tables of another length than the batch's")
    i32, f32, dev = torch.int32, torch.float32, q.get_device()
    with _on(q, stream):
        if o is None:
            o = torch.empty((B, Hq, D), dtype=f32, device=q.device)
        if lse is None:
            lse = torch.empty((B, Hq), dtype=f32, device=q.device)
        if o.shape != shape or lse.shape != (B, Hq):
            raise FdError(-1, "fd_decode_paged_int8: o must have q's shape and lse [batch, num_qo_heads]")
        if workspace is None:
            need = plan_paged(B, Hq, Hkv, D, page_size, ip, ll).workspace_bytes
            workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
        kp, vp, ks, vs = _int8_cache("fd_decode_paged_int8", k_pages_int8, v_pages_int8, k_scale, v_scale, Hkv, D, dev)
        _check(lib().fd_decode_paged_int8(
            B, Hq, Hkv, D, page_size, num_pages, _host_ptr(ip), _host_ptr(ll),
            _need("kv_page_indptr", kv_page_indptr_dev, i32, dev), _need("kv_last_page_len", kv_last_page_len_dev, i32, dev),
            _need("kv_page_indices", kv_page_indices_dev, i32, dev), _need("q", q, torch.bfloat16, dev), kp, vp, ks, vs,
            float(scale), _need("o", o, f32, dev), _need("lse", lse, f32, dev), *_ws(workspace, dev), _stream(stream)),
            "fd_decode_paged_int8")
    return o, lse


def plan_rope(head_dim: int, rotary_dim: int, *, interleaved: bool = False, base: float = 10000.0,
              scaling=None) -> RopeInfo:
    """fd_plan_rope: the rotary frequencies (host only).  scaling: None,
    ("linear", factor), ("bands", factor, trained_len, low, high) or
    ("yarn", factor, trained_len, low, high)."""
    info = RopeInfo()
    kind, args = 0, []
    if scaling is not None:
        if scaling[0] not in ROPE_SCALINGS or len(scaling) != (2 if scaling[0] == "linear" else 5):
            raise FdError(-1, f"plan_rope: unknown scaling {scaling!r}")
        kind, args = ROPE_SCALINGS[scaling[0]], [float(x) for x in scaling[1:]]
    args += [0.0] * (4 - len(args))
    config = RopeConfig(float(base), *args, kind, int(bool(interleaved)))
    _check(lib().fd_plan_rope(head_dim, rotary_dim, ctypes.byref(config), ctypes.byref(info)), "fd_plan_rope")
    return info


def _heads(what: str, x, dev: int):
    """Token stride (elements) of a bf16 [N, H, D] CUDA tensor with contiguous heads."""
    if x.dtype is torch.bfloat16 and x.get_device() == dev and x.dim() == 3:
        n, h, d = x.shape
        token, head, value = x.stride()
        if (value == 1 and (head == d or h <= 1)) or n * h * d == 0:
            return token if n > 1 else max(token, h * d)
    raise FdError(-1, f"{what} must be a bfloat16 CUDA tensor [tokens, heads, head_dim] with contiguous heads")


def _append(name, pool_dtypes, per_row, q, k, v, k_pages, v_pages, append_indptr, kv_page_indptr,
            kv_last_page_len, kv_page_indices, rope, positions, q_out, workspace, stream, scales):
    N, Hkv, D = k.shape
    Hq = 0 if q is None else q.shape[1]
    B = append_indptr.numel() - 1
    if v.shape != k.shape or (q is not None and (q.shape[0] != N or q.shape[2] != D)):
        raise FdError(-1, f"{name}: q, k and v must have the same tokens and head_dim")
    if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or k_pages.shape[2] != Hkv or \
            k_pages.shape[3] != per_row * D or k_pages.dtype not in pool_dtypes or \
            v_pages.dtype not in pool_dtypes:
        raise FdError(-1, f"{name}: pools of another shape or type")
    if kv_page_indptr.numel() != B + 1 or kv_last_page_len.numel() < B:
        raise FdError(-1, f"{name}: kv_page_indptr must have batch+1 and kv_last_page_len batch entries")
    if positions is not None and positions.numel() < N:
        raise FdError(-1, f"{name}: positions must have an entry for every token")
    num_pages, page_size = k_pages.shape[:2]
    i32, dev = torch.int32, k.get_device()
    with _on(k, stream):
        if q is not None and q_out is None:
            q_out = torch.empty((N, Hq, D), dtype=q.dtype, device=q.device)
        if q is not None and q_out.shape != q.shape:
            raise FdError(-1, f"{name}: q_out must have q's shape")
        if workspace is None:
            workspace = torch.zeros(WORKSPACE_HEADER_BYTES, dtype=torch.uint8, device=k.device)
        _check(getattr(lib(), name)(
            B, N, Hq, Hkv, D, page_size, num_pages, None if rope is None else ctypes.byref(rope),
            _ptr(q), 0 if q is None else _heads("q", q, dev), _ptr(k), _heads("k", k, dev), _ptr(v), _heads("v", v, dev),
            _need("append_indptr", append_indptr, i32, dev), _need("kv_page_indptr", kv_page_indptr, i32, dev),
            _need("kv_last_page_len", kv_last_page_len, i32, dev),
            _need("kv_page_indices", kv_page_indices, i32, dev), kv_page_indices.numel(),
            None if positions is None else _need("positions", positions, i32, dev),
            None if q is None else q_out.data_ptr(), 0 if q is None else _heads("q_out", q_out, dev),
            _need("k_pages", k_pages, k_pages.dtype, dev), _need("v_pages", v_pages, v_pages.dtype, dev),
            *scales, *_ws(workspace, dev), _stream(stream)), name)
    return q_out


def append_paged(q, k, v, k_pages, v_pages, append_indptr, kv_page_indptr, kv_last_page_len,
                 kv_page_indices, *, rope=None, positions=None, q_out=None, workspace=None, stream=None):
    """fd_append_paged: rotate q [N,Hq,D] and k [N,Hkv,D] and write k, v into the
    bf16 page pools; returns the rotated queries (q_out; None when q is None).

    All tables are int32 CUDA tensors (include/fd.h); they count the new keys in.
    """
    return _append("fd_append_paged", (torch.bfloat16,), 1, q, k, v, k_pages, v_pages, append_indptr,
                   kv_page_indptr, kv_last_page_len, kv_page_indices, rope, positions, q_out, workspace,
                   stream, ())


def append_paged_fp8(q, k, v, k_pages_fp8, v_pages_fp8, k_scale, v_scale, append_indptr, kv_page_indptr,
                     kv_last_page_len, kv_page_indices, *, rope=None, positions=None, q_out=None,
                     workspace=None, stream=None):
    """fd_append_paged_fp8: append_paged into E4M3 pools (uint8 or
    float8_e4m3fn) with the given per-KV-head scales fp32 [Hkv]."""
    f32 = torch.float32
    if k_scale.numel() != k.shape[1] or v_scale.numel() != k.shape[1]:
        raise FdError(-1, "fd_append_paged_fp8: one scale per KV head")
    return _append("fd_append_paged_fp8", (torch.uint8, torch.float8_e4m3fn), 1, q, k, v, k_pages_fp8,
                   v_pages_fp8, append_indptr, kv_page_indptr, kv_last_page_len, kv_page_indices, rope,
                   positions, q_out, workspace, stream,
                   (_need("k_scale", k_scale, f32, k.get_device()), _need("v_scale", v_scale, f32, k.get_device())))


def append_paged_int4(q, k, v, k_pages_int4, v_pages_int4, k_scale, v_scale, append_indptr,
                      kv_page_indptr, kv_last_page_len, kv_page_indices, *, rope=None, positions=None,
                      q_out=None, workspace=None, stream=None):
    """fd_append_paged_int4: append_paged into packed INT4 pools
    [num_pages, page_size, Hkv, D/2]; writes each new row's scale into k_scale,
    v_scale fp32 [Hkv, num_pages * page_size]."""
    f32 = torch.float32
    rows = k_pages_int4.shape[0] * k_pages_int4.shape[1]
    if k_scale.shape != (k.shape[1], rows) or v_scale.shape != (k.shape[1], rows):
        raise FdError(-1, "fd_append_paged_int4: scales must be [Hkv, num_pages * page_size]")
    return _append("fd_append_paged_int4", (torch.uint8,), 0.5, q, k, v, k_pages_int4, v_pages_int4,
                   append_indptr, kv_page_indptr, kv_last_page_len, kv_page_indices, rope, positions, q_out,
                   workspace, stream, (_need("k_scale", k_scale, f32, k.get_device()), _need("v_scale", v_scale, f32, k.get_device())))


def append_paged_int8(q, k, v, k_pages_int8, v_pages_int8, k_scale, v_scale, append_indptr,
                      kv_page_indptr, kv_last_page_len, kv_page_indices, *, rope=None, positions=None,
                      q_out=None, workspace=None, stream=None):
    """fd_append_paged_int8: append_paged into int8 pools
    [num_pages, page_size, Hkv, D], with the scales fp32 [num_pages, scale_heads(Hkv)]
    of the pages that get keys raised where these need it."""
    _, _, ks, vs = _int8_cache("fd_append_paged_int8", k_pages_int8, v_pages_int8, k_scale, v_scale, k.shape[1],
                               k.shape[2], k.get_device())
    return _append("fd_append_paged_int8", (torch.int8,), 1, q, k, v, k_pages_int8, v_pages_int8,
                   append_indptr, kv_page_indptr, kv_last_page_len, kv_page_indices, rope, positions, q_out,
                   workspace, stream, (ks, vs))


def pages_workspace_bytes(num_pages: int, new_batch: int = 0) -> int:
    """fd_pages_workspace_bytes: workspace of fork_pages (new_batch children) or
    compact_pages (new_batch 0)."""
    out = ctypes.c_int64(0)
    _check(lib().fd_pages_workspace_bytes(num_pages, new_batch, ctypes.byref(out)), "fd_pages_workspace_bytes")
    return out.value


def fork_pages(parent, kv_page_indptr, kv_last_page_len, kv_page_indices, new_page_indptr,
               new_page_entries: int, page_size: int, page_refs, *, new_page_indices=None,
               new_page_refs=None, copy_src=None, copy_dst=None, workspace=None, stream=None):
    """fd_fork_pages: the next step's page tables on the device (int32 CUDA
    tensors; new_page_entries = new_page_indptr[-1], known to the host) ->
    (new_page_indices, new_page_refs, copy_src, copy_dst); hand the last two to
    copy_pages."""
    i32, like, dev = torch.int32, page_refs, page_refs.get_device()
    n_new, n_old, pages = parent.numel(), kv_page_indptr.numel() - 1, page_refs.numel()
    if new_page_indptr.numel() != n_new + 1 or kv_last_page_len.numel() < n_old:
        raise FdError(-1, "fd_fork_pages: new_page_indptr must have new_batch+1 and kv_last_page_len batch entries")
    with _on(like, stream):
        at = like.device
        if new_page_indices is None:
            new_page_indices = torch.empty(new_page_entries, dtype=i32, device=at)
        if new_page_refs is None:
            new_page_refs = torch.empty(pages, dtype=i32, device=at)
        if copy_src is None:
            copy_src = torch.empty(n_new, dtype=i32, device=at)
        if copy_dst is None:
            copy_dst = torch.empty(n_new, dtype=i32, device=at)
        if new_page_indices.numel() < new_page_entries or new_page_refs.numel() != pages or \
                copy_src.numel() < n_new or copy_dst.numel() < n_new:
            raise FdError(-1, "fd_fork_pages: an output is too small")
        if workspace is None:
            workspace = torch.zeros(pages_workspace_bytes(pages, n_new), dtype=torch.uint8, device=like.device)
        _check(lib().fd_fork_pages(
            n_old, n_new, page_size, pages, _need("parent", parent, i32, dev),
            _need("kv_page_indptr", kv_page_indptr, i32, dev),
            _need("kv_last_page_len", kv_last_page_len, i32, dev),
            _need("kv_page_indices", kv_page_indices, i32, dev), kv_page_indices.numel(),
            _need("new_page_indptr", new_page_indptr, i32, dev), new_page_entries,
            _need("page_refs", page_refs, i32, dev), _need("new_page_indices", new_page_indices, i32, dev),
            _need("new_page_refs", new_page_refs, i32, dev), _need("copy_src", copy_src, i32, dev),
            _need("copy_dst", copy_dst, i32, dev), *_ws(workspace, dev),
            _stream(stream)), "fd_fork_pages")
    return new_page_indices, new_page_refs, copy_src, copy_dst


def compact_pages(page_refs, kv_page_indices, max_moves: int, *, limit: int = 0, new_page_indices=None,
                  new_page_refs=None, copy_src=None, copy_dst=None, workspace=None, stream=None):
    """fd_compact_pages: rename the pages in use at or behind `limit` (0: the
    number in use) to the lowest free ones -> (new_page_indices, new_page_refs,
    copy_src, copy_dst); hand the last two (max_moves entries) to copy_pages."""
    i32, like, dev = torch.int32, page_refs, page_refs.get_device()
    pages, entries = page_refs.numel(), kv_page_indices.numel()
    with _on(like, stream):
        at = like.device
        if new_page_indices is None:
            new_page_indices = torch.empty(entries, dtype=i32, device=at)
        if new_page_refs is None:
            new_page_refs = torch.empty(pages, dtype=i32, device=at)
        if copy_src is None:
            copy_src = torch.empty(max_moves, dtype=i32, device=at)
        if copy_dst is None:
            copy_dst = torch.empty(max_moves, dtype=i32, device=at)
        if new_page_indices.numel() < entries or new_page_refs.numel() != pages or \
                copy_src.numel() < max_moves or copy_dst.numel() < max_moves:
            raise FdError(-1, "fd_compact_pages: an output is too small")
        if workspace is None:
            workspace = torch.zeros(pages_workspace_bytes(pages), dtype=torch.uint8, device=like.device)
        _check(lib().fd_compact_pages(
            pages, _need("page_refs", page_refs, i32, dev),
            _need("kv_page_indices", kv_page_indices, i32, dev), entries, int(limit), int(max_moves),
            _need("new_page_indices", new_page_indices, i32, dev),
            _need("new_page_refs", new_page_refs, i32, dev), _need("copy_src", copy_src, i32, dev),
            _need("copy_dst", copy_dst, i32, dev), *_ws(workspace, dev),
            _stream(stream)), "fd_compact_pages")
    return new_page_indices, new_page_refs, copy_src, copy_dst


def copy_pages(pools, src, dst, *, workspace=None, stream=None):
    """fd_copy_pages: page src[i] -> dst[i] (int32 CUDA tensors; src < 0: none)
    of every pool in `pools`, contiguous CUDA tensors [num_pages, ...] (K and V
    of all layers, an INT8 cache's scales; an INT4 cache's scales [Hkv, num_pages * page_size] as
    ``*scales.view(Hkv, num_pages, page_size)``)."""
    if not pools or src.numel() == 0:
        return
    pages, n, dev = pools[0].shape[0], len(pools), src.get_device()
    if dst.numel() != src.numel():
        raise FdError(-1, "fd_copy_pages: src and dst must have the same length")
    ptrs, size = (ctypes.c_void_p * n)(), (ctypes.c_int64 * n)()
    for i, x in enumerate(pools):
        if x.get_device() != dev or dev < 0 or x.shape[0] != pages or not x.is_contiguous():
            raise FdError(-1, "fd_copy_pages: pools must be contiguous CUDA tensors of as many pages, on one device")
        ptrs[i], size[i] = x.data_ptr(), x.nbytes // max(pages, 1)
    if pages == 0:
        return
    with _on(src, stream):
        _check(lib().fd_copy_pages(n, ptrs, size, pages, src.numel(), _need("src", src, torch.int32, dev),
                                   _need("dst", dst, torch.int32, dev),
                                   *((None, 0) if workspace is None else _ws(workspace, dev)),
                                   _stream(stream)), "fd_copy_pages")


def _host_ptr(a):
    if a.size and a.flags.writeable:   # (a.ctypes builds an object that holds the array: 0.8 us of a call)
        return ctypes.addressof(ctypes.c_char.from_buffer(a))
    return a.ctypes.data


def plan_shared(batch: int, num_qo_heads: int, num_kv_heads: int, head_dim: int, prefix_req_indptr,
                prefix_indptr, max_suffix_tokens: int, *, num_sms: int = 0, chunk: int = 0,
                timeout_ns: int | None = None) -> SharedPlan:
    """fd_plan_shared: a plan for these prefixes (host int32 [P+1]: requests and
    keys of each) and room for max_suffix_tokens keys of the requests' own."""
    req, ip = _host_indptr(prefix_req_indptr), _host_indptr(prefix_indptr)
    if req.size != ip.size:
        raise FdError(-1, "prefix_req_indptr and prefix_indptr must have num_prefixes+1 entries")
    plan_ = SharedPlan()
    _check(lib().fd_plan_shared(batch, num_qo_heads, num_kv_heads, head_dim, req.size - 1, _host_ptr(req),
                                _host_ptr(ip), int(max_suffix_tokens), num_sms, chunk, ctypes.byref(plan_)),
           "fd_plan_shared")
    if timeout_ns is not None:
        plan_.timeout_ns = timeout_ns
    return plan_


def plan_shared_paged(batch: int, num_qo_heads: int, num_kv_heads: int, head_dim: int, page_size: int,
                      prefix_req_indptr, prefix_page_indptr, prefix_last_page_len, max_suffix_tokens: int, *,
                      num_sms: int = 0, chunk: int = 0, timeout_ns: int | None = None) -> SharedPlan:
    """fd_plan_shared_paged: plan_shared for prefixes in a paged cache (host
    page-list indptr [P+1] and last-page lengths [P])."""
    req, ip = _host_indptr(prefix_req_indptr), _host_indptr(prefix_page_indptr)
    ll = _host_indptr(prefix_last_page_len)
    if req.size != ip.size or ll.size != ip.size - 1:
        raise FdError(-1, "prefix indptrs must have num_prefixes+1 entries, last-page lengths num_prefixes")
    plan_ = SharedPlan()
    _check(lib().fd_plan_shared_paged(batch, num_qo_heads, num_kv_heads, head_dim, page_size, req.size - 1,
                                      _host_ptr(req), _host_ptr(ip), _host_ptr(ll), int(max_suffix_tokens),
                                      num_sms, chunk, ctypes.byref(plan_)), "fd_plan_shared_paged")
    if timeout_ns is not None:
        plan_.timeout_ns = timeout_ns
    return plan_


def _shared_outputs(name, plan_, q, kv, o, lse, workspace):
    """Shapes of a decode_shared call; allocates what was not given."""
    s = plan_.suffix
    shape = (s.batch, s.num_qo_heads, s.head_dim)
    heads = (s.num_kv_heads, s.head_dim)
    if q.shape != shape:
        raise FdError(-1, f"{name}: q is not of the plan's heads")
    for x in kv:
        if x is not None and x.shape[-2:] != heads:
            raise FdError(-1, f"{name}: K/V are not of the plan's heads")
    if o is None:
        o = torch.empty(shape, dtype=torch.float32, device=q.device)
    elif o.shape != shape:
        raise FdError(-1, f"{name}: o of another shape than q")
    if lse is None:
        lse = torch.empty(shape[:2], dtype=torch.float32, device=q.device)
    elif lse.shape != shape[:2]:
        raise FdError(-1, f"{name}: lse must be [batch, num_qo_heads]")
    if workspace is None:
        workspace = torch.zeros(plan_.workspace_bytes, dtype=torch.uint8, device=q.device)
    return o, lse, workspace, s.batch, s.total_tokens


def _maybe(what, t, dtype, dev):
    return None if t is None else _need(what, t, dtype, dev)


def _decode_shared(name, kv_dtypes, plan_, q, k_prefix, v_prefix, k, v, scales, prefix_req_indptr,
                   prefix_indptr, kv_indptr, scale, o, lse, workspace, stream):
    i32, dev = torch.int32, q.get_device()
    with _on(q, stream):
        o, lse, workspace, B, room = _shared_outputs(name, plan_, q, (k_prefix, v_prefix, k, v), o, lse, workspace)
        P = plan_.num_prefixes
        if prefix_req_indptr.numel() != P + 1 or prefix_indptr.numel() != P + 1 or \
                (room and kv_indptr is None) or (kv_indptr is not None and kv_indptr.numel() != B + 1):
            raise FdError(-1, f"{name}: tables of another length than the plan's")
        if plan_.num_items and (k_prefix is None or v_prefix is None or k_prefix.shape[0] < plan_.prefix_rows or
                                v_prefix.shape[0] < plan_.prefix_rows) or \
                (room and (k is None or v is None or k.shape[0] < room or v.shape[0] < room)):
            raise FdError(-1, f"{name}: K/V hold fewer rows than the plan's")
        for x in (k_prefix, v_prefix, k, v):
            if x is not None and x.dtype not in kv_dtypes:
                raise FdError(-1, f"{name}: K/V of another type")
        _check(getattr(lib(), name)(
            ctypes.byref(plan_), _need("prefix_req_indptr", prefix_req_indptr, i32, dev),
            _need("prefix_indptr", prefix_indptr, i32, dev), _maybe("kv_indptr", kv_indptr, i32, dev),
            _need("q", q, torch.bfloat16, dev), *[None if x is None else _need("K/V", x, x.dtype, dev)
                                             for x in (k_prefix, v_prefix, k, v)], *scales, float(scale),
            _need("o", o, torch.float32, dev), _need("lse", lse, torch.float32, dev), *_ws(workspace, dev),
            _stream(stream)), name)
    return o, lse


def decode_shared(plan, q, k_prefix, v_prefix, k, v, prefix_req_indptr, prefix_indptr, kv_indptr,
                  scale: float, *, o=None, lse=None, workspace=None, stream=None):
    """fd_decode_shared: q [B,Hq,D], prefixes' K/V [Tp,Hkv,D] and the requests' own
    K/V [max_suffix_tokens,Hkv,D] (bf16), tables int32 CUDA tensors -> (O, LSE) fp32."""
    return _decode_shared("fd_decode_shared", (torch.bfloat16,), plan, q, k_prefix, v_prefix, k, v, (),
                          prefix_req_indptr, prefix_indptr, kv_indptr, scale, o, lse, workspace, stream)


def _head_scales(k_scale, v_scale, plan_, q):
    Hkv = plan_.suffix.num_kv_heads
    if k_scale.numel() != Hkv or v_scale.numel() != Hkv:
        raise FdError(-1, "k_scale and v_scale must have one entry per KV head")
    dev = q.get_device()
    return _need("k_scale", k_scale, torch.float32, dev), _need("v_scale", v_scale, torch.float32, dev)


def decode_shared_fp8(plan, q, k_prefix_fp8, v_prefix_fp8, k_fp8, v_fp8, k_scale, v_scale,
                      prefix_req_indptr, prefix_indptr, kv_indptr, scale: float, *, o=None, lse=None,
                      workspace=None, stream=None):
    """fd_decode_shared_fp8: decode_shared over E4M3 K/V (uint8 or float8_e4m3fn)
    with per-KV-head scales fp32 [Hkv]."""
    return _decode_shared("fd_decode_shared_fp8", (torch.uint8, torch.float8_e4m3fn), plan, q, k_prefix_fp8,
                          v_prefix_fp8, k_fp8, v_fp8, _head_scales(k_scale, v_scale, plan, q),
                          prefix_req_indptr, prefix_indptr, kv_indptr, scale, o, lse, workspace, stream)


def _decode_shared_paged(name, kv_dtypes, plan_, q, k_pages, v_pages, scales, prefix_req_indptr,
                         prefix_page_indptr, prefix_last_page_len, prefix_page_indices, kv_page_indptr,
                         kv_last_page_len, kv_page_indices, scale, o, lse, workspace, stream):
    i32, dev = torch.int32, q.get_device()
    with _on(q, stream):
        o, lse, workspace, B, room = _shared_outputs(name, plan_, q, (k_pages, v_pages), o, lse, workspace)
        P = plan_.num_prefixes
        if prefix_req_indptr.numel() != P + 1 or prefix_page_indptr.numel() != P + 1 or \
                prefix_last_page_len.numel() < P or prefix_page_indices.numel() < plan_.prefix_rows or \
                (room and (kv_page_indptr is None or kv_last_page_len is None)) or \
                (kv_page_indptr is not None and kv_page_indptr.numel() != B + 1) or \
                (kv_last_page_len is not None and kv_last_page_len.numel() < B):
            raise FdError(-1, f"{name}: tables of another length than the plan's")
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or k_pages.shape[1] != plan_.page_size or \
                k_pages.dtype not in kv_dtypes or v_pages.dtype not in kv_dtypes:
            raise FdError(-1, f"{name}: pools of another shape or type")
        _check(getattr(lib(), name)(
            ctypes.byref(plan_), k_pages.shape[0], _need("prefix_req_indptr", prefix_req_indptr, i32, dev),
            _need("prefix_page_indptr", prefix_page_indptr, i32, dev),
            _need("prefix_last_page_len", prefix_last_page_len, i32, dev),
            _need("prefix_page_indices", prefix_page_indices, i32, dev),
            _maybe("kv_page_indptr", kv_page_indptr, i32, dev), _maybe("kv_last_page_len", kv_last_page_len, i32, dev),
            _maybe("kv_page_indices", kv_page_indices, i32, dev),
            0 if kv_page_indices is None else kv_page_indices.numel(), _need("q", q, torch.bfloat16, dev),
            _need("k_pages", k_pages, k_pages.dtype, dev), _need("v_pages", v_pages, v_pages.dtype, dev), *scales,
            float(scale), _need("o", o, torch.float32, dev), _need("lse", lse, torch.float32, dev),
            *_ws(workspace, dev), _stream(stream)), name)
    return o, lse


def decode_shared_paged(plan, q, k_pages, v_pages, prefix_req_indptr, prefix_page_indptr,
                        prefix_last_page_len, prefix_page_indices, kv_page_indptr, kv_last_page_len,
                        kv_page_indices, scale: float, *, o=None, lse=None, workspace=None, stream=None):
    """fd_decode_shared_paged: prefixes and the requests' own keys in the same
    bf16 page pools; tables int32 CUDA tensors (include/fd.h) -> (O, LSE) fp32."""
    return _decode_shared_paged("fd_decode_shared_paged", (torch.bfloat16,), plan, q, k_pages, v_pages, (),
                                prefix_req_indptr, prefix_page_indptr, prefix_last_page_len,
                                prefix_page_indices, kv_page_indptr, kv_last_page_len, kv_page_indices,
                                scale, o, lse, workspace, stream)


def decode_shared_paged_fp8(plan, q, k_pages_fp8, v_pages_fp8, k_scale, v_scale, prefix_req_indptr,
                            prefix_page_indptr, prefix_last_page_len, prefix_page_indices,
                            kv_page_indptr, kv_last_page_len, kv_page_indices, scale: float, *, o=None,
                            lse=None, workspace=None, stream=None):
    """fd_decode_shared_paged_fp8: decode_shared_paged over E4M3 page pools with
    per-KV-head scales fp32 [Hkv]."""
    return _decode_shared_paged("fd_decode_shared_paged_fp8", (torch.uint8, torch.float8_e4m3fn), plan, q,
                                k_pages_fp8, v_pages_fp8, _head_scales(k_scale, v_scale, plan, q),
                                prefix_req_indptr, prefix_page_indptr, prefix_last_page_len,
                                prefix_page_indices, kv_page_indptr, kv_last_page_len, kv_page_indices,
                                scale, o, lse, workspace, stream)


def plan_prefill_paged(batch: int, num_qo_heads: int, num_kv_heads: int, head_dim: int, page_size: int, q_indptr,
                       kv_page_indptr, kv_last_page_len, *, causal: bool = True, num_sms: int = 0, chunk: int = 0,
                       timeout_ns: int | None = None) -> PrefillPlan:
    """fd_plan_prefill_paged: a plan for these query tokens and page tables (host
    int32: q_indptr [B+1], kv_page_indptr [B+1], kv_last_page_len [B])."""
    qi, ip, ll = _host_indptr(q_indptr), _host_indptr(kv_page_indptr), _host_indptr(kv_last_page_len)
    if qi.size != batch + 1 or ip.size != batch + 1 or ll.size != batch:
        raise FdError(-1, "indptrs must have batch+1 entries, last-page lengths batch")
    plan_ = PrefillPlan()
    _check(lib().fd_plan_prefill_paged(batch, num_qo_heads, num_kv_heads, head_dim, page_size, _host_ptr(qi),
                                       _host_ptr(ip), _host_ptr(ll), int(bool(causal)), num_sms, chunk,
                                       ctypes.byref(plan_)), "fd_plan_prefill_paged")
    if timeout_ns is not None:
        plan_.timeout_ns = timeout_ns
    return plan_


def prefill_paged_int8(plan, q, k_pages_int8, v_pages_int8, k_scale, v_scale, q_indptr, kv_page_indptr,
                       kv_last_page_len, kv_page_indices, scale: float, *, o=None, lse=None, workspace=None,
                       stream=None):
    """fd_prefill_paged_int8: q [N,Hq,D] bf16 (any token stride, N at least the plan's
    tokens) over an INT8 cache -> (O bf16 [N,Hq,D], LSE fp32 [N,Hq]); tables int32 CUDA
    tensors."""
    name, i32, f32, dev = "fd_prefill_paged_int8", torch.int32, torch.float32, q.get_device()
    B, Hkv, D = plan.batch, plan.num_kv_heads, plan.head_dim
    if q.dim() != 3 or q.shape[0] < plan.num_tokens or q.shape[1:] != (plan.num_qo_heads, D):
        raise FdError(-1, f"{name}: q is not of the plan's tokens and heads")
    if q_indptr.numel() != B + 1 or kv_page_indptr.numel() != B + 1 or kv_last_page_len.numel() < B or \
            kv_page_indices.numel() < plan.num_page_entries:
        raise FdError(-1, f"{name}: tables of another length than the plan's")
    if k_pages_int8.dim() != 4 or k_pages_int8.shape[1] != plan.page_size:
        raise FdError(-1, f"{name}: pools of another shape")
    with _on(q, stream):
        if o is None:
            o = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        if lse is None:
            lse = torch.empty(q.shape[:2], dtype=f32, device=q.device)
        if o.shape != q.shape or lse.shape != q.shape[:2]:
            raise FdError(-1, f"{name}: o must have q's shape and lse [tokens, num_qo_heads]")
        if workspace is None:
            workspace = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=q.device)
        kp, vp, ks, vs = _int8_cache(name, k_pages_int8, v_pages_int8, k_scale, v_scale, Hkv, D, dev)
        _check(lib().fd_prefill_paged_int8(
            ctypes.byref(plan), k_pages_int8.shape[0], _need("q_indptr", q_indptr, i32, dev),
            _need("kv_page_indptr", kv_page_indptr, i32, dev), _need("kv_last_page_len", kv_last_page_len, i32, dev),
            _need("kv_page_indices", kv_page_indices, i32, dev), _ptr(q), _heads("q", q, dev), kp, vp, ks, vs,
            float(scale), _need("o", o, torch.bfloat16, dev), _need("lse", lse, f32, dev), *_ws(workspace, dev),
            _stream(stream)), name)
    return o, lse


def get_device_status(workspace, stream=None) -> int:
    """fd_get_device_status: synchronise, read and clear the kernels' status word."""
    return lib().fd_get_device_status(_ptr(workspace), _stream(stream))


__all__ = [
    "PlanInfo", "FdError", "lib", "build", "plan", "plan_work_items", "decode_split", "merge",
    "decode", "decode_static_workspace", "plan_paged", "decode_paged", "decode_fp8",
    "decode_paged_fp8", "decode_int4", "decode_paged_int4", "decode_paged_int8", "scale_heads",
    "plan_graph", "decode_graph", "merge_states", "get_device_status",
    "SharedPlan", "plan_shared", "plan_shared_paged", "decode_shared", "decode_shared_paged",
    "decode_shared_fp8", "decode_shared_paged_fp8",
    "PrefillPlan", "plan_prefill_paged", "prefill_paged_int8",
    "RopeInfo", "plan_rope", "append_paged", "append_paged_fp8", "append_paged_int4", "append_paged_int8",
    "pages_workspace_bytes", "fork_pages", "compact_pages", "copy_pages", "workspace_bytes", "num_sms",
    "status_string",
    "TILE_TOKENS", "WORKSPACE_HEADER_BYTES", "DEFAULT_TIMEOUT_NS",
]
