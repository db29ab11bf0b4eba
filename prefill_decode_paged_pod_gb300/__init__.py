"""GB300 (sm_103a) POD paged attention: Python binding of the C ABI in include/pod.h.

This module only marshals arguments: host page tables as int32 numpy arrays,
device tensors as raw pointers, the current torch CUDA stream as a handle.
Every step of the computation runs in the library's CUDA kernels; there is no
CPU or PyTorch fallback. If the shared library is missing or cannot be loaded
the import of the binding raises.

    h = pod_plan(p_q_indptr, p_kv_indptr, p_kv_indices, p_last_page_len,
                 d_q_indptr, d_kv_indptr, d_kv_indices, d_last_page_len,
                 num_qo_heads, num_kv_heads, head_dim, page_size,
                 causal, window_left, sm_scale, dtype=torch.bfloat16,
                 p_num_pages=..., d_num_pages=..., has_sinks=False, workspace=ws)
    out_p, lse_p, out_d, lse_d = pod_run(h, q_p, kv_p, q_d, kv_d, ws, sinks=None)

The names and the plan-once / run-many life cycle follow the POD walkthrough
("plan/run 生命周期", "BatchPOD 的 run 差异").
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import Optional

import numpy as np

__all__ = [
    "POD_OK", "PodError", "load_library", "pod_plan", "pod_run", "pod_destroy",
    "pod_workspace_size", "pod_bind_workspace", "pod_last_error", "pod_read_device_status",
    "pod_plan_table", "PodHandle", "LIB_PATH", "DEFAULT_WORKSPACE_BYTES",
    "pod_run_static_scratch", "pod_static_scratch_capacity", "pod_plan_set_decode_fp8",
    "pod_plan_set_prefill_mask", "pod_plan_set_kv_layout", "pod_plan_set_logits_transform",
    "pod_plan_set_rope", "pod_plan_set_graph_capacity", "pod_replan",
    "pod_qk_norm_rope", "pod_append_kv", "pod_norm_rope_append", "pod_gather_kv", "pod_kv_slots",
    "PodTreeHandle", "pod_tree_plan", "pod_tree_run", "pod_tree_workspace_size", "pod_tree_bind_workspace",
    "pod_tree_read_device_status", "pod_tree_plan_table", "pod_tree_destroy",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libpod_gb300.so")
POD_OK = 0
_STATUS = {0: "POD_OK", 1: "POD_ERR_INVALID_ARG", 2: "POD_ERR_UNSUPPORTED", 3: "POD_ERR_WORKSPACE",
           4: "POD_ERR_CUDA", 5: "POD_ERR_DEVICE_STATUS"}
# the pages recommend a 128 MB workspace for typical POD use
DEFAULT_WORKSPACE_BYTES = 128 * 1024 * 1024

_lib = None


class PodError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{_STATUS.get(code, code)}: {msg}")
        self.code = code


def load_library(path: Optional[str] = None):
    """Load the C-ABI library (built by ``__graft_entry__.build()``). Raises if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"POD CUDA library not built: {p} is missing "
                           "(run __graft_entry__.build() or prefill_decode_paged_pod_gb300/_build.py)")
    lib = ctypes.CDLL(p)
    V, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lib.pod_plan.restype = ctypes.c_int
    lib.pod_plan.argtypes = [V, V, V, V, I32, I32, V, V, V, V, I32, I32,
                             I32, I32, I32, I32, I32, I32, ctypes.c_float, ctypes.c_int, I32, I32,
                             V, SZ, V, ctypes.POINTER(V), ctypes.POINTER(SZ)]
    lib.pod_workspace_size.restype = SZ
    lib.pod_workspace_size.argtypes = [V]
    lib.pod_bind_workspace.restype = ctypes.c_int
    lib.pod_bind_workspace.argtypes = [V, V, SZ, V]
    lib.pod_run.restype = ctypes.c_int
    lib.pod_run.argtypes = [V, V, V, V, V, V, V, V, V, V, V, V]
    lib.pod_destroy.restype = ctypes.c_int
    lib.pod_destroy.argtypes = [V]
    lib.pod_last_error.restype = ctypes.c_char_p
    lib.pod_last_error.argtypes = []
    lib.pod_read_device_status.restype = ctypes.c_int
    lib.pod_read_device_status.argtypes = [V, V, V, ctypes.POINTER(I32)]
    lib.pod_plan_table.restype = ctypes.c_int
    lib.pod_plan_table.argtypes = [V, I32, V, ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)]
    lib.pod_run_static_scratch.restype = ctypes.c_int
    lib.pod_run_static_scratch.argtypes = [V, V, V, V, V, V, V, V, V, V, V]
    lib.pod_static_scratch_capacity.restype = SZ
    lib.pod_static_scratch_capacity.argtypes = []
    lib.pod_plan_set_decode_fp8.restype = ctypes.c_int
    lib.pod_plan_set_decode_fp8.argtypes = [V, ctypes.c_float, ctypes.c_float]
    lib.pod_plan_set_rope.restype = ctypes.c_int
    lib.pod_plan_set_rope.argtypes = [V, ctypes.c_float, ctypes.c_float]
    lib.pod_plan_set_logits_transform.restype = ctypes.c_int
    lib.pod_plan_set_logits_transform.argtypes = [V, ctypes.c_float, V]
    lib.pod_plan_set_kv_layout.restype = ctypes.c_int
    lib.pod_plan_set_kv_layout.argtypes = [V, I32, I32]
    lib.pod_plan_set_prefill_mask.restype = ctypes.c_int
    lib.pod_plan_set_prefill_mask.argtypes = [V, V, ctypes.c_int64]
    lib.pod_plan_set_graph_capacity.restype = ctypes.c_int
    lib.pod_plan_set_graph_capacity.argtypes = [V] + [I32] * 6
    lib.pod_replan.restype = ctypes.c_int
    lib.pod_replan.argtypes = [V, V, V, V, V, I32, V, V, V, V, I32, V]
    I64, F32 = ctypes.c_int64, ctypes.c_float
    for fn in (lib.pod_qk_norm_rope, lib.pod_append_kv, lib.pod_norm_rope_append, lib.pod_gather_kv):
        fn.restype = ctypes.c_int
        fn.argtypes = [ctypes.c_char_p, V]
    lib.pod_tree_plan.restype = ctypes.c_int
    lib.pod_tree_plan.argtypes = [V, V, V, V, I32, I32, I32, I32, I32, I32, F32, ctypes.c_int, I32, F32, F32,
                                  I32, I32, I32, V, SZ, V, ctypes.POINTER(V), ctypes.POINTER(SZ)]
    lib.pod_tree_workspace_size.restype = SZ
    lib.pod_tree_workspace_size.argtypes = [V]
    lib.pod_tree_bind_workspace.restype = ctypes.c_int
    lib.pod_tree_bind_workspace.argtypes = [V, V, SZ, V]
    lib.pod_tree_run.restype = ctypes.c_int
    lib.pod_tree_run.argtypes = [V, V, V, V, V, I64, V, V, V, V, V]
    lib.pod_tree_read_device_status.restype = ctypes.c_int
    lib.pod_tree_read_device_status.argtypes = [V, V, V, ctypes.POINTER(I32)]
    lib.pod_tree_plan_table.restype = ctypes.c_int
    lib.pod_tree_plan_table.argtypes = [V, I32, V, I64, ctypes.POINTER(I64)]
    lib.pod_tree_destroy.restype = ctypes.c_int
    lib.pod_tree_destroy.argtypes = [V]
    if path is None:
        _lib = lib
    return lib


def pod_last_error() -> str:
    return load_library().pod_last_error().decode()


def _check(code: int):
    if code != POD_OK:
        raise PodError(code, pod_last_error())


def _i32(a) -> Optional[np.ndarray]:
    if a is None:
        return None
    if hasattr(a, "detach"):
        a = a.detach().cpu().numpy()
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _ptr(a) -> Optional[int]:
    if a is None:
        return None
    if isinstance(a, np.ndarray):
        return a.ctypes.data
    return a.data_ptr()


def _stream(stream=None) -> Optional[int]:
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    if not torch.cuda.is_available():
        return None
    return torch.cuda.current_stream().cuda_stream


def _dtype_code(dtype) -> int:
    import torch
    if dtype in (torch.float16, "float16", "fp16", 0):
        return 0
    if dtype in (torch.bfloat16, "bfloat16", "bf16", 1):
        return 1
    raise PodError(2, f"unsupported dtype {dtype}")


@dataclass
class PodHandle:
    """Owns a plan handle of the C library (released by ``pod_destroy``)."""
    ptr: int
    workspace_bytes: int
    p_rows: int
    d_rows: int
    num_qo_heads: int
    head_dim: int
    dtype: object
    has_sinks: bool
    workspace_ptr: Optional[int] = None
    d_kv_fp8: bool = False      # set by pod_plan_set_decode_fp8
    p_mask: object = None       # custom prefill mask, kept alive while the plan uses it
    alibi: object = None        # ALiBi slopes, kept alive while the plan uses them

    def __del__(self):
        if self.ptr and _lib is not None:
            _lib.pod_destroy(ctypes.c_void_p(self.ptr))
            self.ptr = 0


def pod_plan(p_q_indptr, p_kv_indptr, p_kv_indices, p_last_page_len,
             d_q_indptr, d_kv_indptr, d_kv_indices, d_last_page_len,
             num_qo_heads, num_kv_heads, head_dim, page_size,
             causal=True, window_left=-1, sm_scale=None, *, dtype, p_num_pages, d_num_pages,
             has_sinks=False, num_sms=0, workspace=None, stream=None) -> PodHandle:
    """Plan a POD launch. Index arrays are host int32 (numpy or CPU tensors).

    ``workspace`` is a device uint8 tensor (or None for a host-only plan that
    can be bound later with ``pod_bind_workspace``).
    """
    lib = load_library()
    arrs = [_i32(x) for x in (p_q_indptr, p_kv_indptr, p_kv_indices, p_last_page_len,
                              d_q_indptr, d_kv_indptr, d_kv_indices, d_last_page_len)]
    p_batch = 0 if arrs[0] is None else len(arrs[0]) - 1
    d_batch = 0 if arrs[4] is None else len(arrs[4]) - 1
    handle = ctypes.c_void_p()
    req = ctypes.c_size_t(0)
    ws_ptr = None if workspace is None else workspace.data_ptr()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    code = lib.pod_plan(*[_ptr(a) for a in arrs[:4]], p_batch, int(p_num_pages),
                        *[_ptr(a) for a in arrs[4:]], d_batch, int(d_num_pages),
                        int(num_qo_heads), int(num_kv_heads), int(head_dim), int(page_size),
                        int(bool(causal)), int(window_left),
                        float(sm_scale) if sm_scale is not None else 0.0,
                        _dtype_code(dtype), int(bool(has_sinks)), int(num_sms),
                        ws_ptr, ws_bytes, _stream(stream) if ws_ptr else None,
                        ctypes.byref(handle), ctypes.byref(req))
    if code != POD_OK:
        err = PodError(code, pod_last_error())
        err.required_workspace_bytes = int(req.value)
        raise err
    p_rows = 0 if arrs[0] is None or p_batch == 0 else int(arrs[0][-1])
    d_rows = 0 if arrs[4] is None or d_batch == 0 else int(arrs[4][-1])
    return PodHandle(ptr=handle.value, workspace_bytes=int(req.value), p_rows=p_rows,
                     d_rows=d_rows, num_qo_heads=int(num_qo_heads), head_dim=int(head_dim),
                     dtype=dtype, has_sinks=bool(has_sinks), workspace_ptr=ws_ptr)


def pod_workspace_size(h: PodHandle) -> int:
    return int(load_library().pod_workspace_size(ctypes.c_void_p(h.ptr)))


def pod_bind_workspace(h: PodHandle, workspace, stream=None):
    lib = load_library()
    _check(lib.pod_bind_workspace(ctypes.c_void_p(h.ptr), workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(), _stream(stream)))
    h.workspace_ptr = workspace.data_ptr()


def pod_run(h: PodHandle, q_p, kv_p, q_d, kv_d, workspace, sinks=None,
            out_p=None, lse_p=None, out_d=None, lse_d=None, stream=None):
    """One fused POD launch. Returns (out_p, lse_p, out_d, lse_d); outputs are
    allocated with torch on the inputs' device when not given."""
    import torch
    lib = load_library()
    H, d = h.num_qo_heads, h.head_dim
    dev = None
    for t in (q_p, q_d, workspace):
        if t is not None:
            dev = t.device
            break
    if out_p is None:
        out_p = torch.empty((h.p_rows, H, d), dtype=h.dtype, device=dev)
    if lse_p is None:
        lse_p = torch.empty((h.p_rows, H), dtype=torch.float32, device=dev)
    if out_d is None:
        out_d = torch.empty((h.d_rows, H, d), dtype=h.dtype, device=dev)
    if lse_d is None:
        lse_d = torch.empty((h.d_rows, H), dtype=torch.float32, device=dev)
    for name, t in (("q_p", q_p), ("kv_p", kv_p), ("q_d", q_d), ("kv_d", kv_d)):
        want = torch.float8_e4m3fn if (name == "kv_d" and h.d_kv_fp8) else h.dtype
        if t is not None and (not t.is_contiguous() or t.dtype != want):
            raise PodError(1, f"{name} must be contiguous {want}")
    _check_mask_device(h)
    p_empty, d_empty = h.p_rows == 0, h.d_rows == 0
    code = lib.pod_run(ctypes.c_void_p(h.ptr),
                       None if p_empty else _ptr(q_p), None if p_empty else _ptr(kv_p),
                       None if d_empty else _ptr(q_d), None if d_empty else _ptr(kv_d),
                       _ptr(sinks), _ptr(workspace),
                       None if p_empty else _ptr(out_p), None if p_empty else _ptr(lse_p),
                       None if d_empty else _ptr(out_d), None if d_empty else _ptr(lse_d),
                       _stream(stream))
    _check(code)
    return out_p, lse_p, out_d, lse_d


def pod_static_scratch_capacity() -> int:
    return int(load_library().pod_static_scratch_capacity())


def pod_run_static_scratch(h: PodHandle, q_p, kv_p, q_d, kv_d, sinks=None,
                           out_p=None, lse_p=None, out_d=None, lse_d=None, stream=None):
    """Like pod_run, but the kernels' scratch is the library's fixed device
    array instead of a caller-allocated workspace (for callers that cannot
    allocate device memory). Output tensors are allocated here when not given;
    pass them to keep the call free of allocations. Calls sharing a device must
    not overlap on the GPU."""
    import torch
    lib = load_library()
    H, d = h.num_qo_heads, h.head_dim
    dev = q_p.device if q_p is not None else (q_d.device if q_d is not None else None)
    if out_p is None:
        out_p = torch.empty((h.p_rows, H, d), dtype=h.dtype, device=dev)
    if lse_p is None:
        lse_p = torch.empty((h.p_rows, H), dtype=torch.float32, device=dev)
    if out_d is None:
        out_d = torch.empty((h.d_rows, H, d), dtype=h.dtype, device=dev)
    if lse_d is None:
        lse_d = torch.empty((h.d_rows, H), dtype=torch.float32, device=dev)
    _check_mask_device(h)
    p_empty, d_empty = h.p_rows == 0, h.d_rows == 0
    code = lib.pod_run_static_scratch(
        ctypes.c_void_p(h.ptr),
        None if p_empty else _ptr(q_p), None if p_empty else _ptr(kv_p),
        None if d_empty else _ptr(q_d), None if d_empty else _ptr(kv_d), _ptr(sinks),
        None if p_empty else _ptr(out_p), None if p_empty else _ptr(lse_p),
        None if d_empty else _ptr(out_d), None if d_empty else _ptr(lse_d), _stream(stream))
    _check(code)
    return out_p, lse_p, out_d, lse_d


def pod_destroy(h: PodHandle):
    if h.ptr:
        load_library().pod_destroy(ctypes.c_void_p(h.ptr))
        h.ptr = 0


def pod_read_device_status(h: PodHandle, workspace, stream=None) -> int:
    v = ctypes.c_int32(0)
    code = load_library().pod_read_device_status(ctypes.c_void_p(h.ptr), workspace.data_ptr(),
                                                 _stream(stream), ctypes.byref(v))
    if code not in (POD_OK, 5):
        _check(code)
    return int(v.value)


def pod_plan_table(h: PodHandle, which: int) -> np.ndarray:
    lib = load_library()
    n = ctypes.c_int64(0)
    _check(lib.pod_plan_table(ctypes.c_void_p(h.ptr), int(which), None, 0, ctypes.byref(n)))
    out = np.zeros(max(n.value, 1), dtype=np.int32)
    _check(lib.pod_plan_table(ctypes.c_void_p(h.ptr), int(which), out.ctypes.data, n.value,
                              ctypes.byref(n)))
    return out[:n.value]


# summary indices of pod_plan_table(h, 0), mirroring enum PodSummary in csrc/pod_plan.h
SUMMARY_FIELDS = ("H", "Hk", "d", "ps", "causal", "window", "dtype", "sinks", "num_sms", "grid",
                  "n_p_ctas", "n_d_ctas", "n_tiles", "n_items", "n_groups", "n_mrows", "n_prows",
                  "p_rows", "d_rows", "p_batch", "d_batch", "decode_chunk", "ws_lo", "ws_hi",
                  "p_tma", "d_tma", "p_mask", "rope")


def plan_summary(h: PodHandle) -> dict:
    s = pod_plan_table(h, 0)
    return {k: int(v) for k, v in zip(SUMMARY_FIELDS, s)}


def pod_plan_set_decode_fp8(h: PodHandle, k_scale: float, v_scale: float):
    """The decode cache is FP8 E4M3 codes; K = code * k_scale, V = code * v_scale."""
    _check(load_library().pod_plan_set_decode_fp8(ctypes.c_void_p(h.ptr), float(k_scale),
                                                  float(v_scale)))
    h.d_kv_fp8 = True


def pod_plan_set_prefill_mask(h: PodHandle, packed_mask):
    """Custom prefill mask: uint8 bits (little bit order) of every prefill
    request's [q_len, kv_len] matrix, end to end; None removes it. A CUDA
    tensor for runs; a CPU tensor or numpy array serves host-only plans
    (inspection), whose pointer the library never reads. Switching the mask
    on or off re-plans the handle and releases its workspace: bind again."""
    lib = load_library()
    if packed_mask is None:
        _check(lib.pod_plan_set_prefill_mask(ctypes.c_void_p(h.ptr), None, 0))
        h.p_mask = None
    else:
        if isinstance(packed_mask, np.ndarray):
            packed_mask = np.ascontiguousarray(packed_mask, dtype=np.uint8)
            ptr, nbytes = packed_mask.ctypes.data, packed_mask.nbytes
        else:
            import torch
            if packed_mask.dtype != torch.uint8 or not packed_mask.is_contiguous():
                raise PodError(1, "packed_mask must be a contiguous uint8 tensor")
            ptr, nbytes = packed_mask.data_ptr(), packed_mask.numel()
        _check(lib.pod_plan_set_prefill_mask(ctypes.c_void_p(h.ptr), ptr, int(nbytes)))
        h.p_mask = packed_mask
    h.workspace_bytes = pod_workspace_size(h)
    h.workspace_ptr = None


def pod_plan_set_logits_transform(h: PodHandle, soft_cap: float = 0.0, alibi_slopes=None):
    """Logits soft cap (cap * tanh(x / cap) of the scaled logit; 0 = off) or
    ALiBi slopes (fp32 [H]; a CUDA tensor for runs, any tensor for host-only
    plans), applied by both halves."""
    ptr = None
    if alibi_slopes is not None:
        import torch
        if alibi_slopes.dtype != torch.float32 or not alibi_slopes.is_contiguous() \
                or alibi_slopes.numel() != h.num_qo_heads:
            raise PodError(1, "alibi_slopes must be a contiguous float32 tensor of num_qo_heads")
        ptr = alibi_slopes.data_ptr()
    _check(load_library().pod_plan_set_logits_transform(ctypes.c_void_p(h.ptr), float(soft_cap),
                                                        ptr))
    h.alibi = alibi_slopes


def pod_plan_set_rope(h: PodHandle, rope_scale: float = 1.0, rope_theta: float = 1e4):
    """ROPE_LLAMA on both halves (rope_scale 0 turns it off). Plans the handle
    again and releases its workspace: bind again."""
    _check(load_library().pod_plan_set_rope(ctypes.c_void_p(h.ptr), float(rope_scale),
                                            float(rope_theta)))
    h.workspace_bytes = pod_workspace_size(h)
    h.workspace_ptr = None


_LAYOUTS = {"NHD": 0, "HND": 1, 0: 0, 1: 1}


def pod_plan_set_kv_layout(h: PodHandle, p_layout="NHD", d_layout="NHD"):
    """Page layout of each half's cache: "NHD" [pages, 2, ps, Hk, d] or
    "HND" [pages, 2, Hk, ps, d]."""
    if p_layout not in _LAYOUTS or d_layout not in _LAYOUTS:
        raise PodError(1, f"unknown kv layout {p_layout!r} / {d_layout!r}")
    _check(load_library().pod_plan_set_kv_layout(ctypes.c_void_p(h.ptr), _LAYOUTS[p_layout],
                                                 _LAYOUTS[d_layout]))


def _check_mask_device(h: PodHandle):
    m = h.p_mask
    if m is not None and h.p_rows and not getattr(m, "is_cuda", False):
        raise PodError(1, "the custom prefill mask must be a CUDA uint8 tensor to run")
    if h.alibi is not None and not getattr(h.alibi, "is_cuda", False):
        raise PodError(1, "the ALiBi slopes must be a CUDA float32 tensor to run")


def plan_inputs(inp, workspace=None, num_sms=0, stream=None) -> PodHandle:
    """pod_plan for a ``pod_workloads.PODInputs``-shaped object (tests, bench);
    an FP8 (float8_e4m3fn) decode cache gets pod_plan_set_decode_fp8 with the
    inputs' scales, a packed custom mask on the prefill half
    pod_plan_set_prefill_mask (moved to the GPU when there is one)."""
    mask = getattr(inp.p, "packed_mask", None)
    rope = getattr(inp, "rope", None)
    replans = mask is not None or rope is not None
    h = _plan_inputs(inp, None if replans else workspace, num_sms, stream)
    if rope is not None:
        pod_plan_set_rope(h, *rope)
    import torch
    if inp.d.rows and getattr(inp.d.kv, "dtype", None) == torch.float8_e4m3fn:
        pod_plan_set_decode_fp8(h, inp.k_scale, inp.v_scale)
    cap, slopes = float(getattr(inp, "soft_cap", 0.0) or 0.0), getattr(inp, "alibi", None)
    if cap > 0 or slopes is not None:
        if slopes is not None and torch.cuda.is_available():
            slopes = slopes.to(device="cuda", dtype=torch.float32).contiguous()
        pod_plan_set_logits_transform(h, cap, slopes)
    lp, ld = getattr(inp.p, "kv_layout", "NHD"), getattr(inp.d, "kv_layout", "NHD")
    if (lp, ld) != ("NHD", "NHD"):
        pod_plan_set_kv_layout(h, lp, ld)
    if mask is not None:
        t = torch.from_numpy(np.ascontiguousarray(mask, dtype=np.uint8))
        if torch.cuda.is_available():
            t = t.cuda()
        pod_plan_set_prefill_mask(h, t)
    if replans and workspace is not None:
        pod_bind_workspace(h, workspace, stream)
    return h


def _plan_inputs(inp, workspace, num_sms, stream) -> PodHandle:
    return pod_plan(inp.p.q_indptr, inp.p.kv_indptr, inp.p.kv_indices, inp.p.last_page_len,
                    inp.d.q_indptr, inp.d.kv_indptr, inp.d.kv_indices, inp.d.last_page_len,
                    inp.num_qo_heads, inp.num_kv_heads, inp.head_dim, inp.page_size,
                    inp.causal, inp.window_left, inp.sm_scale, dtype=inp.dtype,
                    p_num_pages=inp.p.num_pages, d_num_pages=inp.d.num_pages,
                    has_sinks=inp.sinks is not None, num_sms=num_sms, workspace=workspace,
                    stream=stream)


def pod_plan_set_graph_capacity(h: PodHandle, max_p_batch: int, max_p_rows: int, max_p_pages: int,
                                max_d_batch: int, max_d_rows: int, max_d_pages: int):
    """Capacity mode for CUDA-graph replay: the workspace layout and launch
    shapes depend on these maxima only; rebind the workspace afterwards. The
    q/out tensors given to pod_run then hold max_*_rows rows."""
    _check(load_library().pod_plan_set_graph_capacity(
        ctypes.c_void_p(h.ptr), int(max_p_batch), int(max_p_rows), int(max_p_pages),
        int(max_d_batch), int(max_d_rows), int(max_d_pages)))
    h.workspace_bytes = pod_workspace_size(h)
    h.p_rows, h.d_rows = int(max_p_rows), int(max_d_rows)


def pod_replan(h: PodHandle, p_q_indptr, p_kv_indptr, p_kv_indices, p_last_page_len,
               d_q_indptr, d_kv_indptr, d_kv_indices, d_last_page_len, stream=None):
    """Plan new page tables into a capacity handle's bound workspace (outside
    any capture); a pod_run captured earlier then replays the new plan."""
    arrs = [_i32(x) for x in (p_q_indptr, p_kv_indptr, p_kv_indices, p_last_page_len,
                              d_q_indptr, d_kv_indptr, d_kv_indices, d_last_page_len)]
    p_batch = 0 if arrs[0] is None else len(arrs[0]) - 1
    d_batch = 0 if arrs[4] is None else len(arrs[4]) - 1
    _check(load_library().pod_replan(ctypes.c_void_p(h.ptr), *[_ptr(a) for a in arrs[:4]], p_batch,
                                     *[_ptr(a) for a in arrs[4:]], d_batch, _stream(stream)))


# ------------------------------------------------------------------ operators around the cache
def pod_kv_slots(kv_indptr, kv_indices, page_size: int, request, position):
    """Slots of key ``position[i]`` of request ``request[i]`` (int64, the
    ``slots`` of pod_append_kv and the others): numpy arrays or tensors of one
    device in, the same kind out. A position outside the request's pages (so any
    negative one), and a request that is not in the table, give -1, the slot of a
    padding row; nothing outside the table is read."""
    if hasattr(kv_indptr, "data_ptr"):
        xp = _torch()
        ask = lambda x: xp.as_tensor(x, device=kv_indptr.device).long()   # noqa: E731
    else:
        xp = np
        ask = lambda x: np.asarray(x).astype(np.int64)                    # noqa: E731
    indptr, indices, request, position = ask(kv_indptr), ask(kv_indices), ask(request), ask(position)
    batch, pages = indptr.shape[0] - 1, indices.shape[0]
    if batch < 1 or pages < 1:
        return xp.full_like(request + position, -1)
    known = (request >= 0) & (request < batch)
    request = xp.where(known, request, 0)
    at = indptr[request] + position // page_size
    inside = known & (position >= 0) & (at < indptr[request + 1]) & (at < pages)
    slots = indices[xp.where(inside, at, 0)] * page_size + position % page_size
    return xp.where(inside, slots, -1)


_KV_FORMATS = {"16bit": 0, "scaled": 1, "block": 2}
_torch_module = None


def _torch():
    """torch, imported on first use, with what the calls below ask of it every
    time: the current device and its current stream (small calls take as long as
    their host side)."""
    global _torch_module, _raw_stream, _current_device
    if _torch_module is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda index: torch.cuda.current_stream(index).cuda_stream)
        _current_device = torch.cuda.current_device
        _torch_module = torch
    return _torch_module


def _device_of(t):
    """Index of a CUDA tensor's device."""
    if t is None or not t.is_cuda:
        raise PodError(1, "the tensors must be CUDA tensors")
    return t.get_device()


def _heads(name, t, dtype, dev, rows=None):
    """[rows, heads, d] with contiguous heads; returns (rows, heads, d, row stride)."""
    try:
        n, h, d = t.shape
        sn, sh, sd = t.stride()
    except ValueError:
        n = -1
    if n < 0 or t.dtype != dtype or t.get_device() != dev:
        raise PodError(1, f"{name} must be a [rows, heads, head_dim] {dtype} tensor on cuda:{dev}")
    if (sd != 1 and d > 1) or (sh != d and h > 1):
        raise PodError(1, f"{name}: the heads of a row must be contiguous")
    if rows is not None and n != rows:
        raise PodError(1, f"{name} has {n} rows, not {rows}")
    return n, h, d, sn if n > 1 else max(sn, h * d) // 8 * 8


def _whole(name, t, shape, dtype, dev):
    """Pointer of a contiguous tensor of this shape."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev or not t.is_contiguous():
        raise PodError(1, f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on cuda:{dev}")
    return t.data_ptr()


def _rotation(positions, rows, rotary_dim, d, dev):
    """(positions pointer, rotary_dim)."""
    R = d if rotary_dim is None else int(rotary_dim)
    if positions is None:
        if R:
            raise PodError(1, "the rotation needs positions")
        return 0, R
    return _whole("positions", positions, (rows,), _torch_module.int32, dev), R


def _status(status, dev):
    if status is None:
        return 0
    if status.dtype != _torch_module.int32 or status.get_device() != dev or status.numel() < 1:
        raise PodError(1, f"status must be an int32 tensor on cuda:{dev}")
    return status.data_ptr()


def _cache_args(kv_cache, kv_scales, kv_layout, dtype, dev):
    """(cache pointer, scales pointer, pages, page size, Hk, d, layout, format)
    of a paged cache: 16-bit, or E4M3 codes with or without scale bytes."""
    hnd = _LAYOUTS.get(kv_layout)
    if hnd is None:
        raise PodError(1, f"unknown kv layout {kv_layout!r}")
    shape, kt = kv_cache.shape, kv_cache.dtype
    if len(shape) != 5 or shape[1] != 2 or kv_cache.get_device() != dev or not kv_cache.is_contiguous():
        raise PodError(1, f"kv_cache must be a contiguous [pages, 2, ...] page pool on cuda:{dev}")
    pages, _, ps, hk, d = shape
    if hnd:
        ps, hk = hk, ps
    sp = 0
    if kt == dtype:
        fmt = 0
        if kv_scales is not None:
            raise PodError(1, "kv_scales given, but the cache is a 16-bit one")
    elif kt != _torch_module.float8_e4m3fn:
        raise PodError(2, f"kv_cache must be {dtype} or float8_e4m3fn, not {kt}")
    elif kv_scales is None:
        fmt = 1
    else:
        fmt = 2
        sp = _whole("kv_scales", kv_scales, shape[:4], _torch_module.uint8, dev)
    return kv_cache.data_ptr(), sp, pages, ps, hk, d, hnd, fmt


def _call(fn, dev, stream, *args):
    """fn(*args, stream) with device `dev` current (it is made so where it is
    not) and, without a given stream, torch's current stream of that device."""
    if stream is None:
        s = _raw_stream(dev)
    else:
        s = stream if isinstance(stream, int) else stream.cuda_stream
    if _current_device() == dev:
        code = fn(*args, s)
    else:
        with _torch_module.cuda.device(dev):
            code = fn(*args, s)
    if code != POD_OK:
        raise PodError(code, pod_last_error())


def _empty(shape, dtype, t, stream):
    """A new output on t's device: memory of the stream that the call writes it on."""
    torch = _torch_module
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=t.device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=t.device) if stream else torch.cuda.default_stream(t.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=t.device)


def _out_rows(name, out, like, rows, heads, d, dtype, dev, stream):
    """(output [rows, heads, d], its row stride): new, or the caller's."""
    if out is None:
        return _empty((rows, heads, d), dtype, like, stream), heads * d
    n, h, dd, stride = _heads(name, out, dtype, dev, rows)
    if h != heads or dd != d:
        raise PodError(1, f"{name} must be {(rows, heads, d)}")
    return out, stride


# struct pod_io_args: 12 pointers, 7 int64, 9 int32, 5 floats
_IO_ARGS = struct.Struct("@12Q7q9i5f")


def pod_qk_norm_rope(q, k, positions=None, *, q_weight=None, k_weight=None, eps=1e-6, rotary_dim=None,
                     interleaved=False, rope_scale=1.0, rope_theta=1e4, q_out=None, k_out=None,
                     stream=None):
    """RMS norm of every head of q [rows, H, d] and k [rows, Hk, d] (where its
    weight is given) and the rotation of the first ``rotary_dim`` elements
    (default all, 0 none) at int32 ``positions``, in one pass. q and k may be
    slices of a fused projection (any row stride that is a multiple of 8);
    either may be None. Returns (q_out, k_out); pass q_out=q, k_out=k to work
    in place."""
    lib = _lib or load_library()
    _torch()
    t = q if q is not None else k
    dev, dtype = _device_of(t), t.dtype
    code = _dtype_code(dtype)
    H = Hk = qs = ks = qos = kos = qp = kp = qop = kop = 0
    if q is not None:
        rows, H, d, qs = _heads("q", q, dtype, dev)
        q_out, qos = _out_rows("q_out", q_out, t, rows, H, d, dtype, dev, stream)
        qp, qop = q.data_ptr(), q_out.data_ptr()
    if k is not None:
        rows, Hk, dk, ks = _heads("k", k, dtype, dev, None if q is None else rows)
        if q is not None and dk != d:
            raise PodError(1, "q and k have different head_dim")
        d = dk
        k_out, kos = _out_rows("k_out", k_out, t, rows, Hk, d, dtype, dev, stream)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    pos, R = _rotation(positions, rows, rotary_dim, d, dev)
    wq = 0 if q_weight is None else _whole("q_weight", q_weight, (d,), dtype, dev)
    wk = 0 if k_weight is None else _whole("k_weight", k_weight, (d,), dtype, dev)
    _call(lib.pod_qk_norm_rope, dev, stream, _IO_ARGS.pack(
        qp, kp, 0, wq, wk, pos, 0, qop, kop, 0, 0, 0, qs, ks, 0, qos, kos, rows, 0, 0, H, Hk, d, 0, 0, code, R,
        bool(interleaved), eps, rope_scale, rope_theta, 1.0, 1.0))
    return (q_out if q is not None else None), (k_out if k is not None else None)


def _written(k, v, kv_cache, kv_scales, kv_layout, slots):
    """Checks of the rows of a write: (device, dtype, rows, k stride, v stride, slots pointer, cache args)."""
    torch = _torch()
    dev, dtype = _device_of(k), k.dtype
    rows, hk, d, ks = _heads("k", k, dtype, dev)
    _, hv, dv, vs = _heads("v", v, dtype, dev, rows)
    cache = _cache_args(kv_cache, kv_scales, kv_layout, dtype, dev)
    if hv != hk or dv != d or cache[4] != hk or cache[5] != d:
        raise PodError(1, "k, v and kv_cache differ in heads or head_dim")
    return dev, dtype, rows, ks, vs, _whole("slots", slots, (rows,), torch.int64, dev), cache


def pod_append_kv(k, v, kv_cache, slots, *, kv_scales=None, k_scale=1.0, v_scale=1.0, kv_layout="NHD",
                  status=None, stream=None):
    """Write rows of k and v [rows, Hk, d] into the int64 ``slots`` of a paged
    cache: a cache of k's dtype takes the values, a float8_e4m3fn one E4M3
    codes, with the per-tensor k_scale and v_scale or, where ``kv_scales``
    (uint8, the cache's shape without head_dim) is given, a power-of-two scale
    per token and KV head. Negative slots are skipped."""
    lib = _lib or load_library()
    dev, dtype, rows, ks, vs, sl, (cache, scales, pages, ps, hk, d, hnd, fmt) = \
        _written(k, v, kv_cache, kv_scales, kv_layout, slots)
    _call(lib.pod_append_kv, dev, stream, _IO_ARGS.pack(
        0, k.data_ptr(), v.data_ptr(), 0, 0, 0, sl, 0, 0, cache, scales, _status(status, dev), 0, ks, vs, 0, 0,
        rows, pages, ps, 0, hk, d, hnd, fmt, _dtype_code(dtype), 0, 0, 0.0, 1.0, 1.0, k_scale, v_scale))


def pod_norm_rope_append(q, k, v, positions, kv_cache, slots, *, q_weight=None, k_weight=None, eps=1e-6,
                         rotary_dim=None, interleaved=False, rope_scale=1.0, rope_theta=1e4,
                         kv_scales=None, k_scale=1.0, v_scale=1.0, kv_layout="NHD", q_out=None,
                         status=None, stream=None):
    """pod_qk_norm_rope and pod_append_kv in one pass: returns q normed and
    rotated (None without q), writes k (normed and rotated) and v into the
    cache."""
    lib = _lib or load_library()
    dev, dtype, rows, ks, vs, sl, (cache, scales, pages, ps, hk, d, hnd, fmt) = \
        _written(k, v, kv_cache, kv_scales, kv_layout, slots)
    H = qs = qos = qp = qop = 0
    if q is not None:
        _, H, dq, qs = _heads("q", q, dtype, dev, rows)
        if dq != d:
            raise PodError(1, "q and k have different head_dim")
        q_out, qos = _out_rows("q_out", q_out, k, rows, H, d, dtype, dev, stream)
        qp, qop = q.data_ptr(), q_out.data_ptr()
    pos, R = _rotation(positions, rows, rotary_dim, d, dev)
    wq = 0 if q_weight is None else _whole("q_weight", q_weight, (d,), dtype, dev)
    wk = 0 if k_weight is None else _whole("k_weight", k_weight, (d,), dtype, dev)
    _call(lib.pod_norm_rope_append, dev, stream, _IO_ARGS.pack(
        qp, k.data_ptr(), v.data_ptr(), wq, wk, pos, sl, qop, 0, cache, scales, _status(status, dev), qs, ks, vs,
        qos, 0, rows, pages, ps, H, hk, d, hnd, fmt, _dtype_code(dtype), R, bool(interleaved), eps, rope_scale,
        rope_theta, k_scale, v_scale))
    return q_out if q is not None else None


def pod_gather_kv(kv_cache, slots, *, dtype, kv_scales=None, k_scale=1.0, v_scale=1.0, kv_layout="NHD",
                  out=None, status=None, stream=None):
    """Cache rows of the int64 ``slots`` back as ``dtype`` values:
    [rows, 2, Hk, d], K then V; a negative slot reads as zeros. The result
    viewed as [rows, 2, 1, Hk, d] is an NHD cache of page size 1."""
    lib = _lib or load_library()
    torch = _torch()
    dev = _device_of(kv_cache)
    code = _dtype_code(dtype)
    cache, scales, pages, ps, hk, d, hnd, fmt = _cache_args(kv_cache, kv_scales, kv_layout, dtype, dev)
    rows = slots.numel()
    sl = _whole("slots", slots, (rows,), torch.int64, dev)
    if out is None:
        out = _empty((rows, 2, hk, d), dtype, kv_cache, stream)
        op = out.data_ptr()
    else:
        op = _whole("out", out, (rows, 2, hk, d), dtype, dev)
    _call(lib.pod_gather_kv, dev, stream, _IO_ARGS.pack(
        0, 0, 0, 0, 0, 0, sl, 0, op, cache, scales, _status(status, dev), 0, 0, 0, 0, 0, rows, pages, ps,
        0, hk, d, hnd, fmt, code, 0, 0, 0.0, 1.0, 1.0, k_scale, v_scale))
    return out


# ------------------------------------------------------------------ tree attention
@dataclass
class PodTreeHandle:
    """Owns a tree plan of the C library (released by ``pod_tree_destroy``)."""
    ptr: int
    workspace_bytes: int
    rows: int
    num_qo_heads: int
    num_kv_heads: int
    head_dim: int
    page_size: int
    num_pages: int
    dtype: object
    kv_format: int
    kv_layout: int
    mask_bytes: int
    has_sinks: bool
    pool_shape: tuple = ()
    workspace_ptr: Optional[int] = None

    def __del__(self):
        if self.ptr and _lib is not None:
            _lib.pod_tree_destroy(ctypes.c_void_p(self.ptr))
            self.ptr = 0


def _workspace(workspace):
    """(pointer, bytes) of a tree plan's workspace. A view with gaps or repeats counts
    more bytes than lie behind its first."""
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise PodError(1, "the workspace must be a contiguous CUDA tensor")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def pod_tree_plan(q_indptr, kv_indptr, kv_indices, last_page_len, num_qo_heads, num_kv_heads, head_dim, page_size,
                  *, dtype, num_pages, sm_scale=None, kv_format="16bit", k_scale=1.0, v_scale=1.0, kv_layout="NHD",
                  has_sinks=False, num_sms=0, workspace=None, stream=None) -> PodTreeHandle:
    """Plan the attention of drafted token trees: request r's
    q_indptr[r+1] - q_indptr[r] tokens are the last keys of its pages. Index
    arrays are host int32. ``kv_format``: "16bit", "scaled" (E4M3, per-tensor
    k_scale and v_scale) or "block" (E4M3 with exponent bytes). Bind a
    workspace before running (here, or with pod_tree_bind_workspace)."""
    lib = load_library()
    arrs = [_i32(x) for x in (q_indptr, kv_indptr, kv_indices, last_page_len)]
    if kv_format not in _KV_FORMATS or kv_layout not in _LAYOUTS:
        raise PodError(1, f"unknown kv_format {kv_format!r} or kv_layout {kv_layout!r}")
    batch = 0 if arrs[0] is None else len(arrs[0]) - 1
    if batch > 0:
        if any(a is None for a in arrs):
            raise PodError(1, "a page table array is missing")
        if len(arrs[1]) != batch + 1 or len(arrs[3]) != batch or len(arrs[2]) < int(arrs[1][-1]):
            raise PodError(1, "the page table arrays do not fit together")
    handle, req = ctypes.c_void_p(), ctypes.c_size_t(0)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else _workspace(workspace)
    code = lib.pod_tree_plan(*[_ptr(a) for a in arrs], max(batch, 0), int(num_pages), int(num_qo_heads),
                             int(num_kv_heads), int(head_dim), int(page_size),
                             float(sm_scale) if sm_scale is not None else 0.0, _dtype_code(dtype),
                             _KV_FORMATS[kv_format], float(k_scale), float(v_scale), _LAYOUTS[kv_layout],
                             int(bool(has_sinks)), int(num_sms), ws_ptr, ws_bytes,
                             _stream(stream) if ws_ptr else None, ctypes.byref(handle), ctypes.byref(req))
    if code != POD_OK:
        err = PodError(code, pod_last_error())
        err.required_workspace_bytes = int(req.value)
        raise err
    n = np.diff(arrs[0].astype(np.int64)) if batch > 0 else np.zeros(0, np.int64)
    return PodTreeHandle(ptr=handle.value, workspace_bytes=int(req.value), rows=int(n.sum()),
                         num_qo_heads=int(num_qo_heads), num_kv_heads=int(num_kv_heads), head_dim=int(head_dim),
                         page_size=int(page_size), num_pages=int(num_pages), dtype=dtype,
                         kv_format=_KV_FORMATS[kv_format], kv_layout=_LAYOUTS[kv_layout],
                         mask_bytes=int((int((n * n).sum()) + 7) // 8), has_sinks=bool(has_sinks),
                         pool_shape=(int(num_pages), 2) + ((int(num_kv_heads), int(page_size)) if _LAYOUTS[kv_layout]
                                                           else (int(page_size), int(num_kv_heads)))
                         + (int(head_dim),), workspace_ptr=ws_ptr)


def pod_tree_workspace_size(h: PodTreeHandle) -> int:
    return int(load_library().pod_tree_workspace_size(ctypes.c_void_p(h.ptr)))


def pod_tree_bind_workspace(h: PodTreeHandle, workspace, stream=None):
    _torch()
    ptr, size = _workspace(workspace)
    _call(load_library().pod_tree_bind_workspace, _device_of(workspace), stream, h.ptr, ptr, size)
    h.workspace_ptr = ptr


def pod_tree_run(h: PodTreeHandle, q, kv, workspace, tree_mask=None, kv_scales=None, sinks=None, out=None, lse=None,
                 stream=None):
    """Attention of the planned trees: q [rows, H, d], kv the paged cache,
    ``tree_mask`` uint8 bits (little bit order) of every request's [n, n]
    matrix end to end (None: chains). Returns (out, lse), lse in base 2."""
    lib = _lib or load_library()
    torch = _torch()
    dev, dtype = _device_of(q), h.dtype
    shape, pool = (h.rows, h.num_qo_heads, h.head_dim), h.pool_shape
    qp = _whole("q", q, shape, dtype, dev)
    cp = _whole("kv", kv, pool, torch.float8_e4m3fn if h.kv_format else dtype, dev)
    sp = mp = mn = kp = 0
    if kv_scales is not None:
        sp = _whole("kv_scales", kv_scales, pool[:4], torch.uint8, dev)
    if tree_mask is not None:
        mn = tree_mask.numel()
        mp = _whole("tree_mask", tree_mask, (mn,), torch.uint8, dev)
        if mn < h.mask_bytes:
            raise PodError(1, f"tree_mask needs {h.mask_bytes} bytes")
    if sinks is not None:
        kp = _whole("sinks", sinks, (h.num_qo_heads,), torch.float32, dev)
    if workspace.get_device() != dev:
        raise PodError(1, f"the workspace must be on cuda:{dev}")
    if out is None:
        out = _empty(shape, dtype, q, stream)
        op = out.data_ptr()
    else:
        op = _whole("out", out, shape, dtype, dev)
    if lse is None:
        lse = _empty(shape[:2], torch.float32, q, stream)
        lp = lse.data_ptr()
    else:
        lp = _whole("lse", lse, shape[:2], torch.float32, dev)
    _call(lib.pod_tree_run, dev, stream, h.ptr, qp, cp, sp, mp, mn, kp, workspace.data_ptr(), op, lp)
    return out, lse


def pod_tree_read_device_status(h: PodTreeHandle, workspace, stream=None) -> int:
    v = ctypes.c_int32(0)
    _torch()
    try:
        _call(lambda st: load_library().pod_tree_read_device_status(h.ptr, workspace.data_ptr(), st, ctypes.byref(v)),
              _device_of(workspace), stream)
    except PodError as e:
        if e.code != 5:
            raise
    return int(v.value)


def pod_tree_plan_table(h: PodTreeHandle, which: int) -> np.ndarray:
    lib = load_library()
    n = ctypes.c_int64(0)
    _check(lib.pod_tree_plan_table(ctypes.c_void_p(h.ptr), int(which), None, 0, ctypes.byref(n)))
    out = np.zeros(max(n.value, 1), dtype=np.int32)
    _check(lib.pod_tree_plan_table(ctypes.c_void_p(h.ptr), int(which), out.ctypes.data, n.value, ctypes.byref(n)))
    return out[:n.value]


def pod_tree_destroy(h: PodTreeHandle):
    if h.ptr:
        load_library().pod_tree_destroy(ctypes.c_void_p(h.ptr))
        h.ptr = 0
