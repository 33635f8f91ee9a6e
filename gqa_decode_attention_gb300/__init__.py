"""GB300-native grouped-query decode attention: Python binding.

A thin ctypes layer over ``libgqa_decode.so`` (the C ABI declared in
``include/gqa_decode.h``).  Functions carry the C entry points' names and
only marshal arguments: torch tensors supply device memory and the current
CUDA stream; every step of the computation runs in the library's kernels.
There is no fallback: if the library is missing, importing a function that
needs it raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgqa_decode.so")

STATUS = {
    0: "GQA_OK",
    1: "GQA_ERR_INVALID_ARG",
    2: "GQA_ERR_UNSUPPORTED",
    3: "GQA_ERR_ALIGNMENT",
    4: "GQA_ERR_NO_MEMORY",
    5: "GQA_ERR_CUDA",
    6: "GQA_ERR_DEVICE_TIMEOUT",
    7: "GQA_ERR_DEVICE_INDEX",
}
GQA_OK = 0

# Every symbol the headers in include/ declare.
EXPORTS = [
    "gqa_status_string", "gqa_version", "gqa_decode", "gqa_decode_num_splits",
    "gqa_decode_workspace_bytes", "gqa_decode_ex", "gqa_decode_dv", "gqa_decode_dv_num_splits",
    "gqa_decode_dv_workspace_bytes", "gqa_decode_dense_engine",
    "gqa_decode_noalloc", "gqa_decode_noalloc_scratch_bytes",
    "gqa_decode_host", "gqa_decode_paged_fp8", "gqa_decode_paged_fp8_dev_scales", "gqa_decode_paged", "gqa_decode_paged_ex",
    "gqa_decode_paged_num_splits", "gqa_decode_paged_workspace_bytes", "gqa_decode_paged_dev_scales",
    "gqa_decode_paged_int4", "gqa_decode_paged_int4_num_splits", "gqa_decode_paged_int4_workspace_bytes",
    "gqa_paged_append", "gqa_paged_gather",
    "gqa_paged_gather_fp8", "gqa_fp8_e4m3fn_to_f32", "gqa_device_status", "gqa_set_wait_limit_ns",
    "gqa_debug_set_fault_mode", "gqa_debug_set_kernel_events", "gqa_debug_read_stream",
    "gqa_decode_paged_engine", "gqa_debug_set_paged_engine",
]


class GQAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {STATUS.get(int(status), status)}")


_lib_handle = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libgqa_decode.so (built by ``gqa_decode_attention_gb300.build``)."""
    global _lib_handle
    if _lib_handle is not None:
        return _lib_handle
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m gqa_decode_attention_gb300.build`")
    lib = ctypes.CDLL(path)
    vp, i, f, st, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int, ctypes.c_size_t
    lib.gqa_status_string.restype = ctypes.c_char_p
    lib.gqa_status_string.argtypes = [st]
    lib.gqa_version.restype = ctypes.c_char_p
    lib.gqa_version.argtypes = []
    lib.gqa_decode.restype = st
    lib.gqa_decode.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, vp]
    lib.gqa_decode_num_splits.restype = i
    lib.gqa_decode_num_splits.argtypes = [i] * 6
    lib.gqa_decode_workspace_bytes.restype = sz
    lib.gqa_decode_workspace_bytes.argtypes = [i] * 7
    lib.gqa_decode_ex.restype = st
    lib.gqa_decode_ex.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, sz, vp]
    lib.gqa_decode_dv.restype = st
    lib.gqa_decode_dv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, vp, sz, vp]
    lib.gqa_decode_dv_num_splits.restype = i
    lib.gqa_decode_dv_num_splits.argtypes = [i] * 7
    lib.gqa_decode_dense_engine.restype = i
    lib.gqa_decode_dense_engine.argtypes = [i] * 7
    lib.gqa_decode_dv_workspace_bytes.restype = sz
    lib.gqa_decode_dv_workspace_bytes.argtypes = [i] * 8
    lib.gqa_decode_noalloc.restype = st
    lib.gqa_decode_noalloc.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp]
    lib.gqa_decode_noalloc_scratch_bytes.restype = sz
    lib.gqa_decode_noalloc_scratch_bytes.argtypes = []
    lib.gqa_decode_host.restype = st
    lib.gqa_decode_host.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, vp]
    lib.gqa_decode_paged_fp8.restype = st
    lib.gqa_decode_paged_fp8.argtypes = [vp, vp, vp, vp, vp, vp, f, f, vp, vp] + [i] * 8 + [f, vp]
    lib.gqa_decode_paged_fp8_dev_scales.restype = st
    lib.gqa_decode_paged_fp8_dev_scales.argtypes = [vp] * 8 + [i, vp, vp] + [i] * 8 + [f, vp]
    lib.gqa_decode_paged.restype = st
    lib.gqa_decode_paged.argtypes = [vp, vp, vp, i, f, f, vp, vp, vp, vp] + [i] * 8 + [f, vp]
    lib.gqa_decode_paged_ex.restype = st
    lib.gqa_decode_paged_ex.argtypes = [vp, vp, vp, i, f, f, vp, vp, vp, vp] + [i] * 8 + [f, i, vp, sz, vp]
    lib.gqa_decode_paged_dev_scales.restype = st
    lib.gqa_decode_paged_dev_scales.argtypes = [vp, vp, vp, i, vp, vp, i, vp, vp, vp, vp] + [i] * 8 + [f, i, vp, sz, vp]
    lib.gqa_decode_paged_num_splits.restype = i
    lib.gqa_decode_paged_num_splits.argtypes = [i] * 8
    lib.gqa_decode_paged_workspace_bytes.restype = sz
    lib.gqa_decode_paged_workspace_bytes.argtypes = [i] * 9
    ll = ctypes.c_longlong
    lib.gqa_decode_paged_int4.restype = st
    lib.gqa_decode_paged_int4.argtypes = [vp] * 8 + [i] * 8 + [f, i, vp, sz, vp]
    lib.gqa_decode_paged_int4_num_splits.restype = i
    lib.gqa_decode_paged_int4_num_splits.argtypes = [i] * 7
    lib.gqa_decode_paged_int4_workspace_bytes.restype = sz
    lib.gqa_decode_paged_int4_workspace_bytes.argtypes = [i] * 8
    lib.gqa_paged_append.restype = st
    lib.gqa_paged_append.argtypes = ([vp, ll, vp, vp, ll, vp, ll, i, vp, vp, vp, f, f, vp, vp, i, vp, vp, vp, vp]
                                     + [i] * 11 + [vp])
    lib.gqa_paged_gather.restype = st
    lib.gqa_paged_gather.argtypes = [i, vp, vp, vp, f, f, vp, vp, i, vp, vp, vp, vp, vp] + [i] * 7 + [vp]
    lib.gqa_paged_gather_fp8.restype = st
    lib.gqa_paged_gather_fp8.argtypes = [vp, vp, vp, vp] + [i] * 7 + [vp]
    lib.gqa_fp8_e4m3fn_to_f32.restype = st
    lib.gqa_fp8_e4m3fn_to_f32.argtypes = [vp, vp, i, vp]
    lib.gqa_device_status.restype = st
    lib.gqa_device_status.argtypes = [vp]
    lib.gqa_set_wait_limit_ns.restype = None
    lib.gqa_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.gqa_debug_set_fault_mode.restype = None
    lib.gqa_debug_set_fault_mode.argtypes = [i]
    lib.gqa_debug_set_kernel_events.restype = None
    lib.gqa_debug_set_kernel_events.argtypes = [vp, vp]
    lib.gqa_decode_paged_engine.restype = i
    lib.gqa_decode_paged_engine.argtypes = [i] * 7
    lib.gqa_debug_set_paged_engine.restype = None
    lib.gqa_debug_set_paged_engine.argtypes = [i]
    lib.gqa_debug_read_stream.restype = st
    lib.gqa_debug_read_stream.argtypes = [vp, sz, vp, vp]
    _lib_handle = lib
    return lib


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status: int, where: str):
    if status != GQA_OK:
        raise GQAError(status, where)


def _need(t: torch.Tensor, name: str, dtype, device_type: str):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device.type != device_type:
        raise ValueError(f"{name}: expected a {device_type} tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _need_shape(t, name: str, shape, dtype, like: torch.Tensor):
    """A caller-supplied tensor the library reads or writes through a raw
    pointer: it must have exactly the shape the call implies (a smaller one
    would be read or written out of bounds), the dtype, and lie contiguous on
    the device of `like`."""
    if t is None:
        return
    _need(t, name, dtype, like.device.type)
    if t.device != like.device:
        raise ValueError(f"{name}: expected a tensor on {like.device}, got {t.device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _dense_shapes(fn: str, q, k, v, out, lse, Dv=None):
    """Shape checks shared by the dense entry points: q [B,Sq,Hq,D],
    k [B,Skv,Hkv,D], v [B,Skv,Hkv,Dv], out [B,Sq,Hq,Dv], lse [B,Hq,Sq]."""
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError(f"{fn}: q, k and v must be 4-D")
    B, Sq, Hq, D = q.shape
    _, Skv, Hkv, _ = k.shape
    Dv = D if Dv is None else Dv
    if tuple(k.shape) != (B, Skv, Hkv, D) or tuple(v.shape) != (B, Skv, Hkv, Dv):
        raise ValueError(f"{fn}: k must be [B,Skv,Hkv,{D}] and v [B,Skv,Hkv,{Dv}] with q's batch")
    for t, n in ((k, "k"), (v, "v")):
        if t.device != q.device:
            raise ValueError(f"{fn}: {n} is on {t.device}, q on {q.device}")
    _need_shape(out, "out", (B, Sq, Hq, Dv), torch.bfloat16, q)
    _need_shape(lse, "lse", (B, Hq, Sq), torch.float32, q)


def _scale_arg(scale):
    return 0.0 if scale is None else float(scale)


# ---------------------------------------------------------------------------
# dense
# ---------------------------------------------------------------------------
def gqa_decode(q, k, v, out=None, lse=None, scale=None, stream=None, with_lse=True):
    """Dense GQA decode.  q [B,Sq,Hq,D], k/v [B,Skv,Hkv,D] bf16 on CUDA.

    Returns (out [B,Sq,Hq,D] bf16, lse [B,Hq,Sq] fp32 or None).
    """
    return gqa_decode_ex(q, k, v, out=out, lse=lse, scale=scale, num_splits=0, workspace=None,
                         stream=stream, with_lse=with_lse)


def gqa_decode_ex(q, k, v, out=None, lse=None, scale=None, num_splits=0, workspace=None, stream=None,
                  with_lse=True):
    """gqa_decode with an explicit split count (0 = automatic) and an optional
    caller workspace (a CUDA uint8 tensor of at least gqa_decode_workspace_bytes)."""
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, "cuda")
    _dense_shapes("gqa_decode_ex", q, k, v, out, lse)
    B, Sq, Hq, D = q.shape
    _, Skv, Hkv, _ = k.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and with_lse:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    st = lib.gqa_decode_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Sq, Skv, Hq, Hkv, D,
                           _scale_arg(scale), int(num_splits), ws_ptr, ws_bytes, _stream(stream))
    _check(st, "gqa_decode_ex")
    return out, lse


def gqa_decode_dv(q, k, v, out=None, lse=None, scale=None, num_splits=0, workspace=None, stream=None,
                  with_lse=True):
    """Dense decode with a score head size Dqk (q, k) different from the value
    head size Dv (v, out): q [B,Sq,Hq,Dqk], k [B,Skv,Hkv,Dqk], v [B,Skv,Hkv,Dv].

    Returns (out [B,Sq,Hq,Dv] bf16, lse [B,Hq,Sq] fp32 or None)."""
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, "cuda")
    B, Sq, Hq, Dqk = q.shape
    _, Skv, Hkv, _ = k.shape
    Dv = v.shape[-1]
    _dense_shapes("gqa_decode_dv", q, k, v, out, lse, Dv=Dv)
    if out is None:
        out = torch.empty((B, Sq, Hq, Dv), dtype=torch.bfloat16, device=q.device)
    if lse is None and with_lse:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    st = lib.gqa_decode_dv(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Sq, Skv, Hq, Hkv, Dqk, Dv,
                           _scale_arg(scale), int(num_splits), ws_ptr, ws_bytes, _stream(stream))
    _check(st, "gqa_decode_dv")
    return out, lse


def gqa_decode_dv_num_splits(B, Sq, Skv, Hq, Hkv, Dqk, Dv) -> int:
    n = load_library().gqa_decode_dv_num_splits(B, Sq, Skv, Hq, Hkv, Dqk, Dv)
    if n < 0:
        raise GQAError(-n, "gqa_decode_dv_num_splits")
    return n


ENGINES = {0: "mma.sync", 1: "tcgen05"}


def gqa_decode_dense_engine(B, Sq, Skv, Hq, Hkv, Dqk, Dv=None) -> str:
    """Kernel engine a dense call of this shape runs: "mma.sync" or "tcgen05"."""
    n = load_library().gqa_decode_dense_engine(B, Sq, Skv, Hq, Hkv, Dqk, Dqk if Dv is None else Dv)
    if n < 0:
        raise GQAError(-n, "gqa_decode_dense_engine")
    return ENGINES[n]


def gqa_decode_dv_workspace_bytes(B, Sq, Skv, Hq, Hkv, Dqk, Dv, num_splits=0) -> int:
    return int(load_library().gqa_decode_dv_workspace_bytes(B, Sq, Skv, Hq, Hkv, Dqk, Dv, int(num_splits)))


def gqa_decode_noalloc(q, k, v, out, lse=None, scale=None, num_splits=0, stream=None):
    """Allocation-free dense decode (fixed in-library scratch, caller-owned
    out / lse; see include/gqa_decode.h).  Allocates nothing, not even outputs."""
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _need(t, n, torch.bfloat16, "cuda")
    _dense_shapes("gqa_decode_noalloc", q, k, v, out, lse)
    B, Sq, Hq, D = q.shape
    _, Skv, Hkv, _ = k.shape
    st = lib.gqa_decode_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Sq, Skv, Hq, Hkv, D,
                                _scale_arg(scale), int(num_splits), _stream(stream))
    _check(st, "gqa_decode_noalloc")
    return out, lse


def gqa_decode_noalloc_scratch_bytes() -> int:
    return int(load_library().gqa_decode_noalloc_scratch_bytes())


def gqa_decode_num_splits(B, Sq, Skv, Hq, Hkv, D) -> int:
    n = load_library().gqa_decode_num_splits(B, Sq, Skv, Hq, Hkv, D)
    if n < 0:
        raise GQAError(-n, "gqa_decode_num_splits")
    return n


def gqa_decode_workspace_bytes(B, Sq, Skv, Hq, Hkv, D, num_splits=0) -> int:
    return int(load_library().gqa_decode_workspace_bytes(B, Sq, Skv, Hq, Hkv, D, int(num_splits)))


def gqa_decode_host(q, k, v, out, lse=None, scale=None, stream=None):
    """End-to-end form on HOST (ideally pinned) tensors; returns when done."""
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _need(t, n, torch.bfloat16, "cpu")
    _dense_shapes("gqa_decode_host", q, k, v, out, lse)
    B, Sq, Hq, D = q.shape
    _, Skv, Hkv, _ = k.shape
    st = lib.gqa_decode_host(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Sq, Skv, Hq, Hkv, D,
                             _scale_arg(scale), _stream(stream))
    _check(st, "gqa_decode_host")
    return out, lse


# ---------------------------------------------------------------------------
# sparse paged FP8
# ---------------------------------------------------------------------------
def gqa_decode_paged_fp8(q, gate, k_pool, v_pool, page_table, topk_idx, k_scale=1.0, v_scale=1.0, out=None,
                         lse=None, scale=None, stream=None, with_lse=True, k_scales=None, v_scales=None):
    """Sparse paged decode over an FP8 E4M3FN pool with a sigmoid gate.

    q, gate [B,Hq,D] bf16; pools uint8 [num_pages, page_size, Hkv, D];
    page_table int32 [B, pages_per_req]; topk_idx int32 [B, topk].
    k_scales / v_scales: optional CUDA fp32 tensors of 1 or Hkv device-side
    scales (replace k_scale / v_scale).
    Returns (out [B,Hq,D] bf16, lse [B,Hq] fp32 or None).
    """
    lib = load_library()
    _need(q, "q", torch.bfloat16, "cuda")
    _need(gate, "gate", torch.bfloat16, "cuda")
    for t, n in ((k_pool, "k_pool"), (v_pool, "v_pool")):
        _need(t, n, torch.uint8, "cuda")
    _need(page_table, "page_table", torch.int32, "cuda")
    _need(topk_idx, "topk_idx", torch.int32, "cuda")
    if q.dim() != 3 or k_pool.dim() != 4 or page_table.dim() != 2 or topk_idx.dim() != 2:
        raise ValueError("gqa_decode_paged_fp8: q [B,Hq,D], pools [pages,page_size,Hkv,D], page_table and "
                         "topk_idx 2-D")
    B, Hq, D = q.shape
    num_pages, page_size, Hkv, _ = k_pool.shape
    if tuple(v_pool.shape) != tuple(k_pool.shape) or k_pool.shape[3] != D:
        raise ValueError("gqa_decode_paged_fp8: v_pool must have k_pool's shape, with q's head size")
    if page_table.shape[0] != B or topk_idx.shape[0] != B:
        raise ValueError("gqa_decode_paged_fp8: page_table and topk_idx need one row per request")
    for t, n in ((k_pool, "k_pool"), (v_pool, "v_pool"), (page_table, "page_table"), (topk_idx, "topk_idx")):
        if t.device != q.device:
            raise ValueError(f"gqa_decode_paged_fp8: {n} is on {t.device}, q on {q.device}")
    _need_shape(gate, "gate", (B, Hq, D), torch.bfloat16, q)
    _need_shape(out, "out", (B, Hq, D), torch.bfloat16, q)
    _need_shape(lse, "lse", (B, Hq), torch.float32, q)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and with_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if k_scales is not None or v_scales is not None:
        _need(k_scales, "k_scales", torch.float32, "cuda")
        _need(v_scales, "v_scales", torch.float32, "cuda")
        st = lib.gqa_decode_paged_fp8_dev_scales(_ptr(q), _ptr(gate), _ptr(k_pool), _ptr(v_pool), _ptr(page_table),
                                                 _ptr(topk_idx), _ptr(k_scales), _ptr(v_scales), k_scales.numel(),
                                                 _ptr(out), _ptr(lse), B, Hq, Hkv, D, page_size,
                                                 page_table.shape[1], num_pages, topk_idx.shape[1],
                                                 _scale_arg(scale), _stream(stream))
        _check(st, "gqa_decode_paged_fp8_dev_scales")
        return out, lse
    st = lib.gqa_decode_paged_fp8(_ptr(q), _ptr(gate), _ptr(k_pool), _ptr(v_pool), _ptr(page_table),
                                  _ptr(topk_idx), float(k_scale), float(v_scale), _ptr(out), _ptr(lse),
                                  B, Hq, Hkv, D, page_size, page_table.shape[1], num_pages,
                                  topk_idx.shape[1], _scale_arg(scale), _stream(stream))
    _check(st, "gqa_decode_paged_fp8")
    return out, lse


GQA_KV_BF16 = 0
GQA_KV_FP8_E4M3FN = 1
GQA_KV_INT8 = 2


def _kv_dtype(k_pool) -> int:
    if k_pool.dtype == torch.bfloat16:
        return GQA_KV_BF16
    if k_pool.dtype == torch.uint8:
        return GQA_KV_FP8_E4M3FN
    if k_pool.dtype == torch.int8:
        return GQA_KV_INT8
    raise TypeError(f"k_pool: expected bfloat16, uint8 (E4M3FN codes) or int8, got {k_pool.dtype}")


def gqa_decode_paged(q, k_pool, v_pool, page_table, seq_lens, k_scale=1.0, v_scale=1.0, out=None, lse=None,
                     scale=None, num_splits=0, workspace=None, stream=None, with_lse=True, k_scales=None,
                     v_scales=None):
    """Paged decode over every token of each request (no top-K).

    q [B,Sq,Hq,D] bf16; pools [num_pages, page_size, Hkv, D] of bf16, of
    uint8 E4M3FN codes or of int8 codes (for 8-bit codes k_scale / v_scale
    apply); page_table int32
    [B, pages_per_req]; seq_lens int32 [B].  num_splits 0 = automatic;
    workspace: optional CUDA uint8 tensor of gqa_decode_paged_workspace_bytes.
    k_scales / v_scales: optional CUDA fp32 tensors of 1 or Hkv device-side
    scales (8-bit pools; replace k_scale / v_scale).
    Returns (out [B,Sq,Hq,D] bf16, lse [B,Hq,Sq] fp32 or None).
    """
    lib = load_library()
    _need(q, "q", torch.bfloat16, "cuda")
    kvd = _kv_dtype(k_pool)
    for t, n in ((k_pool, "k_pool"), (v_pool, "v_pool")):
        _need(t, n, k_pool.dtype, "cuda")
    _need(page_table, "page_table", torch.int32, "cuda")
    _need(seq_lens, "seq_lens", torch.int32, "cuda")
    if q.dim() != 4 or k_pool.dim() != 4 or page_table.dim() != 2:
        raise ValueError("gqa_decode_paged: q [B,Sq,Hq,D], pools [pages,page_size,Hkv,D], page_table 2-D")
    B, Sq, Hq, D = q.shape
    num_pages, page_size, Hkv, _ = k_pool.shape
    if tuple(v_pool.shape) != tuple(k_pool.shape) or k_pool.shape[3] != D:
        raise ValueError("gqa_decode_paged: v_pool must have k_pool's shape, with q's head size")
    if page_table.shape[0] != B or tuple(seq_lens.shape) != (B,):
        raise ValueError("gqa_decode_paged: page_table needs one row and seq_lens one entry per request")
    for t, n in ((k_pool, "k_pool"), (v_pool, "v_pool"), (page_table, "page_table"), (seq_lens, "seq_lens")):
        if t.device != q.device:
            raise ValueError(f"gqa_decode_paged: {n} is on {t.device}, q on {q.device}")
    _need_shape(out, "out", (B, Sq, Hq, D), torch.bfloat16, q)
    _need_shape(lse, "lse", (B, Hq, Sq), torch.float32, q)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and with_lse:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    if k_scales is not None or v_scales is not None:
        _need(k_scales, "k_scales", torch.float32, "cuda")
        _need(v_scales, "v_scales", torch.float32, "cuda")
        st = lib.gqa_decode_paged_dev_scales(_ptr(q), _ptr(k_pool), _ptr(v_pool), kvd, _ptr(k_scales),
                                             _ptr(v_scales), k_scales.numel(), _ptr(page_table), _ptr(seq_lens),
                                             _ptr(out), _ptr(lse), B, Sq, Hq, Hkv, D, page_size,
                                             page_table.shape[1], num_pages, _scale_arg(scale), int(num_splits),
                                             ws_ptr, ws_bytes, _stream(stream))
        _check(st, "gqa_decode_paged_dev_scales")
        return out, lse
    st = lib.gqa_decode_paged_ex(_ptr(q), _ptr(k_pool), _ptr(v_pool), kvd, float(k_scale), float(v_scale),
                                 _ptr(page_table), _ptr(seq_lens), _ptr(out), _ptr(lse), B, Sq, Hq, Hkv, D,
                                 page_size, page_table.shape[1], num_pages, _scale_arg(scale), int(num_splits),
                                 ws_ptr, ws_bytes, _stream(stream))
    _check(st, "gqa_decode_paged_ex")
    return out, lse


def gqa_decode_paged_engine(B, Sq, Hq, Hkv, D, kv_dtype=1, topk_form=False) -> str:
    """Kernel engine a paged call of this shape runs: "mma.sync" or "tcgen05"
    (topk_form: the sparse top-K form; else whole requests with kv_dtype 0
    bf16, 1 FP8, 2 int8)."""
    n = load_library().gqa_decode_paged_engine(B, Sq, Hq, Hkv, D, int(kv_dtype), 1 if topk_form else 0)
    if n < 0:
        raise GQAError(-n, "gqa_decode_paged_engine")
    return ENGINES[n]


def gqa_debug_set_paged_engine(mode: int):
    """mode 1: every later paged call runs on the mma.sync engine; 0: by shape."""
    load_library().gqa_debug_set_paged_engine(int(mode))


def gqa_decode_paged_num_splits(B, Sq, Hq, Hkv, D, kv_dtype, page_size, pages_per_req) -> int:
    return load_library().gqa_decode_paged_num_splits(B, Sq, Hq, Hkv, D, kv_dtype, page_size, pages_per_req)


def gqa_decode_paged_workspace_bytes(B, Sq, Hq, Hkv, D, kv_dtype, page_size, pages_per_req, num_splits=0) -> int:
    return load_library().gqa_decode_paged_workspace_bytes(B, Sq, Hq, Hkv, D, kv_dtype, page_size, pages_per_req,
                                                           num_splits)


# ---------------------------------------------------------------------------
# the paged cache: 4-bit decode, append, gather
# ---------------------------------------------------------------------------
GQA_KV_INT4 = 3


# A decode step runs these calls once a layer, so their checks are written to be cheap: one expression a tensor, the
# message worked out only for a tensor that fails.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on_device_of(dev: int, stream):
    """(guard, stream pointer) of a call on CUDA device `dev`: the stream given, or that device's current one.  The
    guard is entered around the call where another device is current."""
    if dev < 0:
        raise ValueError("expected CUDA tensors")
    if stream is None:
        s = _current_raw_stream(dev) if _current_raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream
    else:
        if stream.device.index != dev:
            raise ValueError(f"stream on {stream.device}, tensors on device {dev}")
        s = stream.cuda_stream
    return (None if dev == torch.cuda.current_device() else torch.cuda.device(dev)), s


def _guarded(guard, fn, *args):
    if guard is None:
        return fn(*args)
    with guard:
        return fn(*args)


def _misfit(fn: str, name: str, t, dtype, dev: int, shape=None):
    want = f"contiguous {dtype}{'' if shape is None else ' ' + str(list(shape))} on cuda:{dev}"
    got = f"{t.dtype} {list(t.shape)} on {t.device}" if isinstance(t, torch.Tensor) else repr(t)
    return ValueError(f"{fn}: {name}: expected {want}, got {got}")


def _fit(fn: str, name: str, t, dtype, dev: int, shape=None):
    """A tensor the library reads or writes through a raw pointer: its type, device, layout and (unless None) shape."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or (shape is not None and t.shape != shape):
        raise _misfit(fn, name, t, dtype, dev, shape)


def _data(t):
    return None if t is None else t.data_ptr()


def _cache(fn: str, dev: int, k_pool, v_pool, kv_params, page_table, seq_lens, k_scales, v_scales):
    """Checks the cache's tensors against each other; returns (kv_dtype, num_pages, page_size, Hkv, D, B,
    pages_per_req, n_scales)."""
    shape = k_pool.shape
    if len(shape) != 4 or page_table.dim() != 2:
        raise ValueError(f"{fn}: pools [num_pages,page_size,Hkv,D or D/2], page_table 2-D")
    num_pages, page_size, Hkv, D = shape
    B, pages_per_req = page_table.shape
    kind = k_pool.dtype
    if kv_params is None:
        kvd = _kv_dtype(k_pool)
    else:
        kvd, D = GQA_KV_INT4, 2 * D
        if kind is not torch.uint8:
            raise _misfit(fn, "k_pool", k_pool, torch.uint8, dev)
        _fit(fn, "kv_params", kv_params, torch.float16, dev, (num_pages, page_size, Hkv, 4))
    if not (v_pool.dtype is kind and page_table.dtype is torch.int32 and seq_lens.dtype is torch.int32
            and v_pool.shape == shape and seq_lens.shape == (B,)
            and k_pool.get_device() == dev and v_pool.get_device() == dev and page_table.get_device() == dev
            and seq_lens.get_device() == dev and k_pool.is_contiguous() and v_pool.is_contiguous()
            and page_table.is_contiguous() and seq_lens.is_contiguous()):
        _fit(fn, "k_pool", k_pool, kind, dev)
        _fit(fn, "v_pool", v_pool, kind, dev, shape)
        _fit(fn, "page_table", page_table, torch.int32, dev)
        _fit(fn, "seq_lens", seq_lens, torch.int32, dev, (B,))
    n_scales = 0
    if k_scales is not None or v_scales is not None:
        if k_scales is None or v_scales is None:
            raise ValueError(f"{fn}: k_scales and v_scales go together")
        n_scales = k_scales.numel()
        _fit(fn, "k_scales", k_scales, torch.float32, dev)
        _fit(fn, "v_scales", v_scales, torch.float32, dev)
        if v_scales.numel() != n_scales:
            raise ValueError(f"{fn}: k_scales and v_scales need the same number of values")
    return kvd, num_pages, page_size, Hkv, D, B, pages_per_req, n_scales


def _new(shape, dtype, like, stream, make=torch.empty):
    """An output the call allocates.  With a stream given it comes from that stream's memory -- the current stream's may
    still be in use by work queued there, which the kernel would not wait for -- and it may be freed while the current
    stream still reads it."""
    if stream is None:
        return make(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        t = make(shape, dtype=dtype, device=like.device)
    t.record_stream(torch.cuda.current_stream(like.device))
    return t


def gqa_decode_paged_int4(q, k_pool, v_pool, kv_params, page_table, seq_lens, out=None, lse=None, scale=None,
                          num_splits=0, workspace=None, stream=None, with_lse=True):
    """Paged decode over every token of each request from a 4-bit cache.

    q [B,Sq,Hq,D] bf16; pools uint8 [num_pages, page_size, Hkv, D/2] (element 2i in the low half of byte i);
    kv_params fp16 [num_pages, page_size, Hkv, 4] (K scale, K zero, V scale, V zero; value = code * scale + zero);
    page_table int32 [B, pages_per_req]; seq_lens int32 [B].  num_splits 0 = automatic; workspace: optional CUDA uint8
    tensor of gqa_decode_paged_int4_workspace_bytes.
    Returns (out [B,Sq,Hq,D] bf16, lse [B,Hq,Sq] fp32 or None).
    """
    lib = _lib_handle or load_library()
    fn = "gqa_decode_paged_int4"
    dev = q.get_device()
    guard, cs = _on_device_of(dev, stream)
    if kv_params is None or q.dim() != 4:
        raise ValueError(f"{fn}: q [B,Sq,Hq,D] and kv_params are needed")
    _, num_pages, page_size, Hkv, D, B, ppr, _ = _cache(fn, dev, k_pool, v_pool, kv_params, page_table, seq_lens, None, None)
    _, Sq, Hq, _ = q.shape
    _fit(fn, "q", q, torch.bfloat16, dev, (B, Sq, Hq, D))
    if out is None:
        out = _new((B, Sq, Hq, D), torch.bfloat16, q, stream)
    else:
        _fit(fn, "out", out, torch.bfloat16, dev, (B, Sq, Hq, D))
    if lse is not None:
        _fit(fn, "lse", lse, torch.float32, dev, (B, Hq, Sq))
    elif with_lse:
        lse = _new((B, Hq, Sq), torch.float32, q, stream)
    ws_bytes = 0
    if workspace is not None:
        if not workspace.is_contiguous() or workspace.get_device() != dev:
            raise ValueError(f"{fn}: workspace: expected a contiguous tensor on cuda:{dev}")
        ws_bytes = workspace.numel() * workspace.element_size()
    st = _guarded(guard, lib.gqa_decode_paged_int4, q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
                  kv_params.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(), _data(lse), B, Sq,
                  Hq, Hkv, D, page_size, ppr, num_pages, _scale_arg(scale), int(num_splits), _data(workspace),
                  ws_bytes, cs)
    if st:
        raise GQAError(st, fn)
    return out, lse


def gqa_decode_paged_int4_num_splits(B, Sq, Hq, Hkv, D, page_size, pages_per_req) -> int:
    n = load_library().gqa_decode_paged_int4_num_splits(B, Sq, Hq, Hkv, D, page_size, pages_per_req)
    if n < 0:
        raise GQAError(-n, "gqa_decode_paged_int4_num_splits")
    return n


def gqa_decode_paged_int4_workspace_bytes(B, Sq, Hq, Hkv, D, page_size, pages_per_req, num_splits=0) -> int:
    return int(load_library().gqa_decode_paged_int4_workspace_bytes(B, Sq, Hq, Hkv, D, page_size, pages_per_req,
                                                                    int(num_splits)))


def _heads_of(fn: str, t, name: str, T, heads, D, dev):
    """Token stride of t [T, heads, D] bf16 whose heads are contiguous."""
    if t.dtype is not torch.bfloat16 or t.get_device() != dev or t.shape != (T, heads, D):
        raise ValueError(f"{fn}: {name} must be bfloat16 [{T},{heads},{D}] on cuda:{dev}, got {t.dtype} "
                         f"{list(t.shape)} on {t.device}")
    s0, s1, s2 = t.stride()
    if T and (s2 != 1 or (heads > 1 and s1 != D)):
        raise ValueError(f"{fn}: the heads of a token of {name} must be contiguous")
    return s0 if T > 1 else heads * D


def gqa_paged_append(k, v, k_pool, v_pool, page_table, seq_lens, cu_tokens=None, q=None, q_out=None, cos_sin=None,
                     interleaved=False, kv_params=None, k_scale=1.0, v_scale=1.0, k_scales=None, v_scales=None,
                     stream=None):
    """Writes T new tokens' k and v [T,Hkv,D] bf16 into a paged cache, k (and q [T,Hq,D]) rotated on the way.

    The token stride of q, k and v is free (slices of a fused projection).  cu_tokens int32 [B+1]: request b owns rows
    cu_tokens[b] .. cu_tokens[b+1]-1 (None: T / B each); seq_lens int32 [B] counts the new tokens too.  cos_sin fp32
    [max_pos, rot_dim]: cosines, then sines (None: no rotation); interleaved: neighbouring pairs instead of i and
    i + rot_dim / 2.  Pools bf16, uint8 (E4M3FN codes), int8, or uint8 of 4-bit codes with kv_params; 8-bit pools take
    k_scale / v_scale or CUDA fp32 k_scales / v_scales of 1 or Hkv values.
    Returns q_out (bf16 [T,Hq,D], allocated when None) or None without q.
    """
    lib = _lib_handle or load_library()
    fn = "gqa_paged_append"
    dev = k_pool.get_device()
    guard, cs = _on_device_of(dev, stream)
    kvd, num_pages, page_size, Hkv, D, B, ppr, n_scales = _cache(fn, dev, k_pool, v_pool, kv_params, page_table, seq_lens,
                                                                 k_scales, v_scales)
    T = k.shape[0]
    k_stride = _heads_of(fn, k, "k", T, Hkv, D, dev)
    v_stride = _heads_of(fn, v, "v", T, Hkv, D, dev)
    Hq = q_stride = 0
    if q is not None:
        Hq = q.shape[1] if q.dim() == 3 else 0
        q_stride = _heads_of(fn, q, "q", T, Hq, D, dev)
        if q_out is None:
            q_out = _new((T, Hq, D), torch.bfloat16, q, stream)
        else:
            _fit(fn, "q_out", q_out, torch.bfloat16, dev, (T, Hq, D))
    elif q_out is not None:
        raise ValueError(f"{fn}: q_out without q")
    if cu_tokens is not None:
        _fit(fn, "cu_tokens", cu_tokens, torch.int32, dev, (B + 1,))
    rot_dim = max_pos = 0
    if cos_sin is not None:
        _fit(fn, "cos_sin", cos_sin, torch.float32, dev)
        if cos_sin.dim() != 2:
            raise ValueError(f"{fn}: cos_sin must be [max_pos, rot_dim]")
        max_pos, rot_dim = cos_sin.shape
    st = _guarded(guard, lib.gqa_paged_append, _data(q), q_stride, _data(q_out), k.data_ptr(), k_stride, v.data_ptr(),
                  v_stride, kvd, k_pool.data_ptr(), v_pool.data_ptr(), _data(kv_params), k_scale, v_scale,
                  _data(k_scales), _data(v_scales), n_scales, page_table.data_ptr(), seq_lens.data_ptr(),
                  _data(cu_tokens), _data(cos_sin), rot_dim, max_pos, 1 if interleaved else 0, T, B, Hq, Hkv, D,
                  page_size, ppr, num_pages, cs)
    if st:
        raise GQAError(st, fn)
    return q_out


def gqa_paged_gather(k_pool, v_pool, page_table, seq_lens, k_out=None, v_out=None, rows=None, starts=None,
                     kv_params=None, k_scale=1.0, v_scale=1.0, k_scales=None, v_scales=None, stream=None):
    """Tokens starts[b] .. seq_lens[b]-1 of each request of a paged cache, dense: k_out, v_out [B,rows,Hkv,D] bf16.

    Output rows past a request's tokens are left as they were.  k_out and v_out None: allocated with zeros, for which
    rows is needed.  Pools, scales and kv_params as gqa_paged_append; starts int32 [B] (None: 0).
    Returns (k_out, v_out).
    """
    lib = _lib_handle or load_library()
    fn = "gqa_paged_gather"
    dev = k_pool.get_device()
    guard, cs = _on_device_of(dev, stream)
    kvd, num_pages, page_size, Hkv, D, B, ppr, n_scales = _cache(fn, dev, k_pool, v_pool, kv_params, page_table, seq_lens,
                                                                 k_scales, v_scales)
    if (k_out is None) != (v_out is None):
        raise ValueError(f"{fn}: k_out and v_out go together")
    if k_out is None:
        if rows is None:
            raise ValueError(f"{fn}: k_out and v_out, or rows, are needed")
        k_out, v_out = (_new((B, rows, Hkv, D), torch.bfloat16, k_pool, stream, torch.zeros) for _ in range(2))
    else:
        if k_out.dim() != 4 or (rows is not None and rows != k_out.shape[1]):
            raise ValueError(f"{fn}: k_out must be [B,rows,Hkv,D]")
        rows = k_out.shape[1]
        _fit(fn, "k_out", k_out, torch.bfloat16, dev, (B, rows, Hkv, D))
        _fit(fn, "v_out", v_out, torch.bfloat16, dev, (B, rows, Hkv, D))
    if starts is not None:
        _fit(fn, "starts", starts, torch.int32, dev, (B,))
    st = _guarded(guard, lib.gqa_paged_gather, kvd, k_pool.data_ptr(), v_pool.data_ptr(), _data(kv_params), k_scale,
                  v_scale, _data(k_scales), _data(v_scales), n_scales, page_table.data_ptr(), seq_lens.data_ptr(),
                  _data(starts), k_out.data_ptr(), v_out.data_ptr(), B, rows, Hkv, D, page_size, ppr, num_pages, cs)
    if st:
        raise GQAError(st, fn)
    return k_out, v_out


def gqa_paged_gather_fp8(pool, page_table, topk_idx, out=None, stream=None):
    """Test hook: the paged kernel's index map as a byte copy -> uint8 [B, topk, Hkv, D]."""
    lib = load_library()
    _need(pool, "pool", torch.uint8, "cuda")
    _need(page_table, "page_table", torch.int32, "cuda")
    _need(topk_idx, "topk_idx", torch.int32, "cuda")
    num_pages, page_size, Hkv, D = pool.shape
    B, topk = topk_idx.shape
    if out is None:
        out = torch.empty((B, topk, Hkv, D), dtype=torch.uint8, device=pool.device)
    st = lib.gqa_paged_gather_fp8(_ptr(pool), _ptr(page_table), _ptr(topk_idx), _ptr(out), B, Hkv, D,
                                  page_size, page_table.shape[1], num_pages, topk, _stream(stream))
    _check(st, "gqa_paged_gather_fp8")
    return out


def gqa_fp8_e4m3fn_to_f32(codes, out=None, stream=None):
    """Test hook: the paged kernel's E4M3FN widening, as fp32."""
    lib = load_library()
    _need(codes, "codes", torch.uint8, "cuda")
    if out is None:
        out = torch.empty(codes.shape, dtype=torch.float32, device=codes.device)
    st = lib.gqa_fp8_e4m3fn_to_f32(_ptr(codes), _ptr(out), codes.numel(), _stream(stream))
    _check(st, "gqa_fp8_e4m3fn_to_f32")
    return out


# ---------------------------------------------------------------------------
# status and controls
# ---------------------------------------------------------------------------
def gqa_device_status(stream=None) -> int:
    """Waits for the stream; returns and clears the device error status code."""
    return int(load_library().gqa_device_status(_stream(stream)))


def gqa_set_wait_limit_ns(ns: int):
    load_library().gqa_set_wait_limit_ns(int(ns))


def gqa_debug_set_fault_mode(mode: int):
    load_library().gqa_debug_set_fault_mode(int(mode))


def gqa_debug_set_kernel_events(before=None, after=None):
    """Measurement hook: torch.cuda.Event pair recorded around the main kernel
    of later calls (None, None stops it)."""
    lib = load_library()
    if before is None or after is None:
        lib.gqa_debug_set_kernel_events(None, None)
    else:
        lib.gqa_debug_set_kernel_events(ctypes.c_void_p(before.cuda_event), ctypes.c_void_p(after.cuda_event))


def gqa_debug_read_stream(buf, sink, stream=None):
    """Measurement hook: reads every byte of the CUDA tensor `buf` once and
    XORs its words into `sink` (a CUDA int32 tensor of one element)."""
    lib = load_library()
    if not buf.is_cuda or not buf.is_contiguous():
        raise ValueError("buf: expected a contiguous CUDA tensor")
    _need(sink, "sink", torch.int32, "cuda")
    st = lib.gqa_debug_read_stream(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink), _stream(stream))
    _check(st, "gqa_debug_read_stream")


def gqa_status_string(status: int) -> str:
    return load_library().gqa_status_string(int(status)).decode()


def gqa_version() -> str:
    return load_library().gqa_version().decode()
