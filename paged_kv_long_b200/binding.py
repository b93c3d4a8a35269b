"""ctypes binding of ``libpa.so`` — argument marshalling only.

Every step of the attention runs in the library's CUDA kernels; this module checks the
torch tensors it is given (device, dtype, shape, contiguity) and passes their device pointers
and the caller's current CUDA stream across the C ABI declared in ``include/pa.h``. There is
no CPU fallback: if the library is missing or a tensor is not on a CUDA device, it raises.
"""
from __future__ import annotations

import collections
import ctypes
import math
import os

PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(PKG, "libpa.so")

PA_F16, PA_BF16 = 0, 1
POLICIES = {"makespan": 0, "cores": 1, "legacy": 2, "balanced": 3}
PA_POLICY_BALANCED = 3
STATUS = {0: "PA_OK", -1: "PA_ERR_INVALID_ARG", -2: "PA_ERR_UNSUPPORTED", -3: "PA_ERR_WORKSPACE",
          -4: "PA_ERR_CUDA", -5: "PA_ERR_TIMEOUT", -6: "PA_ERR_PAGE_INDEX"}
EXPORTED = ("pa_plan", "pa_prefill", "pa_combine", "pa_prefill_noalloc", "pa_device_error",
            "pa_set_wait_timeout_ns",
            "pa_selftest_timeout", "pa_status_string", "pa_cores_policy_splits",
            "pa_legacy_policy_splits", "pa_schedule_items", "pa_kv_append", "pa_pieces",
            "pa_decode_plan", "pa_decode", "pa_batch_plan", "pa_batch_prefill",
            "pa_batch_combine", "pa_batch_schedule_items", "pa_kv_publish",
            "pa_window_plan", "pa_window_prefill", "pa_window_schedule_items",
            "pa_window_decode_plan", "pa_window_decode", "pa_prefix_decode_plan", "pa_prefix_decode",
            "pa_block_tables", "pa_qk_rope_append")


class PaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


class Plan(ctypes.Structure):
    """Mirror of ``pa_plan_t``."""
    _fields_ = [
        ("num_sms", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("group", ctypes.c_int32),
        ("chunk_rows", ctypes.c_int32), ("q_tiles", ctypes.c_int32), ("splits", ctypes.c_int32),
        ("paged", ctypes.c_int32), ("dtype", ctypes.c_int32), ("policy", ctypes.c_int32),
        ("ctas_per_unit", ctypes.c_int32), ("batch", ctypes.c_int32), ("hist_len", ctypes.c_int64),
        ("units", ctypes.c_int64), ("scale", ctypes.c_float),
        ("est_us", ctypes.c_float), ("ws_bytes", ctypes.c_uint64),
    ]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


_lib = None


def lib_path() -> str:
    return _LIB_PATH


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libpa.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libpa.so not built at {p}: run `python -m paged_kv_long_b200.build`")
    lib = ctypes.CDLL(p)
    vp, i32, i64, u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64
    lib.pa_plan.argtypes = [i32, i32, i32, i32, i32, i32, i64, i32, ctypes.c_float, i32, i32, i32,
                            ctypes.POINTER(Plan)]
    lib.pa_plan.restype = i32
    lib.pa_prefill.argtypes = [ctypes.POINTER(Plan), vp, vp, vp, vp, i64, i64, i32, vp, vp, u64, vp]
    lib.pa_prefill.restype = i32
    lib.pa_combine.argtypes = [ctypes.POINTER(Plan), vp, u64, vp, vp]
    lib.pa_combine.restype = i32
    lib.pa_prefill_noalloc.argtypes = [ctypes.POINTER(Plan), vp, vp, vp, vp, i64, i64, i32, vp, vp]
    lib.pa_prefill_noalloc.restype = i32
    lib.pa_device_error.argtypes = [ctypes.POINTER(ctypes.c_int), i32]
    lib.pa_device_error.restype = i32
    lib.pa_set_wait_timeout_ns.argtypes = [u64]
    lib.pa_set_wait_timeout_ns.restype = None
    lib.pa_selftest_timeout.argtypes = [u64, vp]
    lib.pa_selftest_timeout.restype = i32
    lib.pa_status_string.argtypes = [i32]
    lib.pa_status_string.restype = ctypes.c_char_p
    lib.pa_cores_policy_splits.argtypes = [i32, i32, i32]
    lib.pa_cores_policy_splits.restype = i32
    lib.pa_legacy_policy_splits.argtypes = [i32, i32]
    lib.pa_legacy_policy_splits.restype = i32
    lib.pa_schedule_items.argtypes = [ctypes.POINTER(Plan), ctypes.POINTER(ctypes.c_int32), i32]
    lib.pa_schedule_items.restype = i32
    lib.pa_kv_append.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp, i64, i64, i32, vp]
    lib.pa_kv_append.restype = i32
    lib.pa_pieces.argtypes = [i32, i64, i32, ctypes.POINTER(ctypes.c_int32), i32]
    lib.pa_pieces.restype = i32
    lib.pa_decode_plan.argtypes = [i32, i32, i32, i32, i32, i32, i64, i32, ctypes.c_float, i32,
                                   ctypes.POINTER(Plan)]
    lib.pa_decode_plan.restype = i32
    lib.pa_decode.argtypes = [ctypes.POINTER(Plan), vp, vp, vp, vp, i32, vp, i64, vp, vp, u64, vp]
    lib.pa_decode.restype = i32
    lib.pa_batch_plan.argtypes = [i32, i32, i32, i32, i32, i32, vp, vp, i32, ctypes.c_float,
                                  ctypes.POINTER(Plan)]
    lib.pa_batch_plan.restype = i32
    lib.pa_batch_prefill.argtypes = [ctypes.POINTER(Plan), vp, vp, vp, vp, vp, vp, i32, i64, vp,
                                     vp, u64, vp]
    lib.pa_batch_prefill.restype = i32
    lib.pa_batch_combine.argtypes = [ctypes.POINTER(Plan), vp, vp, vp, u64, vp, vp]
    lib.pa_batch_combine.restype = i32
    lib.pa_batch_schedule_items.argtypes = [ctypes.POINTER(Plan), vp, vp,
                                            ctypes.POINTER(ctypes.c_int32), i32]
    lib.pa_batch_schedule_items.restype = i32
    lib.pa_kv_publish.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp, i64, i64, i32, vp]
    lib.pa_kv_publish.restype = i32
    lib.pa_window_plan.argtypes = [i32, i32, i32, i32, i32, i32, vp, vp, i32, i32, i32,
                                   ctypes.c_float, ctypes.POINTER(Plan)]
    lib.pa_window_plan.restype = i32
    lib.pa_window_prefill.argtypes = [ctypes.POINTER(Plan), vp, vp, i32, i32, vp, vp, vp, vp, i32,
                                      i64, vp, vp, u64, vp]
    lib.pa_window_prefill.restype = i32
    lib.pa_window_schedule_items.argtypes = [ctypes.POINTER(Plan), vp, vp, i32, i32,
                                             ctypes.POINTER(ctypes.c_int32), i32]
    lib.pa_window_schedule_items.restype = i32
    lib.pa_window_decode_plan.argtypes = [i32, i32, i32, i32, i32, i32, i64, i32, i32, i32,
                                          ctypes.c_float, ctypes.POINTER(Plan)]
    lib.pa_window_decode_plan.restype = i32
    lib.pa_window_decode.argtypes = [ctypes.POINTER(Plan), i32, i32, vp, vp, vp, vp, i32, vp, i64,
                                     vp, vp, u64, vp]
    lib.pa_window_decode.restype = i32
    lib.pa_prefix_decode_plan.argtypes = [i32, i32, i32, i32, i32, i32, i64, i64, i32,
                                          ctypes.c_float, ctypes.POINTER(Plan)]
    lib.pa_prefix_decode_plan.restype = i32
    lib.pa_prefix_decode.argtypes = [ctypes.POINTER(Plan), i64, vp, vp, vp, vp, vp, i32, vp, i64,
                                     vp, vp, u64, vp]
    lib.pa_prefix_decode.restype = i32
    lib.pa_block_tables.argtypes = [i32, vp, vp, i32, i64, vp, i32, vp, vp, vp, i32, i32, vp, vp,
                                    vp, vp, vp]
    lib.pa_block_tables.restype = i32
    lib.pa_qk_rope_append.argtypes = [i32, i32, i32, i32, i32, i32, vp, i64, vp, i64, vp, i64, vp,
                                      vp, vp, i32, i64, i32, vp, vp, i32, ctypes.c_float, vp, vp,
                                      vp, i64, vp]
    lib.pa_qk_rope_append.restype = i32
    if path is None:
        _lib = lib
    return lib


def _check(status: int, where: str):
    if status != 0:
        raise PaError(status, where)


def _dtype_code(dtype) -> int:
    import torch
    if dtype in ("f16", torch.float16):
        return PA_F16
    if dtype in ("bf16", torch.bfloat16):
        return PA_BF16
    raise ValueError(f"unsupported dtype {dtype}")


def plan(n_q_heads: int, n_kv_heads: int, head_dim: int, page_size: int, chunk_rows: int,
         hist_len: int, dtype="bf16", scale: float = 0.0, splits: int = 0,
         policy: str = "makespan", paged: bool = True, num_sms: int | None = None) -> Plan:
    """pa_plan: split count and workspace for one piece (host only)."""
    if num_sms is None:
        import torch
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    p = Plan()
    st = load_library().pa_plan(num_sms, n_q_heads, n_kv_heads, head_dim, page_size, chunk_rows,
                                hist_len, _dtype_code(dtype), scale, splits, POLICIES[policy],
                                1 if paged else 0, ctypes.byref(p))
    _check(st, "pa_plan")
    return p


def schedule_items(p: Plan):
    """pa_schedule_items: the work items of a balanced plan as an int32 array [n, 4] of
    (row block, kt0, kt1, workspace slot or -1); empty for other plans."""
    import numpy as np
    lib = load_library()
    n = lib.pa_schedule_items(ctypes.byref(p), None, 0)
    _check(0 if n >= 0 else n, "pa_schedule_items")
    buf = (ctypes.c_int32 * max(4 * n, 1))()
    lib.pa_schedule_items(ctypes.byref(p), buf, n)
    return np.frombuffer(buf, dtype=np.int32)[:4 * n].reshape(n, 4).copy()


def pieces(chunk_rows: int, hist_len: int, log2_budget: int = 25) -> list[int]:
    """pa_pieces: the pages' cut of a chunk into pieces (rows of each, in order)."""
    lib = load_library()
    n = lib.pa_pieces(chunk_rows, hist_len, log2_budget, None, 0)
    _check(0 if n >= 0 else n, "pa_pieces")
    buf = (ctypes.c_int32 * max(n, 1))()
    lib.pa_pieces(chunk_rows, hist_len, log2_budget, buf, n)
    return list(buf)[:n]


def kv_append(k_new, v_new, k_pool, v_pool, page_table, hist_len: int, stream=None):
    """pa_kv_append: write the chunk's K/V rows [R, Hkv, D] into the page pools
    [num_pages, PS, Hkv, D] at positions hist_len.. through page_table (see include/pa.h)."""
    import torch
    if k_new.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("k_new must be float16 or bfloat16")
    dt = k_new.dtype
    device = _device_of(k_new, "k_new")
    _require(k_new, "k_new", dt, None, device)
    if k_new.dim() != 3:
        raise ValueError("k_new must be [R, Hkv, D]")
    R, Hkv, D = k_new.shape
    _require(v_new, "v_new", dt, (R, Hkv, D), device)
    _require(k_pool, "k_pool", dt, None, device)
    if k_pool.dim() != 4 or tuple(k_pool.shape[2:]) != (Hkv, D):
        raise ValueError("k_pool must be [num_pages, page_size, Hkv, D]")
    _require(v_pool, "v_pool", dt, tuple(k_pool.shape), device)
    _require(page_table, "page_table", torch.int32, None, device)
    PS = k_pool.shape[1]
    if page_table.numel() < math.ceil((hist_len + R) / PS):
        raise ValueError("page_table is shorter than ceil((hist_len+R)/page_size)")
    _call(device, stream, load_library().pa_kv_append, "pa_kv_append", Hkv, D, PS,
          _dtype_code(dt), k_new.data_ptr(), v_new.data_ptr(), k_pool.data_ptr(),
          v_pool.data_ptr(), page_table.data_ptr(), k_pool.shape[0], hist_len, R)


def kv_publish(k_staged, v_staged, k_pool, v_pool, page_table, first_pos: int, rows: int,
               stream=None):
    """pa_kv_publish: copy staged rows [first_pos, first_pos + rows) of the contiguous staging
    buffers [T, Hkv, D] to their pages (see include/pa.h)."""
    import torch
    if k_staged.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("k_staged must be float16 or bfloat16")
    dt = k_staged.dtype
    device = _device_of(k_staged, "k_staged")
    _require(k_staged, "k_staged", dt, None, device)
    if k_staged.dim() != 3:
        raise ValueError("k_staged must be [T, Hkv, D]")
    T, Hkv, D = k_staged.shape
    if first_pos < 0 or rows < 0 or first_pos + rows > T:
        raise ValueError("rows [first_pos, first_pos + rows) must lie in the staging buffer")
    _require(v_staged, "v_staged", dt, (T, Hkv, D), device)
    _require(k_pool, "k_pool", dt, None, device)
    if k_pool.dim() != 4 or tuple(k_pool.shape[2:]) != (Hkv, D):
        raise ValueError("k_pool must be [num_pages, page_size, Hkv, D]")
    _require(v_pool, "v_pool", dt, tuple(k_pool.shape), device)
    _require(page_table, "page_table", torch.int32, None, device)
    PS = k_pool.shape[1]
    if page_table.numel() < math.ceil((first_pos + rows) / PS):
        raise ValueError("page_table is shorter than ceil((first_pos+rows)/page_size)")
    _call(device, stream, load_library().pa_kv_publish, "pa_kv_publish", Hkv, D, PS,
          _dtype_code(dt), k_staged.data_ptr(), v_staged.data_ptr(), k_pool.data_ptr(),
          v_pool.data_ptr(), page_table.data_ptr(), k_pool.shape[0], first_pos, rows)


def _stream_ptr(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _require_cuda(t, name, dtype=None, shape=None):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _torch_dtype(p: Plan):
    import torch
    return torch.bfloat16 if p.dtype == PA_BF16 else torch.float16


def workspace(p: Plan, device=None):
    """A workspace tensor of plan.ws_bytes (fp32), or None when no split is used."""
    import torch
    if p.ws_bytes == 0:
        return None
    return torch.empty(p.ws_bytes // 4, dtype=torch.float32, device=device or "cuda")


def prefill(p: Plan, q, k_pool, v_pool, page_table, out, ws=None, stream=None):
    """pa_prefill on torch tensors (see include/pa.h for layouts)."""
    import torch
    dt = _torch_dtype(p)
    R, Hq, Hkv, D = p.chunk_rows, p.n_q_heads, p.n_kv_heads, p.head_dim
    device = _device_of(q, "q")
    _require(q, "q", dt, (R, Hq, D), device)
    _require(k_pool, "k_pool", dt, None, device)
    _require(v_pool, "v_pool", dt, tuple(k_pool.shape), device)
    if p.paged:
        if k_pool.dim() != 4 or tuple(k_pool.shape[1:]) != (p.page_size, Hkv, D):
            raise ValueError("k_pool must be [num_pages, page_size, Hkv, D]")
        _require(page_table, "page_table", torch.int32, None, device)
        if page_table.numel() < math.ceil((p.hist_len + R) / p.page_size):
            raise ValueError("page_table is shorter than ceil((H+R)/page_size)")
        num_pages, tab = k_pool.shape[0], page_table.data_ptr()
    else:
        if k_pool.dim() != 3 or tuple(k_pool.shape) != (p.hist_len + R, Hkv, D):
            raise ValueError("contiguous k/v must be [H+R, Hkv, D]")
        num_pages, tab = 0, None
    out_ptr, ws_ptr, ws_bytes = None, None, 0
    if p.splits == 1 or p.policy == PA_POLICY_BALANCED:
        _require(out, "out", torch.float32, (R, Hq, D), device)
        out_ptr = out.data_ptr()
    if p.ws_bytes > 0:
        _require(ws, "ws", torch.float32, None, device)
        ws_ptr, ws_bytes = ws.data_ptr(), ws.numel() * 4
    _call(device, stream, load_library().pa_prefill, "pa_prefill", ctypes.byref(p), q.data_ptr(),
          k_pool.data_ptr(), v_pool.data_ptr(), tab, num_pages, p.hist_len, R, out_ptr, ws_ptr,
          ws_bytes)


def combine(p: Plan, ws, out, stream=None):
    """pa_combine: merge split partials into out (no-op when there are none)."""
    import torch
    if p.ws_bytes == 0:
        return
    device = _device_of(ws, "ws")
    _require(ws, "ws", torch.float32, None, device)
    _require(out, "out", torch.float32, (p.chunk_rows, p.n_q_heads, p.head_dim), device)
    _call(device, stream, load_library().pa_combine, "pa_combine", ctypes.byref(p),
          ws.data_ptr(), ws.numel() * 4, out.data_ptr())


def prefill_combine(p: Plan, q, k_pool, v_pool, page_table, out=None, ws=None, stream=None):
    """pa_prefill followed by pa_combine; allocates out / ws with torch when not given."""
    import torch
    if out is None:
        out = _handed_back(stream, _device_of(q, "q"),
                           _new(stream, torch.empty, (p.chunk_rows, p.n_q_heads, p.head_dim),
                                dtype=torch.float32, device=q.device))
    if p.ws_bytes > 0 and ws is None:
        ws = _new(stream, workspace, p, q.device)
    prefill(p, q, k_pool, v_pool, page_table, out, ws, stream)
    combine(p, ws, out, stream)
    return out


def prefill_noalloc(p: Plan, q, k_pool, v_pool, page_table, out, stream=None):
    """pa_prefill_noalloc: prefill + combine with the library's own device scratch (for
    callers that cannot allocate device memory; see include/pa.h)."""
    import torch
    dt = _torch_dtype(p)
    R, Hq, D = p.chunk_rows, p.n_q_heads, p.head_dim
    device = _device_of(q, "q")
    _require(q, "q", dt, (R, Hq, D), device)
    _require(k_pool, "k_pool", dt, None, device)
    _require(v_pool, "v_pool", dt, tuple(k_pool.shape), device)
    _require(out, "out", torch.float32, (R, Hq, D), device)
    if p.paged:
        _require(page_table, "page_table", torch.int32, None, device)
        num_pages, tab = k_pool.shape[0], page_table.data_ptr()
    else:
        num_pages, tab = 0, None
    _call(device, stream, load_library().pa_prefill_noalloc, "pa_prefill_noalloc",
          ctypes.byref(p), q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), tab, num_pages,
          p.hist_len, R, out.data_ptr())


def decode_plan(n_q_heads: int, n_kv_heads: int, head_dim: int, page_size: int, batch: int,
                max_seq_len: int, dtype="bf16", scale: float = 0.0, splits: int = 0,
                num_sms: int | None = None) -> Plan:
    """pa_decode_plan: split count and workspace for one batched decode step (host only)."""
    if num_sms is None:
        import torch
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    p = Plan()
    st = load_library().pa_decode_plan(num_sms, n_q_heads, n_kv_heads, head_dim, page_size, batch,
                                       max_seq_len, _dtype_code(dtype), scale, splits,
                                       ctypes.byref(p))
    _check(st, "pa_decode_plan")
    return p


def decode(p: Plan, q, k_pool, v_pool, block_table, seq_lens, out=None, ws=None, stream=None):
    """pa_decode followed by pa_combine: one query token per sequence against that sequence's
    paged keys. q [B, Hq, D]; block_table int32 [B, max_pages]; seq_lens int32 [B] (keys of
    each sequence, the new token's included). Returns out fp32 [B, Hq, D]."""
    import torch
    dt = _torch_dtype(p)
    B, Hq, Hkv, D, PS = p.batch, p.n_q_heads, p.n_kv_heads, p.head_dim, p.page_size
    device = _device_of(q, "q")
    _require(q, "q", dt, (B, Hq, D), device)
    _require(k_pool, "k_pool", dt, None, device)
    _require(v_pool, "v_pool", dt, tuple(k_pool.shape), device)
    if k_pool.dim() != 4 or tuple(k_pool.shape[1:]) != (PS, Hkv, D):
        raise ValueError("k_pool must be [num_pages, page_size, Hkv, D]")
    _require(block_table, "block_table", torch.int32, None, device)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [batch, max_pages]")
    _require(seq_lens, "seq_lens", torch.int32, (B,), device)
    if out is None:
        out = _handed_back(stream, device, _new(stream, torch.empty, (B, Hq, D),
                                                dtype=torch.float32, device=q.device))
    _require(out, "out", torch.float32, (B, Hq, D), device)
    ws_ptr, ws_bytes = None, 0
    if p.ws_bytes > 0:
        if ws is None:
            ws = _new(stream, workspace, p, q.device)
        _require(ws, "ws", torch.float32, None, device)
        ws_ptr, ws_bytes = ws.data_ptr(), ws.numel() * 4
    lib = load_library()
    _call(device, stream, lib.pa_decode, "pa_decode", ctypes.byref(p), q.data_ptr(),
          k_pool.data_ptr(), v_pool.data_ptr(), block_table.data_ptr(), block_table.stride(0),
          seq_lens.data_ptr(), k_pool.shape[0], out.data_ptr(), ws_ptr, ws_bytes)
    if p.ws_bytes > 0:
        _call(device, stream, lib.pa_combine, "pa_combine", ctypes.byref(p), ws_ptr, ws_bytes,
              out.data_ptr())
    return out


class BatchPlan:
    """A batched plan with the host length arrays it was made from (pa_batch_plan)."""

    def __init__(self, plan: Plan, q_lens, hist_lens):
        import numpy as np
        self.plan = plan
        self.q_lens = np.array(q_lens, dtype=np.int32)  # copies: the plan's own
        self.hist_lens = np.array(hist_lens, dtype=np.int64)

    def _arrays(self):
        return self.q_lens.ctypes.data, self.hist_lens.ctypes.data


def batch_plan(n_q_heads: int, n_kv_heads: int, head_dim: int, page_size: int, q_lens,
               hist_lens, dtype="bf16", scale: float = 0.0,
               num_sms: int | None = None) -> BatchPlan:
    """pa_batch_plan: the balanced schedule of a batch of chunks (host only)."""
    import numpy as np
    if num_sms is None:
        import torch
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    q_lens = np.ascontiguousarray(q_lens, dtype=np.int32)
    hist_lens = np.ascontiguousarray(hist_lens, dtype=np.int64)
    if q_lens.shape != hist_lens.shape or q_lens.ndim != 1:
        raise ValueError("q_lens and hist_lens must be 1-D of the same length")
    p = Plan()
    st = load_library().pa_batch_plan(num_sms, n_q_heads, n_kv_heads, head_dim, page_size,
                                      len(q_lens), q_lens.ctypes.data, hist_lens.ctypes.data,
                                      _dtype_code(dtype), scale, ctypes.byref(p))
    _check(st, "pa_batch_plan")
    return BatchPlan(p, q_lens, hist_lens)


def batch_schedule_items(bp: BatchPlan):
    """pa_batch_schedule_items: int32 [n, 4] of (global row block, kt0, kt1, slot or -1)."""
    import numpy as np
    lib = load_library()
    ql, hl = bp._arrays()
    n = lib.pa_batch_schedule_items(ctypes.byref(bp.plan), ql, hl, None, 0)
    if n < 0:
        raise PaError(n, "pa_batch_schedule_items")
    out = np.zeros((max(n, 1), 4), dtype=np.int32)
    lib.pa_batch_schedule_items(ctypes.byref(bp.plan), ql, hl,
                                out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), n)
    return out[:n]


def batch_prefill(bp: BatchPlan, q, k_pool, v_pool, block_table, out=None, ws=None,
                  stream=None):
    """pa_batch_prefill followed by pa_batch_combine. q [sum q_lens, Hq, D] (the sequences'
    chunks packed in order); block_table int32 [batch, max_pages]. Returns out fp32
    [sum q_lens, Hq, D]."""
    import torch
    p = bp.plan
    dt = _torch_dtype(p)
    rows, Hq, Hkv, D, PS = p.chunk_rows, p.n_q_heads, p.n_kv_heads, p.head_dim, p.page_size
    device = _device_of(q, "q")
    _require(q, "q", dt, (rows, Hq, D), device)
    _require(k_pool, "k_pool", dt, None, device)
    _require(v_pool, "v_pool", dt, tuple(k_pool.shape), device)
    if k_pool.dim() != 4 or tuple(k_pool.shape[1:]) != (PS, Hkv, D):
        raise ValueError("k_pool must be [num_pages, page_size, Hkv, D]")
    _require(block_table, "block_table", torch.int32, None, device)
    if block_table.dim() != 2 or block_table.shape[0] != p.batch:
        raise ValueError("block_table must be [batch, max_pages]")
    if out is None:
        out = _handed_back(stream, device, _new(stream, torch.empty, (rows, Hq, D),
                                                dtype=torch.float32, device=q.device))
    _require(out, "out", torch.float32, (rows, Hq, D), device)
    ws_ptr, ws_bytes = None, 0
    if p.ws_bytes > 0:
        if ws is None:
            ws = _new(stream, workspace, p, q.device)
        _require(ws, "ws", torch.float32, None, device)
        ws_ptr, ws_bytes = ws.data_ptr(), ws.numel() * 4
    ql, hl = bp._arrays()
    lib = load_library()
    _call(device, stream, lib.pa_batch_prefill, "pa_batch_prefill", ctypes.byref(p), ql, hl,
          q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), block_table.data_ptr(),
          block_table.stride(0), k_pool.shape[0], out.data_ptr(), ws_ptr, ws_bytes)
    _call(device, stream, lib.pa_batch_combine, "pa_batch_combine", ctypes.byref(p), ql, hl, ws_ptr,
          ws_bytes, out.data_ptr())
    return out


class _StepPlan:
    """A plan whose fields the calls of every step and layer need, read out of it once."""

    def __init__(self, plan: Plan):
        self.plan = plan
        self.ref = ctypes.byref(plan)
        self.torch_dtype = _torch_dtype(plan)
        self.q_shape = (plan.chunk_rows, plan.n_q_heads, plan.head_dim)
        self.page_shape = (plan.page_size, plan.n_kv_heads, plan.head_dim)
        self.batch = plan.batch
        self.ws_numel = plan.ws_bytes // 4


class WindowPlan(_StepPlan):
    """A plan with its window and sinks (pa_window_plan with the host length arrays it was made
    from, or pa_window_decode_plan without)."""

    def __init__(self, plan: Plan, window: int, n_sinks: int, q_lens=None, hist_lens=None):
        super().__init__(plan)
        self.window = window
        self.n_sinks = n_sinks
        self.q_lens = q_lens
        self.hist_lens = hist_lens
        if q_lens is not None:
            self.lens_ptrs = (q_lens.ctypes.data, hist_lens.ctypes.data)


def _num_sms(device=None) -> int:
    """SMs of a device, the current one if none is given."""
    import torch
    return torch.cuda.get_device_properties(torch.cuda.current_device() if device is None
                                            else device).multi_processor_count


def _window_args(window, n_sinks):
    """window and n_sinks as the 32-bit C arguments (a larger window sees every key anyway)."""
    window, n_sinks = int(window), int(n_sinks)
    if window < 1 or n_sinks < 0:
        raise ValueError("window must be >= 1 and n_sinks >= 0")
    return min(window, 2**31 - 1), min(n_sinks, 2**31 - 1)


def window_plan(n_q_heads: int, n_kv_heads: int, head_dim: int, page_size: int, q_lens, hist_lens,
                window: int, n_sinks: int = 0, dtype="bf16", scale: float = 0.0,
                num_sms: int | None = None) -> WindowPlan:
    """pa_window_plan: the schedule of a batch of chunks under a sliding window with sinks (host
    only; one sequence is a batch of one)."""
    import numpy as np
    window, n_sinks = _window_args(window, n_sinks)
    q_lens = np.array(q_lens, dtype=np.int32)  # copies: the plan's own
    hist_lens = np.array(hist_lens, dtype=np.int64)
    if q_lens.shape != hist_lens.shape or q_lens.ndim != 1:
        raise ValueError("q_lens and hist_lens must be 1-D of the same length")
    p = Plan()
    st = load_library().pa_window_plan(_num_sms() if num_sms is None else num_sms, n_q_heads,
                                       n_kv_heads, head_dim, page_size, len(q_lens),
                                       q_lens.ctypes.data, hist_lens.ctypes.data, window, n_sinks,
                                       _dtype_code(dtype), scale, ctypes.byref(p))
    _check(st, "pa_window_plan")
    return WindowPlan(p, window, n_sinks, q_lens, hist_lens)


def window_schedule_items(wp: WindowPlan):
    """pa_window_schedule_items: int32 [n, 4] of (global row block, kt0, kt1, slot or -1), kt0 and
    kt1 along the row block's visible KV tiles."""
    import numpy as np
    if wp.q_lens is None:
        raise ValueError("a decode plan has no items")
    args = (ctypes.byref(wp.plan), wp.q_lens.ctypes.data, wp.hist_lens.ctypes.data, wp.window,
            wp.n_sinks)
    n = load_library().pa_window_schedule_items(*args, None, 0)
    if n < 0:
        raise PaError(n, "pa_window_schedule_items")
    out = np.zeros((max(n, 1), 4), dtype=np.int32)
    load_library().pa_window_schedule_items(
        *args, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), n)
    return out[:n]


def window_decode_plan(n_q_heads: int, n_kv_heads: int, head_dim: int, page_size: int, batch: int,
                       max_seq_len: int, window: int, n_sinks: int = 0, dtype="bf16",
                       scale: float = 0.0, num_sms: int | None = None) -> WindowPlan:
    """pa_window_decode_plan: launch and workspace of a decode step under a sliding window with
    sinks (host only)."""
    window, n_sinks = _window_args(window, n_sinks)
    p = Plan()
    st = load_library().pa_window_decode_plan(_num_sms() if num_sms is None else num_sms,
                                              n_q_heads, n_kv_heads, head_dim, page_size, batch,
                                              max_seq_len, window, n_sinks, _dtype_code(dtype),
                                              scale, ctypes.byref(p))
    _check(st, "pa_window_decode_plan")
    return WindowPlan(p, window, n_sinks)


# The calls below run once a layer and step, so their own cost counts: at a decode step's sizes
# the kernels of block_tables and qk_rope_append take 2-7 microseconds, the calls 13-15. A tensor's checks are four attribute reads (the messages come
# from _require_cuda, on failure only), and the stream is read without building a Stream object.


def _require(t, name, dtype, shape, device):
    """t is a contiguous CUDA tensor of this dtype, shape (None: any) and device index."""
    try:
        if (t.dtype is dtype and t.get_device() == device and t.is_contiguous()
                and (shape is None or t.shape == shape)):
            return
    except AttributeError:
        pass
    _require_cuda(t, name, dtype, shape)
    raise ValueError(f"{name} is on cuda:{t.get_device()}, not on cuda:{device}: one device is "
                     "needed")


def _device_of(t, name) -> int:
    """Index of the CUDA device that t (and so the call) is on."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _call(device: int, stream, fn, name, *args):
    """fn(*args, stream) with `device` current, on its current stream unless one is given."""
    import torch
    ptr = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
    if device == torch._C._cuda_getDevice():
        st = fn(*args, ptr)
    else:
        with torch.cuda.device(device):
            st = fn(*args, ptr)
    if st != 0:
        raise PaError(st, name)


def _new(stream, make, *args, **kw):
    """make(*args, **kw): a tensor that this call's kernels write. It comes from the memory of the
    stream that they run on: a block that the current stream has just freed may still be in use by
    that stream's pending work, which `stream` does not wait for."""
    import torch
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _handed_back(stream, device: int, t):
    """A tensor of _new that the caller gets, most likely to use it on the current stream: once
    freed, its memory waits for that stream's work too."""
    import torch
    if stream is not None:
        current = torch.cuda.current_stream(device)
        if current != stream:
            t.record_stream(current)
    return t


def _step_tensors(sp: _StepPlan, q, k_pool, v_pool, block_table, out, ws, stream, device):
    """Checks of the tensors that the window and prefix calls take; (out, ws, its pointer, its
    bytes)."""
    import torch
    dt = sp.torch_dtype
    _require(q, "q", dt, sp.q_shape, device)
    _require(k_pool, "k_pool", dt, None, device)
    pool = k_pool.shape
    if len(pool) != 4 or pool[1:] != sp.page_shape:
        raise ValueError("k_pool must be [num_pages, page_size, Hkv, D]")
    _require(v_pool, "v_pool", dt, pool, device)
    _require(block_table, "block_table", torch.int32, None, device)
    if block_table.dim() != 2 or block_table.shape[0] != sp.batch:
        raise ValueError("block_table must be [batch, max_pages]")
    if out is None:
        out = _handed_back(stream, device, _new(stream, torch.empty_like, q))
    else:
        _require(out, "out", dt, sp.q_shape, device)
    if sp.ws_numel == 0:
        return out, None, None, 0
    if ws is None:
        ws = _new(stream, torch.empty, sp.ws_numel, dtype=torch.float32, device=q.device)
        return out, ws, ws.data_ptr(), 4 * sp.ws_numel
    _require(ws, "ws", torch.float32, None, device)
    return out, ws, ws.data_ptr(), 4 * ws.numel()


def window_decode(wp: WindowPlan, q, k_pool, v_pool, block_table, seq_lens, out=None, ws=None,
                  stream=None):
    """pa_window_decode: one query token per sequence against the last `window` keys and the first
    `n_sinks` of that sequence (see include/pa.h). q [B, Hq, D]; block_table int32
    [B, max_pages]; seq_lens int32 [B]. Returns out [B, Hq, D] of q's type."""
    import torch
    if wp.q_lens is not None:
        raise ValueError("a plan of window_plan runs with window_prefill")
    device = _device_of(q, "q")
    _require(seq_lens, "seq_lens", torch.int32, (wp.batch,), device)
    out, ws, ws_ptr, ws_bytes = _step_tensors(wp, q, k_pool, v_pool, block_table, out, ws, stream,
                                              device)
    _call(device, stream, load_library().pa_window_decode, "pa_window_decode", wp.ref, wp.window,
          wp.n_sinks, q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), block_table.data_ptr(),
          block_table.shape[1], seq_lens.data_ptr(), k_pool.shape[0], out.data_ptr(), ws_ptr,
          ws_bytes)
    return out


def window_prefill(wp: WindowPlan, q, k_pool, v_pool, block_table, out=None, ws=None, stream=None):
    """pa_window_prefill: the chunks of a batch under the plan's sliding window and sinks (see
    include/pa.h). q [sum q_lens, Hq, D] packed in order; block_table int32 [batch, max_pages].
    Returns out [sum q_lens, Hq, D] of q's type."""
    if wp.q_lens is None:
        raise ValueError("a plan of window_decode_plan runs with window_decode")
    device = _device_of(q, "q")
    out, ws, ws_ptr, ws_bytes = _step_tensors(wp, q, k_pool, v_pool, block_table, out, ws, stream,
                                              device)
    _call(device, stream, load_library().pa_window_prefill, "pa_window_prefill", wp.ref,
          *wp.lens_ptrs, wp.window, wp.n_sinks, q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
          block_table.data_ptr(), block_table.shape[1], k_pool.shape[0], out.data_ptr(), ws_ptr,
          ws_bytes)
    return out


class PrefixPlan(_StepPlan):
    """A plan of pa_prefix_decode_plan with its prefix length."""

    def __init__(self, plan: Plan, prefix_len: int):
        super().__init__(plan)
        self.prefix_len = prefix_len


def prefix_decode_plan(n_q_heads: int, n_kv_heads: int, head_dim: int, page_size: int, batch: int,
                       prefix_len: int, max_seq_len: int, dtype="bf16", scale: float = 0.0,
                       num_sms: int | None = None) -> PrefixPlan:
    """pa_prefix_decode_plan: launch and workspace of a decode step over a shared prefix (host
    only)."""
    p = Plan()
    st = load_library().pa_prefix_decode_plan(_num_sms() if num_sms is None else num_sms,
                                              n_q_heads, n_kv_heads, head_dim, page_size, batch,
                                              prefix_len, max_seq_len,
                                              _dtype_code(dtype), scale, ctypes.byref(p))
    _check(st, "pa_prefix_decode_plan")
    return PrefixPlan(p, prefix_len)


def prefix_decode(pp: PrefixPlan, q, k_pool, v_pool, prefix_table, block_table, seq_lens, out=None,
                  ws=None, stream=None):
    """pa_prefix_decode: one query token per sequence, the first prefix_len keys shared by all and
    computed once (see include/pa.h). q [B, Hq, D]; prefix_table int32 [prefix_len / PS];
    block_table int32 [B, max_pages] and seq_lens int32 [B] of whole sequences. Returns out
    [B, Hq, D] of q's type."""
    import torch
    device = _device_of(q, "q")
    _require(prefix_table, "prefix_table", torch.int32, (pp.prefix_len // pp.page_shape[0],),
             device)
    _require(seq_lens, "seq_lens", torch.int32, (pp.batch,), device)
    out, ws, ws_ptr, ws_bytes = _step_tensors(pp, q, k_pool, v_pool, block_table, out, ws, stream,
                                              device)
    _call(device, stream, load_library().pa_prefix_decode, "pa_prefix_decode", pp.ref,
          pp.prefix_len, q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
          prefix_table.data_ptr(), block_table.data_ptr(), block_table.shape[1],
          seq_lens.data_ptr(), k_pool.shape[0], out.data_ptr(), ws_ptr, ws_bytes)
    return out


StepTables = collections.namedtuple("StepTables",
                                    "slots positions cu_q_lens seq_lens pages_used")


def block_tables(q_lens, hist_lens, free_pages, pages_used, block_table, max_rows: int,
                 page_size: int, num_pages: int, out: StepTables | None = None,
                 stream=None) -> StepTables:
    """pa_block_tables: the step's pages taken from the free list into block_table (in place),
    and every new row's pool slot and position (see include/pa.h). q_lens, hist_lens int32 [B];
    free_pages int32 [F]; pages_used int32 [1]; block_table int32 [B, max_pages]. Returns
    StepTables(slots [max_rows], positions [max_rows], cu_q_lens [B + 1], seq_lens [B],
    pages_used [1]), in the tensors of `out` when given (its pages_used not the input's)."""
    import torch
    i32 = torch.int32
    device = _device_of(q_lens, "q_lens")
    _require(q_lens, "q_lens", i32, None, device)
    if q_lens.dim() != 1:
        raise ValueError("q_lens must be [batch]")
    B = q_lens.shape[0]
    _require(hist_lens, "hist_lens", i32, (B,), device)
    _require(free_pages, "free_pages", i32, None, device)
    if free_pages.dim() != 1:
        raise ValueError("free_pages must be 1-D")
    _require(pages_used, "pages_used", i32, (1,), device)
    _require(block_table, "block_table", i32, None, device)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [batch, max_pages]")
    sizes = (max_rows, max_rows, B + 1, B, 1)
    if out is None:  # one allocation for all five
        buf = _handed_back(stream, device, _new(stream, q_lens.new_empty,
                                                2 * max_rows + 2 * B + 2))
        # integer parts have no gradient to track as views: this split takes 1 us less
        out = StepTables._make(torch.unsafe_split_with_sizes(buf, sizes))
    else:
        out = StepTables._make(out)
        for t, name, n in zip(out, StepTables._fields, sizes):
            _require(t, name, i32, (n,), device)
    _call(device, stream, load_library().pa_block_tables, "pa_block_tables", B, q_lens.data_ptr(),
          hist_lens.data_ptr(), page_size, num_pages, free_pages.data_ptr(), free_pages.shape[0],
          pages_used.data_ptr(), out.pages_used.data_ptr(), block_table.data_ptr(),
          block_table.shape[1], max_rows, out.slots.data_ptr(), out.positions.data_ptr(),
          out.cu_q_lens.data_ptr(), out.seq_lens.data_ptr())
    return out


def rope_table(max_pos: int, rot_dim: int, theta: float = 10000.0, device="cuda"):
    """The rotation table that qk_rope_append reads: fp32 [max_pos, rot_dim], row p the cosines
    and then the sines of p * theta^(-2i / rot_dim), i < rot_dim / 2, from angles in 64 bits."""
    import torch
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] \
        * float(theta) ** (-i / rot_dim)
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def _require_rows(t, name, dtype, shape, device):
    """t is [rows, H, D] on the device with contiguous rows; returns its row stride in elements."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, not on cuda:{device}: one device "
                         "is needed")
    rows, heads, D = shape
    s0, s1, s2 = t.stride()
    if (s1 != D and heads > 1) or s2 != 1:
        raise ValueError(f"the heads of a row of {name} must be contiguous")
    if rows <= 1:
        return heads * D
    if s0 < heads * D or s0 % 8:
        raise ValueError(f"the row stride of {name} must be a multiple of 8 and cover the row")
    return s0


def qk_rope_append(q, k, v, positions, slots, rope, k_pool, v_pool, q_weight=None, k_weight=None,
                   eps: float = 1e-6, interleaved: bool = False, q_out=None, stream=None):
    """pa_qk_rope_append: norm (where a weight is given) and rotation of each query and key head,
    the keys and values written into their pool slots (see include/pa.h). q [T, Hq, D], k and v
    [T, Hkv, D], rows of any stride; positions and slots int32 [T] (a negative slot skips the
    row); rope fp32 [max_pos, rot_dim] (rope_table); pools [num_pages, PS, Hkv, D]. Returns
    q_out [T, Hq, D] (q itself may be given, when contiguous)."""
    import torch
    device = _device_of(q, "q")
    dt = q.dtype
    if dt is not torch.float16 and dt is not torch.bfloat16:
        raise TypeError("q must be float16 or bfloat16")
    if q.dim() != 3:
        raise ValueError("q must be [rows, Hq, D]")
    T, Hq, D = q.shape
    _require(k_pool, "k_pool", dt, None, device)
    pool = k_pool.shape
    if len(pool) != 4 or pool[3] != D:
        raise ValueError("k_pool must be [num_pages, page_size, Hkv, D]")
    num_pages, PS, Hkv, _ = pool
    _require(v_pool, "v_pool", dt, pool, device)
    q_stride = _require_rows(q, "q", dt, (T, Hq, D), device)
    k_stride = _require_rows(k, "k", dt, (T, Hkv, D), device)
    v_stride = _require_rows(v, "v", dt, (T, Hkv, D), device)
    _require(positions, "positions", torch.int32, (T,), device)
    _require(slots, "slots", torch.int32, (T,), device)
    _require(rope, "rope", torch.float32, None, device)
    if rope.dim() != 2:
        raise ValueError("rope must be [max_pos, rot_dim]")
    qw = kw = wt = None
    for w in (q_weight, k_weight):
        if w is not None:
            wt = wt or (dt if isinstance(w, torch.Tensor) and w.dtype is dt else torch.float32)
            _require(w, "q_weight and k_weight (both of q's type or both float32)", wt, (D,),
                     device)
    if q_weight is not None:
        qw = q_weight.data_ptr()
    if k_weight is not None:
        kw = k_weight.data_ptr()
    if q_out is None:
        q_out = _handed_back(stream, device, _new(stream, torch.empty_like, q,
                                                  memory_format=torch.contiguous_format))
    else:
        _require(q_out, "q_out", dt, (T, Hq, D), device)
    _call(device, stream, load_library().pa_qk_rope_append, "pa_qk_rope_append", Hq, Hkv, D, PS,
          PA_BF16 if dt is torch.bfloat16 else PA_F16, T, q.data_ptr(), q_stride, k.data_ptr(),
          k_stride, v.data_ptr(), v_stride, positions.data_ptr(), slots.data_ptr(),
          rope.data_ptr(), rope.shape[1], rope.shape[0], 1 if interleaved else 0, qw, kw,
          1 if wt is torch.float32 else 0, eps, q_out.data_ptr(), k_pool.data_ptr(),
          v_pool.data_ptr(), num_pages)
    return q_out


def device_error(reset: bool = True) -> tuple[int, int]:
    """(status, flags) of the library's device-side error word (synchronises the device)."""
    flags = ctypes.c_int(0)
    st = load_library().pa_device_error(ctypes.byref(flags), 1 if reset else 0)
    return st, flags.value


def set_wait_timeout_ns(ns: int):
    load_library().pa_set_wait_timeout_ns(ns)


def selftest_timeout(timeout_ns: int, stream=None):
    _check(load_library().pa_selftest_timeout(timeout_ns, _stream_ptr(stream)), "pa_selftest_timeout")
