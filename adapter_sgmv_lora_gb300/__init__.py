"""Python binding of liblora_sgmv.so (GB300 / sm_103a SGMV LoRA).

Argument marshalling only: every step of the computation runs in the CUDA
library; this module turns torch tensors into pointers, strides and the
current CUDA stream, calls the C ABI declared in ``include/lora_sgmv.h`` and
raises ``LoraError`` on any non-OK status.  There is no fallback: if the
library cannot be loaded, every call raises.

Names follow the C ABI: ``lora_build_routing``, ``lora_set_slot``,
``lora_shrink``, ``lora_expand``, ``lora_workspace_bytes``,
``lora_sgmv_apply``, ``lora_sgmv_apply_noalloc``, ``lora_base_gemm_apply``,
``lora_get_device_status``, ``lora_last_call_path``, ``lora_status_string``;
between the projections ``lora_build_rope``, ``lora_rope_append``,
``lora_attention_workspace_bytes``, ``lora_paged_attention``,
``lora_kv_copy_pages`` and the page bookkeeping ``lora_pages_*`` (class
``Pages``); for the verification of drafted tokens ``lora_base_q4_apply``,
``lora_build_tree``, ``lora_tree_attention_workspace_bytes``,
``lora_tree_attention`` and ``lora_kv_keep_rows``.
"""
from __future__ import annotations

import ctypes
import operator
import os
from dataclasses import dataclass, field, fields
from typing import List, Optional, Sequence

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liblora_sgmv.so")

LORA_OK = 0
STATUS_NAMES = {0: "LORA_OK", 1: "LORA_ERR_NULL", 2: "LORA_ERR_SHAPE", 3: "LORA_ERR_RANK",
                4: "LORA_ERR_SLOT_RANGE", 5: "LORA_ERR_ROUTING", 6: "LORA_ERR_DTYPE",
                7: "LORA_ERR_ALIGN", 8: "LORA_ERR_WORKSPACE", 9: "LORA_ERR_CUDA",
                10: "LORA_ERR_TOO_MANY_GROUPS", 11: "LORA_ERR_NO_PAGES"}
DTYPE_F32, DTYPE_BF16 = 0, 1
DEV_BAD_SLOT, DEV_BAD_OFFSETS, DEV_BAD_END, DEV_TIMEOUT, DEV_BAD_ROW = 1, 2, 4, 8, 16
DEV_BAD_PAGE, DEV_BAD_LENGTH = 32, 64
# Kernel families of lora_last_call_path (include/lora_sgmv.h).
PATH_GENERIC_SHRINK, PATH_GENERIC_EXPAND = 0x1, 0x2
PATH_MMA_SHRINK, PATH_MMA_EXPAND = 0x4, 0x8
PATH_TC_SHRINK, PATH_TC_EXPAND = 0x10, 0x20
PATH_PREP, PATH_BASE_GEMM = 0x80, 0x100
PATH_ROPE, PATH_GENERIC_ROPE = 0x200, 0x400
PATH_MMA_ATTENTION, PATH_GENERIC_ATTENTION, PATH_JOIN = 0x800, 0x1000, 0x2000
PATH_PAGES = 0x4000
PATH_MMA_Q4, PATH_GENERIC_Q4 = 0x8000, 0x10000
PATH_TC_TREE, PATH_GENERIC_TREE, PATH_KEEP, PATH_TC_Q4 = 0x20000, 0x40000, 0x80000, 0x100000
MAX_SLICES = 3


class LoraError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s: %s" % (what, STATUS_NAMES.get(status, str(status))))


class _Slice(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("A_slot_stride", ctypes.c_int64), ("B", ctypes.c_void_p),
                ("B_slot_stride", ctypes.c_int64), ("out_dim", ctypes.c_int32), ("y", ctypes.c_void_p),
                ("y_row_stride", ctypes.c_int64), ("bias", ctypes.c_void_p), ("bias_slot_stride", ctypes.c_int64)]


class _Problem(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("num_tokens", ctypes.c_int32), ("in_dim", ctypes.c_int32),
                ("max_num_loras", ctypes.c_int32), ("max_lora_rank", ctypes.c_int32),
                ("x", ctypes.c_void_p), ("x_row_stride", ctypes.c_int64),
                ("num_slices", ctypes.c_int32), ("slices", _Slice * MAX_SLICES), ("slot_ranks", ctypes.c_void_p)]


class _BaseWeight(ctypes.Structure):
    _fields_ = [("W0", ctypes.c_void_p), ("row_stride", ctypes.c_int64)]


class _Routing(ctypes.Structure):
    _fields_ = [("lora_ids", ctypes.c_void_p), ("grouped_offsets", ctypes.c_void_p),
                ("num_groups", ctypes.c_int32), ("end", ctypes.c_int32), ("token_rows", ctypes.c_void_p),
                ("host_grouped_offsets", ctypes.c_void_p), ("host_lora_ids", ctypes.c_void_p)]


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _KVCache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class _Rope(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("num_tokens", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("layout", ctypes.c_int), ("attention_scale", ctypes.c_float), ("eps", ctypes.c_float),
                ("turns", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("q", _Heads), ("k", _Heads),
                ("v", _Heads), ("q_out", _Heads), ("k_out", _Heads), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("cache_rows", ctypes.c_void_p)]


class _Attention(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("num_heads", ctypes.c_int32), ("q", _Heads), ("out", _Heads),
                ("block_tables", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("max_pages", ctypes.c_int32),
                ("lengths", ctypes.c_void_p), ("scale", ctypes.c_float), ("lse", ctypes.c_void_p)]


class _TreeAttention(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("num_rows", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("q", _Heads), ("out", _Heads), ("block_tables", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("max_pages", ctypes.c_int32), ("lengths", ctypes.c_void_p), ("row_offsets", ctypes.c_void_p),
                ("masks", ctypes.c_void_p), ("mask_words", ctypes.c_int32), ("scale", ctypes.c_float),
                ("lse", ctypes.c_void_p)]


class _Keep(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("block_tables", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("max_pages", ctypes.c_int32), ("lengths", ctypes.c_void_p), ("row_offsets", ctypes.c_void_p),
                ("path", ctypes.c_void_p), ("path_stride", ctypes.c_int64), ("max_kept", ctypes.c_int32),
                ("new_lengths", ctypes.c_void_p)]


class _Q4Weight(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_row_stride", ctypes.c_int64), ("scales", ctypes.c_void_p),
                ("scale_row_stride", ctypes.c_int64), ("zeros", ctypes.c_void_p), ("zero_row_stride", ctypes.c_int64),
                ("group_size", ctypes.c_int32)]


class _Pages(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_seqs", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("tables", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("refs", ctypes.c_void_p), ("free_pages", ctypes.c_void_p), ("num_free", ctypes.c_int32)]


_lib = None
_load_error = None


def library_path() -> str:
    return LIB_PATH


def lib():
    """The loaded library; raises if it is missing or fails to load."""
    global _lib, _load_error
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("liblora_sgmv.so is not built (run adapter_sgmv_lora_gb300/build.py or "
                           "__graft_entry__.build()); there is no fallback")
    L = ctypes.CDLL(LIB_PATH)
    i32 = ctypes.c_int32
    i32p = ctypes.POINTER(ctypes.c_int32)
    vp = ctypes.c_void_p
    L.lora_build_routing.restype = ctypes.c_int
    L.lora_build_routing.argtypes = [i32, i32p, i32p, i32, i32p, i32p, i32p, i32p, i32p, i32p]
    L.lora_build_token_rows.restype = ctypes.c_int
    L.lora_build_token_rows.argtypes = [i32, i32p, i32p, i32, i32p]
    L.lora_set_slot_bias.restype = ctypes.c_int
    L.lora_set_slot_bias.argtypes = [ctypes.POINTER(_Problem), i32, i32, vp, ctypes.c_int, vp]
    L.lora_set_slot.restype = ctypes.c_int
    L.lora_set_slot.argtypes = [ctypes.POINTER(_Problem), i32, i32, i32, ctypes.c_double, i32, vp, vp,
                                ctypes.c_int, vp]
    for name in ("lora_shrink", "lora_expand"):
        f = getattr(L, name)
        f.restype = ctypes.c_int
        f.argtypes = [ctypes.POINTER(_Problem), ctypes.POINTER(_Routing), vp, vp]
    L.lora_workspace_bytes.restype = ctypes.c_size_t
    L.lora_workspace_bytes.argtypes = [ctypes.POINTER(_Problem), i32]
    L.lora_sgmv_apply.restype = ctypes.c_int
    L.lora_sgmv_apply.argtypes = [ctypes.POINTER(_Problem), ctypes.POINTER(_Routing), vp,
                                  ctypes.c_size_t, vp]
    L.lora_sgmv_apply_noalloc.restype = ctypes.c_int
    L.lora_sgmv_apply_noalloc.argtypes = [ctypes.POINTER(_Problem), ctypes.POINTER(_Routing), vp]
    L.lora_get_device_status.restype = ctypes.c_int
    L.lora_get_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
    L.lora_status_string.restype = ctypes.c_char_p
    L.lora_status_string.argtypes = [ctypes.c_int]
    L.lora_base_gemm_apply.restype = ctypes.c_int
    L.lora_base_gemm_apply.argtypes = [ctypes.POINTER(_Problem), ctypes.POINTER(_Routing),
                                       ctypes.POINTER(_BaseWeight), vp, ctypes.c_size_t, vp]
    L.lora_last_call_path.restype = ctypes.c_uint32
    L.lora_last_call_path.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    L.lora_selftest_wait_timeout.restype = ctypes.c_int
    L.lora_selftest_wait_timeout.argtypes = [ctypes.c_uint32, vp]
    f64 = ctypes.c_double
    L.lora_build_rope.restype = ctypes.c_int
    L.lora_build_rope.argtypes = [i32, f64, ctypes.c_int, f64, i32, f64, f64, vp, vp]
    # Descriptors of repeated calls are held as ready-made pointers: plain void pointers here.
    L.lora_rope_append.restype = ctypes.c_int
    L.lora_rope_append.argtypes = [vp, vp, vp]
    L.lora_attention_workspace_bytes.restype = ctypes.c_size_t
    L.lora_attention_workspace_bytes.argtypes = [vp, vp]
    L.lora_paged_attention.restype = ctypes.c_int
    L.lora_paged_attention.argtypes = [vp, vp, vp, ctypes.c_size_t, vp]
    L.lora_kv_copy_pages.restype = ctypes.c_int
    L.lora_kv_copy_pages.argtypes = [vp, i32, vp, vp, i32, vp]
    L.lora_base_q4_apply.restype = ctypes.c_int
    L.lora_base_q4_apply.argtypes = [vp, vp, vp, vp, ctypes.c_size_t, vp]
    L.lora_build_tree.restype = ctypes.c_int
    L.lora_build_tree.argtypes = [i32, vp, i32, vp, vp]
    L.lora_tree_attention_workspace_bytes.restype = ctypes.c_size_t
    L.lora_tree_attention_workspace_bytes.argtypes = [vp, vp]
    L.lora_tree_attention.restype = ctypes.c_int
    L.lora_tree_attention.argtypes = [vp, vp, vp, ctypes.c_size_t, vp]
    L.lora_kv_keep_rows.restype = ctypes.c_int
    L.lora_kv_keep_rows.argtypes = [vp, i32, vp, vp]
    pg = ctypes.POINTER(_Pages)
    L.lora_pages_init.restype = ctypes.c_int
    L.lora_pages_init.argtypes = [pg]
    L.lora_pages_append.restype = ctypes.c_int
    L.lora_pages_append.argtypes = [pg, i32, i32, vp, i32p, i32p]
    L.lora_pages_fork.restype = ctypes.c_int
    L.lora_pages_fork.argtypes = [pg, i32, i32, i32]
    L.lora_pages_trim.restype = ctypes.c_int
    L.lora_pages_trim.argtypes = [pg, i32, i32]
    L.lora_pages_compact.restype = ctypes.c_int
    L.lora_pages_compact.argtypes = [pg, vp, vp, i32p]
    _lib = L
    return L


def _check(rc: int, what: str):
    if rc != LORA_OK:
        raise LoraError(rc, what)


def _stream_handle(stream) -> Optional[int]:
    import torch
    if stream is None:
        # The raw handle: building a Stream object costs more than a small call's kernel.
        # It comes from private functions of torch; a version without them has the public one.
        if torch.cuda.is_initialized():
            try:
                return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
            except AttributeError:
                pass
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


# --------------------------------------------------------------- routing --

def lora_build_routing(req_slot, req_num_tokens, max_num_loras: int, out_ids=None, out_offsets=None) -> dict:
    """Host sort + group (see include/lora_sgmv.h).  Returns numpy arrays.

    out_ids / out_offsets (optional): contiguous int32 arrays of at least
    max_num_loras and max_num_loras + 1 elements (for instance views of
    pinned host tensors) that receive lora_ids and grouped_offsets directly;
    the returned entries are then views of them."""
    L = lib()
    slots = np.ascontiguousarray(np.asarray(req_slot, dtype=np.int32))
    lens = np.ascontiguousarray(np.asarray(req_num_tokens, dtype=np.int32))
    if slots.shape != lens.shape or slots.ndim != 1:
        raise ValueError("req_slot and req_num_tokens must be 1-D and the same length")
    n = int(slots.size)
    S = int(max_num_loras)
    perm = np.zeros(max(n, 1), dtype=np.int32)
    for a, need, name in ((out_ids, max(S, 1), "out_ids"), (out_offsets, max(S, 1) + 1, "out_offsets")):
        if a is not None and (a.dtype != np.int32 or a.ndim != 1 or a.size < need or not a.flags.c_contiguous):
            raise ValueError("%s must be a contiguous int32 array of at least %d elements" % (name, need))
    ids = out_ids if out_ids is not None else np.zeros(max(S, 1), dtype=np.int32)
    offs = out_offsets if out_offsets is not None else np.zeros(max(S, 1) + 1, dtype=np.int32)
    G, end, T = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    p = lambda a: a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    rc = L.lora_build_routing(n, p(slots), p(lens), S, p(perm), p(ids), p(offs), ctypes.byref(G),
                              ctypes.byref(end), ctypes.byref(T))
    _check(rc, "lora_build_routing")
    g = G.value
    keep_ids = ids[:g] if out_ids is not None else ids[:g].copy()
    keep_offs = offs[:g + 1] if out_offsets is not None else offs[:g + 1].copy()
    return {"perm": perm[:n].copy(), "lora_ids": keep_ids, "grouped_offsets": keep_offs,
            "num_groups": g, "end": end.value, "total_tokens": T.value}


def lora_build_token_rows(req_num_tokens, perm, end: int) -> np.ndarray:
    """Rows of the routed tokens in sorted order for an arrival-order batch."""
    L = lib()
    lens = np.ascontiguousarray(np.asarray(req_num_tokens, dtype=np.int32))
    pm = np.ascontiguousarray(np.asarray(perm, dtype=np.int32))
    out = np.zeros(max(int(end), 1), dtype=np.int32)
    p = lambda a: a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    _check(L.lora_build_token_rows(int(lens.size), p(lens), p(pm), int(end), p(out)), "lora_build_token_rows")
    return out[:int(end)].copy()


@dataclass
class Routing:
    """Routing triple: device lora_ids / grouped_offsets tensors, host num_groups / end,
    optionally device token_rows (row of each sorted token, unsorted batches),
    a host copy of grouped_offsets (int32 numpy array) that lets the library
    pick the kernels per group, and a host copy of lora_ids (with the host
    offsets: the mma.sync kernels take the triple as launch parameters)."""
    lora_ids: object
    grouped_offsets: object
    num_groups: int
    end: int
    token_rows: object = None
    host_grouped_offsets: object = None
    host_lora_ids: object = None

    def _c(self) -> _Routing:
        ptr = lambda t: t.data_ptr() if t is not None and t.numel() > 0 else None

        def host(a):
            if a is None:
                return None
            a = np.ascontiguousarray(a, dtype=np.int32)
            self._host_keep.append(a)  # the pointer must outlive the call
            return a.ctypes.data if a.size > 0 else None

        self._host_keep = []
        return _Routing(ptr(self.lora_ids), ptr(self.grouped_offsets), int(self.num_groups), int(self.end),
                        ptr(self.token_rows), host(self.host_grouped_offsets), host(self.host_lora_ids))


def routing_to_device(r: dict, device="cuda", non_blocking=False, host_offsets=False,
                      host_ids=False) -> Routing:
    """Upload the host triple from lora_build_routing (int32 tensors); with
    host_offsets the host copy of grouped_offsets rides along (per-group
    kernel choice), with host_ids also the host copy of lora_ids (the
    mma.sync kernels then take the triple as launch parameters)."""
    import torch
    ids_h = np.ascontiguousarray(r["lora_ids"], dtype=np.int32)[: int(r["num_groups"])]
    ids = torch.from_numpy(np.ascontiguousarray(r["lora_ids"], dtype=np.int32))
    offs_h = np.ascontiguousarray(r["grouped_offsets"], dtype=np.int32)
    offs = torch.from_numpy(offs_h)
    return Routing(ids.to(device, non_blocking=non_blocking), offs.to(device, non_blocking=non_blocking),
                   int(r["num_groups"]), int(r["end"]), None,
                   offs_h.copy() if host_offsets or host_ids else None, ids_h.copy() if host_ids else None)


# --------------------------------------------------------------- problems --

@dataclass
class Slice:
    """One projection slice: stacks A/B (device tensors), element offsets into
    them, slot strides, out_dim, and the output y (2-D tensor) with a column
    offset.  Row stride of y is taken from the tensor."""
    A: object
    A_slot_stride: int
    B: object
    B_slot_stride: int
    out_dim: int
    y: object
    A_offset: int = 0
    B_offset: int = 0
    y_col: int = 0
    bias: object = None          # optional [S, >= out] stack (element offset bias_offset)
    bias_slot_stride: int = 0
    bias_offset: int = 0


@dataclass
class Problem:
    x: object
    slices: List[Slice]
    max_num_loras: int
    max_lora_rank: int
    slot_ranks: object = None    # optional device int32 [S]: true ranks (skip the padding)
    _keep: list = field(default_factory=list)

    def _c(self) -> _Problem:
        import torch
        x = self.x
        if x.dim() != 2 or x.stride(1) != 1:
            raise ValueError("x must be 2-D with unit column stride")
        dt = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}.get(x.dtype)
        if dt is None:
            raise ValueError("x must be float32 or bfloat16")
        if not 1 <= len(self.slices) <= MAX_SLICES:
            raise ValueError("1..3 slices")
        es = x.element_size()
        arr = (_Slice * MAX_SLICES)()
        for j, s in enumerate(self.slices):
            for t in (s.A, s.B, s.y):
                if t.dtype != x.dtype:
                    raise ValueError("x, y, A and B must share one dtype")
            if s.y.dim() != 2 or s.y.stride(1) != 1:
                raise ValueError("y must be 2-D with unit column stride")
            bias_ptr = s.bias.data_ptr() + es * int(s.bias_offset) if s.bias is not None else None
            arr[j] = _Slice(s.A.data_ptr() + es * int(s.A_offset), int(s.A_slot_stride),
                            s.B.data_ptr() + es * int(s.B_offset), int(s.B_slot_stride), int(s.out_dim),
                            s.y.data_ptr() + es * int(s.y_col), int(s.y.stride(0)), bias_ptr,
                            int(s.bias_slot_stride))
        ranks = self.slot_ranks.data_ptr() if self.slot_ranks is not None else None
        return _Problem(dt, int(x.shape[0]), int(x.shape[1]), int(self.max_num_loras),
                        int(self.max_lora_rank), x.data_ptr(), int(x.stride(0)), len(self.slices), arr, ranks)


def fused_problem(x, A_fused, B_fused, y, out_dims: Sequence[int]) -> Problem:
    """Fused stacks A [S, n*R, in], B [S, O, R] and y [T, O] (QKV fusion: A on
    the rank dimension, B on the output dimension)."""
    S, nR, k = A_fused.shape
    n = len(out_dims)
    R = nR // n
    O = int(sum(out_dims))
    assert B_fused.shape == (S, O, R) and nR == n * R
    slices, off = [], 0
    for j, od in enumerate(out_dims):
        slices.append(Slice(A_fused, n * R * k, B_fused, O * R, int(od), y, A_offset=j * R * k,
                            B_offset=off * R, y_col=off))
        off += od
    return Problem(x, slices, S, R)


def per_projection_problem(x, A_list, B_list, y_list, y_cols=None) -> Problem:
    """Separate stacks per projection: A_j [S, R, in], B_j [S, out_j, R]; y_list
    gives each projection's output tensor (or one tensor repeated with y_cols)."""
    slices = []
    S, R, k = A_list[0].shape
    for j, (A, B, y) in enumerate(zip(A_list, B_list, y_list)):
        od = B.shape[1]
        slices.append(Slice(A, R * k, B, od * R, int(od), y, y_col=(y_cols[j] if y_cols else 0)))
    return Problem(x, slices, S, R)


# ---------------------------------------------------------------- calls --

def lora_set_slot(problem: Problem, slice_index: int, slot: int, r: int, lora_alpha: float,
                  use_rslora: bool, A_raw, B_raw, stream=None) -> None:
    import torch
    L = lib()
    raw_dt = DTYPE_BF16 if (A_raw is not None and A_raw.dtype == torch.bfloat16) else DTYPE_F32
    pa = A_raw.data_ptr() if A_raw is not None else None
    pb = B_raw.data_ptr() if B_raw is not None else None
    c = problem._c()
    _check(L.lora_set_slot(ctypes.byref(c), int(slice_index), int(slot), int(r), float(lora_alpha),
                           int(bool(use_rslora)), pa, pb, raw_dt, _stream_handle(stream)),
           "lora_set_slot")


def lora_set_slot_bias(problem: Problem, slice_index: int, slot: int, bias_raw, stream=None) -> None:
    import torch
    L = lib()
    raw_dt = DTYPE_BF16 if (bias_raw is not None and bias_raw.dtype == torch.bfloat16) else DTYPE_F32
    c = problem._c()
    _check(L.lora_set_slot_bias(ctypes.byref(c), int(slice_index), int(slot),
                                bias_raw.data_ptr() if bias_raw is not None else None, raw_dt,
                                _stream_handle(stream)), "lora_set_slot_bias")


def lora_shrink(problem: Problem, routing: Routing, u, stream=None) -> None:
    L = lib()
    c, rr = problem._c(), routing._c()
    _check(L.lora_shrink(ctypes.byref(c), ctypes.byref(rr), u.data_ptr() if u is not None else None,
                         _stream_handle(stream)), "lora_shrink")


def lora_expand(problem: Problem, routing: Routing, u, stream=None) -> None:
    L = lib()
    c, rr = problem._c(), routing._c()
    _check(L.lora_expand(ctypes.byref(c), ctypes.byref(rr), u.data_ptr() if u is not None else None,
                         _stream_handle(stream)), "lora_expand")


def lora_workspace_bytes(problem: Problem, end: int) -> int:
    c = problem._c()
    return int(lib().lora_workspace_bytes(ctypes.byref(c), int(end)))


def new_workspace(problem: Problem, end: int, device="cuda"):
    """A workspace tensor of lora_workspace_bytes(problem, end) bytes."""
    import torch
    nbytes = max(lora_workspace_bytes(problem, end), 256)
    return torch.empty((nbytes + 15) // 16 * 4, dtype=torch.float32, device=device)


def lora_sgmv_apply(problem: Problem, routing: Routing, workspace, stream=None) -> None:
    L = lib()
    c, rr = problem._c(), routing._c()
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(L.lora_sgmv_apply(ctypes.byref(c), ctypes.byref(rr),
                             workspace.data_ptr() if workspace is not None else None, nbytes,
                             _stream_handle(stream)), "lora_sgmv_apply")


def lora_base_gemm_apply(problem: Problem, routing: Routing, W0, workspace, stream=None) -> None:
    """The delta fused into the base projection: every row of each slice's
    y becomes W0_j x (+ the LoRA delta on routed rows), rounded once; y is
    written, not read.  W0: one device tensor [out_j, in] per slice (same
    dtype as x), or (tensor, element offset, row stride) tuples."""
    L = lib()
    c, rr = problem._c(), routing._c()
    arr = (_BaseWeight * MAX_SLICES)()
    if len(W0) != len(problem.slices):
        raise ValueError("one base weight per slice")
    for j, w in enumerate(W0):
        if isinstance(w, tuple):
            t, off, stride = w
        else:
            t, off, stride = w, 0, w.stride(0)
        if t.dtype != problem.x.dtype:
            raise ValueError("W0 must have the dtype of x")
        arr[j] = _BaseWeight(t.data_ptr() + t.element_size() * int(off), int(stride))
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(L.lora_base_gemm_apply(ctypes.byref(c), ctypes.byref(rr), arr,
                                  workspace.data_ptr() if workspace is not None else None, nbytes,
                                  _stream_handle(stream)), "lora_base_gemm_apply")


NOALLOC_MAX_WORKSPACE_BYTES = 16 * 1024 * 1024


def lora_sgmv_apply_noalloc(problem: Problem, routing: Routing, stream=None) -> None:
    """lora_sgmv_apply without a workspace argument, for callers that cannot
    allocate device memory: the intermediate lives in a fixed 16 MiB array
    inside the library.  Calls whose GPU work overlaps race on that array."""
    L = lib()
    c, rr = problem._c(), routing._c()
    _check(L.lora_sgmv_apply_noalloc(ctypes.byref(c), ctypes.byref(rr), _stream_handle(stream)),
           "lora_sgmv_apply_noalloc")


def lora_get_device_status(stream=None) -> int:
    L = lib()
    flags = ctypes.c_uint32(0)
    _check(L.lora_get_device_status(_stream_handle(stream), ctypes.byref(flags)),
           "lora_get_device_status")
    return int(flags.value)


def lora_last_call_path():
    """(path bits, kernel launches) of the most recent library call made on
    this host thread; see lora_last_call_path in include/lora_sgmv.h."""
    n = ctypes.c_uint32(0)
    bits = lib().lora_last_call_path(ctypes.byref(n))
    return int(bits), int(n.value)


def lora_selftest_wait_timeout(polls: int, stream=None) -> None:
    """Launch the failure-path self test: a bounded wait that runs out and
    sets LORA_DEV_TIMEOUT in the device status word (see include/lora_sgmv.h)."""
    _check(lib().lora_selftest_wait_timeout(int(polls), _stream_handle(stream)), "lora_selftest_wait_timeout")


def lora_status_string(status: int) -> str:
    return lib().lora_status_string(int(status)).decode()


class CallBuilder:
    """Pre-marshalled C arguments for repeated calls on fixed buffers (for
    CUDA-graph capture and the benchmark's hot loop): builds the ctypes
    structs once, then each call is a single foreign call."""

    def __init__(self, problem: Problem, routing: Routing, workspace):
        self.L = lib()
        self.c = problem._c()
        self.r = routing._c()
        self.ws = workspace.data_ptr()
        self.nbytes = workspace.numel() * workspace.element_size()
        self._keep = (problem, routing, workspace)
        self._n = ctypes.c_uint32(0)
        self.last_path = 0       # kernel families of the latest apply (lora_last_call_path)
        self.last_launches = 0   # kernels it launched

    def set_routing(self, num_groups: int, end: int) -> None:
        """A new batch in the same device routing buffers: only the host
        num_groups and end change."""
        self.r.num_groups = int(num_groups)
        self.r.end = int(end)

    def apply(self, stream=None) -> None:
        rc = self.L.lora_sgmv_apply(ctypes.byref(self.c), ctypes.byref(self.r), self.ws, self.nbytes,
                                    _stream_handle(stream))
        _check(rc, "lora_sgmv_apply")
        self.last_path = int(self.L.lora_last_call_path(ctypes.byref(self._n)))
        self.last_launches = int(self._n.value)


# ------------------------------------------- attention between projections --
#
# The objects below describe buffers for repeated calls, as CallBuilder does:
# frozen, holding their tensors, with the C structs made once.  New values are
# written into the tensors; other tensors need another object.

ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}
MAX_HEAD_DIM = 256


def _dtype_code(t) -> int:
    import torch
    code = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}.get(t.dtype)
    if code is None:
        raise ValueError("tensors must be float32 or bfloat16")
    return code


def _on_cuda(**tensors) -> None:
    device = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("%s must be a CUDA tensor" % name)
        if device is not None and t.device != device:
            raise ValueError("%s is on another device" % name)
        device = t.device


def _int32(name: str, t, shape) -> None:
    import torch
    if t.dtype != torch.int32 or tuple(t.shape) != tuple(shape):
        raise ValueError("%s must be an int32 tensor of shape %s" % (name, tuple(shape)))
    if t.dim() > 0 and t.shape[-1] > 1 and t.stride(-1) != 1 and 0 not in t.shape:
        raise ValueError("%s must be contiguous along its last dimension" % name)


def _heads(name: str, t, shape, dtype) -> _Heads:
    if t is None:
        return _Heads(None, 0, 0)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s" % (name, tuple(shape)))
    if t.dtype != dtype:
        raise ValueError("%s must have the dtype of the others" % name)
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError("%s must have unit stride in its last dimension" % name)
    return _Heads(t.data_ptr(), t.stride(0), t.stride(1))


def _i32(value, what: str) -> int:
    """A whole number that an int32 argument holds as it is (ctypes would wrap it)."""
    i = int(value)
    if i != value:
        raise ValueError("%s: %r is not a whole number" % (what, value))
    if not -2 ** 31 <= i < 2 ** 31:
        raise LoraError(2, what)
    return i


def lora_build_rope(rotary_dim: int, theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                    original_max_positions: int = 0, low_turns: float = 1.0, high_turns: float = 4.0,
                    frequencies=None, attention_scale: float = 1.0) -> dict:
    """The rotation's frequency table (host; include/lora_sgmv.h): {"turns":
    uint64 [rotary_dim / 2], "rotary_dim", "attention_scale"}.

    scaling: "none", "linear" (position interpolation), "ntk", or "parts" (by
    parts between low_turns and high_turns turns over original_max_positions:
    1 and 4 for Llama 3's rule, 1 and 32 for YaRN's formula, whose
    attention_scale is 0.1 ln(factor) + 1).  The parts blend linearly in the
    turns, as those formulas do.  Checkpoints whose code blends linearly in the
    pair's index between the bounds' pairs need their frequencies given.
    frequencies: rotary_dim / 2 radians per position instead of theta's."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError("scaling must be one of %s" % ", ".join(ROPE_SCALINGS))
    D = _i32(rotary_dim, "lora_build_rope")
    positions = _i32(original_max_positions, "lora_build_rope")
    if D > MAX_HEAD_DIM:
        raise LoraError(2, "lora_build_rope")
    freq = None
    if frequencies is not None:
        freq = np.ascontiguousarray(frequencies, dtype=np.float64)
        if freq.shape != (D // 2,):
            raise ValueError("frequencies must hold rotary_dim / 2 values")
    turns = np.zeros(max(D // 2, 1), dtype=np.uint64)
    rc = lib().lora_build_rope(D, float(theta), ROPE_SCALINGS[scaling], float(factor), positions,
                               float(low_turns), float(high_turns), None if freq is None else freq.ctypes.data,
                               turns.ctypes.data)
    _check(rc, "lora_build_rope")
    return {"turns": turns, "rotary_dim": D, "attention_scale": float(attention_scale)}


@dataclass(frozen=True)
class Rope:
    """The frequency table on the device (int64 tensor holding the uint64 bits)."""
    turns: object
    rotary_dim: int
    attention_scale: float = 1.0

    def __post_init__(self):
        import torch
        t = self.turns
        if t.dtype not in (torch.int64, torch.uint64) or t.dim() != 1 or not t.is_contiguous() or \
                t.numel() < self.rotary_dim // 2:
            raise ValueError("turns must be a contiguous int64 tensor of rotary_dim / 2 values")


def rope_to_device(r: dict, device="cuda") -> Rope:
    """Upload the host table from lora_build_rope."""
    import torch
    return Rope(torch.from_numpy(r["turns"].view(np.int64).copy()).to(device), int(r["rotary_dim"]),
                float(r["attention_scale"]))


@dataclass(frozen=True)
class KVCache:
    """One layer's paged cache: k and v [num_pages, page_size, kv_heads,
    head_dim] with the same strides, unit in the last dimension (head-major
    memory is a permuted view)."""
    k: object
    v: object

    def __post_init__(self):
        k, v = self.k, self.v
        code = _dtype_code(k)
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must be 4-D [pages, page_size, kv_heads, head_dim] of one shape and dtype")
        if k.shape[3] > 1 and (k.stride(3) != 1 or v.stride(3) != 1):
            raise ValueError("k and v must have unit stride in their last dimension")
        if any(k.shape[i] > 1 and k.stride(i) != v.stride(i) for i in range(3)):
            raise ValueError("k and v must have the same strides")
        _on_cuda(k=k, v=v)
        c = _KVCache(code, k.shape[0], k.shape[1], k.shape[2], k.shape[3], k.data_ptr(), v.data_ptr(), k.stride(0),
                     k.stride(1), k.stride(2))
        object.__setattr__(self, "_struct", c)
        object.__setattr__(self, "_ref", ctypes.addressof(c))


@dataclass(frozen=True)
class KVCaches:
    """The layers' caches for lora_kv_copy_pages."""
    layers: Sequence[KVCache]

    def __post_init__(self):
        object.__setattr__(self, "layers", tuple(self.layers))  # the caller's list may change, the structs do not
        if any(c.k.device != self.layers[0].k.device for c in self.layers):
            raise ValueError("the layers must be on one device")
        arr = (_KVCache * max(len(self.layers), 1))(*[c._struct for c in self.layers])
        object.__setattr__(self, "_struct", arr)
        object.__setattr__(self, "_ref", ctypes.addressof(arr))


@dataclass(frozen=True)
class RopeProblem:
    """One lora_rope_append call: q [T, heads, head_dim], k and v [T, kv_heads,
    head_dim] (views of a fused qkv output, for instance), q_out (may be q),
    optionally k_out, a cache with cache_rows int32 [T], and per-head norm
    weights [head_dim].  rope None: no rotation (then positions may be None)."""
    q: object = None
    k: object = None
    v: object = None
    q_out: object = None
    k_out: object = None
    rope: Optional[Rope] = None
    positions: object = None
    interleaved: bool = False
    cache: Optional[KVCache] = None
    cache_rows: object = None
    q_weight: object = None
    k_weight: object = None
    eps: float = 1e-6

    def __post_init__(self):
        x = self.q if self.q is not None else self.k
        if x is None or x.dim() != 3:
            raise ValueError("q or k must be given, 3-D [tokens, heads, head_dim]")
        code = _dtype_code(x)
        T, hd = x.shape[0], x.shape[2]
        H = self.q.shape[1] if self.q is not None else 0
        Hk = self.k.shape[1] if self.k is not None and self.k.dim() == 3 else 0
        rot = self.rope.rotary_dim if self.rope is not None else 0
        _on_cuda(q=self.q, k=self.k, v=self.v, q_out=self.q_out, k_out=self.k_out, positions=self.positions,
                 turns=self.rope.turns if self.rope is not None else None, cache_rows=self.cache_rows,
                 cache=self.cache.k if self.cache is not None else None, q_weight=self.q_weight,
                 k_weight=self.k_weight)
        for name, t in (("positions", self.positions), ("cache_rows", self.cache_rows)):
            if t is not None:
                _int32(name, t, (T,))
        for name, w in (("q_weight", self.q_weight), ("k_weight", self.k_weight)):
            if w is not None and (tuple(w.shape) != (hd,) or w.dtype != x.dtype or (hd > 1 and w.stride(0) != 1)):
                raise ValueError("%s must be a contiguous [head_dim] tensor of q's dtype" % name)
        ptr = lambda t: t.data_ptr() if t is not None else None
        c = _Rope(code, T, H, Hk, hd, rot, int(bool(self.interleaved)),
                  self.rope.attention_scale if self.rope is not None else 1.0, float(self.eps),
                  ptr(self.rope.turns) if self.rope is not None else None, ptr(self.positions),
                  _heads("q", self.q, (T, H, hd), x.dtype), _heads("k", self.k, (T, Hk, hd), x.dtype),
                  _heads("v", self.v, (T, Hk, hd), x.dtype), _heads("q_out", self.q_out, (T, H, hd), x.dtype),
                  _heads("k_out", self.k_out, (T, Hk, hd), x.dtype), ptr(self.q_weight), ptr(self.k_weight),
                  ptr(self.cache_rows))
        object.__setattr__(self, "_struct", c)
        object.__setattr__(self, "_ref", ctypes.addressof(c))
        object.__setattr__(self, "_cache_ref", self.cache._ref if self.cache is not None else None)


def lora_rope_append(problem: RopeProblem, stream=None) -> None:
    """Norm, rotate and store a batch's q/k/v rows in one pass (include/lora_sgmv.h)."""
    _check(lib().lora_rope_append(problem._ref, problem._cache_ref, _stream_handle(stream)), "lora_rope_append")


@dataclass(frozen=True)
class AttentionProblem:
    """One lora_paged_attention call: q and out [B, heads, head_dim] (out may
    be q), block_tables int32 [B, max_pages], lengths int32 [B], scale (None:
    1 / sqrt(head_dim)), optionally lse float32 [B, heads]."""
    q: object
    out: object
    cache: KVCache
    block_tables: object
    lengths: object
    scale: Optional[float] = None
    lse: object = None

    def __post_init__(self):
        import torch
        q, cc = self.q, self.cache._struct
        if q.dim() != 3:
            raise ValueError("q must be 3-D [sequences, heads, head_dim]")
        B, H, hd = q.shape
        if hd != cc.head_dim:
            raise ValueError("q must have the cache's head_dim")
        _on_cuda(q=q, out=self.out, block_tables=self.block_tables, lengths=self.lengths, lse=self.lse,
                 cache=self.cache.k)
        if self.block_tables.dim() != 2:
            raise ValueError("block_tables must be 2-D [sequences, max_pages]")
        M = self.block_tables.shape[1]
        _int32("block_tables", self.block_tables, (B, M))
        _int32("lengths", self.lengths, (B,))
        if self.lse is not None and (self.lse.dtype != torch.float32 or tuple(self.lse.shape) != (B, H) or
                                     not self.lse.is_contiguous()):
            raise ValueError("lse must be a contiguous float32 [sequences, heads] tensor")
        scale = 1.0 / hd ** 0.5 if self.scale is None else float(self.scale)
        dt = self.cache.k.dtype
        c = _Attention(B, H, _heads("q", q, (B, H, hd), dt), _heads("out", self.out, (B, H, hd), dt),
                       self.block_tables.data_ptr() or None, self.block_tables.stride(0) if B > 1 else M, M,
                       self.lengths.data_ptr(), scale, self.lse.data_ptr() if self.lse is not None else None)
        object.__setattr__(self, "_struct", c)
        object.__setattr__(self, "_ref", ctypes.addressof(c))


def lora_attention_workspace_bytes(problem: AttentionProblem) -> int:
    return int(lib().lora_attention_workspace_bytes(problem._ref, problem.cache._ref))


def new_attention_workspace(problem: AttentionProblem):
    """A workspace tensor of lora_attention_workspace_bytes(problem) bytes."""
    import torch
    nbytes = max(lora_attention_workspace_bytes(problem), 256)
    return torch.empty((nbytes + 15) // 16 * 4, dtype=torch.float32, device=problem.q.device)


def lora_paged_attention(problem: AttentionProblem, workspace, stream=None) -> None:
    """Attention of one new token per sequence over its cached pages (include/lora_sgmv.h)."""
    ws, nbytes = None, 0
    if workspace is not None:
        if not workspace.is_cuda or workspace.device != problem.q.device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on q's device")
        ws, nbytes = workspace.data_ptr(), workspace.nbytes
    _check(lib().lora_paged_attention(problem._ref, problem.cache._ref, ws, nbytes, _stream_handle(stream)),
           "lora_paged_attention")


def _page_numbers(name: str, pages) -> np.ndarray:
    """int32 array of page numbers; what numpy would wrap or cut to one is refused."""
    a = np.asarray(pages)
    if a.dtype == np.int32:
        return a
    if a.size > 0:
        if a.dtype.kind not in "iu":
            raise ValueError("%s must hold integers" % name)
        if a.min() < -2 ** 31 or a.max() >= 2 ** 31:
            raise LoraError(2, "lora_kv_copy_pages")
    return a.astype(np.int32)


def lora_kv_copy_pages(caches: KVCaches, src, dst, stream=None) -> None:
    """Copy pages src[i] -> dst[i] (host integers) in every layer's K and V."""
    s = _page_numbers("src", src)
    d = _page_numbers("dst", dst)
    if s.ndim != 1 or s.shape != d.shape:
        raise ValueError("src and dst must be 1-D and the same length")
    # As bytes: copying the list is cheaper than asking an array for its address.
    _check(lib().lora_kv_copy_pages(caches._ref, len(caches.layers), s.tobytes(), d.tobytes(), s.size,
                                    _stream_handle(stream)), "lora_kv_copy_pages")


# ---------------------------------------- verification of drafted tokens --

MAX_MASK_WORDS, MAX_KEPT = 16, 1024


@dataclass(frozen=True)
class Q4Weight:
    """4-bit base weight of one slice: q uint8 [out, ceil(in / 2)] (input 2 i
    in the low half of byte i), scales [out, groups] in the problem's dtype,
    zeros uint8 [out, groups] (None: 8), group_size inputs a group."""
    q: object
    scales: object
    group_size: int
    zeros: object = None

    def __post_init__(self):
        import torch
        for name, t in (("q", self.q), ("scales", self.scales), ("zeros", self.zeros)):
            if t is None and name == "zeros":
                continue
            if t.dim() != 2 or t.shape[0] != self.q.shape[0] or (t.shape[1] > 1 and t.stride(1) != 1):
                raise ValueError("%s must be 2-D [out, ...] with unit column stride" % name)
            if name != "scales" and t.dtype != torch.uint8:
                raise ValueError("%s must be uint8" % name)
        _dtype_code(self.scales)
        if self.zeros is not None and self.zeros.shape != self.scales.shape:
            raise ValueError("zeros must have the shape of scales")
        object.__setattr__(self, "group_size", _i32(self.group_size, "lora_base_q4_apply"))
        if self.group_size < 1:
            raise LoraError(2, "lora_base_q4_apply")
        _on_cuda(q=self.q, scales=self.scales, zeros=self.zeros)


_problem_fields = operator.attrgetter("x", "max_num_loras", "max_lora_rank", "slot_ranks")
_routing_fields = operator.attrgetter(*(f.name for f in fields(Routing)))
_slice_fields = operator.attrgetter(*(f.name for f in fields(Slice)))


@dataclass(frozen=True)
class BaseQ4Problem:
    """One lora_base_q4_apply call: a problem, its routing and a Q4Weight per
    slice.  Routing(None, None, 0, 0) adds no adapter.  The call's arguments are
    made ready here, and again by a call that finds a field of the problem, of
    one of its slices or of the routing set to something else."""
    problem: Problem
    routing: Routing
    weights: Sequence[Q4Weight]

    def __post_init__(self):
        object.__setattr__(self, "weights", tuple(self.weights))
        self._encode()

    def _fields(self) -> list:
        now = [*_problem_fields(self.problem), *_routing_fields(self.routing)]
        for s in self.problem.slices:
            now += _slice_fields(s)
        return now

    def _current(self) -> tuple:
        """(addresses of the call's structs as the fields are now, what they were made from, what they point to)."""
        now, seen = self._fields(), self._made[1]
        if len(now) != len(seen) or not all(map(operator.is_, now, seen)):
            self._encode()
        return self._made

    def _encode(self) -> None:
        x, slices = self.problem.x, self.problem.slices
        if len(self.weights) != len(slices):
            raise ValueError("one base weight per slice")
        c, r = self.problem._c(), self.routing._c()
        arr = (_Q4Weight * MAX_SLICES)()
        rows = lambda t: t.stride(0) if t.shape[0] > 1 else t.shape[1]  # of one row any stride will do
        for j, (w, s) in enumerate(zip(self.weights, slices)):
            if w.scales.dtype != x.dtype:
                raise ValueError("scales must have the dtype of x")
            if w.q.shape != (s.out_dim, (x.shape[1] + 1) // 2):
                raise ValueError("q must have shape [out, ceil(in / 2)]")
            if w.scales.shape[1] != -(-x.shape[1] // w.group_size):
                raise ValueError("scales must have ceil(in / group_size) columns")
            _on_cuda(x=x, y=s.y, q=w.q)
            arr[j] = _Q4Weight(w.q.data_ptr(), rows(w.q), w.scales.data_ptr(), rows(w.scales),
                               w.zeros.data_ptr() if w.zeros is not None else None,
                               rows(w.zeros) if w.zeros is not None else 0, w.group_size)
        object.__setattr__(self, "_made", (tuple(ctypes.addressof(o) for o in (c, r, arr)), self._fields(),
                                           (c, r, arr, self.routing._host_keep)))


def _on_current(t) -> None:
    """Launches go to the current device: the call's tensors must be there."""
    import torch
    if t.device.index != torch.cuda.current_device():
        raise ValueError("the tensors are on %s, which is not the current device" % t.device)


def _workspace(workspace, like):
    _on_current(like)
    if workspace is None:
        return None, 0
    if not workspace.is_cuda or workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return workspace.data_ptr(), workspace.nbytes


def lora_base_q4_apply(problem: BaseQ4Problem, workspace, stream=None) -> None:
    """The base projection on 4-bit weights with the LoRA delta joined before
    the one rounding (include/lora_sgmv.h); workspace as new_workspace makes it."""
    ws, nbytes = _workspace(workspace, problem.problem.x)
    made = problem._current()
    _check(lib().lora_base_q4_apply(*made[0], ws, nbytes, _stream_handle(stream)), "lora_base_q4_apply")


def lora_build_tree(parents, words: Optional[int] = None) -> dict:
    """Masks and depths of a tree of drafted tokens (host; include/lora_sgmv.h):
    parents[i] in [-1, i), -1 where node i hangs on the context's end.  {"masks":
    uint64 [n, words] (words None: as few as hold n bits), "depths": int32 [n]}."""
    par = np.asarray(parents)
    if par.ndim != 1 or (par.size > 0 and par.dtype.kind not in "iu"):
        raise ValueError("parents must be a list of integers")
    if par.size > 0 and (par.min() < -1 or par.max() >= par.size):
        raise LoraError(2, "lora_build_tree")
    par = np.ascontiguousarray(par, dtype=np.int32)
    words = max(1, -(-par.size // 64)) if words is None else _i32(words, "lora_build_tree")
    if not 1 <= words <= MAX_MASK_WORDS:
        raise LoraError(2, "lora_build_tree")
    masks = np.zeros((par.size, words), dtype=np.uint64)
    depths = np.zeros(par.size, dtype=np.int32)
    _check(lib().lora_build_tree(par.size, par.ctypes.data, words, masks.ctypes.data, depths.ctypes.data),
           "lora_build_tree")
    return {"masks": masks, "depths": depths}


@dataclass(frozen=True)
class TreeAttentionProblem:
    """One lora_tree_attention call: q and out [N, heads, head_dim] (out may be
    q), block_tables int32 [B, max_pages], lengths int32 [B] (drafted tokens
    included), row_offsets int32 [B + 1], masks int64 [N, words] holding the
    uint64 bits of lora_build_tree (None: chains), scale (None: 1 /
    sqrt(head_dim)), optionally lse float32 [N, heads]."""
    q: object
    out: object
    cache: KVCache
    block_tables: object
    lengths: object
    row_offsets: object
    masks: object = None
    scale: Optional[float] = None
    lse: object = None

    def __post_init__(self):
        import torch
        q, cc = self.q, self.cache._struct
        if q.dim() != 3:
            raise ValueError("q must be 3-D [rows, heads, head_dim]")
        N, H, hd = q.shape
        if hd != cc.head_dim:
            raise ValueError("q must have the cache's head_dim")
        _on_cuda(q=q, out=self.out, block_tables=self.block_tables, lengths=self.lengths,
                 row_offsets=self.row_offsets, masks=self.masks, lse=self.lse, cache=self.cache.k)
        if self.block_tables.dim() != 2:
            raise ValueError("block_tables must be 2-D [sequences, max_pages]")
        B, M = self.block_tables.shape
        _int32("block_tables", self.block_tables, (B, M))
        _int32("lengths", self.lengths, (B,))
        _int32("row_offsets", self.row_offsets, (B + 1,))
        words = 0
        if self.masks is not None:
            m = self.masks
            if m.dtype not in (torch.int64, torch.uint64) or m.dim() != 2 or m.shape[0] != N or not m.is_contiguous():
                raise ValueError("masks must be a contiguous int64 tensor [rows, words]")
            words = m.shape[1]
        if self.lse is not None and (self.lse.dtype != torch.float32 or tuple(self.lse.shape) != (N, H) or
                                     not self.lse.is_contiguous()):
            raise ValueError("lse must be a contiguous float32 [rows, heads] tensor")
        scale = 1.0 / hd ** 0.5 if self.scale is None else float(self.scale)
        dt = self.cache.k.dtype
        ptr = lambda t: t.data_ptr() if t is not None else None
        c = _TreeAttention(B, N, H, _heads("q", q, (N, H, hd), dt), _heads("out", self.out, (N, H, hd), dt),
                           self.block_tables.data_ptr() or None, self.block_tables.stride(0) if B > 1 else M, M,
                           self.lengths.data_ptr(), self.row_offsets.data_ptr(), ptr(self.masks), words, scale,
                           ptr(self.lse))
        object.__setattr__(self, "_struct", c)
        object.__setattr__(self, "_ref", ctypes.addressof(c))


def lora_tree_attention_workspace_bytes(problem: TreeAttentionProblem) -> int:
    return int(lib().lora_tree_attention_workspace_bytes(problem._ref, problem.cache._ref))


def new_tree_attention_workspace(problem: TreeAttentionProblem):
    """A workspace tensor of lora_tree_attention_workspace_bytes(problem) bytes."""
    import torch
    nbytes = max(lora_tree_attention_workspace_bytes(problem), 256)
    return torch.empty((nbytes + 15) // 16 * 4, dtype=torch.float32, device=problem.q.device)


def lora_tree_attention(problem: TreeAttentionProblem, workspace, stream=None) -> None:
    """Attention of drafted tokens to their context and their own branch over
    the paged cache (include/lora_sgmv.h)."""
    ws, nbytes = _workspace(workspace, problem.q)
    _check(lib().lora_tree_attention(problem._ref, problem.cache._ref, ws, nbytes, _stream_handle(stream)),
           "lora_tree_attention")


@dataclass(frozen=True)
class KeepRowsProblem:
    """One lora_kv_keep_rows call: the layers' caches, block_tables, lengths and
    row_offsets as of the tree attention, path int32 [B, max_kept] (ascending
    drafted tokens, -1 ends a row), optionally new_lengths int32 [B]."""
    caches: KVCaches
    block_tables: object
    lengths: object
    row_offsets: object
    path: object
    new_lengths: object = None

    def __post_init__(self):
        if not self.caches.layers:
            raise ValueError("caches must hold a layer")
        _on_cuda(cache=self.caches.layers[0].k, block_tables=self.block_tables, lengths=self.lengths,
                 row_offsets=self.row_offsets, path=self.path, new_lengths=self.new_lengths)
        if self.block_tables.dim() != 2 or self.path.dim() != 2:
            raise ValueError("block_tables and path must be 2-D")
        B, M = self.block_tables.shape
        K = self.path.shape[1]
        _int32("block_tables", self.block_tables, (B, M))
        _int32("lengths", self.lengths, (B,))
        _int32("row_offsets", self.row_offsets, (B + 1,))
        _int32("path", self.path, (B, K))
        if self.new_lengths is not None:
            _int32("new_lengths", self.new_lengths, (B,))
        c = _Keep(B, self.block_tables.data_ptr() or None, self.block_tables.stride(0) if B > 1 else M, M,
                  self.lengths.data_ptr(), self.row_offsets.data_ptr(), self.path.data_ptr() or None,
                  self.path.stride(0) if B > 1 else K, K,
                  self.new_lengths.data_ptr() if self.new_lengths is not None else None)
        object.__setattr__(self, "_struct", c)
        object.__setattr__(self, "_ref", ctypes.addressof(c))


def lora_kv_keep_rows(problem: KeepRowsProblem, stream=None) -> None:
    """Move the accepted drafted tokens' cache rows up behind the context, in
    every layer (include/lora_sgmv.h)."""
    _on_current(problem.caches.layers[0].k)
    _check(lib().lora_kv_keep_rows(problem.caches._ref, len(problem.caches.layers), problem._ref,
                                   _stream_handle(stream)), "lora_kv_keep_rows")


class Pages:
    """Host bookkeeping of one cache's pages (lora_pages_*): tables [max_seqs,
    max_pages], lengths, refs and the free list are numpy arrays to read or
    upload; only the methods change them."""

    def __init__(self, num_pages: int, page_size: int, max_seqs: int, max_pages: int):
        sizes = [_i32(n, "lora_pages_init") for n in (num_pages, page_size, max_seqs, max_pages)]
        num_pages, page_size, max_seqs, max_pages = sizes
        if min(sizes) < 1:
            raise LoraError(2, "lora_pages_init")
        self.tables = np.empty((max_seqs, max_pages), dtype=np.int32)
        self.lengths = np.empty(max_seqs, dtype=np.int32)
        self.refs = np.empty(num_pages, dtype=np.int32)
        self.free_pages = np.empty(num_pages, dtype=np.int32)
        self._c = _Pages(num_pages, page_size, max_seqs, max_pages, self.tables.ctypes.data, self.lengths.ctypes.data,
                         self.refs.ctypes.data, self.free_pages.ctypes.data, 0)
        _check(lib().lora_pages_init(ctypes.byref(self._c)), "lora_pages_init")

    @property
    def num_free(self) -> int:
        return int(self._c.num_free)

    def append(self, seq: int, num_tokens: int):
        """(cache rows of the new tokens, page copies to run first as (src,
        dst) pairs: at most one)."""
        seq, num_tokens = _i32(seq, "lora_pages_append"), _i32(num_tokens, "lora_pages_append")
        rows = np.empty(max(num_tokens, 0), dtype=np.int32)
        src, dst = ctypes.c_int32(), ctypes.c_int32()
        _check(lib().lora_pages_append(ctypes.byref(self._c), seq, num_tokens, rows.ctypes.data,
                                       ctypes.byref(src), ctypes.byref(dst)), "lora_pages_append")
        return rows, ([(src.value, dst.value)] if src.value >= 0 else [])

    def fork(self, parent: int, child: int, num_tokens: Optional[int] = None) -> None:
        """child shares parent's first num_tokens (None: all of them)."""
        parent, child = _i32(parent, "lora_pages_fork"), _i32(child, "lora_pages_fork")
        if num_tokens is None:
            if not 0 <= parent < self.lengths.size:
                raise LoraError(2, "lora_pages_fork")
            num_tokens = int(self.lengths[parent])
        _check(lib().lora_pages_fork(ctypes.byref(self._c), parent, child, _i32(num_tokens, "lora_pages_fork")),
               "lora_pages_fork")

    def trim(self, seq: int, num_tokens: int = 0) -> None:
        _check(lib().lora_pages_trim(ctypes.byref(self._c), _i32(seq, "lora_pages_trim"),
                                     _i32(num_tokens, "lora_pages_trim")), "lora_pages_trim")

    def compact(self):
        """(src, dst) page moves to run with lora_kv_copy_pages; the tables are already rewritten."""
        n = ctypes.c_int32()
        src = np.empty(self.refs.size, dtype=np.int32)
        dst = np.empty(self.refs.size, dtype=np.int32)
        _check(lib().lora_pages_compact(ctypes.byref(self._c), src.ctypes.data, dst.ctypes.data, ctypes.byref(n)),
               "lora_pages_compact")
        return src[:n.value].copy(), dst[:n.value].copy()
