"""Thin Python binding of ``libpagedkv`` (the C ABI in include/pagedkv.h).

Argument marshalling only: torch tensors supply device pointers, sizes and the
current CUDA stream; every step of the computation runs in the library's kernels.
There is no fallback: if the shared library is missing or fails to load, every call
raises. Function names match the C entry points.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libpagedkv.so")

PKV_OK = 0
STATUS_NAMES = {0: "PKV_OK", 1: "PKV_ERR_NULL", 2: "PKV_ERR_SHAPE", 3: "PKV_ERR_HEADS",
                4: "PKV_ERR_DTYPE", 5: "PKV_ERR_KV_MODE", 6: "PKV_ERR_CAUSAL",
                7: "PKV_ERR_WORKSPACE", 8: "PKV_ERR_ALIGN", 9: "PKV_ERR_UNSUPPORTED",
                10: "PKV_ERR_LAUNCH"}
PKV_F16, PKV_BF16, PKV_F32, PKV_I32 = 1, 2, 3, 4
PKV_SPLIT_AUTO, PKV_SPLIT_PAGES, PKV_SPLIT_FIXED = 0, 1, 2
DEV_BAD_BLOCK, DEV_BAD_SLOT, DEV_BAD_POSITION, DEV_BAD_SEQUENCE, DEV_BAD_EDGE = 1, 2, 4, 8, 16
DEV_TIMEOUT, DEV_NO_BLOCKS = 32, 64
MAX_ROTARY_PAIRS = 128
PRED_BITS = {"cacheShapeOk": 1, "headLayoutOk": 2, "scheduleShapeOk": 4, "ioShapeOk": 8,
             "separateKv": 16, "packedKv": 32, "slotShapeOk": 64}

c_i32, c_i64, c_f32, c_vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class PagedKVError(RuntimeError):
    def __init__(self, call: str, status: int):
        self.status = status
        self.name = STATUS_NAMES.get(status, str(status))
        super().__init__(f"{call} failed: {self.name} ({_status_string(status)})")


class PagedAttentionArgs(ctypes.Structure):
    _fields_ = [("query", c_vp), ("key", c_vp), ("value", c_vp), ("key_cache", c_vp),
                ("value_cache", c_vp), ("cumulative_sequence_length", c_vp),
                ("past_seqlens", c_vp), ("block_table", c_vp), ("slot_mapping", c_vp),
                ("output", c_vp), ("device_status", c_vp), ("cos_cache", c_vp),
                ("sin_cache", c_vp),
                ("num_tokens", c_i64), ("query_hidden", c_i64), ("batch", c_i64),
                ("num_heads", c_i64), ("kv_num_heads", c_i64), ("head_size", c_i64),
                ("block_size", c_i64), ("num_blocks", c_i64), ("max_blocks", c_i64),
                ("rotary_dim", c_i64), ("rotary_positions", c_i64),
                ("rotary_interleaved", c_i32), ("is_causal", c_i32), ("dtype", c_i32),
                ("scale", c_f32), ("split_policy", c_i32), ("fixed_splits", c_i32),
                ("max_splits", c_i32), ("split_min_keys", c_i32), ("rotary_query", c_i32),
                ("reserved", c_i32)]


class PagedPlan(ctypes.Structure):
    _fields_ = [("mode", c_i32), ("group_size", c_i32), ("pages_num_splits", c_i32),
                ("max_splits", c_i32), ("pages_partial_bytes", c_i64),
                ("pages_stats_bytes", c_i64), ("workspace_bytes", c_i64),
                ("decode_item_bound", c_i64), ("prefill_item_bound", c_i64),
                ("partial_slot_bound", c_i64)]


class TensorDesc(ctypes.Structure):
    _fields_ = [("present", c_i32), ("rank", c_i32), ("dtype", c_i32), ("reserved", c_i32),
                ("dims", c_i64 * 4)]


class PagedShapes(ctypes.Structure):
    _fields_ = [(n, TensorDesc) for n in ("query", "key", "value", "key_cache",
                                          "value_cache", "cumulative_sequence_length",
                                          "past_seqlens", "block_table", "slot_mapping",
                                          "output")] + \
               [("num_heads", c_i64), ("kv_num_heads", c_i64), ("is_causal", c_i32),
                ("reserved", c_i32)]


class KVAppendArgs(ctypes.Structure):
    _fields_ = [("source", c_vp), ("value", c_vp), ("total_sequence_length", c_vp),
                ("key_total_sequence_lengths", c_vp), ("cos_cache", c_vp),
                ("sin_cache", c_vp), ("present_key", c_vp), ("present_value", c_vp),
                ("device_status", c_vp), ("batch", c_i64), ("seq_len", c_i64),
                ("num_heads", c_i64), ("kv_num_heads", c_i64), ("head_size", c_i64),
                ("max_cache_seq", c_i64), ("rotary_dim", c_i64), ("rotary_positions", c_i64),
                ("packed", c_i32), ("interleaved", c_i32), ("dtype", c_i32),
                ("reserved", c_i32), ("query", c_vp), ("query_out", c_vp)]


class SparseArgs(ctypes.Structure):
    _fields_ = [("q", c_vp), ("k_pages", c_vp), ("v_pages", c_vp), ("edge_meta", c_vp),
                ("block_tables", c_vp), ("o_partial", c_vp), ("m_partial", c_vp),
                ("l_partial", c_vp), ("device_status", c_vp), ("num_queries", c_i64),
                ("num_edges", c_i64), ("num_seqs", c_i64), ("max_pages", c_i64),
                ("num_pages", c_i64), ("qhead", c_i64), ("hq", c_i64), ("hkv", c_i64),
                ("head_dim", c_i64), ("block_size", c_i64), ("page_size", c_i64),
                ("pages_per_block", c_i64), ("softmax_scale", c_f32), ("dtype", c_i32),
                ("query_positions", c_vp)]


class CombineArgs(ctypes.Structure):
    _fields_ = [("o", c_vp), ("m", c_vp), ("l", c_vp), ("segment_offsets", c_vp),
                ("out", c_vp), ("lse", c_vp), ("num_segments", c_i64), ("lanes", c_i64),
                ("head_dim", c_i64), ("uniform_count", c_i64), ("out_dtype", c_i32),
                ("reserved", c_i32)]


class ScheduleArgs(ctypes.Structure):
    _fields_ = [("past_seqlens", c_vp), ("new_seqlens", c_vp), ("block_table", c_vp),
                ("cumulative_sequence_length", c_vp), ("slot_mapping", c_vp),
                ("positions", c_vp), ("total_seqlens", c_vp), ("free_blocks", c_vp),
                ("device_status", c_vp), ("batch", c_i64), ("max_blocks", c_i64),
                ("num_blocks", c_i64), ("block_size", c_i64), ("num_tokens", c_i64)]


class AppendAxesArgs(ctypes.Structure):
    _fields_ = [("query", c_vp), ("key", c_vp), ("value", c_vp), ("query_out", c_vp),
                ("key_cache", c_vp), ("value_cache", c_vp), ("slot_mapping", c_vp),
                ("positions", c_vp), ("cos_cache", c_vp), ("sin_cache", c_vp),
                ("device_status", c_vp), ("num_tokens", c_i64), ("num_heads", c_i64),
                ("kv_num_heads", c_i64), ("head_size", c_i64), ("block_size", c_i64),
                ("num_blocks", c_i64), ("rotary_dim", c_i64), ("rotary_positions", c_i64),
                ("num_axes", c_i32), ("rotary_interleaved", c_i32), ("dtype", c_i32),
                ("table_dtype", c_i32), ("pair_axis", ctypes.c_uint8 * MAX_ROTARY_PAIRS)]


class CrossAttentionArgs(ctypes.Structure):
    _fields_ = [("query", c_vp), ("key_cache", c_vp), ("value_cache", c_vp),
                ("cumulative_sequence_length", c_vp), ("key_seqlens", c_vp),
                ("block_table", c_vp), ("output", c_vp), ("lse", c_vp),
                ("device_status", c_vp), ("num_tokens", c_i64), ("batch", c_i64),
                ("num_heads", c_i64), ("kv_num_heads", c_i64), ("head_size", c_i64),
                ("block_size", c_i64), ("num_blocks", c_i64), ("max_blocks", c_i64),
                ("max_query_len", c_i64), ("dtype", c_i32), ("scale", c_f32)]


STRUCTS = {"pkv_paged_attention_args": PagedAttentionArgs, "pkv_paged_plan": PagedPlan,
           "pkv_tensor_desc": TensorDesc, "pkv_paged_shapes": PagedShapes,
           "pkv_kv_append_args": KVAppendArgs, "pkv_sparse_args": SparseArgs,
           "pkv_combine_args": CombineArgs, "pkv_schedule_args": ScheduleArgs,
           "pkv_append_axes_args": AppendAxesArgs,
           "pkv_cross_attention_args": CrossAttentionArgs}

_LIB = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libpagedkv (once) and check ABI version and struct layouts. Raises if the
    library is absent: build it with ``__graft_entry__.build()``."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libpagedkv not built ({p} missing); run __graft_entry__.build()")
    lib = ctypes.CDLL(p)
    lib.pkv_abi_version.restype = c_i32
    lib.pkv_status_string.restype = ctypes.c_char_p
    lib.pkv_status_string.argtypes = [c_i32]
    lib.pkv_sizeof_struct.restype = ctypes.c_size_t
    lib.pkv_sizeof_struct.argtypes = [ctypes.c_char_p]
    lib.pkv_launch_count.restype = c_i64
    lib.pkv_profiler_enable.argtypes = [c_i32]
    lib.pkv_profiler_query.argtypes = [ctypes.c_char_p, ctypes.POINTER(ctypes.c_double),
                                       ctypes.POINTER(c_i64)]
    for name, args in (
            ("pkv_paged_attention_plan", [ctypes.POINTER(PagedAttentionArgs),
                                          ctypes.POINTER(PagedPlan)]),
            ("pkv_paged_attention_workspace_size", [ctypes.POINTER(PagedAttentionArgs),
                                                    ctypes.POINTER(ctypes.c_size_t)]),
            ("pkv_paged_attention", [ctypes.POINTER(PagedAttentionArgs), c_vp,
                                     ctypes.c_size_t, c_vp]),
            ("pkv_paged_scatter_kv", [ctypes.POINTER(PagedAttentionArgs), c_vp]),
            ("pkv_paged_contract_check", [ctypes.POINTER(PagedShapes),
                                          ctypes.POINTER(ctypes.c_uint32),
                                          ctypes.POINTER(c_i32)]),
            ("pkv_kv_append_rotary", [ctypes.POINTER(KVAppendArgs), c_vp]),
            ("pkv_sparse_attention_partials_workspace_size",
             [ctypes.POINTER(SparseArgs), ctypes.POINTER(ctypes.c_size_t)]),
            ("pkv_sparse_attention_partials", [ctypes.POINTER(SparseArgs), c_vp,
                                               ctypes.c_size_t, c_vp]),
            ("pkv_combine_partials", [ctypes.POINTER(CombineArgs), c_vp]),
            ("pkv_paged_schedule", [ctypes.POINTER(ScheduleArgs), c_vp]),
            ("pkv_paged_append_rotary_axes", [ctypes.POINTER(AppendAxesArgs), c_vp]),
            ("pkv_cross_attention_workspace_size", [ctypes.POINTER(CrossAttentionArgs),
                                                    ctypes.POINTER(ctypes.c_size_t)]),
            ("pkv_cross_attention", [ctypes.POINTER(CrossAttentionArgs), c_vp,
                                     ctypes.c_size_t, c_vp]),
            ("pkv_testing_wait_limit", [ctypes.c_uint32, c_i32])):
        fn = getattr(lib, name)
        fn.restype = c_i32
        fn.argtypes = args
    if lib.pkv_abi_version() != 3:
        raise RuntimeError("libpagedkv ABI version mismatch")
    for name, cls in STRUCTS.items():
        n = lib.pkv_sizeof_struct(name.encode())
        if n != ctypes.sizeof(cls):
            raise RuntimeError(f"struct {name}: library {n} bytes, binding "
                               f"{ctypes.sizeof(cls)} bytes")
    if path is None:
        _LIB = lib
    return lib


def _status_string(status: int) -> str:
    try:
        return load_library().pkv_status_string(status).decode()
    except Exception:  # noqa: BLE001 - message only
        return ""


def _check(call: str, status: int):
    if status != PKV_OK:
        raise PagedKVError(call, status)


# ----------------------------------------------------------------------------- helpers
def _torch():
    import torch
    return torch


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _made(stream, shape, dtype, device, returned=True):
    """A tensor for a call on ``stream`` (None: the current one). The allocator hands memory
    out in the order of the stream that it is asked on: a block of the current stream's may
    still be in use there by kernels that were enqueued before it was freed, and a call on
    another stream would not wait for them. So it is asked for on the call's stream (in a
    capture there, of the graph's memory); what is returned to the caller, who works on the
    current stream, is given away again only after that stream's use too."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned and stream != current:
        t.record_stream(current)
    return t


def _require(t, dtype, name, device=True):
    torch = _torch()
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if device and not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")


_DT = {"float16": PKV_F16, "bfloat16": PKV_BF16, "float32": PKV_F32, "int32": PKV_I32}


def _dtype_code(t) -> int:
    return _DT.get(str(t.dtype).replace("torch.", ""), 0)


def _desc(t) -> TensorDesc:
    d = TensorDesc()
    if t is None:
        return d
    d.present = 1
    d.rank = t.dim()
    d.dtype = _dtype_code(t)
    for i, s in enumerate(list(t.shape)[:4]):
        d.dims[i] = int(s)
    return d


# ----------------------------------------------------------------------------- paged
def pkv_paged_contract_check(query, key, value, key_cache, value_cache,
                             cumulative_sequence_length, past_seqlens, block_table,
                             slot_mapping, output, *, num_heads: int, kv_num_heads: int,
                             is_causal: int = 1):
    """Shape/dtype contract of the PagedAttention manifest (host only; tensors may live
    on any device). Returns (status, failed_predicates_set, mode)."""
    lib = load_library()
    sh = PagedShapes()
    for name, t in (("query", query), ("key", key), ("value", value),
                    ("key_cache", key_cache), ("value_cache", value_cache),
                    ("cumulative_sequence_length", cumulative_sequence_length),
                    ("past_seqlens", past_seqlens), ("block_table", block_table),
                    ("slot_mapping", slot_mapping), ("output", output)):
        setattr(sh, name, _desc(t))
    sh.num_heads = num_heads
    sh.kv_num_heads = kv_num_heads
    sh.is_causal = is_causal
    failed = ctypes.c_uint32(0)
    mode = c_i32(0)
    st = lib.pkv_paged_contract_check(ctypes.byref(sh), ctypes.byref(failed),
                                      ctypes.byref(mode))
    names = {n for n, bit in PRED_BITS.items() if failed.value & bit}
    return st, names, {1: "separate", 2: "packed"}.get(mode.value)


def make_paged_args(query, key, value, key_cache, value_cache, cumulative_sequence_length,
                    past_seqlens, block_table, slot_mapping=None, output=None, *,
                    num_heads: int, kv_num_heads: int, scale: float = 0.0,
                    is_causal: int = 1, device_status=None, cos_cache=None, sin_cache=None,
                    rotary_dim: int = 0, rotary_interleaved: bool = False,
                    split_policy: int = PKV_SPLIT_AUTO, fixed_splits: int = 0,
                    max_splits: int = 0, split_min_keys: int = 0,
                    rotary_query: bool = False) -> PagedAttentionArgs:
    """Fill the C argument block from tensors (no validation beyond rank checks; the
    library validates). Works for host-only planning too (pointers may be host)."""
    a = PagedAttentionArgs()
    a.query, a.key, a.value = _ptr(query), _ptr(key), _ptr(value)
    a.key_cache, a.value_cache = _ptr(key_cache), _ptr(value_cache)
    a.cumulative_sequence_length = _ptr(cumulative_sequence_length)
    a.past_seqlens = _ptr(past_seqlens)
    a.block_table = _ptr(block_table)
    a.slot_mapping = _ptr(slot_mapping)
    a.output = _ptr(output)
    a.device_status = _ptr(device_status)
    a.cos_cache, a.sin_cache = _ptr(cos_cache), _ptr(sin_cache)
    a.num_tokens = int(query.shape[0])
    a.query_hidden = int(query.shape[1]) if query.dim() == 2 else 0
    a.batch = int(cumulative_sequence_length.shape[0]) - 1
    a.num_heads, a.kv_num_heads = int(num_heads), int(kv_num_heads)
    a.num_blocks, a.block_size = int(key_cache.shape[0]), int(key_cache.shape[1])
    a.head_size = int(key_cache.shape[3])
    a.max_blocks = int(block_table.shape[1])
    a.rotary_dim = int(rotary_dim)
    a.rotary_positions = int(cos_cache.shape[0]) if cos_cache is not None else 0
    a.rotary_interleaved = 1 if rotary_interleaved else 0
    a.is_causal = int(is_causal)
    a.dtype = _dtype_code(query)
    a.scale = float(scale)
    a.split_policy, a.fixed_splits = int(split_policy), int(fixed_splits)
    a.max_splits, a.split_min_keys = int(max_splits), int(split_min_keys)
    a.rotary_query = 1 if rotary_query else 0
    return a


def pkv_paged_attention_plan(args: PagedAttentionArgs) -> PagedPlan:
    plan = PagedPlan()
    _check("pkv_paged_attention_plan",
           load_library().pkv_paged_attention_plan(ctypes.byref(args), ctypes.byref(plan)))
    return plan


def pkv_paged_attention_workspace_size(args: PagedAttentionArgs) -> int:
    n = ctypes.c_size_t(0)
    _check("pkv_paged_attention_workspace_size",
           load_library().pkv_paged_attention_workspace_size(ctypes.byref(args),
                                                             ctypes.byref(n)))
    return int(n.value)


def _check_paged_tensors(query, key, value, key_cache, value_cache, cu, past, bt, slot,
                         output, num_heads, kv_num_heads, is_causal):
    torch = _torch()
    for t, n in ((query, "query"), (key, "key"), (value, "value"), (key_cache, "key_cache"),
                 (value_cache, "value_cache"), (output, "output")):
        _require(t, torch.float16, n)
    for t, n in ((cu, "cumulative_sequence_length"), (past, "past_seqlens"),
                 (bt, "block_table"), (slot, "slot_mapping")):
        _require(t, torch.int32, n)
    st, failed, mode = pkv_paged_contract_check(
        query, key, value, key_cache, value_cache, cu, past, bt, slot, output,
        num_heads=num_heads, kv_num_heads=kv_num_heads, is_causal=is_causal)
    _check(f"pkv_paged_contract_check (false: {sorted(failed)})", st)


def pkv_paged_attention(query, key, value, key_cache, value_cache,
                        cumulative_sequence_length, past_seqlens, block_table,
                        slot_mapping=None, *, num_heads: int, kv_num_heads: int,
                        scale: float = 0.0, is_causal: int = 1, output=None, workspace=None,
                        device_status=None, cos_cache=None, sin_cache=None,
                        rotary_dim: int = 0, rotary_interleaved: bool = False,
                        split_policy: int = PKV_SPLIT_AUTO, fixed_splits: int = 0,
                        max_splits: int = 0, split_min_keys: int = 0,
                        rotary_query: bool = False, stream=None):
    """PagedAttention: scatter new K/V into the caches (in place), then causal GQA
    attention. Returns the fp16 output [num_tokens, num_heads*head_size]."""
    torch = _torch()
    if output is None:
        output = _made(stream, (query.shape[0], num_heads * key_cache.shape[3]),
                       torch.float16, query.device)
    _check_paged_tensors(query, key, value, key_cache, value_cache,
                         cumulative_sequence_length, past_seqlens, block_table,
                         slot_mapping, output, num_heads, kv_num_heads, is_causal)
    if cos_cache is not None:
        _require(cos_cache, torch.float16, "cos_cache")
        _require(sin_cache, torch.float16, "sin_cache")
    a = make_paged_args(query, key, value, key_cache, value_cache,
                        cumulative_sequence_length, past_seqlens, block_table, slot_mapping,
                        output, num_heads=num_heads, kv_num_heads=kv_num_heads, scale=scale,
                        is_causal=is_causal, device_status=device_status,
                        cos_cache=cos_cache, sin_cache=sin_cache, rotary_dim=rotary_dim,
                        rotary_interleaved=rotary_interleaved, split_policy=split_policy,
                        fixed_splits=fixed_splits, max_splits=max_splits,
                        split_min_keys=split_min_keys, rotary_query=rotary_query)
    need = pkv_paged_attention_workspace_size(a)
    if workspace is None or workspace.numel() < need:
        workspace = _made(stream, max(need, 1), torch.uint8, query.device, returned=False)
    _check("pkv_paged_attention",
           load_library().pkv_paged_attention(ctypes.byref(a), workspace.data_ptr(), need,
                                              _stream(stream)))
    return output


def pkv_paged_scatter_kv(query, key, value, key_cache, value_cache,
                         cumulative_sequence_length, past_seqlens, block_table,
                         slot_mapping=None, *, num_heads: int, kv_num_heads: int,
                         device_status=None, cos_cache=None, sin_cache=None,
                         rotary_dim: int = 0, rotary_interleaved: bool = False,
                         stream=None):
    """The ScatterKV pass alone (caches updated in place)."""
    torch = _torch()
    for t, n in ((query, "query"), (key, "key"), (value, "value"),
                 (key_cache, "key_cache"), (value_cache, "value_cache")):
        _require(t, torch.float16, n)
    a = make_paged_args(query, key, value, key_cache, value_cache,
                        cumulative_sequence_length, past_seqlens, block_table, slot_mapping,
                        None, num_heads=num_heads, kv_num_heads=kv_num_heads,
                        device_status=device_status, cos_cache=cos_cache,
                        sin_cache=sin_cache, rotary_dim=rotary_dim,
                        rotary_interleaved=rotary_interleaved)
    _check("pkv_paged_scatter_kv",
           load_library().pkv_paged_scatter_kv(ctypes.byref(a), _stream(stream)))


# ----------------------------------------------------------------------------- append
def make_append_args(source, value, total_sequence_length, key_total_sequence_lengths,
                     present_key, present_value, *, num_heads: int, kv_num_heads: int,
                     batch: int, seq_len: int, packed: bool, cos_cache=None, sin_cache=None,
                     rotary_dim: int = 0, interleaved: bool = False,
                     device_status=None, query=None, query_out=None) -> KVAppendArgs:
    """Fill the C argument block of pkv_kv_append_rotary from tensors."""
    a = KVAppendArgs()
    a.source, a.value = _ptr(source), _ptr(value)
    a.total_sequence_length = _ptr(total_sequence_length)
    a.key_total_sequence_lengths = _ptr(key_total_sequence_lengths)
    a.cos_cache, a.sin_cache = _ptr(cos_cache), _ptr(sin_cache)
    a.present_key, a.present_value = _ptr(present_key), _ptr(present_value)
    a.device_status = _ptr(device_status)
    a.batch, a.seq_len = int(batch), int(seq_len)
    a.num_heads, a.kv_num_heads = int(num_heads), int(kv_num_heads)
    a.head_size = int(present_key.shape[3])
    a.max_cache_seq = int(present_key.shape[2])
    a.rotary_dim = int(rotary_dim)
    a.rotary_positions = int(cos_cache.shape[0]) if cos_cache is not None else 0
    a.packed = 1 if packed else 0
    a.interleaved = 1 if interleaved else 0
    a.dtype = _dtype_code(source)
    a.query, a.query_out = _ptr(query), _ptr(query_out)
    return a


def pkv_kv_append_rotary(source, value, total_sequence_length, key_total_sequence_lengths,
                         present_key, present_value, *, num_heads: int, kv_num_heads: int,
                         batch: int, seq_len: int, packed: bool, cos_cache=None,
                         sin_cache=None, rotary_dim: int = 0, interleaved: bool = False,
                         device_status=None, query=None, query_out=None, stream=None):
    """KV append (+ RoPE of K); with ``query_out`` the query heads are rotated at the
    same positions into it ([batch*seq_len, num_heads*head_size] fp16; ``query`` gives
    the query rows in separate mode)."""
    torch = _torch()
    for t, n in ((source, "source"), (value, "value"), (present_key, "present_key"),
                 (present_value, "present_value"), (cos_cache, "cos_cache"),
                 (sin_cache, "sin_cache"), (query, "query"), (query_out, "query_out")):
        _require(t, torch.float16, n)
    a = make_append_args(source, value, total_sequence_length, key_total_sequence_lengths,
                         present_key, present_value, num_heads=num_heads,
                         kv_num_heads=kv_num_heads, batch=batch, seq_len=seq_len,
                         packed=packed, cos_cache=cos_cache, sin_cache=sin_cache,
                         rotary_dim=rotary_dim, interleaved=interleaved,
                         device_status=device_status, query=query, query_out=query_out)
    _check("pkv_kv_append_rotary",
           load_library().pkv_kv_append_rotary(ctypes.byref(a), _stream(stream)))


# ----------------------------------------------------------------------------- sparse
def make_sparse_args(q, k_pages, v_pages, edge_meta, block_tables, o, m, l, *, qhead: int,
                     block_size: int, page_size: int, pages_per_block: int,
                     softmax_scale: float, device_status=None,
                     query_positions=None) -> SparseArgs:
    a = SparseArgs()
    a.q, a.k_pages, a.v_pages = _ptr(q), _ptr(k_pages), _ptr(v_pages)
    a.edge_meta, a.block_tables = _ptr(edge_meta), _ptr(block_tables)
    a.o_partial, a.m_partial, a.l_partial = _ptr(o), _ptr(m), _ptr(l)
    a.device_status = _ptr(device_status)
    a.num_queries, a.hq, a.head_dim = int(q.shape[0]), int(q.shape[1]), int(q.shape[2])
    a.num_edges = int(edge_meta.shape[0])
    a.num_seqs, a.max_pages = int(block_tables.shape[0]), int(block_tables.shape[1])
    a.num_pages, a.hkv = int(k_pages.shape[0]), int(k_pages.shape[1])
    a.qhead = int(qhead)
    a.block_size, a.page_size = int(block_size), int(page_size)
    a.pages_per_block = int(pages_per_block)
    a.softmax_scale = float(softmax_scale)
    a.dtype = _dtype_code(q)
    a.query_positions = _ptr(query_positions)
    return a


def pkv_sparse_attention_partials_workspace_size(args: SparseArgs) -> int:
    n = ctypes.c_size_t(0)
    _check("pkv_sparse_attention_partials_workspace_size",
           load_library().pkv_sparse_attention_partials_workspace_size(ctypes.byref(args),
                                                                       ctypes.byref(n)))
    return int(n.value)


def pkv_sparse_attention_partials(q, k_pages, v_pages, edge_meta, block_tables, *,
                                  qhead: int, block_size: int, page_size: int,
                                  pages_per_block: int, softmax_scale: float,
                                  o=None, m=None, l=None, workspace=None,
                                  device_status=None, query_positions=None, stream=None):
    """Block-sparse (o, m, l) partials, partial index edge*qhead + lane. q and the pages
    are all fp32 or all fp16; the partials are fp32. ``query_positions`` (int32 per
    query) applies the right-aligned causal mask."""
    torch = _torch()
    dt = torch.float16 if q.dtype == torch.float16 else torch.float32
    for t, n in ((q, "q"), (k_pages, "k_pages"), (v_pages, "v_pages")):
        _require(t, dt, n)
    _require(edge_meta, torch.int32, "edge_meta")
    _require(block_tables, torch.int32, "block_tables")
    _require(query_positions, torch.int32, "query_positions")
    P = int(edge_meta.shape[0]) * qhead
    D = int(q.shape[2])
    if o is None:
        o = _made(stream, (P, D), torch.float32, q.device)
    if m is None:
        m = _made(stream, P, torch.float32, q.device)
    if l is None:
        l = _made(stream, P, torch.float32, q.device)
    a = make_sparse_args(q, k_pages, v_pages, edge_meta, block_tables, o, m, l, qhead=qhead,
                         block_size=block_size, page_size=page_size,
                         pages_per_block=pages_per_block, softmax_scale=softmax_scale,
                         device_status=device_status, query_positions=query_positions)
    need = pkv_sparse_attention_partials_workspace_size(a)
    if workspace is None or workspace.numel() < need:
        workspace = _made(stream, max(need, 1), torch.uint8, q.device, returned=False)
    _check("pkv_sparse_attention_partials",
           load_library().pkv_sparse_attention_partials(ctypes.byref(a), workspace.data_ptr(),
                                                        need, _stream(stream)))
    return o, m, l


# ----------------------------------------------------------------------------- combine
def pkv_combine_partials(o, m, l, segment_offsets=None, *, num_segments: int, lanes: int,
                         uniform_count: int = 0, out=None, out_dtype=None, lse=None,
                         stream=None):
    """LSE merge: output row s*lanes + c from partial rows e*lanes + c, e in segment s."""
    torch = _torch()
    _require(o, torch.float32, "o")
    _require(m, torch.float32, "m")
    _require(l, torch.float32, "l")
    _require(segment_offsets, torch.int32, "segment_offsets")
    D = int(o.shape[-1])
    if out is None:
        out = _made(stream, (num_segments * lanes, D), out_dtype or torch.float32, o.device)
    a = CombineArgs()
    a.o, a.m, a.l = _ptr(o), _ptr(m), _ptr(l)
    a.segment_offsets = _ptr(segment_offsets)
    a.out, a.lse = _ptr(out), _ptr(lse)
    a.num_segments, a.lanes, a.head_dim = int(num_segments), int(lanes), D
    a.uniform_count = int(uniform_count)
    a.out_dtype = _dtype_code(out)
    _check("pkv_combine_partials",
           load_library().pkv_combine_partials(ctypes.byref(a), _stream(stream)))
    return out, lse


# ----------------------------------------------------------------------------- steps
# A decode step makes these calls once a layer, on the host thread that feeds the GPU: the
# argument blocks are packed in one go (fields as in the ctypes structures above) and passed
# as bytes, and a call's tensors are looked at once.
_SCHEDULE_PACK = struct.Struct("@9Q5q")
_AXES_PACK = struct.Struct("@11Q8q4i128s")
_CROSS_PACK = struct.Struct("@9Q9qif")
_STEP = {}   # entry points that take packed blocks


def _step_call(name: str, *args):
    fn = _STEP.get(name)
    if fn is None:
        lib = load_library()
        for pack, cls in ((_SCHEDULE_PACK, ScheduleArgs), (_AXES_PACK, AppendAxesArgs),
                          (_CROSS_PACK, CrossAttentionArgs)):
            assert pack.size == ctypes.sizeof(cls)
        for n, more in (("pkv_paged_schedule", [c_vp]), ("pkv_paged_append_rotary_axes", [c_vp]),
                        ("pkv_cross_attention", [c_vp, ctypes.c_size_t, c_vp])):
            f = lib[n]   # a function object of its own
            f.restype, f.argtypes = c_i32, [ctypes.c_char_p] + more
            _STEP[n] = f
        fn = _STEP[name]
    status = fn(*args)
    if status != PKV_OK:
        raise PagedKVError(name, status)


def _refuse(stream, tensors):
    """Names what is wrong with a call's tensors (see _check_tensors)."""
    for name, t, dtype, shape in tensors:
        if t is None:
            continue
        if t.dtype != dtype:
            raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    for name, t, _, _ in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name}: must be a CUDA tensor")
    here = _torch().cuda.current_device()
    for name, t, _, _ in tensors:
        if t is not None and t.get_device() != here:
            raise ValueError(f"{name}: on device {t.get_device()}, the current one is {here}")
    raise ValueError(f"stream: of device {stream.device_index}, the current one is {here}")


def _check_tensors(stream, tensors) -> int:
    """tensors: (name, tensor or None, dtype, shape) each. They have to be contiguous, of that
    dtype and shape, on the current CUDA device, which is the stream's too. Returns the raw
    stream."""
    device = None
    for _, t, dtype, shape in tensors:
        if t is None:
            continue
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
            _refuse(stream, tensors)
        at = t.get_device()
        if at != device:
            if device is not None or at < 0:
                _refuse(stream, tensors)
            device = at
    torch = _torch()
    if device != torch.cuda.current_device() or (stream is not None and
                                                 stream.device_index != device):
        _refuse(stream, tensors)
    if stream is not None:
        return stream.cuda_stream
    # the current stream's handle without an object for it (a microsecond of the call), where
    # this torch has that
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(device) if raw is not None else torch.cuda.current_stream(device).cuda_stream


def _need(**named):
    for name, t in named.items():
        if t is None:
            raise ValueError(f"{name}: required")


def _at(t) -> int:
    return 0 if t is None else t.data_ptr()


def pkv_paged_schedule(past_seqlens, new_seqlens, block_table, *, num_blocks: int,
                       block_size: int, num_tokens: int, cumulative_sequence_length=None,
                       slot_mapping=None, positions=None, total_seqlens=None,
                       free_blocks=None, device_status=None, stream=None):
    """Block tables, slot maps and cumulative lengths from request lengths, on the GPU.

    ``block_table`` [batch, max_blocks] is updated in place: row b holds its first
    ceil(past / block_size) entries and gets the lowest free blocks for its new tokens.
    Returns (cumulative_sequence_length [batch + 1], slot_mapping [num_tokens], positions
    [num_tokens], total_seqlens [batch], free_blocks [1]), all int32; those not passed in
    are made here. Rows that the pool or ``num_tokens`` cannot take get no tokens."""
    torch = _torch()
    i32 = torch.int32
    if past_seqlens is None or new_seqlens is None or block_table is None:
        _need(past_seqlens=past_seqlens, new_seqlens=new_seqlens, block_table=block_table)
    B = past_seqlens.shape[0] if past_seqlens.dim() == 1 else -1
    MB = block_table.shape[1] if block_table.dim() == 2 else -1
    raw = _check_tensors(stream, (
        ("past_seqlens", past_seqlens, i32, (B,)), ("new_seqlens", new_seqlens, i32, (B,)),
        ("block_table", block_table, i32, (B, MB)),
        ("cumulative_sequence_length", cumulative_sequence_length, i32, (B + 1,)),
        ("slot_mapping", slot_mapping, i32, (num_tokens,)),
        ("positions", positions, i32, (num_tokens,)),
        ("total_seqlens", total_seqlens, i32, (B,)), ("free_blocks", free_blocks, i32, (1,)),
        ("device_status", device_status, i32, (1,))))

    def made(t, n):
        return _made(stream, n, i32, block_table.device) if t is None else t

    cu, slots = made(cumulative_sequence_length, B + 1), made(slot_mapping, num_tokens)
    pos, total = made(positions, num_tokens), made(total_seqlens, B)
    free = made(free_blocks, 1)
    _step_call("pkv_paged_schedule",
               _SCHEDULE_PACK.pack(past_seqlens.data_ptr(), new_seqlens.data_ptr(),
                                   block_table.data_ptr(), cu.data_ptr(), slots.data_ptr(),
                                   pos.data_ptr(), total.data_ptr(), free.data_ptr(),
                                   _at(device_status), B, MB, num_blocks, block_size,
                                   num_tokens), raw)
    return cu, slots, pos, total, free


def rotary_pair_axis(sections, by_turns: bool = False):
    """Axis of each rotary pair, for ``sections`` pairs per axis: one section after the
    other (0 0 0 1 1 2), or the axes by turns while they have pairs left (0 1 2 0 1 0)."""
    left = [int(n) for n in sections]
    if not left or any(n < 0 for n in left):
        raise ValueError(f"sections: numbers of pairs, got {sections!r}")
    if not by_turns:
        return [a for a, n in enumerate(left) for _ in range(n)]
    axis = []
    while any(left):
        for a, n in enumerate(left):
            if n:
                axis.append(a)
                left[a] = n - 1
    return axis


def pkv_paged_append_rotary_axes(query, key, value, key_cache, value_cache, slot_mapping,
                                 positions, *, num_heads: int, kv_num_heads: int,
                                 cos_cache=None, sin_cache=None, rotary_dim: int = 0,
                                 pair_axis=None, rotary_interleaved: bool = False,
                                 query_out=None, rotate_query: bool = True,
                                 device_status=None, stream=None):
    """K and V rows into the paged cache (pool row slot_mapping[i], negative = padding), K
    and Q rotated with ``positions`` [axes, num_tokens]; ``pair_axis`` names the axis of each
    rotary pair (all axis 0 when None). float16 or bfloat16; the tables in that type or
    float32. Packed rows when key and value are None. Returns the rotated queries
    [num_tokens, num_heads * head_size] (made here unless ``query_out`` is given; rows of
    padding are not written), or None without them (``rotate_query`` false, or no query)."""
    torch = _torch()
    if key_cache is None or value_cache is None or slot_mapping is None:
        _need(key_cache=key_cache, value_cache=value_cache, slot_mapping=slot_mapping)
    dt, f32, i32 = key_cache.dtype, torch.float32, torch.int32
    if dt is torch.float16:
        code = PKV_F16
    elif dt is torch.bfloat16:
        code = PKV_BF16
    else:
        raise TypeError(f"key_cache: expected float16 or bfloat16, got {dt}")
    if key_cache.dim() != 4:
        raise ValueError("key_cache: [num_blocks, block_size, kv_num_heads, head_size]")
    NB, BS, _, D = key_cache.shape
    T = slot_mapping.shape[0] if slot_mapping.dim() == 1 else -1
    qh, kvh = num_heads * D, kv_num_heads * D
    pool = (NB, BS, kv_num_heads, D)
    half, axes, rows, tdt, pairs = rotary_dim // 2, 0, 0, f32, b""
    if rotary_dim > 0:
        if positions is None or cos_cache is None or sin_cache is None:
            _need(positions=positions, cos_cache=cos_cache, sin_cache=sin_cache)
        axes = positions.shape[0] if positions.dim() == 2 else -1
        rows = cos_cache.shape[0] if cos_cache.dim() == 2 else -1
        if cos_cache.dtype is dt:
            tdt = dt
        pairs = bytes(half) if pair_axis is None else bytes(list(pair_axis))
        if len(pairs) != half or half > MAX_ROTARY_PAIRS:
            raise ValueError(f"pair_axis: one axis for each of {half} pairs (at most "
                             f"{MAX_ROTARY_PAIRS}), got {len(pairs)}")
    else:
        positions = cos_cache = sin_cache = None
    raw = _check_tensors(stream, (
        ("query", query, dt, (T, qh + 2 * kvh if key is None and value is None else qh)),
        ("key", key, dt, (T, kvh)), ("value", value, dt, (T, kvh)),
        ("query_out", query_out, dt, (T, qh)), ("key_cache", key_cache, dt, pool),
        ("value_cache", value_cache, dt, pool), ("slot_mapping", slot_mapping, i32, (T,)),
        ("positions", positions, i32, (axes, T)), ("cos_cache", cos_cache, tdt, (rows, half)),
        ("sin_cache", sin_cache, tdt, (rows, half)), ("device_status", device_status, i32, (1,))))
    if rotate_query and query is not None and query_out is None:
        query_out = _made(stream, (T, qh), dt, key_cache.device)
    _step_call("pkv_paged_append_rotary_axes",
               _AXES_PACK.pack(_at(query), _at(key), _at(value), _at(query_out),
                               key_cache.data_ptr(), value_cache.data_ptr(),
                               slot_mapping.data_ptr(), _at(positions), _at(cos_cache),
                               _at(sin_cache), _at(device_status), T, num_heads, kv_num_heads,
                               D, BS, NB, rotary_dim, rows, axes,
                               1 if rotary_interleaved else 0, code,
                               PKV_F32 if tdt is f32 else code, pairs), raw)
    return query_out


def make_cross_args(query, key_cache, value_cache, cumulative_sequence_length, key_seqlens,
                    block_table, output, lse=None, *, num_heads: int, kv_num_heads: int,
                    max_query_len: int = 0, scale: float = 0.0,
                    device_status=None) -> CrossAttentionArgs:
    """Fill the C argument block of pkv_cross_attention from tensors."""
    return CrossAttentionArgs(
        query.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
        cumulative_sequence_length.data_ptr(), key_seqlens.data_ptr(), block_table.data_ptr(),
        output.data_ptr(), _ptr(lse), _ptr(device_status), query.shape[0],
        key_seqlens.shape[0], num_heads, kv_num_heads, key_cache.shape[3],
        key_cache.shape[1], key_cache.shape[0], block_table.shape[1], max_query_len,
        _dtype_code(query), scale)


def pkv_cross_attention_workspace_size(args: CrossAttentionArgs) -> int:
    n = ctypes.c_size_t(0)
    _check("pkv_cross_attention_workspace_size",
           load_library().pkv_cross_attention_workspace_size(ctypes.byref(args),
                                                             ctypes.byref(n)))
    return n.value


@functools.lru_cache(maxsize=1024)
def _cross_workspace(device: int, *sizes) -> int:
    """Workspace bytes for these sizes (the fields from num_tokens on) on this device."""
    a = CrossAttentionArgs(*([256] * 8), None, *sizes, 0.0)
    return pkv_cross_attention_workspace_size(a)


_OWN = threading.local()   # (device, raw stream) -> workspace, the last used one last
_OWN_STREAMS = 4


def _own_workspace(need: int, like, stream, raw: int):
    """A workspace for a call that brought none. Each thread keeps one for each of the last
    ``_OWN_STREAMS`` streams that it called on as the current one (an allocation costs a call
    6 us): calls of one thread on one stream run one after the other. One takes up to 61 MB on
    a GPU of 152 SMs, as much as its largest call needed, until the thread ends, has called on
    as many other streams, or calls release_workspaces. A call that is captured gets memory of
    its graph's, one on another stream than the current one its own."""
    torch = _torch()
    if stream is not None or torch.cuda.is_current_stream_capturing():
        return _made(stream, need, torch.uint8, like.device, returned=False)
    kept = _OWN.__dict__
    key = (like.get_device(), raw)
    own = kept.pop(key, None)
    if own is None or own.numel() < need:
        own = None   # its memory may serve the new one
        own = torch.empty(need, dtype=torch.uint8, device=like.device)
    kept[key] = own
    if len(kept) > _OWN_STREAMS:
        del kept[next(iter(kept))]
    return own


def release_workspaces():
    """Gives back the workspaces that pkv_cross_attention keeps for the calling thread (memory
    of torch's caching allocator; calls under way finish undisturbed)."""
    _OWN.__dict__.clear()


def pkv_cross_attention(query, key_cache, value_cache, cumulative_sequence_length,
                        key_seqlens, block_table, *, num_heads: int, kv_num_heads: int,
                        max_query_len: int = 0, scale: float = 0.0, output=None, lse=None,
                        workspace=None, device_status=None, stream=None):
    """Attention of ragged query rows over encoder states in a paged cache: row i of
    sequence b sees the key_seqlens[b] states of table row b. float16 or bfloat16. Returns
    the output [num_tokens, num_heads * head_size]; with ``lse`` (float32 [num_tokens,
    num_heads]) the log-sum-exp of each row's scores is written there. Without a ``workspace``
    (uint8, 256-byte aligned) of at least pkv_cross_attention_workspace_size bytes one of up to
    61 MB is kept for the calling thread and stream (see _own_workspace, release_workspaces)."""
    torch = _torch()
    if (query is None or key_cache is None or value_cache is None or block_table is None or
            cumulative_sequence_length is None or key_seqlens is None):
        _need(query=query, key_cache=key_cache, value_cache=value_cache,
              cumulative_sequence_length=cumulative_sequence_length, key_seqlens=key_seqlens,
              block_table=block_table)
    dt, i32 = query.dtype, torch.int32
    if dt is torch.float16:
        code = PKV_F16
    elif dt is torch.bfloat16:
        code = PKV_BF16
    else:
        raise TypeError(f"query: expected float16 or bfloat16, got {dt}")
    if key_cache.dim() != 4:
        raise ValueError("key_cache: [num_blocks, block_size, kv_num_heads, head_size]")
    NB, BS, _, D = key_cache.shape
    T = query.shape[0] if query.dim() == 2 else -1
    B = key_seqlens.shape[0] if key_seqlens.dim() == 1 else -1
    MB = block_table.shape[1] if block_table.dim() == 2 else -1
    hidden, pool = (T, num_heads * D), (NB, BS, kv_num_heads, D)
    raw = _check_tensors(stream, (
        ("query", query, dt, hidden), ("output", output, dt, hidden),
        ("key_cache", key_cache, dt, pool), ("value_cache", value_cache, dt, pool),
        ("key_seqlens", key_seqlens, i32, (B,)),
        ("cumulative_sequence_length", cumulative_sequence_length, i32, (B + 1,)),
        ("block_table", block_table, i32, (B, MB)),
        ("lse", lse, torch.float32, (T, num_heads)),
        ("workspace", workspace, torch.uint8, None if workspace is None else workspace.shape),
        ("device_status", device_status, i32, (1,))))
    if output is None:
        output = _made(stream, hidden, dt, query.device)
    sizes = (T, B, num_heads, kv_num_heads, D, BS, NB, MB, max_query_len, code)
    need = _cross_workspace(query.get_device(), *sizes)
    if need and (workspace is None or workspace.numel() < need):
        workspace = _own_workspace(need, query, stream, raw)
    _step_call("pkv_cross_attention",
               _CROSS_PACK.pack(query.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
                                cumulative_sequence_length.data_ptr(), key_seqlens.data_ptr(),
                                block_table.data_ptr(), output.data_ptr(), _at(lse),
                                _at(device_status), *sizes, scale),
               _at(workspace), need, raw)
    return output


# ----------------------------------------------------------------------------- runtime
def pkv_launch_count() -> int:
    return int(load_library().pkv_launch_count())


def pkv_profiler_enable(on: bool = True):
    load_library().pkv_profiler_enable(1 if on else 0)


def pkv_profiler_reset():
    load_library().pkv_profiler_reset()


def pkv_profiler_query(kernel: str):
    """(total_ms, launches) of one kernel family since the last reset."""
    ms = ctypes.c_double(0.0)
    n = c_i64(0)
    _check("pkv_profiler_query",
           load_library().pkv_profiler_query(kernel.encode(), ctypes.byref(ms), ctypes.byref(n)))
    return float(ms.value), int(n.value)


def pkv_testing_wait_limit(max_polls: int = 0, withhold_first_copy: bool = False):
    """Testing hook of the tensor-core kernels' bounded waits (see pagedkv.h): a lower
    poll bound and, optionally, a withheld first bulk copy per CTA so that a wait gives
    up. pkv_testing_wait_limit() restores the defaults."""
    _check("pkv_testing_wait_limit",
           load_library().pkv_testing_wait_limit(int(max_polls), 1 if withhold_first_copy else 0))


def pkv_paged_attention_static_workspace(query, key, value, key_cache, value_cache,
                                         cumulative_sequence_length, past_seqlens,
                                         block_table, slot_mapping=None, *, num_heads: int,
                                         kv_num_heads: int, scale: float = 0.0,
                                         output, device_status=None, stream=None, **kw):
    """Paged attention for callers that may not allocate device memory: scratch comes
    from the library's fixed device array (PKV_STATIC_WORKSPACE_BYTES per GPU), so this
    call allocates nothing, not even the output, which the caller passes in. Calls that
    overlap on the GPU share that array and must be serialised."""
    lib = load_library()
    fn = lib.pkv_paged_attention_static_workspace
    fn.restype = c_i32
    fn.argtypes = [ctypes.POINTER(PagedAttentionArgs), c_vp]
    a = make_paged_args(query, key, value, key_cache, value_cache,
                        cumulative_sequence_length, past_seqlens, block_table, slot_mapping,
                        output, num_heads=num_heads, kv_num_heads=kv_num_heads, scale=scale,
                        device_status=device_status, **kw)
    _check("pkv_paged_attention_static_workspace", fn(ctypes.byref(a), _stream(stream)))
    return output
