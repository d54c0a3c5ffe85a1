"""GB300-native batched speculative-sampling verification.

Thin Python binding over the C ABI of ``libspecverify.so`` (declared in
``include/spec_verify.h``, ``include/spec_sample.h``,
``include/spec_lmhead.h``, ``include/spec_tree.h``, ``include/spec_attn.h``,
``include/spec_logits.h``, ``include/spec_chunk.h``, ``include/spec_beam.h``
and ``include/spec_pages.h``).  Every function here only checks and marshals
arguments (shapes, dtypes, device pointers, the current CUDA stream) and calls
the function of the same name in the library; all arithmetic runs in the CUDA
kernels.  PyTorch is used for device memory and streams only.

If the library has not been built the first call raises: there is no CPU
fallback.  Build it with ``__graft_entry__.build()`` (or
``python -m speculative_decoding_verification_65_gb300.build``).
"""
from __future__ import annotations

import ctypes
import functools
import importlib
import math
import os
import struct
import threading

SPEC_F32 = 0
SPEC_BF16 = 1
SPEC_F16 = 2  # attention and appends to the cache only
SPEC_OK = 0
SPEC_EINVAL = 1
SPEC_ECUDA = 2
SPEC_ENOSPACE = 3
SPEC_DEV_OK = 0
SPEC_DEV_WAIT_TIMEOUT = 1
SPEC_MAX_K = 32
SPEC_MAX_V = 1 << 20
SPEC_STAGES = 5
SPEC_SAMPLE_STAGES = 3
SPEC_FILTERED_STAGES = 6
SPEC_LMHEAD_STAGES = 5
SPEC_TREE_MAX_NODES = 1024
SPEC_ATTN_MAX_NODES = 1024
SPEC_ATTN_MAX_HEAD_DIM = 128
SPEC_PLAN_POSITIONS, SPEC_PLAN_STATUS, SPEC_PLAN_MASK = 0, 1, 2
SPEC_LOGITS_MAX_ROWS = 1024
SPEC_LOGITS_MAX_BIAS = 4096
SPEC_CHUNK_MAX_ROWS = 1 << 24
SPEC_BEAM_MAX = 64
SPEC_PAGES_MAX = 1 << 24

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")
_lib = None
_lock = threading.Lock()


class SpecVerifyError(RuntimeError):
    pass


class _AttentionArgs(ctypes.Structure):
    """spec_tree_attention_args (include/spec_attn.h)."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k_new", "v_new", "k_cache", "v_cache")]
                + [(n + "_stride", ctypes.c_int64 * 3)
                   for n in ("q", "k_new", "v_new", "k_cache", "v_cache")]
                + [(n, ctypes.c_void_p) for n in ("page_table", "plan", "out", "out_lse")]
                + [("scale", ctypes.c_float)]
                + [(n, ctypes.c_int32) for n in ("B", "N", "Hq", "Hkv", "D", "page_size",
                                                 "pages_per_seq", "num_pages", "dtype")])


class _CommitArgs(ctypes.Structure):
    """spec_tree_commit_args (include/spec_attn.h)."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k_new", "v_new", "k_cache", "v_cache")]
                + [(n + "_stride", ctypes.c_int64 * 4)
                   for n in ("k_new", "v_new", "k_cache", "v_cache")]
                + [(n, ctypes.c_void_p) for n in ("cache_len", "out_num_accepted", "out_nodes",
                                                  "page_table", "out_len")]
                + [(n, ctypes.c_int32) for n in ("layers", "B", "N", "Hkv", "D", "page_size",
                                                 "pages_per_seq", "num_pages", "elem_size")])


class _LogitsArgs(ctypes.Structure):
    """spec_process_logits_args (include/spec_logits.h)."""
    _fields_ = ([(n, ctypes.c_void_p) for n in (
                    "logits", "out", "history", "history_len", "prompt_len", "draft_tokens",
                    "parent", "n_nodes", "repetition", "frequency", "presence", "bias_tokens",
                    "bias_values", "allowed")]
                + [(n, ctypes.c_int64) for n in ("allowed_stride_b", "allowed_stride_r")]
                + [(n, ctypes.c_int32) for n in ("B", "R", "V", "H", "draft_cols", "bias_cols",
                                                 "dtype")])


class _AppendArgs(ctypes.Structure):
    """spec_chunk_append_args (include/spec_chunk.h)."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k_new", "v_new", "k_cache", "v_cache")]
                + [(n + "_stride", ctypes.c_int64 * 3) for n in ("k_new", "v_new")]
                + [(n + "_stride", ctypes.c_int64 * 4) for n in ("k_cache", "v_cache")]
                + [(n, ctypes.c_void_p) for n in ("row_start", "cache_len", "page_table",
                                                  "out_len")]
                + [(n, ctypes.c_int32) for n in ("layers", "B", "rows", "Hkv", "D", "page_size",
                                                 "pages_per_seq", "num_pages", "elem_size")])


class _ChunkArgs(ctypes.Structure):
    """spec_chunk_attention_args (include/spec_chunk.h)."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k_cache", "v_cache")]
                + [("q_stride", ctypes.c_int64 * 2)]
                + [(n + "_stride", ctypes.c_int64 * 3) for n in ("k_cache", "v_cache")]
                + [(n, ctypes.c_void_p) for n in ("page_table", "plan", "out", "out_lse")]
                + [("scale", ctypes.c_float)]
                + [(n, ctypes.c_int32) for n in ("B", "rows", "Hq", "Hkv", "D", "page_size",
                                                 "pages_per_seq", "num_pages", "dtype")])


class _BeamArgs(ctypes.Structure):
    """spec_beam_select_args (include/spec_beam.h)."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("logits", "scores", "norm", "finished",
                                                "out_tokens", "out_beams", "out_scores")]
                + [(n, ctypes.c_int32) for n in ("B", "K", "V", "n", "end_token", "dtype")])


class _ForkArgs(ctypes.Structure):
    """spec_pages_fork_args (include/spec_pages.h)."""
    _fields_ = ([(n, ctypes.c_void_p) for n in (
                    "table_in", "length_in", "parent", "reserve", "ref_in", "table_out",
                    "length_out", "ref_out", "copies")]
                + [(n, ctypes.c_int32) for n in ("rows_in", "rows_out", "pages_per_seq",
                                                 "page_size", "num_pages")])


class _CompactArgs(ctypes.Structure):
    """spec_pages_compact_args (include/spec_pages.h)."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("table_in", "ref_in", "table_out", "ref_out",
                                                "copies", "used")]
                + [(n, ctypes.c_int32) for n in ("rows", "pages_per_seq", "page_size",
                                                 "num_pages")])


class _CopyArgs(ctypes.Structure):
    """spec_pages_copy_args (include/spec_pages.h)."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k_cache", "v_cache")]
                + [(n + "_stride", ctypes.c_int64 * 4) for n in ("k_cache", "v_cache")]
                + [("copies", ctypes.c_void_p)]
                + [(n, ctypes.c_int32) for n in ("n", "layers", "Hkv", "D", "page_size",
                                                 "num_pages", "elem_size")])


# The same structures packed in one go (the binding's own calls: filling a
# ctypes structure field by field costs more than the smallest kernels).
_pack_attention = struct.Struct("@5Q15q4Qf9i").pack
_pack_commit = struct.Struct("@4Q16q5Q9i4x").pack
_pack_logits = struct.Struct("@14Q2q7i4x").pack
_pack_chunk = struct.Struct("@4Qf").pack
_pack_beam = struct.Struct("@7Q").pack


def library():
    """The loaded ctypes library (raises if it was never built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise SpecVerifyError(
                f"{LIB_PATH} is missing: build the CUDA library first "
                "(__graft_entry__.build()); there is no fallback")
        lib = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        lib.spec_verify_abi_version.restype = i32
        lib.spec_verify_abi_version.argtypes = []
        lib.spec_verify_strerror.restype = ctypes.c_char_p
        lib.spec_verify_strerror.argtypes = [i32]
        lib.spec_verify_workspace_size.restype = sz
        lib.spec_verify_workspace_size.argtypes = [i32, i32, i32, i32]
        lib.spec_verify_workspace_reset.restype = i32
        lib.spec_verify_workspace_reset.argtypes = [vp, sz, vp]
        lib.spec_verify.restype = i32
        lib.spec_verify.argtypes = [vp] * 8 + [i32] * 4 + [vp, sz, vp]
        lib.spec_verify_probs.restype = i32
        lib.spec_verify_probs.argtypes = [vp] * 9 + [i32] * 4 + [vp, sz, vp]
        lib.spec_verify_trace.restype = i32
        lib.spec_verify_trace.argtypes = [vp] * 10 + [i32] * 5 + [vp, sz, vp]
        lib.spec_verify_timed.restype = i32
        lib.spec_verify_timed.argtypes = [vp] * 8 + [i32] * 4 + [vp, sz, vp, vp]
        lib.spec_verify_filtered.restype = i32
        lib.spec_verify_filtered.argtypes = [vp] * 11 + [i32] * 4 + [vp, sz, vp]
        lib.spec_verify_filtered_timed.restype = i32
        lib.spec_verify_filtered_timed.argtypes = [vp] * 10 + [i32] * 4 + [vp, sz, vp, vp]
        lib.spec_verify_noalloc.restype = i32
        lib.spec_verify_noalloc.argtypes = [vp] * 8 + [i32] * 4 + [vp]
        lib.spec_verify_noalloc_max_bytes.restype = sz
        lib.spec_verify_noalloc_max_bytes.argtypes = []
        lib.spec_verify_read_status.restype = i32
        lib.spec_verify_read_status.argtypes = [vp, vp, vp]
        lib.spec_verify_host_arena_size.restype = sz
        lib.spec_verify_host_arena_size.argtypes = [i32, i32, i32, i32]
        lib.spec_verify_host.restype = i32
        lib.spec_verify_host.argtypes = [vp] * 8 + [i32] * 4 + [vp, sz, vp]
        lib.spec_sample_workspace_size.restype = sz
        lib.spec_sample_workspace_size.argtypes = [i32, i32, i32]
        lib.spec_sample.restype = i32
        lib.spec_sample.argtypes = [vp] * 4 + [i32] * 3 + [vp, sz, vp]
        lib.spec_sample_timed.restype = i32
        lib.spec_sample_timed.argtypes = [vp] * 4 + [i32] * 3 + [vp, sz, vp, vp]
        lib.spec_sample_host_arena_size.restype = sz
        lib.spec_sample_host_arena_size.argtypes = [i32, i32, i32]
        lib.spec_sample_host.restype = i32
        lib.spec_sample_host.argtypes = [vp] * 4 + [i32] * 3 + [vp, sz, vp]
        lib.spec_bench_read.restype = i32
        lib.spec_bench_read.argtypes = [vp, sz, vp, vp]
        lib.spec_bench_read_sink_words.restype = i32
        lib.spec_bench_read_sink_words.argtypes = []
        lib.spec_selftest_wait_timeout.restype = i32
        lib.spec_selftest_wait_timeout.argtypes = [vp, ctypes.c_uint64, vp]
        lib.spec_selftest_wait_timeout_noalloc.restype = i32
        lib.spec_selftest_wait_timeout_noalloc.argtypes = [ctypes.c_uint64, vp]
        lib.spec_verify_noalloc_read_status.restype = i32
        lib.spec_verify_noalloc_read_status.argtypes = [vp, vp]
        lib.spec_verify_lmhead_workspace_size.restype = sz
        lib.spec_verify_lmhead_workspace_size.argtypes = [i32] * 5
        lib.spec_verify_lmhead.restype = i32
        lib.spec_verify_lmhead.argtypes = [vp] * 9 + [i32] * 5 + [vp, sz, vp]
        lib.spec_verify_lmhead_timed.restype = i32
        lib.spec_verify_lmhead_timed.argtypes = [vp] * 10 + [i32] * 5 + [vp, sz, vp, vp]
        lib.spec_lmhead_logits.restype = i32
        lib.spec_lmhead_logits.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp]
        lib.spec_verify_filtered_workspace_size.restype = sz
        lib.spec_verify_filtered_workspace_size.argtypes = [i32, i32, i32, i32]
        lib.spec_verify_tree.restype = i32
        lib.spec_verify_tree.argtypes = [vp] * 11 + [i32] * 4 + [vp]
        lib.spec_tree_plan_size.restype = sz
        lib.spec_tree_plan_size.argtypes = [i32, i32]
        lib.spec_tree_plan_offset.restype = sz
        lib.spec_tree_plan_offset.argtypes = [i32] * 3
        lib.spec_tree_plan.restype = i32
        lib.spec_tree_plan.argtypes = [vp] * 4 + [i32] * 5 + [vp, sz, vp]
        lib.spec_tree_attention_workspace_size.restype = sz
        lib.spec_tree_attention_workspace_size.argtypes = [i32] * 4
        lib.spec_tree_attention.restype = i32
        lib.spec_tree_attention.argtypes = [vp, vp, sz, vp]
        lib.spec_selftest_attention_timeout.restype = i32
        lib.spec_selftest_attention_timeout.argtypes = [vp, vp, sz, i32, i32, vp]
        lib.spec_selftest_chunk_timeout.restype = i32
        lib.spec_selftest_chunk_timeout.argtypes = [vp, vp, sz, i32, i32, vp]
        lib.spec_tree_commit.restype = i32
        lib.spec_tree_commit.argtypes = [vp, vp]
        lib.spec_process_logits.restype = i32
        lib.spec_process_logits.argtypes = [vp, vp]
        lib.spec_chunk_append.restype = i32
        lib.spec_chunk_append.argtypes = [vp, vp]
        for name in ("spec_chunk_plan_size", "spec_chunk_plan_status",
                     "spec_chunk_attention_workspace_size"):
            getattr(lib, name).restype = sz
            getattr(lib, name).argtypes = [i32] * 3
        lib.spec_chunk_plan.restype = i32
        lib.spec_chunk_plan.argtypes = [vp] * 3 + [i32] * 6 + [vp, sz, vp]
        lib.spec_beam_workspace_size.restype = sz
        lib.spec_beam_workspace_size.argtypes = [i32] * 5
        lib.spec_pages_workspace_size.restype = sz
        lib.spec_pages_workspace_size.argtypes = [i32] * 2
        for name in ("spec_chunk_attention", "spec_beam_select", "spec_pages_fork",
                     "spec_pages_compact"):
            getattr(lib, name).restype = i32
            getattr(lib, name).argtypes = [vp, vp, sz, vp]
        lib.spec_beam_reorder.restype = i32
        lib.spec_beam_reorder.argtypes = [vp] * 3 + [i32] * 4 + [ctypes.c_int64, vp]
        lib.spec_pages_copy.restype = i32
        lib.spec_pages_copy.argtypes = [vp, vp]
        _lib = lib
        return lib


def _check(rc: int, what: str):
    if rc != SPEC_OK:
        msg = library().spec_verify_strerror(rc).decode()
        raise SpecVerifyError(f"{what} failed: {msg} (status {rc})")


def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return SPEC_F32
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _on(device):
    """The library takes the device from the CUDA runtime's current device, so
    every call is made with the tensors' device current."""
    return _torch().cuda.device(device)


def _stream_handle(stream, device):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def spec_verify_abi_version() -> int:
    return int(library().spec_verify_abi_version())


def spec_verify_workspace_size(B: int, k: int, V: int, dtype: int) -> int:
    return int(library().spec_verify_workspace_size(B, k, V, dtype))


def spec_verify_host_arena_size(B: int, k: int, V: int, dtype: int) -> int:
    return int(library().spec_verify_host_arena_size(B, k, V, dtype))


class _Workspaces(threading.local):
    """One host thread's workspaces by (device, stream).  Calls on a stream run in
    order, but a call is several kernels, and another thread's may come between them."""

    def __init__(self):
        self.of = {}


_ws_cache = _Workspaces()


def workspace(B: int, k: int, V: int, dtype: int, device=None, stream=None):
    """A zeroed workspace tensor big enough for these sizes, cached per
    (host thread, device, stream): a thread's calls in flight on one stream run
    in order, so they can share it."""
    torch = _torch()
    device = torch.device(device if device is not None else "cuda")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    s = stream if stream is not None else torch.cuda.current_stream(device)
    need = spec_verify_workspace_size(B, k, V, dtype)
    if need == 0:
        raise ValueError(f"sizes out of range: B={B} k={k} V={V} dtype={dtype}")
    return _cached_workspace(need, device, s)


def spec_verify_filtered_workspace_size(B: int, k: int, V: int, dtype: int) -> int:
    return int(library().spec_verify_filtered_workspace_size(B, k, V, dtype))


def filtered_workspace(B: int, k: int, V: int, dtype: int, device=None, stream=None):
    """workspace() with room for the top-k cut from group maxima
    (spec_verify_filtered_workspace_size)."""
    torch = _torch()
    device = torch.device(device if device is not None else "cuda")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    s = stream if stream is not None else torch.cuda.current_stream(device)
    need = spec_verify_filtered_workspace_size(B, k, V, dtype)
    if need == 0:
        raise ValueError(f"sizes out of range: B={B} k={k} V={V} dtype={dtype}")
    return _cached_workspace(need, device, s)


def _cached_workspace(need: int, device, s):
    torch = _torch()
    key = (device.index, s.cuda_stream)
    ws = _ws_cache.of.get(key)
    if ws is None or ws.numel() < need:
        with torch.cuda.stream(s):
            ws = torch.zeros(max(need, 1 << 20), dtype=torch.uint8, device=device)
        _ws_cache.of[key] = ws
    return ws


def spec_verify_workspace_reset(ws, stream=None):
    with _on(ws.device):
        _check(library().spec_verify_workspace_reset(_ptr(ws), ws.numel(),
                                                     _stream_handle(stream, ws.device)),
               "spec_verify_workspace_reset")


def spec_verify_read_status(ws, stream=None) -> int:
    st = ctypes.c_int32(-99)
    with _on(ws.device):
        _check(library().spec_verify_read_status(_ptr(ws), ctypes.byref(st),
                                                 _stream_handle(stream, ws.device)),
               "spec_verify_read_status")
    return int(st.value)


def _shapes(target, draft, tokens, u_accept, u_resample, temperature):
    """Shapes and dtypes of the verification inputs: (B, k, V, dtype code)."""
    torch = _torch()
    if target.dim() != 3 or draft.dim() != 3:
        raise ValueError("target must be [B,k+1,V] and draft [B,k,V]")
    B, k1, V = target.shape
    k = k1 - 1
    if tuple(draft.shape) != (B, k, V):
        raise ValueError(f"draft shape {tuple(draft.shape)} != {(B, k, V)}")
    dt = _dtype_code(target)
    if draft.dtype != target.dtype:
        raise TypeError("target and draft must share a dtype")
    for name, t, shape, dtype in (("draft_tokens", tokens, (B, k), torch.int32),
                                  ("u_accept", u_accept, (B, k), torch.float32),
                                  ("u_resample", u_resample, (B,), torch.float32),
                                  ("temperature", temperature, (B,), torch.float32)):
        if tuple(t.shape) != shape or t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")
    return B, k, V, dt


def _check_out(name, t, shape, dtype):
    if tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {shape} tensor, "
                         f"got {t.dtype} {tuple(t.shape)}")


def _dev_out(name, t, shape, dtype, dev):
    """A caller-supplied output: contiguous, of the call's shape and dtype, on
    the inputs' device (the kernels write every element of it)."""
    _check_out(name, t, shape, dtype)
    if not t.is_cuda or t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")


def _check_ws(ws, dev):
    torch = _torch()
    if not ws.is_cuda or ws.device != dev or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous uint8 tensor on {dev}")


def _marshal(target, draft, tokens, u_accept, u_resample, temperature):
    B, k, V, dt = _shapes(target, draft, tokens, u_accept, u_resample, temperature)
    for t in (target, draft, tokens, u_accept, u_resample, temperature):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("all inputs must be contiguous CUDA tensors")
        if t.device != target.device:
            raise ValueError("all inputs must be on one device")
    return B, k, V, dt


def spec_verify(target, draft, tokens, u_accept, u_resample, temperature,
                out_tokens=None, out_num_accepted=None, ws=None, stream=None):
    """Run the verification step on the current (or given) stream.

    target [B,k+1,V] and draft [B,k,V]: float32 or bfloat16 CUDA tensors;
    tokens int32 [B,k]; u_accept float32 [B,k]; u_resample, temperature
    float32 [B].  Returns (out_tokens int32 [B,k+1], out_num_accepted int32
    [B]); asynchronous like any CUDA op."""
    torch = _torch()
    B, k, V, dt = _marshal(target, draft, tokens, u_accept, u_resample, temperature)
    dev = target.device
    if out_tokens is None:
        out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    if out_num_accepted is None:
        out_num_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    _dev_out("out_tokens", out_tokens, (B, k + 1), torch.int32, dev)
    _dev_out("out_num_accepted", out_num_accepted, (B,), torch.int32, dev)
    if ws is None:
        ws = workspace(B, k, V, dt, dev, stream)
    _check_ws(ws, dev)
    with _on(dev):
        rc = library().spec_verify(_ptr(target), _ptr(draft), _ptr(tokens), _ptr(u_accept),
                                   _ptr(u_resample), _ptr(temperature), _ptr(out_tokens),
                                   _ptr(out_num_accepted), B, k, V, dt, _ptr(ws), ws.numel(),
                                   _stream_handle(stream, dev))
    _check(rc, "spec_verify")
    return out_tokens, out_num_accepted


def _filters(B, dev, top_k, top_p):
    torch = _torch()
    for name, t, dtype in (("top_k", top_k, torch.int32), ("top_p", top_p, torch.float32)):
        if t is not None and (tuple(t.shape) != (B,) or t.dtype != dtype or not t.is_cuda
                              or not t.is_contiguous() or t.device != dev):
            raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape ({B},)")


def spec_verify_filtered(target, draft, tokens, u_accept, u_resample, temperature,
                         top_k=None, top_p=None, out_tokens=None, out_num_accepted=None,
                         want_probs=False, ws=None, stream=None):
    """spec_verify with top-k / top-p filtered distributions (see
    include/spec_verify.h): top_k int32 [B] (0 = none), top_p float32 [B]
    (>= 1 = none), either may be None.  Returns (out_tokens, out_num_accepted)
    and, with want_probs, the filtered P, Q [B, k, 2] as a third value."""
    torch = _torch()
    B, k, V, dt = _marshal(target, draft, tokens, u_accept, u_resample, temperature)
    dev = target.device
    _filters(B, dev, top_k, top_p)
    if out_tokens is None:
        out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    if out_num_accepted is None:
        out_num_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    _dev_out("out_tokens", out_tokens, (B, k + 1), torch.int32, dev)
    _dev_out("out_num_accepted", out_num_accepted, (B,), torch.int32, dev)
    probs = torch.empty((B, k, 2), dtype=torch.float32, device=dev) if want_probs else None
    if ws is None:
        ws = filtered_workspace(B, k, V, dt, dev, stream)
    _check_ws(ws, dev)
    with _on(dev):
        rc = library().spec_verify_filtered(_ptr(target), _ptr(draft), _ptr(tokens), _ptr(u_accept),
                                            _ptr(u_resample), _ptr(temperature), _ptr(top_k),
                                            _ptr(top_p), _ptr(out_tokens), _ptr(out_num_accepted),
                                            _ptr(probs), B, k, V, dt, _ptr(ws), ws.numel(),
                                            _stream_handle(stream, dev))
    _check(rc, "spec_verify_filtered")
    if want_probs:
        return out_tokens, out_num_accepted, probs
    return out_tokens, out_num_accepted


def spec_verify_filtered_timed(target, draft, tokens, u_accept, u_resample, temperature,
                               top_k, top_p, out_tokens, out_num_accepted, ws, stage_events,
                               stream=None):
    """spec_verify_filtered recording SPEC_FILTERED_STAGES events: after the
    statistics, the filter (all of its kernels), the accept scan, the draw
    tiles, the final search and the exact draws."""
    torch = _torch()
    B, k, V, dt = _marshal(target, draft, tokens, u_accept, u_resample, temperature)
    dev = target.device
    _filters(B, dev, top_k, top_p)
    _dev_out("out_tokens", out_tokens, (B, k + 1), torch.int32, dev)
    _dev_out("out_num_accepted", out_num_accepted, (B,), torch.int32, dev)
    _check_ws(ws, dev)
    handles = (ctypes.c_void_p * SPEC_FILTERED_STAGES)(
        *[ctypes.c_void_p(e.cuda_event) for e in stage_events])
    with _on(target.device):
        rc = library().spec_verify_filtered_timed(
            _ptr(target), _ptr(draft), _ptr(tokens), _ptr(u_accept), _ptr(u_resample),
            _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(out_tokens), _ptr(out_num_accepted),
            B, k, V, dt, _ptr(ws), ws.numel(), _stream_handle(stream, target.device), handles)
    _check(rc, "spec_verify_filtered_timed")
    return out_tokens, out_num_accepted


def spec_verify_timed(target, draft, tokens, u_accept, u_resample, temperature,
                      out_tokens, out_num_accepted, ws, stage_events, stream=None):
    """spec_verify recording the given torch.cuda.Event objects (SPEC_STAGES of
    them, recorded once beforehand so that they exist) after each stage:
    statistics, accept scan, draw tiles, final search, exact draws."""
    torch = _torch()
    B, k, V, dt = _marshal(target, draft, tokens, u_accept, u_resample, temperature)
    dev = target.device
    _dev_out("out_tokens", out_tokens, (B, k + 1), torch.int32, dev)
    _dev_out("out_num_accepted", out_num_accepted, (B,), torch.int32, dev)
    _check_ws(ws, dev)
    handles = (ctypes.c_void_p * SPEC_STAGES)(*[ctypes.c_void_p(e.cuda_event) for e in stage_events])
    with _on(target.device):
        rc = library().spec_verify_timed(_ptr(target), _ptr(draft), _ptr(tokens), _ptr(u_accept),
                                         _ptr(u_resample), _ptr(temperature), _ptr(out_tokens),
                                         _ptr(out_num_accepted), B, k, V, dt, _ptr(ws), ws.numel(),
                                         _stream_handle(stream, target.device), handles)
    _check(rc, "spec_verify_timed")
    return out_tokens, out_num_accepted


def spec_verify_noalloc(target, draft, tokens, u_accept, u_resample, temperature,
                        out_tokens, out_num_accepted, stream=None):
    """spec_verify without a workspace, for callers that cannot allocate device
    memory when they verify: the library's own fixed scratch array is used
    instead (see include/spec_verify.h).  The output tensors are supplied by
    the caller, so this wrapper allocates nothing either.  Calls that overlap
    on the GPU share that scratch and race."""
    torch = _torch()
    B, k, V, dt = _marshal(target, draft, tokens, u_accept, u_resample, temperature)
    _dev_out("out_tokens", out_tokens, (B, k + 1), torch.int32, target.device)
    _dev_out("out_num_accepted", out_num_accepted, (B,), torch.int32, target.device)
    with _on(target.device):
        rc = library().spec_verify_noalloc(_ptr(target), _ptr(draft), _ptr(tokens), _ptr(u_accept),
                                           _ptr(u_resample), _ptr(temperature), _ptr(out_tokens),
                                           _ptr(out_num_accepted), B, k, V, dt,
                                           _stream_handle(stream, target.device))
    _check(rc, "spec_verify_noalloc")
    return out_tokens, out_num_accepted


def spec_verify_noalloc_read_status(stream=None, device=None) -> int:
    """The device status word of spec_verify_noalloc's scratch (SPEC_DEV_*)."""
    torch = _torch()
    dev = torch.device(device if device is not None else "cuda")
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    st = ctypes.c_int32(-99)
    with torch.cuda.device(dev):
        _check(library().spec_verify_noalloc_read_status(ctypes.byref(st),
                                                         _stream_handle(stream, dev)),
               "spec_verify_noalloc_read_status")
    return int(st.value)


def spec_selftest_wait_timeout_noalloc(limit_ns: int, stream=None, device=None):
    """spec_selftest_wait_timeout on spec_verify_noalloc's scratch."""
    torch = _torch()
    dev = torch.device(device if device is not None else "cuda")
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        _check(library().spec_selftest_wait_timeout_noalloc(int(limit_ns),
                                                            _stream_handle(stream, dev)),
               "spec_selftest_wait_timeout_noalloc")


def spec_verify_noalloc_max_bytes() -> int:
    return int(library().spec_verify_noalloc_max_bytes())


def spec_verify_probs(target, draft, tokens, u_accept, u_resample, temperature,
                      ws=None, stream=None):
    """spec_verify plus the fp32 intermediates P = p_i(g_i), Q = q_i(g_i):
    returns (out_tokens, out_num_accepted, probs [B,k,2])."""
    torch = _torch()
    B, k, V, dt = _marshal(target, draft, tokens, u_accept, u_resample, temperature)
    dev = target.device
    out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    out_n = torch.empty((B,), dtype=torch.int32, device=dev)
    probs = torch.empty((B, k, 2), dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(B, k, V, dt, dev, stream)
    _check_ws(ws, dev)
    with _on(dev):
        rc = library().spec_verify_probs(_ptr(target), _ptr(draft), _ptr(tokens), _ptr(u_accept),
                                         _ptr(u_resample), _ptr(temperature), _ptr(out_tokens),
                                         _ptr(out_n), _ptr(probs), B, k, V, dt, _ptr(ws),
                                         ws.numel(), _stream_handle(stream, dev))
    _check(rc, "spec_verify_probs")
    return out_tokens, out_n, probs


def spec_verify_trace(target, draft, tokens, u_accept, u_resample, temperature,
                      resolve_all=False, want_probs=False, ws=None, stream=None):
    """spec_verify with the trace of each draw (include/spec_verify.h):
    returns (out_tokens, out_num_accepted, draw [B,4] int32, probs or None).
    draw[b] = (fp32 token, listed for the exact draw, token written, the fp32
    distance of u to its cell's nearer edge as float32 bits);
    sequences that draw nothing keep -2 everywhere.  resolve_all lists every
    draw."""
    torch = _torch()
    B, k, V, dt = _marshal(target, draft, tokens, u_accept, u_resample, temperature)
    dev = target.device
    out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    out_n = torch.empty((B,), dtype=torch.int32, device=dev)
    draw = torch.full((B, 4), -2, dtype=torch.int32, device=dev)
    probs = torch.empty((B, k, 2), dtype=torch.float32, device=dev) if want_probs else None
    if ws is None:
        ws = workspace(B, k, V, dt, dev, stream)
    _check_ws(ws, dev)
    with _on(dev):
        rc = library().spec_verify_trace(_ptr(target), _ptr(draft), _ptr(tokens), _ptr(u_accept),
                                         _ptr(u_resample), _ptr(temperature), _ptr(out_tokens),
                                         _ptr(out_n), _ptr(probs), _ptr(draw),
                                         1 if resolve_all else 0, B, k, V, dt, _ptr(ws),
                                         ws.numel(), _stream_handle(stream, dev))
    _check(rc, "spec_verify_trace")
    return out_tokens, out_n, draw, probs


def spec_verify_host(target, draft, tokens, u_accept, u_resample, temperature,
                     arena, out_tokens=None, out_num_accepted=None, stream=None):
    """End-to-end call on HOST tensors (CPU, ideally pinned): the library copies
    the inputs into the device `arena` (a CUDA uint8 tensor of at least
    spec_verify_host_arena_size bytes), verifies, copies the outputs back and
    synchronises.  Returns host (out_tokens, out_num_accepted)."""
    torch = _torch()
    B, k, V, dt = _shapes(target, draft, tokens, u_accept, u_resample, temperature)
    for t in (target, draft, tokens, u_accept, u_resample, temperature):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("host inputs must be contiguous CPU tensors")
    if not arena.is_cuda or arena.dtype != torch.uint8 or not arena.is_contiguous():
        raise ValueError("arena must be a contiguous uint8 CUDA tensor")
    for name, t, shape in (("out_tokens", out_tokens, (B, k + 1)),
                           ("out_num_accepted", out_num_accepted, (B,))):
        if t is not None:
            _check_out(name, t, shape, torch.int32)
            if t.is_cuda:
                raise ValueError(f"{name} must be a host tensor")
    if out_tokens is None:
        out_tokens = torch.empty((B, k + 1), dtype=torch.int32, pin_memory=True)
    if out_num_accepted is None:
        out_num_accepted = torch.empty((B,), dtype=torch.int32, pin_memory=True)
    with _on(arena.device):
        rc = library().spec_verify_host(_ptr(target), _ptr(draft), _ptr(tokens), _ptr(u_accept),
                                        _ptr(u_resample), _ptr(temperature), _ptr(out_tokens),
                                        _ptr(out_num_accepted), B, k, V, dt, _ptr(arena),
                                        arena.numel(), _stream_handle(stream, arena.device))
    _check(rc, "spec_verify_host")
    return out_tokens, out_num_accepted


def spec_sample_workspace_size(R: int, V: int, dtype: int) -> int:
    return int(library().spec_sample_workspace_size(R, V, dtype))


def sample_workspace(R: int, V: int, dtype: int, device=None, stream=None):
    """A zeroed workspace for spec_sample, shared with spec_verify's cache for
    the same (device, stream)."""
    torch = _torch()
    device = torch.device(device if device is not None else "cuda")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    s = stream if stream is not None else torch.cuda.current_stream(device)
    need = spec_sample_workspace_size(R, V, dtype)
    if need == 0:
        raise ValueError(f"sizes out of range: R={R} V={V} dtype={dtype}")
    return _cached_workspace(need, device, s)


def _sample_shapes(logits, u, temperature):
    """Shapes and dtypes of the sampling inputs: (R, V, dtype code)."""
    torch = _torch()
    if logits.dim() != 2:
        raise ValueError("logits must be [R, V]")
    R, V = logits.shape
    dt = _dtype_code(logits)
    for name, t in (("u", u), ("temperature", temperature)):
        if tuple(t.shape) != (R,) or t.dtype != torch.float32:
            raise ValueError(f"{name} must be float32 ({R},), got {t.dtype} {tuple(t.shape)}")
    return R, V, dt


def _marshal_sample(logits, u, temperature):
    R, V, dt = _sample_shapes(logits, u, temperature)
    for t in (logits, u, temperature):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("all inputs must be contiguous CUDA tensors")
        if t.device != logits.device:
            raise ValueError("all inputs must be on one device")
    return R, V, dt


def spec_sample(logits, u, temperature, out=None, ws=None, stream=None):
    """One token per row of logits [R, V] (float32 or bfloat16 CUDA tensor)
    from softmax(logits / T) by inverse CDF with the row's uniform u (float32
    [R] in [0, 1)); temperature float32 [R], 0 = argmax.  Returns int32 [R]
    (-1 on a row error); asynchronous like any CUDA op."""
    torch = _torch()
    R, V, dt = _marshal_sample(logits, u, temperature)
    dev = logits.device
    if out is None:
        out = torch.empty((R,), dtype=torch.int32, device=dev)
    _dev_out("out", out, (R,), torch.int32, dev)
    if ws is None:
        ws = sample_workspace(R, V, dt, dev, stream)
    _check_ws(ws, dev)
    with _on(dev):
        rc = library().spec_sample(_ptr(logits), _ptr(u), _ptr(temperature), _ptr(out), R, V, dt,
                                   _ptr(ws), ws.numel(), _stream_handle(stream, dev))
    _check(rc, "spec_sample")
    return out


def spec_sample_timed(logits, u, temperature, out, ws, stage_events, stream=None):
    """spec_sample recording the given torch.cuda.Event objects
    (SPEC_SAMPLE_STAGES of them, recorded once beforehand) after each stage:
    chunk records, pick, exact draws."""
    torch = _torch()
    R, V, dt = _marshal_sample(logits, u, temperature)
    _dev_out("out", out, (R,), torch.int32, logits.device)
    _check_ws(ws, logits.device)
    handles = (ctypes.c_void_p * SPEC_SAMPLE_STAGES)(
        *[ctypes.c_void_p(e.cuda_event) for e in stage_events])
    with _on(logits.device):
        rc = library().spec_sample_timed(_ptr(logits), _ptr(u), _ptr(temperature), _ptr(out), R, V,
                                         dt, _ptr(ws), ws.numel(),
                                         _stream_handle(stream, logits.device), handles)
    _check(rc, "spec_sample_timed")
    return out


def to_device(case, device="cuda"):
    """Copy a synth.Case's host arrays to device tensors (bf16 bit patterns
    become torch.bfloat16)."""
    import numpy as np
    torch = _torch()

    def logits(a):
        if a.dtype == np.uint16:
            return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).to(device)
        return torch.from_numpy(a).to(device)

    return dict(target=logits(case.target), draft=logits(case.draft),
                tokens=torch.from_numpy(case.tokens).to(device),
                u_accept=torch.from_numpy(case.u_accept).to(device),
                u_resample=torch.from_numpy(case.u_resample).to(device),
                temperature=torch.from_numpy(case.temperature).to(device))


def spec_sample_host_arena_size(R: int, V: int, dtype: int) -> int:
    return int(library().spec_sample_host_arena_size(R, V, dtype))


def spec_sample_host(logits, u, temperature, arena, out=None, stream=None):
    """End-to-end call on HOST tensors (CPU, ideally pinned): the library copies
    the inputs into the device `arena` (a CUDA uint8 tensor of at least
    spec_sample_host_arena_size bytes), samples, copies the tokens back and
    synchronises.  Returns the host int32 [R] tokens."""
    torch = _torch()
    R, V, dt = _sample_shapes(logits, u, temperature)
    for t in (logits, u, temperature):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("host inputs must be contiguous CPU tensors")
    if not arena.is_cuda or arena.dtype != torch.uint8 or not arena.is_contiguous():
        raise ValueError("arena must be a contiguous uint8 CUDA tensor")
    if out is not None:
        _check_out("out", out, (R,), torch.int32)
        if out.is_cuda:
            raise ValueError("out must be a host tensor")
    else:
        out = torch.empty((R,), dtype=torch.int32, pin_memory=True)
    with _on(arena.device):
        rc = library().spec_sample_host(_ptr(logits), _ptr(u), _ptr(temperature), _ptr(out), R, V,
                                        dt, _ptr(arena), arena.numel(),
                                        _stream_handle(stream, arena.device))
    _check(rc, "spec_sample_host")
    return out


def spec_bench_read(buf, sink, stream=None):
    """The benchmark's read-only probe over a CUDA tensor `buf` (16-byte
    aligned, size a multiple of 16 bytes); `sink` is an int32 CUDA tensor of
    at least spec_bench_read_sink_words() elements."""
    with _on(buf.device):
        rc = library().spec_bench_read(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink),
                                       _stream_handle(stream, buf.device))
    _check(rc, "spec_bench_read")


def spec_selftest_wait_timeout(ws, limit_ns: int, stream=None):
    """Launch the bounded-wait self-test on workspace `ws` (see
    include/spec_bench.h); read its outcome with spec_verify_read_status."""
    with _on(ws.device):
        _check(library().spec_selftest_wait_timeout(_ptr(ws), int(limit_ns),
                                                    _stream_handle(stream, ws.device)),
               "spec_selftest_wait_timeout")


def spec_bench_read_sink_words() -> int:
    return int(library().spec_bench_read_sink_words())


def sample_to_device(sc, device="cuda"):
    """Copy a synth.SampleCase's host arrays to device tensors."""
    import numpy as np
    torch = _torch()
    a = sc.logits
    if a.dtype == np.uint16:
        logits = torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).to(device)
    else:
        logits = torch.from_numpy(a).to(device)
    return dict(logits=logits, u=torch.from_numpy(sc.u).to(device),
                temperature=torch.from_numpy(sc.temperature).to(device))


# ------------------------------------------------ LM-head-fused verification

def spec_verify_lmhead_workspace_size(B: int, k: int, V: int, d: int, draft_dtype: int) -> int:
    return int(library().spec_verify_lmhead_workspace_size(B, k, V, d, draft_dtype))


def _marshal_lmhead(hidden, lm_head, draft, tokens, u_accept, u_resample, temperature):
    torch = _torch()
    if hidden.dtype != torch.bfloat16 or lm_head.dtype != torch.bfloat16:
        raise TypeError("hidden and lm_head must be bfloat16")
    if hidden.dim() != 3 or lm_head.dim() != 2 or draft.dim() != 3:
        raise ValueError("hidden [B,k+1,d], lm_head [V,d], draft [B,k,V] expected")
    B, k1, d = hidden.shape
    V = lm_head.shape[0]
    k = k1 - 1
    if lm_head.shape[1] != d or tuple(draft.shape) != (B, k, V):
        raise ValueError("shape mismatch between hidden, lm_head and draft")
    for name, t, shape, dtype in (("tokens", tokens, (B, k), torch.int32),
                                  ("u_accept", u_accept, (B, k), torch.float32),
                                  ("u_resample", u_resample, (B,), torch.float32),
                                  ("temperature", temperature, (B,), torch.float32)):
        if tuple(t.shape) != shape or t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")
    for t in (hidden, lm_head, draft, tokens, u_accept, u_resample, temperature):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("all tensors must be contiguous CUDA tensors")
    return B, k, V, d, _dtype_code(draft)


def _zeros_on(stream, device, n, dtype):
    """A zero-filled device tensor whose fill is ordered before later work on
    `stream` (the current stream when None)."""
    torch = _torch()
    device = torch.device(device if device is not None else "cuda")
    s = stream if stream is not None else torch.cuda.current_stream(device)
    with torch.cuda.stream(s):
        return torch.zeros(n, dtype=dtype, device=device)


def lmhead_workspace(B: int, k: int, V: int, d: int, draft_dtype: int, device=None,
                     stream=None):
    """A zeroed workspace for spec_verify_lmhead, zero-filled on `stream`."""
    torch = _torch()
    need = spec_verify_lmhead_workspace_size(B, k, V, d, draft_dtype)
    if need == 0:
        raise SpecVerifyError("sizes out of range for spec_verify_lmhead")
    return _zeros_on(stream, device, need, torch.uint8)


def spec_verify_lmhead(hidden, lm_head, draft, tokens, u_accept, u_resample, temperature,
                       out_tokens=None, out_num_accepted=None, ws=None, want_probs=False,
                       stream=None):
    """Verification with the target's LM head fused in: target logits
    t = hidden @ lm_head^T are formed on the tensor cores and never stored.
    hidden bf16 [B,k+1,d], lm_head bf16 [V,d], draft [B,k,V] f32 or bf16.
    Returns (out_tokens, out_num_accepted) or, with want_probs, also the fp32
    P = p_i(g_i), Q = q_i(g_i) as [B,k,2]."""
    torch = _torch()
    B, k, V, d, ddt = _marshal_lmhead(hidden, lm_head, draft, tokens, u_accept, u_resample,
                                      temperature)
    dev = hidden.device
    if out_tokens is None:
        out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    if out_num_accepted is None:
        out_num_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    _dev_out("out_tokens", out_tokens, (B, k + 1), torch.int32, dev)
    _dev_out("out_num_accepted", out_num_accepted, (B,), torch.int32, dev)
    if ws is None:
        ws = lmhead_workspace(B, k, V, d, ddt, dev, stream)
    _check_ws(ws, dev)
    probs = torch.empty((B, k, 2), dtype=torch.float32, device=dev) if want_probs else None
    h = _stream_handle(stream, dev)
    with _on(dev):
        if want_probs:
            rc = library().spec_verify_lmhead_timed(
                _ptr(hidden), _ptr(lm_head), _ptr(draft), _ptr(tokens), _ptr(u_accept),
                _ptr(u_resample), _ptr(temperature), _ptr(out_tokens), _ptr(out_num_accepted),
                _ptr(probs), B, k, V, d, ddt, _ptr(ws), ws.numel(), h, None)
        else:
            rc = library().spec_verify_lmhead(
                _ptr(hidden), _ptr(lm_head), _ptr(draft), _ptr(tokens), _ptr(u_accept),
                _ptr(u_resample), _ptr(temperature), _ptr(out_tokens), _ptr(out_num_accepted),
                B, k, V, d, ddt, _ptr(ws), ws.numel(), h)
    _check(rc, "spec_verify_lmhead")
    if want_probs:
        return out_tokens, out_num_accepted, probs
    return out_tokens, out_num_accepted


def spec_verify_lmhead_timed(hidden, lm_head, draft, tokens, u_accept, u_resample, temperature,
                             out_tokens, out_num_accepted, ws, stage_events, stream=None):
    """spec_verify_lmhead recording SPEC_LMHEAD_STAGES events, one after each
    kernel (draft chunk records, statistics GEMM, accept scan, draw GEMM,
    final search)."""
    torch = _torch()
    B, k, V, d, ddt = _marshal_lmhead(hidden, lm_head, draft, tokens, u_accept, u_resample,
                                      temperature)
    dev = hidden.device
    _dev_out("out_tokens", out_tokens, (B, k + 1), torch.int32, dev)
    _dev_out("out_num_accepted", out_num_accepted, (B,), torch.int32, dev)
    _check_ws(ws, dev)
    handles = (ctypes.c_void_p * SPEC_LMHEAD_STAGES)(
        *[ctypes.c_void_p(e.cuda_event) for e in stage_events])
    with _on(hidden.device):
        rc = library().spec_verify_lmhead_timed(
            _ptr(hidden), _ptr(lm_head), _ptr(draft), _ptr(tokens), _ptr(u_accept), _ptr(u_resample),
            _ptr(temperature), _ptr(out_tokens), _ptr(out_num_accepted), None, B, k, V, d, ddt,
            _ptr(ws), ws.numel(), _stream_handle(stream, hidden.device), handles)
    _check(rc, "spec_verify_lmhead_timed")
    return out_tokens, out_num_accepted


def spec_lmhead_logits(hidden, lm_head, out=None, stream=None):
    """The fused GEMM alone, storing out[r][x] = sum_j hidden[r][j] lm_head[x][j]
    (fp32) for checking the tensor-core product.  hidden bf16 [M,d]."""
    torch = _torch()
    if hidden.dtype != torch.bfloat16 or lm_head.dtype != torch.bfloat16:
        raise TypeError("hidden and lm_head must be bfloat16")
    if hidden.dim() != 2 or lm_head.dim() != 2 or lm_head.shape[1] != hidden.shape[1]:
        raise ValueError("hidden [M,d] and lm_head [V,d] expected")
    for t in (hidden, lm_head):
        if not t.is_cuda or not t.is_contiguous() or t.device != hidden.device:
            raise ValueError("hidden and lm_head must be contiguous CUDA tensors on one device")
    M, d = hidden.shape
    V = lm_head.shape[0]
    if out is None:
        out = torch.empty((M, V), dtype=torch.float32, device=hidden.device)
    _dev_out("out", out, (M, V), torch.float32, hidden.device)
    status = _zeros_on(stream, hidden.device, 1, torch.int32)
    with _on(hidden.device):
        rc = library().spec_lmhead_logits(_ptr(hidden), _ptr(lm_head), _ptr(out), M, V, d,
                                          _ptr(status), _stream_handle(stream, hidden.device))
    _check(rc, "spec_lmhead_logits")
    return out, status


# ------------------------------------------------------- tree verification

def spec_verify_tree(target, draft, parent, tokens, n_nodes, u_accept, u_resample, temperature,
                     out_tokens=None, out_nodes=None, out_num_accepted=None, stream=None):
    """Tree verification (include/spec_tree.h) on the current (or given)
    stream.  target and draft [B, N, V]: float32 or bfloat16 CUDA tensors;
    parent, tokens int32 [B, N]; n_nodes int32 [B]; u_accept float32 [B, N];
    u_resample, temperature float32 [B].  Returns (out_tokens int32 [B, N],
    out_nodes int32 [B, N], out_num_accepted int32 [B]); asynchronous like
    any CUDA op."""
    torch = _torch()
    if target.dim() != 3 or tuple(draft.shape) != tuple(target.shape):
        raise ValueError("target and draft must both be [B, N, V]")
    B, N, V = target.shape
    dt = _dtype_code(target)
    if draft.dtype != target.dtype:
        raise TypeError("target and draft must share a dtype")
    dev = target.device
    for name, t, shape, dtype in (("parent", parent, (B, N), torch.int32),
                                  ("tokens", tokens, (B, N), torch.int32),
                                  ("n_nodes", n_nodes, (B,), torch.int32),
                                  ("u_accept", u_accept, (B, N), torch.float32),
                                  ("u_resample", u_resample, (B,), torch.float32),
                                  ("temperature", temperature, (B,), torch.float32)):
        if tuple(t.shape) != shape or t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")
    for t in (target, draft, parent, tokens, n_nodes, u_accept, u_resample, temperature):
        if not t.is_cuda or not t.is_contiguous() or t.device != dev:
            raise ValueError(f"all inputs must be contiguous CUDA tensors on {dev}")
    if out_tokens is None:
        out_tokens = torch.empty((B, N), dtype=torch.int32, device=dev)
    if out_nodes is None:
        out_nodes = torch.empty((B, N), dtype=torch.int32, device=dev)
    if out_num_accepted is None:
        out_num_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    _dev_out("out_tokens", out_tokens, (B, N), torch.int32, dev)
    _dev_out("out_nodes", out_nodes, (B, N), torch.int32, dev)
    _dev_out("out_num_accepted", out_num_accepted, (B,), torch.int32, dev)
    with _on(dev):
        rc = library().spec_verify_tree(_ptr(target), _ptr(draft), _ptr(parent), _ptr(tokens),
                                        _ptr(n_nodes), _ptr(u_accept), _ptr(u_resample),
                                        _ptr(temperature), _ptr(out_tokens), _ptr(out_nodes),
                                        _ptr(out_num_accepted), B, N, V, dt,
                                        _stream_handle(stream, dev))
    _check(rc, "spec_verify_tree")
    return out_tokens, out_nodes, out_num_accepted


def tree_to_device(tc, device="cuda"):
    """Copy a synth.TreeCase's host arrays to device tensors."""
    import numpy as np
    torch = _torch()

    def logits(a):
        if a.dtype == np.uint16:
            return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).to(device)
        return torch.from_numpy(a).to(device)

    return dict(target=logits(tc.target), draft=logits(tc.draft),
                parent=torch.from_numpy(tc.parent).to(device),
                tokens=torch.from_numpy(tc.tokens).to(device),
                n_nodes=torch.from_numpy(tc.n_nodes).to(device),
                u_accept=torch.from_numpy(tc.u_accept).to(device),
                u_resample=torch.from_numpy(tc.u_resample).to(device),
                temperature=torch.from_numpy(tc.temperature).to(device))


# ------------------------------------------- tree attention and cache commit

def _raw(torch):
    """(current stream handle of a device index, current device index) getters: the
    ones that PyTorch's own generated code calls, several times cheaper than
    torch.cuda.current_stream and torch.cuda.current_device."""
    c = torch._C
    return (getattr(c, "_cuda_getCurrentRawStream", None)
            or (lambda i: torch.cuda.current_stream(i).cuda_stream),
            getattr(c, "_cuda_getDevice", None) or torch.cuda.current_device)


_raw_getters = None


def _call_stream(stream, dev, tensors):
    """(stream handle, the stream to allocate on or None for the current one) of
    a call.  Where the call's stream is not the current one, the tensors'
    memory is kept from reuse until the stream has passed the call."""
    global _raw_getters
    if _raw_getters is None:
        _raw_getters = _raw(_torch())
    current = _raw_getters[0](dev.index)
    if stream is None or stream.cuda_stream == current:
        return current, None
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream, stream


def _empty_on(s, shape, dtype, dev):
    """An output allocated for use on stream `s` (None: the current one)."""
    torch = _torch()
    if s is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(s):
        return torch.empty(shape, dtype=dtype, device=dev)


def _launch(dev, what, fn, *args):
    """fn(*args) with `dev` current."""
    if _raw_getters[1]() == dev.index:
        rc = fn(*args)
    else:
        with _on(dev):
            rc = fn(*args)
    if rc != SPEC_OK:
        _check(rc, what)


def _array(name, t, shape, dtype, dev):
    """A contiguous array of the call's shape and dtype on its device."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")
    if not t.is_cuda or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{name} must be a contiguous CUDA tensor on {dev}")
    return t.data_ptr()


def _strided(name, t, dev, step):
    """(address, strides of all dimensions but the last) of a tensor whose last
    dimension is contiguous.  Strides are multiples of `step` elements; a
    dimension of one entry has none."""
    if not t.is_cuda or t.device != dev:
        raise ValueError(f"{name} must be on {dev}")
    shape, st, at = t.shape, t.stride(), t.data_ptr()
    if st[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    st = [s if n != 1 else 0 for n, s in zip(shape[:-1], st)]
    if step > 1 and (at % (2 * step) or any([s % step for s in st])):
        raise ValueError(f"{name}: strides must be multiples of {step} elements and the data "
                         f"{2 * step}-byte aligned")
    return at, st


def _geometry(k_cache, page_table, B, dev):
    """((page_size, pages_per_seq, num_pages), the table's address) of a cache
    [.., pages, slots, heads, D]."""
    P, S = k_cache.shape[-4:-2]
    if page_table is None:
        if P < B:
            raise ValueError(f"a contiguous cache needs a page for each of {B} sequences, got {P}")
        return (S, 1, P), 0
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, pages_per_seq]")
    M = page_table.shape[1]
    return (S, M, P), _array("page_table", page_table, (B, M), _torch().int32, dev)


@functools.lru_cache(maxsize=256)
def _plan_layout(B, N):
    """Bytes of a plan, and the int32 offsets of its readable parts."""
    lib = library()
    return (lib.spec_tree_plan_size(B, N),
            tuple(lib.spec_tree_plan_offset(B, N, i) // 4 for i in range(3)))


class TreePlan:
    """What spec_tree_plan made: `positions` int32 [B, N], `status` int32 [B] and
    `mask` int32 [B, N, W] (bits of ancestors, include/spec_attn.h) are views
    of `data` (int32), which every layer's spec_tree_attention reads."""

    def __init__(self, B, N, geometry, data):
        self.B, self.N, self.geometry, self.data = B, N, geometry, data

    def read_status(self, stream=None):
        """SPEC_DEV_OK, or SPEC_DEV_WAIT_TIMEOUT after a wait inside an attention
        kernel that read this plan gave up.  Synchronises the stream."""
        if self.B == 0:  # no kernel ran, and nothing was written
            return SPEC_DEV_OK
        return spec_verify_read_status(self.data, stream)

    def _part(self, which, shape, strides):
        return self.data.as_strided(shape, strides, _plan_layout(self.B, self.N)[1][which])

    @property
    def positions(self):
        return self._part(SPEC_PLAN_POSITIONS, (self.B, self.N), (self.N, 1))

    @property
    def status(self):
        return self._part(SPEC_PLAN_STATUS, (self.B,), (1,))

    @property
    def mask(self):
        W = 4 * ((self.N + 127) // 128)
        return self._part(SPEC_PLAN_MASK, (self.B, self.N, W), (self.N * W, W, 1))


def spec_tree_plan(parent, n_nodes, cache_len, k_cache, page_table=None, plan=None, stream=None):
    """The plan of a step (include/spec_attn.h): ancestors, positions and schedule of
    B trees of up to N nodes over their caches, made once for all layers.

    parent int32 [B, N] (a chain: parent[n] = n - 1); n_nodes, cache_len int32
    [B]; k_cache [pages, slots, Hkv, D], one layer's cache, asked for its
    geometry only; page_table int32 [B, pages_per_seq], or None for a
    contiguous cache (sequence b owns page b).  `plan` refills a TreePlan of
    the same sizes.  Returns a TreePlan; asynchronous like any CUDA op."""
    torch = _torch()
    if parent.dim() != 2 or k_cache.dim() != 4:
        raise ValueError("parent must be [B, N] and k_cache [pages, slots, Hkv, D]")
    B, N = parent.shape
    dev, i32 = parent.device, torch.int32
    p = _array("parent", parent, (B, N), i32, dev)
    n = _array("n_nodes", n_nodes, (B,), i32, dev)
    c = _array("cache_len", cache_len, (B,), i32, dev)
    geometry, table = _geometry(k_cache, page_table, B, dev)
    need = _plan_layout(B, N)[0]
    if need == 0:
        raise ValueError(f"sizes out of range: B={B} N={N}")
    if plan is not None and ((plan.B, plan.N) != (B, N) or plan.data.device != dev):
        raise ValueError(f"plan is for B={plan.B} N={plan.N} on {plan.data.device}")
    h, s = _call_stream(stream, dev, (parent, n_nodes, cache_len, page_table,
                                      plan.data if plan is not None else None))
    if plan is None:
        plan = TreePlan(B, N, geometry, _empty_on(s, (need // 4,), i32, dev))
    plan.geometry = geometry
    _launch(dev, "spec_tree_plan", (_lib or library()).spec_tree_plan, p, n, c, table, B, N,
            *geometry, plan.data.data_ptr(), need, h)
    return plan


@functools.lru_cache(maxsize=256)
def spec_tree_attention_workspace_size(N: int, Hq: int, Hkv: int, D: int) -> int:
    return int(library().spec_tree_attention_workspace_size(N, Hq, Hkv, D))


_attention_ws = _Workspaces()


def attention_workspace(N: int, Hq: int, Hkv: int, D: int, device=None, stream=None):
    """A workspace for spec_tree_attention, cached per (host thread, device, stream)
    and apart from spec_verify's.  While the stream is being captured into a
    graph it is a new one, in the graph's own memory: a replay may overlap
    later calls on the stream."""
    torch = _torch()
    device = torch.device(device if device is not None else "cuda")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    h, s = _call_stream(stream, device, ())
    return _attention_workspace(N, Hq, Hkv, D, device, h, s)


def _attention_workspace(N, Hq, Hkv, D, device, h, s):
    torch = _torch()
    need = spec_tree_attention_workspace_size(N, Hq, Hkv, D)
    if need == 0:
        raise ValueError(f"sizes out of range: N={N} Hq={Hq} Hkv={Hkv} D={D}")
    if s is not None:
        with torch.cuda.stream(s):
            return _attention_workspace(N, Hq, Hkv, D, device, h, None)
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(need, dtype=torch.uint8, device=device)
    key = (device.index, h)
    ws = _attention_ws.of.get(key)
    if ws is None or ws.numel() < need:
        ws = _attention_ws.of[key] = torch.empty(need, dtype=torch.uint8, device=device)
    return ws


def spec_tree_attention(q, k_new, v_new, k_cache, v_cache, plan, page_table=None, scale=None,
                        out=None, want_lse=False, ws=None, stream=None):
    """Attention of B trees of drafted tokens over a cache (include/spec_attn.h).

    q [B, N, Hq, D]; k_new, v_new [B, N, Hkv, D]: the new tokens' keys and
    values; k_cache, v_cache [pages, slots, Hkv, D], bfloat16 or float16, any
    strides with a contiguous last dimension; plan from spec_tree_plan;
    page_table int32 [B, pages_per_seq] or None; scale 1 / sqrt(D) by default;
    ws of one call at a time, by default this thread's (attention_workspace).
    Returns out [B, N, Hq, D] and, with want_lse, the rows' log-sum-exp
    float32 [B, N, Hq]; asynchronous like any CUDA op."""
    torch = _torch()
    if not q.dim() == k_new.dim() == v_new.dim() == k_cache.dim() == v_cache.dim() == 4:
        raise ValueError("q, k_new, v_new, k_cache and v_cache must have 4 dimensions")
    B, N, Hq, D = q.shape
    Hkv = k_new.shape[2]
    P, S = k_cache.shape[:2]
    if k_new.shape != (B, N, Hkv, D) or v_new.shape != k_new.shape:
        raise ValueError(f"k_new and v_new must be {(B, N, Hkv, D)}")
    if k_cache.shape != (P, S, Hkv, D) or v_cache.shape != k_cache.shape:
        raise ValueError(f"k_cache and v_cache must be [pages, slots, {Hkv}, {D}]")
    dtype = q.dtype
    if dtype != torch.bfloat16 and dtype != torch.float16:
        raise TypeError(f"q must be bfloat16 or float16, got {dtype}")
    if not dtype == k_new.dtype == v_new.dtype == k_cache.dtype == v_cache.dtype:
        raise TypeError("q, k_new, v_new, k_cache and v_cache must share a dtype")
    dev = q.device
    geometry, table = _geometry(k_cache, page_table, B, dev)
    if (plan.B, plan.N, plan.geometry) != (B, N, geometry) or plan.data.device != dev:
        raise ValueError(f"plan is for B={plan.B} N={plan.N}, cache {plan.geometry} on "
                         f"{plan.data.device}; the call is for B={B} N={N}, {geometry} on {dev}")
    q_at, q_st = _strided("q", q, dev, 8)
    kn_at, kn_st = _strided("k_new", k_new, dev, 8)
    vn_at, vn_st = _strided("v_new", v_new, dev, 8)
    kc_at, kc_st = _strided("k_cache", k_cache, dev, 8)
    vc_at, vc_st = _strided("v_cache", v_cache, dev, 8)
    scale = D ** -0.5 if scale is None else float(scale)
    if not 0.0 < scale < float("inf"):
        raise ValueError(f"scale must be finite and positive, got {scale}")
    if table and S % 128 and (S < 8 or S & (S - 1)):
        raise ValueError(f"page size {S}: a multiple of 128, or a power of two from 8")
    h, s = _call_stream(stream, dev, (q, k_new, v_new, k_cache, v_cache, plan.data, page_table,
                                      out, ws))
    if out is None:
        out = _empty_on(s, (B, N, Hq, D), dtype, dev)
    else:
        _dev_out("out", out, (B, N, Hq, D), dtype, dev)
    lse = _empty_on(s, (B, N, Hq), torch.float32, dev) if want_lse else None
    if ws is None:
        ws = _attention_workspace(N, Hq, Hkv, D, dev, h, s)
    else:
        _check_ws(ws, dev)
    args = _pack_attention(q_at, kn_at, vn_at, kc_at, vc_at, *q_st, *kn_st, *vn_st, *kc_st, *vc_st,
                           table, plan.data.data_ptr(), out.data_ptr(),
                           lse.data_ptr() if want_lse else 0, scale, B, N, Hq, Hkv, D, *geometry,
                           SPEC_BF16 if dtype == torch.bfloat16 else SPEC_F16)
    _launch(dev, "spec_tree_attention", (_lib or library()).spec_tree_attention, args,
            ws.data_ptr(), ws.numel(), h)
    return (out, lse) if want_lse else out


def spec_tree_commit(k_new, v_new, k_cache, v_cache, cache_len, out_num_accepted, out_nodes=None,
                     page_table=None, out_len=None, stream=None):
    """Append the accepted path's keys and values to the cache
    (include/spec_attn.h), after spec_verify_tree (out_nodes: its path) or
    spec_verify (out_nodes None: a chain).

    k_new, v_new [B, N, Hkv, D] with caches [pages, slots, Hkv, D], or with a
    leading dimension of layers; bfloat16, float16 or float32, any strides
    with a contiguous last dimension.  Returns the new cache_len int32 [B]
    (-1 for a sequence error, whose cache is left alone)."""
    torch = _torch()
    if k_new.dim() not in (4, 5) or k_cache.dim() != k_new.dim():
        raise ValueError("k_new [.., B, N, Hkv, D] and k_cache [.., pages, slots, Hkv, D] expected")
    *lead, B, N, Hkv, D = k_new.shape
    P, S = k_cache.shape[-4:-2]
    if v_new.shape != k_new.shape:
        raise ValueError("k_new and v_new must have one shape")
    if k_cache.shape != (*lead, P, S, Hkv, D) or v_cache.shape != k_cache.shape:
        raise ValueError(f"k_cache and v_cache must be {(*lead, 'pages', 'slots', Hkv, D)}")
    if k_new.dtype not in (torch.bfloat16, torch.float16, torch.float32):
        raise TypeError(f"k_new must be bfloat16, float16 or float32, got {k_new.dtype}")
    if not k_new.dtype == v_new.dtype == k_cache.dtype == v_cache.dtype:
        raise TypeError("k_new, v_new, k_cache and v_cache must share a dtype")
    dev, i32 = k_new.device, torch.int32
    length = _array("cache_len", cache_len, (B,), i32, dev)
    accepted = _array("out_num_accepted", out_num_accepted, (B,), i32, dev)
    nodes = _array("out_nodes", out_nodes, (B, N), i32, dev) if out_nodes is not None else 0
    geometry, table = _geometry(k_cache, page_table, B, dev)
    at, strides = [], []
    for name, t in (("k_new", k_new), ("v_new", v_new), ("k_cache", k_cache),
                    ("v_cache", v_cache)):
        a, st = _strided(name, t, dev, 1)
        at.append(a)
        strides += st if lead else (0, *st)
    h, s = _call_stream(stream, dev, (k_new, v_new, k_cache, v_cache, cache_len,
                                      out_num_accepted, out_nodes, page_table, out_len))
    if out_len is None:
        out_len = _empty_on(s, (B,), i32, dev)
    else:
        _dev_out("out_len", out_len, (B,), i32, dev)
        if B > 0 and out_len.data_ptr() == length:
            raise ValueError("out_len must not be cache_len itself")
    args = _pack_commit(*at, *strides, length, accepted, nodes, table, out_len.data_ptr(),
                        lead[0] if lead else 1, B, N, Hkv, D, *geometry, k_new.element_size())
    _launch(dev, "spec_tree_commit", (_lib or library()).spec_tree_commit, args, h)
    return out_len


# --------------------------------------------------------- logits processing

def spec_process_logits(logits, history=None, history_len=None, prompt_len=None,
                        draft_tokens=None, parent=None, n_nodes=None, repetition=None,
                        frequency=None, presence=None, bias_tokens=None, bias_values=None,
                        allowed=None, out=None, stream=None):
    """Penalties for repeated tokens, biases and grammar masks on the rows that a
    verification reads next (include/spec_logits.h states the formula).

    logits [B, R, V] float32 or bfloat16; history int32 [B, H] with
    history_len and prompt_len int32 [B]; draft_tokens int32 [B, R - 1] or
    [B, R] (chain: row r follows the first r of them), or with parent int32
    [B, R] the tokens of a tree's nodes; n_nodes int32 [B]: rows past it are
    left alone; repetition, frequency, presence float32 [B]; bias_tokens int32
    and bias_values float32 [B, M] (token -1: unused); allowed int32 words
    [B, R, ceil(V / 32)] (or [B, 1, ..], [1, 1, ..]), bit x % 32 of word
    x / 32 for token x.  Anything may be None.  `out` may be logits itself.
    Returns out; asynchronous like any CUDA op."""
    torch = _torch()
    if logits.dim() != 3:
        raise ValueError("logits must be [B, R, V]")
    B, R, V = logits.shape
    dt = _dtype_code(logits)
    dev, i32, f32 = logits.device, torch.int32, torch.float32
    if not logits.is_cuda or not logits.is_contiguous():
        raise ValueError("logits must be a contiguous CUDA tensor")
    hi = hl = pl = dtok = par = nn = rep = freq = pres = bt = bv = al = 0
    H = cols = M = sb = sr = 0
    if history is not None:
        if history.dim() != 2 or history_len is None or prompt_len is None:
            raise ValueError("history [B, H] comes with history_len and prompt_len [B]")
        H = history.shape[1]
        hi = _array("history", history, (B, H), i32, dev)
        hl = _array("history_len", history_len, (B,), i32, dev)
        pl = _array("prompt_len", prompt_len, (B,), i32, dev)
    elif history_len is not None or prompt_len is not None:
        raise ValueError("history_len and prompt_len come with history")
    if draft_tokens is not None:
        cols = draft_tokens.shape[1] if draft_tokens.dim() == 2 else -1
        if parent is not None and cols != R or parent is None and cols not in (R - 1, R):
            raise ValueError(f"draft_tokens must be [B, {R}]" +
                             ("" if parent is not None else f" or [B, {R - 1}]"))
        dtok = _array("draft_tokens", draft_tokens, (B, cols), i32, dev)
    if parent is not None:
        if draft_tokens is None:
            raise ValueError("parent comes with draft_tokens")
        par = _array("parent", parent, (B, R), i32, dev)
    if n_nodes is not None:
        nn = _array("n_nodes", n_nodes, (B,), i32, dev)
    if repetition is not None:
        rep = _array("repetition", repetition, (B,), f32, dev)
    if frequency is not None:
        freq = _array("frequency", frequency, (B,), f32, dev)
    if presence is not None:
        pres = _array("presence", presence, (B,), f32, dev)
    if (bias_tokens is None) != (bias_values is None):
        raise ValueError("bias_tokens and bias_values come together")
    if bias_tokens is not None:
        if bias_tokens.dim() != 2 or bias_tokens.shape[1] > SPEC_LOGITS_MAX_BIAS:
            raise ValueError(f"bias_tokens must be [B, M], M <= {SPEC_LOGITS_MAX_BIAS}")
        M = bias_tokens.shape[1]
        bt = _array("bias_tokens", bias_tokens, (B, M), i32, dev)
        bv = _array("bias_values", bias_values, (B, M), f32, dev)
    if allowed is not None:
        W = (V + 31) // 32
        if (allowed.dim() != 3 or allowed.shape[0] not in (1, B) or allowed.shape[1] not in (1, R)
                or allowed.shape[2] != W or allowed.dtype != i32 or not allowed.is_cuda
                or allowed.device != dev or allowed.stride(2) != 1 and W > 1):
            raise ValueError(f"allowed must be int32 [{B} or 1, {R} or 1, {W}] on {dev}, its last "
                             "dimension contiguous")
        al = allowed.data_ptr()
        sb = allowed.stride(0) if allowed.shape[0] > 1 else 0
        sr = allowed.stride(1) if allowed.shape[1] > 1 else 0
    h, s = _call_stream(stream, dev, (logits, history, history_len, prompt_len, draft_tokens,
                                        parent, n_nodes, repetition, frequency, presence,
                                        bias_tokens, bias_values, allowed, out))
    if out is None:
        out = _empty_on(s, (B, R, V), logits.dtype, dev)
    else:
        _dev_out("out", out, (B, R, V), logits.dtype, dev)
    args = _pack_logits(logits.data_ptr(), out.data_ptr(), hi, hl, pl, dtok, par, nn, rep, freq,
                        pres, bt, bv, al, sb, sr, B, R, V, H, cols, M, dt)
    _launch(dev, "spec_process_logits", (_lib or library()).spec_process_logits, args, h)
    return out


# --------------------------------------------------- chunks of new tokens
#
# A call's checks depend on its tensors' shapes, strides, dtypes and devices
# alone (addresses apart, which the library checks), so each function keeps what
# they came to by those: with small kernels the checks cost more than the launch.

def _meta(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


class _Checked(dict):
    """What a function's checks came to, by what they depend on."""

    def __call__(self, key, check):
        got = self.get(key)
        if got is None:
            if len(self) >= 4096:
                self.clear()
            got = self[key] = check()
        return got


_checked_append, _checked_plan, _checked_chunk = _Checked(), _Checked(), _Checked()
_checked_beam, _checked_reorder = _Checked(), _Checked()
_checked_fork, _checked_compact, _checked_copy = _Checked(), _Checked(), _Checked()

# The short way of a call that is known (csrc/calls.cpp): by the same things, what its checks came to and
# the words of its arguments but the addresses are kept there, and run(number, a, b, *tensors)
# makes the outputs and the call, or answers None for the long way.
_short = _run = None
_APPEND, _PLAN, _ATTEND, _SELECT, _REORDER, _FORK, _COMPACT, _COPY = range(8)
_AS_ARGS, _WITH_WORKSPACE, _AS_REORDER, _AS_PLAN = range(4)


def _load_calls():
    """The module; without one that was compiled for this PyTorch every call goes the long way."""
    global _short, _run
    if _short is None:
        try:
            if not importlib.import_module(".build", __name__).calls_match():
                raise ImportError("_calls.so is none, or another PyTorch's")
            module = importlib.import_module("._calls", __name__)
        except ImportError:
            _short = False
        else:
            text = ctypes.cast(library().spec_verify_strerror, ctypes.c_void_p).value
            module.setup(SpecVerifyError, text)
            _short, _run = module, module.run
    return _short


def _keep(call, name, style, args, in_at, outs, out_at, dev, kind=-1, need=0, extra=None):
    """What run(*call) does from now on: call = (number, a, b, *tensors), in_at and out_at the
    places of the inputs' and outputs' addresses in args."""
    torch, lib = _torch(), _lib
    if type(lib) is not ctypes.CDLL or not all([t is None or type(t) is torch.Tensor
                                                for t in call[3:]]):
        return
    if _short or _load_calls():
        _short.keep(call, name, ctypes.cast(getattr(lib, name), ctypes.c_void_p).value, style, args,
                    in_at, outs, out_at, kind, need, dev.index, extra)


def _scratch(cache, need, device, h, s, zeroed=False):
    """A workspace of `need` bytes from `cache`, one per (host thread, device, stream).
    While the stream is being captured into a graph it is a new one, in the
    graph's own memory: a replay may overlap later calls on the stream."""
    torch = _torch()
    if s is not None:
        with torch.cuda.stream(s):
            return _scratch(cache, need, device, h, None, zeroed)
    make = torch.zeros if zeroed else torch.empty
    if torch.cuda.is_current_stream_capturing():
        return make(need, dtype=torch.uint8, device=device)
    key = (device.index, h)
    ws = cache.of.get(key)
    if ws is None or ws.numel() < need:
        ws = cache.of[key] = make(need, dtype=torch.uint8, device=device)
        if _short or _load_calls():
            _short.workspace(_kinds.index(cache), device.index, h, ws.data_ptr(), need)
    return ws


_chunk_ws, _beam_ws, _pages_ws = _kinds = _Workspaces(), _Workspaces(), _Workspaces()


def _caches(k_cache, v_cache, lead, Hkv, D, dtype):
    """Checks the caches [*lead, pages, slots, Hkv, D]."""
    P, S = k_cache.shape[-4:-2]
    if k_cache.shape != (*lead, P, S, Hkv, D) or v_cache.shape != k_cache.shape:
        raise ValueError(f"k_cache and v_cache must be {(*lead, 'pages', 'slots', Hkv, D)}")
    if not dtype == k_cache.dtype == v_cache.dtype:
        raise TypeError("keys, values and their caches must share a dtype")


_plain_empty = None


def _new(s, shape, strides, dtype, dev):
    """A contiguous output, of these strides, for use on stream `s` (None: the current
    one).  On the current device and stream it is made by the function that PyTorch's own
    generated code calls, in half of torch.empty's time."""
    global _plain_empty
    if _plain_empty is None:
        guards = getattr(getattr(_torch()._C, "_dynamo", None), "guards", None)
        _plain_empty = getattr(guards, "_empty_strided_cuda", False)
    if s is None and _plain_empty and _raw_getters[1]() == dev.index:
        return _plain_empty(shape, strides, dtype)
    return _empty_on(s, shape, dtype, dev)


def _strides_of(shape):
    st = [1] * len(shape)
    for i in range(len(shape) - 2, -1, -1):
        st[i] = st[i + 1] * max(1, shape[i + 1])
    return tuple(st)


def _ptr_of(t):
    return 0 if t is None else t.data_ptr()


_pack_4q, _pack_5q, _pack_3q = (struct.Struct(f).pack for f in ("@4Q", "@5Q", "@3Q"))


def spec_chunk_append(k_new, v_new, k_cache, v_cache, row_start, cache_len, page_table=None,
                      out_len=None, stream=None):
    """Append new tokens' keys and values to the cache (include/spec_chunk.h).

    k_new, v_new [rows, Hkv, D] with caches [pages, slots, Hkv, D], or both with
    a leading dimension of layers; bfloat16, float16 or float32, any strides
    with a contiguous last dimension; row_start int32 [B + 1]: sequence b's
    tokens are rows row_start[b] .. row_start[b + 1] - 1; cache_len int32 [B].
    Returns the new lengths int32 [B] (-1 for a sequence error, whose cache is
    left alone); asynchronous like any CUDA op."""
    plain = out_len is None and stream is None
    if _run and plain:
        got = _run(_APPEND, 0, 0, k_new, v_new, k_cache, v_cache, row_start, cache_len, page_table)
        if got is not None:
            return got
    torch = _torch()

    def check():
        if k_new.dim() not in (3, 4) or k_cache.dim() != k_new.dim() + 1:
            raise ValueError("k_new [.., rows, Hkv, D] and k_cache [.., pages, slots, Hkv, D] "
                             "expected")
        *lead, T, Hkv, D = k_new.shape
        if v_new.shape != k_new.shape:
            raise ValueError("k_new and v_new must have one shape")
        if k_new.dtype not in (torch.bfloat16, torch.float16, torch.float32):
            raise TypeError(f"k_new must be bfloat16, float16 or float32, got {k_new.dtype}")
        if v_new.dtype != k_new.dtype:
            raise TypeError("k_new and v_new must share a dtype")
        _caches(k_cache, v_cache, lead, Hkv, D, k_new.dtype)
        if cache_len.dim() != 1:
            raise ValueError("cache_len must be [B]")
        dev, i32, B = k_new.device, torch.int32, cache_len.shape[0]
        _array("row_start", row_start, (B + 1,), i32, dev)
        _array("cache_len", cache_len, (B,), i32, dev)
        geometry, _ = _geometry(k_cache, page_table, B, dev)
        strides = []
        for name, t in (("k_new", k_new), ("v_new", v_new), ("k_cache", k_cache),
                        ("v_cache", v_cache)):
            st = _strided(name, t, dev, 1)[1]
            strides += st if lead else (0, *st)
        if out_len is not None:
            _dev_out("out_len", out_len, (B,), i32, dev)
        return (dev, (B,), struct.pack("@14q", *strides),
                struct.pack("@9i4x", lead[0] if lead else 1, B, T, Hkv, D, *geometry,
                            k_new.element_size()))
    dev, shape, strides, sizes = _checked_append(
        (_meta(k_new), _meta(v_new), _meta(k_cache), _meta(v_cache), _meta(row_start),
         _meta(cache_len), _meta(page_table), _meta(out_len)), check)
    h, s = _call_stream(stream, dev, (k_new, v_new, k_cache, v_cache, row_start, cache_len,
                                      page_table, out_len))
    if out_len is None:
        out_len = _new(s, shape, (1,), torch.int32, dev)
    args = b"".join((_pack_4q(k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(),
                              v_cache.data_ptr()), strides,
                     _pack_4q(row_start.data_ptr(), cache_len.data_ptr(), _ptr_of(page_table),
                              out_len.data_ptr()), sizes))
    _launch(dev, "spec_chunk_append", (_lib or library()).spec_chunk_append, args, h)
    if plain:
        _keep((_APPEND, 0, 0, k_new, v_new, k_cache, v_cache, row_start, cache_len, page_table),
              "spec_chunk_append", _AS_ARGS, args, (0, 8, 16, 24, 144, 152, 160), (out_len,), (168,),
              dev)
    return out_len


@functools.lru_cache(maxsize=256)
def _chunk_layout(B, T, G):
    """Bytes of a plan, and the int32 offset of its statuses."""
    lib = library()
    return lib.spec_chunk_plan_size(B, T, G), lib.spec_chunk_plan_status(B, T, G) // 4


class ChunkPlan:
    """What spec_chunk_plan made: `status` int32 [B] is a view of `data` (int32),
    which every layer's spec_chunk_attention reads."""

    def __init__(self, B, rows, group, geometry, data, code=None):
        self.B, self.rows, self.group, self.geometry, self.data = B, rows, group, geometry, data
        self.code = code or self.code_of(geometry)

    def code_of(self, geometry):
        """All that a call's checks depend on of a plan, but its data."""
        return struct.pack("@6q", self.B, self.rows, self.group, *geometry)

    def read_status(self, stream=None):
        """SPEC_DEV_OK, or SPEC_DEV_WAIT_TIMEOUT after a wait inside an attention
        kernel that read this plan gave up.  Synchronises the stream."""
        if self.B == 0:  # no kernel ran, and nothing was written
            return SPEC_DEV_OK
        return spec_verify_read_status(self.data, stream)

    @property
    def status(self):
        at = _chunk_layout(self.B, self.rows, self.group)[1]
        return self.data[at:at + self.B]


def spec_chunk_plan(row_start, kv_len, q, k_cache, page_table=None, plan=None, stream=None):
    """The plan of a step over chunks of new tokens (include/spec_chunk.h), made
    once for all layers.

    row_start int32 [B + 1]; kv_len int32 [B]: positions in the cache, the new
    tokens' included (what spec_chunk_append returned); q [rows, Hq, D] and
    k_cache [pages, slots, Hkv, D], one layer's, asked for their sizes only;
    page_table int32 [B, pages_per_seq], or None for a contiguous cache.
    `plan` refills a ChunkPlan of the same sizes.  Returns a ChunkPlan;
    asynchronous like any CUDA op."""
    plain = plan is None and stream is None
    if _run and plain:
        got = _run(_PLAN, 0, 0, row_start, kv_len, q, k_cache, page_table)
        if got is not None:
            data, (B, T, G, geometry, code) = got
            return ChunkPlan(B, T, G, geometry, data, code)
    torch = _torch()

    def check():
        if kv_len.dim() != 1 or q.dim() != 3 or k_cache.dim() != 4:
            raise ValueError("kv_len must be [B], q [rows, Hq, D] and k_cache "
                             "[pages, slots, Hkv, D]")
        B, (T, Hq), Hkv = kv_len.shape[0], q.shape[:2], k_cache.shape[2]
        if Hkv < 1 or Hq % Hkv:
            raise ValueError(f"{Hq} query heads do not divide among {Hkv} key heads")
        G = Hq // Hkv
        dev, i32 = kv_len.device, torch.int32
        _array("row_start", row_start, (B + 1,), i32, dev)
        _array("kv_len", kv_len, (B,), i32, dev)
        geometry, _ = _geometry(k_cache, page_table, B, dev)
        need = _chunk_layout(B, T, G)[0]
        if need == 0:
            raise ValueError(f"sizes out of range: B={B} rows={T} Hq/Hkv={G}")
        return dev, B, T, G, geometry, need
    dev, B, T, G, geometry, need = _checked_plan(
        (_meta(row_start), _meta(kv_len), q.shape, k_cache.shape, _meta(page_table)), check)
    if plan is not None and ((plan.B, plan.rows, plan.group) != (B, T, G)
                             or plan.data.device != dev):
        raise ValueError(f"plan is for B={plan.B} rows={plan.rows} Hq/Hkv={plan.group} on "
                         f"{plan.data.device}")
    h, s = _call_stream(stream, dev, (row_start, kv_len, page_table,
                                      plan.data if plan is not None else None))
    if plan is None:
        plan = ChunkPlan(B, T, G, geometry, _new(s, (need // 4,), (1,), torch.int32, dev))
    plan.geometry, plan.code = geometry, plan.code_of(geometry)
    _launch(dev, "spec_chunk_plan", (_lib or library()).spec_chunk_plan, row_start.data_ptr(),
            kv_len.data_ptr(), _ptr_of(page_table), B, T, G, *geometry, plan.data.data_ptr(), need,
            h)
    if plain:
        _keep((_PLAN, 0, 0, row_start, kv_len, q, k_cache, page_table), "spec_chunk_plan", _AS_PLAN,
              struct.pack("@5Q6i", 0, 0, 0, 0, need, B, T, G, *geometry), (0, 8, -1, -1, 16),
              (plan.data,), (24,), dev, extra=(B, T, G, geometry, plan.code))
    return plan


@functools.lru_cache(maxsize=256)
def spec_chunk_attention_workspace_size(Hq: int, Hkv: int, D: int) -> int:
    return int(library().spec_chunk_attention_workspace_size(Hq, Hkv, D))


def spec_chunk_attention(q, k_cache, v_cache, plan, page_table=None, scale=None, out=None,
                         want_lse=False, ws=None, stream=None):
    """Causal attention of chunks of new tokens over a cache that holds their keys
    and values already (include/spec_chunk.h).

    q [rows, Hq, D]; k_cache, v_cache [pages, slots, Hkv, D], bfloat16 or
    float16, any strides with a contiguous last dimension; plan from
    spec_chunk_plan; page_table int32 [B, pages_per_seq] or None; scale
    1 / sqrt(D) by default; ws of one call at a time, by default this thread's.
    Returns out [rows, Hq, D] (`out` may be a contiguous q, and shares no memory with other inputs)
    and, with want_lse, the rows' log-sum-exp float32 [rows, Hq]; rows of no sequence are left as they
    are.  Asynchronous like any CUDA op."""
    plain = scale is None and out is None and not want_lse and ws is None and stream is None
    if _run and plain:
        got = _run(_ATTEND, plan.code, 0, q, k_cache, v_cache, plan.data, page_table)
        if got is not None:
            return got
    torch = _torch()

    def check():
        if q.dim() != 3 or not k_cache.dim() == v_cache.dim() == 4:
            raise ValueError("q must be [rows, Hq, D], k_cache and v_cache "
                             "[pages, slots, Hkv, D]")
        T, Hq, D = q.shape
        Hkv, dtype, dev = k_cache.shape[2], q.dtype, q.device
        if dtype != torch.bfloat16 and dtype != torch.float16:
            raise TypeError(f"q must be bfloat16 or float16, got {dtype}")
        _caches(k_cache, v_cache, (), Hkv, D, dtype)
        geometry, _ = _geometry(k_cache, page_table, plan.B, dev)
        if ((plan.rows, plan.group * Hkv, plan.geometry) != (T, Hq, geometry)
                or plan.data.device != dev):
            raise ValueError(f"plan is for rows={plan.rows} Hq/Hkv={plan.group}, cache "
                             f"{plan.geometry} on {plan.data.device}; the call is for rows={T} "
                             f"Hq={Hq} Hkv={Hkv}, {geometry} on {dev}")
        strides = []
        for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache)):
            strides += _strided(name, t, dev, 8)[1]
        S = geometry[0]
        if page_table is not None and S % 128 and (S < 8 or S & (S - 1)):
            raise ValueError(f"page size {S}: a multiple of 128, or a power of two from 8")
        need = spec_chunk_attention_workspace_size(Hq, Hkv, D)
        if need == 0:
            raise ValueError(f"sizes out of range: Hq={Hq} Hkv={Hkv} D={D}")
        if out is not None:
            _dev_out("out", out, (T, Hq, D), dtype, dev)
        return (dev, (T, Hq, D), (Hq * D, D, 1), dtype, need, struct.pack("@8q", *strides),
                struct.pack("@9i", plan.B, T, Hq, Hkv, D, *geometry,
                            SPEC_BF16 if dtype == torch.bfloat16 else SPEC_F16))
    dev, shape, out_st, dtype, need, strides, sizes = _checked_chunk(
        (_meta(q), _meta(k_cache), _meta(v_cache), _meta(page_table), _meta(out), plan.B,
         plan.rows, plan.group, plan.geometry, plan.data.device), check)
    scale = shape[2] ** -0.5 if scale is None else float(scale)
    if not 0.0 < scale < float("inf"):
        raise ValueError(f"scale must be finite and positive, got {scale}")
    at = q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
    if (at[0] | at[1] | at[2]) & 15:
        raise ValueError("q, k_cache and v_cache must be 16-byte aligned")
    h, s = _call_stream(stream, dev, (q, k_cache, v_cache, plan.data, page_table, out, ws))
    if out is None:
        out = _new(s, shape, out_st, dtype, dev)
    lse = _empty_on(s, shape[:2], torch.float32, dev) if want_lse else None
    if ws is None:
        ws = _scratch(_chunk_ws, need, dev, h, s)
    else:
        _check_ws(ws, dev)
    args = b"".join((_pack_3q(*at), strides,
                     _pack_chunk(_ptr_of(page_table), plan.data.data_ptr(), out.data_ptr(),
                                 _ptr_of(lse), scale), sizes))
    _launch(dev, "spec_chunk_attention", (_lib or library()).spec_chunk_attention, args,
            ws.data_ptr(), ws.numel(), h)
    if plain:
        _keep((_ATTEND, plan.code, 0, q, k_cache, v_cache, plan.data, page_table),
              "spec_chunk_attention", _WITH_WORKSPACE, args, (0, 8, 16, 96, 88), (out,), (104,), dev,
              0, need)
    return (out, lse) if want_lse else out


# ------------------------------------------------------------ beam search

@functools.lru_cache(maxsize=256)
def spec_beam_workspace_size(B: int, K: int, V: int, n: int, dtype: int) -> int:
    return int(library().spec_beam_workspace_size(B, K, V, n, dtype))


def spec_beam_select(logits, scores, n, finished=None, norm=None, end_token=0, ws=None,
                     stream=None):
    """The n best continuations of each sequence's beams (include/spec_beam.h).

    logits [B, K, V] float32 or bfloat16; scores float32 [B, K]: the beams'
    log-probabilities so far; finished int32 [B, K]: beams that have ended, with
    end_token as their only candidate; norm float32 [B, K]: what a beam's
    candidates are divided by where they are compared.  ws: zeroed once, of one
    call at a time, by default this thread's.  Returns tokens, beams int32
    [B, n] and scores float32 [B, n], best first (-1, -1 and -inf where there
    are fewer); asynchronous like any CUDA op."""
    plain = ws is None and stream is None
    if _run and plain:
        got = _run(_SELECT, n, end_token, logits, scores, finished, norm)
        if got is not None:
            return got
    torch = _torch()

    def check():
        if logits.dim() != 3:
            raise ValueError("logits must be [B, K, V]")
        B, K, V = logits.shape
        dt = _dtype_code(logits)
        dev, f32 = logits.device, torch.float32
        if not logits.is_cuda or not logits.is_contiguous():
            raise ValueError("logits must be a contiguous CUDA tensor")
        need = spec_beam_workspace_size(B, K, V, n, dt)
        if need == 0:
            raise ValueError(f"sizes out of range: B={B} K={K} V={V} n={n}")
        if not 0 <= end_token < V:
            raise ValueError(f"end_token must be in [0, {V}), got {end_token}")
        _array("scores", scores, (B, K), f32, dev)
        if finished is not None:
            _array("finished", finished, (B, K), torch.int32, dev)
        if norm is not None:
            _array("norm", norm, (B, K), f32, dev)
        return dev, (B, n), need, struct.pack("@6i", B, K, V, n, end_token, dt)
    dev, shape, need, sizes = _checked_beam(
        (_meta(logits), _meta(scores), _meta(finished), _meta(norm), n, end_token), check)
    h, s = _call_stream(stream, dev, (logits, scores, finished, norm, ws))
    st = (n, 1)
    tokens, beams = _new(s, shape, st, torch.int32, dev), _new(s, shape, st, torch.int32, dev)
    best = _new(s, shape, st, torch.float32, dev)
    if ws is None:
        ws = _scratch(_beam_ws, need, dev, h, s, zeroed=True)
    else:
        _check_ws(ws, dev)
    args = _pack_beam(logits.data_ptr(), scores.data_ptr(), _ptr_of(norm), _ptr_of(finished),
                      tokens.data_ptr(), beams.data_ptr(), best.data_ptr()) + sizes
    _launch(dev, "spec_beam_select", (_lib or library()).spec_beam_select, args, ws.data_ptr(),
            ws.numel(), h)
    if plain:
        _keep((_SELECT, n, end_token, logits, scores, finished, norm), "spec_beam_select",
              _WITH_WORKSPACE, args, (0, 8, 24, 16), (tokens, beams, best), (32, 40, 48), dev, 1,
              need)
    return tokens, beams, best


def spec_beam_reorder(state, beams, dim=0, out=None, stream=None):
    """The beams' states in the order of the selected (include/spec_beam.h).

    state [.., B, K, ..] contiguous, of any dtype, B its dimension `dim`; beams
    int32 [B, n] from spec_beam_select.  Returns [.., B, n, ..], where the place
    of a beam -1 is 0; asynchronous like any CUDA op."""
    plain = out is None and stream is None
    if _run and plain:
        got = _run(_REORDER, dim, 0, state, beams)
        if got is not None:
            return got
    torch = _torch()
    if state.dtype.is_complex:  # a view may stand for other numbers than its memory holds
        with torch.cuda.stream(stream):
            state = state.resolve_conj().resolve_neg()
        if out is not None and (out.is_conj() or out.is_neg()):
            raise ValueError("out must not be a conjugated or negated view")

    def check():
        if not 0 <= dim <= state.dim() - 2 or beams.dim() != 2:
            raise ValueError("state must be [.., B, K, ..] with B at `dim`, and beams [B, n]")
        B, K = state.shape[dim:dim + 2]
        n, dev = beams.shape[1], state.device
        if not state.is_cuda or not state.is_contiguous():
            raise ValueError("state must be a contiguous CUDA tensor")
        _array("beams", beams, (B, n), torch.int32, dev)
        shape = (*state.shape[:dim], B, n, *state.shape[dim + 2:])
        if out is not None:
            _dev_out("out", out, shape, state.dtype, dev)
        return (dev, shape, _strides_of(shape), state.dtype,
                (math.prod(state.shape[:dim]), B, K, n,
                 math.prod(state.shape[dim + 2:]) * state.element_size()))
    dev, shape, st, dtype, sizes = _checked_reorder((_meta(state), _meta(beams), _meta(out), dim), check)
    h, s = _call_stream(stream, dev, (state, beams, out))
    if out is None:
        out = _new(s, shape, st, dtype, dev)
    _launch(dev, "spec_beam_reorder", (_lib or library()).spec_beam_reorder, state.data_ptr(),
            beams.data_ptr(), out.data_ptr(), *sizes, h)
    if plain:
        _keep((_REORDER, dim, 0, state, beams), "spec_beam_reorder", _AS_REORDER,
              struct.pack("@3Q4iq", 0, 0, 0, *sizes), (0, 8), (out,), (16,), dev)
    return out


# --------------------------------------------------------- pages of a cache

@functools.lru_cache(maxsize=256)
def spec_pages_workspace_size(rows_out: int, num_pages: int) -> int:
    return int(library().spec_pages_workspace_size(rows_out, num_pages))


def _pages_workspace_size(rows, pages):
    need = spec_pages_workspace_size(rows, pages)
    if need == 0:
        raise ValueError(f"sizes out of range: rows={rows} pages={pages}")
    return need


def _check_outs(given, shapes, dev):
    """The caller's int32 outputs of a call."""
    if given is None:
        return
    if len(given) != len(shapes):
        raise ValueError(f"out must be {len(shapes)} tensors")
    for i, (t, shape) in enumerate(zip(given, shapes)):
        _dev_out(f"out[{i}]", t, shape, _torch().int32, dev)


def _pages_call(name, call, in_at, pointers, sizes, shapes, need, out, ws, dev, h, s):
    """The outputs and the workspace where the caller gave none, and the launch; `call` as
    _keep's, or None."""
    i32 = _torch().int32
    out = tuple(out) if out is not None else tuple([_new(s, *x, i32, dev) for x in shapes])
    if ws is None:
        ws = _scratch(_pages_ws, need, dev, h, s)
    else:
        _check_ws(ws, dev)
    args = b"".join((pointers, _pack_4q(*[t.data_ptr() for t in out]), sizes))
    _launch(dev, name, getattr(_lib or library(), name), args, ws.data_ptr(), ws.numel(), h)
    if call is not None:
        at = len(pointers)
        _keep(call, name, _WITH_WORKSPACE, args, in_at, out, (at, at + 8, at + 16, at + 24), dev, 2,
              need)
    return out


def spec_pages_fork(table, length, parent, ref_count, page_size, reserve=None, out=None, ws=None,
                    stream=None):
    """New rows of a page table from old ones (include/spec_pages.h): row r takes
    over row parent[r], sharing its whole pages, or starts empty (-1).

    table int32 [rows, pages_per_seq], length int32 [rows], parent int32
    [rows_out], ref_count int32 [num_pages] (0: free); reserve int32
    [rows_out]: tokens to have pages for besides.  Returns the new table,
    lengths, reference counts and copies int32 [3, rows_out] for spec_pages_copy
    (before the next call that takes pages).  `out`: those four, none of them an
    input.  Asynchronous like any CUDA op."""
    plain = out is None and ws is None and stream is None
    if _run and plain:
        got = _run(_FORK, page_size, 0, table, length, parent, ref_count, reserve)
        if got is not None:
            return got

    def check():
        if table.dim() != 2 or parent.dim() != 1 or ref_count.dim() != 1:
            raise ValueError("table must be [rows, pages_per_seq], parent [rows_out], "
                             "ref_count [pages]")
        (R0, M), R, P = table.shape, parent.shape[0], ref_count.shape[0]
        dev, i32 = table.device, _torch().int32
        _array("table", table, (R0, M), i32, dev)
        _array("length", length, (R0,), i32, dev)
        _array("parent", parent, (R,), i32, dev)
        _array("ref_count", ref_count, (P,), i32, dev)
        if reserve is not None:
            _array("reserve", reserve, (R,), i32, dev)
        shapes = ((R, M), (R,), (P,), (3, R))
        _check_outs(out, shapes, dev)
        return (dev, tuple((x, _strides_of(x)) for x in shapes), _pages_workspace_size(R, P),
                struct.pack("@5i4x", R0, R, M, page_size, P))
    dev, shapes, need, sizes = _checked_fork(
        (_meta(table), _meta(length), _meta(parent), _meta(ref_count), _meta(reserve), page_size,
         None if out is None else tuple([_meta(t) for t in out])), check)
    h, s = _call_stream(stream, dev, (table, length, parent, ref_count, reserve, ws,
                                      *(out if out is not None else ())))
    pointers = _pack_5q(table.data_ptr(), length.data_ptr(), parent.data_ptr(), _ptr_of(reserve),
                        ref_count.data_ptr())
    call = (_FORK, page_size, 0, table, length, parent, ref_count, reserve) if plain else None
    return _pages_call("spec_pages_fork", call, (0, 8, 16, 32, 24), pointers, sizes, shapes, need, out,
                       ws, dev, h, s)


def spec_pages_compact(table, ref_count, page_size, out=None, ws=None, stream=None):
    """The pages in use to the front of the pool (include/spec_pages.h).

    table int32 [rows, pages_per_seq]: all tables over the pool; ref_count
    int32 [num_pages].  Returns the new table, reference counts, copies int32
    [3, num_pages // 2] for spec_pages_copy and the number of pages in use
    int32 [1].  `out`: those four, none of them an input.  Asynchronous like any
    CUDA op."""
    plain = out is None and ws is None and stream is None
    if _run and plain:
        got = _run(_COMPACT, page_size, 0, table, ref_count)
        if got is not None:
            return got

    def check():
        if table.dim() != 2 or ref_count.dim() != 1:
            raise ValueError("table must be [rows, pages_per_seq], ref_count [pages]")
        (R, M), P = table.shape, ref_count.shape[0]
        dev, i32 = table.device, _torch().int32
        _array("table", table, (R, M), i32, dev)
        _array("ref_count", ref_count, (P,), i32, dev)
        shapes = ((R, M), (P,), (3, P // 2), (1,))
        _check_outs(out, shapes, dev)
        return (dev, tuple((x, _strides_of(x)) for x in shapes), _pages_workspace_size(R, P),
                struct.pack("@4i", R, M, page_size, P))
    dev, shapes, need, sizes = _checked_compact(
        (_meta(table), _meta(ref_count), page_size,
         None if out is None else tuple([_meta(t) for t in out])), check)
    h, s = _call_stream(stream, dev, (table, ref_count, ws, *(out if out is not None else ())))
    pointers = struct.pack("@2Q", table.data_ptr(), ref_count.data_ptr())
    call = (_COMPACT, page_size, 0, table, ref_count) if plain else None
    return _pages_call("spec_pages_compact", call, (0, 8), pointers, sizes, shapes, need, out, ws, dev,
                       h, s)


def spec_pages_copy(k_cache, v_cache, copies, stream=None):
    """Copy pages within the caches, in every layer (include/spec_pages.h).

    k_cache, v_cache [pages, slots, Hkv, D] or with a leading dimension of
    layers, 2 or 4 bytes an element, any strides with a contiguous last
    dimension; copies int32 [3, n]: sources, destinations and numbers of slots
    (-1, -1, 0: nothing).  Asynchronous like any CUDA op."""
    if _run and stream is None and _run(_COPY, 0, 0, k_cache, v_cache, copies):
        return

    def check():
        if k_cache.dim() not in (4, 5) or v_cache.shape != k_cache.shape:
            raise ValueError("k_cache and v_cache must be [.., pages, slots, Hkv, D]")
        if v_cache.dtype != k_cache.dtype or k_cache.element_size() not in (2, 4):
            raise TypeError("k_cache and v_cache must share a dtype of 2 or 4 bytes")
        if copies.dim() != 2 or copies.shape[0] != 3:
            raise ValueError("copies must be [3, n]")
        *lead, P, S, Hkv, D = k_cache.shape
        dev, n = k_cache.device, copies.shape[1]
        _array("copies", copies, (3, n), _torch().int32, dev)
        strides = []
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            st = _strided(name, t, dev, 1)[1]
            strides += st if lead else (0, *st)
        return (dev, struct.pack("@8q", *strides),
                struct.pack("@7i4x", n, lead[0] if lead else 1, Hkv, D, S, P,
                            k_cache.element_size()))
    dev, strides, sizes = _checked_copy((_meta(k_cache), _meta(v_cache), _meta(copies)), check)
    h, _ = _call_stream(stream, dev, (k_cache, v_cache, copies))
    args = b"".join((struct.pack("@2Q", k_cache.data_ptr(), v_cache.data_ptr()), strides,
                     struct.pack("@Q", copies.data_ptr()), sizes))
    _launch(dev, "spec_pages_copy", (_lib or library()).spec_pages_copy, args, h)
    if stream is None:
        _keep((_COPY, 0, 0, k_cache, v_cache, copies), "spec_pages_copy", _AS_ARGS, args, (0, 8, 80), (),
              (), dev)
