"""GB300-native chunked gated-delta-rule (GDN) prefill forward, and the softmax-attention
operators that stand next to it in a hybrid model.

A thin ctypes binding over the C ABI in ``include/gdn_prefill.h`` and
``include/gdn_attention.h``; every step
of the computation runs in the library's CUDA kernels. PyTorch only supplies
device memory and the current stream. There is no fallback: if the compiled
library is missing, importing works but every call raises ``GdnError``.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

__all__ = ["prefill", "prefill_noalloc", "prefill_host", "host_scratch_bytes", "NOALLOC_MAX_SEQS", "workspace_bytes", "check", "last_launch_count",
           "backward", "backward_workspace_bytes",
           "head_norm_rope", "head_norm_rope_backward", "head_norm_rope_backward_workspace_bytes", "paged_append",
           "tree_attention", "tree_attention_workspace_bytes",
           "set_timing_events", "set_test_hooks", "decode", "lib_path", "load", "GdnError",
           "Strides", "Rope", "NormStrides", "Paged", "GDN_OK", "GDN_ERR_ARG", "GDN_ERR_UNSUPPORTED", "GDN_ERR_CUDA",
           "GDN_ERR_DEVICE_STATUS", "GDN_ERR_TIMEOUT", "GDN_ERR_RANGE"]

(GDN_OK, GDN_ERR_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_CUDA, GDN_ERR_DEVICE_STATUS, GDN_ERR_TIMEOUT,
 GDN_ERR_RANGE) = range(7)
NOALLOC_MAX_SEQS = 16384  # GDN_NOALLOC_MAX_SEQS in include/gdn_prefill.h

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_lib", "libgdn_gb300.so")
_lock = threading.Lock()
_lib = None


class GdnError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"gdn error {code}: {message}")
        self.code = code


class Strides(ctypes.Structure):
    _fields_ = [("q", ctypes.c_int64), ("k", ctypes.c_int64), ("v", ctypes.c_int64),
                ("g", ctypes.c_int64), ("beta", ctypes.c_int64), ("out", ctypes.c_int64),
                ("state_is_table", ctypes.c_int32), ("qk_l2norm", ctypes.c_int32)]


class Rope(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("stride", ctypes.c_int64),
                ("positions", ctypes.c_int32), ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class NormStrides(ctypes.Structure):
    _fields_ = [("q", ctypes.c_int64), ("k", ctypes.c_int64), ("q_out", ctypes.c_int64), ("k_out", ctypes.c_int64),
                ("q_grad", ctypes.c_int64), ("k_grad", ctypes.c_int64)]


class Paged(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_page", ctypes.c_int64), ("k_token", ctypes.c_int64),
                ("k_head", ctypes.c_int64), ("v_page", ctypes.c_int64), ("v_token", ctypes.c_int64),
                ("v_head", ctypes.c_int64), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("max_pages", ctypes.c_int32),
                ("B", ctypes.c_int32), ("rows", ctypes.c_int32), ("ctx_lens", ctypes.c_void_p),
                ("cu_rows", ctypes.c_void_p)]


def lib_path() -> str:
    return _LIB_PATH


def load():
    """Load the compiled library (raises GdnError if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise GdnError(GDN_ERR_UNSUPPORTED, f"CUDA library not built: {_LIB_PATH} is missing "
                                                    "(run __graft_entry__.build())")
            lib = ctypes.CDLL(_LIB_PATH)
            vp, i, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
            common = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, ctypes.POINTER(Strides), vp]
            lib.gdn_prefill.argtypes = common + [vp]
            lib.gdn_prefill.restype = i
            lib.gdn_prefill_ex.argtypes = common + [vp, sz, vp]
            lib.gdn_prefill_ex.restype = i
            lib.gdn_prefill_workspace_bytes.argtypes = [i, i, i, i, i, i]
            lib.gdn_prefill_workspace_bytes.restype = sz
            lib.gdn_prefill_check.argtypes = [vp]
            lib.gdn_prefill_check.restype = i
            lib.gdn_last_error.argtypes = []
            lib.gdn_last_error.restype = ctypes.c_char_p
            lib.gdn_last_launch_count.argtypes = []
            lib.gdn_last_launch_count.restype = i
            lib.gdn_prefill_noalloc.argtypes = common + [vp]
            lib.gdn_prefill_noalloc.restype = i
            lib.gdn_prefill_host.argtypes = common + [vp, sz, vp]
            lib.gdn_prefill_host.restype = i
            lib.gdn_prefill_host_scratch_bytes.argtypes = [i, i, i, i, i, i, i]
            lib.gdn_prefill_host_scratch_bytes.restype = sz
            lib.gdn_decode.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, ctypes.POINTER(Strides), vp]
            lib.gdn_decode.restype = i
            lib.gdn_prefill_backward_workspace_bytes.argtypes = [i, i, i, i, i, i]
            lib.gdn_prefill_backward_workspace_bytes.restype = sz
            lib.gdn_prefill_backward.argtypes = [vp] * 14 + [i] * 6 + [ctypes.POINTER(Strides), vp, vp, sz, vp]
            lib.gdn_prefill_backward.restype = i
            f32 = ctypes.c_float
            rope = norm_st = paged = vp  # Rope, NormStrides, Paged: by address
            lib.gdn_head_norm_rope.argtypes = [vp, vp, vp, rope, vp, vp, f32, vp, vp] + [i] * 5 + [norm_st, vp]
            lib.gdn_head_norm_rope.restype = i
            lib.gdn_head_norm_rope_backward_workspace_bytes.argtypes = [i] * 4
            lib.gdn_head_norm_rope_backward_workspace_bytes.restype = sz
            lib.gdn_head_norm_rope_backward.argtypes = ([vp, vp, vp, rope, vp, vp, f32] + [vp] * 6 + [i] * 5
                                                        + [norm_st, vp, sz, vp])
            lib.gdn_head_norm_rope_backward.restype = i
            lib.gdn_paged_append.argtypes = [vp, vp, paged, vp, rope, i, vp, f32, i, i, i, i64, i64, vp]
            lib.gdn_paged_append.restype = i
            lib.gdn_tree_attention_workspace_bytes.argtypes = [i] * 3
            lib.gdn_tree_attention_workspace_bytes.restype = sz
            lib.gdn_tree_attention.argtypes = [vp, paged, vp, i, f32, vp, i, i, i, i, i64, i64, i, vp, sz, vp]
            lib.gdn_tree_attention.restype = i
            lib.gdn_set_timing_events.argtypes = [vp, vp, vp]
            lib.gdn_set_timing_events.restype = None
            lib.gdn_set_test_hooks.argtypes = [i64, i64, i]
            lib.gdn_set_test_hooks.restype = i
            _lib = lib
    return _lib


def _raise(code):
    msg = load().gdn_last_error().decode(errors="replace")
    raise GdnError(code, msg)


def _row_stride(t, name, inner):
    """Row stride (elements) of a [rows, ...] tensor whose per-row part is contiguous."""
    if t.dim() < 2:
        raise GdnError(GDN_ERR_ARG, f"{name} must be at least 2-D ([rows, ...])")
    per_row = 1
    for d in t.shape[1:]:
        per_row *= d
    expect = 1
    for d in range(t.dim() - 1, 0, -1):
        if t.shape[d] != 1 and t.stride(d) != expect:
            raise GdnError(GDN_ERR_ARG, f"{name}: the part of each row must be contiguous")
        expect *= t.shape[d]
    if per_row < inner:
        raise GdnError(GDN_ERR_ARG, f"{name}: rows hold {per_row} elements, need {inner}")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), per_row)


def workspace_bytes(B, T, nv, varlen, dk=128, dv=128) -> int:
    return int(load().gdn_prefill_workspace_bytes(B, T, nv, dk, dv, 1 if varlen else 0))


# The library takes raw device addresses, so a host tensor or a wrong element type
# handed to it would reach a kernel; these checks turn that into a GdnError first.
def _check_rows(torch, named):
    for name, t, dt in named:
        if t.dtype != dt:
            raise GdnError(GDN_ERR_ARG, f"{name} must be {dt}, got {t.dtype}")
        if not t.is_cuda:
            raise GdnError(GDN_ERR_ARG, f"{name} must be a CUDA tensor")


def _check_state(torch, state, state_is_table, name="state"):
    if not state.is_cuda:
        raise GdnError(GDN_ERR_ARG, f"{name} must be a CUDA tensor")
    if state_is_table:
        if state.dtype != torch.int64 or not state.is_contiguous():
            raise GdnError(GDN_ERR_ARG, f"a {name} table must be a contiguous int64 tensor of device addresses")
    elif state.dtype != torch.float32 or not state.is_contiguous():
        raise GdnError(GDN_ERR_ARG, f"{name} must be a contiguous fp32 tensor [B, nv, dk, dv]")


def _check_aux(torch, cu_seqlens, workspace):
    if cu_seqlens is not None and (cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda
                                   or not cu_seqlens.is_contiguous()):
        raise GdnError(GDN_ERR_ARG, "cu_seqlens must be a contiguous int32 CUDA tensor")
    if workspace is not None and (not workspace.is_cuda or not workspace.is_contiguous()):
        raise GdnError(GDN_ERR_ARG, "workspace must be a contiguous CUDA tensor")


def _io_rows(torch, q, k, v, g, beta, last):
    return (("q", q, torch.bfloat16), ("k", k, torch.bfloat16), ("v", v, torch.bfloat16),
            ("g", g, torch.float32), ("beta", beta, torch.float32), last)


def prefill(q, k, v, g, beta, state, out, *, nk: int, nv: int, B: int | None = None, T: int | None = None,
            cu_seqlens=None, state_is_table: bool = False, workspace=None, stream=None, dk: int = 128,
            dv: int = 128, qk_l2norm: bool = False) -> None:
    """Enqueue one GDN prefill on ``stream`` (default: torch's current stream).

    q, k: bf16 CUDA tensors [rows, nk*dk] (or [rows, nk, dk]); v: bf16 [rows, nv*dv];
    g, beta: fp32 [rows, nv]; out: bf16 [rows, nv*dv]. ``state``: fp32 CUDA tensor
    [B, nv, dk, dv] updated in place, or (``state_is_table``) an int64 CUDA tensor of
    B device addresses of [nv, dk, dv] fp32 states. Dense batches give ``B`` and ``T``
    (rows = B*T); varlen batches give ``cu_seqlens`` (int32 CUDA [B+1]).
    ``workspace`` (uint8 CUDA tensor) passes caller-provided scratch (``gdn_prefill_ex``).
    ``qk_l2norm`` normalises every q and k head row inside the kernels (fused prologue).
    """
    import torch

    lib = load()
    _check_rows(torch, _io_rows(torch, q, k, v, g, beta, ("out", out, torch.bfloat16)))
    _check_state(torch, state, state_is_table)
    _check_aux(torch, cu_seqlens, workspace)
    rows = q.shape[0]
    if cu_seqlens is not None:
        B = cu_seqlens.numel() - 1
        T = rows
    elif B is None or T is None:
        raise GdnError(GDN_ERR_ARG, "dense batches need B and T")
    st = Strides(_row_stride(q, "q", nk * dk), _row_stride(k, "k", nk * dk), _row_stride(v, "v", nv * dv),
                 _row_stride(g, "g", nv), _row_stride(beta, "beta", nv), _row_stride(out, "out", nv * dv),
                 1 if state_is_table else 0, 1 if qk_l2norm else 0)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    args = [q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), state.data_ptr(),
            out.data_ptr(), B, T, nk, nv, dk, dv, ctypes.byref(st),
            None if cu_seqlens is None else cu_seqlens.data_ptr()]
    if workspace is None:
        rc = lib.gdn_prefill(*args, stream)
    else:
        rc = lib.gdn_prefill_ex(*args, workspace.data_ptr() if workspace.numel() else None,
                                workspace.numel() * workspace.element_size(), stream)
    if rc != GDN_OK:
        _raise(rc)


def prefill_noalloc(q, k, v, g, beta, state, out, *, nk: int, nv: int, B: int | None = None,
                    T: int | None = None, cu_seqlens=None, state_is_table: bool = False, stream=None,
                    dk: int = 128, dv: int = 128, qk_l2norm: bool = False) -> None:
    """``prefill`` through ``gdn_prefill_noalloc``: the library allocates no device
    memory during the call (its varlen schedule lives in a static device array of
    ``NOALLOC_MAX_SEQS`` entries). For callers that cannot allocate mid-call.
    Calls that overlap on the GPU race on that shared array."""
    import torch

    lib = load()
    _check_rows(torch, _io_rows(torch, q, k, v, g, beta, ("out", out, torch.bfloat16)))
    _check_state(torch, state, state_is_table)
    _check_aux(torch, cu_seqlens, None)
    if cu_seqlens is not None:
        B = cu_seqlens.numel() - 1
        T = q.shape[0]
    elif B is None or T is None:
        raise GdnError(GDN_ERR_ARG, "dense batches need B and T")
    st = Strides(_row_stride(q, "q", nk * dk), _row_stride(k, "k", nk * dk), _row_stride(v, "v", nv * dv),
                 _row_stride(g, "g", nv), _row_stride(beta, "beta", nv), _row_stride(out, "out", nv * dv),
                 1 if state_is_table else 0, 1 if qk_l2norm else 0)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    rc = lib.gdn_prefill_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                                 state.data_ptr(), out.data_ptr(), B, T, nk, nv, dk, dv, ctypes.byref(st),
                                 None if cu_seqlens is None else cu_seqlens.data_ptr(), stream)
    if rc != GDN_OK:
        _raise(rc)


def host_scratch_bytes(B, T, nk, nv, varlen, dk=128, dv=128) -> int:
    """Device scratch of ``prefill_host`` (``gdn_prefill_host_scratch_bytes``)."""
    return int(load().gdn_prefill_host_scratch_bytes(B, T, nk, nv, dk, dv, 1 if varlen else 0))


def prefill_host(q, k, v, g, beta, state, out, *, nk: int, nv: int, B: int | None = None, T: int | None = None,
                 cu_seqlens=None, scratch=None, stream=None, dk: int = 128, dv: int = 128,
                 qk_l2norm: bool = False) -> None:
    """``gdn_prefill_host``: the prefill over page-locked host tensors (``pin_memory()``),
    packed as for ``prefill`` (q, k [rows, nk*dk] bf16; v, out [rows, nv*dv] bf16; g, beta
    [rows, nv] fp32; state [B, nv, dk, dv] fp32, updated in place; cu_seqlens int32 [B+1]).
    Enqueued on ``stream`` (default: torch's current CUDA stream); the host tensors must
    stay untouched until that stream passes the call. ``scratch``: optional uint8 CUDA
    tensor of ``host_scratch_bytes(...)`` bytes (else allocated stream-ordered)."""
    import torch

    lib = load()
    named = [("q", q, torch.bfloat16), ("k", k, torch.bfloat16), ("v", v, torch.bfloat16), ("g", g, torch.float32),
             ("beta", beta, torch.float32), ("state", state, torch.float32), ("out", out, torch.bfloat16)]
    if cu_seqlens is not None:
        named.append(("cu_seqlens", cu_seqlens, torch.int32))
    for name, t, dt in named:
        if t.device.type != "cpu" or not t.is_pinned():
            raise GdnError(GDN_ERR_ARG, f"{name} must be a page-locked CPU tensor (pin_memory())")
        if t.dtype != dt or not t.is_contiguous():
            raise GdnError(GDN_ERR_ARG, f"{name} must be a contiguous {dt} tensor")
    if scratch is not None and (not scratch.is_cuda or scratch.dtype != torch.uint8):
        raise GdnError(GDN_ERR_ARG, "scratch must be a uint8 CUDA tensor")
    rows = q.shape[0]
    if cu_seqlens is not None:
        B = cu_seqlens.numel() - 1
        T = rows
    elif B is None or T is None:
        raise GdnError(GDN_ERR_ARG, "dense batches need B and T")
    st = Strides(nk * dk, nk * dk, nv * dv, nv, nv, nv * dv, 0, 1 if qk_l2norm else 0)
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    rc = lib.gdn_prefill_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                              state.data_ptr(), out.data_ptr(), B, T, nk, nv, dk, dv, ctypes.byref(st),
                              None if cu_seqlens is None else cu_seqlens.data_ptr(),
                              None if scratch is None or not scratch.numel() else scratch.data_ptr(),
                              0 if scratch is None else scratch.numel(), stream)
    if rc != GDN_OK:
        _raise(rc)


def decode(q, k, v, g, beta, state, out, *, nk: int, nv: int, state_is_table: bool = False, stream=None,
           dk: int = 128, dv: int = 128, qk_l2norm: bool = False) -> None:
    """Enqueue one single-token decode step for every row (sequence) b of q/k/v/g/beta/out:
    the state of sequence b (``state[b]``, or the b-th pointer of a table) is advanced by
    that token and the token's output written to ``out[b]``. Same layouts as ``prefill``."""
    import torch

    lib = load()
    _check_rows(torch, _io_rows(torch, q, k, v, g, beta, ("out", out, torch.bfloat16)))
    _check_state(torch, state, state_is_table)
    st = Strides(_row_stride(q, "q", nk * dk), _row_stride(k, "k", nk * dk), _row_stride(v, "v", nv * dv),
                 _row_stride(g, "g", nv), _row_stride(beta, "beta", nv), _row_stride(out, "out", nv * dv),
                 1 if state_is_table else 0, 1 if qk_l2norm else 0)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    rc = lib.gdn_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), state.data_ptr(),
                        out.data_ptr(), q.shape[0], nk, nv, dk, dv, ctypes.byref(st), stream)
    if rc != GDN_OK:
        _raise(rc)


def backward_workspace_bytes(B, T, nv, varlen, dk=128, dv=128) -> int:
    return int(load().gdn_prefill_backward_workspace_bytes(B, T, nv, dk, dv, 1 if varlen else 0))


def backward(q, k, v, g, beta, h0, dout, dq, dk, dv, dg, dbeta, *, nk: int, nv: int, dST=None, dh0=None,
             B: int | None = None, T: int | None = None, cu_seqlens=None, state_is_table: bool = False,
             workspace=None, stream=None, dk_dim: int = 128, dv_dim: int = 128) -> None:
    """Enqueue the backward of ``prefill`` (``gdn_prefill_backward``): the chunked form
    on the tensor cores, 4 launches (5 with ``cu_seqlens``).

    q, k, v, g, beta, cu_seqlens, state_is_table: as ``prefill``; ``h0`` is the initial
    state the forward started from. ``dout`` fp32 [rows, nv*dv] (dL/do), ``dST`` fp32
    [B, nv, dk, dv] or None. Outputs (fp32): dq, dk [rows, nk*dk], dv [rows, nv*dv],
    dg, dbeta [rows, nv], dh0 [B, nv, dk, dv] or None.
    """
    import torch

    lib = load()
    _check_rows(torch, _io_rows(torch, q, k, v, g, beta, ("dout", dout, torch.float32)))
    _check_state(torch, h0, state_is_table, name="h0")
    _check_aux(torch, cu_seqlens, workspace)
    for name, t in (("dout", dout), ("dq", dq), ("dk", dk), ("dv", dv), ("dg", dg), ("dbeta", dbeta),
                    ("dST", dST), ("dh0", dh0)):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or not t.is_cuda):
            raise GdnError(GDN_ERR_ARG, f"{name} must be a contiguous fp32 CUDA tensor")
    rows = q.shape[0]
    if cu_seqlens is not None:
        B = cu_seqlens.numel() - 1
        T = rows
    elif B is None or T is None:
        raise GdnError(GDN_ERR_ARG, "dense batches need B and T")
    st = Strides(_row_stride(q, "q", nk * dk_dim), _row_stride(k, "k", nk * dk_dim), _row_stride(v, "v", nv * dv_dim),
                 _row_stride(g, "g", nv), _row_stride(beta, "beta", nv), nv * dv_dim,
                 1 if state_is_table else 0, 0)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream

    def ptr(t):
        return None if t is None else t.data_ptr()

    ws_ptr, ws_size = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    rc = lib.gdn_prefill_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), h0.data_ptr(),
                                  dout.data_ptr(), ptr(dST), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dg.data_ptr(),
                                  dbeta.data_ptr(), ptr(dh0), B, T, nk, nv, dk_dim, dv_dim, ctypes.byref(st),
                                  ptr(cu_seqlens), ws_ptr, ws_size, stream)
    if rc != GDN_OK:
        _raise(rc)


# ---- the softmax-attention operators (include/gdn_attention.h) ----------------------------
# A decode step makes several of these calls a layer, each a few microseconds on the GPU, so the
# checks below touch every attribute of a tensor once and take the common layout first.

_torch = None   # torch, once one of the calls below has been made
_codes = {}     # torch dtype -> the ABI's number
_cards = 0      # devices of this process
# The ABI's structs, packed: the bytes of Rope, NormStrides and Paged (a fraction of a ctypes object's cost)
_ROPE = struct.Struct("@QQqiii4x").pack
_STRIDES = struct.Struct("@6q").pack
_PAGED = struct.Struct("@QQqqqqqqiiQqiii4xQQ").pack


def _setup():
    global _torch, _cards
    import torch

    load()
    _cards = torch.cuda.device_count()
    _codes.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    _torch = torch
    return torch


def _stream_of(stream, t):
    if stream is None:  # the handle itself: a torch.cuda.Stream around it costs a sixth of a call
        return _torch._C._cuda_getCurrentRawStream(t.get_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _one_card(**tensors):
    """All tensors have to be on the current device, where the launch goes. Asked where there are several devices; else
    a CUDA tensor has nowhere else to be, and the question costs up to a tenth of a call."""
    here = _torch._C._cuda_getDevice()
    for name, t in tensors.items():
        if t is not None and t.get_device() != here:
            raise GdnError(GDN_ERR_ARG, f"{name} is on {t.device}, the current device is cuda:{here}")


def _act_code(t, name, most):
    """The ABI's number of an activation type: bf16 0, fp16 1, fp32 2 (up to `most`)."""
    code = _codes.get(t.dtype, 9)
    if code > most:
        raise GdnError(GDN_ERR_ARG, f"{name} must be {' or '.join(('bfloat16', 'float16', 'float32')[:most + 1])}, got {t.dtype}")
    return code


def _act(t, name, dtype, rows, inner):
    """Checks [rows, ...] activations with `inner` contiguous elements a row; (address, row stride)."""
    if t.dtype is not dtype or not t.is_cuda:
        raise GdnError(GDN_ERR_ARG, f"{name} must be a {dtype} CUDA tensor, got {t.dtype} on {t.device}")
    if t.numel() == rows * inner and t.is_contiguous():  # packed rows, however they are split up
        return t.data_ptr(), inner
    stride = _row_stride(t, name, inner)
    if t.shape[0] != rows:
        raise GdnError(GDN_ERR_ARG, f"{name} has {t.shape[0]} rows, need {rows}")
    if t.numel() != rows * inner:  # [B, T, ...] in place of [B * T, ...], or heads that no one would touch
        raise GdnError(GDN_ERR_ARG, f"{name}: rows hold {t.numel() // rows} elements, need just {inner}")
    return t.data_ptr(), stride


def _vector(t, name, dtype, n):
    """The address of a contiguous CUDA vector of n elements, or None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or not t.is_cuda or t.numel() != n or not t.is_contiguous():
        raise GdnError(GDN_ERR_ARG, f"{name} must be a contiguous {dtype} CUDA tensor of {n} elements")
    return t.data_ptr()


def _rope(cos, sin, interleaved):
    """The tables as the ABI's struct, packed."""
    if cos is None or sin is None:
        if cos is not sin:
            raise GdnError(GDN_ERR_ARG, "cos and sin must be given together")
        return None
    f32, shape = _torch.float32, cos.shape
    if cos.dtype is not f32 or sin.dtype is not f32 or not cos.is_cuda or not sin.is_cuda or len(shape) != 2 or sin.shape != shape:
        raise GdnError(GDN_ERR_ARG, "cos and sin must be fp32 CUDA tensors [positions, rot/2], both alike")
    n, half = shape
    stride = half
    if not (cos.is_contiguous() and sin.is_contiguous()):
        st = cos.stride()
        if sin.stride() != st or (st[1] != 1 and half > 1):
            raise GdnError(GDN_ERR_ARG, "cos and sin must be contiguous in a row, with the same row stride")
        stride = st[0] if n > 1 else max(st[0], half)
    return _ROPE(cos.data_ptr(), sin.data_ptr(), stride, n, 2 * half, 1 if interleaved else 0)


def _scratch(workspace):
    if workspace is None:
        return None, 0
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise GdnError(GDN_ERR_ARG, "workspace must be a contiguous CUDA tensor")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _heads_given(q, k, nq, nkv):
    if (q is None) != (nq == 0) or (k is None) != (nkv == 0) or (q is None and k is None):
        raise GdnError(GDN_ERR_ARG, "q (k) is None just where nq (nkv) is 0, and one of them is given")
    return q if q is not None else k


_NONE = (None, 0)


def head_norm_rope(q, k, positions, cos, sin, q_out, k_out, *, nq: int, nkv: int, head_dim: int = 128, q_weight=None,
                   k_weight=None, eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
    """RMS norm of every query and key head row, then the position rotation, in one pass
    (``gdn_head_norm_rope``): y = rotate(x / sqrt(mean(x^2) + eps) * weight).

    q, q_out: [rows, nq*head_dim] (or [rows, nq, head_dim]); k, k_out likewise with nkv heads; bf16, fp16 or
    fp32, all alike. Either may be None with a head count of 0; q_out may be q itself, k_out k. ``q_weight``,
    ``k_weight``: fp32 [head_dim], shared by the heads (None: ones). ``positions``: int32 [rows] into the fp32
    tables ``cos``, ``sin`` [positions, rot/2] (both None: no rotation); the first ``rot`` values of a head are
    turned, in pairs (i, i + rot/2), or (2i, 2i + 1) if ``interleaved``. head_dim is 64 or 128."""
    torch = _torch or _setup()
    x = _heads_given(q, k, nq, nkv)
    if _cards > 1:
        _one_card(q=q, k=k, positions=positions, cos=cos, sin=sin, q_out=q_out, k_out=k_out, q_weight=q_weight, k_weight=k_weight)
    code, rows, dt, wq, wk = _act_code(x, "q" if nq else "k", 2), x.shape[0], x.dtype, nq * head_dim, nkv * head_dim
    if (nq and q_out is None) or (nkv and k_out is None):
        raise GdnError(GDN_ERR_ARG, "q_out or k_out is missing")
    qp, qs = _act(q, "q", dt, rows, wq) if nq else _NONE
    kp, ks = _act(k, "k", dt, rows, wk) if nkv else _NONE
    qo, qos = _act(q_out, "q_out", dt, rows, wq) if nq else _NONE
    ko, kos = _act(k_out, "k_out", dt, rows, wk) if nkv else _NONE
    rc = _lib.gdn_head_norm_rope(qp, kp, _vector(positions, "positions", torch.int32, rows), _rope(cos, sin, interleaved),
                                 _vector(q_weight, "q_weight", torch.float32, head_dim),
                                 _vector(k_weight, "k_weight", torch.float32, head_dim), eps, qo, ko, rows, nq, nkv,
                                 head_dim, code, _STRIDES(qs, ks, qos, kos, 0, 0), _stream_of(stream, x))
    if rc != GDN_OK:
        _raise(rc)


def head_norm_rope_backward_workspace_bytes(rows, nq, nkv, head_dim=128) -> int:
    return int(load().gdn_head_norm_rope_backward_workspace_bytes(rows, nq, nkv, head_dim))


def head_norm_rope_backward(q, k, positions, cos, sin, q_grad, k_grad, dq, dk, dq_weight=None, dk_weight=None, *,
                            nq: int, nkv: int, head_dim: int = 128, q_weight=None, k_weight=None, eps: float = 1e-6,
                            interleaved: bool = False, workspace=None, stream=None) -> None:
    """The backward of ``head_norm_rope`` (``gdn_head_norm_rope_backward``). q, k and the rest as given to the
    forward; ``q_grad``, ``k_grad``: dL/dq_out, dL/dk_out; outputs ``dq``, ``dk`` of the same type (may be
    q_grad, k_grad themselves) and, where given, ``dq_weight``, ``dk_weight``: fp32 [head_dim], overwritten with
    the sums over all rows and heads."""
    torch = _torch or _setup()
    x = _heads_given(q, k, nq, nkv)
    if _cards > 1:
        _one_card(q=q, k=k, positions=positions, cos=cos, sin=sin, q_grad=q_grad, k_grad=k_grad, dq=dq, dk=dk, dq_weight=dq_weight,
                  dk_weight=dk_weight, q_weight=q_weight, k_weight=k_weight, workspace=workspace)
    code, rows, dt, wq, wk = _act_code(x, "q" if nq else "k", 2), x.shape[0], x.dtype, nq * head_dim, nkv * head_dim
    if (nq and (dq is None or q_grad is None)) or (nkv and (dk is None or k_grad is None)):
        raise GdnError(GDN_ERR_ARG, "a gradient tensor is missing")
    qp, qs = _act(q, "q", dt, rows, wq) if nq else _NONE
    kp, ks = _act(k, "k", dt, rows, wk) if nkv else _NONE
    gq, gqs = _act(q_grad, "q_grad", dt, rows, wq) if nq else _NONE
    gk, gks = _act(k_grad, "k_grad", dt, rows, wk) if nkv else _NONE
    dqp, dqs = _act(dq, "dq", dt, rows, wq) if nq else _NONE
    dkp, dks = _act(dk, "dk", dt, rows, wk) if nkv else _NONE
    ws, size = _scratch(workspace)
    f32 = torch.float32
    rc = _lib.gdn_head_norm_rope_backward(qp, kp, _vector(positions, "positions", torch.int32, rows), _rope(cos, sin, interleaved),
                                          _vector(q_weight, "q_weight", f32, head_dim), _vector(k_weight, "k_weight", f32, head_dim),
                                          eps, gq, gk, dqp, dkp, _vector(dq_weight, "dq_weight", f32, head_dim),
                                          _vector(dk_weight, "dk_weight", f32, head_dim), rows, nq, nkv, head_dim, code,
                                          _STRIDES(qs, ks, dqs, dks, gqs, gks), ws, size, _stream_of(stream, x))
    if rc != GDN_OK:
        _raise(rc)


def _paged(x, k_cache, v_cache, block_table, ctx_lens, cu_rows, nkv, d, rows):
    """The cache and the batch of `rows` rows like x as the ABI's struct."""
    dt, shape, ks, vs = x.dtype, k_cache.shape, k_cache.stride(), v_cache.stride()
    if k_cache.dtype is not dt or v_cache.dtype is not dt or not k_cache.is_cuda or not v_cache.is_cuda:
        raise GdnError(GDN_ERR_ARG, f"k_cache and v_cache must be {dt} CUDA tensors")
    if len(shape) != 4 or shape[2] != nkv or shape[3] != d or v_cache.shape != shape or ks[3] != 1 or vs[3] != 1:
        raise GdnError(GDN_ERR_ARG, f"k_cache and v_cache must be [pages, page_size, {nkv}, {d}], the last dimension contiguous")
    i32, table = _torch.int32, block_table.shape
    if block_table.dtype is not i32 or not block_table.is_cuda or len(table) != 2:
        raise GdnError(GDN_ERR_ARG, "block_table must be an int32 CUDA tensor [B, max_pages]")
    B, most = table
    stride = most
    if not block_table.is_contiguous():
        ts = block_table.stride()
        if ts[1] != 1 and most > 1:
            raise GdnError(GDN_ERR_ARG, "block_table must be contiguous in a row")
        stride = max(ts[0], most) if B < 2 else ts[0]
    return _PAGED(k_cache.data_ptr(), v_cache.data_ptr(), ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], shape[0], shape[1],
                  block_table.data_ptr(), stride, most, B, rows, _vector(ctx_lens, "ctx_lens", i32, B) or 0,
                  _vector(cu_rows, "cu_rows", i32, B + 1) or 0)


def paged_append(k, v, k_cache, v_cache, block_table, ctx_lens, *, nkv: int, head_dim: int = 128, cu_rows=None,
                 positions=None, cos=None, sin=None, norm: bool = False, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, stream=None) -> None:
    """Write new keys and values into a paged cache (``gdn_paged_append``), the keys normed (``norm``) and rotated
    on the way.

    k, v: bf16 or fp16 [rows, nkv*head_dim]; k_cache, v_cache: [pages, page_size, nkv, head_dim] of the same type,
    any strides with a contiguous last dimension; block_table: int32 [B, max_pages]; ctx_lens: int32 [B], each
    sequence's tokens before this call; cu_rows: int32 [B + 1], the rows of each sequence (None: row b belongs to
    sequence b). Row i of sequence b becomes its token ctx_lens[b] + i. ``positions``: int32 [rows] for the
    rotation (None: the token's index); ``cos``, ``sin``, ``interleaved``, ``k_weight``: as ``head_norm_rope``."""
    torch = _torch or _setup()
    if _cards > 1:
        _one_card(k=k, v=v, k_cache=k_cache, v_cache=v_cache, block_table=block_table, ctx_lens=ctx_lens, cu_rows=cu_rows,
                  positions=positions, cos=cos, sin=sin, k_weight=k_weight)
    code, rows, w = _act_code(k, "k", 1), k.shape[0], nkv * head_dim
    kp, ks = _act(k, "k", k.dtype, rows, w)
    vp, vs = _act(v, "v", k.dtype, rows, w)
    rc = _lib.gdn_paged_append(kp, vp, _paged(k, k_cache, v_cache, block_table, ctx_lens, cu_rows, nkv, head_dim, rows),
                               _vector(positions, "positions", torch.int32, rows), _rope(cos, sin, interleaved),
                               1 if norm else 0, _vector(k_weight, "k_weight", torch.float32, head_dim), eps, nkv, head_dim,
                               code, ks, vs, _stream_of(stream, k))
    if rc != GDN_OK:
        _raise(rc)


def tree_attention_workspace_bytes(nq, nkv, head_dim=128) -> int:
    return int(load().gdn_tree_attention_workspace_bytes(nq, nkv, head_dim))


def tree_attention(q, k_cache, v_cache, block_table, ctx_lens, out, *, nq: int, nkv: int, head_dim: int = 128,
                   cu_rows=None, mask=None, max_rows: int | None = None, scale: float | None = None, workspace=None,
                   stream=None) -> None:
    """Attention of decode tokens or drafted trees over a paged cache (``gdn_tree_attention``); the new tokens' keys
    and values are in the cache already (``paged_append``), whose arguments these share.

    q, out: [rows, nq*head_dim] of the cache's type, nq a multiple of nkv. Every row sees the ctx_lens[b] tokens of
    its sequence's context; of its sequence's new rows it sees those whose bit is set in ``mask`` (int64 [rows,
    words], bit j % 64 of word j // 64 for new row j), or without a mask those up to itself. A row that sees
    nothing gives zeros. ``max_rows``: the most rows of a sequence, by which the kernel is chosen; ``scale``:
    1/sqrt(head_dim) by default; ``workspace``: uint8 CUDA tensor of ``tree_attention_workspace_bytes(...)``."""
    torch = _torch or _setup()
    if _cards > 1:
        _one_card(q=q, k_cache=k_cache, v_cache=v_cache, block_table=block_table, ctx_lens=ctx_lens, out=out, cu_rows=cu_rows,
                  mask=mask, workspace=workspace)
    code, rows, w = _act_code(q, "q", 1), q.shape[0], nq * head_dim
    qp, qs = _act(q, "q", q.dtype, rows, w)
    op, os_ = _act(out, "out", q.dtype, rows, w)
    cache = _paged(q, k_cache, v_cache, block_table, ctx_lens, cu_rows, nkv, head_dim, rows)
    words, mp = 0, None
    if mask is not None:
        shape = mask.shape
        if mask.dtype != torch.int64 or not mask.is_cuda or len(shape) != 2 or shape[0] != rows or not mask.is_contiguous():
            raise GdnError(GDN_ERR_ARG, f"mask must be a contiguous int64 CUDA tensor [{rows}, words]")
        words, mp = shape[1], mask.data_ptr()
        if words == 0 and rows:  # no address either, which the library takes for no mask
            raise GdnError(GDN_ERR_ARG, "mask must have at least one word a row")
    ws, size = _scratch(workspace)
    rc = _lib.gdn_tree_attention(qp, cache, mp, words, max(head_dim, 1) ** -0.5 if scale is None else scale, op, nq, nkv, head_dim,
                                 code, qs, os_, max_rows or 0, ws, size, _stream_of(stream, q))
    if rc != GDN_OK:
        _raise(rc)


def check(stream=None) -> None:
    """Synchronise the stream and raise if a kernel reported a device-side error."""
    import torch

    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    rc = load().gdn_prefill_check(stream)
    if rc != GDN_OK:
        _raise(rc)


def last_launch_count() -> int:
    return int(load().gdn_last_launch_count())


def set_timing_events(before_wy=None, before_spine=None, after_spine=None) -> None:
    """Have later calls on this thread record these torch.cuda.Events (or None) before
    the WY-solve kernel, between the kernels and after the spine kernel. torch creates
    an event's CUDA handle on its first record, so record each once beforehand."""
    def handle(e):
        return None if e is None else e.cuda_event
    load().gdn_set_timing_events(handle(before_wy), handle(before_spine), handle(after_spine))


def set_test_hooks(wait_limit_ns: int = 0, consumer_delay_ns: int = 0, skip_hand_off_chunk: int = -1) -> None:
    """Test hooks (``gdn_set_test_hooks``) for later prefill calls on this thread: a
    short wait limit, a consumer delay before the hand-off wait of odd chunks, and a
    skipped hand-off arrival. All defaults switch them off."""
    rc = load().gdn_set_test_hooks(int(wait_limit_ns), int(consumer_delay_ns), int(skip_hand_off_chunk))
    if rc != GDN_OK:
        _raise(rc)
