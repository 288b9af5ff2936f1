"""Thin ctypes binding of libkda_b200.so (declared in include/kda.h).

Argument marshalling only: shapes and dtypes are read off torch tensors, output
and workspace buffers are allocated with torch on the tensors' device, and the
C entry points do all of the work on the current (or given) CUDA stream.  There
is no CPU path: if the library is missing, every call raises :class:`KDAError`.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import Dict, Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libkda_b200.so"

KDA_OK = 0
_STATUS = {
    0: "KDA_OK", 1: "KDA_ERR_INVALID_ARG", 2: "KDA_ERR_UNSUPPORTED", 3: "KDA_ERR_CUDA",
    4: "KDA_ERR_TIMEOUT", 5: "KDA_ERR_WORKSPACE", 6: "KDA_ERR_BAD_SEQLENS", 7: "KDA_ERR_RANGE",
}
KDA_F32, KDA_BF16 = 0, 1
KDA_GATE_CHANNEL, KDA_GATE_HEAD, KDA_GATE_NONE = 0, 1, 2
KDA_NORM_RMS, KDA_NORM_L2 = 0, 1

_lock = threading.Lock()
_lib = None


class KDAError(RuntimeError):
    """A libkda_b200 call returned a status other than KDA_OK."""

    def __init__(self, status: int, message: str):
        self.status = status
        super().__init__(f"{_STATUS.get(status, status)}: {message}")


def library_path() -> str:
    """Path of the in-tree CUDA library (built by ``__graft_entry__.build()``)."""
    return os.environ.get("KDA_B200_LIB", os.path.join(_HERE, _LIB_NAME))


def _declare(lib):
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    fp = ctypes.POINTER(f)
    lib.kda_chunk_fwd_workspace_size.restype = sz
    lib.kda_chunk_fwd_workspace_size.argtypes = [i, i, i, i, i, i, i, i]
    lib.kda_chunk_fwd.restype = i
    lib.kda_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i,
                                  vp, vp, vp, sz, vp]
    lib.kda_recurrent_step.restype = i
    lib.kda_recurrent_step.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, vp]
    lib.kda_chunk_fwd_gated.restype = i
    lib.kda_chunk_fwd_gated.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i,
                                        vp, vp, vp, sz, vp]
    lib.kda_recurrent_step_gated.restype = i
    lib.kda_recurrent_step_gated.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, vp]
    lib.kda_chunk_bwd_workspace_size.restype = sz
    lib.kda_chunk_bwd_workspace_size.argtypes = [i, i, i, i, i, i, i, i]
    lib.kda_chunk_bwd.restype = i
    lib.kda_chunk_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i,
                                  vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.kda_chunk_bwd_gated.restype = i
    lib.kda_chunk_bwd_gated.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i,
                                        vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.kda_chunk_fwd_plan.restype = i
    lib.kda_chunk_fwd_plan.argtypes = [i, i, i, i, i, i, i, i, sz]
    lib.kda_chunk_fwd_fused_workspace_size.restype = sz
    lib.kda_chunk_fwd_fused_workspace_size.argtypes = [i, i, i, i, i, i, i, i]
    lib.kda_chunk_fwd_save.restype = i
    lib.kda_chunk_fwd_save.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i,
                                       vp, vp, vp, sz, vp]
    lib.kda_chunk_bwd_saved.restype = i
    lib.kda_chunk_bwd_saved.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i,
                                        vp, vp, vp, vp, vp, vp, vp, sz, vp]
    for name in ("kda_linear_chunk_fwd_workspace_size", "kda_linear_chunk_bwd_workspace_size"):
        getattr(lib, name).restype = sz
        getattr(lib, name).argtypes = [i, i, i, i, i, i, i, i]
    lib.kda_linear_chunk_fwd.restype = i
    lib.kda_linear_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp, vp, vp, sz, vp]
    lib.kda_linear_chunk_bwd.restype = i
    lib.kda_linear_chunk_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i,
                                         vp, vp, vp, vp, vp, sz, vp]
    lib.kda_linear_recurrent_step.restype = i
    lib.kda_linear_recurrent_step.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, vp, vp]
    ll = ctypes.c_int64
    lib.kda_qk_norm_rope.restype = i
    lib.kda_qk_norm_rope.argtypes = [vp] * 6 + [i] * 6 + [ll] * 6 + [i, i, f, i, vp, vp, vp]
    lib.kda_qk_norm_rope_bwd_workspace_size.restype = sz
    lib.kda_qk_norm_rope_bwd_workspace_size.argtypes = [i]
    lib.kda_qk_norm_rope_bwd.restype = i
    lib.kda_qk_norm_rope_bwd.argtypes = [vp] * 8 + [i] * 6 + [ll] * 6 + [i, i, f, i, vp, vp, vp, vp, vp, sz, vp]
    lib.kda_workspace_status.restype = i
    lib.kda_workspace_status.argtypes = [vp, sz, vp]
    lib.kda_set_stage_events.restype = i
    lib.kda_set_stage_events.argtypes = [ctypes.POINTER(vp), i]
    lib.kda_debug_drop_copy.restype = i
    lib.kda_debug_drop_copy.argtypes = [ctypes.c_longlong]
    lib.kda_linear_debug_drop_copy.restype = i
    lib.kda_linear_debug_drop_copy.argtypes = [ctypes.c_longlong]
    lib.kda_last_error.restype = ctypes.c_char_p
    lib.kda_last_error.argtypes = []
    lib.kda_version.restype = ctypes.c_char_p
    lib.kda_version.argtypes = []
    del fp
    return lib


def lib():
    """Load (once) and return the ctypes handle of libkda_b200.so."""
    global _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise KDAError(3, f"CUDA library not found at {path}; build it with "
                                  "`python -c 'import __graft_entry__ as g; g.build()'`")
            _lib = _declare(ctypes.CDLL(path))
    return _lib


def _check(status: int):
    if status != KDA_OK:
        raise KDAError(status, lib().kda_last_error().decode(errors="replace"))


def _validate_default() -> bool:
    """``KDA_VALIDATE=1`` in the environment turns on ``check`` by default."""
    return os.environ.get("KDA_VALIDATE", "0") not in ("", "0", "false", "False")


def _check_device_status(workspace: torch.Tensor, stream) -> None:
    """Synchronise on the call's stream and raise if a kernel left an error
    (bad cu_seqlens, a bounded wait that gave up, an fp16-range overflow)."""
    _check(lib().kda_workspace_status(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                      _stream_ptr(stream, workspace.device)))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return KDA_F32
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    raise TypeError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream: Optional[torch.cuda.Stream], device) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _used_on(stream: Optional[torch.cuda.Stream], device, *tensors) -> None:
    """Buffers the binding allocates come from the caching allocator on the
    current stream.  When the call runs on another stream, mark them as used
    there, so that their memory is not handed out again (after the caller, or
    this function's return, drops them) before that stream's work is done."""
    if stream is None or stream.cuda_stream == torch.cuda.current_stream(device).cuda_stream:
        return
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _need(t: torch.Tensor, name: str, dtype=None, device=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _dims(t: torch.Tensor, name: str, n: int):
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got shape {tuple(t.shape)}")


def _shape(t: Optional[torch.Tensor], name: str, shape):
    """The kernels take every size from q (and v, cu_seqlens): a tensor of any
    other shape would be read or written out of bounds, so it is refused here."""
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _num_seqs(B: int, cu_seqlens) -> int:
    if cu_seqlens is None:
        return B
    _dims(cu_seqlens, "cu_seqlens", 1)
    if B != 1:
        raise ValueError(f"cu_seqlens requires B == 1 (sequences packed along T), got B={B}")
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must hold N + 1 >= 1 offsets")
    return cu_seqlens.numel() - 1


def chunk_fwd_workspace_size(B: int, T: int, H: int, dk: int, dv: int,
                             num_seqs: int, varlen: bool, dtype: torch.dtype) -> int:
    """Workspace bytes ``chunk_fwd`` needs (``kda_chunk_fwd_workspace_size``)."""
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return int(lib().kda_chunk_fwd_workspace_size(B, T, H, dk, dv, num_seqs,
                                                  int(bool(varlen)), code))


def chunk_fwd_plan(B: int, T: int, H: int, dk: int, dv: int, num_seqs: int, varlen: bool,
                   dtype: torch.dtype, workspace_bytes: Optional[int] = None) -> int:
    """1 if ``chunk_fwd`` with a workspace of ``workspace_bytes`` (default: the
    full ``chunk_fwd_workspace_size``) runs the fused single pass, 0 for the
    two-kernel form, -1 if neither fits (``kda_chunk_fwd_plan``)."""
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    if workspace_bytes is None:
        workspace_bytes = chunk_fwd_workspace_size(B, T, H, dk, dv, num_seqs, varlen, dtype)
    return int(lib().kda_chunk_fwd_plan(B, T, H, dk, dv, num_seqs, int(bool(varlen)), code,
                                        int(workspace_bytes)))


def chunk_fwd_fused_workspace_size(B: int, T: int, H: int, dk: int, dv: int,
                                   num_seqs: int, varlen: bool, dtype: torch.dtype) -> int:
    """Workspace bytes of the fused single pass (``kda_chunk_fwd_fused_workspace_size``;
    0 for fp32 inputs)."""
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return int(lib().kda_chunk_fwd_fused_workspace_size(B, T, H, dk, dv, num_seqs,
                                                        int(bool(varlen)), code))


def _gate_of(log_alpha, channel_ndim: int, shape_channel, shape_head, device=None) -> int:
    """Gate kind from log_alpha's shape: None -> no gate (DeltaNet), one value
    per head -> Gated DeltaNet, one value per key channel -> KDA."""
    if log_alpha is None:
        return KDA_GATE_NONE
    if tuple(log_alpha.shape) == tuple(shape_channel):
        gate = KDA_GATE_CHANNEL
    elif tuple(log_alpha.shape) == tuple(shape_head):
        gate = KDA_GATE_HEAD
    else:
        raise ValueError(f"log_alpha must be {tuple(shape_channel)} (per channel), {tuple(shape_head)} "
                         f"(per head) or None, got {tuple(log_alpha.shape)}")
    _need(log_alpha, "log_alpha", torch.float32, device)
    return gate


def chunk_fwd(q, k, v, log_alpha, beta, initial_state=None, cu_seqlens=None,
              output_final_state: bool = True, o=None, final_state=None,
              workspace=None, stream=None, check: Optional[bool] = None,
              _save: bool = False) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunkwise forward (``kda_chunk_fwd_gated``).

    q, k [B, T, H, dk]; v [B, T, H, dv]; beta [B, T, H];
    log_alpha [B, T, H, dk] (KDA), [B, T, H] (Gated DeltaNet) or None (DeltaNet);
    initial_state [N, H, dk, dv] fp32 or None; cu_seqlens int32 [N+1] or None.
    Returns (o [B, T, H, dv], final_state [N, H, dk, dv] or None).

    Errors found by the kernels while they run (cu_seqlens rejected on the
    device, a bounded wait that gave up, a bf16-path value beyond the fp16
    range) are written to the workspace's status word and are NOT raised by
    default, since reading them needs a synchronisation.  ``check=True`` (or
    ``KDA_VALIDATE=1`` in the environment) synchronises after the call and
    raises :class:`KDAError` for them; otherwise pass a ``workspace`` and read
    it later with :func:`workspace_status`.
    """
    _dims(q, "q", 4)
    _dims(v, "v", 4)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    N = _num_seqs(B, cu_seqlens)
    for t, n, shape in ((k, "k", (B, T, H, dk)), (v, "v", (B, T, H, dv)), (beta, "beta", (B, T, H)),
                        (initial_state, "initial_state", (N, H, dk, dv)), (o, "o", (B, T, H, dv)),
                        (final_state, "final_state", (N, H, dk, dv))):
        _shape(t, n, shape)
    dev = q.device
    gate = _gate_of(log_alpha, 4, (B, T, H, dk), (B, T, H), dev)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, dev)
    _need(beta, "beta", torch.float32, dev)
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    for t, n, dt in ((initial_state, "initial_state", torch.float32), (o, "o", q.dtype),
                     (final_state, "final_state", torch.float32)):
        if t is not None:
            _need(t, n, dt, dev)
    made = []
    if o is None:
        o = torch.empty(B, T, H, dv, dtype=q.dtype, device=q.device)
        made.append(o)
    if final_state is None and output_final_state:
        final_state = torch.empty(N, H, dk, dv, dtype=torch.float32, device=q.device)
        made.append(final_state)
    size_fn = chunk_bwd_workspace_size if _save else chunk_fwd_workspace_size
    ws_bytes = size_fn(B, T, H, dk, dv, N, cu_seqlens is not None, q.dtype)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
        made.append(workspace)
    _used_on(stream, q.device, *made)
    call = lib().kda_chunk_fwd_save if _save else lib().kda_chunk_fwd_gated
    _check(call(
        _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(initial_state),
        _ptr(cu_seqlens), B, T, H, dk, dv, N, _dtype_code(q), gate, _ptr(o), _ptr(final_state),
        _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream, q.device)))
    if check if check is not None else _validate_default():
        _check_device_status(workspace, stream)
    if _save:
        return o, final_state, workspace
    return o, final_state


def chunk_fwd_train(q, k, v, log_alpha, beta, initial_state=None, cu_seqlens=None,
                    output_final_state: bool = True, o=None, final_state=None, stream=None,
                    check: Optional[bool] = None):
    """``chunk_fwd`` for training (``kda_chunk_fwd_save``): returns (o, final_state,
    saved), where ``saved`` is a backward-sized workspace that also holds what
    ``chunk_bwd`` would recompute.  Pass it as ``chunk_bwd(..., saved=saved)`` with
    the same inputs, unchanged, to skip the recomputation."""
    return chunk_fwd(q, k, v, log_alpha, beta, initial_state, cu_seqlens, output_final_state, o,
                     final_state, None, stream, check, _save=True)


def chunk_bwd_workspace_size(B: int, T: int, H: int, dk: int, dv: int,
                             num_seqs: int, varlen: bool, dtype: torch.dtype) -> int:
    """Workspace bytes ``chunk_bwd`` needs (``kda_chunk_bwd_workspace_size``)."""
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return int(lib().kda_chunk_bwd_workspace_size(B, T, H, dk, dv, num_seqs,
                                                  int(bool(varlen)), code))


def chunk_bwd(q, k, v, log_alpha, beta, d_o, initial_state=None, d_final_state=None,
              cu_seqlens=None, output_d_initial_state: bool = True, workspace=None,
              stream=None, saved=None, check: Optional[bool] = None) -> Dict[str, Optional[torch.Tensor]]:
    """Gradients of the chunkwise forward (``kda_chunk_bwd_gated``).

    Inputs as ``chunk_fwd``: log_alpha [B, T, H, dk] (KDA), [B, T, H] (Gated
    DeltaNet) or None (DeltaNet); d_o like o; d_final_state [N, H, dk, dv] fp32
    or None.  Returns a dict with dq, dk, dv (input dtype), dlog_alpha (shaped
    like log_alpha, None without a gate), dbeta (fp32) and dS0 [N, H, dk, dv]
    (fp32, or None when ``output_d_initial_state`` is false).  With ``saved``
    (the third result of ``chunk_fwd_train`` on the same inputs) the forward is
    not recomputed (``kda_chunk_bwd_saved``); ``workspace`` must then be None.
    ``check`` as in :func:`chunk_fwd`.
    """
    _dims(q, "q", 4)
    _dims(v, "v", 4)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    N = _num_seqs(B, cu_seqlens)
    for t, n, shape in ((k, "k", (B, T, H, dk)), (v, "v", (B, T, H, dv)), (beta, "beta", (B, T, H)),
                        (d_o, "d_o", (B, T, H, dv)), (initial_state, "initial_state", (N, H, dk, dv)),
                        (d_final_state, "d_final_state", (N, H, dk, dv))):
        _shape(t, n, shape)
    dev = q.device
    gate = _gate_of(log_alpha, 4, (B, T, H, dk), (B, T, H), dev)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (d_o, "d_o")):
        _need(t, n, q.dtype, dev)
    _need(beta, "beta", torch.float32, dev)
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    for t, n in ((initial_state, "initial_state"), (d_final_state, "d_final_state")):
        if t is not None:
            _need(t, n, torch.float32, dev)
    g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
         "dlog_alpha": None if log_alpha is None else torch.empty_like(log_alpha),
         "dbeta": torch.empty_like(beta),
         "dS0": (torch.empty(N, H, dk, dv, dtype=torch.float32, device=q.device)
                 if output_d_initial_state else None)}
    ws_bytes = chunk_bwd_workspace_size(B, T, H, dk, dv, N, cu_seqlens is not None, q.dtype)
    call = lib().kda_chunk_bwd_gated
    if saved is not None:
        if workspace is not None:
            raise ValueError("pass either saved or workspace, not both")
        _need(saved, "saved", torch.uint8, dev)
        if saved.numel() < ws_bytes:
            raise ValueError(f"saved holds {saved.numel()} bytes; these sizes need {ws_bytes} "
                             "(it must come from chunk_fwd_train on the same inputs)")
        workspace, call = saved, lib().kda_chunk_bwd_saved
    made = list(g.values())
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
        made.append(workspace)
    _used_on(stream, q.device, *made)
    _check(call(
        _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(initial_state),
        _ptr(cu_seqlens), _ptr(d_o), _ptr(d_final_state), B, T, H, dk, dv, N, _dtype_code(q), gate,
        _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dlog_alpha"]), _ptr(g["dbeta"]),
        _ptr(g["dS0"]), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream, q.device)))
    if check if check is not None else _validate_default():
        _check_device_status(workspace, stream)
    return g


def debug_drop_copy(wait_cycles: int) -> None:
    """Arm the one-shot failure-path test hook (``kda_debug_drop_copy``)."""
    _check(lib().kda_debug_drop_copy(int(wait_cycles)))


def workspace_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise and return the device status code left in ``workspace``."""
    return int(lib().kda_workspace_status(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                          _stream_ptr(stream, workspace.device)))


def set_stage_events(events) -> None:
    """Record ``events`` (4 ``torch.cuda.Event``s) at the stage boundaries of
    the following ``chunk_fwd`` calls on this thread; ``None`` stops it."""
    if events is None:
        _check(lib().kda_set_stage_events(None, 0))
        return
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check(lib().kda_set_stage_events(arr, len(events)))


def recurrent_step(q, k, v, log_alpha, beta, state, o=None, stream=None) -> torch.Tensor:
    """One decoding step (``kda_recurrent_step_gated``); ``state`` is updated in place.

    q, k [B, H, dk]; v [B, H, dv]; beta [B, H]; state [B, H, dk, dv] fp32;
    log_alpha [B, H, dk] (KDA), [B, H] (Gated DeltaNet) or None (DeltaNet).
    Returns o [B, H, dv] in q's dtype.
    """
    _dims(q, "q", 3)
    _dims(v, "v", 3)
    B, H, dk = q.shape
    dv = v.shape[-1]
    for t, n, shape in ((k, "k", (B, H, dk)), (v, "v", (B, H, dv)), (beta, "beta", (B, H)),
                        (state, "state", (B, H, dk, dv)), (o, "o", (B, H, dv))):
        _shape(t, n, shape)
    dev = q.device
    gate = _gate_of(log_alpha, 3, (B, H, dk), (B, H), dev)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, dev)
    _need(beta, "beta", torch.float32, dev)
    _need(state, "state", torch.float32, dev)
    if o is not None:
        _need(o, "o", q.dtype, dev)
    if o is None:
        o = torch.empty(B, H, dv, dtype=q.dtype, device=q.device)
        _used_on(stream, q.device, o)
    _check(lib().kda_recurrent_step_gated(
        _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(state),
        B, H, dk, dv, _dtype_code(q), gate, _ptr(o), _stream_ptr(stream, q.device)))
    return o


# ------------------------------------------- linear attention, decay per head --
# These calls are short enough that the host's part shows, so the checks run over
# all tensors at once and name what is wrong only where something is.
def _on(device):
    """The library launches on the current device; make that the tensors' device
    for the call where it is another."""
    return (_HERE_DEVICE if torch.cuda.current_device() == device.index else torch.cuda.device(device))


_HERE_DEVICE = contextlib.nullcontext()


def _loaded():
    """:func:`lib` without its lock, once it is loaded."""
    return _lib if _lib is not None else lib()


def _current_raw_stream():
    """The current stream's handle by device index: torch's own short way to it, which is not
    public, where this torch has it, else the public one (1 us more a call)."""
    return getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


_current_raw = _current_raw_stream()


def _raw_stream(stream, device) -> int:
    return _current_raw(device.index) if stream is None else stream.cuda_stream


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _verify(device, specs) -> None:
    """Each (tensor or None, name, shape, dtype) is contiguous, of that shape and
    type, on ``device``, a GPU; a shape or dtype of None may be any."""
    for t, _, shape, dtype in specs:
        if t is not None and not ((shape is None or t.shape == shape) and (dtype is None or t.dtype is dtype)
                                  and t.device == device and t.is_contiguous()):
            break
    else:
        if device.type == "cuda":
            return
    for t, name, shape, _ in specs:
        if shape is not None:
            _shape(t, name, shape)
    for t, name, _, dtype in specs:
        if t is not None:
            _need(t, name, dtype, device)


def _workspace_args(workspace):
    return (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)


def _run_status(status: int, workspace, stream, device, check: bool) -> None:
    if status != KDA_OK:
        _check(status)
    if check:
        _check_device_status(workspace, stream if stream is not None else torch.cuda.current_stream(device))


def linear_chunk_fwd_workspace_size(B: int, T: int, H: int, dk: int, dv: int,
                                    num_seqs: int, varlen: bool, dtype: torch.dtype) -> int:
    """Workspace bytes ``linear_chunk_fwd`` needs (``kda_linear_chunk_fwd_workspace_size``)."""
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return _loaded().kda_linear_chunk_fwd_workspace_size(B, T, H, dk, dv, num_seqs, int(varlen), code)


def linear_chunk_bwd_workspace_size(B: int, T: int, H: int, dk: int, dv: int,
                                    num_seqs: int, varlen: bool, dtype: torch.dtype) -> int:
    """Workspace bytes ``linear_chunk_bwd`` needs (``kda_linear_chunk_bwd_workspace_size``)."""
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return _loaded().kda_linear_chunk_bwd_workspace_size(B, T, H, dk, dv, num_seqs, int(varlen), code)


def linear_chunk_fwd(q, k, v, log_decay=None, initial_state=None, cu_seqlens=None,
                     output_final_state: bool = True, o=None, final_state=None, workspace=None,
                     stream=None, check: Optional[bool] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Linear attention with one fixed decay per head, chunkwise (``kda_linear_chunk_fwd``):
    S_t = e^log_decay S_{t-1} + k_t v_t^T, o_t = dk^-1/2 S_t^T q_t.

    q, k [B, T, H, dk]; v [B, T, H, dv]; log_decay [H] fp32 or None (no decay);
    initial_state [N, H, dk, dv] fp32 or None; cu_seqlens int32 [N+1] or None.
    Returns (o [B, T, H, dv], final_state [N, H, dk, dv] or None).  The decays
    are constants: they get no gradient.  ``check`` as in :func:`chunk_fwd`.
    """
    _dims(q, "q", 4)
    _dims(v, "v", 4)
    B, T, H, dk = q.shape
    dv = v.shape[3]
    N = _num_seqs(B, cu_seqlens)
    dev, dtype, f32, state = q.device, q.dtype, torch.float32, (N, H, dk, dv)
    _verify(dev, ((q, "q", None, dtype), (k, "k", (B, T, H, dk), dtype), (v, "v", (B, T, H, dv), dtype),
                  (log_decay, "log_decay", (H,), f32), (initial_state, "initial_state", state, f32),
                  (cu_seqlens, "cu_seqlens", None, torch.int32), (o, "o", (B, T, H, dv), dtype),
                  (final_state, "final_state", state, f32), (workspace, "workspace", None, None)))
    code = _dtype_code(q)
    check = _validate_default() if check is None else check
    made = []
    if o is None:
        o = torch.empty_like(v)
        made.append(o)
    if final_state is None and output_final_state:
        final_state = torch.empty(state, dtype=f32, device=dev) if initial_state is None else torch.empty_like(initial_state)
        made.append(final_state)
    if workspace is None:
        size = _loaded().kda_linear_chunk_fwd_workspace_size(B, T, H, dk, dv, N, cu_seqlens is not None, code)
        if check or size != 256:        # 256: the status alone, which nobody would read
            workspace = torch.empty(max(size, 1), dtype=torch.uint8, device=dev)
            made.append(workspace)
    if stream is not None:
        _used_on(stream, dev, *made)
    with _on(dev):
        status = _loaded().kda_linear_chunk_fwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), _addr(log_decay), _addr(initial_state), _addr(cu_seqlens),
            B, T, H, dk, dv, N, code, o.data_ptr(), _addr(final_state),
            *_workspace_args(workspace), _raw_stream(stream, dev))
        _run_status(status, workspace, stream, dev, check)
    return o, final_state


def linear_chunk_bwd(q, k, v, log_decay, d_o, initial_state=None, d_final_state=None, cu_seqlens=None,
                     output_d_initial_state: bool = True, workspace=None, stream=None,
                     check: Optional[bool] = None) -> Dict[str, Optional[torch.Tensor]]:
    """Gradients of :func:`linear_chunk_fwd` (``kda_linear_chunk_bwd``).

    Inputs as ``linear_chunk_fwd``; d_o like o; d_final_state [N, H, dk, dv] fp32
    or None.  Returns a dict with dq, dk, dv (input dtype) and dS0 [N, H, dk, dv]
    (fp32, or None when ``output_d_initial_state`` is false).
    """
    _dims(q, "q", 4)
    _dims(v, "v", 4)
    B, T, H, dk = q.shape
    dv = v.shape[3]
    N = _num_seqs(B, cu_seqlens)
    dev, dtype, f32, state = q.device, q.dtype, torch.float32, (N, H, dk, dv)
    _verify(dev, ((q, "q", None, dtype), (k, "k", (B, T, H, dk), dtype), (v, "v", (B, T, H, dv), dtype),
                  (d_o, "d_o", (B, T, H, dv), dtype), (log_decay, "log_decay", (H,), f32),
                  (initial_state, "initial_state", state, f32), (d_final_state, "d_final_state", state, f32),
                  (cu_seqlens, "cu_seqlens", None, torch.int32), (workspace, "workspace", None, None)))
    code = _dtype_code(q)
    check = _validate_default() if check is None else check
    g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
         "dS0": torch.empty(state, dtype=f32, device=dev) if output_d_initial_state else None}
    made = list(g.values())
    if workspace is None:
        size = _loaded().kda_linear_chunk_bwd_workspace_size(B, T, H, dk, dv, N, cu_seqlens is not None, code)
        if check or size != 256:        # 256: the status alone, which nobody would read
            workspace = torch.empty(max(size, 1), dtype=torch.uint8, device=dev)
            made.append(workspace)
    if stream is not None:
        _used_on(stream, dev, *made)
    with _on(dev):
        status = _loaded().kda_linear_chunk_bwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), _addr(log_decay), _addr(initial_state), _addr(cu_seqlens),
            d_o.data_ptr(), _addr(d_final_state), B, T, H, dk, dv, N, code, g["dq"].data_ptr(), g["dk"].data_ptr(),
            g["dv"].data_ptr(), _addr(g["dS0"]), *_workspace_args(workspace), _raw_stream(stream, dev))
        _run_status(status, workspace, stream, dev, check)
    return g


def linear_recurrent_step(q, k, v, log_decay, state, o=None, stream=None) -> torch.Tensor:
    """One token of :func:`linear_chunk_fwd`'s recurrence (``kda_linear_recurrent_step``);
    ``state`` is updated in place.

    q, k [B, H, dk]; v [B, H, dv]; log_decay [H] fp32 or None; state [B, H, dk, dv]
    fp32.  Returns o [B, H, dv] in q's dtype.
    """
    _dims(q, "q", 3)
    _dims(v, "v", 3)
    B, H, dk = q.shape
    dv = v.shape[2]
    dev, dtype, f32 = q.device, q.dtype, torch.float32
    _verify(dev, ((q, "q", None, dtype), (k, "k", (B, H, dk), dtype), (v, "v", (B, H, dv), dtype),
                  (log_decay, "log_decay", (H,), f32), (state, "state", (B, H, dk, dv), f32),
                  (o, "o", (B, H, dv), dtype)))
    code = _dtype_code(q)
    if o is None:
        o = torch.empty_like(v)
        if stream is not None:
            _used_on(stream, dev, o)
    with _on(dev):
        status = _loaded().kda_linear_recurrent_step(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), _addr(log_decay), state.data_ptr(), B, H, dk, dv, code,
            o.data_ptr(), _raw_stream(stream, dev))
    if status != KDA_OK:
        _check(status)
    return o


def linear_debug_drop_copy(wait_cycles: int) -> None:
    """Arm the one-shot failure-path test hook of the next bf16 :func:`linear_chunk_fwd`
    (``kda_linear_debug_drop_copy``)."""
    _check(lib().kda_linear_debug_drop_copy(int(wait_cycles)))


# ------------------------------------------------ norm and rotation of q and k --
def _rows(t: torch.Tensor, name: str, dtype, device):
    """Element strides of batch, token and head of rows that may lie apart: only
    their channels are contiguous."""
    if t.device != device or device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor on {device}, got {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    s, n = t.stride(), t.shape
    if s[-1] != 1 and n[-1] > 1:
        raise ValueError(f"the channels of {name} must be contiguous")
    # a dimension of one element is never stepped over, whatever stride torch gives it
    return (s[0] if n[0] != 1 else 0, s[1] if len(n) == 4 and n[1] != 1 else 0, s[-2] if n[-2] != 1 else 0)


def _norm_args(q, k, q_weight, k_weight, inv_freq, positions, norm, more):
    """Checks the arguments the norm and its gradients share; returns the sizes and
    strides as the C calls take them and the norm's code.  ``more`` names the tensors
    shaped like q and like k."""
    ndim = q.dim()
    if ndim not in (3, 4):
        raise ValueError(f"q must have 3 or 4 dimensions, got shape {tuple(q.shape)}")
    _dims(k, "k", ndim)
    qshape, kshape = q.shape, k.shape
    lead, Hq, Hk, d = qshape[:-2], qshape[-2], kshape[-2], qshape[-1]
    if kshape[:-2] != lead or kshape[-1] != d:
        _shape(k, "k", (*lead, Hk, d))
    B, T = lead if ndim == 4 else (lead[0], 1)
    rot = 0
    if inv_freq is not None:
        _dims(inv_freq, "inv_freq", 1)
        rot = 2 * inv_freq.shape[0]
        if ndim == 3 and positions is None:
            raise ValueError("a rotation of single tokens needs their positions")
    code = {"rms": KDA_NORM_RMS, "l2": KDA_NORM_L2}.get(norm)
    if code is None:
        raise ValueError(f"norm must be 'rms' or 'l2', got {norm!r}")
    dev, dtype, f32 = q.device, q.dtype, torch.float32
    _verify(dev, ((q_weight, "q_weight", (d,), f32), (k_weight, "k_weight", (d,), f32),
                  (inv_freq, "inv_freq", None, f32), (positions, "positions", lead, torch.int32),
                  *[(t, n, qshape if of_q else kshape, dtype) for t, n, of_q in more]))
    return (B, T, Hq, Hk, d, rot, *_rows(q, "q", dtype, dev), *_rows(k, "k", dtype, dev)), code


def qk_norm_rope(q, k, q_weight=None, k_weight=None, inv_freq=None, positions=None, norm: str = "l2",
                 eps: float = 1e-6, interleaved: bool = False, q_out=None, k_out=None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Norm of queries and keys per head and position rotation in one pass
    (``kda_qk_norm_rope``), as they go into the attention calls of this module.

    q [B, T, Hq, d], k [B, T, Hk, d] (or single tokens [B, Hq, d], [B, Hk, d]),
    which may be slices of a joint projection; ``norm`` "l2" (unit rows) or "rms";
    q_weight, k_weight [d] fp32 or None; inv_freq [rotary_dim / 2] fp32 turns the
    first rotary_dim channels by position * inv_freq (None: no rotation), in pairs
    (j, j + rotary_dim / 2) or, with ``interleaved``, (2j, 2j + 1); positions int32
    [B, T] ([B] for single tokens), None: 0 .. T-1.  Returns (q_out, k_out),
    contiguous and of the inputs' dtype.
    """
    sizes, code = _norm_args(q, k, q_weight, k_weight, inv_freq, positions, norm,
                             ((q_out, "q_out", True), (k_out, "k_out", False)))
    dev, dt = q.device, _dtype_code(q)
    made = []
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        made.append(q_out)
    if k_out is None:
        k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
        made.append(k_out)
    if stream is not None:
        _used_on(stream, dev, *made)
    with _on(dev):
        status = _loaded().kda_qk_norm_rope(
            q.data_ptr(), k.data_ptr(), _addr(q_weight), _addr(k_weight), _addr(inv_freq), _addr(positions), *sizes,
            dt, code, eps, interleaved, q_out.data_ptr(), k_out.data_ptr(), _raw_stream(stream, dev))
    if status != KDA_OK:
        _check(status)
    return q_out, k_out


def qk_norm_rope_bwd(q, k, d_q_out, d_k_out, q_weight=None, k_weight=None, inv_freq=None, positions=None,
                     norm: str = "l2", eps: float = 1e-6, interleaved: bool = False, workspace=None,
                     stream=None) -> Dict[str, Optional[torch.Tensor]]:
    """Gradients of :func:`qk_norm_rope` (``kda_qk_norm_rope_bwd``): q, k its inputs,
    d_q_out, d_k_out the cotangents of its outputs.  Returns a dict with dq, dk
    (contiguous) and dq_weight, dk_weight [d] fp32 (None without that weight)."""
    sizes, code = _norm_args(q, k, q_weight, k_weight, inv_freq, positions, norm,
                             ((d_q_out, "d_q_out", True), (d_k_out, "d_k_out", False)))
    dev, dt = q.device, _dtype_code(q)
    g = {"dq": torch.empty_like(q, memory_format=torch.contiguous_format),
         "dk": torch.empty_like(k, memory_format=torch.contiguous_format),
         "dq_weight": None if q_weight is None else torch.empty_like(q_weight),
         "dk_weight": None if k_weight is None else torch.empty_like(k_weight)}
    made = list(g.values())
    if workspace is not None:
        _need(workspace, "workspace", None, dev)
    elif q_weight is not None or k_weight is not None:
        workspace = torch.empty(max(_loaded().kda_qk_norm_rope_bwd_workspace_size(sizes[4]), 1), dtype=torch.uint8, device=dev)
        made.append(workspace)
    if stream is not None:
        _used_on(stream, dev, *made)
    with _on(dev):
        status = _loaded().kda_qk_norm_rope_bwd(
            q.data_ptr(), k.data_ptr(), d_q_out.data_ptr(), d_k_out.data_ptr(), _addr(q_weight), _addr(k_weight),
            _addr(inv_freq), _addr(positions), *sizes, dt, code, eps, interleaved, g["dq"].data_ptr(),
            g["dk"].data_ptr(), _addr(g["dq_weight"]), _addr(g["dk_weight"]), _addr(workspace),
            0 if workspace is None else workspace.nbytes, _raw_stream(stream, dev))
    if status != KDA_OK:
        _check(status)
    return g
