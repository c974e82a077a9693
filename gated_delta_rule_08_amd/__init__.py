"""Python binding of libgdr, the gated delta-rule mixer for MI355X (gfx950).

Argument marshalling only: each function checks that the torch tensors it is
given agree with one another (device, dtype, contiguity, shapes), passes their
device pointers and the current HIP stream to the C ABI declared in
``include/gdr.h``, and raises :class:`GdrError` on a non-zero status.  All
arithmetic runs in the library's HIP kernels.  If ``libgdr.so`` has not been
built, importing works but every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

__all__ = [
    "GdrError", "GATES", "library_path", "load_library", "gdr_decode_step",
    "gdr_decode_multi", "gdr_chunk_prefill", "gdr_chunk_prefill_varlen",
    "gdr_chunk_prefill_varlen_workspace_bytes", "gdr_chunk_prefill_workspace_bytes", "gdr_status_string",
    "gdr_abi_version", "EXPORTED_SYMBOLS", "gdr_decode_step_ex", "gdr_chunk_prefill_ex",
    "PRO_L2NORM_QK", "PRO_SIGMOID", "gdr_chunk_backward", "gdr_chunk_backward_workspace_bytes",
    "gdr_chunk_backward_workspace_bytes_ranged",
    "gdr_decode_multi_ex", "gdr_chunk_prefill_varlen_ex", "SCHED_FUSED", "SCHED_SPLIT",
    "gdr_chunk_prefill_noalloc", "gdr_attn_prefill", "gdr_attn_prefill_varlen", "gdr_attn_backward",
    "gdr_attn_backward_workspace_bytes", "gdr_attn_decode", "gdr_attn_decode_workspace_bytes", "gdr_attn_append",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
GATES = {"gdn": 0, "kda": 1}
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
# input prologue flags of the *_ex calls (include/gdr.h: GDR_PRO_*)
PRO_L2NORM_QK = 1
PRO_SIGMOID = 2
# schedule of the bf16 chunked prefill (include/gdr.h: GDR_SCHED_*); neither
# bit = the default (fused for GDN, split for KDA)
SCHED_FUSED = 4
SCHED_SPLIT = 8
EXPORTED_SYMBOLS = ("gdr_decode_step", "gdr_decode_step_ex", "gdr_chunk_prefill_ex",
                    "gdr_chunk_prefill_noalloc",
                    "gdr_chunk_prefill_workspace_bytes_ex",
                    "gdr_chunk_prefill_varlen_workspace_bytes_ex",
                    "gdr_decode_multi_ex", "gdr_chunk_prefill_varlen_ex",
                    "gdr_chunk_backward", "gdr_chunk_backward_workspace_bytes",
                    "gdr_chunk_backward_workspace_bytes_ranged",
                    "gdr_decode_multi", "gdr_chunk_prefill",
                    "gdr_chunk_prefill_varlen", "gdr_chunk_prefill_varlen_workspace_bytes",
                    "gdr_chunk_prefill_workspace_bytes", "gdr_status_string",
                    "gdr_abi_version",
                    "gdr_attn_prefill", "gdr_attn_prefill_varlen", "gdr_attn_backward",
                    "gdr_attn_backward_workspace_bytes", "gdr_attn_decode",
                    "gdr_attn_decode_workspace_bytes", "gdr_attn_append")
CHUNK = 64
_lib = None


class GdrError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


def library_path() -> str:
    return os.environ.get("GDR_LIBRARY", os.path.join(_PKG, "libgdr.so"))


def load_library():
    """Load libgdr.so and declare the C signatures.  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise GdrError(-100, "libgdr.so is not built (%s); run "
                       "`python -m gated_delta_rule_08_amd.build`" % path)
    lib = ctypes.CDLL(path)
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.gdr_decode_step.argtypes = [i, i, i, i, i, i, f] + [vp] * 8
    lib.gdr_decode_step.restype = i
    lib.gdr_decode_step_ex.argtypes = [i] * 7 + [f] + [vp] * 8
    lib.gdr_decode_step_ex.restype = i
    lib.gdr_chunk_prefill_ex.argtypes = [i] * 9 + [f] + [vp] * 9 + [ctypes.c_size_t, vp]
    lib.gdr_chunk_prefill_ex.restype = i
    lib.gdr_chunk_prefill_noalloc.argtypes = [i] * 9 + [f] + [vp] * 9
    lib.gdr_chunk_prefill_noalloc.restype = i
    lib.gdr_chunk_backward.argtypes = [i] * 8 + [f] + [vp] * 15 + [ctypes.c_size_t, vp]
    lib.gdr_chunk_backward.restype = i
    lib.gdr_chunk_backward_workspace_bytes.argtypes = [i] * 8
    lib.gdr_chunk_backward_workspace_bytes.restype = ctypes.c_size_t
    lib.gdr_chunk_backward_workspace_bytes_ranged.argtypes = [i] * 9
    lib.gdr_chunk_backward_workspace_bytes_ranged.restype = ctypes.c_size_t
    lib.gdr_decode_multi_ex.argtypes = [i] * 8 + [f] + [vp] * 9
    lib.gdr_decode_multi_ex.restype = i
    lib.gdr_chunk_prefill_varlen_ex.argtypes = [i] * 10 + [f] + [vp] * 9 + [i, vp, vp, ctypes.c_size_t, vp]
    lib.gdr_chunk_prefill_varlen_ex.restype = i
    lib.gdr_decode_multi.argtypes = [i] * 7 + [f] + [vp] * 9
    lib.gdr_decode_multi.restype = i
    lib.gdr_chunk_prefill.argtypes = [i] * 8 + [f] + [vp] * 9 + [ctypes.c_size_t, vp]
    lib.gdr_chunk_prefill.restype = i
    lib.gdr_chunk_prefill_workspace_bytes.argtypes = [i] * 8
    lib.gdr_chunk_prefill_workspace_bytes.restype = ctypes.c_size_t
    lib.gdr_chunk_prefill_varlen.argtypes = [i] * 9 + [f] + [vp] * 9 + [i, vp, vp, ctypes.c_size_t, vp]
    lib.gdr_chunk_prefill_varlen.restype = i
    lib.gdr_chunk_prefill_varlen_workspace_bytes.argtypes = [i] * 8
    lib.gdr_chunk_prefill_varlen_workspace_bytes.restype = ctypes.c_size_t
    lib.gdr_chunk_prefill_workspace_bytes_ex.argtypes = [i] * 9
    lib.gdr_chunk_prefill_workspace_bytes_ex.restype = ctypes.c_size_t
    lib.gdr_chunk_prefill_varlen_workspace_bytes_ex.argtypes = [i] * 9
    lib.gdr_chunk_prefill_varlen_workspace_bytes_ex.restype = ctypes.c_size_t
    lib.gdr_attn_prefill.argtypes = [i] * 9 + [f] + [vp] * 6
    lib.gdr_attn_prefill.restype = i
    lib.gdr_attn_prefill_varlen.argtypes = [i] * 10 + [f] + [vp] * 8
    lib.gdr_attn_prefill_varlen.restype = i
    lib.gdr_attn_backward.argtypes = [i] * 9 + [f] + [vp] * 10 + [ctypes.c_size_t, vp]
    lib.gdr_attn_backward.restype = i
    lib.gdr_attn_backward_workspace_bytes.argtypes = [i] * 9
    lib.gdr_attn_backward_workspace_bytes.restype = ctypes.c_size_t
    lib.gdr_attn_decode.argtypes = [i] * 10 + [f] + [vp] * 9 + [ctypes.c_size_t, vp]
    lib.gdr_attn_decode.restype = i
    lib.gdr_attn_decode_workspace_bytes.argtypes = [i] * 9
    lib.gdr_attn_decode_workspace_bytes.restype = ctypes.c_size_t
    lib.gdr_attn_append.argtypes = [i] * 8 + [vp] * 8
    lib.gdr_attn_append.restype = i
    lib.gdr_status_string.argtypes = [i]
    lib.gdr_status_string.restype = ctypes.c_char_p
    lib.gdr_abi_version.argtypes = []
    lib.gdr_abi_version.restype = i
    _lib = lib
    return lib


def gdr_status_string(status: int) -> str:
    return load_library().gdr_status_string(int(status)).decode()


def gdr_abi_version() -> int:
    return load_library().gdr_abi_version()


def _check(status: int) -> None:
    if status != 0:
        raise GdrError(status, gdr_status_string(status))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _stream_object(stream, device):
    """A stream argument as torch's object.  Handle 0 is the device's default stream (torch would make a new one)."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else torch.cuda.default_stream(device)


def _workspace(need: int, device, stream):
    """A workspace of `need` bytes for one call launched on `stream`.

    The caching allocator ties a block to the stream current at allocation
    and may hand it out again once the tensor is freed, so a block used by a
    launch on another stream is recorded on that stream: it is not reused
    before the launch's work there has completed.
    """
    if not need:
        return None
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    if stream is not None:
        s = _stream_object(stream, device)
        if s.cuda_stream != torch.cuda.current_stream(device).cuda_stream:
            ws.record_stream(s)
    return ws


def _same_device(*ts):
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("all tensors must be on the GPU")
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("all tensors must be on one device")


def gdr_decode_step(gate: str, q, k, v, alpha, beta, state, o, scale: float = 1.0,
                    stream=None) -> None:
    """One decode step; ``state`` [B,H,dk,dv] fp32 is updated in place.

    q, k [B,H,dk] and v, o [B,H,dv] share a dtype (fp32 or bf16); alpha is
    [B,H] (gate "gdn") or [B,H,dk] (gate "kda"); beta [B,H]; fp32 gates.
    """
    _decode_step(None, gate, q, k, v, alpha, beta, state, o, scale, stream)


def gdr_decode_step_ex(gate: str, q, k, v, alpha, beta, state, o, flags: int = 0,
                       scale: float = 1.0, stream=None) -> None:
    """:func:`gdr_decode_step` with an input prologue: ``flags`` ORs
    PRO_L2NORM_QK (q, k are raw and get L2-normalised) and PRO_SIGMOID
    (alpha, beta are logits)."""
    _decode_step(int(flags), gate, q, k, v, alpha, beta, state, o, scale, stream)


def _decode_step(flags, gate, q, k, v, alpha, beta, state, o, scale, stream):
    B, H, dk = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or v.shape != (B, H, dv) or o.shape != (B, H, dv):
        raise ValueError("q, k, v, o shapes disagree")
    if alpha.shape != ((B, H, dk) if gate == "kda" else (B, H)) or beta.shape != (B, H):
        raise ValueError("alpha / beta shapes disagree with the gate mode")
    if state.shape != (B, H, dk, dv) or state.dtype != torch.float32:
        raise ValueError("state must be fp32 [B,H,dk,dv]")
    if not (q.dtype == k.dtype == v.dtype == o.dtype) or q.dtype not in _DTYPES:
        raise ValueError("q, k, v, o must share dtype fp32 or bf16")
    if alpha.dtype != torch.float32 or beta.dtype != torch.float32:
        raise ValueError("alpha and beta must be fp32")
    _same_device(q, k, v, alpha, beta, state, o)
    lib = load_library()
    ptrs = (_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state), _ptr(o), _stream(stream))
    if flags is None:
        _check(lib.gdr_decode_step(GATES[gate], _DTYPES[q.dtype], B, H, dk, dv, float(scale), *ptrs))
    else:
        _check(lib.gdr_decode_step_ex(GATES[gate], _DTYPES[q.dtype], flags, B, H, dk, dv, float(scale),
                                      *ptrs))


def gdr_decode_multi_ex(gate: str, q, k, v, alpha, beta, state, o, states=None, flags: int = 0,
                        scale: float = 1.0, stream=None) -> None:
    """:func:`gdr_decode_multi` with an input prologue (``flags`` as in
    :func:`gdr_decode_step_ex`), applied to every token."""
    _decode_multi(int(flags), gate, q, k, v, alpha, beta, state, o, states, scale, stream)


def gdr_decode_multi(gate: str, q, k, v, alpha, beta, state, o, states=None,
                     scale: float = 1.0, stream=None) -> None:
    """T decode steps per head (the verify step of speculative decoding).

    q, k [B,T,H,dk] and v, o [B,T,H,dv] share a dtype; alpha [B,T,H] (gdn) or
    [B,T,H,dk] (kda) and beta [B,T,H] are fp32; ``state`` [B,H,dk,dv] fp32 is
    read as S_0 and overwritten with S_T.  ``states`` (optional, fp32
    [B,T,H,dk,dv]) receives the state after every token.  T <= 64.
    """
    _decode_multi(None, gate, q, k, v, alpha, beta, state, o, states, scale, stream)


def _decode_multi(flags, gate, q, k, v, alpha, beta, state, o, states, scale, stream):
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or v.shape != (B, T, H, dv) or o.shape != (B, T, H, dv):
        raise ValueError("q, k, v, o shapes disagree")
    if alpha.shape != ((B, T, H, dk) if gate == "kda" else (B, T, H)) or beta.shape != (B, T, H):
        raise ValueError("alpha / beta shapes disagree with the gate mode")
    if state.shape != (B, H, dk, dv) or state.dtype != torch.float32:
        raise ValueError("state must be fp32 [B,H,dk,dv]")
    if states is not None and (states.shape != (B, T, H, dk, dv) or states.dtype != torch.float32):
        raise ValueError("states must be fp32 [B,T,H,dk,dv]")
    if not (q.dtype == k.dtype == v.dtype == o.dtype) or q.dtype not in _DTYPES:
        raise ValueError("q, k, v, o must share dtype fp32 or bf16")
    if alpha.dtype != torch.float32 or beta.dtype != torch.float32:
        raise ValueError("alpha and beta must be fp32")
    _same_device(q, k, v, alpha, beta, state, o, states)
    lib = load_library()
    rest = (B, T, H, dk, dv, float(scale), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
            _ptr(state), _ptr(o), _ptr(states), _stream(stream))
    if flags is None:
        _check(lib.gdr_decode_multi(GATES[gate], _DTYPES[q.dtype], *rest))
    else:
        _check(lib.gdr_decode_multi_ex(GATES[gate], _DTYPES[q.dtype], flags, *rest))


def gdr_chunk_prefill_workspace_bytes(gate: str, dtype, B: int, T: int, H: int, dk: int,
                                      dv: int, chunk: int = CHUNK, flags: int = 0) -> int:
    """Workspace bytes of a chunked prefill with these prologue and schedule
    ``flags`` (0: the default schedule)."""
    return int(load_library().gdr_chunk_prefill_workspace_bytes_ex(
        GATES[gate], _DTYPES[dtype], int(flags), B, T, H, dk, dv, chunk))


def gdr_chunk_prefill(gate: str, q, k, v, alpha, beta, state_in, state_out, o,
                      scale: float = 1.0, workspace=None, chunk: int = CHUNK,
                      stream=None) -> None:
    """Chunked prefill; writes o [B,T,H,dv] and state_out [B,H,dk,dv] (fp32).

    q, k [B,T,H,dk] and v, o [B,T,H,dv] share a dtype; alpha [B,T,H] (gdn) or
    [B,T,H,dk] (kda) and beta [B,T,H] are fp32; state_in may be None.
    workspace: a device tensor of at least gdr_chunk_prefill_workspace_bytes
    bytes, or None to have one allocated for this call.
    """
    _chunk_prefill(None, gate, q, k, v, alpha, beta, state_in, state_out, o, scale, workspace,
                   chunk, stream)


def gdr_chunk_prefill_ex(gate: str, q, k, v, alpha, beta, state_in, state_out, o, flags: int = 0,
                         scale: float = 1.0, workspace=None, chunk: int = CHUNK,
                         stream=None) -> None:
    """:func:`gdr_chunk_prefill` with an input prologue and a schedule choice:
    ``flags`` ORs the PRO_* bits of :func:`gdr_decode_step_ex` with at most
    one of SCHED_FUSED, SCHED_SPLIT (bf16 only)."""
    _chunk_prefill(int(flags), gate, q, k, v, alpha, beta, state_in, state_out, o, scale,
                   workspace, chunk, stream)


def gdr_chunk_prefill_noalloc(gate: str, q, k, v, alpha, beta, state_in, state_out, o, flags: int = 0,
                              scale: float = 1.0, chunk: int = CHUNK, stream=None) -> None:
    """:func:`gdr_chunk_prefill_ex` without a workspace: the split schedule
    uses the library's fixed 96 MiB device scratch (one per GPU), so the call
    allocates nothing.  Calls overlapping in time on one GPU race on it."""
    _chunk_prefill(int(flags), gate, q, k, v, alpha, beta, state_in, state_out, o, scale, None,
                   chunk, stream, noalloc=True)


def _chunk_prefill(flags, gate, q, k, v, alpha, beta, state_in, state_out, o, scale, workspace,
                   chunk, stream, noalloc=False):
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or v.shape != (B, T, H, dv) or o.shape != (B, T, H, dv):
        raise ValueError("q, k, v, o shapes disagree")
    if alpha.shape != ((B, T, H, dk) if gate == "kda" else (B, T, H)) or beta.shape != (B, T, H):
        raise ValueError("alpha / beta shapes disagree with the gate mode")
    for s in (state_in, state_out):
        if s is not None and (s.shape != (B, H, dk, dv) or s.dtype != torch.float32):
            raise ValueError("states must be fp32 [B,H,dk,dv]")
    if not (q.dtype == k.dtype == v.dtype == o.dtype) or q.dtype not in _DTYPES:
        raise ValueError("q, k, v, o must share dtype fp32 or bf16")
    if alpha.dtype != torch.float32 or beta.dtype != torch.float32:
        raise ValueError("alpha and beta must be fp32")
    _same_device(q, k, v, alpha, beta, state_in, state_out, o, workspace)
    if noalloc:
        _check(load_library().gdr_chunk_prefill_noalloc(
            GATES[gate], _DTYPES[q.dtype], flags, B, T, H, dk, dv, chunk, float(scale), _ptr(q), _ptr(k),
            _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state_in), _ptr(state_out), _ptr(o), _stream(stream)))
        return
    if workspace is None:  # allocate what this call needs (callers that time or capture pass their own)
        workspace = _workspace(gdr_chunk_prefill_workspace_bytes(gate, q.dtype, B, T, H, dk, dv, chunk,
                                                                 flags or 0), q.device, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    lib = load_library()
    rest = (float(scale), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state_in),
            _ptr(state_out), _ptr(o), _ptr(workspace), ws_bytes, _stream(stream))
    if flags is None:
        _check(lib.gdr_chunk_prefill(GATES[gate], _DTYPES[q.dtype], B, T, H, dk, dv, chunk, *rest))
    else:
        _check(lib.gdr_chunk_prefill_ex(GATES[gate], _DTYPES[q.dtype], flags, B, T, H, dk, dv, chunk,
                                        *rest))


def gdr_chunk_prefill_varlen_workspace_bytes(gate: str, dtype, N: int, max_T: int, H: int,
                                             dk: int, dv: int, chunk: int = CHUNK,
                                             flags: int = 0) -> int:
    return int(load_library().gdr_chunk_prefill_varlen_workspace_bytes_ex(
        GATES[gate], _DTYPES[dtype], int(flags), N, max_T, H, dk, dv, chunk))


def gdr_chunk_prefill_varlen_ex(gate: str, q, k, v, alpha, beta, cu_seqlens, state_slots, states,
                                o, has_state=None, max_seqlen: Optional[int] = None, flags: int = 0,
                                scale: float = 1.0, workspace=None, chunk: int = CHUNK,
                                stream=None) -> None:
    """:func:`gdr_chunk_prefill_varlen` with an input prologue (``flags`` as
    in :func:`gdr_chunk_prefill_ex`)."""
    _prefill_varlen(int(flags), gate, q, k, v, alpha, beta, cu_seqlens, state_slots, states, o,
                    has_state, max_seqlen, scale, workspace, chunk, stream)


def gdr_chunk_prefill_varlen(gate: str, q, k, v, alpha, beta, cu_seqlens, state_slots, states, o,
                             has_state=None, max_seqlen: Optional[int] = None, scale: float = 1.0,
                             workspace=None, chunk: int = CHUNK, stream=None) -> None:
    """Chunked prefill of packed variable-length sequences with pooled states.

    q, k [total_T,H,dk] and v, o [total_T,H,dv] share a dtype; alpha
    [total_T,H] (gdn) or [total_T,H,dk] (kda) and beta [total_T,H] are fp32;
    cu_seqlens [N+1], state_slots [N] and has_state [N] (optional) are int32
    device tensors; states [n_slots,H,dk,dv] fp32 is read and written in
    place.  max_seqlen bounds every sequence length; if None it is read from
    cu_seqlens (one device-to-host copy).
    """
    _prefill_varlen(None, gate, q, k, v, alpha, beta, cu_seqlens, state_slots, states, o,
                    has_state, max_seqlen, scale, workspace, chunk, stream)


def _prefill_varlen(flags, gate, q, k, v, alpha, beta, cu_seqlens, state_slots, states, o,
                    has_state, max_seqlen, scale, workspace, chunk, stream):
    total_T, H, dk = q.shape
    dv = v.shape[-1]
    N = cu_seqlens.numel() - 1
    if N < 0 or state_slots.shape != (N,) or (has_state is not None and has_state.shape != (N,)):
        raise ValueError("cu_seqlens must be [N+1], state_slots and has_state [N]")
    for t in (cu_seqlens, state_slots, has_state):
        if t is not None and t.dtype != torch.int32:
            raise ValueError("cu_seqlens, state_slots and has_state must be int32")
    if k.shape != q.shape or v.shape != (total_T, H, dv) or o.shape != (total_T, H, dv):
        raise ValueError("q, k, v, o shapes disagree")
    if alpha.shape != ((total_T, H, dk) if gate == "kda" else (total_T, H)) or beta.shape != (total_T, H):
        raise ValueError("alpha / beta shapes disagree with the gate mode")
    if states.dim() != 4 or states.shape[1:] != (H, dk, dv) or states.dtype != torch.float32:
        raise ValueError("states must be fp32 [n_slots,H,dk,dv]")
    if not (q.dtype == k.dtype == v.dtype == o.dtype) or q.dtype not in _DTYPES:
        raise ValueError("q, k, v, o must share dtype fp32 or bf16")
    if alpha.dtype != torch.float32 or beta.dtype != torch.float32:
        raise ValueError("alpha and beta must be fp32")
    _same_device(q, k, v, alpha, beta, cu_seqlens, state_slots, has_state, states, o, workspace)
    if max_seqlen is None:
        cu = cu_seqlens.cpu()
        max_seqlen = int((cu[1:] - cu[:-1]).max()) if N > 0 else 0
    if workspace is None:
        workspace = _workspace(gdr_chunk_prefill_varlen_workspace_bytes(
            gate, q.dtype, N, max_seqlen, H, dk, dv, chunk, flags or 0), q.device, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    lib = load_library()
    rest = (N, total_T, int(max_seqlen), H, dk, dv, chunk, float(scale), _ptr(q), _ptr(k), _ptr(v),
            _ptr(alpha), _ptr(beta), _ptr(cu_seqlens), _ptr(state_slots), _ptr(has_state),
            _ptr(states), states.shape[0], _ptr(o), _ptr(workspace), ws_bytes, _stream(stream))
    if flags is None:
        _check(lib.gdr_chunk_prefill_varlen(GATES[gate], _DTYPES[q.dtype], *rest))
    else:
        _check(lib.gdr_chunk_prefill_varlen_ex(GATES[gate], _DTYPES[q.dtype], flags, *rest))


def gdr_chunk_backward_workspace_bytes(gate: str, dtype, B: int, T: int, H: int, dk: int, dv: int,
                                       chunk: int = CHUNK) -> int:
    return int(load_library().gdr_chunk_backward_workspace_bytes(
        GATES[gate], _DTYPES[dtype], B, T, H, dk, dv, chunk))


def gdr_chunk_backward_workspace_bytes_ranged(gate: str, dtype, B: int, T: int, H: int, dk: int,
                                              dv: int, range_chunks: int, chunk: int = CHUNK) -> int:
    """Workspace with which the backward runs in ranges of ``range_chunks``
    chunks (any workspace from the one-chunk size up is accepted; the widest
    ranges that fit are taken)."""
    return int(load_library().gdr_chunk_backward_workspace_bytes_ranged(
        GATES[gate], _DTYPES[dtype], B, T, H, dk, dv, chunk, range_chunks))


def gdr_chunk_backward(gate: str, q, k, v, alpha, beta, state_in, grad_o, grad_state_out,
                       grad_q, grad_k, grad_v, grad_alpha, grad_beta, grad_state_in=None,
                       scale: float = 1.0, workspace=None, chunk: int = CHUNK, stream=None) -> None:
    """Gradients of sum(grad_o * o) + sum(grad_state_out * S_T) through the
    chunked prefill, written into grad_* (shapes and dtypes of the inputs;
    grad_alpha, grad_beta, grad_state_in fp32).  state_in, grad_state_out and
    grad_state_in may be None.  workspace: a device tensor of at least
    gdr_chunk_backward_workspace_bytes bytes (one pass) or of fewer, down to
    gdr_chunk_backward_workspace_bytes_ranged(..., 1) (chunk ranges), or None
    to allocate the one-pass size."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or v.shape != (B, T, H, dv) or grad_o.shape != (B, T, H, dv):
        raise ValueError("q, k, v, grad_o shapes disagree")
    if grad_q.shape != q.shape or grad_k.shape != q.shape or grad_v.shape != v.shape:
        raise ValueError("gradient shapes must match the inputs")
    ash = (B, T, H, dk) if gate == "kda" else (B, T, H)
    if alpha.shape != ash or beta.shape != (B, T, H) or grad_alpha.shape != ash or grad_beta.shape != (B, T, H):
        raise ValueError("alpha / beta (or their gradients) disagree with the gate mode")
    for st in (state_in, grad_state_out, grad_state_in):
        if st is not None and (st.shape != (B, H, dk, dv) or st.dtype != torch.float32):
            raise ValueError("states must be fp32 [B,H,dk,dv]")
    if not (q.dtype == k.dtype == v.dtype == grad_o.dtype == grad_q.dtype == grad_k.dtype == grad_v.dtype) \
            or q.dtype not in _DTYPES:
        raise ValueError("q, k, v, grad_o and grad_q/k/v must share dtype fp32 or bf16")
    for t in (alpha, beta, grad_alpha, grad_beta):
        if t.dtype != torch.float32:
            raise ValueError("gates and their gradients must be fp32")
    _same_device(q, k, v, alpha, beta, state_in, grad_o, grad_state_out, grad_q, grad_k, grad_v,
                 grad_alpha, grad_beta, grad_state_in, workspace)
    if workspace is None:
        workspace = _workspace(gdr_chunk_backward_workspace_bytes(gate, q.dtype, B, T, H, dk, dv, chunk),
                               q.device, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().gdr_chunk_backward(
        GATES[gate], _DTYPES[q.dtype], B, T, H, dk, dv, chunk, float(scale), _ptr(q), _ptr(k), _ptr(v),
        _ptr(alpha), _ptr(beta), _ptr(state_in), _ptr(grad_o), _ptr(grad_state_out), _ptr(grad_q),
        _ptr(grad_k), _ptr(grad_v), _ptr(grad_alpha), _ptr(grad_beta), _ptr(grad_state_in),
        _ptr(workspace), ws_bytes, _stream(stream)))



# The attention calls are short (a decode step of a small batch takes a few
# microseconds on the GPU), so their checks keep to what a call costs: integer
# device numbers, plain integers as pointers, the raw stream handle.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _attn_device(*ts) -> int:
    """The device number all of the tensors (None ones apart) are on."""
    dev = None
    for t in ts:
        if t is not None:
            n = t.get_device()
            if n != dev:
                if n < 0:
                    raise ValueError("all tensors must be on the GPU")
                if dev is not None:
                    raise ValueError("all tensors must be on one device")
                dev = n
            if not t.is_contiguous():
                raise ValueError("all tensors must be contiguous")
    return dev


def _attn_launch(dev: int, stream, fn, *args) -> None:
    """fn(*args, stream) with `dev` current: a launch belongs to the tensors'
    device, whichever device is current, and by default to its current stream."""
    if stream is None:
        stream = _raw_stream(dev)
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    if dev == torch.cuda.current_device():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status:
        _check(status)


def _on_stream(dev: int, stream):
    """The call's stream as the current one, for torch's own work on its tensors."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(_stream_object(stream, dev))


def _attn_types(q, *ts) -> int:
    """The dtype code of q, which every other tensor shares."""
    dtype = q.dtype
    for t in ts:
        if t.dtype != dtype:
            raise ValueError("q, k, v, o (pages, gradients) must share dtype fp32 or bf16")
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("q, k, v, o (pages, gradients) must share dtype fp32 or bf16")
    return code


def _attn_heads(Hq: int, Hkv: int) -> None:
    if Hq % Hkv if Hkv and Hq else Hq != Hkv:
        raise ValueError("the query heads must be a multiple of the key heads")


def _attn_int(x: int) -> int:
    """x as a C int, of which ctypes would drop the bits above 32: a window, a sink count or a bound beyond it
    says the same as the largest, a size beyond it is refused as that is, and anything negative as -1 is."""
    return -1 if x < 0 else x if x < 0x7fffffff else 0x7fffffff


def _int32(name, t, shape) -> None:
    if t.dtype != torch.int32 or t.shape != shape:
        raise ValueError("%s must be int32 %s" % (name, list(shape)))


def _attn_workspace(workspace, need: int, dev: int, stream):
    """(pointer, bytes, tensor) of the caller's workspace or of one made for this call."""
    if workspace is None:
        if not need:
            return None, 0, None
        workspace = _workspace(need, torch.device("cuda", dev), stream)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def gdr_attn_prefill(q, k, v, o, lse=None, window: int = 0, sinks: int = 0, scale: Optional[float] = None,
                     stream=None) -> None:
    """Causal attention of a prompt, full (``window`` 0) or over the last
    ``window`` positions and the first ``sinks`` keys.

    q, o [B,Tq,Hq,d] and k, v [B,Tk,Hkv,d] share a dtype (fp32 or bf16), d is
    64 or 128 and Hq a multiple of Hkv; the queries are the last Tq of the Tk
    positions.  ``lse`` (optional, fp32 [B,Tq,Hq]) receives the log-sum-exp
    that :func:`gdr_attn_backward` needs.  ``scale`` defaults to d ** -0.5.
    """
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B,Tq,Hq,d], k and v [B,Tk,Hkv,d]")
    B, Tq, Hq, d = shape = q.shape
    _, Tk, Hkv, _ = k.shape
    if k.shape != (B, Tk, Hkv, d) or v.shape != (B, Tk, Hkv, d) or o.shape != shape:
        raise ValueError("q, k, v, o shapes disagree")
    _attn_heads(Hq, Hkv)
    code = _attn_types(q, k, v, o)
    if lse is not None and (lse.shape != shape[:3] or lse.dtype != torch.float32):
        raise ValueError("lse must be fp32 [B,Tq,Hq]")
    dev = _attn_device(q, k, v, o, lse)
    _attn_launch(dev, stream, load_library().gdr_attn_prefill, code, B, Tq, Tk, Hq, Hkv, d, _attn_int(window), _attn_int(sinks),
                 d ** -0.5 if scale is None else scale, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                 None if lse is None else lse.data_ptr())


def gdr_attn_prefill_varlen(q, k, v, cu_q, cu_k, o, lse=None, max_seqlen_q: Optional[int] = None, window: int = 0,
                            sinks: int = 0, scale: Optional[float] = None, stream=None) -> None:
    """:func:`gdr_attn_prefill` of packed sequences: q, o [total_q,Hq,d], k, v
    [total_k,Hkv,d], lse [total_q,Hq]; cu_q and cu_k [N+1] are int32 device
    offsets.  max_seqlen_q bounds every sequence's queries; if None it is read
    from cu_q (one device-to-host copy on the call's stream)."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [total_q,Hq,d], k and v [total_k,Hkv,d]")
    total_q, Hq, d = shape = q.shape
    total_k, Hkv, _ = k.shape
    if k.shape != (total_k, Hkv, d) or v.shape != (total_k, Hkv, d) or o.shape != shape:
        raise ValueError("q, k, v, o shapes disagree")
    _attn_heads(Hq, Hkv)
    code = _attn_types(q, k, v, o)
    N = cu_q.numel() - 1
    if N < 0:
        raise ValueError("cu_q must be [N+1]")
    _int32("cu_q", cu_q, (N + 1,))
    _int32("cu_k", cu_k, (N + 1,))
    if lse is not None and (lse.shape != shape[:2] or lse.dtype != torch.float32):
        raise ValueError("lse must be fp32 [total_q,Hq]")
    dev = _attn_device(q, k, v, cu_q, cu_k, o, lse)
    if max_seqlen_q is None:
        with _on_stream(dev, stream):  # cu_q may be this stream's work
            cu = cu_q.cpu()
        max_seqlen_q = int((cu[1:] - cu[:-1]).max().clamp(min=0)) if N > 0 else 0
    _attn_launch(dev, stream, load_library().gdr_attn_prefill_varlen, code, N, total_q, total_k, _attn_int(max_seqlen_q), Hq, Hkv, d,
                 _attn_int(window), _attn_int(sinks), d ** -0.5 if scale is None else scale, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                 cu_q.data_ptr(), cu_k.data_ptr(), o.data_ptr(), None if lse is None else lse.data_ptr())


def gdr_attn_backward_workspace_bytes(dtype, B: int, Tq: int, Tk: int, Hq: int, Hkv: int, d: int, window: int = 0,
                                      sinks: int = 0) -> int:
    return int(load_library().gdr_attn_backward_workspace_bytes(
        _DTYPES[dtype], *map(_attn_int, (B, Tq, Tk, Hq, Hkv, d, window, sinks))))


def gdr_attn_backward(q, k, v, o, lse, grad_o, grad_q, grad_k, grad_v, window: int = 0, sinks: int = 0,
                      scale: Optional[float] = None, workspace=None, stream=None) -> None:
    """Gradients of sum(grad_o * o) through :func:`gdr_attn_prefill`, written
    into grad_q, grad_k, grad_v (shapes and dtype of q, k, v).  o and lse are
    what the forward wrote for the same q, k, v, window, sinks and scale.
    workspace: a device tensor of at least gdr_attn_backward_workspace_bytes
    bytes, or None to have one allocated for this call."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B,Tq,Hq,d], k and v [B,Tk,Hkv,d]")
    B, Tq, Hq, d = shape = q.shape
    _, Tk, Hkv, _ = kshape = k.shape
    if kshape != (B, Tk, Hkv, d) or v.shape != kshape or o.shape != shape:
        raise ValueError("q, k, v, o shapes disagree")
    if grad_o.shape != shape or grad_q.shape != shape or grad_k.shape != kshape or grad_v.shape != kshape:
        raise ValueError("gradient shapes must match the inputs")
    _attn_heads(Hq, Hkv)
    code = _attn_types(q, k, v, o, grad_o, grad_q, grad_k, grad_v)
    if lse.shape != shape[:3] or lse.dtype != torch.float32:
        raise ValueError("lse must be fp32 [B,Tq,Hq]")
    dev = _attn_device(q, k, v, o, lse, grad_o, grad_q, grad_k, grad_v, workspace)
    need = 0 if workspace is not None else gdr_attn_backward_workspace_bytes(q.dtype, B, Tq, Tk, Hq, Hkv, d, window, sinks)
    ws, ws_bytes, workspace = _attn_workspace(workspace, need, dev, stream)
    _attn_launch(dev, stream, load_library().gdr_attn_backward, code, B, Tq, Tk, Hq, Hkv, d, _attn_int(window), _attn_int(sinks),
                 d ** -0.5 if scale is None else scale, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                 lse.data_ptr(), grad_o.data_ptr(), grad_q.data_ptr(), grad_k.data_ptr(), grad_v.data_ptr(), ws, ws_bytes)


def _page_checks(k_pages, v_pages, page_table, Hkv, d, N):
    if k_pages.dim() != 4 or page_table.dim() != 2:
        raise ValueError("k_pages and v_pages must be [num_pages,Hkv,page_size,d], page_table [sequences,max_pages]")
    num_pages, _, page, _ = shape = k_pages.shape
    if shape != (num_pages, Hkv, page, d) or v_pages.shape != shape:
        raise ValueError("k_pages and v_pages must be [num_pages,Hkv,page_size,d]")
    max_pages = page_table.shape[1]
    _int32("page_table", page_table, (N, max_pages))
    return page, num_pages, max_pages


def gdr_attn_decode_workspace_bytes(dtype, B: int, Hq: int, Hkv: int, d: int, page_size: int, max_pages: int,
                                    window: int = 0, sinks: int = 0) -> int:
    return int(load_library().gdr_attn_decode_workspace_bytes(
        _DTYPES[dtype], *map(_attn_int, (B, Hq, Hkv, d, page_size, max_pages, window, sinks))))


def gdr_attn_decode(q, k, v, k_pages, v_pages, page_table, lengths, o, window: int = 0, sinks: int = 0,
                    scale: Optional[float] = None, workspace=None, stream=None) -> None:
    """One decode step of attention over a paged cache: the new token's k, v
    [B,Hkv,d] are written at position lengths[b] of each sequence and its q
    [B,Hq,d] attends from there, the mask as in :func:`gdr_attn_prefill`.

    k_pages, v_pages [num_pages,Hkv,page_size,d] are updated in place
    (page_size a power of two); page_table [B,max_pages] and lengths [B] are
    int32 device tensors (lengths are not advanced).  workspace: a device
    tensor of at least gdr_attn_decode_workspace_bytes bytes, or None to have
    one allocated for this call.
    """
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [B,Hq,d], k and v [B,Hkv,d]")
    B, Hq, d = shape = q.shape
    Hkv = k.shape[1]
    if k.shape != (B, Hkv, d) or v.shape != (B, Hkv, d) or o.shape != shape:
        raise ValueError("q, k, v, o shapes disagree")
    _attn_heads(Hq, Hkv)
    code = _attn_types(q, k, v, o, k_pages, v_pages)
    page, num_pages, max_pages = _page_checks(k_pages, v_pages, page_table, Hkv, d, B)
    _int32("lengths", lengths, (B,))
    dev = _attn_device(q, k, v, k_pages, v_pages, page_table, lengths, o, workspace)
    need = 0 if workspace is not None else gdr_attn_decode_workspace_bytes(q.dtype, B, Hq, Hkv, d, page, max_pages, window,
                                                                           sinks)
    ws, ws_bytes, workspace = _attn_workspace(workspace, need, dev, stream)
    _attn_launch(dev, stream, load_library().gdr_attn_decode, code, B, Hq, Hkv, d, page, num_pages, max_pages, _attn_int(window), _attn_int(sinks),
                 d ** -0.5 if scale is None else scale, q.data_ptr(), k.data_ptr(), v.data_ptr(), k_pages.data_ptr(),
                 v_pages.data_ptr(), page_table.data_ptr(), lengths.data_ptr(), o.data_ptr(), ws, ws_bytes)


def gdr_attn_append(k, v, cu_seqlens, lengths, k_pages, v_pages, page_table, stream=None) -> None:
    """Writes packed keys and values k, v [total,Hkv,d] to the pages of N
    sequences: token i of sequence n (cu_seqlens [N+1], int32) goes to
    position lengths[n] + i.  Pages, page_table [N,max_pages] and lengths [N]
    as in :func:`gdr_attn_decode`; lengths are not advanced."""
    if k.dim() != 3:
        raise ValueError("k and v must be [total,Hkv,d]")
    total, Hkv, d = shape = k.shape
    if v.shape != shape:
        raise ValueError("k and v shapes disagree")
    code = _attn_types(k, v, k_pages, v_pages)
    N = lengths.numel()
    _int32("lengths", lengths, (N,))
    _int32("cu_seqlens", cu_seqlens, (N + 1,))
    page, num_pages, max_pages = _page_checks(k_pages, v_pages, page_table, Hkv, d, N)
    dev = _attn_device(k, v, cu_seqlens, lengths, k_pages, v_pages, page_table)
    _attn_launch(dev, stream, load_library().gdr_attn_append, code, N, total, Hkv, d, page, num_pages, max_pages,
                 k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), lengths.data_ptr(), k_pages.data_ptr(),
                 v_pages.data_ptr(), page_table.data_ptr())
