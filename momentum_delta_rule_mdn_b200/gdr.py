"""The gated delta rule (include/mdn.h, mdn_gdr_*): argument marshalling only.

Per value head, with alpha = exp(alpha_log):

    vtilde_t = v_t - alpha_t S_{t-1}^T k_t
    S_t      = alpha_t S_{t-1} + beta_t k_t vtilde_t^T
    o_t      = scale S_t^T q_t            (scale defaults to d ** -0.5)

q and k have Hk heads, v and the gates H (a multiple of Hk); value head h uses
key head h // (H // Hk).  q, k, v are float32 or bfloat16, gates and states
float32.  Every tensor is contiguous and on one CUDA device, which need not be
the current one; ``stream`` (default: that device's current stream) is the
stream of the work and of the tensors allocated for it.
"""
from __future__ import annotations

import contextlib
import functools
import math
from typing import Optional

import torch

from . import _lib
from .api import _check, _dtype_code, _ptr, library


class _On:
    """Makes ``device`` current and ``stream`` (if given) its current stream, so that
    scratch is allocated, used and freed in that stream's order; gives the stream's
    handle.  With no stream on the current device there is nothing to switch."""
    __slots__ = ("device", "stream", "stack")

    def __init__(self, device: torch.device, stream: Optional[torch.cuda.Stream]):
        if device.type != "cuda":
            raise ValueError(f"tensors must be on a CUDA device, got {device}")
        if stream is not None and stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
        self.device, self.stream, self.stack = device, stream, None

    def __enter__(self) -> int:
        if self.stream is not None or self.device.index != torch.cuda.current_device():
            self.stack = contextlib.ExitStack()
            self.stack.enter_context(torch.cuda.device(self.device))
            self.stack.enter_context(torch.cuda.stream(self.stream))
        return torch._C._cuda_getCurrentRawStream(self.device.index)

    def __exit__(self, *exc):
        if self.stack is not None:
            self.stack.close()


def _need(t, like, dtype, shape, name):
    if t is None:
        return
    if (t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
            or t.get_device() != like.get_device()):
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {like.device}, got "
                         f"{t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()} on {t.device}")


def _fits(*sizes) -> bool:
    """Whether sizes fit the library's ints (a conversion would keep the low 32 bits)."""
    return all(0 <= n < 1 << 31 for n in sizes)


def _heads(q, ref, ref_name, lead):
    """(rows..., Hk, H, d) of a call, its tensors' shapes checked against each other."""
    if q.dim() != lead + 2 or ref.dim() != lead + 2:
        raise ValueError(f"q and {ref_name}: expected {lead + 2} dimensions, got {q.dim()} and "
                         f"{ref.dim()}")
    Hk, d, H = q.shape[-2], q.shape[-1], ref.shape[-2]
    if H % max(Hk, 1) or (Hk == 0) != (H == 0):
        raise ValueError(f"{ref_name} has {H} heads, which is no multiple of q's {Hk}")
    return Hk, H, d


def _scale(scale, d) -> float:
    s = d ** -0.5 if scale is None else float(scale)
    if not math.isfinite(s):
        raise ValueError(f"scale must be finite, got {s}")
    return s


def _workspace(ws, need, like):
    """(pointer, bytes, tensor) of a call's scratch."""
    if ws is None:
        if need == 0:
            return None, 0, None
        ws = like.new_empty(need, dtype=torch.uint8)
    elif ws.device != like.device or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError("workspace: expected a contiguous uint8 tensor on the tensors' device")
    return ws.data_ptr(), ws.numel(), ws


def _cu(cu_seqlens, like):
    if (cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_contiguous() or cu_seqlens.dim() != 1
            or cu_seqlens.numel() < 1):
        raise ValueError("cu_seqlens: expected a contiguous int32 tensor of N+1 offsets")
    if cu_seqlens.device != like.device:
        raise ValueError("cu_seqlens must be on the same device as q")
    return cu_seqlens.numel() - 1


def gdr_chunk_workspace_size(B: int, T: int, Hk: int, H: int, d: int, C: int = 64,
                             dtype: torch.dtype = torch.bfloat16, flags: int = 0, *,
                             packed: bool = False, backward: bool = False) -> int:
    """Scratch bytes of the chunk calls (packed: B sequences in T tokens); 0 if unsupported."""
    if not _fits(B, T, Hk, H, d, C):
        return 0
    return _chunk_bytes(B, T, Hk, H, d, C, dtype, int(flags), packed, backward)


@functools.lru_cache(maxsize=1024)
def _chunk_bytes(B, T, Hk, H, d, C, dtype, flags, packed, backward):
    code = _lib.MDN_BF16 if dtype == torch.bfloat16 else _lib.MDN_F32
    name = f"mdn_gdr_chunk_{'bwd' if backward else 'fwd'}{'_varlen' if packed else ''}_workspace_size"
    return int(getattr(library(), name)(B, T, Hk, H, d, d, C, code, flags))


def _fwd(q, k, v, alpha_log, beta, scale, cu_seqlens, S0, C, out, want_vtilde, workspace, flags,
         stream):
    packed = cu_seqlens is not None
    lead = 1 if packed else 2
    Hk, H, d = _heads(q, v, "v", lead)
    rows = tuple(q.shape[:lead])
    N = _cu(cu_seqlens, q) if packed else rows[0]
    code = _dtype_code(q)
    _need(q, q, q.dtype, q.shape, "q")
    _need(k, q, q.dtype, q.shape, "k")
    _need(v, q, q.dtype, rows + (H, d), "v")
    _need(alpha_log, q, torch.float32, rows + (H,), "alpha_log")
    _need(beta, q, torch.float32, rows + (H,), "beta")
    _need(S0, q, torch.float32, (N, H, d, d), "S0")
    flags = int(flags)
    scale = _scale(scale, d)
    with _On(q.device, stream) as s:
        if out is None:
            o, vt = torch.empty_like(v), torch.empty_like(v) if want_vtilde else None
            S_T = q.new_empty((N, H, d, d), dtype=torch.float32)
            flags |= _lib.MDN_ZERO_BEHIND if packed else 0
        else:
            o, vt, S_T = out
            _need(o, q, q.dtype, v.shape, "o")
            _need(vt, q, q.dtype, v.shape, "vtilde")
            _need(S_T, q, torch.float32, (N, H, d, d), "S_T")
        T = rows[-1]
        ws, ws_bytes, _hold = _workspace(
            workspace, _chunk_bytes(N, T, Hk, H, d, C, q.dtype, flags, packed, False), q)
        lib = library()
        if packed:
            status = lib.mdn_gdr_chunk_fwd_varlen(
                _ptr(q), _ptr(k), _ptr(v), code, _ptr(alpha_log), _ptr(beta), scale,
                _ptr(cu_seqlens), N, T, _ptr(S0), Hk, H, d, d, C, _ptr(o), _ptr(vt), _ptr(S_T),
                ws, ws_bytes, flags, s)
        else:
            status = lib.mdn_gdr_chunk_fwd(
                _ptr(q), _ptr(k), _ptr(v), code, _ptr(alpha_log), _ptr(beta), scale, _ptr(S0), N, T,
                Hk, H, d, d, C, _ptr(o), _ptr(vt), _ptr(S_T), ws, ws_bytes, flags, s)
    _check(status, "mdn_gdr_chunk_fwd" + ("_varlen" if packed else ""))
    return o, vt, S_T


def gdr_chunk_fwd(q, k, v, alpha_log, beta, scale: Optional[float] = None, S0=None, C: int = 64, *,
                  out=None, want_vtilde: bool = True, workspace: Optional[torch.Tensor] = None,
                  flags: int = 0, stream: Optional[torch.cuda.Stream] = None):
    """Gated delta rule over whole sequences.  Returns (o, vtilde or None, S_T).

    q, k: [B,T,Hk,d]; v: [B,T,H,d]; alpha_log, beta: [B,T,H]; S0: [B,H,d,d] or
    None.  ``out`` may hold preallocated (o, vtilde or None, S_T); S_T may be S0.
    vtilde is what :func:`gdr_chunk_bwd` needs (``want_vtilde=False`` leaves it out)."""
    return _fwd(q, k, v, alpha_log, beta, scale, None, S0, C, out, want_vtilde, workspace, flags,
                stream)


def gdr_chunk_fwd_varlen(q, k, v, alpha_log, beta, cu_seqlens: torch.Tensor,
                         scale: Optional[float] = None, S0=None, C: int = 64, *, out=None,
                         want_vtilde: bool = True, workspace: Optional[torch.Tensor] = None,
                         flags: int = 0, stream: Optional[torch.cuda.Stream] = None):
    """The same over N sequences packed along the token axis.

    q, k: [total_T,Hk,d]; v: [total_T,H,d]; gates [total_T,H]; cu_seqlens: int32
    [N+1] on the device, cu_seqlens[N] <= total_T (rows of ``out`` behind it are
    left as they were; of newly allocated outputs they are zero); S0: [N,H,d,d]."""
    return _fwd(q, k, v, alpha_log, beta, scale, cu_seqlens, S0, C, out, want_vtilde, workspace,
                flags, stream)


_GRADS = ("dq", "dk", "dv", "dalpha_log", "dbeta", "dS0")


def _bwd(q, k, alpha_log, beta, cu_seqlens, scale, vtilde, d_o, S0, dS_T, C, workspace, flags,
         stream):
    packed = cu_seqlens is not None
    lead = 1 if packed else 2
    Hk, H, d = _heads(q, vtilde, "vtilde", lead)
    rows = tuple(q.shape[:lead])
    N = _cu(cu_seqlens, q) if packed else rows[0]
    code = _dtype_code(q)
    _need(q, q, q.dtype, q.shape, "q")
    _need(k, q, q.dtype, q.shape, "k")
    _need(vtilde, q, q.dtype, rows + (H, d), "vtilde")
    _need(d_o, q, q.dtype, rows + (H, d), "d_o")
    _need(alpha_log, q, torch.float32, rows + (H,), "alpha_log")
    _need(beta, q, torch.float32, rows + (H,), "beta")
    _need(S0, q, torch.float32, (N, H, d, d), "S0")
    _need(dS_T, q, torch.float32, (N, H, d, d), "dS_T")
    flags = int(flags) | (_lib.MDN_ZERO_BEHIND if packed else 0)
    scale = _scale(scale, d)
    with _On(q.device, stream) as s:
        g = [*map(torch.empty_like, (q, k, vtilde, alpha_log, beta)),
             q.new_empty((N, H, d, d), dtype=torch.float32)]
        T = rows[-1]
        ws, ws_bytes, _hold = _workspace(
            workspace, _chunk_bytes(N, T, Hk, H, d, C, q.dtype, flags, packed, True), q)
        outs = [t.data_ptr() for t in g]
        lib = library()
        if packed:
            status = lib.mdn_gdr_chunk_bwd_varlen(
                _ptr(q), _ptr(k), code, _ptr(alpha_log), _ptr(beta), scale, _ptr(cu_seqlens), N, T,
                _ptr(S0), _ptr(vtilde), _ptr(d_o), _ptr(dS_T), Hk, H, d, d, C, *outs, ws, ws_bytes,
                flags, s)
        else:
            status = lib.mdn_gdr_chunk_bwd(
                _ptr(q), _ptr(k), code, _ptr(alpha_log), _ptr(beta), scale, _ptr(S0), _ptr(vtilde),
                _ptr(d_o), _ptr(dS_T), N, T, Hk, H, d, d, C, *outs, ws, ws_bytes, flags, s)
    _check(status, "mdn_gdr_chunk_bwd" + ("_varlen" if packed else ""))
    return dict(zip(_GRADS, g))


def gdr_chunk_bwd(q, k, alpha_log, beta, scale: Optional[float], vtilde, d_o, S0=None, dS_T=None,
                  C: int = 64, *, workspace: Optional[torch.Tensor] = None, flags: int = 0,
                  stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Gradients of <d_o, o> + <dS_T, S_T> from the ``vtilde`` that
    :func:`gdr_chunk_fwd` saved.  Returns a dict: dq, dk, dv in q's type (dq and
    dk summed over the value heads of a key head), dalpha_log, dbeta, dS0 float32."""
    return _bwd(q, k, alpha_log, beta, None, scale, vtilde, d_o, S0, dS_T, C, workspace, flags,
                stream)


def gdr_chunk_bwd_varlen(q, k, alpha_log, beta, cu_seqlens: torch.Tensor, scale: Optional[float],
                         vtilde, d_o, S0=None, dS_T=None, C: int = 64, *,
                         workspace: Optional[torch.Tensor] = None, flags: int = 0,
                         stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Gradients of :func:`gdr_chunk_fwd_varlen` (zero in the rows behind the last sequence)."""
    return _bwd(q, k, alpha_log, beta, cu_seqlens, scale, vtilde, d_o, S0, dS_T, C, workspace,
                flags, stream)


def gdr_step(q, k, v, alpha_log, beta, scale: Optional[float], S: torch.Tensor, *,
             S_out: Optional[torch.Tensor] = None, o: Optional[torch.Tensor] = None,
             vtilde: Optional[torch.Tensor] = None, want_vtilde: bool = True,
             stream: Optional[torch.cuda.Stream] = None):
    """One decode token: q, k [B,Hk,d]; v [B,H,d]; gates [B,H]; S [B,H,d,d] float32,
    updated in place, or kept with the new state written to ``S_out``.
    Returns (o, vtilde or None)."""
    Hk, H, d = _heads(q, v, "v", 1)
    B = q.shape[0]
    code = _dtype_code(q)
    _need(q, q, q.dtype, (B, Hk, d), "q")
    _need(k, q, q.dtype, (B, Hk, d), "k")
    _need(v, q, q.dtype, (B, H, d), "v")
    _need(alpha_log, q, torch.float32, (B, H), "alpha_log")
    _need(beta, q, torch.float32, (B, H), "beta")
    _need(S, q, torch.float32, (B, H, d, d), "S")
    _need(S_out, q, torch.float32, (B, H, d, d), "S_out")
    _need(o, q, q.dtype, (B, H, d), "o")
    _need(vtilde, q, q.dtype, (B, H, d), "vtilde")
    S_out = S if S_out is None else S_out
    scale = _scale(scale, d)
    with _On(q.device, stream) as s:
        if o is None:
            o = torch.empty_like(v)
        if vtilde is None and want_vtilde:
            vtilde = torch.empty_like(v)
        status = library().mdn_gdr_step(
            _ptr(q), _ptr(k), _ptr(v), code, _ptr(alpha_log), _ptr(beta), scale, _ptr(S),
            _ptr(S_out), B, Hk, H, d, d, _ptr(o), _ptr(vtilde), 0, s)
    _check(status, "mdn_gdr_step")
    return o, vtilde
