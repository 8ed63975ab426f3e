"""Group norm with an activation, channels last (include/mdn.h,
mdn_group_norm_*): argument marshalling only.

    xhat = (x - mean) rstd,  n = xhat weight + bias
    y = act(n) without a gate,  y = n act(gate) with one

x is [N, L, C], its C channels in ``groups`` groups of neighbours; statistics are
over the L x C/groups values of a group.  The output of a token mixer,
[B, T, H, d], normed token by token and head by head, is
``o.view(B * T, 1, H * d)`` with ``groups=H``.
"""
from __future__ import annotations

import functools
import math
from typing import Optional

import torch

from . import _lib
from .api import _check, _dtype_code, _ptr, library
from .gdr import _fits, _need, _On, _workspace

_ACT = {"none": _lib.MDN_ACT_NONE, "silu": _lib.MDN_ACT_SILU}


def _common(x, groups, weight, bias, gate, act):
    if act not in _ACT:
        raise ValueError(f"act must be one of {sorted(_ACT)}, got {act!r}")
    if x.dim() != 3:
        raise ValueError(f"x: expected [N, L, C], got {x.dim()} dimensions")
    N, L, C = x.shape
    if groups < 1 or C == 0 or C % groups:
        raise ValueError(f"{C} channels do not divide into {groups} groups")
    if max(N, L, C) >= 1 << 31:  # the library's ints would keep the low 32 bits
        raise ValueError(f"x: sizes must be below 2^31, got {tuple(x.shape)}")
    if (weight is None) != (bias is None):
        raise ValueError("weight and bias: give both or neither")
    code = _dtype_code(x)
    _need(x, x, x.dtype, x.shape, "x")
    _need(gate, x, x.dtype, x.shape, "gate")
    _need(weight, x, torch.float32, (C,), "weight")
    _need(bias, x, torch.float32, (C,), "bias")
    return N, L, C, code


def group_norm_workspace_size(N: int, L: int, C: int, groups: int,
                              dtype: torch.dtype = torch.bfloat16, backward: bool = False) -> int:
    """Scratch bytes of :func:`group_norm_fwd` or :func:`group_norm_bwd`."""
    if not _fits(N, L, C, groups):
        return 0
    return _bytes(N, L, C, groups, _lib.MDN_BF16 if dtype == torch.bfloat16 else _lib.MDN_F32, backward)


@functools.lru_cache(maxsize=1024)
def _bytes(N, L, C, groups, code, backward):
    return int(library().mdn_group_norm_workspace_size(N, L, C, groups, code, int(backward)))


def group_norm_fwd(x, groups: int, weight=None, bias=None, gate=None, eps: float = 1e-5,
                   act: str = "silu", *, out=None, workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None):
    """Returns (y, mean, rstd): y of x's shape and type, mean and rstd [N, groups]
    float32 (what :func:`group_norm_bwd` needs).  ``out`` may hold them preallocated.
    Groups of no rows (L = 0) have mean 0 and rstd eps ** -0.5, those of no spread."""
    N, L, C, code = _common(x, groups, weight, bias, gate, act)
    with _On(x.device, stream) as s:
        if out is None:
            y, mean = torch.empty_like(x), x.new_empty((N, groups), dtype=torch.float32)
            rstd = torch.empty_like(mean)
        else:
            y, mean, rstd = out
            _need(y, x, x.dtype, x.shape, "y")
            _need(mean, x, torch.float32, (N, groups), "mean")
            _need(rstd, x, torch.float32, (N, groups), "rstd")
        ws, ws_bytes, _hold = _workspace(workspace, _bytes(N, L, C, groups, code, False), x)
        status = library().mdn_group_norm_fwd(
            _ptr(x), _ptr(gate), code, _ptr(weight), _ptr(bias), N, L, C, groups, float(eps),
            _ACT[act], _ptr(y), _ptr(mean), _ptr(rstd), ws, ws_bytes, s)
        _check(status, "mdn_group_norm_fwd")
        if L == 0:  # the library has no rows to take statistics of and writes none
            mean.zero_()
            rstd.fill_(float(eps) ** -0.5 if eps > 0 else math.inf)
    return y, mean, rstd


def group_norm_bwd(x, groups: int, mean, rstd, dy, weight=None, bias=None, gate=None,
                   act: str = "silu", *, workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Gradients from the forward pass's mean and rstd.  Returns a dict: dx (x's
    type), with a gate dgate, with weight and bias dweight and dbias (float32)."""
    N, L, C, code = _common(x, groups, weight, bias, gate, act)
    _need(dy, x, x.dtype, x.shape, "dy")
    _need(mean, x, torch.float32, (N, groups), "mean")
    _need(rstd, x, torch.float32, (N, groups), "rstd")
    with _On(x.device, stream) as s:
        g = {"dx": torch.empty_like(x)}
        if gate is not None:
            g["dgate"] = torch.empty_like(x)
        if weight is not None:
            g["dweight"], g["dbias"] = torch.empty_like(weight), torch.empty_like(bias)
        ws, ws_bytes, _hold = _workspace(workspace, _bytes(N, L, C, groups, code, True), x)
        status = library().mdn_group_norm_bwd(
            _ptr(x), _ptr(gate), code, _ptr(weight), _ptr(bias), _ptr(mean), _ptr(rstd), _ptr(dy),
            N, L, C, groups, _ACT[act], _ptr(g["dx"]), _ptr(g.get("dgate")), _ptr(g.get("dweight")),
            _ptr(g.get("dbias")), ws, ws_bytes, s)
    _check(status, "mdn_group_norm_bwd")
    return g
