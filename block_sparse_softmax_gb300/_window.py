"""Attention with a sliding window and sinks: ``attn_fwd_window`` and ``attn_bwd_window``."""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _check, _lib, _need, _scale, _stream_of


def _same_device(device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}, got {t.device}")


def attn_fwd_window(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window: int, *,
                    sinks: int = 0, scale: Optional[float] = None, q_offset: int = 0,
                    k_offset: int = 0, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """O [B,H,Lq,d] bf16 and LSE [B,H,Lq] fp32 of attention in which query i sees key j when
    0 <= t and (t < window or j + k_offset < sinks), t = (i + q_offset) - (j + k_offset): the
    last ``window`` positions up to its own and the sequence's first ``sinks`` positions.
    k and v may have fewer heads than q (grouped query heads).  A query that sees no key gets
    O = 0, LSE = -inf."""
    B, H, Lq, d = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    _need(q, "q", torch.bfloat16, (B, H, Lq, d))
    _need(k, "k", torch.bfloat16, (B, Hkv, Lk, d))
    _need(v, "v", torch.bfloat16, (B, Hkv, Lk, d))
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, Lq), device=q.device, dtype=torch.float32) if lse is None else lse
    _need(out, "out", torch.bfloat16, (B, H, Lq, d))
    _need(lse, "lse", torch.float32, (B, H, Lq))
    _same_device(q.device, k=k, v=v, out=out, lse=lse)
    with torch.cuda.device(q.device):
        st = _lib.load().attn_fwd_window(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, Hkv,
            Lq, Lk, d, _scale(scale, d), int(window), int(sinks), int(q_offset), int(k_offset),
            _stream_of(q))
    _check(st, "attn_fwd_window")
    return out, lse


def attn_bwd_window_workspace_bytes(B: int, H: int, H_kv: int, Lq: int, Lk: int, d: int,
                                    window: int, sinks: int = 0, q_offset: int = 0,
                                    k_offset: int = 0) -> int:
    return int(_lib.load().attn_bwd_window_workspace_bytes(B, H, H_kv, Lq, Lk, d, int(window),
                                                           int(sinks), int(q_offset),
                                                           int(k_offset)))


def attn_bwd_window(q, k, v, o, lse, dout, window: int, *, sinks: int = 0,
                    scale: Optional[float] = None, q_offset: int = 0, k_offset: int = 0,
                    workspace: Optional[torch.Tensor] = None, dq=None, dk=None, dv=None,
                    delta=None):
    """Gradients (dq, dk, dv) bf16 of attn_fwd_window with the same window, sinks, offsets and
    scale, and delta = rowsum(dO * O) fp32, by recomputation.  dk and dv are the same in every
    run; dq's last bit may differ (fp32 additions in the order the key tiles finish)."""
    B, H, Lq, d = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    for name, t in (("q", q), ("o", o), ("dout", dout)):
        _need(t, name, torch.bfloat16, (B, H, Lq, d))
    for name, t in (("k", k), ("v", v)):
        _need(t, name, torch.bfloat16, (B, Hkv, Lk, d))
    _need(lse, "lse", torch.float32, (B, H, Lq))
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    delta = torch.empty((B, H, Lq), device=q.device, dtype=torch.float32) if delta is None else delta
    _need(dq, "dq", torch.bfloat16, (B, H, Lq, d))
    _need(dk, "dk", torch.bfloat16, (B, Hkv, Lk, d))
    _need(dv, "dv", torch.bfloat16, (B, Hkv, Lk, d))
    _need(delta, "delta", torch.float32, (B, H, Lq))
    nbytes = attn_bwd_window_workspace_bytes(B, H, Hkv, Lq, Lk, d, window, sinks, q_offset, k_offset)
    if workspace is None:
        workspace = torch.empty(max(16, nbytes), device=q.device, dtype=torch.uint8)
    _same_device(q.device, k=k, v=v, o=o, lse=lse, dout=dout, dq=dq, dk=dk, dv=dv, delta=delta,
                 workspace=workspace)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    with torch.cuda.device(q.device):
        st = _lib.load().attn_bwd_window(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), delta.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), B, H, Hkv, Lq, Lk, d, _scale(scale, d),
            int(window), int(sinks), int(q_offset), int(k_offset), _stream_of(q))
    _check(st, "attn_bwd_window")
    return dq, dk, dv, delta
