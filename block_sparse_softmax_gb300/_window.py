"""Attention with a sliding window and sinks: ``attn_fwd_window`` and ``attn_bwd_window``."""
from __future__ import annotations

import functools
from typing import Optional, Tuple

import torch

from . import OK, AttnError, _lib, _need, _scale

# These calls serve single tokens, where the host's share of a call counts: the checks below cost
# a few attribute reads per tensor where all is well, and look for what is wrong only where it is
# not.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_empty = torch.empty


def _is(t: torch.Tensor, name: str, dtype: torch.dtype, shape, device: int) -> int:
    """The address of a contiguous CUDA tensor of this type and shape on this device."""
    if (t.dtype is dtype and t.is_contiguous() and t.get_device() == device and t.shape == shape
            and device >= 0):
        return t.data_ptr()
    _need(t, name, dtype, shape)
    raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")


_entry = {}


def _run(name: str, device: int, *args) -> None:
    """One library call on the device's current stream; raises on a status other than OK."""
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(_lib.load(), name)
    if device == _current_device():
        st = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(device))
    if st != OK:
        raise AttnError(st, name)


def _out(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape, like: torch.Tensor):
    """(tensor, address) of an output: the caller's, checked, or a new one on ``like``'s device."""
    if t is None:
        t = _empty(shape, dtype=dtype, device=like.device)
        return t, t.data_ptr()
    return t, _is(t, name, dtype, shape, like.get_device())


def _workspace(workspace: Optional[torch.Tensor], nbytes: int, like: torch.Tensor) -> torch.Tensor:
    """The caller's workspace, checked, or a new one of ``nbytes``."""
    if workspace is None:
        return _empty(max(16, nbytes), dtype=torch.uint8, device=like.device)
    if workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {like.device}")
    return workspace


def attn_fwd_window(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window: int, *,
                    sinks: int = 0, scale: Optional[float] = None, q_offset: int = 0,
                    k_offset: int = 0, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """O [B,H,Lq,d] bf16 and LSE [B,H,Lq] fp32 of attention in which query i sees key j when
    0 <= t and (t < window or j + k_offset < sinks), t = (i + q_offset) - (j + k_offset): the
    last ``window`` positions up to its own and the sequence's first ``sinks`` positions.
    k and v may have fewer heads than q (grouped query heads).  A query that sees no key gets
    O = 0, LSE = -inf."""
    B, H, Lq, d = q_shape = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    dev, bf16, fp32 = q.get_device(), torch.bfloat16, torch.float32
    qp = _is(q, "q", bf16, q_shape, dev)
    kp = _is(k, "k", bf16, (B, Hkv, Lk, d), dev)
    vp = _is(v, "v", bf16, (B, Hkv, Lk, d), dev)
    out, op = _out(out, "out", bf16, q_shape, q)
    lse, lp = _out(lse, "lse", fp32, (B, H, Lq), q)
    _run("attn_fwd_window", dev, qp, kp, vp, op, lp, B, H, Hkv, Lq, Lk, d, _scale(scale, d),
         int(window), int(sinks), int(q_offset), int(k_offset))
    return out, lse


def attn_bwd_window_workspace_bytes(B: int, H: int, H_kv: int, Lq: int, Lk: int, d: int,
                                    window: int, sinks: int = 0, q_offset: int = 0,
                                    k_offset: int = 0) -> int:
    return int(_lib.load().attn_bwd_window_workspace_bytes(B, H, H_kv, Lq, Lk, d, int(window),
                                                           int(sinks), int(q_offset),
                                                           int(k_offset)))


_bwd_bytes = functools.lru_cache(maxsize=256)(attn_bwd_window_workspace_bytes)


def attn_bwd_window(q, k, v, o, lse, dout, window: int, *, sinks: int = 0,
                    scale: Optional[float] = None, q_offset: int = 0, k_offset: int = 0,
                    workspace: Optional[torch.Tensor] = None, dq=None, dk=None, dv=None,
                    delta=None):
    """Gradients (dq, dk, dv) bf16 of attn_fwd_window with the same window, sinks, offsets and
    scale, and delta = rowsum(dO * O) fp32, by recomputation.  dk and dv are the same in every
    run; dq's last bit may differ (fp32 additions in the order the key tiles finish)."""
    B, H, Lq, d = q_shape = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    k_shape, rows = (B, Hkv, Lk, d), (B, H, Lq)
    dev, bf16, fp32 = q.get_device(), torch.bfloat16, torch.float32
    qp, op = _is(q, "q", bf16, q_shape, dev), _is(o, "o", bf16, q_shape, dev)
    dop = _is(dout, "dout", bf16, q_shape, dev)
    kp, vp = _is(k, "k", bf16, k_shape, dev), _is(v, "v", bf16, k_shape, dev)
    lp = _is(lse, "lse", fp32, rows, dev)
    dq, dqp = _out(dq, "dq", bf16, q_shape, q)
    dk, dkp = _out(dk, "dk", bf16, k_shape, q)
    dv, dvp = _out(dv, "dv", bf16, k_shape, q)
    delta, dep = _out(delta, "delta", fp32, rows, q)
    window, sinks, q_offset, k_offset = int(window), int(sinks), int(q_offset), int(k_offset)
    ws = _workspace(workspace, 0 if workspace is not None else _bwd_bytes(
        B, H, Hkv, Lq, Lk, d, window, sinks, q_offset, k_offset), q)
    _run("attn_bwd_window", dev, qp, kp, vp, op, lp, dop, dqp, dkp, dvp, dep, ws.data_ptr(),
         ws.numel() * ws.element_size(), B, H, Hkv, Lq, Lk, d, _scale(scale, d), window, sinks,
         q_offset, k_offset)
    return dq, dk, dv, delta
