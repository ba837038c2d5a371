"""Attention with a sliding window and sinks, from its definition in 64 bits, and how far a
kernel with bf16 products may be from it (test infrastructure only).

Query i at position i + q_offset sees key j at position j + k_offset when, with t the query's
position minus the key's, 0 <= t and (t < window or the key's position < sinks).  Rows that see
nothing have O = 0, LSE = -inf and no gradient.

The bounds count the roundings that such a kernel makes, each by at most half a step of its type
(bf16: 2^-8 of the value, fp32: 2^-24), element by element:

  delta   error of a scaled score: d products, exact in fp32, summed in fp32.  Every partial sum
          is at most sum |q||k|, and an addition may be truncated instead of rounded, so
          delta = scale * sum|q||k| * d * 2^-23.
  P       exp(S - LSE): relative 2 delta (score and normaliser) + 2^-19 (the exponential's and
          the logarithm's own error, and the fp32 sum of the row), and 2^-8 as an operand of P V
          or P^T dO (`p_round` where a kernel holds it in more bits).
  O       sum P |v| times P's error, + 2^-8 |O| for its own rounding.
  D       dO . O with the rounded O: sum |dO| (O's error), + fp32; for rows of few keys
          sum_j P_ij dP_ij in fp32: P's error before any rounding to bf16.  Which rows those are
          `few_keys` says; without it, the rows of at most 16 keys.
  dS      scale P (dP - D): P's error on |dS|, 2^-8 |dS| as an operand, scale P (D's error + dP's).
  dQ, dK  sums of dS's error times |k|, |q|, + 2^-8 of the result.
"""
from __future__ import annotations

import math

import torch

BF16 = 2.0 ** -8


def window_mask(Lq, Lk, window, sinks=0, q_offset=0, k_offset=0, device="cpu"):
    """Boolean [Lq, Lk]: which pairs are allowed."""
    i = torch.arange(Lq, device=device)[:, None] + q_offset
    j = torch.arange(Lk, device=device)[None, :] + k_offset
    return (j <= i) & ((i - j < window) | (j < sinks))


def few_keys(Lq, Lk, window, sinks=0, q_offset=0, k_offset=0, device="cpu"):
    """Boolean [Lq]: the rows whose D attn_bwd_window takes from its definition.  They see at most
    64 keys, and lie near the first key or past the last one (the window holds the first key, or
    reaches past the last but 64), or window and sinks together are at most 32 keys."""
    n = window_mask(Lq, Lk, window, sinks, q_offset, k_offset, device).sum(1)
    own = torch.arange(Lq, device=device) + q_offset - k_offset
    near = (own < 64) | (own - window + 1 >= Lk - 64)
    held = max(0, min(sinks - k_offset, Lk))
    if window + held <= 32 or Lk <= 64:
        near = torch.ones_like(near)
    return near & (n <= 64)


def _grouped(x, H):
    return x.repeat_interleave(H // x.shape[1], dim=1)


def forward(q, k, v, mask, scale):
    """(O, LSE, P) in 64 bits for q [B,H,Lq,d], k and v [B,Hkv,Lk,d]."""
    H = q.shape[1]
    q, k, v = q.double(), _grouped(k, H).double(), _grouped(v, H).double()
    S = torch.where(mask, scale * (q @ k.transpose(-1, -2)), -math.inf)
    lse = torch.logsumexp(S, -1)
    seen = mask.any(-1)
    P = torch.exp(S - torch.where(seen, lse, 0.0)[..., None])
    P = torch.where(mask, P, 0.0)
    return P @ v, torch.where(seen, lse, -math.inf), P


def forward_bounds(q, k, v, mask, scale, p_round=BF16, sums=0.0):
    """(bound of O, bound of LSE) element by element.  p_round: what rounding P takes off it;
    sums: the fp32 sums over the keys, relative to sum P |v| (beside a P in bf16 they vanish)."""
    H, d = q.shape[1], q.shape[-1]
    O, lse, P = forward(q, k, v, mask, scale)
    kk = _grouped(k, H).double()
    size = scale * (q.double().abs() @ kk.abs().transpose(-1, -2))
    delta = torch.where(mask, size, 0.0).amax(-1, keepdim=True) * d * 2.0 ** -23
    spread = P @ _grouped(v, H).double().abs()
    p_rel = 2 * delta + 2.0 ** -19
    p_rel = p_rel + sums
    bound_o = spread * (p_round * (1 + p_rel) + p_rel) + O.abs() * BF16 * (1 + BF16) + spread * BF16 * (
        p_round + p_rel) + 1e-30
    bound_l = delta[..., 0] + torch.nan_to_num(lse, neginf=0.0).abs() * 2.0 ** -22 + 2.0 ** -18
    return bound_o, bound_l


def backward(q, k, v, do, mask, scale):
    """(dq, dk, dv, D) in 64 bits; dk and dv summed over the query heads of their group."""
    B, H, Lq, d = q.shape
    Hkv = k.shape[1]
    O, _, P = forward(q, k, v, mask, scale)
    kk, vv, do, qq = _grouped(k, H).double(), _grouped(v, H).double(), do.double(), q.double()
    D = (do * O).sum(-1, keepdim=True)
    dS = scale * P * (do @ vv.transpose(-1, -2) - D)
    fold = lambda x: x.reshape(B, Hkv, H // Hkv, *x.shape[2:]).sum(2)  # noqa: E731
    return (dS @ kk, fold(dS.transpose(-1, -2) @ qq), fold(P.transpose(-1, -2) @ do), D[..., 0])


def backward_bounds(q, k, v, do, mask, scale, few_rows=None):
    """(bounds of dq, dk, dv, D) element by element; few_rows: `few_keys` of the call."""
    B, H, Lq, d = q.shape
    Hkv = k.shape[1]
    O, lse, P = forward(q, k, v, mask, scale)
    bound_o, bound_l = forward_bounds(q, k, v, mask, scale)
    kk, vv, qq = _grouped(k, H).double(), _grouped(v, H).double(), q.double().abs()
    doa = do.double().abs()
    size = scale * (qq @ kk.abs().transpose(-1, -2))
    delta = torch.where(mask, size, 0.0).amax(-1, keepdim=True) * d * 2.0 ** -23
    # the kernel's P uses the saved LSE, which is off by its bound
    p_rel = 2 * (delta + bound_l[..., None]) + 2.0 ** -19
    dP = do.double() @ vv.transpose(-1, -2)
    dP_size = doa @ vv.abs().transpose(-1, -2)
    D = (do.double() * O).sum(-1, keepdim=True)
    D_err = (doa * bound_o).sum(-1, keepdim=True) + (doa * (O.abs() + bound_o)).sum(
        -1, keepdim=True) * d * 2.0 ** -23
    few = (P * (1 + p_rel) * (dP.abs() * p_rel + dP_size * d * 2.0 ** -23)).sum(-1, keepdim=True)
    if few_rows is None:
        few_rows = mask.sum(-1) <= 16
    D_err = torch.where(few_rows[:, None], few + (P * dP.abs()).sum(
        -1, keepdim=True) * 2.0 ** -19, D_err)
    dS = (scale * P * (dP - D)).abs()
    dS_err = scale * P * (1 + p_rel) * (D_err + dP_size * d * 2.0 ** -23 + (dP.abs() + D.abs()) * 2.0 ** -22)
    dS_err = dS_err + dS * p_rel
    dS_err = dS_err * (1 + BF16) + dS * BF16
    P_err = P * (p_rel + BF16 * (1 + p_rel))
    fold = lambda x: x.reshape(B, Hkv, H // Hkv, *x.shape[2:]).sum(2)  # noqa: E731
    dq, dk, dv, _ = backward(q, k, v, do, mask, scale)
    sums = 2.0 ** -22 * (mask.shape[0] + mask.shape[1]) ** 0.5       # fp32 sums over tiles
    eq = dS_err @ kk.abs() + sums * (dS @ kk.abs())
    ek = fold((dS_err + sums * dS).transpose(-1, -2) @ qq)
    ev = fold((P_err + sums * P).transpose(-1, -2) @ doa)
    out = [e * (1 + BF16) + g.abs() * BF16 + 1e-30 for e, g in ((eq, dq), (ek, dk), (ev, dv))]
    return (*out, D_err[..., 0] + 1e-30)
