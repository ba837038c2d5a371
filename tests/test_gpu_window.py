"""Attention with a sliding window and sinks on the GPU, forward and backward, element by element
against its definition in 64 bits, within bounds that count the kernel's roundings
(`oracle/window.py`)."""
import math

import pytest
import torch

from oracle import window as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bss():
    import block_sparse_softmax_gb300 as m
    m.library()
    return m


def inputs(B, H, Hkv, Lq, Lk, d, seed, sinks=0):
    g = torch.Generator("cuda").manual_seed(seed)
    shapes = [(B, H, Lq, d), (B, Hkv, Lk, d), (B, Hkv, Lk, d), (B, H, Lq, d)]
    q, k, v, do = (torch.randn(s, generator=g, device="cuda") for s in shapes)
    k[:, :, :sinks] += 0.5 * q.mean(dim=(1, 2), keepdim=True)
    return [t.bfloat16() for t in (q, k, v, do)]


def check_forward(o, lse, q, k, v, mask, scale):
    O, L, _ = ref.forward(q, k, v, mask, scale)
    bo, bl = ref.forward_bounds(q, k, v, mask, scale)
    empty = torch.isneginf(L)
    assert torch.equal(torch.isneginf(lse), empty)
    assert torch.all(o[empty] == 0)
    assert torch.isfinite(o).all()
    assert ((o.double() - O).abs() <= bo).all(), ((o.double() - O).abs() / bo).max()
    off = (lse.double() - L).abs()[~empty]
    assert (off <= bl[~empty]).all(), (off / bl[~empty]).max()


SHAPES = [
    # B, H, Hkv, Lq, Lk, d, window, sinks, q_offset, k_offset
    (1, 1, 1, 1, 1, 128, 1, 0, 0, 0),            # one token
    (2, 4, 2, 1, 700, 64, 100, 4, 699, 0),       # one query against many keys
    (1, 2, 1, 300, 300, 128, 1, 0, 0, 0),        # each query sees itself
    (1, 2, 2, 300, 300, 64, 1, 1, 0, 0),
    (1, 4, 2, 777, 777, 128, 128, 4, 0, 0),      # a window of one block
    (1, 4, 4, 777, 777, 64, 127, 0, 0, 0),
    (1, 2, 1, 1000, 1000, 128, 129, 130, 0, 0),  # sinks past a block
    (2, 2, 2, 640, 640, 64, 300, 128, 0, 0),
    (1, 2, 1, 1100, 1100, 128, 513, 1, 0, 0),
    (1, 3, 1, 500, 500, 64, 10 ** 12, 0, 0, 0),  # a window past every length: causal
    (1, 3, 3, 500, 500, 128, 40, 10 ** 12, 0, 0),  # every key a sink: causal
    (1, 4, 1, 100, 900, 128, 256, 4, 800, 0),    # a prompt's next chunk
    (1, 2, 2, 200, 300, 64, 50, 0, 320, 0),      # some queries past the window of every key
    (1, 2, 2, 200, 300, 128, 50, 3, 320, 0),     # ... but not of the sinks
    (1, 2, 1, 300, 200, 128, 64, 0, 0, 150),     # the first queries before every key
    (1, 2, 1, 300, 200, 64, 64, 160, 0, 150),    # a chunk with the last of the sinks
    (1, 2, 1, 130, 260, 128, 64, 4, 2 ** 40, 2 ** 40 - 130),  # far positions
    (1, 1, 1, 64, 64, 64, 8, 2, 2 ** 40, 0),     # nothing but sinks is near
    (2, 4, 2, 3, 3, 128, 50, 4, 0, 0),           # three tokens
    (1, 2, 1, 9, 9, 64, 5, 1, 0, 0),
    (1, 2, 2, 200, 200, 64, 9, 7, 0, 0),         # every row sees at most 16 keys
    (1, 2, 2, 200, 200, 128, 10, 7, 0, 0),       # ... 17
    (1, 2, 2, 100, 12, 128, 50, 0, 0, 0),        # 12 keys, queries run past them
    (1, 2, 2, 100, 40, 64, 50, 3, 5, 0),
    (1, 2, 1, 0, 70, 64, 5, 0, 0, 0),            # no query
]


@pytest.mark.parametrize("B,H,Hkv,Lq,Lk,d,window,sinks,qo,ko", SHAPES)
def test_forward_and_backward(bss, B, H, Hkv, Lq, Lk, d, window, sinks, qo, ko):
    q, k, v, do = inputs(B, H, Hkv, Lq, Lk, d, Lq + 3 * Lk + window % 1000, min(sinks, Lk))
    scale = 1.0 / math.sqrt(d)
    mask = ref.window_mask(Lq, Lk, window, sinks, qo, ko, "cuda")
    opt = dict(sinks=sinks, q_offset=qo, k_offset=ko)
    o, lse = bss.attn_fwd_window(q, k, v, window, **opt)
    got = bss.attn_bwd_window(q, k, v, o, lse, do, window, **opt)
    torch.cuda.synchronize()
    assert bss.attn_poll_status() == 0
    check_forward(o, lse, q, k, v, mask, scale)
    want = ref.backward(q, k, v, do, mask, scale)
    bound = ref.backward_bounds(q, k, v, do, mask, scale)
    for name, a, w, b in zip(("dq", "dk", "dv", "delta"), got, want, bound):
        off = (a.double() - w).abs()
        assert torch.isfinite(a).all(), name
        assert (off <= b).all(), f"{name}: {(off / b).max().item():.3g} of its bound"
    unseen = ~mask.any(0)
    assert torch.all(got[1][:, :, unseen] == 0) and torch.all(got[2][:, :, unseen] == 0)
    assert torch.all(got[0][:, :, ~mask.any(1)] == 0)


@pytest.mark.parametrize("d", [64, 128])
def test_no_key(bss, d):
    q, k, v, do = inputs(1, 2, 1, 70, 0, d, 1)
    o, lse = bss.attn_fwd_window(q, k, v, 5)
    dq, dk, dv, delta = bss.attn_bwd_window(q, k, v, o, lse, do, 5)
    assert bss.attn_poll_status() == 0
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse))
    assert torch.all(dq == 0) and torch.all(delta == 0) and dk.numel() == dv.numel() == 0
