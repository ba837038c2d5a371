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
    (1, 2, 1, 1, 2000, 128, 1500, 4, 1999, 0),   # CTAs that share a tile's keys: one query
    (1, 2, 2, 300, 2500, 64, 2300, 4, 2200, 0),
    (1, 40, 8, 100, 1300, 64, 1200, 3, 1200, 0),   # ... two CTAs a tile
    (1, 50, 25, 128, 1500, 128, 1400, 0, 1372, 0),
    (1, 4, 2, 1100, 1100, 128, 1000, 2, 0, 0),   # ... and the first tiles have too few for all
    (1, 2, 1, 700, 1500, 64, 900, 300, 1400, 0),  # ... the last queries see sinks alone
    (1, 2, 2, 700, 1500, 128, 900, 0, 2000, 0),  # ... or nothing
    (2, 2, 1, 1000, 700, 64, 10 ** 12, 0, 0, 400),  # ... or the first ones do not
    (1, 50, 50, 2100, 2100, 64, 100, 1200, 0, 0),  # sink tiles for three waves of CTAs
    (1, 48, 48, 1100, 1100, 64, 100, 1100, 0, 0),
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


def test_same_bits_every_run(bss):
    """O, LSE, dK and dV come out the same in every run; dQ is summed in fp32 in the order the key
    tiles finish, so two runs differ by at most a rounding of the sum (2^-8) and of the terms."""
    q, k, v, do = inputs(1, 4, 2, 1500, 1500, 128, 3, 4)
    o, lse = bss.attn_fwd_window(q, k, v, 300, sinks=4)
    first = bss.attn_bwd_window(q, k, v, o, lse, do, 300, sinks=4)
    for _ in range(3):
        o2, lse2 = bss.attn_fwd_window(q, k, v, 300, sinks=4)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        again = bss.attn_bwd_window(q, k, v, o, lse, do, 300, sinks=4)
        assert torch.equal(first[1], again[1]) and torch.equal(first[2], again[2])
        assert torch.equal(first[3], again[3])
        mask = ref.window_mask(1500, 1500, 300, 4, device="cuda")
        bound = ref.backward_bounds(q, k, v, do, mask, 128 ** -0.5)[0]
        assert ((first[0].double() - again[0].double()).abs() <= bound).all()


@pytest.mark.parametrize("windows", [(100, 333), (800, 1100)])
def test_two_streams_at_once(bss, windows):
    """Two calls at a time on streams of their own, with workspaces of their own."""
    a = inputs(1, 8, 2, 900, 900, 64, 1)
    b = inputs(1, 4, 4, 1200, 1200, 128, 2)
    want = []
    for (q, k, v, do), w in ((a, windows[0]), (b, windows[1])):
        o, lse = bss.attn_fwd_window(q, k, v, w, sinks=2)
        want.append((o, lse) + bss.attn_bwd_window(q, k, v, o, lse, do, w, sinks=2)[1:3])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for st, (q, k, v, do), w in zip(streams, (a, b), windows):
            with torch.cuda.stream(st):
                o, lse = bss.attn_fwd_window(q, k, v, w, sinks=2)
                got.append((o, lse) + bss.attn_bwd_window(q, k, v, o, lse, do, w, sinks=2)[1:3])
        torch.cuda.synchronize()
        for x, y in zip(want, got):
            assert all(torch.equal(s, t) for s, t in zip(x, y))
    assert bss.attn_poll_status() == 0


def test_captured_and_replayed(bss):
    """A training step captured in a graph gives, on new contents of its inputs, what the eager
    calls give, also while eager calls on the same tensors run in between."""
    q, k, v, do = inputs(1, 4, 2, 700, 700, 128, 4)
    run = lambda: (lambda o, l: (o, l) + bss.attn_bwd_window(q, k, v, o, l, do, 130, sinks=3))(  # noqa: E731
        *bss.attn_fwd_window(q, k, v, 130, sinks=3))
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for seed in (5, 6):
        for t, new in zip((q, k, v, do), inputs(1, 4, 2, 700, 700, 128, seed)):
            t.copy_(new)
        eager = run()
        graph.replay()
        torch.cuda.synchronize()
        for n in (0, 1, 3, 4, 5):                   # dQ is compared below
            assert torch.equal(held[n], eager[n])
        mask = ref.window_mask(700, 700, 130, 3, device="cuda")
        off = (held[2].double() - ref.backward(q, k, v, do, mask, 128 ** -0.5)[0]).abs()
        assert (off <= ref.backward_bounds(q, k, v, do, mask, 128 ** -0.5)[0]).all()
    assert bss.attn_poll_status() == 0


def test_writes_nothing_else(bss):
    """Outputs inside larger buffers: what lies before and behind them stays."""
    q, k, v, do = inputs(1, 2, 1, 200, 333, 64, 8)
    bufs = {}

    def inside(name, like):
        big = torch.full((like.numel() + 512,), 7.0, device="cuda", dtype=like.dtype)
        bufs[name] = big
        return big[256:256 + like.numel()].view(like.shape)

    lse = torch.empty(1, 2, 200, device="cuda")
    o, l = bss.attn_fwd_window(q, k, v, 50, sinks=1, q_offset=133, out=inside("o", q), lse=inside("l", lse))
    bss.attn_bwd_window(q, k, v, o, l, do, 50, sinks=1, q_offset=133, dq=inside("dq", q),
                        dk=inside("dk", k), dv=inside("dv", v), delta=inside("delta", lse),
                        workspace=inside("ws", torch.empty(bss.attn_bwd_window_workspace_bytes(
                            1, 2, 1, 200, 333, 64, 50, 1, 133) // 4, device="cuda")))
    torch.cuda.synchronize()
    assert bss.attn_poll_status() == 0
    for name, big in bufs.items():
        assert torch.all(big[:256] == 7) and torch.all(big[-256:] == 7), name


def test_refuses_what_it_cannot_take(bss):
    q, k, v, do = inputs(1, 2, 1, 64, 64, 64, 9)
    with pytest.raises(ValueError, match="contiguous"):
        bss.attn_fwd_window(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, 4)
    with pytest.raises(ValueError, match="bfloat16"):
        bss.attn_fwd_window(q.half(), k.half(), v.half(), 4)
    with pytest.raises(ValueError, match="shape"):
        bss.attn_fwd_window(q, k, v[:, :, :32], 4)
    with pytest.raises(bss.AttnError, match="INVALID_ARG"):
        bss.attn_fwd_window(q, k, v, 0)
    o, lse = bss.attn_fwd_window(q, k, v, 4)
    with pytest.raises(bss.AttnError, match="WORKSPACE"):
        bss.attn_bwd_window(q, k, v, o, lse, do, 4, workspace=torch.empty(64, device="cuda"))


@pytest.mark.parametrize("L,window,sinks", [(2, 50, 0), (63, 47, 1), (35, 173, 1), (300, 20, 1)])
def test_gradients_of_few_keys(bss, L, window, sinks):
    """Where rows see few keys, of which a sink has most of the weight, dQ and dK are as exact as
    the roundings of dS and of the result leave them: two of at most 2^-8, which over independent
    terms average 2^-8 / sqrt(3), and dS's terms partly cancel in dQ: within 2^-7 in norm."""
    g = torch.Generator("cuda").manual_seed(L)
    q, k, v, do = (torch.randn(1, 4, L, 128, generator=g, device="cuda") for _ in range(4))
    lead = 0.4 * torch.randn(1, 4, 1, 128, generator=g, device="cuda")
    q, k = q + lead, torch.cat([k[:, :, :sinks] + 2 * lead, k[:, :, sinks:]], 2)
    q, k, v, do = (t.bfloat16() for t in (q, k, v, do))
    o, lse = bss.attn_fwd_window(q, k, v, window, sinks=sinks)
    got = bss.attn_bwd_window(q, k, v, o, lse, do, window, sinks=sinks)
    mask = ref.window_mask(L, L, window, sinks, device="cuda")
    want = ref.backward(q, k, v, do, mask, 128 ** -0.5)
    for a, w in zip(got[:3], want[:3]):
        assert (a.double() - w).norm() <= 2.0 ** -7 * w.norm()
    # D itself: fp32 throughout, so within its few terms' 2^-20
    terms = (want[3].abs().amax() + (do.double().abs() * v.double().abs().amax()).sum(-1).amax()) * 2.0 ** -16
    if L <= 64 or window + sinks <= 32:
        assert (got[3].double() - want[3]).abs().amax() <= terms


def test_a_launch_after_a_timeout_stops(bss):
    """With a timeout in the status word a launch stops at once, block by block, and returns; once
    the word is read and cleared the same calls are right."""
    q, k, v, do = inputs(1, 8, 2, 1000, 1000, 128, 12)
    o, lse = bss.attn_fwd_window(q, k, v, 100, sinks=3)
    bss.attn_watchdog_selftest(1 << 16)
    held = torch.full_like(q, 7.0)
    bss.attn_fwd_window(q, k, v, 100, sinks=3, out=held)
    bss.attn_bwd_window(q, k, v, o, lse, do, 100, sinks=3)
    bss.attn_bwd_window(*(t[..., :64].contiguous() for t in (q, k, v, o)), lse, do[..., :64].contiguous(), 100)
    bss.attn_fwd(q, k, v, causal=True, out=held)
    bss.attn_fwd(q[..., :64].contiguous(), k[..., :64].contiguous(), v[..., :64].contiguous())
    bss.attn_bwd(q, k, v, o, lse, do, causal=True)
    assert bss.attn_poll_status() == bss.ERR_TIMEOUT
    assert torch.all(held == 7)
    assert bss.attn_poll_status() == 0
    mask = ref.window_mask(1000, 1000, 100, 3, device="cuda")
    o, lse = bss.attn_fwd_window(q, k, v, 100, sinks=3, out=held)
    got = bss.attn_bwd_window(q, k, v, o, lse, do, 100, sinks=3)
    check_forward(o, lse, q, k, v, mask, 128 ** -0.5)
    for a, w, b in zip(got, ref.backward(q, k, v, do, mask, 128 ** -0.5),
                       ref.backward_bounds(q, k, v, do, mask, 128 ** -0.5)):
        assert ((a.double() - w).abs() <= b).all()
    assert bss.attn_poll_status() == 0


@pytest.mark.parametrize("B,H,Hkv,Lq,Lk,d,window,sinks,qo,ko", [
    # forward: more query tiles than the device has SMs, so that a CTA takes several, d=128
    (1, 40, 8, 1100, 1100, 128, 100, 4, 0, 0),
    (1, 48, 16, 1300, 1300, 128, 1, 0, 0, 0),      # one block each but for its neighbour's edge
    (1, 64, 8, 1200, 700, 128, 300, 0, 0, 0),      # the last tiles see nothing
    (2, 40, 40, 900, 900, 128, 513, 130, 0, 0),
    (1, 50, 10, 1000, 900, 128, 200, 2, 0, 300),   # ... the first ones
    (1, 70, 70, 1000, 1000, 128, 10 ** 12, 0, 0, 0),
    (1, 64, 4, 1500, 800, 64, 260, 1, 100, 0),     # the same at d=64
    # backward: walks of more than 20 tiles over at least 152 key tiles, a CTA each
    (6, 16, 2, 1600, 1600, 128, 700, 4, 0, 0),
    (6, 16, 2, 1600, 1600, 64, 700, 0, 0, 0),
    (1, 8, 8, 2750, 2750, 64, 2500, 3, 0, 0),
    (1, 8, 8, 2750, 2750, 128, 10 ** 12, 0, 0, 0),
])
def test_many_items_and_long_walks(bss, B, H, Hkv, Lq, Lk, d, window, sinks, qo, ko):
    """What small shapes do not reach: a CTA that goes from query tile to query tile with one Q
    buffer, and key tiles whose walks are long enough for a CTA of their own."""
    test_forward_and_backward(bss, B, H, Hkv, Lq, Lk, d, window, sinks, qo, ko)


@pytest.mark.parametrize("H,Hkv,Lq,Lk,d,window,sinks,qo,ko", [
    (4, 4, 2, 2, 128, 50, 0, 0, 0),
    (4, 2, 63, 63, 128, 47, 1, 0, 0),
    (4, 1, 64, 64, 64, 1000, 0, 0, 0),
    (4, 4, 300, 300, 128, 20, 1, 0, 0),            # every row sees at most 21 keys
    (4, 2, 300, 300, 64, 28, 4, 0, 0),             # ... 32
    (4, 2, 300, 300, 64, 29, 4, 0, 0),             # ... 33: the first 64 rows alone
    (2, 2, 300, 300, 128, 150, 3, 0, 0),
    (2, 1, 300, 300, 128, 64, 0, 0, 0),
    (2, 2, 200, 300, 64, 50, 0, 320, 0),           # rows past the last key
    (2, 2, 200, 300, 128, 100, 10, 250, 0),
    (2, 1, 300, 200, 128, 64, 0, 0, 150),          # a later chunk of keys
    (2, 1, 300, 200, 64, 300, 160, 0, 150),
    (2, 2, 500, 40, 128, 50, 3, 5, 0),             # few keys there are
    (2, 2, 100, 65, 64, 70, 0, 0, 0),
])
def test_rows_of_few_keys(bss, H, Hkv, Lq, Lk, d, window, sinks, qo, ko):
    """Rows of up to 64 keys, of which a sink may have most of the weight, take D from its
    definition: D is off by fp32 sums alone and dQ and dK by what rounding dS and the result leaves.
    (D from the rounded O is up to 2^-8 |dO| |O| off, several times these bounds.)"""
    g = torch.Generator("cuda").manual_seed(Lq + Lk + window)
    q, do = (torch.randn(1, H, Lq, d, generator=g, device="cuda") for _ in range(2))
    k, v = (torch.randn(1, Hkv, Lk, d, generator=g, device="cuda") for _ in range(2))
    lead = 0.4 * torch.randn(1, Hkv, 1, d, generator=g, device="cuda")
    q = q + lead.repeat_interleave(H // Hkv, 1)
    k[:, :, :max(0, min(sinks - ko, Lk))] += 2 * lead
    q, k, v, do = (t.bfloat16() for t in (q, k, v, do))
    opt = dict(sinks=sinks, q_offset=qo, k_offset=ko)
    o, lse = bss.attn_fwd_window(q, k, v, window, **opt)
    got = bss.attn_bwd_window(q, k, v, o, lse, do, window, **opt)
    assert bss.attn_poll_status() == 0
    mask = ref.window_mask(Lq, Lk, window, sinks, qo, ko, "cuda")
    few = ref.few_keys(Lq, Lk, window, sinks, qo, ko, "cuda")
    want = ref.backward(q, k, v, do, mask, d ** -0.5)
    bound = ref.backward_bounds(q, k, v, do, mask, d ** -0.5, few)
    for name, a, w, b in zip(("dq", "dk", "dv", "delta"), got, want, bound):
        off = (a.double() - w).abs()
        assert (off <= b).all(), f"{name}: {(off / b).max().item():.3g} of its bound"
    # the other way to take D would not be within them
    seen = few & (mask.sum(1) > 1)
    if seen.any():
        rough = (do.double() * o.double()).sum(-1)
        assert ((rough - want[3]).abs() > bound[3])[:, :, seen].any()


@pytest.mark.parametrize("B,H,Hkv,Lq,Lk,d,window,sinks,qo,ko", [
    (2, 12, 3, 1111, 1111, 64, 70, 8, 0, 0),       # as many sinks as share a kernel of their own
    (2, 12, 3, 1111, 1111, 64, 70, 9, 0, 0),       # ... one more
    (1, 16, 16, 37, 37, 128, 5, 8, 0, 0),
    (3, 4, 1, 203, 203, 128, 1000, 5, 0, 0),       # a window past every length
    (1, 6, 2, 100, 900, 128, 256, 7, 800, 0),      # a prompt's next chunk
    (1, 4, 2, 500, 700, 64, 60, 7, 900, 4),        # three of seven sinks, queries past the window
    (1, 2, 1, 300, 6, 128, 4, 8, 0, 0),            # nothing but sinks
    (1, 2, 2, 400, 200, 64, 30, 130, 0, 123),      # seven of 130
    (1, 200, 100, 40, 40, 64, 7, 2, 0, 0),
    (1, 16, 4, 5300, 5300, 128, 300, 4, 0, 0),     # a last wave of key tiles that is cut, in 9
    (1, 16, 4, 5000, 5000, 64, 100, 1, 0, 0),      # ... a query tile each
    (1, 8, 8, 2500, 2500, 128, 50, 8, 0, 0),       # ... not, its walks being short
    (20, 16, 1, 1100, 1100, 64, 100, 4, 0, 0),     # ... of a launch of a CTA an item
    (2, 6, 2, 5200, 5200, 64, 130, 3, 0, 0),
    (1, 4, 2, 700, 700, 128, 20, 12, 0, 0),        # every row of few keys: more sinks than share a kernel
    (1, 4, 4, 700, 700, 64, 32, 0, 0, 0),          # ... none
    (2, 4, 1, 500, 40, 128, 50, 13, 5, 0),         # ... no more keys than that
    (1, 4, 2, 300, 64, 64, 10, 40, 0, 0),
])
def test_few_sinks(bss, B, H, Hkv, Lq, Lk, d, window, sinks, qo, ko):
    test_forward_and_backward(bss, B, H, Hkv, Lq, Lk, d, window, sinks, qo, ko)


@pytest.mark.parametrize("H,Hkv,L,d,window,sinks", [(8, 2, 4000, 128, 24, 4), (4, 4, 3001, 64, 20, 8),
                                                    (8, 1, 2500, 128, 700, 1), (6, 3, 2000, 64, 100, 5)])
def test_gradients_of_sinks(bss, H, Hkv, L, d, window, sinks):
    """A sink's dK and dV add up thousands of queries, so elements near 0 show what rounding P and dS
    leaves: two bf16 parts hold all but 2^-15 of each, which over independent terms adds up to
    2^-15 / sqrt(3) of the root of their squares' sum; 2^-12, 14 of those, covers every element and
    the fp32 scores and sums.  (A single bf16 part leaves 2^-8 / sqrt(3).)  dK so where every row
    takes D from its definition; else D's rounded O adds 2^-8 / sqrt(3) of the root of sum dO^2 O^2,
    a row, and 6 of those count."""
    g = torch.Generator("cuda").manual_seed(L)
    q, do = (torch.randn(1, H, L, d, generator=g, device="cuda") for _ in range(2))
    k, v = (torch.randn(1, Hkv, L, d, generator=g, device="cuda") for _ in range(2))
    lead = 0.4 * torch.randn(1, Hkv, 1, d, generator=g, device="cuda")
    q = q + lead.repeat_interleave(H // Hkv, 1)
    k[:, :, :sinks] += 2 * lead
    q, k, v, do = (t.bfloat16() for t in (q, k, v, do))
    o, lse = bss.attn_fwd_window(q, k, v, window, sinks=sinks)
    _, dk, dv, _ = bss.attn_bwd_window(q, k, v, o, lse, do, window, sinks=sinks)
    assert bss.attn_poll_status() == 0
    scale = d ** -0.5
    O, _, P = ref.forward(q, k, v, ref.window_mask(L, L, window, sinks, device="cuda"), scale)
    P, qq, dd = P[..., :sinks], q.double(), do.double()
    vv = v[:, :, :sinks].double().repeat_interleave(H // Hkv, 1)
    dS = scale * P * (dd @ vv.transpose(-1, -2) - (dd * O).sum(-1, keepdim=True))
    fold = lambda x: x.reshape(1, Hkv, H // Hkv, sinks, d).sum(2)  # noqa: E731
    each = lambda a, b: fold((a ** 2).transpose(-1, -2) @ b ** 2).sqrt()  # noqa: E731
    for got, a, b in ((dv, P, dd), (dk, dS, qq)):
        want = fold(a.transpose(-1, -2) @ b)
        tail = 2.0 ** -12 * each(a, b)
        if got is dk and window + sinks > 32:
            off_d = 2.0 ** -8 / 3 ** 0.5 * ((dd * O) ** 2).sum(-1, keepdim=True).sqrt()
            tail = tail + 6 * each(scale * P * off_d, qq)
        off = (got[:, :, :sinks].double() - want).abs()
        bound = 2.0 ** -8 * want.abs() + tail
        assert (off <= bound).all(), (off / bound).max()


def test_rows_of_few_keys_with_more_sinks(bss):
    """The rows' D where every row takes it from its definition and the sinks are too many for a
    kernel of their own."""
    for args in ((4, 2, 700, 700, 128, 20, 12, 0, 0), (4, 4, 500, 40, 64, 50, 13, 5, 0),
                 (2, 1, 300, 64, 128, 10, 40, 0, 0), (4, 4, 600, 600, 64, 32, 0, 0, 0)):
        test_rows_of_few_keys(bss, *args)


def test_sinks_without_a_key(bss):
    q, k, v, do = inputs(1, 2, 1, 90, 0, 128, 1)
    o, lse = bss.attn_fwd_window(q, k, v, 10, sinks=4)
    dq, dk, dv, delta = bss.attn_bwd_window(q, k, v, o, lse, do, 10, sinks=4)
    assert bss.attn_poll_status() == 0
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse))
    assert torch.all(dq == 0) and torch.all(delta == 0) and dk.numel() == dv.numel() == 0
