"""Chunks of new tokens over the paged cache, and rows with pages of their own, at the edges of what
the calls take, on the GPU."""
import math

import pytest
import torch

from oracle import window as ref
from test_gpu_paged import Cache, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bss():
    import block_sparse_softmax_gb300 as m
    m.library()
    return m


@pytest.mark.parametrize("e4m3", [False, True])
def test_as_many_sequences_as_there_may_be(bss, e4m3):
    """65536 sequences of one token each: a row's output is its value's, its LSE its score."""
    S, H, Hkv, d, page, P = 65536, 64, 4, 64, 16, 500
    g = torch.Generator("cuda").manual_seed(1)
    k, v = (torch.randn(P, Hkv, page, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    scales = {}
    if e4m3:
        k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
        scales = dict(k_scale=torch.full((Hkv,), 0.5, device="cuda"), v_scale=torch.full((Hkv,), 0.5, device="cuda"))
    q = torch.randn(S, H, d, generator=g, device="cuda").bfloat16()
    table = torch.randint(0, P, (S, 1), generator=g, device="cuda").int()
    lens = torch.ones(S, dtype=torch.int32, device="cuda")
    lens[12345] = 0                                       # more new tokens than it has
    o, lse = bss.attn_fwd_paged(q, k, v, table, lens, torch.arange(S + 1, device="cuda").int(), **scales)
    assert bss.attn_poll_status() == bss.ERR_BAD_PAGES
    f = 0.5 if e4m3 else 1.0
    at = table[:, 0].long()
    # one key: P is 1 (2^7 as fp16), and O the value itself
    want = (v[at, :, 0].float() * f).bfloat16().repeat_interleave(H // Hkv, 1)
    assert (o[12345] == 0).all() and torch.isneginf(lse[12345]).all()
    o[12345], want[12345] = 0, 0
    assert torch.equal(o, want)
    for a in range(0, S, 8192):
        x = q[a:a + 8192].double() * (k[at[a:a + 8192], :, 0].double() * f).repeat_interleave(H // Hkv, 1)
        score = x.sum(-1) / 8
        # a product's and a sum's roundings, and those of the scale's product and log's
        off = (x.abs().sum(-1) / 8 * 72 + score.abs() * 4) * 2.0 ** -24 + 2.0 ** -22
        bad = (lse[a:a + 8192].double() - score).abs() > off
        if a <= 12345 < a + 8192:
            bad[12345 - a] = False
        assert not bad.any()


@pytest.mark.parametrize("page,columns", [(16, 3), (64, 20)])
def test_more_rows_than_a_launch_takes(bss, page, columns):
    """Selected pages of 65536 rows and some more: each row's attention, those past the 65536th, too;
    rows of no sequence are left as they were."""
    T, H, Hkv, d = 65536 + 77, 2, 1, 64
    n = 30 * page
    c = Cache([n], Hkv, d, page, 3)
    g = torch.Generator("cuda").manual_seed(page)
    q = torch.randn(T, H, d, generator=g, device="cuda").bfloat16()
    places = torch.rand(T, 30, generator=g, device="cuda").argsort(-1)[:, :columns].sort(-1).values
    pages = c.table[0][places][:, None].contiguous()
    lens = torch.randint(0, columns * page + 1, (T,), generator=g, device="cuda").int()
    lens[::1001] = -1
    lens[-1] = columns * page
    o, lse = torch.full_like(q, 7.0), torch.full((T, H), 3.0, device="cuda")
    wide = torch.randn(T, 3, H, d, device="cuda").bfloat16()
    wide[:, 1] = q                                        # strided rows
    for workspace in (None, torch.empty(max(1, bss.attn_decode_paged_workspace_bytes(
            65536, H, Hkv, d, columns, page)), dtype=torch.uint8, device="cuda")):
        bss.attn_decode_selected(wide[:, 1], c.k, c.v, pages, lens, out=o, lse=lse, workspace=workspace)
        assert bss.attn_poll_status() == 0
        gone = lens < 0
        assert (o[gone] == 7.0).all() and (lse[gone] == 3.0).all()
        empty = lens == 0
        assert (o[empty] == 0).all() and torch.isneginf(lse[empty]).all()
        for t in (0, 1, 2, 65534, 65535, 65536, 65537, 65600, T - 2, T - 1):
            m = lens[t].item()
            if m <= 0:
                continue
            at = torch.cat([torch.arange(x * page, (x + 1) * page) for x in places[t].tolist()])[:m]
            args = (q[t][None, :, None], c.k64[0][:, at][None], c.v64[0][:, at][None],
                    torch.ones(1, m, dtype=torch.bool, device="cuda"), 1.0 / math.sqrt(d))
            O, L, _ = ref.forward(*args)
            bo, bl = ref.forward_bounds(*args)
            assert ((o[t].double() - O[0, :, 0]).abs() <= bo[0, :, 0]).all(), t
            assert ((lse[t].double() - L[0, :, 0]).abs() <= bl[0, :, 0]).all(), t
        o.fill_(7.0), lse.fill_(3.0)
