"""Chunks of new tokens over the paged cache at the edges of what the call takes, on the GPU."""
import pytest
import torch

from test_gpu_paged import ints

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
