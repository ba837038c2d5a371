"""Refusals of the windowed and paged calls, without a GPU: the C ABI returns a status before any
device work, the binding raises on tensors it cannot take."""
import ctypes

import pytest
import torch

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6


@pytest.fixture(scope="module")
def lib():
    from block_sparse_softmax_gb300 import build
    build.build()
    from block_sparse_softmax_gb300 import _lib
    return _lib.load()


P = ctypes.c_void_p(16 * 1000)            # aligned, never dereferenced
ODD = ctypes.c_void_p(16 * 1000 + 2)


def test_window_forward(lib):
    def call(q=P, o=P, lse=P, B=1, H=4, Hkv=2, Lq=64, Lk=64, d=64, scale=0.1, window=8, sinks=0, qo=0,
             ko=0):
        return lib.attn_fwd_window(q, P, P, o, lse, B, H, Hkv, Lq, Lk, d, scale, window, sinks, qo, ko,
                                   None)
    assert call(d=96) == UNSUPPORTED
    for bad in (dict(q=None), dict(q=ODD), dict(o=ODD), dict(lse=ODD), dict(B=0), dict(Hkv=3),
                dict(Lq=-1), dict(Lk=-1), dict(scale=0.0), dict(scale=float("inf")), dict(window=0),
                dict(window=-5), dict(sinks=-1), dict(qo=-1), dict(ko=-1)):
        assert call(**bad) == INVALID, bad
    assert call(Lk=2 ** 31 - 1) == call(Lq=2 ** 31 - 1) == UNSUPPORTED
    assert call(Lq=0, q=None, o=None, lse=None) == 0      # nothing to do


def test_window_backward(lib):
    size = lib.attn_bwd_window_workspace_bytes
    base = (1, 4, 2, 4096, 4096, 64, 256, 4, 0, 0)
    full = size(*base)
    assert full >= 4 * 4096 * 64 * 4
    assert size(1, 4, 3, 4096, 4096, 64, 256, 4, 0, 0) == 0
    assert size(1, 4, 2, 4096, 4096, 96, 256, 4, 0, 0) == 0
    assert size(1, 4, 2, 4096, 4096, 64, 0, 4, 0, 0) == 0
    assert size(1, 4, 2, 4096, 4096, 64, 256, -1, 0, 0) == 0

    # however many keys are sinks, the parts of their walks stay within 8 a multiprocessor
    for sinks in (1, 4, 1000, 16384):
        assert size(2, 16, 16, 16384, 16384, 128, 1, sinks, 0, 0) <= (
            2 * 16 * 16384 * 128 * 4 + 152 * 8 * 2 * 128 * 128 * 4)

    def call(ws=P, nbytes=full, B=1, H=4, Hkv=2, d=64, window=256, sinks=4, q=P, lse=P):
        return lib.attn_bwd_window(q, P, P, P, lse, P, P, P, P, P, ws, nbytes, B, H, Hkv, 4096, 4096, d,
                                   0.1, window, sinks, 0, 0, None)
    assert call(nbytes=full - 1) == WORKSPACE
    assert call(d=32) == UNSUPPORTED
    for bad in (dict(ws=None), dict(ws=ODD), dict(q=ODD), dict(lse=None), dict(Hkv=3), dict(window=0),
                dict(sinks=-1)):
        assert call(**bad) == INVALID, bad


def test_decode(lib):
    full = lib.attn_decode_paged_workspace_bytes(3, 8, 2, 128, 400, 16)
    assert full > 0
    assert lib.attn_decode_paged_workspace_bytes(3, 8, 3, 128, 400, 16) == 0
    assert lib.attn_decode_paged_workspace_bytes(3, 8, 2, 96, 400, 16) == 0
    assert lib.attn_decode_paged_workspace_bytes(0, 8, 2, 128, 4, 16) == 0
    assert lib.attn_decode_paged_workspace_bytes(3, 8, 2, 128, 4, 16) == 0      # small: none needed
    assert lib.attn_decode_paged_workspace_bytes(3, 8, 2, 128, 400, 24) == 0
    assert lib.attn_decode_paged_workspace_bytes(3, 8, 2, 128, 0, 16) == 0
    assert lib.attn_decode_paged_workspace_bytes(9000, 8, 2, 128, 400, 16) <= 16e6

    def call(q=P, qs=8 * 128, ks=2 * 16 * 128, vs=2 * 16 * 128, kind=0, kscale=None, vscale=None,
             table=P, ws=P, nbytes=full, S=3, H=8, Hkv=2, d=128, M=400, n=20, page=16, scale=0.1, window=0,
             sinks=0):
        return lib.attn_decode_paged(q, qs, P, P, ks, vs, kind, kscale, vscale, table, P, P, P, ws, nbytes,
                                     S, H, Hkv, d, M, n, page, scale, window, sinks, None)
    assert call(nbytes=full - 1) == WORKSPACE
    for bad in (dict(d=96), dict(kind=2), dict(page=8), dict(page=24), dict(page=2048),
                dict(S=70000, nbytes=1 << 40)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(q=None), dict(q=ODD), dict(table=None), dict(ws=None), dict(S=0), dict(Hkv=3),
                dict(M=0), dict(n=0), dict(qs=8 * 128 - 8), dict(qs=8 * 128 + 4), dict(ks=2 * 16 * 128 - 8),
                dict(vs=2 * 16 * 128 + 4), dict(scale=-1.0), dict(window=-1), dict(sinks=-1),
                dict(sinks=4), dict(kscale=P), dict(kind=1), dict(kind=1, kscale=P),
                dict(kind=1, kscale=P, vscale=P, ks=2 * 16 * 128 + 8)):
        assert call(**bad) == INVALID, bad


def test_pages(lib):
    def reserve(t=P, n=P, start=P, S=3, M=4, pages=20, page=16):
        return lib.attn_kv_reserve(t, P, P, n, start, S, M, pages, page, None)
    for bad in (dict(t=None), dict(t=ODD), dict(n=None), dict(start=None), dict(S=0), dict(M=0),
                dict(pages=0)):
        assert reserve(**bad) == INVALID, bad
    for bad in (dict(S=70000), dict(page=12), dict(page=2048), dict(pages=(1 << 30) + 1)):
        assert reserve(**bad) == UNSUPPORTED, bad

    def fork(a=P, F=2, src=P):
        return lib.attn_kv_fork(P, P, P, a, P, F, src, P, 3, 4, 20, 16, None)
    assert fork(a=None) == fork(src=None) == fork(F=-1) == INVALID
    assert fork(F=0, a=None, src=None) == 0
    assert lib.attn_kv_free(P, P, P, None, 2, 3, 4, 20, 16, None) == INVALID
    assert lib.attn_kv_free(P, P, P, None, 0, 3, 4, 20, 16, None) == 0
    assert lib.attn_kv_evict(P, P, P, 0, 0, 3, 4, 20, 16, None) == INVALID
    assert lib.attn_kv_evict(P, P, P, 5, -1, 3, 4, 20, 16, None) == INVALID
    assert lib.attn_kv_compact(P, P, P, None, P, 3, 4, 20, None) == INVALID
    assert lib.attn_kv_compact(P, P, P, P, P, 3, 4, 0, None) == INVALID

    def copy(k=P, stride=2 * 16 * 64, kind=0, n=3, src=P, count=None, page=16):
        return lib.attn_kv_copy_pages(k, P, stride, stride, kind, src, P, n, count, 20, 2, 64, page, None)
    for bad in (dict(k=None), dict(k=ODD), dict(stride=2 * 16 * 64 - 8), dict(n=-1), dict(src=None),
                dict(count=ODD)):
        assert copy(**bad) == INVALID, bad
    assert copy(kind=3) == copy(page=17) == UNSUPPORTED
    assert copy(n=0, src=None) == 0

    def write(T=4, row=2 * 64, kind=0, scale=None, new=P):
        return lib.attn_kv_write(new, P, row, row, P, P, 2 * 16 * 64, 2 * 16 * 64, kind, scale, scale, P, P,
                                 P, T, 3, 4, 20, 2, 64, 16, None)
    for bad in (dict(T=-1), dict(row=64), dict(row=2 * 64 + 4), dict(kind=1), dict(scale=P), dict(new=ODD)):
        assert write(**bad) == INVALID, bad
    assert write(T=0, new=None) == 0
    assert lib.attn_status_string(7) == b"ATTN_ERR_BAD_PAGES"
    assert lib.attn_status_string(8) == b"ATTN_ERR_NO_PAGES"


def test_binding_refuses_cpu_tensors(lib):
    import block_sparse_softmax_gb300 as bss
    q = torch.zeros(1, 1, 128, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        bss.attn_fwd_window(q, q, q, 4)
    with pytest.raises(ValueError, match="CUDA"):
        bss.attn_bwd_window(q, q, q, q, torch.zeros(1, 1, 128), q, 4)
    c = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16)
    t, n = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        bss.attn_decode_paged(q[0, :, 0][None], c, c, t, n)
    with pytest.raises(ValueError, match="CUDA"):
        bss.attn_kv_reserve(t, n, n, n, 16)
    with pytest.raises(ValueError, match="CUDA"):
        bss.attn_kv_copy_pages(c, c, n, n)


def test_no_workspace_for_lengths_that_are_refused(lib):
    """Lengths that attn_bwd_window refuses get no size, whatever the sinks; the longest allowed do."""
    size = lib.attn_bwd_window_workspace_bytes
    most = 0x7FFFFF00
    for Lq, Lk in ((128, 2 ** 31 - 1), (2 ** 31 - 1, 128), (128, most + 1), (2 ** 31 - 1, 2 ** 31 - 1)):
        for sinks in (0, 4, 2 ** 31 - 1):
            assert size(1, 1, 1, Lq, Lk, 64, 256, sinks, 0, 0) == 0, (Lq, Lk, sinks)
    acc = 128 * 64 * 4
    for sinks in (0, 4, most):
        assert acc <= size(1, 1, 1, 128, most, 64, 256, sinks, 0, 0) <= acc + 152 * 8 * 2 * 128 * 64 * 4, sinks


def test_decode_takes_the_route_that_measured_faster(lib):
    """A CTA a unit (no workspace) or the units' steps shared evenly, at sizes where the two were
    timed 4 % or more apart (rows as long as the table)."""
    def shared(S, H, Hkv, tokens):
        return lib.attn_decode_paged_workspace_bytes(S, H, Hkv, 128, tokens // 16, 16) > 0
    # S, H, H_kv, tokens a row: one CTA a unit is faster
    for case in ((1, 16, 4, 64), (1, 16, 4, 256), (64, 16, 4, 1024), (512, 16, 4, 1024), (1, 16, 1, 256),
                 (32, 16, 1, 512), (64, 16, 1, 768), (128, 16, 1, 1024), (16, 64, 2, 512), (128, 16, 4, 16),
                 (512, 16, 4, 64), (1024, 16, 4, 512)):
        assert not shared(*case), case
    # ... sharing is
    for case in ((1, 16, 1, 768), (1, 16, 1, 1024), (8, 16, 1, 1024), (32, 16, 1, 1024), (1, 64, 2, 1024),
                 (512, 16, 4, 16), (1024, 16, 4, 16), (1024, 16, 4, 32)):
        assert shared(*case), case
