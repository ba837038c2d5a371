"""Sizes that the calls over chunks and selected pages take, without a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from block_sparse_softmax_gb300 import build
    build.build()
    from block_sparse_softmax_gb300 import _lib
    return _lib.load()


P = ctypes.c_void_p(16 * 1000)            # aligned, never dereferenced


def test_selection_workspace_is_bounded(lib):
    """Scores go through in turns of 2^26, or of one row; beside them a few numbers a row and head."""
    size = lib.attn_select_pages_workspace_bytes
    for T, S, H, Hkv, M in ((10 ** 6, 3, 8, 2, 32768), (100, 3, 256, 256, 32768), (100, 100, 256, 256, 32768),
                            (100, 3, 1024, 1024, 32768), (100, 3, 2048, 2048, 32768), (5, 5, 8192, 4096, 32768),
                            (5000, 3, 65535, 65535, 16), (3, 1, 8, 8, 100)):
        scores = max(1 << 26, Hkv * M)
        rows = max(1, scores // (Hkv * M))
        got = size(T, S, H, Hkv, 128, M, 16, 5, 1, 0)
        assert 4 * min(T, rows // 8 * 8 or rows, 65528) * Hkv * M <= got, (T, Hkv, M)
        assert got <= 4 * scores + 4 * 16 * 152 * max(32, Hkv) + 256, (T, Hkv, M, got)


def test_many_sequences_of_many_rows_are_taken(lib):
    """A batch's rows and heads count, not its sequences times its tiles."""
    UNSUPPORTED, WORKSPACE = 2, 6

    def call(T, S, H, Hkv):
        assert lib.attn_fwd_paged_workspace_bytes(T, S, H, Hkv, 128, 400, 16) > 0
        return lib.attn_fwd_paged(P, H * 128, P, P, Hkv * 16 * 128, Hkv * 16 * 128, 0, None, None, P, P, P, P, P, P,
                                  0, T, S, H, Hkv, 128, 400, 20, 16, 0.1, 0, 0, None)
    for case in ((65536, 65536, 64, 8), (65536, 65536, 128, 8), (10 ** 6, 20000, 16, 4), (3, 1, 2, 2)):
        assert call(*case) == WORKSPACE, case             # (of 0 bytes)
