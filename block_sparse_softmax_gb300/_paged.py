"""Paged key/value caches: ``attn_decode_paged``, ``attn_fwd_paged``, ``attn_select_pages``,
``attn_decode_selected`` and the ``attn_kv_*`` calls.

A cache is a pair of tensors [n_pages, H_kv, page_size, d] (bf16, or e4m3 with a scale per K/V
head); its bookkeeping is three int32 tensors on the same device, changed in place: ``page_table``
[S, max_pages] (-1 where a sequence holds no page), ``seq_lens`` [S] and ``refs`` [n_pages] (0 for
a free page).  A fresh cache has -1 in every entry and 0 in every length and count.  What is wrong
in them is found on the device: ``attn_poll_status`` then returns ``ERR_BAD_PAGES``, or
``ERR_NO_PAGES`` where too few pages were free.  A call for an empty batch (no sequence, token,
fork or copy) does nothing; outputs without rows are returned.
"""
from __future__ import annotations

import functools
from typing import Optional, Tuple

import torch

from . import _lib, _need, _scale
from ._window import _is, _out, _run, _workspace

KV_BF16 = 0
KV_E4M3 = 1
_DECODE_ROWS = 65536
_INT, _BF16, _FP32, _E4M3 = torch.int32, torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _cache(k_cache: torch.Tensor, v_cache: torch.Tensor, dev: int):
    """(k address, v address, k page stride, v page stride, dtype code) of a checked cache."""
    kind, shape = k_cache.dtype, k_cache.shape
    if (v_cache.dtype is kind and v_cache.shape == shape and (kind is _BF16 or kind is _E4M3)
            and len(shape) == 4 and k_cache.is_contiguous() and v_cache.is_contiguous()
            and k_cache.get_device() == dev and v_cache.get_device() == dev and dev >= 0):
        page = shape[1] * shape[2] * shape[3]
        return (k_cache.data_ptr(), v_cache.data_ptr(), page, page,
                KV_BF16 if kind is _BF16 else KV_E4M3)
    if kind is not _BF16 and kind is not _E4M3:
        raise ValueError(f"k_cache must be torch.bfloat16 or torch.float8_e4m3fn, got {kind}")
    if len(shape) != 4:
        raise ValueError("k_cache must have 4 dimensions [n_pages, H_kv, page_size, d]")
    if v_cache.dtype is not kind or v_cache.shape != shape:
        raise ValueError(f"v_cache must be {kind} of shape {tuple(shape)}, got {v_cache.dtype} of "
                         f"{tuple(v_cache.shape)}")
    P, Hkv, page, d = shape
    strides = []
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.get_device() != dev or dev < 0:
            raise ValueError(f"{name} must be a CUDA tensor on the call's device, got {t.device}")
        if t.is_contiguous():
            strides.append(Hkv * page * d)
        elif P > 1 and t[0].is_contiguous():
            strides.append(t.stride(0))
        else:
            raise ValueError(f"a page of {name} must be contiguous")
    return (k_cache.data_ptr(), v_cache.data_ptr(), strides[0], strides[1],
            KV_BF16 if kind is _BF16 else KV_E4M3)


def _scales(code: int, k_scale, v_scale, Hkv: int, dev: int):
    """The scales' addresses: both for an e4m3 cache, none for a bf16 one."""
    if code == KV_BF16:
        if k_scale is None and v_scale is None:
            return None, None
    elif k_scale is not None and v_scale is not None:
        return (_is(k_scale, "k_scale", _FP32, (Hkv,), dev),
                _is(v_scale, "v_scale", _FP32, (Hkv,), dev))
    raise ValueError("k_scale and v_scale belong to e4m3 caches, both of them, and to no others")


def _table(page_table: torch.Tensor, dev: int):
    """(address, rows, max_pages) of a checked page table."""
    shape = page_table.shape
    if len(shape) != 2:
        raise ValueError("page_table must have 2 dimensions [S, max_pages]")
    return _is(page_table, "page_table", _INT, shape, dev), shape[0], shape[1]


def _state(page_table, seq_lens, refs):
    """(device, table, lengths and counts addresses, S, max_pages, n_pages) of a checked state."""
    dev = page_table.get_device()
    tp, S, M = _table(page_table, dev)
    P = refs.numel()
    return (dev, tp, _is(seq_lens, "seq_lens", _INT, (S,), dev), _is(refs, "refs", _INT, (P,), dev),
            S, M, P)


def _rows(t: torch.Tensor, name: str, shape: Tuple[int, int, int], dev: int) -> int:
    """The row stride of a bf16 [n, heads, d] tensor whose rows are contiguous."""
    if dev >= 0 and t.get_device() == dev and t.dtype is _BF16 and t.shape == shape:
        if t.is_contiguous() or shape[0] == 0:
            return shape[1] * shape[2]
        if t[0].is_contiguous():
            return t.stride(0) if shape[0] > 1 else shape[1] * shape[2]
        raise ValueError(f"a row of {name} must be contiguous")
    _need(t, name, _BF16, shape)
    raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")


def attn_decode_paged_workspace_bytes(S: int, H: int, H_kv: int, d: int, max_pages: int,
                                      page_size: int) -> int:
    return int(_lib.load().attn_decode_paged_workspace_bytes(S, H, H_kv, d, max_pages, page_size))


_decode_bytes = functools.lru_cache(maxsize=256)(attn_decode_paged_workspace_bytes)


def attn_decode_paged(q, k_cache, v_cache, page_table, seq_lens, *, window: int = 0,
                      sinks: int = 0, scale: Optional[float] = None, k_scale=None, v_scale=None,
                      workspace: Optional[torch.Tensor] = None, out=None, lse=None):
    """Attention of one new token per sequence over a paged cache: O [S,H,d] bf16 and LSE [S,H]
    fp32.  q [S,H,d] bf16 (rows may be strided).  The query of sequence s stands at position
    seq_lens[s] - 1, its key already in the cache; with ``window`` > 0 it sees the last
    ``window`` positions and the first ``sinks`` ones, with 0 every one.  A sequence of length 0
    gets O = 0, LSE = -inf.  The table may have more rows than q has sequences: they are ignored,
    and so are the lengths past the S-th."""
    dev = q.get_device()
    kp, vp, ks, vs, code = _cache(k_cache, v_cache, dev)
    P, Hkv, page, d = k_cache.shape
    q_shape = q.shape
    if len(q_shape) != 3:
        raise ValueError("q must have 3 dimensions [S, H, d]")
    S, H, _ = q_shape
    q_stride = _rows(q, "q", (S, H, d), dev)
    ksp, vsp = _scales(code, k_scale, v_scale, Hkv, dev)
    tp, rows, M = _table(page_table, dev)
    if rows < S:
        raise ValueError(f"page_table has {rows} rows for {S} sequences")
    lp = _is(seq_lens, "seq_lens", _INT, (rows,), dev)
    out, op = _out(out, "out", _BF16, (S, H, d), q)
    lse, ep = _out(lse, "lse", _FP32, (S, H), q)
    if S == 0:                                # no sequence asks for anything
        return out, lse
    wp, nbytes = None, 0
    if workspace is None:
        nbytes = _decode_bytes(S, H, Hkv, d, M, page)
    if workspace is not None or nbytes:       # small calls need none
        workspace = _workspace(workspace, nbytes, q)
        wp, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _run("attn_decode_paged", dev, q.data_ptr(), q_stride, kp, vp, ks, vs, code, ksp, vsp, tp, lp,
         op, ep, wp, nbytes, S, H, Hkv, d, M, P, page, _scale(scale, d), int(window), int(sinks))
    return out, lse


def attn_fwd_paged_workspace_bytes(T: int, S: int, H: int, H_kv: int, d: int, max_pages: int,
                                   page_size: int) -> int:
    return int(_lib.load().attn_fwd_paged_workspace_bytes(T, S, H, H_kv, d, max_pages, page_size))


_chunk_bytes = functools.lru_cache(maxsize=256)(attn_fwd_paged_workspace_bytes)


def _rows_of(q, page_table, seq_lens, cu_q, dev: int):
    """(T, H, d, S, max_pages, table, lengths and cu_q addresses) of a ragged batch of new tokens."""
    if len(q.shape) != 3:
        raise ValueError("q must have 3 dimensions [T, H, d]")
    T, H, d = q.shape
    tp, rows, M = _table(page_table, dev)
    S = cu_q.numel() - 1
    if not 0 <= S <= rows:
        raise ValueError(f"page_table has {rows} rows, cu_q {S + 1} entries for one less sequences")
    return (T, H, d, S, M, tp, _is(seq_lens, "seq_lens", _INT, (rows,), dev),
            _is(cu_q, "cu_q", _INT, (S + 1,), dev))


def attn_fwd_paged(q, k_cache, v_cache, page_table, seq_lens, cu_q, *, window: int = 0,
                   sinks: int = 0, scale: Optional[float] = None, k_scale=None, v_scale=None,
                   workspace: Optional[torch.Tensor] = None, out=None, lse=None):
    """Attention of a chunk of new tokens per sequence over a paged cache: O [T,H,d] bf16 and LSE
    [T,H] fp32.  Rows cu_q[s] .. cu_q[s+1]-1 of q [T,H,d] bf16 (rows may be strided) are the last
    tokens of sequence s, their keys already in the cache: row t stands at position i =
    seq_lens[s] - (cu_q[s+1] - t) and sees the keys j <= i, with ``window`` > 0 only those with
    j > i - window or j < sinks.  Rows before cu_q[0] or from cu_q[S] on belong to no sequence:
    their rows of ``out`` and ``lse`` are left as they were.  At most 128 query heads share a K/V
    head.  The table may have more rows than cu_q names sequences: they are ignored."""
    dev = q.get_device()
    kp, vp, ks, vs, code = _cache(k_cache, v_cache, dev)
    P, Hkv, page, d = k_cache.shape
    T, H, _, S, M, tp, lp, cp = _rows_of(q, page_table, seq_lens, cu_q, dev)
    q_stride = _rows(q, "q", (T, H, d), dev)
    ksp, vsp = _scales(code, k_scale, v_scale, Hkv, dev)
    out, op = _out(out, "out", _BF16, (T, H, d), q)
    lse, ep = _out(lse, "lse", _FP32, (T, H), q)
    if T == 0 or S == 0:                      # no row of a sequence
        return out, lse
    ws = _workspace(workspace, 0 if workspace is not None else _chunk_bytes(
        T, S, H, Hkv, d, M, page), q)
    _run("attn_fwd_paged", dev, q.data_ptr(), q_stride, kp, vp, ks, vs, code, ksp, vsp, tp, lp, cp,
         op, ep, ws.data_ptr(), ws.numel() * ws.element_size(), T, S, H, Hkv, d, M, P, page,
         _scale(scale, d), int(window), int(sinks))
    return out, lse


def attn_kv_pool(k_cache, k_means, page_table, start, seq_lens, *, k_scale=None) -> None:
    """The mean keys of the pages that became full between start[s] and seq_lens[s] tokens (start
    as attn_kv_reserve returns it; 0 for all of a sequence's full pages) go to ``k_means``
    [n_pages,H_kv,d] fp32; other pages' stay as they are.  start may be shorter than the table."""
    dev = k_cache.get_device()
    # (one cache alone: the second one's place is taken by the first)
    kp, _, ks, _, code = _cache(k_cache, k_cache, dev)
    P, Hkv, page, d = k_cache.shape
    mp = _is(k_means, "k_means", _FP32, (P, Hkv, d), dev)
    tp, rows, M = _table(page_table, dev)
    S = start.numel()
    if rows < S:
        raise ValueError(f"page_table has {rows} rows for {S} sequences")
    sp, lp = _is(start, "start", _INT, (S,), dev), _is(seq_lens, "seq_lens", _INT, (rows,), dev)
    if (code == KV_E4M3) != (k_scale is not None):
        raise ValueError("k_scale belongs to an e4m3 cache and to no other")
    ksp = None if k_scale is None else _is(k_scale, "k_scale", _FP32, (Hkv,), dev)
    if S == 0:
        return
    _run("attn_kv_pool", dev, kp, ks, code, ksp, mp, tp, sp, lp, S, M, P, Hkv, d, page)


def attn_select_pages_workspace_bytes(T: int, S: int, H: int, H_kv: int, d: int, max_pages: int,
                                      page_size: int, top_r: int, local_pages: int = 1,
                                      first_pages: int = 0) -> int:
    return int(_lib.load().attn_select_pages_workspace_bytes(
        T, S, H, H_kv, d, max_pages, page_size, top_r, local_pages, first_pages))


_select_bytes = functools.lru_cache(maxsize=256)(attn_select_pages_workspace_bytes)


def attn_select_pages(q, k_means, page_table, seq_lens, cu_q, top_r: int, page_size: int, *,
                      local_pages: int = 1, first_pages: int = 0,
                      workspace: Optional[torch.Tensor] = None, pages=None, lens=None):
    """For each new token and K/V head the pages it reads: the first ``first_pages`` of its
    sequence, the last ``local_pages`` up to its own, and the ``top_r`` others whose mean keys
    (``k_means`` [n_pages,H_kv,d] fp32, attn_kv_pool) score highest against the sum of the query
    heads that share the K/V head, ties to the lower place.  q, page_table, seq_lens and cu_q as
    for attn_fwd_paged.  Returns pages [T,H_kv,first+local+top] int32 (in ascending order of their
    place, then -1) and lens [T] int32, the tokens in them (-1 for a row of no sequence), as
    attn_decode_selected takes them."""
    dev = q.get_device()
    T, H, d, S, M, tp, lp, cp = _rows_of(q, page_table, seq_lens, cu_q, dev)
    if len(k_means.shape) != 3:
        raise ValueError("k_means must have 3 dimensions [n_pages, H_kv, d]")
    P, Hkv, _ = k_means.shape
    mp = _is(k_means, "k_means", _FP32, (P, Hkv, d), dev)
    q_stride = _rows(q, "q", (T, H, d), dev)
    top_r, local_pages, first_pages = int(top_r), int(local_pages), int(first_pages)
    R = top_r + local_pages + first_pages
    if top_r < 0 or local_pages < 1 or first_pages < 0:
        raise ValueError("top_r and first_pages must be at least 0, local_pages at least 1")
    if T * Hkv * R >= 1 << 31:
        raise ValueError(f"pages would have {T * Hkv * R} entries; at most 2^31 - 1 are supported")
    pages, pp = _out(pages, "pages", _INT, (T, Hkv, R), q)
    lens, np_ = _out(lens, "lens", _INT, (T,), q)
    if T == 0:
        return pages, lens
    if S == 0:                                # every row is one of no sequence
        return pages.fill_(-1), lens.fill_(-1)
    page_size = int(page_size)
    ws = _workspace(workspace, 0 if workspace is not None else _select_bytes(
        T, S, H, Hkv, d, M, page_size, top_r, local_pages, first_pages), q)
    _run("attn_select_pages", dev, q.data_ptr(), q_stride, mp, tp, lp, cp, pp, np_, ws.data_ptr(),
         ws.numel() * ws.element_size(), T, S, H, Hkv, d, M, P, page_size, top_r, local_pages,
         first_pages)
    return pages, lens


def attn_decode_selected(q, k_cache, v_cache, pages, lens, *, scale: Optional[float] = None,
                         k_scale=None, v_scale=None, workspace: Optional[torch.Tensor] = None,
                         out=None, lse=None):
    """Attention of rows that read pages of their own per K/V head: O [T,H,d] bf16 and LSE [T,H]
    fp32.  Row t's query heads of K/V head h see the first lens[t] tokens of the pages
    pages[t,h,:] (attn_select_pages); a row with lens[t] < 0 is of no sequence, its rows of ``out``
    and ``lse`` are left as they were.  q [T,H,d] bf16 (rows may be strided).  The library takes
    65536 rows at a time; longer batches go to it in parts, and a ``workspace`` is one for a part."""
    dev = q.get_device()
    kp, vp, ks, vs, code = _cache(k_cache, v_cache, dev)
    P, Hkv, page, d = k_cache.shape
    if len(q.shape) != 3 or len(pages.shape) != 3:
        raise ValueError("q must have 3 dimensions [T, H, d], pages 3 [T, H_kv, max_pages]")
    T, H, _ = q.shape
    M = pages.shape[2]
    q_stride = _rows(q, "q", (T, H, d), dev)
    ksp, vsp = _scales(code, k_scale, v_scale, Hkv, dev)
    pp, lp = _is(pages, "pages", _INT, (T, Hkv, M), dev), _is(lens, "lens", _INT, (T,), dev)
    out, op = _out(out, "out", _BF16, (T, H, d), q)
    lse, ep = _out(lse, "lse", _FP32, (T, H), q)
    if T == 0:
        return out, lse
    if T > _DECODE_ROWS:
        if workspace is None:
            workspace = _workspace(None, _decode_bytes(_DECODE_ROWS, H, Hkv, d, M, page), q)
        for a in range(0, T, _DECODE_ROWS):
            b = min(T, a + _DECODE_ROWS)
            attn_decode_selected(q[a:b], k_cache, v_cache, pages[a:b], lens[a:b], scale=scale,
                                 k_scale=k_scale, v_scale=v_scale, workspace=workspace,
                                 out=out[a:b], lse=lse[a:b])
        return out, lse
    wp, nbytes = None, 0
    if workspace is None:
        nbytes = _decode_bytes(T, H, Hkv, d, M, page)
    if workspace is not None or nbytes:       # small calls need none
        workspace = _workspace(workspace, nbytes, q)
        wp, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _run("attn_decode_selected", dev, q.data_ptr(), q_stride, kp, vp, ks, vs, code, ksp, vsp, pp, lp,
         op, ep, wp, nbytes, T, H, Hkv, d, M, P, page, _scale(scale, d))
    return out, lse


def attn_kv_reserve(page_table, seq_lens, refs, n_new, page_size: int, *, start=None):
    """Room for n_new[s] more tokens in every sequence.  Returns ``start`` [S] int32, the position
    of each sequence's first new token, or -1 throughout when the call was refused (then nothing
    changed, and attn_poll_status says why).  n_new may be shorter than the table: the other
    sequences get none."""
    dev, tp, lp, rp, S, M, P = _state(page_table, seq_lens, refs)
    n = n_new.numel()
    np_ = _is(n_new, "n_new", _INT, (n,), dev)
    if n > S:
        raise ValueError(f"n_new has {n} entries for {S} sequences")
    start, sp = _out(start, "start", _INT, (n,), n_new)
    if n == 0:
        return start
    _run("attn_kv_reserve", dev, tp, lp, rp, np_, sp, n, M, P, int(page_size))
    return start


def attn_kv_write(k_new, v_new, k_cache, v_cache, page_table, start, cu_new, *, k_scale=None,
                  v_scale=None) -> None:
    """Keys and values of new tokens into their pages: rows cu_new[s] .. cu_new[s+1]-1 of k_new
    and v_new [T,H_kv,d] bf16 (rows may be strided) become sequence s's tokens start[s], ...;
    rows from cu_new[S] on are left out.  An e4m3 cache gets round(x / scale[h]), saturated at
    448."""
    dev = k_cache.get_device()
    kp, vp, ks, vs, code = _cache(k_cache, v_cache, dev)
    P, Hkv, page, d = k_cache.shape
    T = k_new.shape[0]
    k_row = _rows(k_new, "k_new", (T, Hkv, d), dev)
    v_row = _rows(v_new, "v_new", (T, Hkv, d), dev)
    ksp, vsp = _scales(code, k_scale, v_scale, Hkv, dev)
    tp, rows, M = _table(page_table, dev)
    S = start.numel()
    if rows < S:
        raise ValueError(f"page_table has {rows} rows for {S} sequences")
    sp, cp = _is(start, "start", _INT, (S,), dev), _is(cu_new, "cu_new", _INT, (S + 1,), dev)
    if S == 0:                                # every row is one of no sequence
        return
    _run("attn_kv_write", dev, k_new.data_ptr(), v_new.data_ptr(), k_row, v_row, kp, vp, ks, vs, code,
         ksp, vsp, tp, sp, cp, T, S, M, P, Hkv, d, page)


def attn_kv_fork(page_table, seq_lens, refs, parents, children, page_size: int, *, copy_src=None,
                 copy_dst=None):
    """Sequence children[f] becomes a copy of parents[f].  Full pages are shared; of a last page
    that is not full the child takes its own: returns (copy_src, copy_dst) [F] int32, the copies
    to make with attn_kv_copy_pages in every layer's cache (-1: none).  A child must be empty,
    occur once and not be a parent too."""
    dev, tp, lp, rp, S, M, P = _state(page_table, seq_lens, refs)
    F = parents.numel()
    pp = _is(parents, "parents", _INT, (F,), dev)
    cp = _is(children, "children", _INT, (F,), dev)
    copy_src, csp = _out(copy_src, "copy_src", _INT, (F,), parents)
    copy_dst, cdp = _out(copy_dst, "copy_dst", _INT, (F,), parents)
    _run("attn_kv_fork", dev, tp, lp, rp, pp, cp, F, csp, cdp, S, M, P, int(page_size))
    return copy_src, copy_dst


def attn_kv_free(page_table, seq_lens, refs, seqs, page_size: int) -> None:
    """The listed sequences (int32) give back their pages and become empty; one that is listed
    twice is freed once."""
    dev, tp, lp, rp, S, M, P = _state(page_table, seq_lens, refs)
    n = seqs.numel()
    _run("attn_kv_free", dev, tp, lp, rp, _is(seqs, "seqs", _INT, (n,), dev), n, S, M, P,
         int(page_size))


def attn_kv_evict(page_table, seq_lens, refs, window: int, sinks: int, page_size: int) -> None:
    """Every sequence gives back the pages that attn_decode_paged with this window and sinks no
    longer reads, now or at a greater length."""
    dev, tp, lp, rp, S, M, P = _state(page_table, seq_lens, refs)
    _run("attn_kv_evict", dev, tp, lp, rp, int(window), int(sinks), S, M, P, int(page_size))


def attn_kv_compact(page_table, refs, *, copy_src=None, copy_dst=None, count=None):
    """The pages in use move to the lowest indices; table and counts follow.  Returns (copy_src,
    copy_dst [n_pages], count [1]) int32: the copies to make with attn_kv_copy_pages in every
    layer's cache."""
    dev = page_table.get_device()
    tp, S, M = _table(page_table, dev)
    P = refs.numel()
    rp = _is(refs, "refs", _INT, (P,), dev)
    copy_src, csp = _out(copy_src, "copy_src", _INT, (P,), refs)
    copy_dst, cdp = _out(copy_dst, "copy_dst", _INT, (P,), refs)
    count, cp = _out(count, "count", _INT, (1,), refs)
    _run("attn_kv_compact", dev, tp, rp, csp, cdp, cp, S, M, P)
    return copy_src, copy_dst, count


def attn_kv_copy_pages(k_cache, v_cache, copy_src, copy_dst, count=None) -> None:
    """Page copy_src[i] of both caches to page copy_dst[i], for every i (the first ``count[0]`` of
    them when ``count``, int32 on the device, is given); a pair of two negative entries is left
    out.  No page may be both a source and a destination, and a destination may occur once."""
    dev = k_cache.get_device()
    kp, vp, ks, vs, code = _cache(k_cache, v_cache, dev)
    P, Hkv, page, d = k_cache.shape
    n = copy_src.numel()
    cp = None if count is None else _is(count, "count", _INT, (1,), dev)
    _run("attn_kv_copy_pages", dev, kp, vp, ks, vs, code,
         _is(copy_src, "copy_src", _INT, (n,), dev), _is(copy_dst, "copy_dst", _INT, (n,), dev), n,
         cp, P, Hkv, d, page)
