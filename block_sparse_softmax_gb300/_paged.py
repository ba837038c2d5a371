"""Paged key/value caches: ``attn_decode_paged`` and the ``attn_kv_*`` calls.

A cache is a pair of tensors [n_pages, H_kv, page_size, d] (bf16, or e4m3 with a scale per K/V
head); its bookkeeping is three int32 tensors on the same device, changed in place: ``page_table``
[S, max_pages] (-1 where a sequence holds no page), ``seq_lens`` [S] and ``refs`` [n_pages] (0 for
a free page).  A fresh cache has -1 in every entry and 0 in every length and count.  What is wrong
in them is found on the device: ``attn_poll_status`` then returns ``ERR_BAD_PAGES``, or
``ERR_NO_PAGES`` where too few pages were free.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _check, _lib, _need, _scale, _stream_of
from ._window import _same_device

KV_BF16 = 0
KV_E4M3 = 1
_KV_DTYPES = {torch.bfloat16: KV_BF16, torch.float8_e4m3fn: KV_E4M3}


def _cache(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale, v_scale, scales: bool = True):
    """(n_pages, H_kv, page_size, d, dtype code, page strides) of a checked cache."""
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype not in _KV_DTYPES:
            raise ValueError(f"{name} must be torch.bfloat16 or torch.float8_e4m3fn, got {t.dtype}")
        if t.dim() != 4:
            raise ValueError(f"{name} must have 4 dimensions [n_pages, H_kv, page_size, d]")
        if t.shape[0] > 0 and not t[0].is_contiguous():
            raise ValueError(f"a page of {name} must be contiguous")
    if v_cache.dtype != k_cache.dtype or v_cache.shape != k_cache.shape:
        raise ValueError(f"v_cache must be {k_cache.dtype} of shape {tuple(k_cache.shape)}, got "
                         f"{v_cache.dtype} of {tuple(v_cache.shape)}")
    P, Hkv, page, d = k_cache.shape
    if scales:
        if (k_cache.dtype == torch.float8_e4m3fn) != (k_scale is not None) or (
                k_scale is None) != (v_scale is None):
            raise ValueError("k_scale and v_scale belong to e4m3 caches, and to no others")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None:
                _need(t, name, torch.float32, (Hkv,))
    _same_device(k_cache.device, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale)
    # a single page has no distance to the next
    ks = k_cache.stride(0) if P > 1 else Hkv * page * d
    vs = v_cache.stride(0) if P > 1 else Hkv * page * d
    return P, Hkv, page, d, _KV_DTYPES[k_cache.dtype], ks, vs


def _state(page_table, seq_lens, refs):
    """(S, max_pages, n_pages) of a checked page table, lengths (or None) and counts (or None)."""
    if page_table.dim() != 2:
        raise ValueError("page_table must have 2 dimensions [S, max_pages]")
    S, M = page_table.shape
    _need(page_table, "page_table", torch.int32, (S, M))
    if seq_lens is not None:
        _need(seq_lens, "seq_lens", torch.int32, (S,))
    P = 0
    if refs is not None:
        P = refs.numel()
        _need(refs, "refs", torch.int32, (P,))
    _same_device(page_table.device, seq_lens=seq_lens, refs=refs)
    return S, M, P


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _rows(t: torch.Tensor, name: str, shape: Tuple[int, int, int]) -> int:
    """The row stride of a bf16 [n, heads, d] tensor whose rows are contiguous."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if shape[0] > 0 and not t[0].is_contiguous():
        raise ValueError(f"a row of {name} must be contiguous")
    return t.stride(0) if shape[0] > 1 else shape[1] * shape[2]


def attn_decode_paged_workspace_bytes(S: int, H: int, H_kv: int, d: int) -> int:
    return int(_lib.load().attn_decode_paged_workspace_bytes(S, H, H_kv, d))


def attn_decode_paged(q, k_cache, v_cache, page_table, seq_lens, *, window: int = 0,
                      sinks: int = 0, scale: Optional[float] = None, k_scale=None, v_scale=None,
                      workspace: Optional[torch.Tensor] = None, out=None, lse=None):
    """Attention of one new token per sequence over a paged cache: O [S,H,d] bf16 and LSE [S,H]
    fp32.  q [S,H,d] bf16 (rows may be strided).  The query of sequence s stands at position
    seq_lens[s] - 1, its key already in the cache; with ``window`` > 0 it sees the last
    ``window`` positions and the first ``sinks`` ones, with 0 every one.  A sequence of length 0
    gets O = 0, LSE = -inf.  The table may have more rows than q has sequences: they are ignored,
    and so are the lengths past the S-th."""
    P, Hkv, page, d, code, ks, vs = _cache(k_cache, v_cache, k_scale, v_scale)
    if q.dim() != 3:
        raise ValueError("q must have 3 dimensions [S, H, d]")
    S, H = q.shape[0], q.shape[1]
    q_stride = _rows(q, "q", (S, H, d))
    rows, M, _ = _state(page_table, seq_lens, None)
    if rows < S:
        raise ValueError(f"page_table has {rows} rows for {S} sequences")
    out = torch.empty((S, H, d), device=q.device, dtype=torch.bfloat16) if out is None else out
    lse = torch.empty((S, H), device=q.device, dtype=torch.float32) if lse is None else lse
    _need(out, "out", torch.bfloat16, (S, H, d))
    _need(lse, "lse", torch.float32, (S, H))
    if workspace is None:
        nbytes = attn_decode_paged_workspace_bytes(S, H, Hkv, d)
        workspace = torch.empty(max(16, nbytes), device=q.device, dtype=torch.uint8)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _same_device(q.device, k_cache=k_cache, page_table=page_table, out=out, lse=lse,
                 workspace=workspace)
    with torch.cuda.device(q.device):
        st = _lib.load().attn_decode_paged(
            q.data_ptr(), q_stride, k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, code,
            _ptr(k_scale), _ptr(v_scale), page_table.data_ptr(), seq_lens.data_ptr(),
            out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), S, H, Hkv, d, M, P, page,
            _scale(scale, d), int(window), int(sinks), _stream_of(q))
    _check(st, "attn_decode_paged")
    return out, lse


def attn_kv_reserve(page_table, seq_lens, refs, n_new, page_size: int, *, start=None):
    """Room for n_new[s] more tokens in every sequence.  Returns ``start`` [S] int32, the position
    of each sequence's first new token, or -1 throughout when the call was refused (then nothing
    changed, and attn_poll_status says why).  n_new may be shorter than the table: the other
    sequences get none."""
    S, M, P = _state(page_table, seq_lens, refs)
    n = n_new.numel()
    _need(n_new, "n_new", torch.int32, (n,))
    if n > S:
        raise ValueError(f"n_new has {n} entries for {S} sequences")
    start = torch.empty((n,), device=page_table.device, dtype=torch.int32) if start is None else start
    _need(start, "start", torch.int32, (n,))
    _same_device(page_table.device, n_new=n_new, start=start)
    with torch.cuda.device(page_table.device):
        st = _lib.load().attn_kv_reserve(page_table.data_ptr(), seq_lens.data_ptr(),
                                         refs.data_ptr(), n_new.data_ptr(), start.data_ptr(), n, M,
                                         P, int(page_size), _stream_of(page_table))
    _check(st, "attn_kv_reserve")
    return start


def attn_kv_write(k_new, v_new, k_cache, v_cache, page_table, start, cu_new, *, k_scale=None,
                  v_scale=None) -> None:
    """Keys and values of new tokens into their pages: rows cu_new[s] .. cu_new[s+1]-1 of k_new
    and v_new [T,H_kv,d] bf16 (rows may be strided) become sequence s's tokens start[s], ...;
    rows from cu_new[S] on are left out.  An e4m3 cache gets round(x / scale[h]), saturated at
    448."""
    P, Hkv, page, d, code, ks, vs = _cache(k_cache, v_cache, k_scale, v_scale)
    T = k_new.shape[0]
    k_row = _rows(k_new, "k_new", (T, Hkv, d))
    v_row = _rows(v_new, "v_new", (T, Hkv, d))
    rows, M, _ = _state(page_table, None, None)
    S = start.numel()
    if rows < S:
        raise ValueError(f"page_table has {rows} rows for {S} sequences")
    _need(start, "start", torch.int32, (S,))
    _need(cu_new, "cu_new", torch.int32, (S + 1,))
    _same_device(k_cache.device, k_new=k_new, v_new=v_new, page_table=page_table, start=start,
                 cu_new=cu_new)
    with torch.cuda.device(k_cache.device):
        st = _lib.load().attn_kv_write(
            k_new.data_ptr(), v_new.data_ptr(), k_row, v_row, k_cache.data_ptr(),
            v_cache.data_ptr(), ks, vs, code, _ptr(k_scale), _ptr(v_scale), page_table.data_ptr(),
            start.data_ptr(), cu_new.data_ptr(), T, S, M, P, Hkv, d, page, _stream_of(k_cache))
    _check(st, "attn_kv_write")


def attn_kv_fork(page_table, seq_lens, refs, parents, children, page_size: int, *, copy_src=None,
                 copy_dst=None):
    """Sequence children[f] becomes a copy of parents[f].  Full pages are shared; of a last page
    that is not full the child takes its own: returns (copy_src, copy_dst) [F] int32, the copies
    to make with attn_kv_copy_pages in every layer's cache (-1: none).  A child must be empty,
    occur once and not be a parent too."""
    S, M, P = _state(page_table, seq_lens, refs)
    F = parents.numel()
    dev = page_table.device
    copy_src = torch.empty((F,), device=dev, dtype=torch.int32) if copy_src is None else copy_src
    copy_dst = torch.empty((F,), device=dev, dtype=torch.int32) if copy_dst is None else copy_dst
    for name, t in (("parents", parents), ("children", children), ("copy_src", copy_src),
                    ("copy_dst", copy_dst)):
        _need(t, name, torch.int32, (F,))
    _same_device(dev, parents=parents, children=children, copy_src=copy_src, copy_dst=copy_dst)
    with torch.cuda.device(dev):
        st = _lib.load().attn_kv_fork(page_table.data_ptr(), seq_lens.data_ptr(), refs.data_ptr(),
                                      parents.data_ptr(), children.data_ptr(), F,
                                      copy_src.data_ptr(), copy_dst.data_ptr(), S, M, P,
                                      int(page_size), _stream_of(page_table))
    _check(st, "attn_kv_fork")
    return copy_src, copy_dst


def attn_kv_free(page_table, seq_lens, refs, seqs, page_size: int) -> None:
    """The listed sequences (int32) give back their pages and become empty; one that is listed
    twice is freed once."""
    S, M, P = _state(page_table, seq_lens, refs)
    n = seqs.numel()
    _need(seqs, "seqs", torch.int32, (n,))
    _same_device(page_table.device, seqs=seqs)
    with torch.cuda.device(page_table.device):
        st = _lib.load().attn_kv_free(page_table.data_ptr(), seq_lens.data_ptr(), refs.data_ptr(),
                                      seqs.data_ptr(), n, S, M, P, int(page_size),
                                      _stream_of(page_table))
    _check(st, "attn_kv_free")


def attn_kv_evict(page_table, seq_lens, refs, window: int, sinks: int, page_size: int) -> None:
    """Every sequence gives back the pages that attn_decode_paged with this window and sinks no
    longer reads, now or at a greater length."""
    S, M, P = _state(page_table, seq_lens, refs)
    with torch.cuda.device(page_table.device):
        st = _lib.load().attn_kv_evict(page_table.data_ptr(), seq_lens.data_ptr(), refs.data_ptr(),
                                       int(window), int(sinks), S, M, P, int(page_size),
                                       _stream_of(page_table))
    _check(st, "attn_kv_evict")


def attn_kv_compact(page_table, refs, *, copy_src=None, copy_dst=None, count=None):
    """The pages in use move to the lowest indices; table and counts follow.  Returns (copy_src,
    copy_dst [n_pages], count [1]) int32: the copies to make with attn_kv_copy_pages in every
    layer's cache."""
    S, M, P = _state(page_table, None, refs)
    dev = page_table.device
    copy_src = torch.empty((P,), device=dev, dtype=torch.int32) if copy_src is None else copy_src
    copy_dst = torch.empty((P,), device=dev, dtype=torch.int32) if copy_dst is None else copy_dst
    count = torch.empty((1,), device=dev, dtype=torch.int32) if count is None else count
    _need(copy_src, "copy_src", torch.int32, (P,))
    _need(copy_dst, "copy_dst", torch.int32, (P,))
    _need(count, "count", torch.int32, (1,))
    _same_device(dev, copy_src=copy_src, copy_dst=copy_dst, count=count)
    with torch.cuda.device(dev):
        st = _lib.load().attn_kv_compact(page_table.data_ptr(), refs.data_ptr(),
                                         copy_src.data_ptr(), copy_dst.data_ptr(),
                                         count.data_ptr(), S, M, P, _stream_of(page_table))
    _check(st, "attn_kv_compact")
    return copy_src, copy_dst, count


def attn_kv_copy_pages(k_cache, v_cache, copy_src, copy_dst, count=None) -> None:
    """Page copy_src[i] of both caches to page copy_dst[i], for every i (the first ``count[0]`` of
    them when ``count``, int32 on the device, is given); a pair of two negative entries is left
    out.  No page may be both a source and a destination, and a destination may occur once."""
    P, Hkv, page, d, code, ks, vs = _cache(k_cache, v_cache, None, None, scales=False)
    n = copy_src.numel()
    _need(copy_src, "copy_src", torch.int32, (n,))
    _need(copy_dst, "copy_dst", torch.int32, (n,))
    if count is not None:
        _need(count, "count", torch.int32, (1,))
    _same_device(k_cache.device, copy_src=copy_src, copy_dst=copy_dst, count=count)
    with torch.cuda.device(k_cache.device):
        st = _lib.load().attn_kv_copy_pages(k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, code,
                                            copy_src.data_ptr(), copy_dst.data_ptr(), n,
                                            _ptr(count), P, Hkv, d, page, _stream_of(k_cache))
    _check(st, "attn_kv_copy_pages")
