"""The operators for serving and training with a bounded key/value memory, as measured cases.

Three groups that belong together:
  * attention with a sliding window and a few first tokens that stay visible (sinks): a prompt
    (`attn_fwd_window`) and a training step (`attn_fwd_window` and `attn_bwd_window`);
  * attention of one new token per sequence over a paged key/value cache (`attn_decode_paged`),
    with or without that window, over bf16 or e4m3 pages;
  * the pages themselves: a decoding step's eviction, reservation and write (`attn_kv_evict`,
    `attn_kv_reserve`, `attn_kv_write`), forking (`attn_kv_fork`, `attn_kv_copy_pages`) and
    compaction (`attn_kv_compact`, `attn_kv_copy_pages`).

Each is computed in two ways: by elementary torch operations in 32 bits (`own` False), and by the
package's entry points (`own` True).  `exact` follows the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

PAIR = 0.6180339887498949   # spreads the sequences' lengths over their range
LEAST = 1e-30               # a sum of exponentials that is below this is an empty row's


# ----------------------------------------------------------------------------
# the cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # a prompt through a windowed layer with four sinks, grouped heads, 16384 tokens: the
        # longest prompt of the repository's own workloads
        dict(name="window-prompt-16384", op="window", B=2, H=16, Hkv=4, Lq=16384, Lk=16384, d=128,
             window=1024, sinks=4, past=0, grad=False),
        # the next chunk of a long prompt: 500 queries at the end of 8191 cached keys
        dict(name="window-chunk-500", op="window", B=1, H=16, Hkv=4, Lq=500, Lk=8191, d=128,
             window=2048, sinks=4, past=0, grad=False),
        # a training step at head dimension 64, sequences of odd length, one K/V head a query head
        dict(name="window-train-2000-d64", op="window", B=4, H=16, Hkv=16, Lq=2000, Lk=2000, d=64,
             window=256, sinks=0, past=0, grad=True),
        # a long training step with grouped heads and sinks that every query sees
        dict(name="window-train-16384", op="window", B=1, H=16, Hkv=4, Lq=16384, Lk=16384, d=128,
             window=1024, sinks=4, past=0, grad=True),
        # one conversation that has just begun: latency alone counts
        dict(name="decode-one-300", op="decode", S=1, H=16, Hkv=4, d=128, page=16, longest=300,
             ragged=False, window=0, sinks=0, kv="bf16"),
        # a batch of conversations of very different lengths
        dict(name="decode-32-ragged-8192", op="decode", S=32, H=16, Hkv=4, d=128, page=64,
             longest=8192, ragged=True, window=0, sinks=0, kv="bf16"),
        # two documents of 131071 tokens: few rows, a long cache
        dict(name="decode-2-131071", op="decode", S=2, H=8, Hkv=8, d=128, page=128, longest=131071,
             ragged=False, window=0, sinks=0, kv="bf16"),
        # a full server over an 8-bit cache
        dict(name="decode-128-e4m3-16384", op="decode", S=128, H=16, Hkv=4, d=128, page=64,
             longest=16384, ragged=True, window=0, sinks=0, kv="e4m3"),
        # endless streams: each sequence reads its sinks and its window out of a long cache
        dict(name="decode-64-window-d64", op="decode", S=64, H=16, Hkv=16, d=64, page=32,
             longest=16384, ragged=True, window=1000, sinks=4, kv="bf16"),
        # the bookkeeping of one decoding step, and its new keys and values
        dict(name="pages-step-256", op="step", S=256, Hkv=4, d=128, page=32, longest=4096, fresh=1,
             window=1024, sinks=4, kv="bf16"),
        # every conversation is continued in four ways (parallel samples, beams)
        dict(name="pages-fork-32x4", op="fork", S=32, ways=4, Hkv=4, d=128, page=64, longest=2047),
        # a fragmented cache is packed together
        dict(name="pages-compact-16384", op="compact", S=256, pages=16384, Hkv=4, d=128, page=64,
             keep=0.5),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "decode", "decode", "decode", "decode", "step",
                     "fork", "compact"])
    d = rng.choice([64, 128, 128])
    H, Hkv = rng.choice([(16, 16), (16, 4), (8, 8), (8, 1), (6, 2), (16, 2), (20, 1)])
    if op == "window":
        grad = rng.random() < 0.5
        Lk = _spread(rng, 1, 16384)
        B = 1 if Lk > 8000 else rng.choice([1, 2])
        # a prompt, or a prompt's next chunk
        Lq = Lk if grad or rng.random() < 0.5 else _spread(rng, 1, Lk)
        window = _spread(rng, 1, 4096)
        if B * H * Lq * min(Lk, window) > 1.5e8:
            window = max(1, int(1.5e8 / (B * H * Lq)))
        # now and then the queries lie past the last key, as against an earlier chunk of keys: some
        # may see none
        past = _spread(rng, 1, 2 * window) if rng.random() < 0.2 else 0
        return dict(op=op, B=B, H=min(H, 16), Hkv=Hkv if H <= 16 else 1, Lq=Lq, Lk=Lk, d=d,
                    window=window, sinks=rng.choice([0, 1, 4, 4, 130]), past=past, grad=grad)
    page = rng.choice([16, 32, 64, 128])
    kv = rng.choice(["bf16", "bf16", "e4m3"])
    if op == "decode":
        S = _spread(rng, 1, 128)
        longest = _spread(rng, 1, min(131072, max(1, (1 << 28) // (S * Hkv * d))))
        w = rng.random() < 0.4
        return dict(op=op, S=S, H=H, Hkv=Hkv, d=d, page=page, longest=longest,
                    ragged=rng.random() < 0.7, window=_spread(rng, 1, 4096) if w else 0,
                    sinks=rng.choice([0, 1, 4, 70]) if w else 0, kv=kv)
    if op == "step":
        w = rng.random() < 0.5
        return dict(op=op, S=_spread(rng, 1, 256), Hkv=Hkv, d=d, page=page,
                    longest=_spread(rng, 1, 4096), fresh=_spread(rng, 1, 64),
                    window=_spread(rng, 1, 1024) if w else 0, sinks=4 if w else 0, kv=kv)
    if op == "fork":
        return dict(op=op, S=_spread(rng, 1, 32), ways=rng.choice([1, 2, 4, 7]), Hkv=Hkv, d=d,
                    page=page, longest=_spread(rng, 1, 2048))
    return dict(op=op, S=_spread(rng, 1, 256), pages=_spread(rng, 8, (1 << 20) // page // Hkv),
                Hkv=Hkv, d=d, page=page, keep=round(rng.uniform(0.05, 0.95), 2))


def _lens(case):
    """The sequences' lengths: the longest, and where they are ragged the others spread below it,
    one of seven empty."""
    S, longest = case["S"], case["longest"]
    n = np.full(S, longest, np.int64)
    if case.get("ragged", True):
        s = np.arange(S)
        n = 1 + np.floor((longest - 1) * (1.0 - (s * PAIR) % 1.0)).astype(np.int64)
        n[s % 7 == 3] = 0
    return n


# ----------------------------------------------------------------------------
# what a user's program has in hand
# ----------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed) * 7919 + 13)
    st = dict(case)
    op = case["op"]
    if op == "window":
        B, H, Hkv, Lq, Lk, d = (case[x] for x in ("B", "H", "Hkv", "Lq", "Lk", "d"))
        q, k, v = _randn(g, B, H, Lq, d), _randn(g, B, Hkv, Lk, d), _randn(g, B, Hkv, Lk, d)
        lead = _randn(g, B, Hkv, 1, d) * 0.4     # what draws every query to the first tokens
        q += lead.repeat_interleave(H // Hkv, dim=1)
        k[:, :, :case["sinks"]] += 2.0 * lead
        st.update(q=q.bfloat16(), k=k.bfloat16(), v=v.bfloat16(), q_offset=Lk - Lq + case["past"])
        if case["grad"]:
            st.update(do=_randn(g, B, H, Lq, d).bfloat16())
        return st
    if op == "compact":
        return _prepare_compact(st, case, g)
    S, Hkv, d, page = case["S"], case["Hkv"], case["d"], case["page"]
    n = _lens(case)
    fresh = case.get("fresh", 0)
    rows = S * (1 + case.get("ways", 0))
    width = max(1, -(-(int(n.max()) + fresh) // page))
    held = -(-n // page)
    spare = S * (-(-fresh // page) + 1) + rows + 5
    pages = int(held.sum()) + spare
    order = torch.randperm(pages, generator=g, device="cuda")
    table = torch.full((rows, width), -1, dtype=torch.int64, device="cuda")
    slot = torch.arange(width, device="cuda")[None, :]
    held_t = torch.as_tensor(held, device="cuda")
    base = torch.cumsum(held_t, 0) - held_t
    used = slot < held_t[:, None]
    at = torch.where(used, base[:, None] + slot, 0)
    table[:S] = torch.where(used, order[at], -1)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[order[:int(held.sum())]] = 1
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    lens[:S] = torch.as_tensor(n, device="cuda", dtype=torch.int32)
    st.update(table=table.int(), lens=lens, refs=refs, scale_k=None, scale_v=None)
    shape = (pages, Hkv, page, d)
    kc, vc = torch.empty(shape, device="cuda", dtype=torch.bfloat16), torch.empty(
        shape, device="cuda", dtype=torch.bfloat16)
    kc.normal_(generator=g)
    vc.normal_(generator=g)
    if case.get("kv") == "e4m3":
        st.update(scale_k=0.01 + 0.01 * torch.rand(Hkv, generator=g, device="cuda"),
                  scale_v=0.01 + 0.01 * torch.rand(Hkv, generator=g, device="cuda"))
        kc, vc = (torch.div(c, s[None, :, None, None]).clamp_(-448, 448).to(torch.float8_e4m3fn)
                  for c, s in ((kc, st["scale_k"]), (vc, st["scale_v"])))
    st.update(kc=kc, vc=vc)
    if op == "decode":
        st.update(q=_randn(g, S, case["H"], d).bfloat16())
    elif op == "step":
        # sequences take `fresh` new tokens each; every fifth one has none this time
        news = torch.full((S,), fresh, dtype=torch.int32, device="cuda")
        news[4::5] = 0
        cu = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
        cu[1:] = torch.cumsum(news, 0)
        total = fresh * (S - S // 5)
        st.update(news=news, cu=cu, k_new=_randn(g, total, Hkv, d).bfloat16(),
                  v_new=_randn(g, total, Hkv, d).bfloat16())
    else:
        parents = torch.arange(S, dtype=torch.int32, device="cuda").repeat_interleave(case["ways"])
        st.update(parents=parents,
                  children=torch.arange(S, rows, dtype=torch.int32, device="cuda"))
    return st


def _prepare_compact(st, case, g):
    """Sequences that hold `keep` of the pages, scattered; one page in eight is held twice."""
    S, pages, Hkv, d, page = (case[x] for x in ("S", "pages", "Hkv", "d", "page"))
    live = max(1, min(pages, int(pages * case["keep"])))
    width = -(-live // S) + -(-live // 8 // S) + 1
    order = torch.randperm(pages, generator=g, device="cuda")[:live]
    entries = torch.cat([order, order[:live // 8]])
    table = torch.full((S * width,), -1, dtype=torch.int64, device="cuda")
    spots = torch.randperm(S * width, generator=g, device="cuda")[:entries.numel()]
    table[spots] = entries
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs.index_add_(0, entries, torch.ones_like(entries, dtype=torch.int32))
    kc, vc = (torch.empty((pages, Hkv, page, d), device="cuda", dtype=torch.bfloat16)
              for _ in range(2))
    kc.normal_(generator=g)
    vc.normal_(generator=g)
    st.update(table=table.reshape(S, width).int(), refs=refs, kc=kc, vc=vc)
    return st


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(state):
    op = state["op"]
    if op == "window":
        return _window_own(state) if own else _window_plain(state)
    if op == "decode":
        return _decode_own(state) if own else _decode_plain(state)
    if op == "step":
        return _step_own(state) if own else _step_plain(state)
    if op == "fork":
        return _fork_own(state) if own else _fork_plain(state)
    return _compact_own(state) if own else _compact_plain(state)


def _package():
    import block_sparse_softmax_gb300
    return block_sparse_softmax_gb300


def _window_own(st):
    bss = _package()
    opt = dict(sinks=st["sinks"], q_offset=st["q_offset"])
    o, lse = bss.attn_fwd_window(st["q"], st["k"], st["v"], st["window"], **opt)
    if not st["grad"]:
        return o, lse
    dq, dk, dv, _ = bss.attn_bwd_window(st["q"], st["k"], st["v"], o, lse, st["do"], st["window"],
                                        **opt)
    return o, lse, dq, dk, dv


def _softmax(s):
    """Probabilities and log of the normaliser of scores in which masked pairs are -inf; a row with
    no pair left has probabilities 0 and -inf."""
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    lse = torch.where(total > LEAST, top + torch.log(total), torch.full_like(total, -math.inf))
    return p / total.clamp_min(LEAST), lse[..., 0]


def _window_plain(st):
    H, Hkv, d = st["H"], st["Hkv"], st["d"]
    scale = 1.0 / math.sqrt(d)
    B, Lq, Lk = st["B"], st["Lq"], st["Lk"]
    q = st["q"].float().reshape(B, Hkv, H // Hkv, Lq, d)
    k, v = st["k"].float()[:, :, None], st["v"].float()[:, :, None]
    i = torch.arange(Lq, device="cuda")[:, None] + st["q_offset"]
    j = torch.arange(Lk, device="cuda")[None, :]
    hidden = (j > i) | ((i - j >= st["window"]) & (j >= st["sinks"]))
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(hidden, -math.inf)
    p, lse = _softmax(s)
    del s
    o = torch.matmul(p, v)
    out = o.reshape(B, H, Lq, d).bfloat16(), lse.reshape(B, H, Lq)
    if not st["grad"]:
        return out
    do = st["do"].float().reshape(B, Hkv, H // Hkv, Lq, d)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    ds = torch.matmul(do, v.transpose(-1, -2))
    ds = ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq = torch.matmul(ds, k).reshape(B, H, Lq, d)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2)
    return out + (dq.bfloat16(), dk.bfloat16(), dv.bfloat16())


def _decode_own(st):
    return _package().attn_decode_paged(st["q"], st["kc"], st["vc"], st["table"], st["lens"],
                                        window=st["window"], sinks=st["sinks"],
                                        k_scale=st["scale_k"], v_scale=st["scale_v"])


def _decode_plain(st):
    S, H, Hkv, d, page = (st[x] for x in ("S", "H", "Hkv", "d", "page"))
    at = st["table"].clamp_min(0).long()
    width = at.shape[1]

    def gathered(cache, scale):
        x = cache.view(torch.uint8)[at].view(cache.dtype).float()     # [S, width, Hkv, page, d]
        x = x.permute(0, 2, 1, 3, 4).reshape(S, Hkv, width * page, d)
        return x if scale is None else x * scale[None, :, None, None]

    k, v = gathered(st["kc"], st["scale_k"]), gathered(st["vc"], st["scale_v"])
    q = st["q"].float().reshape(S, Hkv, H // Hkv, d)
    j = torch.arange(width * page, device="cuda")[None, :]
    n = st["lens"][:S, None].long()
    seen = j < n
    if st["window"]:
        seen &= (j >= n - st["window"]) | (j < st["sinks"])
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    p, lse = _softmax(s.masked_fill_(~seen[:, None, None, :], -math.inf))
    return torch.matmul(p, v).reshape(S, H, d).bfloat16(), lse.reshape(S, H)


def _values(cache, scale):
    return cache if scale is None else cache.float() * scale[None, :, None, None]


def _step_own(st):
    bss = _package()
    table, lens, refs = st["table"].clone(), st["lens"].clone(), st["refs"].clone()
    if st["window"]:
        bss.attn_kv_evict(table, lens, refs, st["window"], st["sinks"], st["page"])
    start = bss.attn_kv_reserve(table, lens, refs, st["news"], st["page"])
    bss.attn_kv_write(st["k_new"], st["v_new"], st["kc"], st["vc"], table, start, st["cu"],
                      k_scale=st["scale_k"], v_scale=st["scale_v"])
    return table, lens, refs, start, _values(st["kc"], st["scale_k"]), _values(st["vc"],
                                                                             st["scale_v"])


def _step_plain(st):
    page = st["page"]
    table, lens, refs = st["table"].long(), st["lens"].long(), st["refs"].clone()
    slot = torch.arange(table.shape[1], device="cuda")[None, :]
    if st["window"]:
        gone = (table >= 0) & (slot * page >= st["sinks"])
        gone &= (slot + 1) * page <= lens[:, None] - st["window"]
        refs.index_add_(0, table.clamp_min(0).flatten(), -gone.flatten().int())
        table = torch.where(gone, -1, table)
    start, news = lens, st["news"].long()
    lens = lens + news
    before, after = (start + page - 1) // page, (lens + page - 1) // page
    free = torch.argsort((refs > 0).int(), stable=True)
    taken = torch.cumsum(after - before, 0)
    fill = (slot >= before[:, None]) & (slot < after[:, None])
    pick = (taken - (after - before))[:, None] + slot - before[:, None]
    table = torch.where(fill, free[pick.clamp(0, free.numel() - 1)], table)
    refs[free] += (torch.arange(free.numel(), device="cuda") < taken[-1]).int()
    # the sequence of each new token, and its place there
    t = torch.arange(st["k_new"].shape[0], device="cuda")
    s = torch.searchsorted(st["cu"].long(), t, right=True) - 1
    pos = start[s] + t - st["cu"].long()[s]
    at, row = table[s, pos // page], pos % page
    for_k, for_v = st["k_new"], st["v_new"]
    if st["scale_k"] is not None:
        for_k = (for_k.float() / st["scale_k"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        for_v = (for_v.float() / st["scale_v"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    word = torch.uint8 if st["scale_k"] is not None else torch.bfloat16
    st["kc"].view(word)[at, :, row] = for_k.view(word)
    st["vc"].view(word)[at, :, row] = for_v.view(word)
    return table.int(), lens.int(), refs, start.int(), _values(st["kc"], st["scale_k"]), _values(
        st["vc"], st["scale_v"])


def _fork_own(st):
    bss = _package()
    table, lens, refs = st["table"].clone(), st["lens"].clone(), st["refs"].clone()
    src, dst = bss.attn_kv_fork(table, lens, refs, st["parents"], st["children"], st["page"])
    bss.attn_kv_copy_pages(st["kc"], st["vc"], src, dst)
    return table, lens, refs, src, dst, st["kc"], st["vc"]


def _fork_plain(st):
    page = st["page"]
    table, lens, refs = st["table"].long(), st["lens"].long(), st["refs"].clone()
    parents, children = st["parents"].long(), st["children"].long()
    slot = torch.arange(table.shape[1], device="cuda")[None, :]
    n = lens[parents]
    full, part = n // page, (n % page > 0)
    shared = table[parents]
    kept = (slot < full[:, None]) & (shared >= 0)
    free = torch.argsort((refs > 0).int(), stable=True)
    taken = torch.cumsum(part.long(), 0)
    dst = torch.where(part, free[taken - 1], -1)
    src = torch.where(part, shared.gather(1, full.clamp_max(table.shape[1] - 1)[:, None])[:, 0], -1)
    refs.index_add_(0, shared.clamp_min(0).flatten(), kept.flatten().int())
    refs[free] += (torch.arange(free.numel(), device="cuda") < taken[-1]).int()
    rows = torch.where(kept, shared, -1)
    rows = torch.where((slot == full[:, None]) & part[:, None], dst[:, None], rows)
    table[children] = rows
    lens[children] = n
    moved = src >= 0
    st["kc"][dst[moved]] = st["kc"][src[moved]]
    st["vc"][dst[moved]] = st["vc"][src[moved]]
    return table.int(), lens.int(), refs, src.int(), dst.int(), st["kc"], st["vc"]


def _compact_own(st):
    bss = _package()
    table, refs = st["table"].clone(), st["refs"].clone()
    src, dst, count = bss.attn_kv_compact(table, refs)
    bss.attn_kv_copy_pages(st["kc"], st["vc"], src, dst, count)
    return table, refs, src, dst, count, st["kc"], st["vc"]


def _compact_plain(st):
    table, refs = st["table"].long(), st["refs"]
    pages = refs.numel()
    live = refs > 0
    at = torch.arange(pages, device="cuda")
    inside = at < live.sum()
    src, dst = torch.nonzero(live & ~inside)[:, 0], torch.nonzero(~live & inside)[:, 0]
    to = at.clone()
    to[src] = dst
    table = torch.where(table >= 0, to[table.clamp_min(0)], -1)
    refs = torch.zeros_like(refs).index_put((to[live],), refs[live])
    st["kc"][dst] = st["kc"][src]
    st["vc"][dst] = st["vc"][src]
    tail = torch.full((pages - src.numel(),), -1, device="cuda")
    return (table.int(), refs, torch.cat([src, tail]).int(), torch.cat([dst, tail]).int(),
            torch.tensor([src.numel()], device="cuda", dtype=torch.int32), st["kc"], st["vc"])


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def _pairs(case):
    """Allowed (query, key) pairs of one head of a windowed case."""
    pos = np.arange(case["Lq"], dtype=np.int64) + case["Lk"] - case["Lq"] + case["past"]
    upto = np.minimum(pos + 1, case["Lk"])                            # keys not in the future
    low = np.clip(pos + 1 - case["window"], 0, case["Lk"])            # the window's first key
    return int(np.maximum(upto - low, 0).sum() + np.minimum(low, case["sinks"]).sum())


def work(case):
    op = case["op"]
    if op == "window":
        B, H, Hkv, Lq, Lk, d = (case[x] for x in ("B", "H", "Hkv", "Lq", "Lk", "d"))
        rows, keys = B * H * Lq * d, B * Hkv * Lk * d
        pairs = B * H * _pairs(case)
        if not case["grad"]:      # q, k, v in; o and lse out; two products
            return {"bytes": 2 * (2 * rows + 2 * keys) + 4 * B * H * Lq, "flops": 4 * d * pairs}
        # q, k, v, do in; o, lse, dq, dk, dv out; two products and five
        return {"bytes": 2 * (4 * rows + 4 * keys) + 4 * B * H * Lq, "flops": 14 * d * pairs}
    if op == "compact":
        held = min(case["pages"], max(1, int(case["pages"] * case["keep"])))
        width = -(-held // case["S"]) + -(-held // 8 // case["S"]) + 1
        each = 2 * case["Hkv"] * case["page"] * case["d"] * 2         # a page of K and one of V
        moves = held * (1.0 - held / case["pages"])                   # as scattered as these are
        return {"bytes": moves * each * 2 + 8 * case["S"] * width + 16 * case["pages"], "flops": 0}
    n = _lens(case)
    item = 1 if case.get("kv") == "e4m3" else 2
    Hkv, d, page = case["Hkv"], case["d"], case["page"]
    held = int((-(-n // page)).sum())
    if op == "decode":
        seen = n
        if case["window"]:
            seen = np.minimum(n, case["window"]) + np.minimum(
                np.maximum(0, n - case["window"]), case["sinks"])
        seen = int(seen.sum())
        return {"bytes": 2 * seen * Hkv * d * item + case["S"] * case["H"] * (4 * d + 4)
                + 4 * seen // page + 4 * case["S"], "flops": 4 * seen * case["H"] * d}
    if op == "step":
        total = case["fresh"] * (case["S"] - case["S"] // 5)
        return {"bytes": 2 * total * Hkv * d * (2 + item) + 8 * held + 16 * case["S"], "flops": 0}
    parts = int((n % page > 0).sum()) * case["ways"]
    return {"bytes": 4 * parts * Hkv * page * d * 2 + 8 * held * case["ways"], "flops": 0}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "window":
        return _window_exact(case, st)
    if case["op"] == "decode":
        return _decode_exact(case, st)
    return _pages_exact(case, st)


def _attend(q, k, v, seen):
    """softmax over the keys that `seen` allows, row by row, in 64 bits: (p, lse, o)."""
    x = (q @ k.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
    p = torch.where(seen, p, torch.zeros_like(p))
    return p, lse, p @ v


def _window_exact(case, st):
    B, H, Hkv, Lq, Lk, d = (case[x] for x in ("B", "H", "Hkv", "Lq", "Lk", "d"))
    W, sinks, off = case["window"], min(case["sinks"], Lk), st["q_offset"]
    G = H // Hkv
    q, k, v = (st[x].double() for x in "qkv")
    o = torch.zeros(B, H, Lq, d, device="cuda", dtype=torch.float64)
    lse = torch.zeros(B, H, Lq, device="cuda", dtype=torch.float64)
    grads = [torch.zeros_like(t) for t in (q, k, v)]
    rows = 512
    for h in range(H):
        for r in range(0, Lq, rows):
            e = min(Lq, r + rows)
            lo, hi = min(Lk, max(0, r + off - W + 1)), min(Lk, e + off)
            # the sinks below the window's first key, then the window
            keys = torch.cat([torch.arange(min(sinks, lo)), torch.arange(lo, max(lo, hi))]).cuda()
            i = torch.arange(r, e, device="cuda")[:, None] + off
            seen = (keys[None] <= i) & ((keys[None] > i - W) | (keys[None] < sinks))
            kk, vv = k[:, h // G, keys], v[:, h // G, keys]
            p, lse[:, h, r:e], oo = _attend(q[:, h, r:e], kk, vv, seen)
            o[:, h, r:e] = oo
            if case["grad"]:
                do = st["do"][:, h, r:e].double()
                dp = do @ vv.transpose(-1, -2)
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(d)
                grads[0][:, h, r:e] = ds @ kk
                grads[1][:, h // G].index_add_(1, keys, ds.transpose(-1, -2) @ q[:, h, r:e])
                grads[2][:, h // G].index_add_(1, keys, p.transpose(-1, -2) @ do)
    return (o, lse, *grads) if case["grad"] else (o, lse)


def _decode_exact(case, st):
    S, H, Hkv, d = (case[x] for x in ("S", "H", "Hkv", "d"))
    G = H // Hkv
    o = torch.zeros(S, H, d, device="cuda", dtype=torch.float64)
    lse = torch.full((S, H), -math.inf, device="cuda", dtype=torch.float64)
    n = _lens(case)
    for s in range(S):
        length = int(n[s])
        if length == 0:
            continue
        at = st["table"][s, :-(-length // case["page"])].long()

        def lay(cache, scale):
            x = cache.view(torch.uint8)[at].view(cache.dtype).double().transpose(0, 1)
            x = x.reshape(Hkv, -1, d)[:, :length]
            return x if scale is None else x * scale.double()[:, None, None]

        k, v = lay(st["kc"], st["scale_k"]), lay(st["vc"], st["scale_v"])
        j = torch.arange(length, device="cuda")
        seen = torch.ones_like(j, dtype=torch.bool)
        if case["window"]:
            seen = (j >= length - case["window"]) | (j < case["sinks"])
        _, l, x = _attend(st["q"][s].double().reshape(Hkv, G, d), k, v, seen)
        lse[s], o[s] = l.reshape(H), x.reshape(H, d)
    return o, lse


def _pages_exact(case, st):
    """The bookkeeping followed entry by entry on the host; the caches get what it says."""
    op = case["op"]
    table = st["table"].cpu().tolist()
    refs = st["refs"].cpu().tolist()
    page = case["page"]
    kc, vc = st["kc"], st["vc"]

    def lowest_free():
        x = refs.index(0)
        refs[x] = 1
        return x

    whole = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    moves = []
    if op == "compact":
        live = sum(r > 0 for r in refs)
        holes = [x for x in range(live) if refs[x] == 0]
        late = [x for x in range(live, len(refs)) if refs[x] > 0]
        to = dict(zip(late, holes))
        moves = list(zip(late, holes))
        for a, b in moves:
            refs[b], refs[a] = refs[a], 0
        table = [[to.get(e, e) for e in row] for row in table]
        pad = [-1] * (len(refs) - len(moves))
        lists = [whole(late + pad), whole(holes + pad), whole([len(moves)])]
        head = [whole(table), whole(refs)] + lists
    elif op == "fork":
        lens = st["lens"].cpu().tolist()
        src, dst = [], []
        for a, b in zip(st["parents"].cpu().tolist(), st["children"].cpu().tolist()):
            lens[b] = lens[a]
            src.append(-1)
            dst.append(-1)
            for m in range(lens[a] // page):
                table[b][m] = table[a][m]
                refs[table[a][m]] += 1
            if lens[a] % page:
                m = lens[a] // page
                src[-1], dst[-1] = table[a][m], lowest_free()
                table[b][m] = dst[-1]
        moves = [(a, b) for a, b in zip(src, dst) if a >= 0]
        head = [whole(table), whole(lens), whole(refs), whole(src), whole(dst)]
    else:
        lens = st["lens"].cpu().tolist()
        news = st["news"].cpu().tolist()
        if case["window"]:
            for s, row in enumerate(table):
                for m, e in enumerate(row):
                    if e >= 0 and m * page >= case["sinks"] and (
                            m + 1) * page <= lens[s] - case["window"]:
                        refs[e] -= 1
                        row[m] = -1
        start = list(lens)
        places = []
        for s in range(case["S"]):
            for x in range(news[s]):
                if lens[s] % page == 0:
                    table[s][lens[s] // page] = lowest_free()
                places.append((table[s][lens[s] // page], lens[s] % page))
                lens[s] += 1
        head = [whole(table), whole(lens), whole(refs), whole(start)]
        kd, vd = _values(kc, st["scale_k"]).double(), _values(vc, st["scale_v"]).double()
        at = torch.tensor(places, device="cuda").reshape(-1, 2)

        def rounded(x, scale):
            if scale is None:
                return x.double()
            y = (x.float() / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            return (y.float() * scale[:, None]).double()

        kd[at[:, 0], :, at[:, 1]] = rounded(st["k_new"], st["scale_k"])
        vd[at[:, 0], :, at[:, 1]] = rounded(st["v_new"], st["scale_v"])
        return head + [kd, vd]
    if moves:
        a, b = (torch.tensor(x, device="cuda") for x in zip(*moves))
        kc[b], vc[b] = kc[a], vc[a]
    return head + [kc.double(), vc.double()]
