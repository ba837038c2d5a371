"""Serving long sequences over a paged key/value cache, as measured cases.

Operators that read the same cache, with the summary that one of them needs:
  * attention of a chunk of new tokens per sequence (`attn_fwd_paged`): a prompt's next chunk, a few
    draft tokens to verify, or both beside single tokens in one ragged batch; with or without a
    window and sinks, over bf16 or e4m3 pages;
  * the pages' mean keys (`attn_kv_pool`), made when a page is full;
  * for every new token and K/V head the pages that score highest (`attn_select_pages`), and
    attention over these (`attn_decode_selected`).

Each is computed in two ways: by elementary torch operations in 32 bits (`own` False; scores that
decide which pages are taken, and means, in 64), and by the package's entry points (`own` True).
`exact` follows the definitions in 64 bits.
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
        # eight short conversations, five draft tokens each to verify: latency alone counts
        dict(name="chunk-draft-8x5", op="chunk", S=8, H=16, Hkv=4, d=128, page=16, longest=300,
             ragged=False, fresh=5, mixed=False, window=0, sinks=0, kv="bf16"),
        # the next chunk of one prompt, of an odd length
        dict(name="chunk-500-8191", op="chunk", S=1, H=16, Hkv=4, d=128, page=64, longest=8191,
             ragged=False, fresh=500, mixed=False, window=0, sinks=0, kv="bf16"),
        # a serving step: 32 conversations of very different lengths, every fourth in the middle of
        # its prompt, the others with a token each
        dict(name="chunk-mixed-32-8192", op="chunk", S=32, H=16, Hkv=4, d=128, page=64, longest=8192,
             ragged=True, fresh=512, mixed=True, window=0, sinks=0, kv="bf16"),
        # the last chunk of a document of 131071 tokens, one K/V head a query head
        dict(name="chunk-1024-131071", op="chunk", S=1, H=8, Hkv=8, d=128, page=128, longest=131071,
             ragged=False, fresh=1024, mixed=False, window=0, sinks=0, kv="bf16"),
        # four prompts over an 8-bit cache
        dict(name="chunk-e4m3-4x1000-16384", op="chunk", S=4, H=16, Hkv=4, d=128, page=32,
             longest=16384, ragged=False, fresh=1000, mixed=False, window=0, sinks=0, kv="e4m3"),
        # windowed layers of head dimension 64, chunks of six prompts
        dict(name="chunk-window-6x700-d64", op="chunk", S=6, H=16, Hkv=16, d=64, page=16,
             longest=4096, ragged=True, fresh=700, mixed=False, window=1000, sinks=4, kv="bf16"),
        # the mean keys of a prompt's pages
        dict(name="pool-prompt-16384", op="pool", S=1, Hkv=4, d=128, page=64, longest=16384,
             ragged=False, fresh=16384, kv="bf16"),
        # ... of the pages that 256 conversations have filled, a chunk of 64 tokens each
        dict(name="pool-256x64-e4m3", op="pool", S=256, Hkv=4, d=128, page=32, longest=4096,
             ragged=True, fresh=64, kv="e4m3"),
        # one conversation of 8192 tokens that reads 16 of its 128 pages
        dict(name="select-one-8192", op="select", S=1, H=16, Hkv=4, d=128, page=64, longest=8192,
             ragged=False, fresh=1, top=12, local=3, first=1, kv="bf16"),
        # a batch of conversations of very different lengths
        dict(name="select-64-ragged-16384", op="select", S=64, H=16, Hkv=4, d=128, page=64,
             longest=16384, ragged=True, fresh=1, top=28, local=3, first=1, kv="bf16"),
        # two documents of 131071 tokens in small pages, over an 8-bit cache
        dict(name="select-2-131071-e4m3", op="select", S=2, H=8, Hkv=8, d=128, page=16,
             longest=131071, ragged=False, fresh=1, top=256, local=8, first=1, kv="e4m3"),
        # a chunk of 500 tokens of a long prompt, each with pages of its own
        dict(name="select-chunk-500-65535", op="select", S=1, H=16, Hkv=4, d=128, page=64,
             longest=65535, ragged=False, fresh=500, top=28, local=3, first=1, kv="bf16"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "chunk", "select", "select", "select", "pool"])
    d = rng.choice([64, 128, 128])
    H, Hkv = rng.choice([(16, 16), (16, 4), (8, 8), (8, 1), (6, 2), (16, 2), (16, 1)])
    page = rng.choice([16, 32, 64, 128])
    kv = rng.choice(["bf16", "bf16", "e4m3"])
    S = _spread(rng, 1, 64)
    # what all sequences' keys of a head may come to
    longest = _spread(rng, 1, min(131072, max(1, (1 << 27) // (S * Hkv * d))))
    ragged = rng.random() < 0.6
    case = dict(op=op, S=S, H=H, Hkv=Hkv, d=d, page=page, longest=longest, ragged=ragged, kv=kv)
    if op == "chunk":
        case.update(fresh=_spread(rng, 1, min(longest, 2048)), mixed=rng.random() < 0.4)
        case["fresh"] = max(1, min(case["fresh"], int(6e10 // (S * H * d * longest))))
        w = rng.random() < 0.4
        case.update(window=_spread(rng, 1, 4096) if w else 0,
                    sinks=rng.choice([0, 1, 4, 4, 130]) if w else 0)
    elif op == "pool":
        del case["H"]
        case["longest"] = max(longest, page)          # a page at least becomes full
        case.update(fresh=_spread(rng, page, case["longest"]))
    else:
        case.update(fresh=1 if rng.random() < 0.5 else _spread(rng, 1, min(longest, 128)),
                    top=_spread(rng, 1, 64), local=rng.choice([1, 2, 3, 8]),
                    first=rng.choice([0, 1, 1, 2]))
        # keys that the rows read, and the scores of their pages
        read = (case["top"] + case["local"] + case["first"]) * page
        rows = S * case["fresh"] * Hkv
        if rows * read > 1 << 22 or rows * longest // page > 1 << 22:
            case["fresh"] = max(1, min((1 << 22) // (S * Hkv * read),
                                       (1 << 22) // (S * Hkv * max(1, longest // page))))
    return case


def _lens(case):
    """The sequences' lengths: the longest, and where they are ragged the others spread below it,
    one of seven empty."""
    S, longest = case["S"], case["longest"]
    n = np.full(S, longest, np.int64)
    if case["ragged"]:
        s = np.arange(S)
        n = 1 + np.floor((longest - 1) * (1.0 - (s * PAIR) % 1.0)).astype(np.int64)
        n[s % 7 == 3] = 0
    return n


def _news(case):
    """New tokens of each sequence, the last of its length."""
    n = _lens(case)
    want = np.full(case["S"], case["fresh"], np.int64)
    if case.get("mixed"):
        want[np.arange(case["S"]) % 4 != 0] = 1
    return np.minimum(n, want)


# ----------------------------------------------------------------------------
# what a user's program has in hand
# ----------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed) * 6151 + 29)
    st = dict(case)
    S, Hkv, d, page = case["S"], case["Hkv"], case["d"], case["page"]
    n, news = _lens(case), _news(case)
    held = -(-n // page)
    width = max(1, int(held.max()))
    pages = int(held.sum()) + 5
    order = torch.randperm(pages, generator=g, device="cuda")
    slot = torch.arange(width, device="cuda")[None, :]
    held_t = torch.as_tensor(held, device="cuda")
    base = torch.cumsum(held_t, 0) - held_t
    used = slot < held_t[:, None]
    table = torch.where(used, order[torch.where(used, base[:, None] + slot, 0)], -1)
    cu = np.concatenate([[0], np.cumsum(news)])
    total = int(cu[-1])
    shape = (pages, Hkv, page, d)
    kc, vc = torch.empty(shape, device="cuda", dtype=torch.bfloat16), torch.empty(
        shape, device="cuda", dtype=torch.bfloat16)
    kc.normal_(generator=g)
    vc.normal_(generator=g)
    topics = _randn(g, 24, Hkv, d) * 0.5
    if case["op"] == "select":              # a page's keys have something in common
        kc += topics[torch.randint(24, (pages,), generator=g, device="cuda")][:, :, None].bfloat16()
    scale_k = scale_v = None
    if case["kv"] == "e4m3":
        scale_k = 0.01 + 0.01 * torch.rand(Hkv, generator=g, device="cuda")
        scale_v = 0.01 + 0.01 * torch.rand(Hkv, generator=g, device="cuda")
        kc, vc = (torch.div(c, s[None, :, None, None]).clamp_(-448, 448).to(torch.float8_e4m3fn)
                  for c, s in ((kc, scale_k), (vc, scale_v)))
    st.update(table=table.int(), kc=kc, vc=vc, scale_k=scale_k, scale_v=scale_v,
              lens=torch.as_tensor(n, device="cuda", dtype=torch.int32),
              cu=torch.as_tensor(cu, device="cuda", dtype=torch.int32),
              host_lens=n.tolist(), host_news=news.tolist(), host_cu=cu.tolist())
    if case["op"] == "pool":
        st.update(start=torch.as_tensor(n - news, device="cuda", dtype=torch.int32),
                  means=torch.zeros(pages, Hkv, d, device="cuda"))
        del st["vc"]
        return st
    q = _randn(g, total, Hkv, case["H"] // Hkv, d)
    if case["op"] == "select":
        q += topics[torch.randint(24, (total,), generator=g, device="cuda")][:, :, None]
        st.update(means=torch.empty(pages, Hkv, d, device="cuda"))
        for p in range(0, pages, 1024):
            x = _values(kc[p:p + 1024], scale_k)
            st["means"][p:p + 1024] = (x.sum(2) / page).float()
    st.update(q=q.reshape(total, case["H"], d).bfloat16())
    return st


def _values(cache, scale):
    """What a cache's elements stand for, in 64 bits."""
    x = cache.double()
    return x if scale is None else x * scale.double()[None, :, None, None]


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(state):
    op = state["op"]
    if op == "chunk":
        return _chunk_own(state) if own else _chunk_plain(state)
    if op == "pool":
        return _pool_own(state) if own else _pool_plain(state)
    return _select_own(state) if own else _select_plain(state)


def _package():
    import block_sparse_softmax_gb300
    return block_sparse_softmax_gb300


def _chunk_own(st):
    return _package().attn_fwd_paged(st["q"], st["kc"], st["vc"], st["table"], st["lens"], st["cu"],
                                     window=st["window"], sinks=st["sinks"], k_scale=st["scale_k"],
                                     v_scale=st["scale_v"])


def _softmax(s):
    """Probabilities and log of the normaliser of scores in which masked pairs are -inf; a row with
    no pair left has probabilities 0 and -inf."""
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    lse = torch.where(total > LEAST, top + torch.log(total), torch.full_like(total, -math.inf))
    return p / total.clamp_min(LEAST), lse[..., 0]


def _gathered(cache, at, scale):
    """[..., R] pages of a cache as [..., Hkv, R * page, d] in 32 bits."""
    x = cache.view(torch.uint8)[at].view(cache.dtype).float()
    x = x.transpose(-4, -3).flatten(-3, -2)
    return x if scale is None else x * scale[:, None, None]


def _chunk_plain(st):
    H, Hkv, d, page = (st[x] for x in ("H", "Hkv", "d", "page"))
    G = H // Hkv
    o = torch.empty_like(st["q"])
    lse = torch.empty(o.shape[:2], device="cuda")
    groups = {}                       # sequences with as many new tokens go together
    for s, new in enumerate(st["host_news"]):
        if new:
            groups.setdefault(new, []).append(s)
    for new, seqs in groups.items():
        longest = max(st["host_lens"][s] for s in seqs)
        at = st["table"][seqs, :-(-longest // page)].clamp_min(0).long()
        k, v = _gathered(st["kc"], at, st["scale_k"]), _gathered(st["vc"], at, st["scale_v"])
        rows = torch.tensor([[st["host_cu"][s] + i for i in range(new)] for s in seqs], device="cuda")
        q = st["q"][rows].float().reshape(len(seqs), new, Hkv, G, d).permute(0, 2, 3, 1, 4)
        n = st["lens"][seqs].long()
        pos = (n[:, None] - new + torch.arange(new, device="cuda"))[:, :, None]      # [seqs, new, 1]
        j = torch.arange(at.shape[1] * page, device="cuda")
        seen = j <= pos
        if st["window"]:
            seen &= (j > pos - st["window"]) | (j < st["sinks"])
        s = torch.matmul(q.reshape(len(seqs), Hkv, G * new, d), k.transpose(-1, -2))
        s = s.mul_(1.0 / math.sqrt(d)).view(len(seqs), Hkv, G, new, -1)
        p, l = _softmax(s.masked_fill_(~seen[:, None, None], -math.inf))
        del s
        y = torch.matmul(p.view(len(seqs), Hkv, G * new, -1), v).view(len(seqs), Hkv, G, new, d)
        o[rows] = y.permute(0, 3, 1, 2, 4).reshape(len(seqs), new, H, d).bfloat16()
        lse[rows] = l.permute(0, 3, 1, 2).reshape(len(seqs), new, H)
    return o, lse


def _pool_own(st):
    _package().attn_kv_pool(st["kc"], st["means"], st["table"], st["start"], st["lens"],
                            k_scale=st["scale_k"])
    return st["means"]


def _pool_plain(st):
    page = st["page"]
    slot = torch.arange(st["table"].shape[1], device="cuda")[None, :]
    full = (slot >= st["start"][:, None] // page) & (slot < st["lens"][:, None] // page)
    at = st["table"][full].long()
    x = st["kc"].view(torch.uint8)[at].view(st["kc"].dtype)
    st["means"][at] = (_values(x, st["scale_k"]).sum(2) / page).float()
    return st["means"]


def _select_own(st):
    bss = _package()
    pages, lens = bss.attn_select_pages(st["q"], st["means"], st["table"], st["lens"], st["cu"],
                                        st["top"], st["page"], local_pages=st["local"],
                                        first_pages=st["first"])
    o, lse = bss.attn_decode_selected(st["q"], st["kc"], st["vc"], pages, lens,
                                      k_scale=st["scale_k"], v_scale=st["scale_v"])
    return pages, lens, o, lse


def _select_plain(st):
    S, H, Hkv, d, page = (st[x] for x in ("S", "H", "Hkv", "d", "page"))
    top, local, first, fresh = (st[x] for x in ("top", "local", "first", "fresh"))
    T, most = st["q"].shape[0], first + local + top
    if T == 0:
        return (torch.empty(0, Hkv, most, device="cuda", dtype=torch.int32),
                torch.empty(0, device="cuda", dtype=torch.int32), torch.empty_like(st["q"]),
                torch.empty(0, H, device="cuda"))
    # a row's sequence and place; the scores of every page of its sequence's, in 64 bits
    rows = torch.arange(T, device="cuda")
    s = torch.searchsorted(st["cu"].long(), rows, right=True) - 1
    n = st["lens"].long()[s] - st["cu"].long()[s + 1] + rows + 1      # tokens it sees
    qsum = st["q"].double().reshape(T, Hkv, H // Hkv, d).sum(2)
    table = st["table"].long()
    width = table.shape[1]
    padded = torch.zeros(S, fresh, Hkv, d, device="cuda", dtype=torch.float64)
    padded[s, rows - st["cu"].long()[s]] = qsum
    means = st["means"].double()[table.clamp_min(0)]                  # [S, width, Hkv, d]
    score = torch.einsum("sihd,smhd->sihm", padded, means)[s, rows - st["cu"].long()[s]]
    slot = torch.arange(width, device="cuda")[None, :]
    held = (n[:, None] + page - 1) // page
    own_page = (slot < held) & ((slot < first) | (slot >= held - local)) & (table[s] >= 0)
    other = (slot < held) & ~own_page & (table[s] >= 0)
    score = score.masked_fill(~other[:, None], -math.inf)
    rank = torch.argsort(torch.argsort(score, dim=-1, descending=True, stable=True), dim=-1)
    taken = own_page[:, None] | (other[:, None] & (rank < top))
    # the pages taken, in ascending order of their places
    place = torch.where(taken, slot[None], width)
    place = torch.sort(place, dim=-1).values[..., :most]
    if place.shape[-1] < most:
        place = torch.cat([place, place.new_full((T, Hkv, most - place.shape[-1]), width)], -1)
    some = place < width
    pages = torch.where(some, table[s][:, None].expand(T, Hkv, width).gather(
        2, place.clamp_max(width - 1)), -1)
    lens = (some[:, 0].sum(-1) - 1) * page + n - (held[:, 0] - 1) * page
    o = torch.empty_like(st["q"])
    lse = torch.empty(T, H, device="cuda")
    chunk = max(1, (1 << 28) // (Hkv * most * page * d))
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    for r in range(0, T, chunk):
        at = pages[r:r + chunk].clamp_min(0)
        k, v = (c.view(torch.uint8)[at, head].view(c.dtype).float().flatten(2, 3)
                for c in (st["kc"], st["vc"]))
        if st["scale_k"] is not None:
            k, v = k * st["scale_k"][:, None, None], v * st["scale_v"][:, None, None]
        q = st["q"][r:r + chunk].float().reshape(-1, Hkv, H // Hkv, d)
        x = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
        seen = torch.arange(most * page, device="cuda") < lens[r:r + chunk, None]
        p, l = _softmax(x.masked_fill_(~seen[:, None, None], -math.inf))
        o[r:r + chunk] = torch.matmul(p, v).reshape(-1, H, d).bfloat16()
        lse[r:r + chunk] = l.reshape(-1, H)
    return pages.int(), lens.int(), o, lse


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    n, news = _lens(case), _news(case)
    Hkv, d, page = case["Hkv"], case["d"], case["page"]
    item = 1 if case["kv"] == "e4m3" else 2
    if case["op"] == "pool":
        full = int((n // page - (n - news) // page).sum())
        return {"bytes": full * Hkv * d * (page * item + 4) + 4 * full + 8 * case["S"],
                "flops": full * Hkv * d * page}
    H, total = case["H"], int(news.sum())
    ends = total * H * (4 * d + 4)                                    # q in, o and lse out
    if case["op"] == "select":
        # the mean keys of every sequence's pages, once; the pages taken, for each row by itself
        # (a sequence's rows may share them: no more than it holds)
        most = case["first"] + case["local"] + case["top"]
        read = int(sum(min(int(x), int(w) * most * page) for x, w in zip(n, news)))
        pairs = int(sum(min(int(x), most * page) * int(w) for x, w in zip(n, news)))
        held = int((-(-n // page) * (news > 0)).sum())
        scored = int((-(-n // page) * news).sum())
        return {"bytes": 2 * read * Hkv * d * item + 4 * held * (Hkv * d + 1) + ends
                + 4 * total * (Hkv * most + 1),
                "flops": 4 * pairs * H * d + 2 * scored * Hkv * d}
    pairs = keys = 0
    W, sinks = case["window"], case["sinks"]
    for x, w in zip(n.tolist(), news.tolist()):
        if not w:
            continue
        pos = np.arange(x - w, x, dtype=np.int64)
        low = np.maximum(pos + 1 - W, 0) if W else np.zeros_like(pos)
        pairs += int((pos + 1 - low + np.minimum(low, sinks)).sum())
        keys += int(x - low[0] + min(low[0], sinks))
    return {"bytes": 2 * keys * Hkv * d * item + ends + 4 * keys // page + 8 * case["S"],
            "flops": 4 * pairs * H * d}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "pool":
        return _pool_exact(case, st)
    return _chunk_exact(case, st) if case["op"] == "chunk" else _select_exact(case, st)


def _attend(q, k, v, seen=None):
    """Softmax attention over the keys that `seen` allows (every row sees one): (o, lse)."""
    x = (q @ k.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    if seen is not None:
        x = torch.where(seen, x, torch.full_like(x, -math.inf))
    lse = torch.logsumexp(x, -1)
    return torch.exp(x - lse[..., None]) @ v, lse


def _chunk_exact(case, st):
    H, Hkv, d, page = (case[x] for x in ("H", "Hkv", "d", "page"))
    G = H // Hkv
    o = torch.zeros(st["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.zeros(o.shape[:2], device="cuda", dtype=torch.float64)
    rows = 256
    for s, (n, new) in enumerate(zip(st["host_lens"], st["host_news"])):
        at = st["table"][s, :-(-n // page)].long()
        for h in range(Hkv if new else 0):
            k, v = (c[at, h].double().reshape(-1, d)[:n] * (1.0 if f is None else f[h].double())
                    for c, f in ((st["kc"], st["scale_k"]), (st["vc"], st["scale_v"])))
            for r in range(0, new, rows):
                e = min(new, r + rows)
                i = torch.arange(n - new + r, n - new + e, device="cuda")[:, None]
                lo = max(0, n - new + r + 1 - case["window"]) if case["window"] else 0
                keys = torch.cat([torch.arange(min(case["sinks"], lo), device="cuda"),
                                  torch.arange(lo, n - new + e, device="cuda")])
                seen = keys[None] <= i
                if case["window"]:
                    seen &= (i - keys[None] < case["window"]) | (keys[None] < case["sinks"])
                a, b = st["host_cu"][s] + r, st["host_cu"][s] + e
                q = st["q"][a:b, h * G:(h + 1) * G].double().transpose(0, 1)
                y, l = _attend(q, k[keys], v[keys], seen)
                o[a:b, h * G:(h + 1) * G] = y.transpose(0, 1)
                lse[a:b, h * G:(h + 1) * G] = l.transpose(0, 1)
    return o, lse


def _pool_exact(case, st):
    page = case["page"]
    out = st["means"].double()
    for s, (n, new) in enumerate(zip(st["host_lens"], st["host_news"])):
        for m in range((n - new) // page, n // page):
            x = st["table"][s, m]
            out[x] = _values(st["kc"][x][None], st["scale_k"])[0].mean(1)
    return out


def _select_exact(case, st):
    H, Hkv, d, page = (case[x] for x in ("H", "Hkv", "d", "page"))
    G, most = H // Hkv, case["first"] + case["local"] + case["top"]
    T = st["q"].shape[0]
    pages = np.full((T, Hkv, most), -1, np.int64)
    lens = np.zeros(T, np.int64)
    o = torch.zeros(st["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.zeros(T, H, device="cuda", dtype=torch.float64)
    host = st["table"].cpu().numpy()
    for s, (n, new) in enumerate(zip(st["host_lens"], st["host_news"])):
        if not new:
            continue
        held = -(-n // page)
        means = st["means"][st["table"][s, :held].long()].double().cpu().numpy()
        a = st["host_cu"][s]
        q = st["q"][a:a + new].double().cpu().numpy().reshape(new, Hkv, G, d)
        for h in range(Hkv):
            total = q[:, h].sum(1) @ means[:, h].T                    # [new, held]
            for i in range(new):
                sees = n - new + i + 1
                mine = -(-sees // page)
                kept = [m for m in range(mine) if m < case["first"] or m >= mine - case["local"]]
                rest = [m for m in range(mine) if m not in set(kept)] if mine > len(kept) else []
                rest.sort(key=lambda m: (-total[i, m], m))
                kept = sorted(kept + rest[:case["top"]])
                pages[a + i, h, :len(kept)] = host[s, kept]
                lens[a + i] = sees - (mine - len(kept)) * page
                at = torch.as_tensor(host[s, kept], device="cuda").long()
                k, v = (c[at, h].double().reshape(-1, d)[:lens[a + i]] *
                        (1.0 if f is None else f[h].double())
                        for c, f in ((st["kc"], st["scale_k"]), (st["vc"], st["scale_v"])))
                o[a + i, h * G:(h + 1) * G], lse[a + i, h * G:(h + 1) * G] = _attend(
                    st["q"][a + i, h * G:(h + 1) * G].double(), k, v)
    return torch.as_tensor(pages).int(), torch.as_tensor(lens).int(), o, lse
