"""The paged key/value cache on the GPU: attention of one new token per sequence against its
definition in 64 bits (bounds of `oracle/window.py`), and the pages' bookkeeping, writes and copies
against `oracle/pages.py`, number by number."""
import math
import random

import pytest
import torch

from oracle import window as ref
from oracle.pages import Pages

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def bss():
    import block_sparse_softmax_gb300 as m
    m.library()
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Cache:
    """A filled cache: lengths as given, pages in a random order, garbage (NaN) wherever no token
    lies.  `inter`: K and V pages interleaved in one tensor."""

    def __init__(self, lens, Hkv, d, page, seed, e4m3=False, inter=False, extra=3, window=0, sinks=0):
        g = torch.Generator("cuda").manual_seed(seed)
        S = len(lens)
        held = [-(-max(0, n) // page) for n in lens]
        P, M = sum(held) + extra, max(1, max(held)) + 1
        order = torch.randperm(P, generator=g, device="cuda").tolist()
        both = torch.full((P, 2, Hkv, page, d), float("nan"), device="cuda")
        self.k64 = [torch.randn(Hkv, n, d, generator=g, device="cuda") for n in lens]
        self.v64 = [torch.randn(Hkv, n, d, generator=g, device="cuda") for n in lens]
        self.k_scale = self.v_scale = None
        if e4m3:
            self.k_scale = 0.01 + 0.02 * torch.rand(Hkv, generator=g, device="cuda")
            self.v_scale = 0.01 + 0.02 * torch.rand(Hkv, generator=g, device="cuda")

        def held_as(x, scale):          # the values the cache holds, and what they stand for
            if scale is None:
                return x.bfloat16().float(), x.bfloat16().double()
            y = (x / scale[:, None, None]).clamp(-448, 448).to(E4M3).float()
            return y, y.double() * scale.double()[:, None, None]

        self.table = torch.full((S, M), -1, dtype=torch.int32, device="cuda")
        for s, n in enumerate(lens):
            kx, self.k64[s] = held_as(self.k64[s], self.k_scale)
            vx, self.v64[s] = held_as(self.v64[s], self.v_scale)
            for m in range(held[s]):
                x = order.pop()
                a, e = m * page, min(n, (m + 1) * page)
                # a page that nobody sees any more is not even in the table
                if window and e <= n - window and a >= sinks:
                    continue
                self.table[s, m] = x
                both[x, 0, :, :e - a] = kx[:, a:e]
                both[x, 1, :, :e - a] = vx[:, a:e]
                for j in range(a, e):
                    if window and j < n - window and j >= sinks:
                        both[x, :, :, j - a] = float("nan")
        kind = E4M3 if e4m3 else torch.bfloat16
        if inter:
            both = both.to(kind)
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = both[:, 0].to(kind).contiguous(), both[:, 1].to(kind).contiguous()
        self.lens = ints(lens)


def check_decode(bss, c, q, lens, window, sinks, **kw):
    S, H, d = q.shape
    scale = 1.0 / math.sqrt(d)
    o, lse = bss.attn_decode_paged(q, c.k, c.v, c.table, c.lens, window=window, sinks=sinks,
                                   k_scale=c.k_scale, v_scale=c.v_scale, **kw)
    torch.cuda.synchronize()
    assert bss.attn_poll_status() == 0
    for s, n in enumerate(lens):
        if n == 0:
            assert torch.all(o[s] == 0) and torch.all(torch.isneginf(lse[s]))
            continue
        mask = ref.window_mask(1, n, window or n, sinks, n - 1, 0, "cuda")
        args = q[s].reshape(1, H, 1, d), c.k64[s][None], c.v64[s][None], mask, scale
        O, L, _ = ref.forward(*args)
        bo, bl = ref.forward_bounds(*args)
        off = (o[s].double() - O[0, :, 0]).abs()
        assert (off <= bo[0, :, 0]).all(), (s, n, (off / bo[0, :, 0]).max())
        off = (lse[s].double() - L[0, :, 0]).abs()
        assert (off <= bl[0, :, 0]).all(), (s, n, (off / bl[0, :, 0]).max())
    return o, lse


CASES = [
    # lens, H, Hkv, d, page, window, sinks
    ([1], 1, 1, 128, 16, 0, 0),
    ([300], 16, 4, 128, 16, 0, 0),
    ([0, 1, 15, 16, 17, 63, 64, 65, 0, 128, 200], 8, 2, 128, 16, 0, 0),
    ([0, 0, 0], 4, 4, 64, 32, 0, 0),
    ([5, 1000, 33, 257, 0, 64], 6, 2, 64, 64, 0, 0),
    ([777, 12, 2049], 16, 1, 128, 128, 0, 0),      # 16 query heads on one K/V head
    ([500, 31, 1025], 20, 1, 64, 32, 0, 0),        # ... 20: two groups of rows
    ([130, 70], 66, 2, 128, 16, 0, 0),             # ... 33
    ([4000, 1, 2600], 8, 8, 64, 1024, 0, 0),
    ([20011], 2, 1, 128, 32, 0, 0),                # one sequence over every CTA
    ([1000, 40, 3, 0, 999], 8, 2, 128, 16, 100, 4),
    ([1000, 40, 3, 0, 999], 8, 2, 64, 64, 1, 0),   # each token sees itself
    ([1000, 40, 3, 0, 999], 16, 2, 128, 32, 37, 70),   # sinks past a page
    ([600, 601, 615, 616], 4, 4, 64, 16, 600, 1),  # the window just falls behind
    ([900, 17], 9, 3, 128, 64, 10 ** 12, 10 ** 12),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,H,Hkv,d,page,window,sinks", CASES)
def test_decode(bss, lens, H, Hkv, d, page, window, sinks, e4m3):
    c = Cache(lens, Hkv, d, page, sum(lens) + H + page, e4m3, window=window, sinks=sinks)
    g = torch.Generator("cuda").manual_seed(H + len(lens))
    q = torch.randn(len(lens), H, d, generator=g, device="cuda").bfloat16()
    # a table with little room takes a block per K/V head, a wide one shares all steps evenly
    for columns in (0, 1100 // page):
        c.table = torch.cat([c.table, ints([[-1] * columns] * len(lens))], 1)
        a = check_decode(bss, c, q, lens, window, sinks)
        b = check_decode(bss, c, q, lens, window, sinks)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_of_many_sequences(bss):
    rng = random.Random(5)
    lens = [rng.choice([0, 1, 7, 64, rng.randint(1, 500)]) for _ in range(300)]
    c = Cache(lens, 2, 64, 16, 9)
    q = torch.randn(300, 4, 64, device="cuda").bfloat16()
    check_decode(bss, c, q, lens, 0, 0)


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_takes_strided_queries_and_interleaved_caches(bss, e4m3):
    lens = [70, 0, 333, 18]
    c = Cache(lens, 2, 128, 32, 3, e4m3, inter=True)
    qkv = torch.randn(4, 8 + 2 + 2, 128, device="cuda").bfloat16()
    check_decode(bss, c, qkv[:, :8], lens, 0, 0)


def random_pages(rng, S, M, P, page, steps=12):
    """A state that calls have led to, with shared and evicted pages, beside its host double."""
    h = Pages(S, M, P, page)
    for _ in range(steps):
        x = rng.random()
        if x < 0.6:
            h.reserve([rng.choice([0, 1, rng.randint(0, 2 * page)]) for _ in range(S)])
        elif x < 0.75:
            empty = [s for s in range(S) if h.lens[s] == 0]
            full = [s for s in range(S) if h.lens[s]]
            if empty and full:
                children = rng.sample(empty, min(len(empty), 3))
                h.fork([rng.choice(full) for _ in children], children)
        elif x < 0.9:
            h.free([rng.randrange(S)])
        else:
            h.evict(2 * page, 1)
    return h


def on_gpu(h):
    return ints(h.table), ints(h.lens), ints(h.refs)


def same(h, table, lens, refs):
    assert table.tolist() == h.table
    assert lens.tolist() == h.lens
    assert refs.tolist() == h.refs


@pytest.mark.parametrize("seed", range(8))
def test_bookkeeping_follows_the_host(bss, seed):
    rng = random.Random(seed)
    S, M, page = rng.choice([(1, 4, 16), (9, 20, 16), (40, 33, 32)])
    P = rng.choice([S * 3, S * 6, 1500])
    h = random_pages(rng, S, M, P, page)
    t, n, r = on_gpu(h)
    for _ in range(25):
        x = rng.random()
        if x < 0.45:
            new = [rng.choice([0, 1, rng.randint(0, 3 * page)]) for _ in range(S)]
            want = h.reserve(new)
            start = bss.attn_kv_reserve(t, n, r, ints(new), page)
            assert start.tolist() == (want if want is not None else [-1] * S)
            assert (bss.attn_poll_status() == 0) == (want is not None)
        elif x < 0.65:
            empty = [s for s in range(S) if h.lens[s] == 0]
            rest = [s for s in range(S) if h.lens[s]] or [s for s in range(S) if s not in empty[:1]]
            children = rng.sample(empty, min(len(empty), rng.randint(1, 4)))
            rest = [s for s in rest if s not in children]
            if not children or not rest:
                continue
            parents = [rng.choice(rest) for _ in children]
            want = h.fork(parents, children)
            src, dst = bss.attn_kv_fork(t, n, r, ints(parents), ints(children), page)
            none = [-1] * len(children)
            assert (src.tolist(), dst.tolist()) == (want if want is not None else (none, none))
            assert bss.attn_poll_status() == (0 if want is not None else bss.ERR_NO_PAGES)
        elif x < 0.8:
            seqs = [rng.randrange(S) for _ in range(rng.randint(1, 4))]
            seqs.append(seqs[0])                       # listed twice: freed once
            h.free(seqs)
            bss.attn_kv_free(t, n, r, ints(seqs), page)
            assert bss.attn_poll_status() == 0
        elif x < 0.9:
            w, k = rng.randint(1, 4 * page), rng.choice([0, 1, 4, page + 1])
            h.evict(w, k)
            bss.attn_kv_evict(t, n, r, w, k, page)
            assert bss.attn_poll_status() == 0
        else:
            src, dst = h.compact()
            a, b, count = bss.attn_kv_compact(t, r)
            assert count.tolist() == [len(src)]
            tail = [-1] * (P - len(src))
            assert a.tolist() == src + tail and b.tolist() == dst + tail
            assert bss.attn_poll_status() == 0
        same(h, t, n, r)


@pytest.mark.parametrize("e4m3,Hkv,d,page", [(False, 2, 128, 16), (False, 3, 64, 64),
                                             (True, 2, 64, 16), (True, 1, 128, 128)])
def test_write_and_copy(bss, e4m3, Hkv, d, page):
    rng = random.Random(page + d)
    h = random_pages(rng, 7, 12, 60, page)
    t, n, r = on_gpu(h)
    kind, word = (E4M3, torch.uint8) if e4m3 else (torch.bfloat16, torch.int16)
    both = torch.randint(-100, 100, (60, 2, Hkv, page, d), device="cuda").to(kind)
    scales = [0.01 + torch.rand(Hkv, device="cuda") for _ in range(2)] if e4m3 else [None, None]
    new = [rng.choice([0, 1, rng.randint(0, page)]) for _ in range(7)]
    start = bss.attn_kv_reserve(t, n, r, ints(new), page)
    assert h.reserve(new) == start.tolist()
    cu = [2]                                           # rows before and behind them are left out
    for x in new:
        cu.append(cu[-1] + x)
    total = cu[-1] + 5
    qkv = 30 * torch.randn(total, 3 * Hkv, d, device="cuda").bfloat16()
    qkv[cu[0], Hkv:] = float("nan")                    # a NaN stays one, and
    qkv[cu[0] + 1:cu[0] + 2, Hkv:] = float("inf")      # in e4m3 infinity is 448
    k_new, v_new = qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]
    want = both.clone()
    for s, x in enumerate(new):
        for i in range(x):
            pos = start.tolist()[s] + i
            at = h.table[s][pos // page]
            for j, (src, scale) in enumerate(zip((k_new, v_new), scales)):
                row = src[cu[s] + i]
                if e4m3:
                    row = (row.float() / scale[:, None]).clamp(-448, 448).to(E4M3)
                want.view(word)[at, j, :, pos % page] = row.contiguous().view(word)
    bss.attn_kv_write(k_new, v_new, both[:, 0], both[:, 1], t, start, ints(cu), k_scale=scales[0],
                      v_scale=scales[1])
    assert bss.attn_poll_status() == 0
    assert torch.equal(both.view(word), want.view(word))
    # copies: pairs, none, and a count that cuts the list
    src, dst = [3, -1, 7, 3, 9], [50, -1, 51, 52, 53]
    for count in (None, 4):
        for a, b in list(zip(src, dst))[:count]:
            if a >= 0:
                want.view(word)[b] = want.view(word)[a]
        bss.attn_kv_copy_pages(both[:, 0], both[:, 1], ints(src), ints(dst),
                               None if count is None else ints([count]))
        assert bss.attn_poll_status() == 0
        assert torch.equal(both.view(word), want.view(word))
        both.view(word)[53] = 0
        want.view(word)[53] = 0


def test_serving_run(bss):
    """Prompts through the windowed forward, then decoding steps over pages with eviction, forks
    and a compaction in between: every token's output as the windowed forward gives it for the
    whole sequence."""
    g = torch.Generator("cuda").manual_seed(11)
    H, Hkv, d, page, window, sinks, rows = 4, 2, 64, 16, 40, 3, 6
    prompts, steps = [70, 5, 33], 60
    P, M = 60, 12
    table, lens, refs = ints([[-1] * M] * rows), ints([0] * rows), ints([0] * P)
    kc, vc = (torch.full((P, Hkv, page, d), float("nan"), device="cuda").bfloat16() for _ in range(2))
    seqs = {}                                          # row -> (q, k, v) of its tokens so far

    def draw(n):
        return [torch.randn(x, n, d, generator=g, device="cuda").bfloat16() for x in (H, Hkv, Hkv)]

    for s, n in enumerate(prompts):
        seqs[s] = draw(n)

    def put(news):
        """The newest news[s] tokens of every row into the cache."""
        cu = [0]
        for x in news:
            cu.append(cu[-1] + x)
        k_new = torch.cat([seqs[s][1][:, -x:].transpose(0, 1) for s, x in enumerate(news) if x])
        v_new = torch.cat([seqs[s][2][:, -x:].transpose(0, 1) for s, x in enumerate(news) if x])
        start = bss.attn_kv_reserve(table, lens, refs, ints(news), page)
        bss.attn_kv_write(k_new.contiguous(), v_new.contiguous(), kc, vc, table, start, ints(cu))

    put(prompts + [0] * (rows - 3))
    for step in range(steps):
        if step == 20:
            src, dst = bss.attn_kv_fork(table, lens, refs, ints([0, 0]), ints([3, 5]), page)
            bss.attn_kv_copy_pages(kc, vc, src, dst)
            seqs[3], seqs[5] = [x.clone() for x in seqs[0]], [x.clone() for x in seqs[0]]
        if step == 30:
            bss.attn_kv_free(table, lens, refs, ints([0]), page)
            del seqs[0]
        if step in (35, 50):
            src, dst, count = bss.attn_kv_compact(table, refs)
            bss.attn_kv_copy_pages(kc, vc, src, dst, count)
            live = int((refs > 0).sum())
            assert torch.all(refs[:live] > 0)
        bss.attn_kv_evict(table, lens, refs, window, sinks, page)
        for s in seqs:
            seqs[s] = [torch.cat([a, b], 1) for a, b in zip(seqs[s], draw(1))]
        put([1 if s in seqs else 0 for s in range(rows)])
        q = torch.zeros(rows, H, d, device="cuda").bfloat16()
        for s in seqs:
            q[s] = seqs[s][0][:, -1]
        o, lse = bss.attn_decode_paged(q, kc, vc, table, lens, window=window, sinks=sinks)
        assert bss.attn_poll_status() == 0
        for s in range(rows):
            if s not in seqs:
                assert torch.all(o[s] == 0)
                continue
            n = seqs[s][0].shape[1]
            assert int(lens[s]) == n
            args = [x[None] for x in seqs[s]]
            mask = ref.window_mask(1, n, window, sinks, n - 1, 0, "cuda")
            O, L, _ = ref.forward(args[0][:, :, -1:], *args[1:], mask, d ** -0.5)
            bo, bl = ref.forward_bounds(args[0][:, :, -1:], *args[1:], mask, d ** -0.5)
            assert ((o[s].double() - O[0, :, 0]).abs() <= bo[0, :, 0]).all(), (step, s)
            assert ((lse[s].double() - L[0, :, 0]).abs() <= bl[0, :, 0]).all()
            if step == steps - 1:
                whole, _ = bss.attn_fwd_window(*[x.contiguous() for x in args], window, sinks=sinks)
                assert ((whole[0, :, -1].double() - O[0, :, 0]).abs() <= bo[0, :, 0]).all()
    held = sum(len({int(x) for x in table[s] if x >= 0}) for s in seqs)
    assert held <= 5 * (-(-window // page) + 2)        # memory stays bounded by window and sinks


def test_decode_leaves_out_bad_pages(bss):
    """A page out of range and a length past the table are reported, and nothing is read there."""
    lens = [100, 40, 64]
    c = Cache(lens, 2, 64, 16, 21)
    q = torch.randn(3, 4, 64, device="cuda").bfloat16()
    good, _ = bss.attn_decode_paged(q, c.k, c.v, c.table, c.lens)
    assert bss.attn_poll_status() == 0
    c.table[0, 2] = c.k.shape[0] + 5                 # tokens 32 .. 47 of sequence 0
    o, lse = bss.attn_decode_paged(q, c.k, c.v, c.table, c.lens)
    assert bss.attn_poll_status() == bss.ERR_BAD_PAGES
    assert torch.equal(o[1:], good[1:])
    mask = torch.ones(1, 100, dtype=torch.bool, device="cuda")
    mask[:, 32:48] = False
    args = q[0].reshape(1, 4, 1, 64), c.k64[0][None], c.v64[0][None], mask, 0.125
    assert ((o[0].double() - ref.forward(*args)[0][0, :, 0]).abs() <= ref.forward_bounds(*args)[0][0, :, 0]).all()
    c.table[0, 2] = -7
    bss.attn_decode_paged(q, c.k, c.v, c.table, c.lens)
    assert bss.attn_poll_status() == bss.ERR_BAD_PAGES
    c = Cache(lens, 2, 64, 16, 21)
    c.lens[1] = 10 ** 6
    o, _ = bss.attn_decode_paged(q, c.k, c.v, c.table, c.lens)
    assert bss.attn_poll_status() == bss.ERR_BAD_PAGES
    assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])
    c.lens[1] = -3
    o, lse = bss.attn_decode_paged(q, c.k, c.v, c.table, c.lens)
    assert bss.attn_poll_status() == bss.ERR_BAD_PAGES
    assert torch.all(o[1] == 0) and torch.all(torch.isneginf(lse[1]))


def test_decode_of_the_most_sequences(bss):
    """65536 rows, one in nine with tokens; the answer of each is its own."""
    S = 65536
    lens = torch.zeros(S, dtype=torch.int32)
    lens[::9] = torch.arange(len(range(0, S, 9)), dtype=torch.int32) % 40
    held = (lens + 15) // 16
    table = torch.full((S, 3), -1, dtype=torch.int32)
    at = 0
    base = torch.cumsum(held, 0) - held
    for m in range(3):
        table[:, m] = torch.where(held > m, base + m, -1)
    at = int(held.sum())
    k, v = (torch.randn(at, 1, 16, 64, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(S, 1, 64, device="cuda").bfloat16()
    o, lse = bss.attn_decode_paged(q, k, v, table.cuda(), lens.cuda())
    assert bss.attn_poll_status() == 0
    empty = lens.cuda() == 0
    assert torch.all(o[empty] == 0) and torch.all(torch.isneginf(lse[empty]))
    for s in list(range(0, 900, 9)) + [S - 7, S // 2 // 9 * 9]:
        n = int(lens[s])
        if n == 0:
            continue
        kk, vv = (x[table[s, :int(held[s])].long().cuda()].transpose(0, 1).reshape(1, -1, 64)[:, :n] for x in (k, v))
        mask = torch.ones(1, n, dtype=torch.bool, device="cuda")
        args = q[s].reshape(1, 1, 1, 64), kk[None], vv[None], mask, 0.125
        assert ((o[s].double() - ref.forward(*args)[0][0, :, 0]).abs() <= ref.forward_bounds(*args)[0][0, :, 0]).all(), s


def test_decode_with_far_pages(bss):
    """Offsets past 32 bits: a cache of over 2^32 elements whose last pages are in use."""
    page, Hkv, d = 1024, 8, 128
    P = (1 << 32) // (page * Hkv * d) + 3
    k = torch.empty(P, Hkv, page, d, device="cuda", dtype=torch.bfloat16)
    v = torch.empty_like(k)
    last = [P - 1, 0, P - 2]
    for t in (k, v):
        t[last] = torch.randn(3, Hkv, page, d, device="cuda").bfloat16()
    table, lens = ints([[P - 1, 0, P - 2]]), ints([2900])
    q = torch.randn(1, 8, d, device="cuda").bfloat16()
    o, _ = bss.attn_decode_paged(q, k, v, table, lens)
    bss.attn_kv_copy_pages(k, v, ints([P - 1]), ints([P - 3]))
    new = torch.randn(1, Hkv, d, device="cuda").bfloat16()
    bss.attn_kv_write(new, new, k, v, table, ints([2900]), ints([0, 1]))
    assert bss.attn_poll_status() == 0
    assert torch.equal(k[P - 3], k[P - 1]) and torch.equal(v[P - 3], v[P - 1])
    assert torch.equal(k[P - 2, :, 2900 - 2048], new[0])
    kk, vv = (t[last].transpose(0, 1).reshape(Hkv, -1, d)[:, :2900][None] for t in (k, v))
    mask = torch.ones(1, 2900, dtype=torch.bool, device="cuda")
    kk = kk.clone()
    args = q.reshape(1, 8, 1, d), kk, vv, mask, d ** -0.5
    assert ((o[0].double() - ref.forward(*args)[0][0, :, 0]).abs() <= ref.forward_bounds(*args)[0][0, :, 0]).all()


def test_refused_bookkeeping_changes_nothing(bss):
    h = random_pages(random.Random(3), 6, 5, 40, 16, steps=4)
    h.free([5])
    h.free([4])
    t, n, r = on_gpu(h)
    full = [s for s in range(4) if h.lens[s]][0]
    cases = [
        lambda: bss.attn_kv_reserve(t, n, r, ints([0, -1, 0, 0, 0, 0]), 16),
        lambda: bss.attn_kv_reserve(t, n, r, ints([10 ** 9, 0, 0, 0, 0, 0]), 16),
        lambda: bss.attn_kv_reserve(t, n, r, ints([81, 0, 0, 0, 0, 0]), 16),           # past max_pages
        lambda: bss.attn_kv_fork(t, n, r, ints([full, full]), ints([5, 5]), 16)[0],    # a child twice
        lambda: bss.attn_kv_fork(t, n, r, ints([full]), ints([full]), 16)[0],
        lambda: bss.attn_kv_fork(t, n, r, ints([5]), ints([5]), 16)[0],                # its own parent
        lambda: bss.attn_kv_fork(t, n, r, ints([full, 4]), ints([4, 5]), 16)[0],       # a child as parent
        lambda: bss.attn_kv_fork(t, n, r, ints([9]), ints([5]), 16)[0],
        lambda: bss.attn_kv_fork(t, n, r, ints([full]), ints([-1]), 16)[0],
    ]
    for i, call in enumerate(cases):
        got = call()
        assert bss.attn_poll_status() == bss.ERR_BAD_PAGES, i
        assert torch.all(got == -1), i
        same(h, t, n, r)
    # too few pages
    small = Pages(3, 8, 4, 16)
    t, n, r = on_gpu(small)
    assert torch.all(bss.attn_kv_reserve(t, n, r, ints([40, 20, 1]), 16) == -1)
    assert bss.attn_poll_status() == bss.ERR_NO_PAGES
    same(small, t, n, r)
    bss.attn_kv_free(t, n, r, ints([7, -2, 1]), 16)      # sequences that do not exist
    assert bss.attn_poll_status() == bss.ERR_BAD_PAGES
    same(small, t, n, r)
    # fewer entries than rows: the others get nothing
    assert bss.attn_kv_reserve(t, n, r, ints([17]), 16).tolist() == [0]
    small.reserve([17, 0, 0])
    same(small, t, n, r)


def test_the_longest_sequence(bss):
    """Lengths count in 32 bits: a table with room for more neither grows a sequence past the last
    length nor decodes past it."""
    most, page = 0x7FFFFF00, 1024
    table = torch.zeros(1, 2 ** 21 + 1, dtype=torch.int32, device="cuda")
    refs = ints([1, 0, 0, 0])
    lens = ints([most - 256])
    assert bss.attn_kv_reserve(table, lens, refs, ints([257]), page).tolist() == [-1]
    assert bss.attn_poll_status() == bss.ERR_BAD_PAGES and lens.tolist() == [most - 256]
    assert bss.attn_kv_reserve(table, lens, refs, ints([256]), page).tolist() == [most - 256]
    assert bss.attn_poll_status() == 0 and lens.tolist() == [most]
    g = torch.Generator("cuda").manual_seed(1)
    k, v = (torch.randn(1, 1, page, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(1, 2, 64, generator=g, device="cuda").bfloat16()
    o, lse = bss.attn_decode_paged(q, k, v, table, lens, window=100, sinks=3)
    assert bss.attn_poll_status() == 0
    rows = [0, 1, 2] + [(most - 100 + i) % page for i in range(100)]
    mask = torch.ones(1, 103, dtype=torch.bool, device="cuda")
    args = q.reshape(1, 2, 1, 64), k[:, :, rows].double(), v[:, :, rows].double(), mask, 0.125
    assert ((o.double() - ref.forward(*args)[0][:, :, 0]).abs() <= ref.forward_bounds(*args)[0][:, :, 0]).all()
    lens[0] = 0x7FFFFFFF
    cut, _ = bss.attn_decode_paged(q, k, v, table, lens, window=100, sinks=3)
    assert bss.attn_poll_status() == bss.ERR_BAD_PAGES and torch.equal(cut, o)


def test_bookkeeping_of_many_pages(bss):
    """More pages than one turn of the scan takes, and tables that a second launch rewrites."""
    P, S, M, page = 70001, 700, 120, 16
    g = torch.Generator().manual_seed(1)
    held = torch.randperm(P, generator=g)[:60000]
    table = torch.full((S * M,), -1, dtype=torch.int64)
    table[:60000] = held
    table = table[torch.randperm(S * M, generator=g)].reshape(S, M)
    refs = torch.zeros(P, dtype=torch.int32)
    refs[held] = 1
    t, r = table.int().cuda(), refs.cuda()
    src, dst, count = bss.attn_kv_compact(t, r)
    assert bss.attn_poll_status() == 0
    at = torch.arange(P)
    want_src, want_dst = at[(refs > 0) & (at >= 60000)], at[(refs == 0) & (at < 60000)]
    assert int(count) == len(want_src)
    assert torch.equal(src.cpu().long()[:len(want_src)], want_src) and torch.all(src[len(want_src):] == -1)
    assert torch.equal(dst.cpu().long()[:len(want_src)], want_dst)
    to = at.clone()
    to[want_src] = want_dst
    assert torch.equal(t.cpu().long(), torch.where(table >= 0, to[table.clamp_min(0)], -1))
    assert torch.equal(r.cpu(), (at < 60000).int())
    # 9000 pages at once, past the list in shared memory; the lowest first
    n = torch.zeros(S, dtype=torch.int32, device="cuda")
    t2 = torch.full((S, M), -1, dtype=torch.int32, device="cuda")
    r2 = (torch.arange(P) % 3 > 0).int().cuda()
    new = torch.full((S,), 13 * page - 3, dtype=torch.int32, device="cuda")
    start = bss.attn_kv_reserve(t2, n, r2, new, page)
    assert bss.attn_poll_status() == 0 and torch.all(start == 0)
    assert torch.equal(t2[:, :13].cpu().long().flatten(), 3 * torch.arange(13 * S))
    assert torch.all(t2[:, 13:] == -1)


def test_two_graphs_and_streams(bss):
    """Two captured decodings that share a workspace, replayed one after the other on new contents,
    and two eager ones at once on streams and workspaces of their own."""
    lens = [[300, 0, 77, 1024], [64, 500, 3]]
    caches = [Cache(l, 2, 128, 32, 31 + i) for i, l in enumerate(lens)]
    qs = [torch.randn(len(l), 8, 128, device="cuda").bfloat16() for l in lens]
    ws = torch.empty(16 + max(bss.attn_decode_paged_workspace_bytes(len(l), 8, 2, 128, c.table.shape[1], 32)
                         for l, c in zip(lens, caches)), device="cuda", dtype=torch.uint8)
    ws.fill_(255)
    run = lambda i, **kw: bss.attn_decode_paged(qs[i], caches[i].k, caches[i].v, caches[i].table,  # noqa: E731
                                                caches[i].lens, **kw)
    for i in range(2):
        run(i)
    torch.cuda.synchronize()
    graphs, held = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(run(i, workspace=ws))
        graphs.append(g)
    for turn in range(3):
        for i in (0, 1):
            qs[i].copy_(torch.randn_like(qs[i]))
        caches[0].lens.copy_(ints([300 - 50 * turn, 0, 77, 1024 - turn]))
        want = [run(i) for i in range(2)]
        for i in (1, 0, 1):
            graphs[i].replay()
        torch.cuda.synchronize()
        for w, x in zip(want, held):
            assert torch.equal(w[0], x[0]) and torch.equal(w[1], x[1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append(run(i))
        torch.cuda.synchronize()
        for w, x in zip(want, got):
            assert torch.equal(w[0], x[0]) and torch.equal(w[1], x[1])
    assert bss.attn_poll_status() == 0


def test_paged_refusals(bss):
    c = Cache([40], 2, 64, 16, 1)
    q = torch.randn(1, 4, 64, device="cuda").bfloat16()
    for bad in (dict(k_cache=c.k.transpose(1, 2).contiguous().transpose(1, 2)), dict(v_cache=c.v[:-1]),
                dict(k_cache=c.k.half()), dict(q=q.float()), dict(q=q[:, ::2]), dict(page_table=c.table.long()),
                dict(seq_lens=c.lens.repeat(2)), dict(k_scale=torch.ones(2, device="cuda")),
                dict(k_cache=c.k.to(E4M3), v_cache=c.v.to(E4M3))):
        args = dict(q=q, k_cache=c.k, v_cache=c.v, page_table=c.table, seq_lens=c.lens) | bad
        with pytest.raises(ValueError):
            bss.attn_decode_paged(**args)
    with pytest.raises(bss.AttnError, match="INVALID_ARG"):
        bss.attn_decode_paged(q, c.k, c.v, c.table, c.lens, sinks=3)
    with pytest.raises(bss.AttnError, match="WORKSPACE"):
        bss.attn_decode_paged(q, c.k, c.v, c.table.repeat(1, 50), c.lens, workspace=torch.empty(64, device="cuda"))
    with pytest.raises(bss.AttnError, match="UNSUPPORTED"):
        bss.attn_kv_reserve(c.table, c.lens, ints([0] * c.k.shape[0]), ints([1]), 24)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,H,Hkv,d,page", [([300, 1, 64], 8, 2, 128, 16), ([700, 33], 16, 1, 64, 32),
                                               ([2100, 900], 16, 4, 64, 64), ([3000, 70], 20, 1, 128, 128)])
def test_decode_loses_nothing_to_P(bss, lens, H, Hkv, d, page, e4m3):
    """P enters its product in two bf16 parts (all but 2^-15 of it) over bf16 pages, in fp16 (2^-11)
    over e4m3 ones: what is left is the rounding of O itself, and fp32 sums of a term a key, off by
    at most 2^-23 of sum P |v| each.  Where O is small beside the values it averages, a P in bf16
    alone is 2^-8 of sum P |v| off."""
    c = Cache(lens, Hkv, d, page, 7 * d + page, e4m3)
    g = torch.Generator("cuda").manual_seed(d)
    q = torch.randn(len(lens), H, d, generator=g, device="cuda").bfloat16()
    for columns in (0, 1100 // page):
        c.table = torch.cat([c.table, ints([[-1] * columns] * len(lens))], 1)
        o, _ = check_decode(bss, c, q, lens, 0, 0)
        for s, n in enumerate(lens):
            mask = ref.window_mask(1, n, n, 0, n - 1, 0, "cuda")
            args = q[s].reshape(1, H, 1, d), c.k64[s][None], c.v64[s][None], mask, d ** -0.5
            bound, _ = ref.forward_bounds(*args, p_round=2.0 ** (-11 if e4m3 else -15), sums=n * 2.0 ** -23)
            off = (o[s].double() - ref.forward(*args)[0][0, :, 0]).abs()
            assert (off <= bound[0, :, 0]).all(), (s, n, (off / bound[0, :, 0]).max())


def test_decode_of_an_infinite_value(bss):
    """An infinity among the values that are seen comes out as one, in its own column alone."""
    c = Cache([100, 40], 2, 64, 16, 5)
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    want, _ = bss.attn_decode_paged(q, c.k, c.v, c.table, c.lens)
    c.v[c.table[0, 1], 1, 3, 7] = float("inf")
    c.v[c.table[0, 2], 0, 0, 9] = -float("inf")
    got, _ = bss.attn_decode_paged(q, c.k, c.v, c.table, c.lens)
    want[0, 2:, 7] = float("inf")
    want[0, :2, 9] = -float("inf")
    assert torch.equal(got, want)
    assert bss.attn_poll_status() == 0


@pytest.mark.parametrize("columns", [4, 70000])
def test_compaction_reports_bad_entries(bss, columns):
    """An entry past the last page is reported and left as it is, for small tables and for large
    ones, which a launch of their own rewrites, whether or not a page moves."""
    for refs, moved in (([1, 1, 0, 0], 0), ([0, 1, 1, 0], 1)):
        table = torch.full((1, columns), -1, dtype=torch.int32, device="cuda")
        table[0, -3:] = ints([9, 1, 2 if moved else 0])
        r = ints(refs)
        src, dst, count = bss.attn_kv_compact(table, r)
        assert bss.attn_poll_status() == bss.ERR_BAD_PAGES
        assert int(count) == moved and r.tolist() == [1, 1, 0, 0]
        assert table[0, -3:].tolist() == [9, 1, 0] and torch.all(table[0, :-3] == -1)
        assert src.tolist() == [2 if moved else -1, -1, -1, -1]
        assert dst.tolist() == [0 if moved else -1, -1, -1, -1]
        table[0, -3] = -1
        bss.attn_kv_compact(table, r)
        assert bss.attn_poll_status() == 0


def test_an_empty_batch(bss):
    """No sequence, no token, no fork: nothing happens, and the outputs have no rows."""
    c = Cache([40, 3], 2, 64, 16, 6)
    before = [t.clone() for t in (c.k, c.v, c.table, c.lens)]
    refs = torch.zeros(c.k.shape[0], dtype=torch.int32, device="cuda")
    none, bf = ints([]), dict(dtype=torch.bfloat16, device="cuda")
    for columns in (0, 100):                           # either route
        wide = torch.cat([c.table, ints([[-1] * columns] * 2)], 1)
        for table, lens in ((wide, c.lens), (wide[:0], c.lens[:0])):
            o, lse = bss.attn_decode_paged(torch.empty(0, 4, 64, **bf), c.k, c.v, table, lens)
            assert o.shape == (0, 4, 64) and o.dtype == torch.bfloat16
            assert lse.shape == (0, 4) and lse.dtype == torch.float32
    start = bss.attn_kv_reserve(c.table, c.lens, refs, none, 16)
    assert start.shape == (0,) and start.dtype == torch.int32
    rows = torch.randn(3, 2, 64, device="cuda").bfloat16()
    bss.attn_kv_write(rows, rows, c.k, c.v, c.table, none, ints([3]))       # rows of no sequence
    bss.attn_kv_write(rows[:0], rows[:0], c.k, c.v, c.table, ints([40, 3]), ints([0, 0, 0]))
    src, dst = bss.attn_kv_fork(c.table, c.lens, refs, none, none, 16)
    bss.attn_kv_copy_pages(c.k, c.v, src, dst)
    bss.attn_kv_free(c.table, c.lens, refs, none, 16)
    assert bss.attn_poll_status() == 0
    assert all(torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a,
                           b.view(torch.int16) if b.dtype == torch.bfloat16 else b)
               for a, b in zip(before, (c.k, c.v, c.table, c.lens)))
    with pytest.raises(ValueError):
        bss.attn_decode_paged(torch.empty(0, 4, 32, **bf), c.k, c.v, c.table, c.lens)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,H,Hkv,d,page,window,sinks", [
    ([1008], 16, 1, 128, 16, 0, 0),                # a tight table, units shared by several CTAs
    ([700, 0, 1, 1023], 20, 1, 64, 32, 0, 0),
    ([1024 - 64, 17], 66, 2, 128, 64, 300, 5),
    ([13, 0, 16, 1] * 160, 4, 1, 64, 16, 0, 0),    # many units of one page
])
def test_decode_of_tight_tables_shared_evenly(bss, lens, H, Hkv, d, page, window, sinks, e4m3):
    c = Cache(lens, Hkv, d, page, sum(lens) + d, e4m3, window=window, sinks=sinks)
    c.table = c.table[:, :-(-max(lens) // page)].contiguous()       # no more room than the longest takes
    assert bss.attn_decode_paged_workspace_bytes(len(lens), H, Hkv, d, c.table.shape[1], page) > 0
    q = torch.randn(len(lens), H, d, generator=torch.Generator("cuda").manual_seed(H), device="cuda").bfloat16()
    a = check_decode(bss, c, q, lens, window, sinks)
    b = check_decode(bss, c, q, lens, window, sinks)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
