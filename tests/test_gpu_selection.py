"""Mean keys and selected pages where they are hardest, on the GPU: sums that cancel, scores that tie,
the widest tables, offsets in disorder, and the attention of a sparse layer in a cache whose pages are
shared and moved."""
import math
import random

import pytest
import torch

from oracle import window as ref
from oracle.select import select_pages
from test_gpu_paged import ints

pytestmark = pytest.mark.gpu

BAD_PAGES = 7


@pytest.fixture(scope="module")
def bss():
    import block_sparse_softmax_gb300 as m
    m.library()
    return m


# ----------------------------------------------------------------------------
# mean keys
# ----------------------------------------------------------------------------

def check_means(bss, k):
    """`k` [pages, heads, page, d] bf16: every mean is the exact sum's, rounded once.  (The sum itself
    is rounded to 64 bits by math.fsum, by 2^-53 of it.)"""
    P, Hkv, page, d = k.shape
    means = torch.full((P, Hkv, d), 5.0, device="cuda")
    bss.attn_kv_pool(k, means, ints([list(range(P))]), ints([0]), ints([P * page]))
    assert bss.attn_poll_status() == 0
    columns = k.double().transpose(2, 3).reshape(-1, page).tolist()
    want = torch.tensor([math.fsum(c) / page for c in columns], dtype=torch.float64).view(P, Hkv, d)
    off = (means.double().cpu() - want).abs()
    assert (off <= (2.0 ** -24 + 2.0 ** -50) * want.abs()).all(), (off / want.abs().clamp_min(1e-300)).max()


def test_pool_of_three_magnitudes(bss):
    """Numbers that cancel down to one that neither the sum nor its rest holds beside them."""
    k = torch.zeros(4, 1, 16, 64, device="cuda", dtype=torch.bfloat16)
    # rows that one warp's lanes of different rows hold, in either order
    for p, order in enumerate(((0, 4, 8, 12, 1), (12, 8, 4, 0, 3), (0, 1, 2, 3, 4), (15, 0, 7, 9, 2))):
        for r, x in zip(order, (2.0 ** 51, 2.0 ** 26, 1.0, -(2.0 ** 51), -(2.0 ** 26))):
            k[p, 0, r] = x
    check_means(bss, k)
    k[1, 0, :, 5:9] *= -(2.0 ** -70)
    k[2, 0, :, 40] *= 2.0 ** 70
    k[3, 0, 5, 63] = 2.0 ** -133                          # the smallest number there is
    check_means(bss, k)


@pytest.mark.parametrize("page,d,Hkv", [(16, 64, 2), (64, 128, 3), (128, 64, 1), (1024, 128, 1), (1024, 64, 2)])
def test_pool_of_wide_ranges(bss, page, d, Hkv):
    """Elements spread over some or all binades, half of them cancelling the other half but for little."""
    g = torch.Generator("cuda").manual_seed(page + d)
    P = 3
    x = torch.randn(P, Hkv, page, d, generator=g, device="cuda")
    e = torch.randint(-20, 21, x.shape, generator=g, device="cuda")
    e[1] = torch.randint(-60, 61, e[1].shape, generator=g, device="cuda")
    e[2] = torch.randint(-132, 116, e[2].shape, generator=g, device="cuda")
    k = torch.ldexp(x, e).clamp(-3e38, 3e38).bfloat16()
    half = page // 2
    perm = torch.randperm(half, generator=g, device="cuda")
    k[:, :, half:, ::2] = -k[:, :, perm, ::2]             # every other column: sums of 0 but for
    k[:, :, page - 1, ::4] = torch.ldexp(x[:, :, 0, ::4], e[:, :, 1, ::4]).clamp(-3e38, 3e38).bfloat16()
    check_means(bss, k)


def test_pool_of_scales_past_the_range(bss):
    """A mean times its scale that leaves fp32's range is infinite, not a NaN."""
    k = torch.full((1, 3, 16, 64), 448.0, device="cuda").to(torch.float8_e4m3fn)
    k[0, 1] = torch.full((16, 64), -448.0, device="cuda").to(torch.float8_e4m3fn)
    means = torch.zeros(1, 3, 64, device="cuda")
    bss.attn_kv_pool(k, means, ints([[0]]), ints([0]), ints([16]),
                     k_scale=torch.tensor([2.0 ** 120, 2.0 ** 120, 2.0 ** 110], device="cuda"))
    assert (means[0, 0] == math.inf).all() and (means[0, 1] == -math.inf).all()
    assert (means[0, 2] == 448.0 * 2.0 ** 110).all()


# ----------------------------------------------------------------------------
# selection
# ----------------------------------------------------------------------------

def check_selected(bss, q, means, table, lens, cu, news, top, page, local=1, first=0):
    pages, got = bss.attn_select_pages(q, means, table, ints(lens), ints(cu), top, page, local_pages=local,
                                       first_pages=first)
    assert bss.attn_poll_status() == 0
    want, n = select_pages(q, means, table, lens, cu, news, top, page, local, first)
    assert torch.equal(pages.cpu(), want) and torch.equal(got.cpu(), n)
    return pages


# pages of a row: few and many that are undecided (32 are ranked at once), and more columns than a
# table whose rows are short has
@pytest.mark.parametrize("rows", [1, 9])
@pytest.mark.parametrize("n", [25, 300, 2500])
def test_products_that_cancel(bss, n, rows):
    """Scores that only what 64 bits lose beside 2^60 tells apart."""
    page, d = 16, 128
    g = torch.Generator("cuda").manual_seed(n)
    table = torch.randperm(n, generator=g, device="cuda").int()[None]
    q = torch.zeros(rows, 2, d, device="cuda", dtype=torch.bfloat16)
    q[:, 0, 0], q[:, 0, 32], q[:, 0, 64] = 2.0 ** 60, 1.0, -(2.0 ** 60)       # a lane's three
    means = torch.zeros(n, 1, d, device="cuda")
    means[:, 0, 0] = means[:, 0, 64] = 1.0
    means[:, 0, 32] = torch.randint(-63, 64, (n,), generator=g, device="cuda").float()
    args = [n * page - rows // 2], [0, rows], [rows]
    for top in (1, 7, 20):
        check_selected(bss, q, means, table, *args, top, page)
    q = q.roll(5, -1)
    q[:, 0, 37] = 0.0                                     # ... and lanes' sums of them
    q[:, 1, 21] = 1.0
    means = means.roll(5, -1)
    means[:, 0, 21] = means[:, 0, 37]
    for top in (1, 7):
        check_selected(bss, q, means, table, *args, top, page)
    # the same in the group's sum: heads of 2^60, 1 and -2^60
    q = torch.zeros(rows, 3, d, device="cuda", dtype=torch.bfloat16)
    q[:, 0, 3], q[:, 1, 3], q[:, 2, 3] = 2.0 ** 60, 1.0, -(2.0 ** 60)
    means = torch.zeros(n, 1, d, device="cuda")
    means[:, 0, 3] = torch.randint(-63, 64, (n,), generator=g, device="cuda").float()
    for top in (1, 7):
        check_selected(bss, q, means, table, *args, top, page)


@pytest.mark.parametrize("rows", [1, 9])
@pytest.mark.parametrize("n", [25, 300, 2500])
@pytest.mark.parametrize("d,spread", [(128, 0), (128, 12), (64, 20), (128, 20)])
def test_sums_of_the_same_numbers_tie(bss, d, spread, n, rows):
    """Means that are one another's permutations score alike under a query of one value, in whatever
    order they are added; the lower places are taken."""
    page = 16
    g = torch.Generator("cuda").manual_seed(n + d + spread)
    table = torch.randperm(n, generator=g, device="cuda").int()[None]
    q = torch.full((rows, 2, d), 1.375, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(d, generator=g, device="cuda")
    x = torch.ldexp(x, torch.randint(-spread // 2, spread // 2 + 1, (d,), generator=g, device="cuda"))
    means = torch.stack([x[torch.randperm(d, generator=g, device="cuda")] for _ in range(n)])[:, None].contiguous()
    # (the rows end in the last page: all see the same others)
    args = [n * page - 1], [0, rows], [rows]
    for top in (1, 7, 20):
        pages = check_selected(bss, q, means, table, *args, top, page)
        assert torch.equal(pages[:, 0, :top], table[:, :top].expand(rows, -1))
    # one of them is larger by a unit of its smallest element's last place
    at = table[0, n * 2 // 3].item()
    col = means[at, 0].abs().argmin()
    means[at, 0, col] = torch.nextafter(means[at, 0, col], means.new_tensor(math.inf))
    for top in (1, 20):
        pages = check_selected(bss, q, means, table, *args, top, page)
        assert (pages[:, 0, :-1] == at).any(-1).all()


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("d,n", [(128, 2049), (64, 4000), (128, 4500)])
def test_wide_tables(bss, d, n, rows):
    """Tables of more columns than a small block picks from: ordinary scores, pages given back, ties
    and near ties, scores that are not finite."""
    page, top = 16, 60
    g = torch.Generator("cuda").manual_seed(n + rows)
    table = torch.randperm(n, generator=g, device="cuda").int()[None]
    q = torch.randn(rows, 4, d, generator=g, device="cuda").bfloat16()
    means = torch.randn(n, 2, d, generator=g, device="cuda")
    few = slice(0, 1) if rows == 1 else slice(18, 21)     # rows that are looked at
    picked = list(range(rows))[few]

    def check(means, table, top, local=1, first=0, q=q):
        pages, got = bss.attn_select_pages(q, means, table, ints([n * page - 3]), ints([0, rows]), top, page,
                                           local_pages=local, first_pages=first)
        assert bss.attn_poll_status() == 0
        for r in picked:
            end = n * page - 3 - rows + r + 1
            want, m = select_pages(q[r:r + 1], means, table, [end], [0, 1], [1], top, page, local, first)
            assert torch.equal(pages[r].cpu(), want[0]) and got[r].item() == m[0].item()

    check(means, table, top)
    holes = table.clone()
    holes[0, torch.randperm(n - 9, generator=g, device="cuda")[:n // 3]] = -1
    check(means, holes, top, 3, 2)
    check(means, holes, n, 3, 2)                          # more than there are
    alike = means[:1].repeat(n, 1, 1)
    check(alike, table, top)
    for step in (2.0 ** -23, 2.0 ** -18):
        near = alike.clone()
        col = torch.randint(0, d, (n,), generator=g, device="cuda")
        near[torch.arange(n), 0, col] *= 1 + step * torch.randint(-3, 4, (n,), generator=g, device="cuda")
        check(near, table, 1)
        check(near, table, top)
    check(alike, table, 7, q=q * 0)
    odd = means.clone()
    for x in (math.nan, math.inf, -math.inf):
        odd[torch.randperm(n, generator=g, device="cuda")[:30], :, 3] = x
    check(odd, table, top)
    odd[:, :, 5] = math.nan                               # nothing but NaN: the lower places
    check(odd, table, top)


@pytest.mark.parametrize("rows", [1, 9])
@pytest.mark.parametrize("n", [25, 300, 2500])
def test_scores_past_the_range(bss, n, rows):
    """Scores that 32 bits make infinite or 0 are told apart; a query that is not finite has scores
    that are infinite or no numbers."""
    page, d = 16, 128
    g = torch.Generator("cuda").manual_seed(n)
    table = torch.randperm(n, generator=g, device="cuda").int()[None]
    q = torch.randn(rows, 2, d, generator=g, device="cuda").bfloat16()
    means = torch.randn(n, 1, d, generator=g, device="cuda")
    args = [n * page - rows // 2], [0, rows], [rows]
    for a, b in ((100, 60), (-100, -45), (-20, -120), (120, -100)):
        for top in (1, 20):
            check_selected(bss, torch.ldexp(q.float(), torch.tensor(a, device="cuda")).bfloat16(),
                           torch.ldexp(means, torch.tensor(b, device="cuda")), table, *args, top, page)
    for x in (math.inf, -math.inf, math.nan):
        far = q.clone()
        far[:, 1, 7] = x
        check_selected(bss, far, means, table, *args, 20, page)
        few = means.clone()
        few[::3, 0, 7] = 0.0                              # infinity times 0
        few[1::5, 0, 90] = math.inf
        check_selected(bss, far, few, table, *args, 20, page)
        check_selected(bss, q, few, table, *args, 20, page)
    far[:, 1, 7], far[:, 0, 7] = math.inf, -math.inf      # ... and their sum
    check_selected(bss, far, means, table, *args, 20, page)


def test_selection_reports_offsets_in_disorder(bss):
    """... as the dense layer's call does; what it writes may be handed on."""
    page, d = 16, 64
    table = ints([[0, 1, 2, 3]] * 4)
    means = torch.zeros(4, 1, d, device="cuda")
    lens = ints([60, 60, 60, 60])
    k = torch.zeros(4, 1, page, d, device="cuda", dtype=torch.bfloat16)
    for T in (3, 40):
        q = torch.zeros(T, 2, d, device="cuda", dtype=torch.bfloat16)
        for cu in ([0, 2, 1, 2, 3], [3, 2, 1, 0, 0], [0, 1, 2, 3, 2]):
            pages, n = bss.attn_select_pages(q, means, table, lens, ints(cu), 2, page)
            assert bss.attn_poll_status() == BAD_PAGES, cu
            assert ((pages >= -1) & (pages < 4)).all() and ((n >= -1) & (n <= 64)).all()
            bss.attn_decode_selected(q, k, k, pages, n)
            torch.cuda.synchronize()
            bss.attn_poll_status()
        # (three of the four pages: two whole ones and the 12 tokens of the last)
        pages, n = bss.attn_select_pages(q, means, table, lens, ints([0, 1, 1, 2, 3]), 2, page)
        assert bss.attn_poll_status() == 0 and n[:3].tolist() == [44, 44, 44] and (n[3:] == -1).all()


@pytest.mark.parametrize("news", [[100, 60], [1, 1, 70, 2, 1, 60, 3, 0, 40, 1]])
def test_wide_tables_of_many_rows(bss, news):
    """... and of more rows and heads than multiprocessors, of one chunk or of chunks beside single
    tokens."""
    page, d, n = 16, 64, 2600
    g = torch.Generator("cuda").manual_seed(len(news))
    S, T = len(news), sum(news)
    table = torch.stack([torch.randperm(n, generator=g, device="cuda") for _ in range(S)]).int()
    table[:, 5:900:7] = -1
    means = torch.randn(n, 2, d, generator=g, device="cuda")
    means[1::2] = means[::2]                              # ties
    q = torch.randn(T, 2, d, generator=g, device="cuda").bfloat16()
    cu = [0]
    for x in news:
        cu.append(cu[-1] + x)
    lens = [n * page - 37 * s for s in range(S)]
    pages, got = bss.attn_select_pages(q, means, table, ints(lens), ints(cu), 21, page, local_pages=2, first_pages=1)
    assert bss.attn_poll_status() == 0
    for s, new in enumerate(news):
        for i in {0, new // 2, new - 1} if new else ():
            t, end = cu[s] + i, lens[s] - new + i + 1
            want, m = select_pages(q[t:t + 1], means, table[s:s + 1], [end], [0, 1], [1], 21, page, 2, 1)
            assert torch.equal(pages[t].cpu(), want[0]) and got[t].item() == m[0].item(), (s, i)


def test_selections_on_two_streams(bss):
    """Pooling, selection and its attention on two streams at once, in caches of their own, are what they
    are one after the other."""
    H, Hkv, d, page = 8, 2, 128, 16
    steps = []
    for i, (lens, news) in enumerate((([5000, 300, 41], [1, 200, 3]), ([2000] * 40, [1] * 40))):
        g = torch.Generator("cuda").manual_seed(i)
        held = [-(-n // page) for n in lens]
        P, S = sum(held), len(lens)
        table = torch.full((S, max(held)), -1, dtype=torch.int32, device="cuda")
        order = torch.randperm(P, generator=g, device="cuda").int()
        for s in range(S):
            table[s, :held[s]] = order[sum(held[:s]):sum(held[:s + 1])]
        k, v = (torch.randn(P, Hkv, page, d, generator=g, device="cuda").bfloat16() for _ in range(2))
        q = torch.randn(sum(news), H, d, generator=g, device="cuda").bfloat16()
        cu = ints([sum(news[:s]) for s in range(S + 1)])
        steps.append((q, k, v, torch.zeros(P, Hkv, d, device="cuda"), table, ints(lens), cu, ints([0] * S)))

    def step(q, k, v, means, table, lens, cu, start):
        bss.attn_kv_pool(k, means, table, start, lens)
        pages, n = bss.attn_select_pages(q, means, table, lens, cu, 12, page, local_pages=2, first_pages=1)
        return (means.clone(), pages, n) + bss.attn_decode_selected(q, k, v, pages, n)

    want = [step(*x) for x in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(10):
        got = []
        for x, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                got.append(step(*x))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for x, y in zip(a, b):
                assert torch.equal(x, y)
    assert bss.attn_poll_status() == 0


# ----------------------------------------------------------------------------
# a sparse layer
# ----------------------------------------------------------------------------

def test_a_sparse_layer_of_a_server(bss):
    """Step after step in one cache, over forks, compaction and freed sequences: the attention of each
    row is that over the tokens of its chosen pages, the last of them not whole."""
    S, H, Hkv, d, page, P = 6, 8, 2, 64, 16, 300
    G = H // Hkv
    g = torch.Generator("cuda").manual_seed(11)
    kc = torch.full((P, Hkv, page, d), float("nan"), device="cuda", dtype=torch.bfloat16)
    vc = kc.clone()
    means = torch.full((P, Hkv, d), float("nan"), device="cuda")
    table = torch.full((S, 40), -1, dtype=torch.int32, device="cuda")
    lens, refs = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (S, P))
    keys = [torch.zeros(Hkv, 0, d, device="cuda", dtype=torch.float64) for _ in range(S)]
    values = [x.clone() for x in keys]
    rng = random.Random(6)
    for step in range(8):
        if step in (3, 6):                                # the second goes on as the sixth, too
            bss.attn_kv_free(table, lens, refs, ints([5]), page)
            src, dst = bss.attn_kv_fork(table, lens, refs, ints([1]), ints([5]), page)
            bss.attn_kv_copy_pages(kc, vc, src, dst)
            keys[5], values[5] = keys[1], values[1]
        if step in (4, 7):
            bss.attn_kv_free(table, lens, refs, ints([0]), page)
            keys[0], values[0] = keys[0][:, :0], values[0][:, :0]
            src, dst, count = bss.attn_kv_compact(table, refs)
            bss.attn_kv_copy_pages(kc, vc, src, dst, count)
            means.fill_(float("nan"))
            bss.attn_kv_pool(kc, means, table, torch.zeros_like(lens), lens)
        news = [rng.choice([0, 1, 5, 40, 70]) for _ in range(S)]
        cu = [0]
        for n in news:
            cu.append(cu[-1] + n)
        T = cu[-1]
        if T == 0:
            continue
        q = torch.randn(T, H, d, generator=g, device="cuda").bfloat16()
        k, v = (torch.randn(T, Hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2))
        start = bss.attn_kv_reserve(table, lens, refs, ints(news), page)
        bss.attn_kv_write(k, v, kc, vc, table, start, ints(cu))
        bss.attn_kv_pool(kc, means, table, start, lens)
        for s in range(S):
            keys[s] = torch.cat([keys[s], k[cu[s]:cu[s + 1]].transpose(0, 1).double()], 1)
            values[s] = torch.cat([values[s], v[cu[s]:cu[s + 1]].transpose(0, 1).double()], 1)
        have = [x.shape[1] for x in keys]
        pages = check_selected(bss, q, means, table, have, cu, news, 2, page, 2, 1)
        pages, n = bss.attn_select_pages(q, means, table, lens, ints(cu), 2, page, local_pages=2, first_pages=1)
        o, lse = bss.attn_decode_selected(q, kc, vc, pages, n)
        assert bss.attn_poll_status() == 0
        slots = table.tolist()
        for t in rng.sample(range(T), min(T, 25)):
            s = max(i for i in range(S) if cu[i] <= t)
            own = have[s] - (cu[s + 1] - t)
            for h in range(Hkv):
                seen = []
                for x in pages[t, h].tolist():
                    if x >= 0:
                        m = slots[s].index(x)
                        seen += [j for j in range(m * page, (m + 1) * page) if j <= own]
                assert len(seen) == n[t].item()
                args = (q[t, h * G:(h + 1) * G][None, :, None], keys[s][h, seen][None, None],
                        values[s][h, seen][None, None],
                        torch.ones(1, len(seen), dtype=torch.bool, device="cuda"), 1.0 / math.sqrt(d))
                O, L, _ = ref.forward(*args)
                bo, bl = ref.forward_bounds(*args)
                assert ((o[t, h * G:(h + 1) * G].double() - O[0, :, 0]).abs() <= bo[0, :, 0]).all(), (step, t, h)
                assert ((lse[t, h * G:(h + 1) * G].double() - L[0, :, 0]).abs() <= bl[0, :, 0]).all(), (step, t, h)
