"""Chunks of new tokens over the paged cache, and attention over selected pages, on the GPU: against
their definitions in 64 bits (bounds of `oracle/window.py`), selections number by number."""
import math
import random

import pytest
import torch

from oracle import window as ref
from oracle.select import page_means, select_pages
from test_gpu_paged import Cache, ints

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
BAD_PAGES = 7


@pytest.fixture(scope="module")
def bss():
    import block_sparse_softmax_gb300 as m
    m.library()
    return m


def ragged(news, H, d, seed, before=0, after=0):
    """(q [T,H,d], cu) of new tokens per sequence, with rows of nobody before and after them."""
    g = torch.Generator("cuda").manual_seed(seed)
    cu = [before]
    for n in news:
        cu.append(cu[-1] + n)
    return torch.randn(cu[-1] + after, H, d, generator=g, device="cuda").bfloat16(), cu


def check_rows(q, o, lse, c, lens, news, cu, window=0, sinks=0, skip=(), scale=None):
    H, d = q.shape[1:]
    scale = scale or 1.0 / math.sqrt(d)
    for s, (n, new) in enumerate(zip(lens, news)):
        if new == 0 or s in skip:
            continue
        a, b = cu[s], cu[s + 1]
        mask = ref.window_mask(new, n, window or n, sinks, n - new, 0, "cuda")
        args = (q[a:b].transpose(0, 1)[None], c.k64[s][None], c.v64[s][None], mask, scale)
        O, L, _ = ref.forward(*args)
        bo, bl = ref.forward_bounds(*args)
        if getattr(c, "k_scale", None) is not None:
            # over e4m3 pages P enters its product as fp16, 2^7 times itself relative to a maximum
            # that the row's largest reaches: what is below 2^-14 there is off by at most half of
            # fp16's last step, 2^-25, so a P_j by 2^-32 of the largest, which l holds whole
            bo = bo + 2.0 ** -32 * (mask.double() @ c.v64[s].abs().repeat_interleave(H // c.v64[s].shape[0], 0))
        off = (o[a:b].transpose(0, 1)[None].double() - O).abs()
        assert (off <= bo).all(), (s, n, new, (off / bo).max())
        off = (lse[a:b].transpose(0, 1)[None].double() - L).abs()
        assert (off <= bl).all(), (s, n, new, (off / bl).max())


def check_chunk(bss, c, q, cu, lens, news, window=0, sinks=0, **kw):
    o, lse = bss.attn_fwd_paged(q, c.k, c.v, c.table, c.lens, ints(cu), window=window, sinks=sinks,
                                k_scale=c.k_scale, v_scale=c.v_scale, **kw)
    torch.cuda.synchronize()
    assert bss.attn_poll_status() == 0
    check_rows(q, o, lse, c, lens, news, cu, window, sinks, scale=kw.get("scale"))
    return o, lse


CASES = [
    # lens, new tokens, H, Hkv, d, page, window, sinks
    ([1], [1], 1, 1, 128, 16, 0, 0),
    ([300], [5], 16, 4, 128, 16, 0, 0),
    ([17, 0, 200, 64, 129, 128], [17, 0, 1, 64, 1, 128], 8, 2, 128, 16, 0, 0),
    ([5, 1000, 33, 257, 0, 64], [5, 130, 33, 1, 0, 3], 6, 2, 64, 64, 0, 0),       # 3 heads: tiles of 42 tokens
    ([777, 12, 2049], [300, 12, 65], 16, 1, 128, 128, 0, 0),
    ([500, 31, 1025], [33, 31, 1], 20, 1, 64, 32, 0, 0),
    ([130, 70], [2, 70], 256, 2, 128, 16, 0, 0),                                  # 128 heads of a group
    ([130, 70], [2, 70], 198, 2, 64, 16, 0, 0),                                   # ... 99
    ([4000, 1, 2600], [1000, 1, 129], 8, 8, 64, 1024, 0, 0),
    ([20011], [3], 2, 1, 128, 32, 0, 0),                                          # few rows, many keys
    ([9000, 3000], [1, 1], 4, 4, 128, 16, 0, 0),
    ([1000, 40, 3, 0, 999], [200, 40, 1, 0, 1], 8, 2, 128, 16, 100, 4),
    ([1000, 40, 3, 0, 999], [999, 7, 3, 0, 130], 8, 2, 64, 64, 1, 0),             # each token sees itself
    ([1000, 40, 3, 0, 2999], [100, 40, 3, 0, 1], 16, 2, 128, 32, 37, 70),         # sinks past a page
    ([3000, 601, 615], [700, 601, 100], 4, 4, 64, 16, 600, 130),
    ([900, 17], [900, 17], 9, 3, 128, 64, 10 ** 12, 10 ** 12),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,news,H,Hkv,d,page,window,sinks", CASES)
def test_chunk(bss, lens, news, H, Hkv, d, page, window, sinks, e4m3):
    seen = window + max(news) - 1 if window else 0       # what some row of a sequence sees
    c = Cache(lens, Hkv, d, page, sum(lens) + H + page, e4m3, window=seen, sinks=sinks)
    q, cu = ragged(news, H, d, H + len(lens))
    a = check_chunk(bss, c, q, cu, lens, news, window, sinks)
    b = check_chunk(bss, c, q, cu, lens, news, window, sinks)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_of_many_items(bss, d, e4m3):
    """More tiles than the GPU has SMs, of very different lengths."""
    rng = random.Random(d)
    lens = [rng.choice([0, 1, 130, rng.randint(1, 3000)]) for _ in range(70)]
    news = [min(n, rng.choice([1, 1, 40, 300])) for n in lens]
    c = Cache(lens, 2, d, 32, d, e4m3)
    q, cu = ragged(news, 16, d, 3)
    check_chunk(bss, c, q, cu, lens, news)


def test_chunk_of_single_tokens_is_decoding(bss):
    lens = [1, 40, 700, 0, 1500]
    c = Cache(lens, 2, 128, 16, 5)
    q, cu = ragged([1, 1, 1, 0, 1], 8, 128, 4)
    o, lse = check_chunk(bss, c, q, cu, lens, [1, 1, 1, 0, 1])
    rows = torch.tensor([0, 1, 2, 4], device="cuda")
    full = torch.zeros(5, 8, 128, device="cuda", dtype=torch.bfloat16)
    full[rows] = q
    od, ld = bss.attn_decode_paged(full, c.k, c.v, c.table, c.lens)
    assert (o.float() - od[rows].float()).abs().max() <= 0.03
    assert (lse - ld[rows]).abs().max() <= 1e-4


@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_of_no_sequence_are_left_alone(bss, e4m3):
    lens, news = [300, 17, 90], [40, 17, 1]
    c = Cache(lens, 2, 128, 16, 7, e4m3, inter=True)
    q, cu = ragged(news, 8, 128, 1, before=5, after=11)
    wide = torch.full((q.shape[0], 3, 8, 128), float("nan"), device="cuda", dtype=torch.bfloat16)
    wide[:, 1] = q
    q = wide[:, 1]                                       # strided rows
    o = torch.full((q.shape[0], 8, 128), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((q.shape[0], 8), 3.0, device="cuda")
    # (the table's last rows are of sequences that the batch does not hold)
    c.table = torch.cat([c.table, torch.full_like(c.table, 10 ** 6)])
    c.lens = torch.cat([c.lens, c.lens * 0 - 5])
    check_chunk(bss, c, q, cu, lens, news, out=o, lse=lse)
    for x, v in ((o, 7.0), (lse, 3.0)):
        assert (x[:5] == v).all() and (x[-11:] == v).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_reports_bad_pages(bss, d, e4m3):
    lens, news = [300, 400, 500, 20], [40, 50, 60, 20]
    c = Cache(lens, 2, d, 16, 7, e4m3)
    q, cu = ragged(news, 8, d, 1)
    args = dict(k_scale=c.k_scale, v_scale=c.v_scale)
    for bad in (-1, 10 ** 6, -(10 ** 9)):
        table = c.table.clone()
        table[1, 3] = bad
        o, lse = bss.attn_fwd_paged(q, c.k, c.v, table, c.lens, ints(cu), **args)
        assert bss.attn_poll_status() == BAD_PAGES
        check_rows(q, o, lse, c, lens, news, cu, skip=(1,))
        # a bad entry's keys are left out
        keep = torch.ones(400, dtype=torch.bool, device="cuda")
        keep[48:64] = False
        mask = ref.window_mask(50, 400, 400, 0, 350, 0, "cuda")[:, keep]
        w = (q[cu[1]:cu[2]].transpose(0, 1)[None], c.k64[1][None, :, keep], c.v64[1][None, :, keep], mask,
             1.0 / math.sqrt(d))
        O, L, _ = ref.forward(*w)
        bo, bl = ref.forward_bounds(*w)
        assert ((o[cu[1]:cu[2]].transpose(0, 1)[None].double() - O).abs() <= bo).all()
        assert ((lse[cu[1]:cu[2]].transpose(0, 1)[None].double() - L).abs() <= bl).all()
    # past the last token nothing is looked at
    table = c.table.clone()
    table[0, 19:] = 10 ** 6
    o, lse = bss.attn_fwd_paged(q, c.k, c.v, table, c.lens, ints(cu), **args)
    assert bss.attn_poll_status() == 0
    check_rows(q, o, lse, c, lens, news, cu)


def test_chunk_reports_bad_lengths(bss):
    lens, news = [300, 40, 50], [40, 40, 50]
    c = Cache(lens, 2, 128, 16, 7)
    q, cu = ragged(news, 8, 128, 1)
    # more new tokens than the sequence has: the first 15 rows stand before its first token
    n = ints([300, 25, 50])
    o, lse = bss.attn_fwd_paged(q, c.k, c.v, c.table, n, ints(cu))
    assert bss.attn_poll_status() == BAD_PAGES
    assert (o[40:55] == 0).all() and torch.isneginf(lse[40:55]).all()
    check_rows(q, o, lse, c, lens, news, cu, skip=(1,))
    c.k64[1], c.v64[1] = c.k64[1][:, :25], c.v64[1][:, :25]
    check_rows(q, o, lse, c, [300, 25, 50], [0, 25, 0], [40, 55, 80])
    for bad in (-3, 10 ** 6, 0x7FFFFFFF, -0x80000000):
        o, lse = bss.attn_fwd_paged(q, c.k, c.v, c.table, ints([300, bad, 50]), ints(cu))
        assert bss.attn_poll_status() == BAD_PAGES
        check_rows(q, o, lse, c, lens, news, cu, skip=(1,))


def test_offsets_in_disorder_are_refused(bss):
    """... on the device: nothing is written, and it is reported; the selection's rows each find some
    sequence or none."""
    c = Cache([300, 40, 50], 2, 128, 16, 7)
    q, _ = ragged([40, 40, 50], 8, 128, 1)
    o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 3.0, device="cuda")
    means = torch.zeros(c.k.shape[0], 2, 128, device="cuda")
    for cu in ([0, 90, 40, 130], [130, 90, 40, 0], [-5, 40, 80, 10 ** 6], [0, 0, 0, 0],
               [-2 ** 31, 2 ** 31 - 1, -1, 7]):
        bss.attn_fwd_paged(q, c.k, c.v, c.table, c.lens, ints(cu), out=o, lse=lse)
        if cu != sorted(cu):
            assert bss.attn_poll_status() == BAD_PAGES
            assert (o == 7.0).all() and (lse == 3.0).all()
        elif cu == [0, 0, 0, 0]:
            assert bss.attn_poll_status() == 0 and (o == 7.0).all()
        else:                                            # more new tokens than there are
            assert bss.attn_poll_status() == BAD_PAGES
            o.fill_(7.0), lse.fill_(3.0)
        pages, lens = bss.attn_select_pages(q, means, c.table, c.lens, ints(cu), 3, 16)
        bss.attn_decode_selected(q, c.k, c.v, pages, lens)
        torch.cuda.synchronize()
        bss.attn_poll_status()


@pytest.mark.parametrize("e4m3", [False, True])
def test_chunk_in_a_graph_and_on_streams(bss, e4m3):
    """A captured call follows the lengths, and two calls may run at once."""
    lens, news = [700, 2000], [100, 30]
    c = Cache(lens, 2, 128, 16, 3, e4m3)
    q, cu = ragged([130, 130], 8, 128, 2)
    n, b = ints([0, 0]), ints([0, 0, 0])
    nbytes = bss.attn_fwd_paged_workspace_bytes(260, 2, 8, 2, 128, c.table.shape[1], 16)
    ws = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [(torch.empty_like(q), torch.empty(260, 8, device="cuda")) for _ in range(2)]
    args = dict(k_scale=c.k_scale, v_scale=c.v_scale)
    side = [torch.cuda.Stream() for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side[0]):
        bss.attn_fwd_paged(q, c.k, c.v, c.table, n, b, workspace=ws[0], out=outs[0][0], lse=outs[0][1], **args)
        side[0].synchronize()
        with torch.cuda.graph(graph, stream=side[0]):
            bss.attn_fwd_paged(q, c.k, c.v, c.table, n, b, workspace=ws[0], out=outs[0][0],
                               lse=outs[0][1], **args)
    torch.cuda.synchronize()
    for news in ([100, 30], [1, 130], [130, 0]):
        cu = [0, news[0], sum(news)]
        n.copy_(ints(lens))
        b.copy_(ints(cu))
        torch.cuda.synchronize()
        with torch.cuda.stream(side[1]):
            bss.attn_fwd_paged(q, c.k, c.v, c.table, n, b, workspace=ws[1], out=outs[1][0],
                               lse=outs[1][1], **args)
        graph.replay()
        torch.cuda.synchronize()
        assert bss.attn_poll_status() == 0
        for o, lse in outs:
            check_rows(q, o, lse, c, lens, news, cu)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_of_large_scores(bss, d, e4m3):
    """Scores of some thousands, rows whose keys all score far below 0, zeros; the smallest and the
    largest numbers; rows with an element that is hundreds of times the others."""
    c = Cache([500, 64], 2, d, 16, 3, e4m3)
    q, cu = ragged([100, 64], 4, d, 2)
    for f in (60.0, -60.0, 0.0, 2.0 ** -130, 2.0 ** -100):
        check_chunk(bss, c, (q.float() * f).bfloat16(), cu, [500, 64], [100, 64])
    check_chunk(bss, c, (q.float() * 2.0 ** 100).bfloat16(), cu, [500, 64], [100, 64], scale=2.0 ** -103)
    check_chunk(bss, c, (q.float() * 2.0 ** -100).bfloat16(), cu, [500, 64], [100, 64], scale=2.0 ** -120)
    for at in (0, d - 1):
        far = q.clone()
        far[::2, :, at] = 700.0
        far[1::4, :, at] = -90.0
        check_chunk(bss, c, far, cu, [500, 64], [100, 64])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_numbers_that_are_not_finite(bss, d, e4m3):
    """A NaN among the keys reaches the rows that see it, one among the values its own column of the
    rows of its 128 keys' block and later; other sequences are as they were."""
    lens, news = [300, 200], [40, 60]
    c = Cache(lens, 2, d, 16, 7, e4m3)
    q, cu = ragged(news, 8, d, 1)
    args = dict(k_scale=c.k_scale, v_scale=c.v_scale)
    kind = c.k.dtype
    bits = torch.tensor([0xFF if e4m3 else 0x7FC0], device="cuda", dtype=torch.int32)
    nan = bits.to(torch.uint8 if e4m3 else torch.int16).view(kind)[0]
    page = c.table[1, 50 // 16].item()

    def planted(x, h, col):
        y = x.view(torch.uint8 if e4m3 else torch.int16).clone()
        y[page, h, 50 % 16, col] = nan.view(torch.uint8 if e4m3 else torch.int16)
        return y.view(kind)

    o, lse = bss.attn_fwd_paged(q, c.k, planted(c.v, 0, 5), c.table, c.lens, ints(cu), **args)
    check_rows(q, o, lse, c, lens, news, cu, skip=(1,))
    hit = o[cu[1]:].isnan()
    assert hit[:, :4, 5].all() and hit.sum() == hit[:, :4, 5].numel() and lse.isfinite().all()
    o, lse = bss.attn_fwd_paged(q, planted(c.k, 1, d - 1), c.v, c.table, c.lens, ints(cu), **args)
    check_rows(q, o, lse, c, lens, news, cu, skip=(1,))
    assert o[cu[1]:, 4:].isnan().all() and lse[cu[1]:, 4:].isnan().all()
    assert o[cu[1]:, :4].isfinite().all()
    assert bss.attn_poll_status() == 0


def test_far_pages(bss):
    """Pages past 4 GB of the cache, and row offsets of q past 32 bits of bytes."""
    P, page = 70000, 256
    kc = torch.zeros(P, 1, page, 128, device="cuda", dtype=torch.bfloat16)
    vc = torch.zeros_like(kc)
    c = Cache([600], 1, 128, page, 8)
    table = ints([[P - 1, P - 2, P - 3]])
    for m in range(3):
        x = c.table[0, m].item()
        kc[P - 1 - m], vc[P - 1 - m] = c.k[x], c.v[x]
    q, cu = ragged([200], 4, 128, 2)
    o, lse = bss.attn_fwd_paged(q, kc, vc, table, ints([600]), ints(cu))
    assert bss.attn_poll_status() == 0
    check_rows(q, o, lse, c, [600], [200], cu)
    means = torch.zeros(P, 1, 128, device="cuda")
    bss.attn_kv_pool(kc, means, table, ints([0]), ints([600]))
    assert torch.equal(means[P - 2:].double().flip(0), page_means(c.k64[0], page)[:2].float().double())
    pages, lens = bss.attn_select_pages(q, means, table, ints([600]), ints(cu), 2, page)
    o2, lse2 = bss.attn_decode_selected(q, kc, vc, pages, lens)
    assert bss.attn_poll_status() == 0
    check_rows(q, o2, lse2, c, [600], [200], cu)         # all of its pages


# ----------------------------------------------------------------------------
# mean keys
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,page,Hkv", [(128, 16, 3), (64, 16, 1), (128, 64, 4), (64, 128, 2), (128, 1024, 1)])
def test_pool(bss, d, page, Hkv, e4m3):
    lens = [5 * page + 3, 0, page, page - 1, 2 * page, 9 * page]
    start = [0, 0, 0, 0, page + 1, 4 * page - 1]
    c = Cache(lens, Hkv, d, page, 5, e4m3, inter=True)
    c.table = torch.cat([c.table, torch.full_like(c.table[:1], 10 ** 6)])      # a row that start does not name
    means = torch.full((c.k.shape[0], Hkv, d), 5.0, device="cuda")
    want = means.double()
    for s, n in enumerate(lens):
        for m in range(start[s] // page, n // page):
            want[c.table[s, m]] = page_means(c.k64[s], page)[m]
    c.table[5, 6] = -1                                   # given back
    bss.attn_kv_pool(c.k, means, c.table, ints(start), torch.cat([c.lens, ints([7])]), k_scale=c.k_scale)
    assert bss.attn_poll_status() == 0
    lost = (want - 5.0).abs().sum((1, 2)) * (means - 5.0).abs().sum((1, 2)) == 0
    assert lost.sum() == c.k.shape[0] - sum(n // page - a // page for n, a in zip(lens, start)) + 1
    assert ((means.double() - want).abs() <= 2.0 ** -24 * want.abs())[~lost].all()


def test_pool_of_numbers_that_cancel(bss):
    """A mean whose sum loses everything in 32 bits, the largest numbers, infinities and NaN."""
    page = 16
    k = torch.zeros(3, 1, page, 64, device="cuda", dtype=torch.bfloat16)
    k[0, 0, 0], k[0, 0, 7], k[0, 0, 9], k[0, 0, 15] = 2.0 ** 60, 3.0, -(2.0 ** 60), 2.0 ** -10
    k[1] = torch.finfo(torch.bfloat16).max
    k[2, 0, 3, 0], k[2, 0, 4, 1], k[2, 0, 5, 2], k[2, 0, 6, 2] = math.inf, math.nan, math.inf, -math.inf
    means = torch.zeros(3, 1, 64, device="cuda")
    bss.attn_kv_pool(k, means, ints([[0, 1, 2]]), ints([0]), ints([48]))
    assert (means[0] == (3.0 + 2.0 ** -10) / 16).all()
    assert (means[1] == torch.finfo(torch.bfloat16).max).all()
    assert means[2, 0, 0] == math.inf and means[2, 0, 1:3].isnan().all() and (means[2, 0, 3:] == 0).all()


def test_pool_reports_bad_pages(bss):
    c = Cache([64, 64], 1, 64, 16, 5)
    means = torch.full((c.k.shape[0], 1, 64), 5.0, device="cuda")
    table = c.table.clone()
    table[0, 1] = 10 ** 6
    bss.attn_kv_pool(c.k, means, table, ints([0, 0]), c.lens)
    assert bss.attn_poll_status() == BAD_PAGES
    assert (means[c.table[1, :4].long()] != 5.0).any(-1).all() and (means[c.table[0, 1].long()] == 5.0).all()
    for n in (-1, 10 ** 6):
        bss.attn_kv_pool(c.k, means, c.table, ints([0, 0]), ints([64, n]))
        assert bss.attn_poll_status() == BAD_PAGES
    bss.attn_kv_pool(c.k, means, table, ints([-1, 0]), c.lens)      # nothing was reserved there
    assert bss.attn_poll_status() == 0


# ----------------------------------------------------------------------------
# selection, and attention over it
# ----------------------------------------------------------------------------

def select_and_check(bss, q, means, table, lens, cu, news, top, page, local, first, **kw):
    pages, got = bss.attn_select_pages(q, means, table, ints(lens), ints(cu), top, page, local_pages=local,
                                       first_pages=first, **kw)
    assert bss.attn_poll_status() == 0
    want, n = select_pages(q, means, table, lens, cu, news, top, page, local, first)
    assert torch.equal(pages.cpu(), want) and torch.equal(got.cpu(), n)
    return pages, got


SELECT = [
    # lens, new tokens, H, Hkv, d, page, top, local, first
    ([1], [1], 1, 1, 128, 16, 1, 1, 0),
    ([300], [1], 16, 4, 128, 16, 3, 2, 1),
    ([17, 0, 200, 640, 129, 128], [17, 0, 1, 64, 1, 128], 8, 2, 128, 16, 2, 1, 0),
    ([5, 1000, 33, 257, 0, 64], [5, 130, 33, 1, 0, 3], 6, 2, 64, 64, 0, 2, 2),
    ([777, 12, 2049], [300, 12, 65], 16, 1, 128, 32, 7, 3, 1),
    ([20011, 900], [1, 1], 2, 1, 128, 16, 100, 8, 1),
    ([9000], [21], 4, 4, 64, 16, 33, 1, 0),
    ([500, 31], [10, 3], 33, 1, 64, 32, 40, 1, 3),      # more than there are
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,news,H,Hkv,d,page,top,local,first", SELECT)
def test_select_and_decode(bss, lens, news, H, Hkv, d, page, top, local, first, e4m3):
    c = Cache(lens, Hkv, d, page, sum(lens) + H, e4m3)
    q, cu = ragged(news, H, d, H + len(lens), before=2, after=3)
    means = torch.full((c.k.shape[0], Hkv, d), float("nan"), device="cuda")
    bss.attn_kv_pool(c.k, means, c.table, ints([0] * len(lens)), c.lens, k_scale=c.k_scale)
    pages, n = select_and_check(bss, q, means, c.table, lens, cu, news, top, page, local, first)
    assert (n[:2] == -1).all() and (n[-3:] == -1).all()
    o = torch.full((q.shape[0], H, d), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((q.shape[0], H), 3.0, device="cuda")
    # a table with little room takes a block per K/V head, a wide one shares all steps evenly
    for columns in (0, 1100 // page):
        wide = torch.cat([pages, pages.new_full((q.shape[0], Hkv, columns), -1)], 2).contiguous()
        bss.attn_decode_selected(q, c.k, c.v, wide, n, k_scale=c.k_scale, v_scale=c.v_scale, out=o, lse=lse)
        torch.cuda.synchronize()
        assert bss.attn_poll_status() == 0
        for x, v in ((o, 7.0), (lse, 3.0)):
            assert (x[:2] == v).all() and (x[-3:] == v).all()
        G = H // Hkv
        place = {x: (s, m) for s in range(len(lens)) for m, x in enumerate(c.table[s].tolist()) if x >= 0}
        rng = random.Random(1)
        for t in rng.sample(range(2, 2 + sum(news)), min(12, sum(news))):
            for h in range(Hkv):
                keys, s = [], None
                for x in pages[t, h].tolist():
                    if x >= 0:
                        s, m = place[x]
                        keys += range(m * page, (m + 1) * page)
                keys = keys[:n[t].item()]
                mask = torch.ones(1, len(keys), dtype=torch.bool, device="cuda")
                args = (q[t, h * G:(h + 1) * G][None, :, None], c.k64[s][h, keys][None, None],
                        c.v64[s][h, keys][None, None], mask, 1.0 / math.sqrt(d))
                O, L, _ = ref.forward(*args)
                bo, bl = ref.forward_bounds(*args)
                assert ((o[t, h * G:(h + 1) * G].double() - O[0, :, 0]).abs() <= bo[0, :, 0]).all(), (t, h)
                assert ((lse[t, h * G:(h + 1) * G].double() - L[0, :, 0]).abs() <= bl[0, :, 0]).all(), (t, h)


def test_every_page_selected_is_decoding(bss):
    lens = [700, 33, 0, 64]
    c = Cache(lens, 2, 128, 16, 4)
    q = torch.randn(4, 8, 128, device="cuda").bfloat16()
    means = torch.zeros(c.k.shape[0], 2, 128, device="cuda")
    pages, n = bss.attn_select_pages(q[[0, 1, 3]], means, c.table, c.lens, ints([0, 1, 2, 2, 3]), 60, 16)
    assert n.tolist() == [700, 33, 64]
    o, lse = bss.attn_decode_selected(q[[0, 1, 3]], c.k, c.v, pages, n)
    od, ld = bss.attn_decode_paged(q, c.k, c.v, c.table, c.lens)
    assert (o.float() - od[[0, 1, 3]].float()).abs().max() <= 2.0 ** -7
    assert (lse - ld[[0, 1, 3]]).abs().max() <= 1e-5


@pytest.mark.parametrize("rows,n", [(3, 40), (70, 40), (2, 300), (20, 300)])
def test_ties_and_near_ties(bss, rows, n):
    """Equal scores go to the lower place; scores that 32 bits cannot tell apart are told apart."""
    page, d = 16, 128
    g = torch.Generator("cuda").manual_seed(rows + n)
    table = torch.randperm(n, generator=g, device="cuda").int()[None]
    base = torch.randn(1, d, generator=g, device="cuda")
    means = base.repeat(n, 1)[:, None].contiguous()                  # all alike
    q = torch.randn(rows, 4, d, generator=g, device="cuda").bfloat16()
    # the first token of the last page and those after it, or before it
    args = ([n * page - 15 + rows % 16], [0, rows], [rows])
    pages, _ = select_and_check(bss, q, means, table, *args, 5, page, 1, 0)
    assert torch.equal(pages[-1, 0], table[0, [0, 1, 2, 3, 4, n - 1]])
    for step in (2.0 ** -23, 2.0 ** -22, 2.0 ** -18, 2.0 ** -12):
        # one element of each differs by a few units of its last place: sums that round alike
        near = means.clone()
        units = torch.randint(-3, 4, (n,), generator=g, device="cuda")
        col = torch.randint(0, d, (n,), generator=g, device="cuda")
        near[torch.arange(n), 0, col] *= 1 + step * units
        for top in (1, 7, 20):
            select_and_check(bss, q, near, table, *args, top, page, 1, 0)
    # a group whose heads cancel: the sum's own rounding
    q2 = torch.cat([q[:, :2] * 256, -q[:, :2] * 256 + q[:, 2:]], 1)
    mixed = means + torch.randn(n, 1, d, generator=g, device="cuda") * 1e-3
    for top in (1, 7, 20):
        select_and_check(bss, q2, mixed, table, *args, top, page, 1, 0)
    # all of them 0
    select_and_check(bss, q * 0, mixed, table, *args, 7, page, 1, 0)


def test_scores_that_are_not_finite(bss):
    page, d, n = 16, 64, 30
    table = torch.arange(n, device="cuda").int()[None]
    means = torch.randn(n, 1, d, device="cuda")
    means[3, 0, 5], means[9, 0, 7], means[4, 0, 2] = math.nan, math.inf, -math.inf
    q = torch.ones(1, 2, d, device="cuda").bfloat16()
    for top in (1, 5, 27, 28, 29):
        pages, _ = bss.attn_select_pages(q, means, table, ints([n * page]), ints([0, 1]), top, page)
        score = (means[:29, 0].double() @ q[0].double().sum(0)).tolist()
        order = sorted(range(29), key=lambda m: (score[m] != score[m], -score[m] if score[m] == score[m] else 0, m))
        assert pages[0, 0].tolist() == sorted(order[:top]) + [n - 1]
    assert bss.attn_poll_status() == 0


def test_pages_given_back_are_not_selected(bss):
    lens, page = [400], 16
    c = Cache(lens, 2, 64, page, 4)
    q, cu = ragged([3], 4, 64, 1)
    means = torch.randn(c.k.shape[0], 2, 64, device="cuda")
    c.table[0, [0, 3, 7, 8, 22]] = -1
    select_and_check(bss, q, means, c.table, lens, cu, [3], 5, page, 4, 2)
    select_and_check(bss, q, means, c.table, lens, cu, [3], 50, page, 4, 2)
    for bad in (10 ** 6, -7):
        c.table[0, 5] = bad
        bss.attn_select_pages(q, means, c.table, ints(lens), ints(cu), 5, page)
        assert bss.attn_poll_status() == BAD_PAGES
    # decoding reports what it is given, and leaves it out
    pages = ints([[[c.table[0, 1], 10 ** 6]] * 2])
    bss.attn_decode_selected(q[:1], c.k, c.v, pages, ints([20]))
    assert bss.attn_poll_status() == BAD_PAGES
    bss.attn_decode_selected(q[:1], c.k, c.v, pages, ints([33]))
    assert bss.attn_poll_status() == BAD_PAGES


def test_rows_in_several_launches(bss):
    """More scores than the workspace holds at once."""
    n, page, d = 30000, 16, 64
    T = 2400                                             # 2400 rows of 30000 slots: two launches
    table = torch.randperm(n, device="cuda").int()[None]
    means = torch.randn(n, 1, d, device="cuda")
    q = torch.randn(T, 1, d, device="cuda").bfloat16()
    pages, lens = bss.attn_select_pages(q, means, table, ints([n * page]), ints([0, T]), 20, page)
    assert bss.attn_poll_status() == 0
    rows = [0, 1, 1000, 2231, 2232, 2233, 2239, 2240, 2399]
    ends = [n * page - T + 1 + r for r in rows]
    for r, end in zip(rows, ends):
        want, m = select_pages(q[r:r + 1], means, table, [end], [0, 1], [1], 20, page, 1, 0)
        assert torch.equal(pages[r].cpu(), want[0]) and lens[r].item() == m[0].item()


def test_a_step_of_a_server(bss):
    """Reserve, write, pool, then a dense layer and a sparse one, step after step, in one cache; the
    sparse layer's summaries survive forks and compaction."""
    S, H, Hkv, d, page, P = 6, 8, 2, 128, 16, 400
    g = torch.Generator("cuda").manual_seed(3)
    kc = torch.full((P, Hkv, page, d), float("nan"), device="cuda", dtype=torch.bfloat16)
    vc = kc.clone()
    means = torch.full((P, Hkv, d), float("nan"), device="cuda")
    table = torch.full((S, 40), -1, dtype=torch.int32, device="cuda")
    lens, refs = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (S, P))

    class Seen:
        k64 = [torch.zeros(Hkv, 0, d, device="cuda", dtype=torch.float64) for _ in range(S)]
        v64 = [x.clone() for x in k64]

    rng = random.Random(2)
    have = [0] * S
    for step in range(7):
        if step == 4:                                    # the second goes on as the sixth, too
            bss.attn_kv_free(table, lens, refs, ints([5]), page)
            src, dst = bss.attn_kv_fork(table, lens, refs, ints([1]), ints([5]), page)
            bss.attn_kv_copy_pages(kc, vc, src, dst)
            Seen.k64[5], Seen.v64[5], have[5] = Seen.k64[1], Seen.v64[1], have[1]
        if step == 5:
            src, dst, count = bss.attn_kv_compact(table, refs)
            bss.attn_kv_copy_pages(kc, vc, src, dst, count)
            means.fill_(float("nan"))
            bss.attn_kv_pool(kc, means, table, torch.zeros_like(lens), lens)
        news = [rng.choice([0, 1, 1, 40, 70]) for _ in range(S)]
        q, cu = ragged(news, H, d, step, after=4)
        T = q.shape[0]
        k, v = (torch.randn(T, Hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2))
        start = bss.attn_kv_reserve(table, lens, refs, ints(news), page)
        bss.attn_kv_write(k, v, kc, vc, table, start, ints(cu))
        bss.attn_kv_pool(kc, means, table, start, lens)
        for s, n in enumerate(news):
            have[s] += n
            Seen.k64[s] = torch.cat([Seen.k64[s], k[cu[s]:cu[s + 1]].transpose(0, 1).double()], 1)
            Seen.v64[s] = torch.cat([Seen.v64[s], v[cu[s]:cu[s + 1]].transpose(0, 1).double()], 1)
        o, lse = bss.attn_fwd_paged(q, kc, vc, table, lens, ints(cu))
        assert bss.attn_poll_status() == 0
        check_rows(q, o, lse, Seen, have, news, cu)
        pages, n = select_and_check(bss, q, means, table, have, cu, news, 2, page, 1, 1)
        o, lse = bss.attn_decode_selected(q, kc, vc, pages, n)
        pages, n = select_and_check(bss, q, means, table, have, cu, news, 40, page, 1, 1)
        o, lse = bss.attn_decode_selected(q, kc, vc, pages, n)      # every page: as the dense layer
        assert bss.attn_poll_status() == 0
        check_rows(q, o, lse, Seen, have, news, cu)


def test_selection_in_a_graph(bss):
    lens = [700, 300]
    c = Cache(lens, 2, 128, 16, 3)
    q, _ = ragged([20, 20], 8, 128, 2)
    means = torch.zeros(c.k.shape[0], 2, 128, device="cuda")
    n, b, start = ints(lens), ints([0, 20, 40]), ints([0, 0])
    bss.attn_kv_pool(c.k, means, c.table, start, n)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()

    def call():
        bss.attn_kv_pool(c.k, means, c.table, start, n)
        pages, m = bss.attn_select_pages(q, means, c.table, n, b, 4, 16)
        return (pages, m) + bss.attn_decode_selected(q, c.k, c.v, pages, m)

    with torch.cuda.stream(side):
        call()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out = call()
    for cu in ([0, 20, 40], [0, 1, 2], [3, 30, 31]):
        b.copy_(ints(cu))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = call()
        for x, y in zip(out[:2], want[:2]):
            assert torch.equal(x, y)
        for x, y in zip(out[2:], want[2:]):
            assert torch.equal(x[cu[0]:cu[2]], y[cu[0]:cu[2]])
    assert bss.attn_poll_status() == 0


# (equal prompts: the last turn's tiles are cut once more; 60 tiles a K/V head of whole ones, of ones
# that are cut already, and beside sequences of a few keys; with and without a window)
TAIL = [
    ([9000] * 3, [1900, 1920, 1900], 8, 2, 128, 0, 0),
    ([4200] * 4 + [3, 900, 0], [1024] * 4 + [1, 1, 0], 16, 4, 128, 0, 0),
    ([6000] * 5, [1100] * 5, 8, 8, 64, 2500, 3),
    ([20000], [2600], 8, 2, 64, 0, 0),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,news,H,Hkv,d,window,sinks", TAIL)
def test_chunk_of_equal_tiles(bss, lens, news, H, Hkv, d, window, sinks, e4m3):
    c = Cache(lens, Hkv, d, 64, d + Hkv, e4m3)
    q, cu = ragged(news, H, d, 4)
    check_chunk(bss, c, q, cu, lens, news, window=window, sinks=sinks)


@pytest.mark.parametrize("S", [257, 1300])
def test_chunk_of_many_sequences(bss, S):
    """More sequences than the plan sorts, and than it has threads; a few of them long."""
    rng = random.Random(S)
    lens = [rng.choice([0, 1, 17, 40]) for _ in range(S)]
    news = [min(n, rng.choice([0, 1, 1, 3])) for n in lens]
    for s, n, new in ((5, 9000, 70), (S // 2, 2500, 300), (S - 1, 9000, 1)):
        lens[s], news[s] = n, new
    c = Cache(lens, 2, 64, 32, S)
    q, cu = ragged(news, 8, 64, 5)
    check_chunk(bss, c, q, cu, lens, news)


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_launch_after_a_timeout_stops(bss, e4m3):
    """With a timeout in the status word a launch stops, block by block, with parts to be joined or
    without, and leaves its outputs; once the word is read and cleared the same call is right."""
    for lens, news in (([300, 40], [5, 40]), ([9000], [300])):
        c = Cache(lens, 2, 128, 16, 9, e4m3)
        q, cu = ragged(news, 8, 128, 2)
        o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 3.0, device="cuda")
        bss.attn_watchdog_selftest(1 << 16)
        for _ in range(2):
            bss.attn_fwd_paged(q, c.k, c.v, c.table, c.lens, ints(cu), k_scale=c.k_scale, v_scale=c.v_scale,
                               out=o, lse=lse)
        assert bss.attn_poll_status() == bss.ERR_TIMEOUT
        assert (o == 7.0).all() and (lse == 3.0).all()
        check_chunk(bss, c, q, cu, lens, news)
