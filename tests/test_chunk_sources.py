"""What the chunk kernel does once a bounded wait has run out, read off its source (no GPU): the roles
of whole warps take the same way with all of their lanes, or those that stay wait for the others at
the next vote without end; and the oracle of the selection against plain counting."""
import os
import re

import torch

from oracle.select import page_means, select_pages

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_sparse_softmax_gb300", "csrc")


def spans(text, name):
    """Where the arguments of every call of `name` begin and end."""
    for m in re.finditer(name + r"\(", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        yield m.end(), at


def test_a_warp_of_the_chunk_kernel_leaves_a_wait_as_one():
    with open(os.path.join(CSRC, "chunk.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    begin = text.index("attn_fwd_paged_kernel(")
    text = text[begin:text.index("chunk_join_kernel(")]
    mma = text.index("if (elect_one()) {", text.index("warp == 13")), text.index("warp == 14")   # one thread
    votes = list(spans(text, "__all_sync"))
    waits = [m.start() for m in re.finditer(r"\bwait_bar(_relaxed)?\(", text)]
    assert len(waits) >= 15
    for at in waits:
        if mma[0] <= at < mma[1] or any(a <= at < b for a, b in votes):
            continue
        # the outcome is kept, and voted on before anybody leaves
        statement = max(text.rfind(c, 0, at) for c in ";{}")
        assert re.search(r"\bfine = ", text[statement:at]), text[statement:at + 60]
        vote = text.index("__all_sync(0xFFFFFFFFu, fine)", at)
        between = text[at:vote]
        between = between[:between.rfind("return")] if between.rstrip().endswith("return") else between
        assert not re.search(r"\b(break|return|continue)\b", between), between


def test_page_means_and_selected_pages_by_hand():
    k = torch.arange(2 * 7 * 4, dtype=torch.float64).reshape(2, 7, 4)
    m = page_means(k, 2)
    assert m.shape == (3, 2, 4) and m[1, 1].tolist() == ((k[1, 2] + k[1, 3]) / 2).tolist()
    # one K/V head, two query heads: the pages' scores are those of the heads' sum
    means = torch.tensor([[[1.0]], [[5.0]], [[3.0]], [[5.0]], [[9.0]], [[float("nan")]]])
    table = torch.tensor([[4, 3, 2, 1, 0, -1], [5, 4, -1, 0, 1, 2]])
    q = torch.tensor([[[2.0], [-1.0]], [[1.0], [1.0]], [[-1.0], [0.0]], [[7.0], [7.0]]])
    # rows 1 and 2 of the batch are the last of 20 tokens in pages of 4, row 3 of 23 of the second
    pages, lens = select_pages(q, means, table, [20, 23], [1, 3, 4], [2, 1], 2, 4, 1, 1)
    assert lens.tolist() == [-1, 15, 16, 15]
    assert pages[1, 0].tolist() == [4, 3, 1, 0]       # 5 at places 1 and 3 beats 3
    assert pages[2, 0].tolist() == [4, 2, 1, 0] or pages[2, 0].tolist() == [4, 3, 2, 0]
    assert pages[0].eq(-1).all()
    # ties go to the lower place: scores -5, -3, -5 at places 1, 2, 3
    assert pages[2, 0].tolist() == [4, 3, 2, 0]
    # the second sequence: places 0 and 5 anyway, of 1, 3, 4 the pages 4 (126) and 1 (70)
    assert pages[3, 0].tolist() == [5, 4, 1, 2]


def test_chosen_pages_are_the_best_ones():
    g = torch.Generator().manual_seed(1)
    q, means = torch.randn(5, 4, 8, generator=g), torch.randn(40, 2, 8, generator=g)
    table = torch.randperm(40, generator=g)[None]
    pages, lens = select_pages(q, means, table, [40 * 16], [0, 5], [5], 7, 16, 2, 1)
    for t in range(5):
        for h in range(2):
            x = (q[t, 2 * h:2 * h + 2].sum(0).double() * means[:, h].double()).sum(1)
            chosen = set(pages[t, h].tolist())
            rest = [p for m, p in enumerate(table[0].tolist()) if 1 <= m < 38]
            best = sorted(rest, key=lambda p: -x[p])[:7]
            assert chosen == set(best) | {table[0, i].item() for i in (0, 38, 39)}
        assert lens[t].item() == 9 * 16 + 16 - (4 - t)
