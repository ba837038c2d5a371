"""What a kernel does once a bounded wait has run out, read off the sources (no GPU): a block has to
take the same way with all of its warps, and a warp with all of its lanes, or those that stay wait
for the others at the next barrier or vote without end."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_sparse_softmax_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh"))))
def test_a_block_reads_the_timeout_as_one(name):
    """The status word decides whether a block goes on only by way of a vote of the whole block."""
    text = source(name)
    for m in re.finditer(r"== *ATTN_ERR_TIMEOUT", text):
        line = text[text.rfind("\n", 0, m.start()) + 1:text.find("\n", m.end())]
        assert "__syncthreads_or(" in line, line.strip()


# where the roles of whole warps begin in each kernel (the others' waits are one lane's)
WHOLE_WARPS = {"window_fwd.cu": "regs_set<kWinOut", "window_bwd.cu": "regs_set<WinBwdRegs<D>::kMid",
               "bwd.cu": "regs_set<BwdRegs<D>::kMid", "fwd.cu": "regs_set<FwdRegs<SPARSE>::kHigh",
               "fwd_wide.cu": "regs_set<kWideHigh"}


def votes(text):
    """The spans of the arguments of every __all_sync."""
    for m in re.finditer(r"__all_sync\(", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        yield m.end(), at


@pytest.mark.parametrize("name", sorted(WHOLE_WARPS))
def test_a_warp_leaves_a_wait_as_one(name):
    """The roles of whole warps vote on every bounded wait's outcome, at the wait, or (`fine`) at
    the end of the tile or round, up to where nobody leaves."""
    text = source(name)
    begin = text.index(WHOLE_WARPS[name])
    text = text[begin:text.index("tmem_dealloc", begin)]
    spans = list(votes(text))
    waits = [m.start() for m in re.finditer(r"\bwait_bar(_relaxed)?\(", text)]
    assert len(waits) >= 4
    for at in waits:
        line = text[text.rfind("\n", 0, at):text.find("\n", at)].strip()
        if any(a <= at < b for a, b in spans):
            continue
        statement = max(text.rfind(c, 0, at) for c in ";{}")
        assert re.search(r"\bfine = ", text[statement:at]), line
        vote = text.index("__all_sync(0xFFFFFFFFu, fine)", at)
        assert not re.search(r"\b(break|return|continue)\b", text[at:vote]), line
