"""The kernels that fill LDS rings by direct loads let other waves overwrite a
slot after a barrier: before it, every wave has to have waited for its own LDS
reads.  The builtin barrier, unlike __syncthreads(), waits for nothing by itself,
and no test on a GPU shows such a wait's absence reliably, so the sources are
read: the waits before every builtin barrier inside a ring's loop have to count
LDS operations down to zero.  (In a wait's number vmcnt is in bits 3:0 and
15:14, expcnt in 6:4, lgkmcnt in 11:8.)
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "structured_sparse_transformer_amd", "csrc")
WAIT = re.compile(r"__builtin_amdgcn_s_waitcnt\(([^;]*)\);")


def lgkmcnt(expression):
    """The field of a wait's number, terms without names alone."""
    number = 0
    for term in expression.split("|"):
        term = term.strip()
        while term.startswith("(") and term.endswith(")"):
            term = term[1:-1].strip()
        if re.search("[A-Za-z]", term.replace("0xF", "")):   # the load count's bits, of vmcnt
            continue
        number |= eval(term)   # noqa: S307  numbers and shifts
    return number >> 8 & 15


def test_the_field_is_read():
    assert lgkmcnt("4 | (7 << 4) | (15 << 8)") == 15 and lgkmcnt("0 | (7 << 4) | (0 << 8)") == 0
    assert lgkmcnt("0xF | (7 << 4) | (0 << 8) | (3 << 14)") == 0
    assert lgkmcnt("(n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8)") == 15


# source, the text that opens the ring's loop, the text after it
LOOPS = [("sp24_spmm_loop.inc", "auto stage = [&]", "static_assert(kSlots == 2"),
         ("sp24_linear.hip", "for (int j = 0; j < rounds; ++j) {", "if constexpr (kTail) {"),
         ("sp24_dw.hip", "__builtin_amdgcn_s_barrier();\n", "__syncthreads();   // the mask table"),
         ("sp24_ns.hip", "__builtin_amdgcn_s_barrier();\n", "__syncthreads();   // the ring is idle")]


@pytest.mark.parametrize("name,opening,closing", LOOPS, ids=[n for n, _, _ in LOOPS])
def test_reads_are_waited_for_before_a_slot_is_free(name, opening, closing):
    text = open(os.path.join(CSRC, name)).read()
    start = text.index(opening) + len(opening)
    text = text[start: text.index(closing, start)]
    before = text.split("__builtin_amdgcn_s_barrier();")[:-1]
    assert before
    for part in before:
        # the last wait, or both sides of an if and else
        waits = [(m.start(), lgkmcnt(m.group(1))) for m in WAIT.finditer(part)]
        assert waits
        last = waits[-2:] if re.search(r"\belse\s*$", part[: waits[-1][0]]) else waits[-1:]
        assert all(field == 0 for _, field in last), part[-400:]
