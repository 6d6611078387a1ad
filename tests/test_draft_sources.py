"""Rules that the kernels for drafted tokens keep in their sources; no GPU."""
from __future__ import annotations

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_command_execution_gb300", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _block(text, at):
    """The text between the brace at or behind `at` and the one that ends it."""
    begin = text.index("{", at)
    depth = 0
    for i in range(begin, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[begin + 1:i]
    raise AssertionError("braces do not match")


@pytest.mark.parametrize("name,kernels", [("cache_drafts_f32.cu", ("drafts_f32_kernel", "weigh_f32_kernel")),
                                          ("cache_drafts_mma.cu", ("drafts_mma_kernel", "weigh_mma_kernel"))])
def test_a_barrier_between_a_tiles_mask_and_the_next_one_in_its_place(name, kernels):
    """Which tokens of a tile are there is read by every warp, and overwritten (draft_place) by the first warps for the
    tile after next: on every path a barrier of the CTA lies between the two, and one between the writing and the
    reading a turn later."""
    text = _source(name)
    for kernel in kernels:
        body = _block(text, text.index(f"{kernel}("))
        loop = _block(body, re.search(r"for \(int i = 0; i < g\.tiles; \+\+i\)", body).start())
        reads = [m.start() for m in re.finditer(r"s_tile\[buffer\]\.here", loop)]
        writes = [m.start() for m in re.finditer(r"draft_place\(p, s_tile\[buffer\]", loop)]
        assert reads and len(writes) == 1 and reads[-1] < writes[0], kernel

        def depth(i):
            return loop.count("{", 0, i) - loop.count("}", 0, i)
        # (barriers of the loop's own body: what is in an inner block may be passed by)
        barriers = [m.start() for m in re.finditer(r"__syncthreads\(\);", loop) if depth(m.start()) == 0]
        assert any(reads[-1] < b < writes[0] for b in barriers), kernel
        assert any(b > writes[0] for b in barriers), kernel
