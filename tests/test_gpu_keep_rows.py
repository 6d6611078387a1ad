"""What the accepted drafts' move and the eviction do with rows whose lengths, counts or pages are not as they should be, or only
look so."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import cacheutil as U
import draftutil as D
import tensor_command_execution_gb300 as T

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("length", [65, 10 ** 6, 2 ** 31 - 1])
@pytest.mark.parametrize("budget,recent", [(30, 4), (0, 0), (63, 63)])
def test_evict_leaves_a_row_longer_than_its_table_alone(length, budget, recent):
    """Nothing of it is moved, zeroed or released; its length is held to the table's 64 tokens."""
    c = U.Cache("bf16", [64, 64], 2, 32, 8)
    w, lengths, refs = torch.rand(2, 2, 64, device="cuda"), c.lengths.clone(), D.counts(c)
    lengths[1] = length
    k, v, w2, status = c.k.clone(), c.v.clone(), w.clone(), _status()
    got, out_refs = T.cache_evict(c.tables, lengths, refs, [(k, v, w2)], budget=budget, recent=recent, status=status)
    assert int(status) == T.cache.BAD_INDEX and got.tolist() == [budget, 64]
    page, slot = D.slots(c, 1, 64)
    assert torch.equal(k[page, slot], c.k[page, slot]) and torch.equal(v[page, slot], c.v[page, slot]) and torch.equal(w2[1], w[1])
    assert torch.equal(out_refs[page.unique()], refs[page.unique()])
    assert int(out_refs.sum()) == 8 + -(-budget // 8)


@pytest.mark.parametrize("count", [0, -1])
def test_only_counts_above_one_say_that_others_hold_a_page(count):
    """A caller that keeps no counts (or wrong ones) is not told of other holders."""
    c = U.Cache("bf16", [26, 26], 2, 32, 8)
    refs, status = D.counts(c), _status()
    refs[c.tables[1, :4].long()] = count
    path = _i32([[0, 2, 3, 5, -1, -1]] * 2)
    k, v = c.k.clone(), c.v.clone()
    got, out_refs = T.cache_accept(c.tables, c.lengths, refs, path, _i32([4, 4]), [k, v], status=status)
    T.cache_status(status)
    assert got.tolist() == [24, 24] and out_refs[c.tables[1, :3].long()].tolist() == [count] * 3
    for r in range(2):
        page, slot = D.slots(c, r, 26)
        for x, y in ((k, c.k), (v, c.v)):
            want = y[page, slot].clone()
            want[20:24] = want[[20, 22, 23, 25]]
            assert torch.equal(x[page, slot], want)
    w = torch.rand(2, 2, 32, device="cuda")
    k, v, mine = c.k.clone(), c.v.clone(), w.clone()
    got, out_refs = T.cache_evict(c.tables, c.lengths, refs, [(k, v, mine)], budget=9, recent=2, status=status)
    T.cache_status(status)
    assert got.tolist() == [9, 9] and out_refs[c.tables[1, :2].long()].tolist() == [count] * 2
    for r in range(2):
        page, slot = D.slots(c, r, 26)
        for h in range(2):
            of = torch.tensor(D.evicted(w[r, h].tolist(), 26, 9, 2), device="cuda")
            assert torch.equal(k[page[:9], slot[:9], h], c.k[page[of], slot[of], h]) and torch.equal(mine[r, h, :9], w[r, h, of])


def test_accept_asks_only_for_the_pages_that_its_moves_meet():
    """Drafts that stay in their slots may lie in a page that another row holds too, and a page that no accepted draft comes
    from or goes to need not exist."""
    drafts, page = 10, 4  # drafts in slots 8 to 17: columns 2, 3 and 4
    c = U.Cache("bf16", [18, 18, 18], 2, 32, page)
    refs, tables, status = D.counts(c), c.tables.clone(), _status()
    refs[tables[0, 2].long()] = 2
    tables[1, 3] = -1
    refs[tables[2, 3].long()] = 2  # (written to)
    path = _i32([[0, 1, 2, 3, 5, 7, -1, -1, -1, -1], [0, 9] + [-1] * 8, [0, 1, 2, 3, 5] + [-1] * 5])
    counts, moved = [6, 2, 5], [[0, 1, 2, 3, 5, 7], [0, 9], []]
    k, v = c.k.clone(), c.v.clone()
    got, out_refs = T.cache_accept(tables, c.lengths, refs, path, _i32(counts), [k, v], drafts=drafts, status=status)
    # (the second row's missing page was to be released)
    assert int(status) == T.cache.SHARED_PAGE | T.cache.BAD_PAGE
    assert got.tolist() == [14, 10, 8]
    for r in range(3):
        at, slot = D.slots(c, r, 18)
        there = torch.ones(18, dtype=torch.bool, device="cuda")
        there[12:16] = r != 1
        for x, y in ((k, c.k), (v, c.v)):
            want = y[at, slot].clone()
            want[8:8 + len(moved[r])] = want[[8 + i for i in moved[r]]]
            assert torch.equal(x[at, slot][there], want[there])
    assert out_refs[tables[0].long()].tolist() == [1, 1, 2, 1, 0]
