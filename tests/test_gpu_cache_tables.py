"""The cache operators on tables, pools and lengths that a program may hand them in earnest: entries that name no page,
and as many pools as a model has."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import cacheutil as U
import tensor_command_execution_gb300 as T

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


class _Rest:
    """A cache's rows without the tokens whose table entry names no page."""

    def __init__(self, cache, lengths):
        self.tokens = []
        for r, n in enumerate(lengths):
            table = cache.tables[r].tolist()
            at = [(table[i // cache.page], i % cache.page) for i in range(n) if 0 <= table[i // cache.page] < cache.pages]
            page, slot = (torch.tensor([a[j] for a in at], dtype=torch.long) for j in range(2))
            self.tokens.append(tuple(x[page.cuda(), slot.cuda()].cpu().double() for x in (cache.k, cache.v)))
        self.lengths = [len(k) for k, _ in self.tokens]

    def rows(self, r, n):
        return self.tokens[r]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 100, 33])
@pytest.mark.parametrize("page", [3, 16])
@pytest.mark.parametrize("long", [False, True])
def test_attention_over_what_bad_entries_leave(kind, dim, page, long):
    """Entries below zero and past the pool, at the start, inside and at the end of rows, one row with nothing else,
    and lengths past the table: each row is the attention over exactly the tokens that are left."""
    lengths = [3000, 1500, 40, 17, 2900, 1] if long else [200, 64, 40, 17, 130, 1]
    # (tables far longer than the rows: work is dealt out evenly and split; else clusters take the rows)
    c = U.Cache(kind, lengths, 2, dim, page, columns=max(-(-n // page) for n in lengths) + (6000 // page if long else 0))
    bad = [-1, -5, c.pages, 0x7fffffff, -(1 << 31)]
    rng = np.random.RandomState(dim + page)
    for r, n in enumerate(lengths[:-1]):
        need = -(-n // page)
        where = [0] if r == 0 else [need - 1] if r == 1 else list(range(need)) if r == 3 else rng.permutation(need)[: 1 + need // 3]
        for i, j in enumerate(where):
            c.tables[r, int(j)] = bad[(r + i) % len(bad)]
    given = list(lengths)
    if not long:  # past the table: held to it
        full = -(-max(lengths) // page)
        c.tables[2, :full] = c.tables[0, :full]
        c.tables[2, 0] = c.tables[5, 0]
        given[2], lengths[2] = full * page + 1, full * page
    gen = torch.Generator(device="cuda").manual_seed(1)
    q = (2 * torch.randn(len(lengths), 6, dim, generator=gen, device="cuda")).to(U.TYPES[kind])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = T.attention_decode(q, c.k, c.v, c.tables, _i32(given), return_lse=True, status=status)
    with pytest.raises(T.CmdError, match="page" if long else "page.*length"):
        T.cache_status(status)
    rest = _Rest(c, lengths)
    assert rest.lengths[3] == 0 and 0 < rest.lengths[0] < lengths[0]
    want, want_lse, bound, lse_bound = U.attended(q, rest, rest.lengths, dim ** -0.5)
    # (a weight of a 16-bit cache is held as two 16-bit numbers)
    split = {"f32": 0.0, "f16": 2.0 ** -21, "bf16": 2.0 ** -16}[kind]
    top = torch.stack([v.abs().amax() if len(v) else torch.zeros(()).double() for _, v in rest.tokens])
    bound = bound + split * top[:, None, None] + U.ROUND[kind] * want.abs() * (1 + 2.0 ** -10) + U.TINY[kind]
    assert bool(((out.cpu().double() - want).abs() <= bound).all())
    empty = torch.isinf(want_lse)
    assert torch.equal(lse.cpu() == -torch.inf, empty)
    assert bool(((lse.cpu().double() - want_lse).abs().masked_fill(empty, 0.0) <= lse_bound).all())


@pytest.mark.parametrize("pools", [3, 9, 64, 71])
def test_as_many_pools_as_a_model_has(pools):
    """A key and a value pool for each layer: short and long lists of pools, and one call for each 64 of more, whose
    tables, lengths and counts are the same. Pages of different sizes and alignment."""
    rng = np.random.RandomState(pools)
    lengths, page = [37, 16, 5, 0, 21], 8
    c = U.Cache("bf16", lengths, 1, 8, page, spare=14, columns=7)
    t = c.tables.cpu().numpy()
    refs = np.zeros(c.pages, dtype=np.int32)
    for r, n in enumerate(c.need):
        refs[t[r, :n]] += 1
    parents, grow = [4, 0, 0, 4, -1, 2], [1, 9, 0, 3, 8, 1]
    want = U.select_reference(t, lengths, refs, parents, grow, page)
    assert len(want[3]) >= 2 and (want[1] > 0).all()

    def make():
        gen = torch.Generator(device="cuda").manual_seed(9)
        unit = int(rng.choice([1, 2, 4, 8, 16]))
        return [torch.randint(0, 255, (c.pages, page, unit * (1 + i % 3)), generator=gen, dtype=torch.uint8, device="cuda") for i in range(pools)]

    def calls(f, all_pools):
        got = [f(all_pools[i:i + 64]) for i in range(0, len(all_pools), 64)]
        for g in got[1:]:
            assert all(torch.equal(x, y) for x, y in zip(g, got[0]))
        return got[0]
    mine = make()
    expect = [p.clone() for p in mine]
    for p in expect:
        for a, b in want[3]:
            p[b] = p[a]
    got = calls(lambda some: T.cache_select(c.tables, c.lengths, _i32(refs), _i32(parents), some, page_size=page, grow=_i32(grow)), mine)
    assert all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(mine, expect))
    # compaction of what the selection left
    used = want[2] > 0
    n = int(used.sum())
    of, to = np.flatnonzero(used & (np.arange(c.pages) >= n)), np.flatnonzero(~used & (np.arange(c.pages) < n))
    assert len(of)
    for p in expect:
        p[torch.from_numpy(to).cuda()] = p[torch.from_numpy(of).cuda()]
    tables, refs_out, where = calls(lambda some: T.cache_compact(got[0], got[1], got[2], some, page_size=page), mine)
    assert all(torch.equal(a, b) for a, b in zip(mine, expect))
    assert where[torch.from_numpy(of).cuda()].tolist() == to.tolist()
    assert bool((refs_out[:n] > 0).all()) and int(refs_out[n:].abs().sum()) == 0
    if pools > 64:
        with pytest.raises(ValueError, match="64"):
            T.cache_select(c.tables, c.lengths, _i32(refs), _i32(parents), mine, page_size=page)
