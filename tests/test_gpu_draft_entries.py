"""Attention of drafted tokens over tables with entries that name no page: each row is the attention over exactly the tokens
that are left, in every kernel."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import cacheutil as U
import draftutil as D
import tensor_command_execution_gb300 as T
from test_gpu_cache_tables import _Rest
from test_gpu_drafts import _i32, _near, _randn

pytestmark = pytest.mark.gpu


def _check(kind, bases, drafts, hq, hk, dim, page, where, entries, columns=0, repeats=1):
    """bases: tokens before the drafts. where(j): whether a row's page j, of those that hold no draft, has one of
    `entries` in its place."""
    totals = [n + drafts for n in bases]
    c = U.Cache(kind, totals, hk, dim, page, columns=max([columns] + [-(-n // page) for n in totals]))
    some = 0
    for r, n in enumerate(bases):
        for j in range(n // page):
            if where(j):
                c.tables[r, j] = entries(c)[some % len(entries(c))]
                some += 1
    q, parents = _randn(len(bases), drafts, hq, dim, kind=kind, seed=1), D.trees(len(bases), drafts, "tree")
    rest = _Rest(c, totals)
    rest.k = c.k
    want, want_lse, want_w, bound, lse_bound, w_bound = D.drafted(q, rest, rest.lengths, parents, dim ** -0.5)
    top = torch.stack([v.abs().amax() for _, v in rest.tokens])
    bound = bound + D.split_error(kind) * top[:, None, None, None] + U.ROUND[kind] * want.abs() * (1 + 2.0 ** -10) + U.TINY[kind]
    tables, first = c.tables.cpu().numpy(), None
    for _ in range(repeats):
        status, weights = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(len(bases), hk, tables.shape[1] * page, device="cuda")
        out, lse = T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, parents=_i32(parents), weights=weights, return_lse=True, status=status)
        assert int(status) == (T.cache.BAD_PAGE if some else 0)
        if first is None:
            first = out, lse, weights
            _near(out, want, bound, "out")
            _near(lse, want_lse, lse_bound, "lse")
            for r, n in enumerate(totals):
                left = [t for t in range(n) if 0 <= tables[r, t // page] < c.pages]
                _near(weights[r][:, left], want_w[r], w_bound[r] + 2.0 ** -24 * want_w[r], "weights")
                gone = np.setdiff1d(np.arange(weights.shape[2]), left)
                assert bool((weights[r][:, gone] == 0).all())
        assert all(torch.equal(a, b) for a, b in zip((out, lse, weights), first))


# kind, drafts, query heads, kv heads, dim, page, columns: 32 bits with blocks of 16 and of 64 query rows, the warp-level
# kernels (few queries in short tables, wide heads, rows of 4-byte words, odd rows), the CTA-wide ones by both kinds of copies
KERNELS = [("f32", 3, 4, 2, 64, 16, 0), ("f32", 40, 4, 2, 80, 8, 0), ("bf16", 3, 8, 2, 64, 16, 0), ("f16", 24, 8, 2, 192, 8, 0),
           ("bf16", 6, 4, 2, 100, 8, 0), ("bf16", 5, 4, 2, 33, 16, 0), ("bf16", 40, 8, 2, 64, 16, 0), ("f16", 40, 16, 2, 128, 8, 0),
           ("bf16", 12, 8, 2, 128, 3, 900), ("f32", 1, 4, 2, 64, 16, 0), ("bf16", 1, 4, 2, 64, 16, 0), ("bf16", 1, 4, 2, 33, 16, 0)]


@pytest.mark.parametrize("kernel", KERNELS)
def test_masks_that_change_from_tile_to_tile(kernel):
    """Long rows whose tiles have other tokens missing each: whoever took a tile by another one's mask would be seen."""
    _check(*kernel[:1], [1900, 700, 40], *kernel[1:6], lambda j: (j * j) % 7 in (2, 4), lambda c: [-5, c.pages, 0x7fffffff, -(1 << 31)],
           columns=kernel[6], repeats=8)


@pytest.mark.parametrize("kernel", KERNELS)
def test_entries_of_minus_one_are_reported(kernel):
    """... what a table holds where there is no page is no page inside a row's length either: alone, beside other bad
    entries, as a row's first and as its last before the drafts."""
    for where in (lambda j: j == 1, lambda j: j in (0, 4), lambda j: j % 3 == 0):
        _check(*kernel[:1], [700, 130, 40], *kernel[1:6], where, lambda c: [-1], columns=kernel[6])
    _check(*kernel[:1], [700, 130, 40], *kernel[1:6], lambda j: j % 4 == 0, lambda c: [-1, c.pages], columns=kernel[6])
    _check(*kernel[:1], [700, 130, 40], *kernel[1:6], lambda j: False, lambda c: [-1], columns=kernel[6])


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("beyond", [1, 10 ** 6, None])
def test_a_length_beyond_the_table_is_held_to_it(kernel, beyond):
    kind, drafts, hq, hk, dim, page, columns = kernel
    c = U.Cache(kind, [64 + drafts, 30 + drafts], hk, dim, page, columns=columns or None)
    c.tables.clamp_(max=c.pages - 1)
    most = c.tables.shape[1] * page
    q, given, held = _randn(2, drafts, hq, dim, kind=kind), c.lengths.clone(), c.lengths.clone()
    given[0], held[0] = 2 ** 31 - 1 if beyond is None else most + beyond, most
    got = []
    for lengths in (given, held):
        status, weights = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(2, hk, most, device="cuda")
        out, lse = T.attention_drafts(q, c.k, c.v, c.tables, lengths, weights=weights, return_lse=True, status=status)
        assert int(status) == (T.cache.BAD_INDEX if lengths is given else 0)
        got.append((out, lse, weights))
    assert all(torch.equal(a, b) for a, b in zip(*got))
