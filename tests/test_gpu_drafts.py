"""Attention of drafted tokens over a paged cache, and the weights that it adds up, against plain forms in 64 bits."""
from __future__ import annotations

import math

import pytest
import torch

import cacheutil as U
import draftutil as D
import tensor_command_execution_gb300 as T
from tensor_command_execution_gb300.cache import cmd_drafts_workspace

pytestmark = pytest.mark.gpu


def _randn(*shape, kind, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(U.TYPES[kind])


def _near(got, want, bound, what=""):
    off = (got.detach().cpu().double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {float((off / bound.clamp(min=1e-300)).max()):.3g} of the bound"


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _check(kind, lengths, drafts, hq, hk, dim, page, order="slots", tree="tree", softcap=0.0, window=0, scale=None, seed=0,
           junk=None, pad=0, q=None, weigh=True):
    """lengths: tokens before the drafts (-1: a row without any token)."""
    totals = [n + drafts if n >= 0 else 0 for n in lengths]
    c = U.Cache(kind, totals, hk, dim, page, order, seed=seed, junk=junk, pad=pad)
    q = _randn(len(lengths), drafts, hq, dim, kind=kind, seed=seed + 1) if q is None else q
    parents = None if tree is None else D.trees(len(lengths), drafts, tree, seed)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    weights = torch.rand(len(lengths), hk, c.tables.shape[1] * page + 3, device="cuda") if weigh else None
    before = weights.clone() if weigh else None
    out, lse = T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, parents=None if parents is None else _i32(parents), scale=scale,
                                  softcap=softcap, window=window, weights=weights, return_lse=True, status=status)
    T.cache_status(status)
    if parents is None:
        parents = D.trees(len(lengths), drafts, "chain")
    want, want_lse, want_w, bound, lse_bound, w_bound = D.drafted(q, c, totals, parents, dim ** -0.5 if scale is None else scale, softcap, window)
    top = torch.stack([c.rows(r, n)[1].abs().amax() if n else torch.zeros(()).double() for r, n in enumerate(totals)])
    bound = bound + D.split_error(kind) * top[:, None, None, None] + U.ROUND[kind] * want.abs() * (1 + 2.0 ** -10) + U.TINY[kind]
    _near(out, want, bound, "out")
    none = torch.isinf(want_lse)
    assert torch.equal(torch.isinf(lse.cpu()) & (lse.cpu() < 0), none)
    _near(torch.where(none.cuda(), 0.0, lse), torch.where(none, 0.0, want_lse), lse_bound, "lse")
    if weigh:
        for r, n in enumerate(totals):
            total = before[r, :, :n].cpu().double() + want_w[r]
            _near(weights[r, :, :n], total, w_bound[r] + 2.0 ** -24 * total, "weights")
            assert torch.equal(weights[r, :, n:], before[r, :, n:])
    return c, q, out, lse


KINDS = ["f32", "f16", "bf16"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("drafts", [1, 2, 3, 7, 16, 17, 33, 64, 100])
@pytest.mark.parametrize("tree", [None, "tree", "forest", "star"])
def test_numbers_of_drafts_and_trees(kind, drafts, tree):
    _check(kind, [0, 1, 130, -1, 63], drafts, 4, 2, 64, 16, tree=tree)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("tree", ["tree", "forest", "padded", None])
def test_the_largest_trees(kind, tree):
    _check(kind, [0, 37], 256, 2, 1, 32, 16, tree=tree)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hk", [(8, 8), (8, 2), (32, 4), (7, 1), (10, 5), (24, 2), (33, 1), (48, 3)])
def test_heads(kind, hq, hk):
    _check(kind, [0, 15, 130, 333], 5, hq, hk, 64, 16)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [1, 8, 20, 33, 40, 64, 72, 80, 96, 128, 136, 192, 256])
@pytest.mark.parametrize("drafts", [3, 12, 40])
def test_dims(kind, dim, drafts):
    _check(kind, [3, 64, 201], drafts, 6, 2, dim, 8)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("page", [1, 3, 16, 24, 32, 128])
@pytest.mark.parametrize("order", ["slots", "heads", "both"])
def test_pages(kind, page, order):
    _check(kind, [0, 2, 31, 97, 256, 413], 9, 8, 2, 128, page, order)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("softcap,window", [(20.0, 0), (0.0, 1), (0.0, 3), (0.0, 17), (5.0, 100), (0.0, 1000), (0.0, 2 ** 31 - 1)])
@pytest.mark.parametrize("tree", [None, "tree"])
def test_cap_and_window(kind, softcap, window, tree):
    _check(kind, [0, 1, 16, 99, 100, 101, 400], 20, 4, 2, 96, 16, softcap=softcap, window=window, tree=tree)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("drafts", [2, 24])
def test_long_rows_are_split_and_joined(kind, drafts):
    _check(kind, [20011, 5, -1, 4097], drafts, 4, 1, 64, 32, seed=2)


def test_many_rows():
    """More rows than one launch takes, most of them without a token or short."""
    rng = torch.Generator().manual_seed(5)
    _check("bf16", [int(x) - 1 for x in torch.randint(0, 5, (1100,), generator=rng)], 3, 2, 1, 16, 2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("drafts", [4, 40])
def test_padding_gives_zeros(kind, drafts):
    """Drafts without a parent, drafts of those, and nothing else disturbed."""
    _, _, out, lse = _check(kind, [0, 33, 200], drafts, 4, 2, 64, 16, tree="padded", seed=3)
    for r, p in enumerate(D.trees(3, drafts, "padded", 3)):
        for i, path in enumerate(D.seen_by(p)):
            if path is None:
                assert bool((out[r, i] == 0).all()) and bool((lse[r, i] == -math.inf).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf, "lowest"])
@pytest.mark.parametrize("drafts", [4, 40])
def test_what_is_not_in_the_row_does_not_enter(kind, junk, drafts):
    junk = torch.finfo(U.TYPES[kind]).min if junk == "lowest" else junk
    _check(kind, [0, 1, 37, 128, 129], drafts, 4, 2, 128, 32, junk=junk)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dim,drafts", [(64, 6), (128, 40), (256, 6), (33, 6)])
def test_other_branches_do_not_enter(kind, junk, dim, drafts):
    """Two chains from the same tokens: the keys and values of one are not finite. The other's outputs are the same bits as
    without; the first one's are not finite."""
    parents = [[-1, -1] + list(range(drafts - 2))]
    c = U.Cache(kind, [70 + drafts], 2, dim, 16)
    q = _randn(1, drafts, 4, dim, kind=kind, seed=4)
    want, want_lse = T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, parents=_i32(parents), return_lse=True)
    page, slot = D.slots(c, 0, 70 + drafts)
    odd = torch.arange(71, 70 + drafts, 2, device="cuda")
    c.v[page[odd], slot[odd]] = junk
    w0 = torch.zeros(1, 2, c.tables.shape[1] * 16, device="cuda")
    got = T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, parents=_i32(parents), weights=w0)
    assert torch.equal(got[:, ::2], want[:, ::2])
    assert not bool(torch.isfinite(got[:, 1::2]).any())
    c.k[page[odd], slot[odd]] = junk
    w1 = torch.zeros_like(w0)
    got, lse = T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, parents=_i32(parents), return_lse=True, weights=w1)
    assert torch.equal(got[:, ::2], want[:, ::2]) and torch.equal(lse[:, ::2], want_lse[:, ::2])
    even = torch.arange(70, 70 + drafts, 2, device="cuda")
    # (the first chain's own tokens have weights from it alone)
    assert torch.equal(w1[:, :, even], w0[:, :, even])


@pytest.mark.parametrize("kind", KINDS)
def test_tokens_before_a_window_do_not_enter(kind):
    """Within a tree, where the window begins differs from draft to draft."""
    drafts, window = 8, 20
    lengths = [70 + drafts, 33 + drafts]
    q = _randn(2, drafts, 4, 64, kind=kind)
    got = []
    for junk in (None, math.nan, math.inf):
        c = U.Cache(kind, lengths, 2, 64, 16)
        for r, n in enumerate(lengths):
            page, slot = D.slots(c, r, n - drafts - window + 1)
            if junk is not None:
                c.k[page, slot], c.v[page, slot] = junk, junk
        got.append(T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, window=window))
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("kind", KINDS)
def test_extreme_scores(kind):
    _check(kind, [50, 3], 5, 2, 1, 32, 16, scale=30.0)
    c = U.Cache(kind, [40], 1, 32, 16)
    c.k[...] = 0
    c.k[..., 0] = -math.inf
    q = torch.zeros(1, 4, 1, 32, device="cuda", dtype=U.TYPES[kind])
    q[..., 0] = 1
    w = torch.full((1, 1, 48), 0.5, device="cuda")
    out, lse = T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, return_lse=True, weights=w)
    assert torch.equal(out, torch.zeros_like(out)) and bool((lse == -math.inf).all()) and bool((w == 0.5).all())


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 100, 33, 256])
@pytest.mark.parametrize("above", [9.0, 17.5, 20.0])
def test_small_weights_beside_a_dominant_token(kind, dim, above):
    """The first token takes all but e^-above of the softmax of each other one and has a value of zero: the output is
    what the small weights add up to. The bound is that of the one-token attention's test, but that f16 weights are held no
    finer than 2^-36 of the largest: they are lifted by 2^11, and half of f16's smallest step is 2^-25."""
    n, drafts = 8192, 3
    c = U.Cache(kind, [n], 1, dim, 32)
    gen = torch.Generator(device="cuda").manual_seed(3)
    first = (int(c.tables[0, 0]), 0)
    c.k.copy_(0.05 * torch.randn(c.k.shape, generator=gen, device="cuda"))
    c.v.copy_(64.0 + 64.0 * torch.rand(c.v.shape, generator=gen, device="cuda"))
    c.k[..., 0] = 0
    c.k[first] = 0
    c.k[first + (0, 0)] = above * dim ** 0.5
    c.v[first] = 0
    q = torch.randn(1, drafts, 2, dim, generator=gen, device="cuda").to(U.TYPES[kind])
    q[..., 0] = 1
    rows = 256
    got, lse = T.attention_drafts(q.expand(rows, -1, -1, -1), c.k, c.v, c.tables.expand(rows, -1), c.lengths.expand(rows), return_lse=True)
    want, want_lse, _, bound, lse_bound, _ = D.drafted(q, c, [n], D.trees(1, drafts, "chain"), dim ** -0.5)
    assert float(want.min()) > 1e-4
    split = {"f32": 0.0, "f16": 2.0 ** -22, "bf16": 2.0 ** -16}[kind] * want + {"f16": n * 2.0 ** -36}.get(kind, 0.0) * 128.0
    bound = bound + split + U.ROUND[kind] * want.abs() * (1 + 2.0 ** -10) + U.TINY[kind]
    _near(got, want.expand(rows, -1, -1, -1), bound.expand(rows, -1, -1, -1))
    _near(lse, want_lse.expand(rows, -1, -1), lse_bound.expand(rows, -1, -1))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("drafts", [3, 24])
def test_strides(kind, drafts):
    """Rows of the cache padded (to an odd and to a vector's pitch), queries out of a fused projection and broadcast, outputs
    and weights inside wider tensors, tables and parents transposed."""
    for pad in (1, 2, 8):
        _check(kind, [5, 77, 140], drafts, 4, 2, 64, 16, pad=pad)
    wide = _randn(3, drafts, 12, 65, kind=kind, seed=9)
    _check(kind, [5, 77, 140], drafts, 4, 2, 64, 16, q=wide[:, :, 3:7, 1:])
    _check(kind, [5, 77, 140], drafts, 4, 2, 64, 16, q=wide[:1, :1, 3:4, :64].expand(3, drafts, 4, 64))
    c = U.Cache(kind, [30 + drafts, 31 + drafts], 2, 64, 16)
    q, parents = _randn(2, drafts, 4, 64, kind=kind), _i32(D.trees(2, drafts, "tree"))
    want, want_lse = T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, parents=parents, return_lse=True)
    room = torch.full((drafts, 2, 9, 64), 7.0, device="cuda", dtype=U.TYPES[kind])
    room_lse = torch.full((4, 2, drafts, 2), 7.0, device="cuda")
    weights = torch.zeros(2, 3, c.tables.shape[1] * 16 + 5, device="cuda")
    lengths = torch.stack([c.lengths, c.lengths], 1)[:, 0]
    out, lse = T.attention_drafts(q, c.k, c.v, c.tables.t().contiguous().t(), lengths, parents=parents.t().contiguous().t(),
                                  out=room.transpose(0, 1)[:, :, 2:6], lse=room_lse[..., 0].permute(1, 2, 0), return_lse=True,
                                  weights=weights[:, 1:])
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert bool((room[:, :, :2] == 7).all()) and bool((room[:, :, 6:] == 7).all()) and bool((room_lse[..., 1] == 7).all())
    assert bool((weights[:, 0] == 0).all())
    for r, n in enumerate(c.lengths.tolist()):
        # (every draft's query heads give one in all; sums of n terms in 32 bits)
        total = weights[r, 1:].double().sum(-1)
        assert bool(((total - drafts * 2).abs() < (n + 64) * 2.0 ** -22 * drafts * 2).all()) and bool((weights[r, :, n:] == 0).all())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("drafts", [2, 30])
def test_bad_pages_and_lengths(kind, drafts):
    """What is wrong with a row is reported, and leaves the others as they were; a page that does not exist is skipped."""
    totals = [64 + drafts] * 5
    c = U.Cache(kind, totals, 2, 64, 16)
    q = _randn(5, drafts, 4, 64, kind=kind)
    good, good_lse = T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, return_lse=True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tables, lengths = c.tables.clone(), c.lengths.clone()
    tables[1, 2], tables[2, 1] = -7, c.pages
    lengths[3], lengths[4] = -5, drafts - 1
    weights = torch.zeros(5, 2, tables.shape[1] * 16, device="cuda")
    out, lse = T.attention_drafts(q, c.k, c.v, tables, lengths, return_lse=True, status=status, weights=weights)
    assert int(status) == T.cache.BAD_PAGE | T.cache.BAD_INDEX
    # (the work is split otherwise among fewer tokens)
    assert float((out[0] - good[0]).abs().max()) < 8 * U.ROUND[kind] + 2.0 ** -15 and bool((out[3:] == 0).all()) and bool((lse[3:] == -math.inf).all())
    assert bool((weights[1, :, 32:48] == 0).all()) and bool((weights[2, :, 16:32] == 0).all()) and bool((weights[3:] == 0).all())
    for r, (lo, hi) in ((1, (32, 48)), (2, (16, 32))):
        k, v = c.rows(r, 64 + drafts)
        x = q[r].cpu().double().reshape(drafts, 2, 2, 64)
        s = torch.einsum("ihgd,thd->ihgt", x, k) / 8
        t = torch.arange(64 + drafts)
        s = s.masked_fill(((t >= lo) & (t < hi)) | (t[None] > 64 + torch.arange(drafts)[:, None])[:, None, None], -math.inf)
        want = torch.einsum("ihgt,thd->ihgd", torch.softmax(s, -1), v).reshape(drafts, 4, 64)
        # (two roundings of the type, of values up to 4)
        assert float((out[r].cpu().double() - want).abs().max()) < 8 * U.ROUND[kind] + 2.0 ** -15
    parents = [[-1] + [i - 1 for i in range(1, drafts)] for _ in range(5)]
    parents[1][drafts - 1] = drafts - 1
    status.zero_()
    out = T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, parents=_i32(parents), status=status)
    assert int(status) == T.cache.BAD_INDEX and bool((out[1, -1] == 0).all())
    assert torch.equal(out[1, :-1], good[1, :-1]) and torch.equal(out[2:], good[2:])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,softcap", [(0, 0.0), (50, 10.0)])
def test_one_draft_is_the_one_token_attention(kind, window, softcap):
    """The same function, to the bounds of both."""
    c = U.Cache(kind, [1, 33, 700], 2, 64, 16)
    q = _randn(3, 8, 64, kind=kind)
    a, a_lse = T.attention_decode(q, c.k, c.v, c.tables, c.lengths, window=window, softcap=softcap, return_lse=True)
    b, b_lse = T.attention_drafts(q[:, None], c.k, c.v, c.tables, c.lengths, window=window, softcap=softcap, return_lse=True)
    want, want_lse, bound, lse_bound = U.attended(q, c, [1, 33, 700], 0.125, softcap, window)
    assert bool(((a_lse - b_lse[:, 0]).abs().cpu().double() <= 2 * lse_bound).all())
    split = D.split_error(kind) * 5.0
    assert bool(((a - b[:, 0]).abs().cpu().double() <= 2 * (bound + split) + 2 * U.ROUND[kind] * want.abs() * (1 + 2.0 ** -7) + 2 * U.TINY[kind]).all())


def test_no_rows_and_no_heads():
    c = U.Cache("bf16", [20], 2, 64, 16)
    out = T.attention_drafts(_randn(0, 3, 4, 64, kind="bf16"), c.k, c.v, c.tables[:0], c.lengths[:0])
    assert out.shape == (0, 3, 4, 64)
    out = T.attention_drafts(_randn(1, 3, 0, 64, kind="bf16"), c.k[:, :, :0], c.v[:, :, :0], c.tables, c.lengths)
    assert out.shape == (1, 3, 0, 64)


def test_pools_past_32_bits():
    """Pages whose elements lie past 2^32."""
    pages = (1 << 32) // (16 * 64) + 40
    both = torch.empty(pages, 16, 1, 64, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([[0, pages - 1, pages - 17]], dtype=torch.int32, device="cuda")
    both[at[0].long()] = _randn(3, 16, 1, 64, kind="bf16")
    q = _randn(1, 5, 2, 64, kind="bf16", seed=1)
    n = _i32([44])
    small = both[at[0].long()].clone()
    weights = torch.zeros(2, 1, 1, 48, device="cuda")
    a = T.attention_drafts(q, both, both, at, n, weights=weights[0])
    b = T.attention_drafts(q, small, small, _i32([[0, 1, 2]]), n, weights=weights[1])
    assert torch.equal(a, b) and torch.equal(weights[0], weights[1])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_given_workspaces_and_repeated_calls(kind):
    """Workspaces of any contents; the same bits every time."""
    c = U.Cache(kind, [3000, 40, 900], 2, 64, 16)
    q, parents = _randn(3, 12, 8, 64, kind=kind), _i32(D.trees(3, 12, "tree"))
    need = cmd_drafts_workspace(3, 12, 8, 2, 64, c.tables.shape[1] * 16)
    got = []
    for fill in (0, 255, 127):
        w = torch.zeros(3, 2, c.tables.shape[1] * 16, device="cuda")
        work = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        got.append((*T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, parents=parents, return_lse=True, weights=w, workspace=work), w))
    for x in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(x, got[0]))
    short = torch.zeros(need - 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(T.CmdError, match="workspace"):
        T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, parents=parents, workspace=short, weights=got[0][2])


def test_captured_and_replayed():
    """In a graph, on other lengths, trees and numbers than it was captured with."""
    c = U.Cache("bf16", [300, 90, 40], 2, 64, 16, columns=30)
    q, parents = _randn(3, 10, 4, 64, kind="bf16"), _i32(D.trees(3, 10, "tree"))
    weights = torch.zeros(3, 2, 480, device="cuda")
    out = torch.empty_like(q)

    def call():
        T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, parents=parents, out=out, weights=weights)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for seed, lengths in enumerate(([300, 90, 40], [0, 11, 33], [299, 10, 0])):
        q.copy_(_randn(3, 10, 4, 64, kind="bf16", seed=seed + 5))
        parents.copy_(_i32(D.trees(3, 10, "padded", seed)))
        c.lengths.copy_(_i32(lengths))
        weights.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got, w = out.clone(), weights.clone()
        weights.zero_()
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, got) and torch.equal(weights, w), seed


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("drafts,dim", [(5, 64), (40, 128), (40, 200)])
@pytest.mark.parametrize("junk", [math.nan, math.inf])
def test_padding_may_hold_anything(kind, drafts, dim, junk):
    """Queries, keys and values of padding are not finite, in rows that are split over many CTAs."""
    lengths = [9000 + drafts, 70 + drafts]
    c = U.Cache(kind, lengths, 2, dim, 16)
    q = _randn(2, drafts, 4, dim, kind=kind, seed=6)
    parents = D.trees(2, drafts, "tree", 6)
    for r in range(2):
        parents[r][drafts // 2] = -2
    want, want_lse = T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, parents=_i32(parents), return_lse=True)
    w0, w1 = (torch.zeros(2, 2, c.tables.shape[1] * 16, device="cuda") for _ in range(2))
    T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, parents=_i32(parents), weights=w0)
    for r, n in enumerate(lengths):
        page, slot = D.slots(c, r, n)
        for i, path in enumerate(D.seen_by(parents[r])):
            if path is None:
                at = n - drafts + i
                q[r, i], c.k[page[at], slot[at]], c.v[page[at], slot[at]] = junk, junk, junk
                assert bool((want[r, i] == 0).all()) and bool((want_lse[r, i] == -math.inf).all())
    got, lse = T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, parents=_i32(parents), return_lse=True, weights=w1)
    assert torch.equal(got, want) and torch.equal(lse, want_lse) and torch.equal(w0, w1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hk,dim,page", [(8, 8, 64, 16), (32, 4, 128, 16), (7, 1, 64, 3), (24, 2, 256, 1), (33, 1, 72, 16), (48, 3, 100, 8),
                                            (4, 2, 33, 16), (130, 1, 64, 32)])
def test_weights_of_one_token(kind, hq, hk, dim, page):
    """One new token's scores are kept (16-bit rows of whole 16-byte vectors), or worked out again."""
    _check(kind, [0, 1, 15, 130, -1, 1500], 1, hq, hk, dim, page, tree=None)
    _check(kind, [0, 40, 200], 1, hq, hk, dim, page, tree=None, softcap=5.0, window=30)
    _check(kind, [0, 40, 200], 1, hq, hk, dim, page, tree="padded", seed=2)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("drafts,hq,hk,dim,page", [(2, 4, 4, 64, 16), (8, 4, 2, 128, 8), (5, 3, 1, 72, 3), (16, 4, 2, 128, 16), (3, 16, 2, 80, 24),
                                                   (31, 1, 1, 64, 128)])
def test_few_queries_of_long_tables(kind, drafts, hq, hk, dim, page):
    """Up to 32 query rows to a kv head, in tables long enough for the CTA-wide instructions, and in shorter ones."""
    _check(kind, [0, 1, 100, 700, -1, 1300], drafts, hq, hk, dim, page, tree="padded")
    _check(kind, [1300, 20], drafts, hq, hk, dim, page, tree="tree", softcap=5.0, window=60, junk=float("nan"))
    _check(kind, [0, 1, 100, -1, 200], drafts, hq, hk, dim, page, tree="padded")
    _check(kind, [200, 20], drafts, hq, hk, dim, page, tree="tree", softcap=5.0, window=60, junk=float("nan"))


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hq,hk,dim,page", [(8, 2, 128, 16), (3, 3, 33, 8), (20, 1, 256, 1)])
def test_one_draft_with_parents(kind, hq, hk, dim, page):
    """-1 is one token's attention, exactly; less, or a parent that does not exist (reported), is a row without any."""
    totals = [700, 20, 1, 0, 40, 300]
    c = U.Cache(kind, totals, hk, dim, page)
    q = _randn(6, 1, hq, dim, kind=kind, seed=1)
    parents, status = _i32([[-1], [-2], [-1], [-1], [0], [-2147483648]]), torch.zeros(1, dtype=torch.int32, device="cuda")
    tokens = c.tables.shape[1] * page
    w, plain = (torch.rand(6, hk, tokens, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda") for _ in range(2))
    start = w.clone()
    out, lse = T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, parents=parents, weights=w, return_lse=True, status=status)
    with pytest.raises(T.CmdError):
        T.cache_status(status)
    want, want_lse = T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, weights=plain, return_lse=True)
    assert torch.equal(want[:, 0], T.attention_decode(q[:, 0], c.k, c.v, c.tables, c.lengths))
    for r in range(6):
        if r in (0, 2):
            assert torch.equal(out[r], want[r]) and torch.equal(lse[r], want_lse[r]) and torch.equal(w[r], plain[r])
        else:
            assert not bool(out[r].any()) and bool((lse[r] == -math.inf).all()) and torch.equal(w[r], start[r])


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("drafts,hq,hk,dim,page", [(16, 28, 2, 192, 8), (5, 8, 2, 256, 16), (40, 8, 1, 136, 64), (2, 4, 4, 200, 24), (9, 30, 1, 256, 8)])
def test_weights_of_wide_heads(kind, drafts, hq, hk, dim, page):
    """Heads of more than 128 dims, with more query rows to a head than a launch takes."""
    _check(kind, [0, 1, 100, 700, -1], drafts, hq, hk, dim, page, tree="padded")
    _check(kind, [300, 20], drafts, hq, hk, dim, page, tree="tree", softcap=5.0, window=60)


@pytest.mark.parametrize("drafts", [1, 3])
def test_weights_of_tables_with_room_for_millions(drafts):
    """Scores that would take more than a GiB are not kept; tables, weights and lengths of rows far apart."""
    lengths, columns = [700, 3, 2100], 100_000
    totals = [n + drafts for n in lengths]
    c = U.Cache("bf16", totals, 8, 64, 16, columns=columns)
    q = _randn(3, drafts, 64, 64, kind="bf16", seed=1)
    weights = torch.zeros(3, 8, columns * 16, device="cuda")
    out, lse = T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, weights=weights, return_lse=True)
    _, _, want, _, _, bound = D.drafted(q, c, totals, D.trees(3, drafts, "chain"), 0.125)
    for r, n in enumerate(totals):
        _near(weights[r, :, :n], want[r], bound[r] + 2.0 ** -24 * want[r], "weights")
        assert not bool(weights[r, :, n:].any())


def test_two_streams_at_once():
    """Calls on two streams over one cache, each with its own workspace and outputs, again and again."""
    c = U.Cache("bf16", [3000, 40, 900, 260], 2, 128, 16)
    calls = []
    for seed in range(2):
        q, parents = _randn(4, 10, 8, 128, kind="bf16", seed=seed), _i32(D.trees(4, 10, "tree", seed))
        calls.append((q, parents, T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, parents=parents)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            w = torch.zeros(4, 2, c.tables.shape[1] * 16, device="cuda")
            s.wait_stream(torch.cuda.current_stream())
            got[i].append((T.attention_drafts(calls[i][0], c.k, c.v, c.tables, c.lengths, parents=calls[i][1], weights=w, stream=s), w))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, calls[i][2]) and torch.equal(w, got[i][0][1]) for x, w in got[i])


def test_a_step_with_drafts():
    """Room for the drafts, their keys at their own positions, attention, the accepted branch and its slots: the cache is
    what it would be had the accepted tokens come one by one; captured in a graph too."""
    drafts, tree = 7, [-1, 0, 0, 1, 1, 3, 2]
    depth = _i32([0, 1, 1, 2, 2, 3, 2])
    turns = T.rope_turns(64)
    gen = torch.Generator(device="cuda").manual_seed(0)

    def start():
        c = U.Cache("bf16", [33, 16, 5], 2, 64, 16, spare=12, columns=6)
        return c, D.counts(c)
    tokens = _i32([[3, 5, 6, 7, 8, 9, 4], [1, 2, 2, 4, 4, 4, 4], [9, 8, 7, 6, 5, 4, 3]])
    choices = _i32([[5, 8, 0, 0, 0, 0, 0], [2, 4, 0, 4, 0, 0, 0], [0, 0, 0, 0, 0, 0, 0]])
    want_path = [[0, 1, 4], [0, 1, 3, 5], [0]]
    parents = _i32([tree] * 3)
    q, k, v = (torch.randn(3, drafts, h, 64, generator=gen, device="cuda").bfloat16() for h in (8, 2, 2))
    same, grow = _i32([0, 1, 2]), _i32([drafts] * 3)
    rows = same.repeat_interleave(drafts)

    def step(c, refs):
        t, n, r = T.cache_select(c.tables, c.lengths, refs, same, [c.k, c.v], page_size=16, grow=grow)
        positions = n[:, None] - drafts + depth
        x, y = T.rope(q, k, positions, turns)
        slots = (n[:, None] - drafts + torch.arange(drafts, dtype=torch.int32, device="cuda")).flatten()
        T.cache_append(y.flatten(0, 1), v.flatten(0, 1), c.k, c.v, t, slots, rows=rows)
        out = T.attention_drafts(x, c.k, c.v, t, n, parents=parents)
        path, counts, last = T.draft_path(tokens, choices, parents=parents)
        n, r = T.cache_accept(t, n, r, path, counts, [c.k, c.v], drafts=drafts)
        return out, t, n, r, path, counts, last, c.k, c.v

    c, refs = start()
    got = [x.clone() for x in step(c, refs)]
    out, t, n, r, path, counts, last = got[:7]
    assert [p[:k] for p, k in zip(path.tolist(), counts.tolist())] == want_path
    assert n.tolist() == [33 + 3, 16 + 4, 5 + 1]
    # the same tokens, one at a time
    one, refs1 = start()
    t1, n1, r1 = one.tables, one.lengths, refs1
    for step_ in range(4):
        alive = [step_ < len(w) for w in want_path]
        node = [w[min(step_, len(w) - 1)] for w in want_path]
        t1, n1, r1 = T.cache_select(t1, n1, r1, same, [one.k, one.v], page_size=16, grow=_i32([int(a) for a in alive]))
        pick = torch.tensor(node, device="cuda")
        kk, vv, qq = (x[torch.arange(3, device="cuda"), pick] for x in (k, v, q))
        pos = torch.where(torch.tensor(alive, device="cuda"), n1 - 1, -1)
        turned = T.cache_append(kk, vv, one.k, one.v, t1, pos.int(), q=qq, turns=turns)
        single = T.attention_decode(turned, one.k, one.v, t1, n1)
        for row in range(3):
            if alive[row]:
                # (the same function: two roundings of values below 4)
                assert float((single[row].float() - out[row, node[row]].float()).abs().max()) < 8 * U.ROUND["bf16"]
    assert torch.equal(n1, n)
    for row, length in enumerate(n.tolist()):
        at = torch.arange(length, device="cuda")
        for x, y in ((got[7], one.k), (got[8], one.v)):
            assert torch.equal(x[t[row].long()[at // 16], at % 16], y[t1[row].long()[at // 16], at % 16])
    assert int(r.sum()) == int(r1.sum()) == sum(-(-x // 16) for x in n.tolist())
    # captured
    c, refs = start()
    kc, vc = c.k.clone(), c.v.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c, refs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        again = step(c, refs)
    for _ in range(2):
        c.k.copy_(kc)
        c.v.copy_(vc)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(again, got))
