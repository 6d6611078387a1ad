"""What a paged cache keeps: the accepted branch, its slots, and the tokens of the largest weights."""
from __future__ import annotations

import math
import random

import numpy as np
import pytest
import torch

import cacheutil as U
import draftutil as D
import tensor_command_execution_gb300 as T

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _bits(x):
    return x.contiguous().view({2: torch.int16, 4: torch.int32}[x.element_size()])


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---- the accepted branch -------------------------------------------------------------------------------------------

@pytest.mark.parametrize("rows,drafts", [(1, 1), (5, 2), (3, 31), (7, 32), (9, 33), (130, 64), (6, 255), (2, 256)])
@pytest.mark.parametrize("tree", [None, "tree", "forest", "star", "padded"])
def test_path(rows, drafts, tree):
    """Few tokens, so that several drafts go on with the same one and branches are long."""
    parents = D.trees(rows, drafts, tree or "chain", seed=rows)
    rng = np.random.RandomState(drafts)
    for words in (1, 2, 50):
        tokens, choices = rng.randint(0, words, (rows, drafts)), rng.randint(0, words, (rows, drafts))
        status = _status()
        path, counts, last = T.draft_path(_i32(tokens), _i32(choices), parents=None if tree is None else _i32(parents), status=status)
        T.cache_status(status)
        for r in range(rows):
            want, end = D.walked(tokens[r], choices[r], parents[r])
            assert path[r].tolist() == want + [-1] * (drafts - len(want)) and int(counts[r]) == len(want) and int(last[r]) == end


def test_path_strides_and_invalid_parents():
    rng = np.random.RandomState(0)
    tokens, choices = rng.randint(0, 2, (6, 9)), rng.randint(0, 2, (6, 9))
    parents = D.trees(6, 9, "tree")
    want = T.draft_path(_i32(tokens), _i32(choices), parents=_i32(parents))
    out = (torch.empty(9, 6, dtype=torch.int32, device="cuda").t(), torch.empty(12, dtype=torch.int32, device="cuda")[::2],
           torch.empty(6, dtype=torch.int32, device="cuda"))
    got = T.draft_path(_i32(tokens).t().contiguous().t(), _i32(choices)[:, :9], parents=_i32(parents).t().contiguous().t(), out=out)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and got[0].data_ptr() == out[0].data_ptr()
    one = T.draft_path(_i32(tokens)[:1].expand(6, 9), _i32(choices)[:1].expand(6, 9), parents=_i32(parents)[:1].expand(6, 9))
    assert torch.equal(one[0], want[0][:1].expand(6, 9))
    status = _status()
    parents[2][4] = 4
    T.draft_path(_i32(tokens), _i32(choices), parents=_i32(parents), status=status)
    assert int(status) == T.cache.BAD_INDEX
    assert T.draft_path(_i32(tokens)[:0], _i32(choices)[:0])[0].shape == (0, 9)


# ---- its slots -----------------------------------------------------------------------------------------------------

def _accept(kind, base, drafts, heads, dim, page, order="slots", pools=2, seed=0, pad=0, full=False):
    rng = random.Random(seed)
    totals = [n + drafts if n >= 0 else 0 for n in base]
    c = U.Cache(kind, totals, heads, dim, page, order, seed=seed, pad=pad)
    caches = [c.k, c.v]
    while len(caches) < pools:
        caches += [c.k.clone(), c.v.clone()]
    caches = caches[:pools]
    counts = [rng.choice([0, 1, drafts, rng.randint(0, drafts)]) for _ in base]
    path = np.full((len(base), drafts), -7)
    for r, n in enumerate(counts):
        path[r, :n] = range(n) if full else sorted(rng.sample(range(drafts), n))
    refs = D.counts(c)
    before = [x.clone() for x in caches]
    status = _status()
    lengths, out_refs = T.cache_accept(c.tables, c.lengths, refs, _i32(path), _i32(counts), caches, drafts=drafts, status=status)
    T.cache_status(status)
    want_refs = refs.clone()
    for r, n in enumerate(base):
        keep = n + counts[r] if n >= 0 else 0
        assert int(lengths[r]) == keep
        want_refs[c.tables[r, -(-keep // page): c.need[r]].long()] -= 1
        if n < 0:
            continue
        at, slot = D.slots(c, r, totals[r])
        for x in before:
            of = torch.tensor([n + int(p) for p in path[r, :counts[r]]], dtype=torch.long, device="cuda")
            x[at[n:keep], slot[n:keep]] = x[at[of], slot[of]].clone()
    assert torch.equal(out_refs, want_refs)
    for x, y in zip(before, caches):
        assert torch.equal(_bits(x), _bits(y))


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("drafts", [1, 2, 5, 33, 256])
@pytest.mark.parametrize("page", [1, 3, 16, 64])
def test_accept(kind, drafts, page):
    _accept(kind, [0, 1, 15, -1, 16, 70], drafts, 2, 64, page, seed=drafts)


@pytest.mark.parametrize("heads,dim,order,pad", [(8, 128, "heads", 0), (1, 1, "slots", 0), (3, 33, "slots", 0), (2, 72, "both", 0),
                                                 (5, 256, "slots", 0), (2, 64, "slots", 1), (2, 64, "slots", 4), (70, 20, "heads", 0)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_accept_layouts(kind, heads, dim, order, pad):
    _accept(kind, [3, 0, 40], 12, heads, dim, 8, order, pad=pad, pools=4)


@pytest.mark.parametrize("pools", [1, 3, 64])
def test_accept_pools(pools):
    _accept("bf16", [9, 100], 10, 2, 32, 16, pools=pools)
    _accept("bf16", [9, 100], 10, 2, 32, 16, pools=pools, full=True)


def test_accept_many_rows():
    _accept("bf16", [r % 5 - 1 for r in range(700)], 6, 1, 16, 4)


@pytest.mark.parametrize("wrong", ["order", "twice", "past", "below", "count", "negative", "page", "shared", "short", "long"])
def test_accept_leaves_a_wrong_row_alone(wrong):
    drafts, n = 6, 20 + 6
    c = U.Cache("bf16", [n] * 3, 2, 64, 8)
    path, counts = np.tile([0, 2, 3, 5, -1, -1], (3, 1)), np.array([4, 4, 4])
    tables, lengths, refs = c.tables.clone(), c.lengths.clone(), D.counts(c)
    bit, keep = T.cache.BAD_INDEX, 20
    if wrong == "order":
        path[1] = [0, 3, 2, 5, -1, -1]
    elif wrong == "twice":
        path[1] = [0, 2, 2, 5, -1, -1]
    elif wrong == "past":
        path[1, 3] = 6
    elif wrong == "below":
        path[1, 0] = -1
    elif wrong == "count":
        counts[1] = 7
    elif wrong == "negative":
        counts[1] = -1
    elif wrong == "page":
        tables[1, 2], bit = c.pages, T.cache.BAD_PAGE
    elif wrong == "shared":
        refs[c.tables[1, 2].long()], bit = 2, T.cache.SHARED_PAGE
    elif wrong == "short":
        lengths[1], keep = 5, 5
    elif wrong == "long":
        lengths[1], keep = 10 ** 6, None
    k, v, status = c.k.clone(), c.v.clone(), _status()
    got, out_refs = T.cache_accept(tables, lengths, refs, _i32(path), _i32(counts), [k, v], status=status)
    assert int(status) == bit
    assert got[0] == 24 and got[2] == 24
    if keep is None:  # (held to the table, whose last tokens are the drafts then)
        assert int(got[1]) == tables.shape[1] * 8 - drafts + 4
        return
    assert int(got[1]) == keep
    for r in (0, 1, 2):
        page, slot = D.slots(c, r, n)
        for x, y in ((k, c.k), (v, c.v)):
            want = y[page, slot].clone()
            if r != 1:
                want[20:24] = want[[20, 22, 23, 25]]
            ok = torch.ones(n, dtype=torch.bool) if not (wrong == "page" and r == 1) else torch.arange(n) // 8 != 2
            assert torch.equal(x[page, slot][ok], want[ok])
    assert int(out_refs[c.tables[0, 3].long()]) == 0 and int(out_refs[c.tables[0, 2].long()]) == 1


# ---- eviction ------------------------------------------------------------------------------------------------------

def _evict(kind, lengths, heads, dim, page, budget, recent, order="slots", layers=1, seed=0, pad=0, fill=None):
    c = U.Cache(kind, lengths, heads, dim, page, order, seed=seed, pad=pad)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    tokens = c.tables.shape[1] * page + 2
    stack = []
    for i in range(layers):
        w = torch.exp(2 * torch.randn(len(lengths), heads, tokens, generator=gen, device="cuda"))
        if fill is not None:
            w = fill(w, gen)
        stack.append((c.k if i == 0 else torch.randn_like(c.k), c.v if i == 0 else torch.randn_like(c.v), w))
    before = [[x.clone() for x in layer] for layer in stack]
    refs, status = D.counts(c), _status()
    got, out_refs = T.cache_evict(c.tables, c.lengths, refs, stack, budget=budget, recent=recent, status=status)
    T.cache_status(status)
    want_refs = refs.clone()
    for r, n in enumerate(lengths):
        keep = min(n, budget)
        assert int(got[r]) == keep
        want_refs[c.tables[r, -(-keep // page): c.need[r]].long()] -= 1
        if keep == n:
            continue
        at, slot = D.slots(c, r, n)
        for k, v, w in before:
            values = w[r].tolist()
            for h in range(heads):
                of = torch.tensor(D.evicted(values[h], n, budget, recent), dtype=torch.long, device="cuda")
                for x in (k, v):
                    x[at[:keep], slot[:keep], h] = x[at[of], slot[of], h].clone()
                kept = w[r, h, of].clone()
                w[r, h, :n] = 0
                w[r, h, :keep] = kept
    assert torch.equal(out_refs, want_refs)
    for a, b in zip(before, stack):
        for x, y in zip(a, b):
            assert torch.equal(_bits(x), _bits(y))


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (20, 0), (20, 7), (20, 20), (64, 10), (150, 40), (0, 0)])
@pytest.mark.parametrize("page", [1, 3, 16, 64])
def test_evict(kind, budget, recent, page):
    _evict(kind, [0, 1, 20, 21, 65, 200], 2, 64, page, budget, recent)


@pytest.mark.parametrize("heads,dim,order,pad", [(8, 128, "heads", 0), (1, 1, "slots", 0), (3, 33, "slots", 0), (2, 72, "both", 0),
                                                 (5, 256, "slots", 0), (2, 64, "slots", 1), (2, 64, "slots", 4), (9, 20, "heads", 0)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_evict_layouts(kind, heads, dim, order, pad):
    _evict(kind, [300, 10, 90], heads, dim, 8, 60, 13, order, pad=pad)


@pytest.mark.parametrize("layers", [2, 32])
def test_evict_layers(layers):
    _evict("bf16", [120, 10, 51], 2, 16, 16, 50, 5, layers=layers)


@pytest.mark.parametrize("length,budget", [(5000, 700), (50001, 40000), (50001, 3), (70000, 69999)])
def test_evict_long_rows(length, budget):
    """Among them rows whose weights do not fit in shared memory."""
    _evict("bf16", [length, 100], 1, 8, 16, budget, min(budget, 30))


def _equal(w, gen):
    return torch.full_like(w, 0.25)


def _few_values(w, gen):
    return torch.randint(0, 3, w.shape, generator=gen, device="cuda").float()


def _signed(w, gen):
    return torch.randn(w.shape, generator=gen, device="cuda") * torch.tensor([1e-42, 1.0, 1e38], device="cuda")[torch.randint(0, 3, w.shape, generator=gen, device="cuda")]


def _odd(w, gen):
    some = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, 1.0, -math.nan], device="cuda")
    return some[torch.randint(0, 7, w.shape, generator=gen, device="cuda")]


def _close(w, gen):
    return (torch.randint(0, 1 << 12, w.shape, generator=gen, device="cuda", dtype=torch.int32) + 0x3f800000).view(torch.float32)


@pytest.mark.parametrize("fill", [_equal, _few_values, _signed, _odd, _close])
@pytest.mark.parametrize("budget,recent", [(100, 0), (333, 50), (1, 0)])
def test_evict_weights_of_every_kind(fill, budget, recent):
    """Equal ones (the earliest stay), negative and tiny ones, zeros of both signs (equal), infinities, NaN (last)."""
    _evict("bf16", [400, 1500], 2, 16, 16, budget, recent, fill=fill)


@pytest.mark.parametrize("wrong", ["page", "tail page", "shared", "long"])
def test_evict_leaves_a_wrong_row_alone(wrong):
    c = U.Cache("bf16", [60, 60], 2, 32, 8)
    w = torch.rand(2, 2, 64, device="cuda")
    tables, lengths, refs = c.tables.clone(), c.lengths.clone(), D.counts(c)
    bit = T.cache.BAD_PAGE
    if wrong == "page":
        tables[1, 0] = -1
    elif wrong == "tail page":
        tables[1, 7] = c.pages + 5
    elif wrong == "shared":
        refs[c.tables[1, 2].long()], bit = 2, T.cache.SHARED_PAGE
    else:
        lengths[1], bit = -3, T.cache.BAD_INDEX
    k, v, w2, status = c.k.clone(), c.v.clone(), w.clone(), _status()
    got, out_refs = T.cache_evict(tables, lengths, refs, [(k, v, w2)], budget=30, recent=4, status=status)
    assert int(status) & bit and got.tolist() == [30, 60 if wrong != "long" else 0]
    page, slot = D.slots(c, 1, 60)
    assert torch.equal(k[page, slot], c.k[page, slot]) and torch.equal(v[page, slot], c.v[page, slot]) and torch.equal(w2[1], w[1])
    assert int(out_refs[c.tables[0, 4].long()]) == 0 and torch.equal(out_refs[page.unique()], refs[page.unique()])
    refs[c.tables[1, 5].long()] = 3  # (a page past the budget may be shared: it is only given up)
    if wrong == "shared":
        refs[c.tables[1, 2].long()] = 1
        got, out_refs = T.cache_evict(c.tables, c.lengths, refs, [(k, v, w2)], budget=30, recent=4)
        assert got.tolist() == [30, 30] and int(out_refs[c.tables[1, 5].long()]) == 2


def test_given_outputs_and_nothing_to_do():
    c = U.Cache("bf16", [60, 30], 2, 32, 8)
    refs, w = D.counts(c), torch.rand(2, 2, 64, device="cuda")
    out = (torch.full((2,), 7, dtype=torch.int32, device="cuda"), torch.full((c.pages,), 7, dtype=torch.int32, device="cuda"))
    got = T.cache_evict(c.tables, c.lengths, refs, [(c.k, c.v, w)], budget=100, out=out)
    assert got[0] is out[0] and torch.equal(out[0], c.lengths) and torch.equal(out[1], refs)
    got = T.cache_evict(c.tables[:0], c.lengths[:0], refs, [(c.k, c.v, w[:0])], budget=3, out=(out[0][:0], out[1].zero_()))
    assert torch.equal(out[1], refs)
    got = T.cache_accept(c.tables[:0], c.lengths[:0], refs, torch.zeros(0, 4, dtype=torch.int32, device="cuda"), c.lengths[:0], [c.k],
                         out=(out[0][:0], out[1].zero_()))
    assert torch.equal(out[1], refs)


# ---- streams and graphs --------------------------------------------------------------------------------------------

def _calls():
    c = U.Cache("bf16", [46, 26], 2, 64, 16, spare=4, columns=4)
    refs = D.counts(c)
    rng = np.random.RandomState(1)
    tokens, choices = _i32(rng.randint(0, 2, (2, 6))), _i32(rng.randint(0, 2, (2, 6)))
    parents = _i32(D.trees(2, 6, "tree"))
    q = torch.randn(2, 6, 4, 64, device="cuda").bfloat16()
    w = torch.rand(2, 2, 64, device="cuda")

    def drafts(s, q, t, n, p, kc, vc, w):
        return T.attention_drafts(q, kc, vc, t, n, parents=p, weights=w, stream=s), kc, vc, w

    def accept(s, t, n, r, path, counts, kc, vc):
        return *T.cache_accept(t, n, r, path, counts, [kc, vc], stream=s), kc, vc

    def evict(s, t, n, r, kc, vc, w):
        return *T.cache_evict(t, n, r, [(kc, vc, w)], budget=20, recent=5, stream=s), kc, vc, w
    path = torch.tensor([[0, 2, 5, -1, -1, -1], [1, 3, -1, -1, -1, -1]], dtype=torch.int32, device="cuda")
    return [(drafts, (q, c.tables, c.lengths, parents, c.k, c.v, w), 3),
            (lambda s, t, x, p: T.draft_path(t, x, parents=p, stream=s), (tokens, choices, parents), 0),
            (accept, (c.tables, c.lengths, refs, path, _i32([3, 2]), c.k, c.v), 2),
            (evict, (c.tables, c.lengths, refs, c.k, c.v, w), 3)]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("which", range(4))
def test_inputs_freed_after_the_call_stay_until_the_stream_is_done(which, raw):
    """A call on a busy stream, its inputs dropped right after and their memory asked for again on the current stream."""
    call, tensors, written = _calls()[which]
    want = [x.clone() for x in call(None, *[x.clone() for x in tensors])]
    side = torch.cuda.Stream()
    mine = [x.clone() for x in tensors]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # (about 0.1 s)
    got = call(side.cuda_stream if raw else side, *mine)
    like = [(x.shape, x.dtype) for x in mine[: len(mine) - written]]
    mine = x = None
    over = [torch.zeros(s, dtype=d, device="cuda") for s, d in like for _ in range(4)]
    torch.cuda.synchronize()
    assert over and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("which", range(1, 4))
def test_captured_and_replayed(which):
    call, tensors, written = _calls()[which]
    start = [x.clone() for x in tensors]
    mine = [x.clone() for x in tensors]
    want = [x.clone() for x in call(None, *mine)]
    side = torch.cuda.Stream()
    mine = [x.clone() for x in tensors]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = call(None, *mine)
    for _ in range(3):
        for x, y in zip(mine, start):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_budget_beyond_the_table():
    """... keeps every row as it is, with no more workspace than the table's tokens ask for."""
    c = U.Cache("bf16", [60, 30], 2, 32, 8)
    refs, w = D.counts(c), torch.rand(2, 2, 64, device="cuda")
    before = [x.clone() for x in (c.k, c.v, w)]
    lengths, out = T.cache_evict(c.tables, c.lengths, refs, [(c.k, c.v, w)], budget=2 ** 31 - 1, recent=2 ** 31 - 1)
    assert torch.equal(lengths, c.lengths) and torch.equal(out, refs)
    assert all(torch.equal(a, b) for a, b in zip(before, (c.k, c.v, w)))


def test_evicted_rows_go_on():
    """Rows are held to their budget, grow again, and are attended to: what is left is a cache like any other."""
    c = U.Cache("f32", [50, 20, 90], 2, 64, 8, spare=6, columns=14)
    w = torch.rand(3, 2, 14 * 8, device="cuda")
    refs = D.counts(c)
    kept = [D.evicted(w[r, h].tolist(), n, 32, 5) if n > 32 else list(range(n)) for r, n in enumerate((50, 20, 90)) for h in range(2)]
    keys, values = ([[x[D.slots(c, r, n)][:, h].clone() for h in range(2)] for r, n in enumerate((50, 20, 90))] for x in (c.k, c.v))
    lengths, refs = T.cache_evict(c.tables, c.lengths, refs, [(c.k, c.v, w)], budget=32, recent=5)
    tables, lengths, refs = T.cache_select(c.tables, lengths, refs, _i32([0, 1, 2]), [c.k, c.v], page_size=8, grow=_i32([1, 1, 1]))
    assert lengths.tolist() == [33, 21, 33]
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(3, h, 64, generator=gen, device="cuda") for h in (4, 2, 2))
    T.cache_append(k, v, c.k, c.v, tables, lengths - 1)
    out = T.attention_decode(q, c.k, c.v, tables, lengths)
    for r in range(3):
        for h in range(2):
            kk = torch.cat([keys[r][h][kept[2 * r + h]], k[r, h][None]]).double()
            vv = torch.cat([values[r][h][kept[2 * r + h]], v[r, h][None]]).double()
            for i in (2 * h, 2 * h + 1):
                want = torch.softmax(kk @ q[r, i].double() / 8, 0) @ vv
                # (33 terms of values below 5 and scores below 8 in 32 bits)
                assert float((out[r, i].double() - want).abs().max()) < 64 * 2.0 ** -24 * 5 * 8


@pytest.mark.parametrize("kind,heads,dim,order,pad", [("bf16", 2, 64, "slots", 0), ("f32", 3, 33, "heads", 0), ("f16", 1, 256, "slots", 0),
                                                      ("bf16", 8, 128, "heads", 0), ("bf16", 2, 96, "both", 1), ("f32", 20, 40, "slots", 0)])
@pytest.mark.parametrize("budget,recent", [(3001, 100), (513, 512), (4999, 4999)])
def test_evict_long_lists(kind, heads, dim, order, pad, budget, recent):
    """Lists that several CTAs move side by side, most tokens by a few slots, or by thousands."""
    _evict(kind, [5000, 3002, 40], heads, dim, 16, budget, recent, order, pad=pad)
