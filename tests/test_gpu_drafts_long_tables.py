"""Cases of test_gpu_drafts whose few queries and short tables take the warp-level instructions there, in tables with room for
2048 tokens, where they take the CTA-wide ones; and every kernel in a graph that goes on with other lengths."""
from __future__ import annotations

import math

import pytest
import torch

import cacheutil as U
import draftutil as D
import tensor_command_execution_gb300 as T
import test_gpu_drafts as S

pytestmark = pytest.mark.gpu

KINDS = ["f16", "bf16"]


@pytest.fixture()
def room(monkeypatch):
    class Room(U.Cache):
        def __init__(self, kind, lengths, heads, dim, page, *args, columns=0, **named):
            super().__init__(kind, lengths, heads, dim, page, *args, columns=max([columns, -(-2048 // page)] + [-(-n // page) for n in lengths]),
                             **named)
    monkeypatch.setattr(U, "Cache", Room)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("drafts", [2, 7, 16])
@pytest.mark.parametrize("tree", [None, "tree", "forest", "star"])
def test_numbers_of_drafts_and_trees(room, kind, drafts, tree):
    S.test_numbers_of_drafts_and_trees(kind, drafts, tree)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hk", [(8, 8), (8, 2), (7, 1), (10, 5)])
def test_heads(room, kind, hq, hk):
    S.test_heads(kind, hq, hk)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [8, 40, 64, 72, 96, 128])
@pytest.mark.parametrize("drafts", [3, 10])
def test_dims(room, kind, dim, drafts):
    S.test_dims(kind, dim, drafts)


@pytest.mark.parametrize("page", [1, 3, 16, 24, 32, 128])
@pytest.mark.parametrize("order", ["slots", "heads", "both"])
def test_pages(room, page, order):
    S._check("bf16", [0, 2, 31, 97, 256, 413], 4, 8, 2, 128, page, order)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("softcap,window", [(20.0, 0), (0.0, 1), (0.0, 3), (0.0, 17), (5.0, 100), (0.0, 1000), (0.0, 2 ** 31 - 1)])
def test_cap_and_window(room, kind, softcap, window):
    S._check(kind, [0, 1, 16, 99, 100, 101, 400], 6, 4, 2, 96, 16, softcap=softcap, window=window)


@pytest.mark.parametrize("kind", KINDS)
def test_padding_gives_zeros(room, kind):
    S.test_padding_gives_zeros(kind, 4)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf, "lowest"])
def test_what_is_not_in_the_row_does_not_enter(room, kind, junk):
    S.test_what_is_not_in_the_row_does_not_enter(kind, junk, 4)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dim", [64, 128])
def test_other_branches_do_not_enter(room, kind, junk, dim):
    S.test_other_branches_do_not_enter(kind, junk, dim, 6)


@pytest.mark.parametrize("kind", KINDS)
def test_windows_and_extreme_scores(room, kind):
    S.test_tokens_before_a_window_do_not_enter(kind)
    S._check(kind, [50, 3], 5, 2, 1, 32, 16, scale=30.0)


def test_strides_and_bad_tables(room):
    S.test_strides("bf16", 3)
    S.test_bad_pages_and_lengths("bf16", 2)


def test_many_rows(room):
    S.test_many_rows()


def test_pools_past_32_bits():
    """Pages whose elements lie past 2^32."""
    pages = (1 << 32) // (16 * 64) + 40
    both = torch.empty(pages, 16, 1, 64, dtype=torch.bfloat16, device="cuda")
    at = torch.full((1, 130), -5, dtype=torch.int32, device="cuda")
    at[0, :3] = torch.tensor([0, pages - 1, pages - 17])
    both[at[0, :3].long()] = S._randn(3, 16, 1, 64, kind="bf16")
    q, n = S._randn(1, 5, 2, 64, kind="bf16", seed=1), torch.tensor([44], dtype=torch.int32, device="cuda")
    small, near = both[at[0, :3].long()].clone(), at.clone()
    near[0, :3] = torch.arange(3)
    weights = torch.zeros(2, 1, 1, 130 * 16, device="cuda")
    a = T.attention_drafts(q, both, both, at, n, weights=weights[0])
    b = T.attention_drafts(q, small, small, near, n, weights=weights[1])
    assert torch.equal(a, b) and torch.equal(weights[0], weights[1])


@pytest.mark.parametrize("kind,drafts,hq,dim,page,columns", [
    ("bf16", 1, 8, 128, 16, 40), ("bf16", 1, 8, 33, 16, 40), ("f32", 1, 8, 64, 16, 40),      # one token
    ("bf16", 3, 8, 128, 16, 20), ("f16", 4, 8, 64, 16, 70), ("bf16", 6, 6, 192, 8, 40),      # warp-level, teams or not
    ("bf16", 3, 8, 100, 16, 40), ("f16", 3, 8, 33, 16, 40),
    ("bf16", 3, 8, 128, 16, 200), ("f16", 40, 16, 64, 8, 40), ("bf16", 24, 8, 128, 3, 200),  # CTA-wide, by both kinds of copies
    ("f32", 4, 8, 80, 16, 40), ("f32", 30, 8, 80, 16, 40)])                                  # 32 bits, blocks of 16 and of 64
def test_captured_with_weights_and_replayed(kind, drafts, hq, dim, page, columns):
    """On other lengths, trees and numbers than it was captured with: what a call gives."""
    most = columns * page
    c = U.Cache(kind, [most, most // 2, drafts], 2, dim, page, columns=columns)
    q, parents = S._randn(3, drafts, hq, dim, kind=kind), S._i32(D.trees(3, drafts, "tree"))
    c.tables.clamp_(max=c.pages - 1)  # (rows grow into others' pages: they are only read)
    weights, out, lse = torch.zeros(3, 2, most, device="cuda"), torch.empty_like(q), torch.empty(3, drafts, hq, device="cuda")

    def call():
        T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, parents=parents, out=out, lse=lse, return_lse=True, weights=weights)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for seed, lengths in enumerate(([most, most // 2, drafts], [drafts, 0, most], [0, 0, 0], [most - 1, most, drafts + 1])):
        q.copy_(S._randn(3, drafts, hq, dim, kind=kind, seed=seed + 5))
        parents.copy_(S._i32(D.trees(3, drafts, "padded", seed)))
        c.lengths.copy_(S._i32(lengths))
        weights.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (out, lse, weights)]
        weights.zero_()
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, lse, weights))), seed
        assert bool(torch.isfinite(out).all()) and bool((lse[2] == -math.inf).all()) == (lengths[2] == 0 or all(x is None for x in D.seen_by(parents[2].tolist())))
