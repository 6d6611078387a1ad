"""The operators of a paged cache against their plain forms in 64 bits."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import tensor_command_execution_gb300 as T
import cacheutil as U
from tensor_command_execution_gb300.cache import cmd_attention_workspace

pytestmark = pytest.mark.gpu


def _randn(*shape, kind, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(U.TYPES[kind])


def _near(got, want, bound, what=""):
    off = (got.detach().cpu().double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {float((off / bound.clamp(min=1e-300)).max()):.3g} of the bound"


def _same_bits(a, b):
    kind = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


# ---- rotary positions ----------------------------------------------------------------------------------------------

ROPE_SHAPES = [  # batch, tokens, q heads, k heads, dim, rotated
    (2, 5, 4, 2, 128, 128), (1, 1, 1, 1, 64, 64), (3, 7, 3, 3, 80, 32), (1, 9, 5, 1, 72, 72), (2, 3, 2, 2, 256, 256),
    (1, 4, 130, 2, 64, 48), (1, 6, 2, 1, 10, 6), (2, 4, 3, 1, 33, 20), (1, 2, 1, 1, 2, 2), (1, 3, 2, 2, 16, 0),
    (2, 3001, 1, 1, 16, 8), (1, 5003, 2, 0, 32, 32),
    (2, 9, 17, 3, 72, 36), (1, 7, 20, 20, 80, 40), (1, 5, 9, 2, 20, 12), (2, 3, 31, 1, 36, 36), (1, 8, 3, 3, 22, 10),
]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("shape", ROPE_SHAPES, ids=str)
def test_rope_and_its_gradient(shape, layout, kind):
    b, t, hq, hk, dim, rot = shape
    q, k = _randn(b, t, hq, dim, kind=kind), _randn(b, t, hk, dim, kind=kind, seed=1)
    turns = T.rope_turns(rot, 10000.0)
    positions = torch.randint(-(1 << 31), (1 << 31) - 1, (b, t), dtype=torch.int64).to(torch.int32)
    positions.view(-1)[0] = 0
    for f, backward, scale in ((T.rope, False, 1.0), (T.rope_backward, True, 1.25)):
        got = f(q, k, positions.cuda(), turns, layout=layout, scale=scale)
        for x, y in zip((q, k), got):
            want = U.rotated(x, positions, turns, layout, scale, backward)
            _near(y, want, U.rope_bound(x, want, rot // 2, layout, scale, kind), (f.__name__, shape))
            assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_gradient_against_differences(layout):
    """The rotation is linear, so a difference quotient with step 1 is its derivative up to rounding: the gradient
    of sum(w * rope(x)) is rope_backward(w)."""
    x, w = _randn(1, 3, 2, 24, kind="f32"), _randn(1, 3, 2, 24, kind="f32", seed=1)
    positions = torch.tensor([[3, 70000, 1 << 30]], dtype=torch.int32, device="cuda")
    turns = T.rope_turns(16, 10000.0)
    grad, none = T.rope_backward(w, None, positions, turns, layout=layout, scale=0.75)
    assert none is None
    base = T.rope(x, None, positions, turns, layout=layout, scale=0.75)[0].double()
    for e in range(x.numel()):
        step = x.clone()
        step.view(-1)[e] += 1.0
        moved = T.rope(step, None, positions, turns, layout=layout, scale=0.75)[0].double()
        quotient = float(((moved - base) * w.double()).sum() / (step.view(-1)[e].double() - x.view(-1)[e].double()))
        # two rotations, of values up to 6, rounded to 2^-24 in two places of a pair, times weights up to 4
        assert abs(quotient - float(grad.view(-1)[e])) < 2 * 2 * 8 * 2.0 ** -24 * 12 * 4


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_strides_and_in_place(layout, kind):
    """Heads outermost, slices of a fused projection, an element off the vector alignment, broadcast inputs and
    positions, and in place."""
    turns = T.rope_turns(32, 500000.0, scaling="linear", factor=4.0)
    positions = torch.arange(6, dtype=torch.int32, device="cuda") * 1000

    def check(q, k, pos, out=None):
        want = [U.rotated(x, pos.expand(x.shape[:-2]), turns, layout, 1.0) for x in (q, k)]
        bounds = [U.rope_bound(x, w, 16, layout, 1.0, kind) for x, w in zip((q, k), want)]
        got = T.rope(q, k, pos, turns, layout=layout, out=out)
        for y, w, e in zip(got, want, bounds):
            _near(y, w, e)
        return got

    heads_first = _randn(2, 3, 6, 48, kind=kind).transpose(1, 2)
    check(heads_first, _randn(2, 1, 6, 48, kind=kind).transpose(1, 2), positions.expand(2, 6))
    fused = _randn(6, 5, 48, kind=kind)
    before = fused.clone()
    got = check(fused[:, :3], fused[:, 3:4], positions, out=(fused[:, :3], fused[:, 3:4]))
    assert got[0].data_ptr() == fused.data_ptr() and torch.equal(fused[:, 4], before[:, 4])
    odd = _randn(6 * 4 * 49 + 1, kind=kind)[1:].view(6, 4, 49)[..., :48]
    check(odd[:, :2], odd[:, 2:], positions)
    wide = _randn(1, 6, 2, 48, kind=kind).expand(3, 6, 2, 48)
    check(wide, wide[:, :, :1], positions.expand(3, 6))
    check(fused[:0, :3], fused[:0, 3:4], positions[:0])


def test_rope_every_pair_of_a_long_context():
    """Positions up to 2^31 - 1: the angle is as good there as at 1."""
    for p in (1, 4095, 131071, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31), -1):
        x = torch.ones(1, 1, 256, device="cuda")
        turns = T.rope_turns(256, 1e6, scaling="parts", factor=32.0, original_length=4096.0)
        pos = torch.tensor([p], dtype=torch.int32, device="cuda")
        y = T.rope(x, None, pos, turns)[0]
        want = U.rotated(x, pos, turns, "half", 1.0)
        _near(y, want, U.rope_bound(x, want, 128, "half", 1.0, "f32"), p)


def test_rope_in_autograd():
    """The pair as a differentiable function, with a broadcast input: its gradient is the sum over what it fed."""
    turns, pos = T.rope_turns(32), torch.arange(7, dtype=torch.int32, device="cuda") * 999

    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return T.rope(x, None, pos.expand(x.shape[:2]), turns, layout="interleaved", scale=1.5)[0]

        @staticmethod
        def backward(ctx, g):
            return T.rope_backward(g, None, pos.expand(g.shape[:2]), turns, layout="interleaved", scale=1.5)[0]

    x = _randn(1, 7, 3, 40, kind="f32").requires_grad_()
    w = _randn(4, 7, 3, 40, kind="f32", seed=1)
    (Rope.apply(x.expand(4, 7, 3, 40)) * w).sum().backward()
    want = U.rotated(w, pos.expand(4, 7), turns, "interleaved", 1.5, backward=True).sum(0, keepdim=True)
    bound = U.rope_bound(w, w.cpu().double() * 0, 16, "interleaved", 1.5, "f32").sum(0, keepdim=True) + 8 * 2.0 ** -24 * want.abs()
    _near(x.grad, want, bound + 4 * 2.0 ** -24 * w.cpu().double().abs().sum(0, keepdim=True) * 1.5)


# ---- append --------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("order", ["slots", "heads", "both"])
@pytest.mark.parametrize("layout,dim,rot,page", [("half", 128, 128, 16), ("interleaved", 80, 40, 7), ("half", 33, 10, 1)])
def test_append(kind, order, layout, dim, rot, page):
    lengths = [19, 1, 40, 3]
    c = U.Cache(kind, lengths, 2, dim, page, order)
    rows, positions = [], []
    for r, n in enumerate(lengths):  # each row's tokens but its first ones, and a padding token
        rows += [r] * (n - n // 2 + 1)
        positions += list(range(n // 2, n)) + [-1]
    order_ = np.random.RandomState(3).permutation(len(rows))
    rows, positions = np.array(rows)[order_], np.array(positions)[order_]
    n = len(rows)
    q, k, v = (_randn(n, h, dim, kind=kind, seed=s) for s, h in ((4, 6), (5, 2), (6, 2)))
    turns = T.rope_turns(rot, 10000.0)
    want_k, want_v = c.k.clone(), c.v.clone()
    pos = torch.tensor(positions, dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got_q = T.cache_append(k, v, c.k, c.v, c.tables, pos.cuda(), rows=torch.tensor(rows, dtype=torch.int32).cuda(), q=q,
                           turns=turns, layout=layout, scale=1.5, status=status)
    T.cache_status(status)
    want_q = U.rotated(q, pos, turns, layout, 1.5)
    _near(got_q, want_q, U.rope_bound(q, want_q, rot // 2, layout, 1.5, kind))
    turned = U.rotated(k, pos, turns, layout, 1.5)
    bound = U.rope_bound(k, turned, rot // 2, layout, 1.5, kind)
    written = torch.zeros(c.pages, page, dtype=torch.bool)
    for i in range(n):
        if positions[i] < 0:
            continue
        at, slot = int(c.tables[rows[i], positions[i] // page]), positions[i] % page
        written[at, slot] = True
        _near(c.k[at, slot], turned[i], bound[i])
        assert _same_bits(c.v[at, slot], v[i])
    keep = ~written.cuda()
    assert _same_bits(c.k[keep], want_k[keep]) and _same_bits(c.v[keep], want_v[keep])


def test_append_without_rotation_or_rows():
    c = U.Cache("bf16", [5, 9, 2], 3, 24, 4)
    k, v = _randn(3, 3, 24, kind="bf16"), _randn(3, 3, 24, kind="bf16", seed=1)
    pos = torch.tensor([4, 8, 1], dtype=torch.int32, device="cuda")
    assert T.cache_append(k, v, c.k, c.v, c.tables, pos) is None
    for r, p in enumerate([4, 8, 1]):
        page = int(c.tables[r, p // 4])
        assert _same_bits(c.k[page, p % 4], k[r]) and _same_bits(c.v[page, p % 4], v[r])


def test_append_reports_what_it_cannot_store():
    """A page number outside the pool, a row outside the tables and a position past them: nothing is stored for
    those tokens, the others are, and the status says so."""
    c = U.Cache("f32", [8, 8], 1, 8, 4, columns=2)
    before = c.k.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.tables[1, 1] = c.pages
    k, v = _randn(5, 1, 8, kind="f32"), _randn(5, 1, 8, kind="f32", seed=1)
    rows = torch.tensor([0, 1, 2, -1, 0], dtype=torch.int32, device="cuda")
    pos = torch.tensor([3, 5, 0, 0, 8], dtype=torch.int32, device="cuda")
    T.cache_append(k, v, c.k, c.v, c.tables, pos, rows=rows, status=status)
    with pytest.raises(T.CmdError) as e:
        T.cache_status(status)
    assert e.value.name == "CMD_ERR_ARG" and "page" in str(e.value) and "row" in str(e.value)
    T.cache_status(status)  # (cleared)
    before[int(c.tables[0, 0]), 3] = k[0]
    assert torch.equal(c.k, before)


# ---- attention -------------------------------------------------------------------------------------------------------

def _attend(kind, lengths, hq, hk, dim, page, order="slots", softcap=0.0, window=0, seed=0, junk=math.nan, pad=0, scale=None,
            q=None):
    """Both ways of dealing out the work: with tables as long as the rows (few short rows go to teams of CTAs), and with
    tables that could hold far more tokens."""
    q = 2 * _randn(len(lengths), hq, dim, kind=kind, seed=seed + 1) if q is None else q
    most = -(-max(lengths) // page)
    for columns in (max(most, 1), most + 5000 // page):
        c = U.Cache(kind, lengths, hk, dim, page, order, seed=seed, junk=junk, pad=pad, columns=columns)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = T.attention_decode(q, c.k, c.v, c.tables, c.lengths, softcap=softcap, window=window, scale=scale,
                                      return_lse=True, status=status)
        T.cache_status(status)
        want, want_lse, bound, lse_bound = U.attended(q, c, lengths, dim ** -0.5 if scale is None else scale, softcap, window)
        # the weights of 16-bit caches are held as two 16-bit numbers: 2^-16 of each (bf16), 2^-21 (f16)
        split = {"f32": 0.0, "f16": 2.0 ** -21, "bf16": 2.0 ** -16}[kind]
        top = torch.stack([c.rows(r, n)[1].abs().amax() if n else torch.zeros(()).double() for r, n in enumerate(lengths)])
        bound = bound + split * top[:, None, None] + U.ROUND[kind] * want.abs() * (1 + 2.0 ** -10) + U.TINY[kind]
        _near(out, want, bound, "out")
        empty = torch.isinf(want_lse)
        assert torch.equal(torch.isinf(lse.cpu()) & (lse.cpu() < 0), empty)
        _near(torch.where(empty.cuda(), 0.0, lse), torch.where(empty, 0.0, want_lse), lse_bound, "lse")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lengths", [[1], [64], [65], [700], [1500], [2048], [0], [33, 2000], [512, 0, 1, 900]], ids=str)
@pytest.mark.parametrize("window", [0, 150])
def test_attention_few_short_rows(kind, lengths, window):
    """Teams of one, two, four and eight CTAs, with no, one and several tiles to a CTA."""
    _attend(kind, lengths, 6, 2, 80, 16, window=window)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,hk", [(8, 8), (8, 2), (32, 4), (7, 1), (10, 5), (24, 2), (33, 1), (48, 3)])
def test_attention_heads(kind, hq, hk):
    _attend(kind, [0, 1, 15, 16, 17, 130, 333], hq, hk, 64, 16)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [1, 8, 20, 33, 40, 64, 72, 80, 96, 128, 136, 192, 256])
def test_attention_dims(kind, dim):
    _attend(kind, [3, 64, 201], 6, 2, dim, 8)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("page", [1, 3, 16, 24, 32, 128])
@pytest.mark.parametrize("order", ["slots", "heads", "both"])
def test_attention_pages(kind, page, order):
    _attend(kind, [0, 2, 31, 97, 256, 413], 8, 2, 128, page, order)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("softcap,window", [(20.0, 0), (0.0, 1), (0.0, 17), (5.0, 100), (0.0, 1000)])
def test_attention_cap_and_window(kind, softcap, window):
    _attend(kind, [0, 1, 16, 99, 100, 101, 400], 8, 2, 96, 16, softcap=softcap, window=window)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_attention_long_rows_are_split_and_joined(kind):
    """Rows whose tiles go to many CTAs, next to short ones."""
    _attend(kind, [20011, 5, 0, 4097], 4, 1, 64, 32, seed=2)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_attention_many_rows(kind):
    """More rows than one launch takes, most of them empty or short."""
    rng = np.random.RandomState(5)
    _attend(kind, [int(x) for x in rng.randint(0, 4, 2100)], 2, 1, 16, 2)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf, "lowest"])
def test_attention_ignores_what_is_not_in_the_row(kind, junk):
    """Slots past a row's length and pages of no row, and with a window the tokens before it."""
    junk = torch.finfo(U.TYPES[kind]).min if junk == "lowest" else junk
    _attend(kind, [0, 1, 37, 128, 129], 8, 2, 128, 32, junk=junk)
    lengths, window = [70, 33], 20
    c = U.Cache(kind, lengths, 2, 64, 16)
    clean = U.Cache(kind, lengths, 2, 64, 16)
    for r, n in enumerate(lengths):
        for i in range(n - window):
            c.k[c.tables[r, i // 16].item(), i % 16] = junk
            c.v[c.tables[r, i // 16].item(), i % 16] = junk
    q = _randn(2, 4, 64, kind=kind)
    a = T.attention_decode(q, c.k, c.v, c.tables, c.lengths, window=window)
    b = T.attention_decode(q, clean.k, clean.v, clean.tables, clean.lengths, window=window)
    assert _same_bits(a, b)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_attention_extreme_scores(kind):
    """Scores far apart (one token takes all), and a row whose scores are all -infinity."""
    _attend(kind, [50, 50], 2, 1, 32, 16, scale=30.0)
    c = U.Cache(kind, [40], 1, 32, 16)
    c.k[...] = 0
    c.k[..., 0] = -math.inf
    q = torch.zeros(1, 1, 32, device="cuda", dtype=U.TYPES[kind])
    q[..., 0] = 1
    out, lse = T.attention_decode(q, c.k, c.v, c.tables, c.lengths, return_lse=True)
    assert torch.equal(out, torch.zeros_like(out)) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_attention_strides(kind):
    """Rows of the cache padded (to an odd and to a vector's pitch), queries out of a fused projection, outputs into
    a wider tensor."""
    for pad in (1, 8):
        _attend(kind, [5, 77, 140], 4, 2, 64, 16, pad=pad)
    wide = _randn(3, 12, 65, kind=kind, seed=9)
    _attend(kind, [5, 77, 140], 4, 2, 64, 16, q=wide[:, 3:7, 1:])
    c = U.Cache(kind, [30, 31], 2, 64, 16)
    q = _randn(2, 4, 64, kind=kind)
    room = torch.full((2, 9, 64), 7.0, device="cuda", dtype=U.TYPES[kind])
    got = T.attention_decode(q, c.k, c.v, c.tables, c.lengths, out=room[:, 2:6])
    assert _same_bits(got, T.attention_decode(q, c.k, c.v, c.tables, c.lengths))
    assert bool((room[:, :2] == 7).all()) and bool((room[:, 6:] == 7).all())


def test_attention_skips_bad_pages_and_lengths():
    c = U.Cache("bf16", [64, 64, 64], 2, 64, 16)
    good = T.attention_decode(_randn(3, 4, 64, kind="bf16"), c.k, c.v, c.tables, c.lengths)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.tables[1, 2] = -5
    c.tables[2, 0] = c.pages
    got = T.attention_decode(_randn(3, 4, 64, kind="bf16"), c.k, c.v, c.tables, c.lengths, status=status)
    with pytest.raises(T.CmdError, match="page"):
        T.cache_status(status)
    assert _same_bits(got[0], good[0]) and bool(torch.isfinite(got).all())
    lengths = torch.tensor([64, -3, 1 << 30], dtype=torch.int32, device="cuda")
    c.tables[2, 0] = c.tables[0, 0]
    got = T.attention_decode(_randn(3, 4, 64, kind="bf16"), c.k, c.v, c.tables, lengths, status=status)
    with pytest.raises(T.CmdError, match="length"):
        T.cache_status(status)
    assert _same_bits(got[0], good[0]) and bool((got[1] == 0).all())


def test_attention_on_streams_and_in_a_graph():
    """Other streams with workspaces of their own, twice the same bits, and a captured step whose lengths change."""
    c = U.Cache("bf16", [3000, 40, 700], 2, 128, 16)
    q = _randn(3, 8, 128, kind="bf16")
    want = T.attention_decode(q, c.k, c.v, c.tables, c.lengths)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = [T.attention_decode(q, c.k, c.v, c.tables, c.lengths, stream=s) for s in side for _ in range(3)]
    torch.cuda.synchronize()
    assert all(_same_bits(x, want) for x in got)
    out, lengths = torch.empty_like(q), c.lengths.clone()
    ws = torch.full((cmd_attention_workspace(8, 2, 128),), 255, dtype=torch.uint8, device="cuda")  # (any contents)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        T.attention_decode(q, c.k, c.v, c.tables, lengths, out=out, workspace=ws)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert _same_bits(out, want)
    lengths.copy_(torch.tensor([17, 0, 699]))
    g.replay()
    torch.cuda.synchronize()
    assert _same_bits(out, T.attention_decode(q, c.k, c.v, c.tables, lengths))


def test_a_whole_step_in_a_graph():
    """Selection, append and attention captured without buffers of their own; replayed, they do what the calls do."""
    c = U.Cache("bf16", [33, 16, 5], 2, 64, 16, spare=12, columns=4)
    refs = torch.zeros(c.pages, dtype=torch.int32, device="cuda")
    for r, n in enumerate(c.need):
        refs[c.tables[r, :n].long()] += 1
    parents, one = torch.tensor([1, 0, 0], dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")
    q, k, v = (_randn(3, h, 64, kind="bf16", seed=h) for h in (8, 2, 2))
    turns, pools = T.rope_turns(64), [c.k, c.v]

    def step():
        t, n, r = T.cache_select(c.tables, c.lengths, refs, parents, pools, page_size=16, grow=one)
        x = T.cache_append(k, v, c.k, c.v, t, n - 1, q=q, turns=turns)
        return t, n, r, T.attention_decode(x, c.k, c.v, t, n)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [x.clone() for x in step()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = step()
    for new in ([1, 0, 0], [1, 0, 0], [2, 2, -1]):  # (the last takes the pages of rows 0 and 1)
        parents.copy_(torch.tensor(new))
        g.replay()
        torch.cuda.synchronize()
        if new[2] == 0:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        else:
            assert got[1].tolist() == [6, 6, 1] and int((got[2] > 0).sum()) == 3


# ---- pages -----------------------------------------------------------------------------------------------------------

def _select_case(seed, rows, new_rows, page, columns, spare, longest, grow, dim=16, heads=2, kind="bf16", order="slots"):
    rng = np.random.RandomState(seed)
    lengths = [int(x) for x in rng.randint(0, longest + 1, rows)]
    c = U.Cache(kind, lengths, heads, dim, page, order, spare=spare, columns=columns, seed=seed)
    refs = np.zeros(c.pages, dtype=np.int32)
    t = c.tables.cpu().numpy()
    for r, n in enumerate(c.need):
        refs[t[r, :n]] += 1
    held = np.flatnonzero(refs == 0)[:1]
    refs[held] = 1  # a page held by no row
    parents = rng.randint(-1, rows, new_rows)
    return c, lengths, refs, parents, rng.randint(0, grow + 1, new_rows)


@pytest.mark.parametrize("rows,new_rows,page,columns,spare,longest,grow", [
    (4, 4, 4, 8, 40, 20, 3), (1, 9, 16, 3, 30, 37, 1), (7, 3, 1, 40, 10, 30, 5), (40, 64, 8, 12, 300, 80, 16),
    (300, 300, 16, 9, 900, 128, 1), (5, 5, 4, 6, 2, 20, 8), (16, 33, 4, 3, 12, 12, 9), (2000, 3000, 2, 5, 9000, 8, 2),
], ids=str)
@pytest.mark.parametrize("order", ["slots", "heads", "both"])
def test_select(rows, new_rows, page, columns, spare, longest, grow, order):
    """Against the row-by-row selection: ample room, a pool that runs out, tables that are too short."""
    c, lengths, refs, parents, more = _select_case(rows + page, rows, new_rows, page, columns, spare, longest, grow, order=order)
    want = U.select_reference(c.tables.cpu().numpy(), lengths, refs, parents, more, page)
    pools = [p.clone() if order != "heads" else p.transpose(1, 2).clone() for p in (c.k, c.v)]
    expect = [p.clone() for p in pools]
    for p in expect:
        for a, b in want[3]:
            p[b] = p[a]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def i32(x):
        return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")
    got = T.cache_select(c.tables, c.lengths, i32(refs), i32(parents), pools, page_size=page, grow=i32(more), status=status)
    for g, w, n in zip(got, want, ("tables", "lengths", "refs")):
        assert np.array_equal(g.cpu().numpy(), w), n
    for p, w in zip(pools, expect):
        assert _same_bits(p, w)
    dropped = any(n == 0 and (p >= 0 and lengths[p] or m) for n, p, m in zip(want[1], parents, more))
    if dropped:
        with pytest.raises(T.CmdError) as e:
            T.cache_status(status)
        assert e.value.name == "CMD_ERR_LIMIT"
    else:
        T.cache_status(status)


def test_select_shared_pages_stay_shared():
    """Two generations of forks: shared pages are counted, a fork's copy holds its parent's values, and dropping all
    rows frees everything."""
    c = U.Cache("f32", [37], 1, 8, 16, spare=8, columns=5)
    refs = torch.zeros(c.pages, dtype=torch.int32, device="cuda")
    refs[c.tables[0, :3].long()] = 1
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    pools = [c.k, c.v]
    t, n, r = T.cache_select(c.tables, c.lengths, refs, zero, pools, page_size=16)
    assert n.tolist() == [37] * 3 and sorted(r.tolist(), reverse=True)[:5] == [3, 3, 1, 1, 1] and int(r.sum()) == 9
    for i in (1, 2):
        assert torch.equal(c.k[int(t[i, 2])][:5], c.k[int(t[0, 2])][:5]) and int(t[i, 2]) != int(t[0, 2])
    t, n, r = T.cache_select(t, n, r, torch.tensor([2, 2], dtype=torch.int32, device="cuda"), pools, page_size=16,
                             grow=torch.tensor([11, 12], dtype=torch.int32, device="cuda"))
    assert n.tolist() == [48, 49] and int(r.sum()) == 3 + 4 and int((r > 0).sum()) == 2 + 1 + 2
    t, n, r = T.cache_select(t, n, r, torch.tensor([-1], dtype=torch.int32, device="cuda"), pools, page_size=16)
    assert n.tolist() == [0] and int(r.abs().sum()) == 0 and bool((t == -1).all())


def test_select_bad_indices():
    c = U.Cache("f32", [20, 20], 1, 8, 8, spare=4, columns=4)
    refs = torch.zeros(c.pages, dtype=torch.int32, device="cuda")
    for i in range(2):
        refs[c.tables[i, :3].long()] = 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.tables[1, 2] = c.pages + 7
    parents = torch.tensor([0, 7, -9, 1, 1], dtype=torch.int32, device="cuda")
    t, n, r = T.cache_select(c.tables, c.lengths, refs, parents, [c.k], page_size=8, status=status,
                             grow=torch.tensor([0, 0, 0, 0, -4], dtype=torch.int32, device="cuda"))
    assert n.tolist() == [20, 0, 0, 20, 20]
    with pytest.raises(T.CmdError, match="page.*row"):
        T.cache_status(status)


@pytest.mark.parametrize("pages,rows,page,move", [(1, 1, 4, 0), (40, 5, 4, 7), (601, 9, 8, 150), (9000, 50, 2, 2000), (64, 4, 16, 0)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_compact(pages, rows, page, move, kind):
    rng = np.random.RandomState(pages)
    live = max(1, pages // 2)
    numbers = rng.permutation(np.concatenate([rng.permutation(live)[: live - move],
                                              live + rng.permutation(pages - live)[:move]])).astype(np.int32)
    columns = -(-live // rows) + 1
    t = np.full((rows, columns), 0x7ffffff0, dtype=np.int32)
    lengths = []
    for r in range(rows):
        part = numbers[r * (columns - 1):(r + 1) * (columns - 1)]
        part = part[: max(0, len(part) - r % 2)]  # (pages held outside the tables)
        t[r, : len(part)] = part
        lengths.append(len(part) * page - (r % page if len(part) else 0))
    refs = np.zeros(pages, dtype=np.int32)
    refs[numbers] = rng.randint(1, 4, len(numbers))
    pools = [_randn(pages, page, 3, 10, kind=kind), _randn(pages, 2, 6, kind=kind, seed=1)]
    used = refs > 0
    n = int(used.sum())
    of, to = np.flatnonzero(used & (np.arange(pages) >= n)), np.flatnonzero(~used & (np.arange(pages) < n))
    where = np.where(used, np.arange(pages), -1)
    where[of] = to
    want_refs = np.zeros(pages, dtype=np.int32)
    want_refs[where[used]] = refs[used]
    want_t = np.full_like(t, -1)
    for r in range(rows):
        k = -(-lengths[r] // page)
        want_t[r, :k] = where[t[r, :k]]
    expect = [p.clone() for p in pools]
    for p, e in zip(pools, expect):
        e[torch.from_numpy(to).cuda()] = p[torch.from_numpy(of).cuda()]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = T.cache_compact(torch.from_numpy(t).cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                          torch.from_numpy(refs).cuda(), pools, page_size=page, status=status)
    T.cache_status(status)
    assert np.array_equal(got[0].cpu().numpy(), want_t) and np.array_equal(got[1].cpu().numpy(), want_refs)
    assert np.array_equal(got[2].cpu().numpy(), where)
    for p, e in zip(pools, expect):
        assert _same_bits(p, e)


def test_pages_of_any_alignment():
    """Pages of an odd number of bytes' alignment, padded strides, and a base off the vector alignment."""
    for make in (lambda: _randn(12, 3, 7, kind="bf16"), lambda: _randn(12, 4, 16, kind="bf16")[:, :3],
                 lambda: _randn(12 * 8 + 1, kind="bf16")[1:].view(12, 8), lambda: _randn(12, 5, kind="f32"),
                 lambda: _randn(12, 4, 6, kind="bf16").transpose(1, 2), lambda: torch.randint(0, 255, (12, 9), dtype=torch.uint8, device="cuda")):
        pool = make()
        want = pool.clone()
        refs = torch.tensor([0, 1, 0, 0, 1, 1, 0, 0, 0, 1, 0, 1], dtype=torch.int32, device="cuda")
        tables = torch.tensor([[9, 11], [4, 1]], dtype=torch.int32, device="cuda")
        lengths = torch.tensor([2, 2], dtype=torch.int32, device="cuda")
        t, r, m = T.cache_compact(tables, lengths, refs, [pool], page_size=1)
        assert t.tolist() == [[2, 3], [4, 1]] and m.tolist() == [-1, 1, -1, -1, 4, 0, -1, -1, -1, 2, -1, 3]
        assert r.tolist() == [1] * 5 + [0] * 7
        used = [i for i, x in enumerate(refs.tolist()) if x]
        n = len(used)
        pairs = list(zip([i for i in used if i >= n], [i for i in range(n) if i not in used]))
        for a, b in pairs:
            want[b] = want[a]
        assert torch.equal(pool, want)


@pytest.mark.parametrize("kind,dim", [("bf16", 256), ("f32", 256), ("bf16", 255)])
def test_a_pool_past_32_bits(kind, dim):
    """Pages at element offsets above 2^32: appended to, attended to, copied by a selection and moved by a compaction
    as the same values in a small pool are."""
    pages, page, heads = (1 << 32) // (16 * 16 * dim) + 40, 16, 16
    big = [torch.empty(pages, page, heads, dim, device="cuda", dtype=U.TYPES[kind]) for _ in range(2)]
    assert big[0].stride(0) * (pages - 9) > 1 << 32
    small = U.Cache(kind, [40, 20], heads, dim, page)
    where = {p: pages - 9 + p for p in range(small.pages)}
    assert small.pages <= 9
    for a, b in zip(big, (small.k, small.v)):
        a[pages - 9: pages - 9 + small.pages] = b
    tables = torch.tensor([[where[p] if p < small.pages else -1 for p in row] for row in small.tables.tolist()],
                          dtype=torch.int32, device="cuda")
    q, k, v = (_randn(2, h, dim, kind=kind, seed=h) for h in (32, heads, heads))
    pos, turns = small.lengths - 1, T.rope_turns(dim // 2 * 2)
    a = T.cache_append(k, v, big[0], big[1], tables, pos, q=q, turns=turns)
    b = T.cache_append(k, v, small.k, small.v, small.tables, pos, q=q, turns=turns)
    assert _same_bits(a, b)
    want = T.attention_decode(b, small.k, small.v, small.tables, small.lengths)
    assert _same_bits(T.attention_decode(a, big[0], big[1], tables, small.lengths), want)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[tables[0, :3].long()] = 1
    refs[tables[1, :2].long()] = 1
    parents = torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda")
    t, n, refs = T.cache_select(tables, small.lengths, refs, parents, big, page_size=page)
    assert int(t[1, 2]) == 0  # (the copy went to the front of the pool)
    t, refs, _ = T.cache_compact(t, n, refs, big, page_size=page)
    assert int(t.max()) == 5 and int((refs > 0).sum()) == 6
    got = T.attention_decode(a[parents.long()], big[0], big[1], t, n)
    at = parents.long()
    assert _same_bits(got, T.attention_decode(b[at], small.k, small.v, small.tables[at], small.lengths[at]))


# ---- refusals ----------------------------------------------------------------------------------------------------------

def test_refusals_of_tensors():
    x, i = torch.zeros(2, 1, 8, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    t, turns = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), T.rope_turns(8)
    c = torch.zeros(4, 2, 1, 8, device="cuda")
    for bad, error, words in (
            (lambda: T.rope(x.double(), None, i, turns), TypeError, "float32"),
            (lambda: T.rope(x, None, i.long(), turns), TypeError, "positions"),
            (lambda: T.rope(x, None, i, turns.int()), ValueError, "turns"),
            (lambda: T.rope(x, None, i, turns[::2]), ValueError, "turns"),
            (lambda: T.rope(x, None, i.cpu(), turns), ValueError, "positions is not on a GPU"),
            (lambda: T.rope(x, None, i, None, layout="half"), None, None),
            (lambda: T.rope(x, None, i[:1], turns), T.CmdError, "positions"),
            (lambda: T.rope(x.expand(2, 3, 8), None, i, turns, out=(x.expand(2, 3, 8), None)), T.CmdError, "overlaps itself"),
            (lambda: T.attention_decode(x[0], c, c, t, i), ValueError, "rank"),
            (lambda: T.attention_decode(x, c, c, t, i, scale=-1.0), T.CmdError, "scale"),
            (lambda: T.attention_decode(x.half(), c, c, t, i), T.CmdError, "element type"),
            (lambda: T.attention_decode(x, c, c, t, i, workspace=torch.empty(64, device="cuda")), T.CmdError, "workspace"),
            (lambda: T.attention_decode(x, c, c, t, i, status=torch.zeros(2, dtype=torch.int32, device="cuda")), ValueError, "status"),
            (lambda: T.cache_append(x, x, c, c.clone(), t, i, q=x), T.CmdError, "rotates"),
            (lambda: T.cache_append(x, x, c, c.clone(), t, i, q_out=5), TypeError, "q_out is no tensor"),
            (lambda: T.attention_decode(x, c, c, t, i, status=3), TypeError, "status is no tensor"),
            (lambda: T.attention_decode(x, c, c, t, i, window=1 << 40), ValueError, "window"),
            (lambda: T.attention_decode(x, c, c, t, i, softcap="1"), TypeError, "real number"),
            (lambda: T.cache_select(t, i, i, i, [c], page_size=2), ValueError, "pages in its first dim"),
            (lambda: T.cache_select(t, i, torch.zeros(4, dtype=torch.int32, device="cuda"), i, [c[..., ::2]], page_size=2), ValueError, "dense"),
            (lambda: T.cache_select(t, i, torch.zeros(4, dtype=torch.int32, device="cuda"), i, c, page_size=2), TypeError, "list or tuple"),
            (lambda: T.cache_compact(t, i, i, [], page_size=2, out=(t, i)), TypeError, "tuple of 3"),
            (lambda: T.cache_compact(t, i, i, [], page_size=2, out=(t, i, i.clone())), T.CmdError, "overlaps")):
        if error is None:
            bad()
            continue
        with pytest.raises(error, match=words):
            bad()
