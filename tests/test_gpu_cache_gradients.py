"""Rotary positions inside autograd, through the entry points themselves."""
from __future__ import annotations

import pytest
import torch

import cacheutil as U
import tensor_command_execution_gb300 as T

pytestmark = pytest.mark.gpu


def _randn(*shape, kind="f32", seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(U.TYPES[kind])


POS = torch.tensor([[3, 70000, 1 << 30, 5]], dtype=torch.int32)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("backward", [False, True])
def test_gradients_are_recorded(kind, layout, backward):
    """Results that depend on an input whose gradient is asked for carry it, also from weights that are broadcast."""
    f = T.rope_backward if backward else T.rope
    q, k = _randn(1, 4, 3, 24, kind=kind).requires_grad_(), _randn(1, 4, 2, 24, kind=kind, seed=1).requires_grad_()
    w = _randn(1, 4, 3, 24, kind=kind, seed=2)
    turns, pos = T.rope_turns(16), POS.cuda()
    a, b = f(q, k, pos, turns, layout=layout, scale=0.75)
    assert a.requires_grad and b.requires_grad
    ((a * w).sum() + b.sum()).backward()
    for x, up in ((q, w), (k, torch.ones_like(k))):
        want = U.rotated(up, POS, turns, layout, 0.75, backward=not backward)
        bound = U.rope_bound(up, want, 8, layout, 0.75, kind)
        assert bool(((x.grad.cpu().double() - want).abs() <= bound).all())
    # one of the two, and none
    a, b = f(q.detach(), k, pos, turns, layout=layout)
    assert b.requires_grad
    (g,) = torch.autograd.grad(b.sum(), k)
    assert g.shape == k.shape and bool(torch.isfinite(g).all())
    a, b = f(q, None, pos, turns, layout=layout)
    assert a.requires_grad and b is None
    with torch.no_grad():
        assert not f(q, k, pos, turns, layout=layout)[0].requires_grad
    assert not f(q.detach(), k.detach(), pos, turns, layout=layout)[0].requires_grad


def test_gradients_on_a_stream_and_of_gradients():
    x, pos, turns = _randn(1, 4, 2, 16).requires_grad_(), POS.cuda(), T.rope_turns(16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = T.rope(x, None, pos, turns, stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    w = _randn(1, 4, 2, 16, seed=1).requires_grad_()
    (g,) = torch.autograd.grad((y * w).sum(), x, create_graph=True)
    want = U.rotated(w, POS, turns, "half", 1.0, backward=True)
    assert bool(((g.detach().cpu().double() - want).abs() <= U.rope_bound(w, want, 8, "half", 1.0, "f32")).all())
    u = _randn(1, 4, 2, 16, seed=2)
    (h,) = torch.autograd.grad((g * u).sum(), w)  # g is linear in w: the gradient is the rotation of u
    want = U.rotated(u, POS, turns, "half", 1.0)
    assert bool(((h.cpu().double() - want).abs() <= U.rope_bound(u, want, 8, "half", 1.0, "f32")).all())


def test_outputs_given_record_no_gradient():
    x, pos, turns = _randn(4, 2, 16).requires_grad_(), POS[0].cuda(), T.rope_turns(16)
    room = torch.empty(4, 2, 16, device="cuda")
    for q, out in ((x, room), (x.detach(), room.clone().requires_grad_())):
        with pytest.raises(ValueError, match="gradient"):
            T.rope(q, None, pos, turns, out=(out, None))
    with torch.no_grad():
        assert T.rope(x, None, pos, turns, out=(room, None))[0] is room


def test_autograd_hears_of_what_is_written():
    """A tensor that a gradient still needs, overwritten by an operator: an error, not a wrong gradient."""
    c = U.Cache("f32", [9, 3], 2, 16, 4, spare=3, columns=4)
    pos, turns = c.lengths - 1, T.rope_turns(16)
    q, k = _randn(2, 2, 16), _randn(2, 2, 16, seed=1)
    refs = torch.zeros(c.pages, dtype=torch.int32, device="cuda")
    for r, n in enumerate(c.need):
        refs[c.tables[r, :n].long()] = 1

    def needs(x):  # a graph that has x in it
        w = torch.ones((), device="cuda", requires_grad=True)
        return (w * x).sum()
    for x, write in (
            (q, lambda: T.rope(q, None, pos, turns, out=(q, None))),
            (k, lambda: T.rope_backward(None, k, pos, turns, out=(None, k))),
            (c.k, lambda: T.cache_append(k, k, c.k, c.v, c.tables, pos)),
            (c.v, lambda: T.cache_append(k, k, c.k, c.v, c.tables, pos)),
            (q, lambda: T.attention_decode(k, c.k, c.v, c.tables, c.lengths, out=q)),
            (c.v, lambda: T.cache_select(c.tables, c.lengths, refs, torch.zeros(2, dtype=torch.int32, device="cuda"), [c.k, c.v], page_size=4)),
            (c.k, lambda: T.cache_compact(c.tables, c.lengths, refs, [c.k, c.v], page_size=4))):
        y = needs(x)
        write()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    with torch.inference_mode():  # (tensors without a version)
        z = torch.zeros(2, 2, 16, device="cuda")
        assert T.rope(z, None, pos, turns, out=(z, None))[0] is z


def test_views_that_hold_negated_numbers_are_refused():
    x = torch._neg_view(_randn(4, 2, 16))
    with pytest.raises(ValueError, match="negat"):
        T.rope(x, None, POS[0].cuda(), T.rope_turns(16))
