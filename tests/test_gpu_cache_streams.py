"""The cache operators on streams other than their tensors' own."""
from __future__ import annotations

import pytest
import torch

import cacheutil as U
import tensor_command_execution_gb300 as T

pytestmark = pytest.mark.gpu


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _calls():
    """Each operator with its tensors, as (name, call of a stream and the tensors, tensors)."""
    c = U.Cache("f32", [40, 20], 2, 64, 16, spare=4, columns=4)
    refs = torch.zeros(c.pages, dtype=torch.int32, device="cuda")
    for r, n in enumerate(c.need):
        refs[c.tables[r, :n].long()] = 1
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(2, h, 64, generator=gen, device="cuda") for h in (4, 2, 2))
    x, pos, turns = torch.randn(300, 4, 64, generator=gen, device="cuda"), torch.arange(300, dtype=torch.int32, device="cuda"), T.rope_turns(64)

    def append(s, k, v, kc, vc, t, n, q, turns, rows):
        return T.cache_append(k, v, kc, vc, t, n, q=q, turns=turns, rows=rows, stream=s), kc, vc

    def select(s, t, n, r, parents, grow, kc, vc):
        return *T.cache_select(t, n, r, parents, [kc, vc], page_size=16, grow=grow, stream=s), kc, vc

    def compact(s, t, n, r, kc, vc):
        return *T.cache_compact(t, n, r, [kc, vc], page_size=16, stream=s), kc, vc
    return [
        ("rope", lambda s, x, y, pos, turns: T.rope(x, y, pos, turns, stream=s), (x, x[:, :2].clone(), pos, turns)),
        ("rope_backward", lambda s, x, pos, turns: T.rope_backward(x, None, pos, turns, stream=s)[:1], (x, pos, turns)),
        ("cache_append", append, (k, v, c.k, c.v, c.tables, c.lengths - 1, q, turns, _i32(0, 1))),
        ("attention_decode", lambda s, q, kc, vc, t, n: (T.attention_decode(q, kc, vc, t, n, stream=s),), (q, c.k, c.v, c.tables, c.lengths)),
        ("cache_select", select, (c.tables, c.lengths, refs, _i32(1, 0, 1), _i32(1, 2, 3), c.k, c.v)),
        ("cache_compact", compact, (c.tables, c.lengths, refs, c.k, c.v)),
    ]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("which", range(6))
def test_inputs_freed_after_the_call_stay_until_the_stream_is_done(which, raw):
    """A call on a busy stream, its inputs dropped right after and their memory asked for again on the current stream:
    the work still reads the inputs. (What takes their place are zeros: valid pages, rows and lengths.)"""
    name, call, tensors = _calls()[which]
    want = [x.clone() for x in call(None, *[x.clone() for x in tensors])]
    outputs = {"cache_append": 2, "cache_select": 2, "cache_compact": 2}.get(name, 0)  # (results that are inputs too)
    side = torch.cuda.Stream()
    mine = [x.clone() for x in tensors]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # (about 0.1 s)
    got = call(side.cuda_stream if raw else side, *mine)
    kept = mine[2:4] if name == "cache_append" else mine[-2:] if outputs else []
    like = [(x.shape, x.dtype) for x in mine if not any(x is y for y in kept)]
    mine = x = None
    over = [torch.zeros(s, dtype=d, device="cuda") for s, d in like for _ in range(4)]
    torch.cuda.synchronize()
    assert over and all(torch.equal(a, b) for a, b in zip(got, want)), name
