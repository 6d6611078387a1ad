"""The serving path of a paged key-value cache, as cases that can be measured.

Five operators work on one cache: rotary positions (forward, and backward for training), the append of new tokens'
keys and values (rotated on the way), the attention of one new token per sequence, the selection of the sequences
that go on (fork, free, grow: a beam search's step, or the batch's turnover), and compaction. A cache is a pool of
pages, logically [pages, page slots, key-value heads, head dim]; a table row lists a sequence's pages in order.

Each case runs in a plain form (elementary torch operations, 32-bit arithmetic, one rounding at the end) or, with
`own`, through the framework's entry points. `exact` gives the computed outputs from the definition in 64 bits.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---- the cases ----------------------------------------------------------------------------------------------------

def listed():
    return [
        # queries and keys of a training batch, forward: half layout over the whole head, grouped key heads
        dict(name="rope_train", kind="rope", dtype="bf16", batch=4, seq=4096, hq=32, hk=8, dim=128, rot=128,
             layout="half", backward=False, start=0, base=10000.0, factor=1.0, scale=1.0),
        # the gradient of a partly rotated head in 32 bits at far positions: interleaved pairs, odd lengths, equal
        # head counts, frequencies slowed four times and the rotated part scaled for a long context
        dict(name="rope_grad_far", kind="rope", dtype="f32", batch=3, seq=1537, hq=12, hk=12, dim=80, rot=32,
             layout="interleaved", backward=True, start=262139, base=500000.0, factor=4.0, scale=1.1),
        # one decode step of a small batch: latency counts
        dict(name="append_decode", kind="append", dtype="bf16", rows=16, new=1, hq=32, hk=8, dim=128, rot=128,
             layout="half", page=16, order="slots", longest=2048, mix=1),
        # prompts of several ragged sequences entering the cache at once, half of each head rotated, head-major pages
        dict(name="append_prompts", kind="append", dtype="f16", rows=7, new=1171, hq=24, hk=8, dim=128, rot=64,
             layout="half", page=64, order="heads", longest=4096, mix=2),
        # a single conversation's next token: the smallest call
        dict(name="attend_one", kind="attend", dtype="bf16", rows=1, hq=32, hk=8, dim=128, page=16, order="slots",
             longest=700, shortest=700, softcap=0.0, window=0, mix=3),
        # a serving batch with ragged lengths, an empty row among them
        dict(name="attend_batch", kind="attend", dtype="bf16", rows=64, hq=64, hk=8, dim=128, page=16, order="slots",
             longest=8192, shortest=0, softcap=0.0, window=0, mix=4),
        # two very long documents: the work has to be split over the cache's length and joined
        dict(name="attend_long", kind="attend", dtype="f16", rows=2, hq=16, hk=2, dim=128, page=64, order="heads",
             longest=393217, shortest=262147, softcap=0.0, window=0, mix=5),
        # 32-bit numbers, one key head for each query head, an uncommon head dim and page size, capped scores
        # within a sliding window
        dict(name="attend_f32", kind="attend", dtype="f32", rows=24, hq=16, hk=16, dim=80, page=24, order="slots",
             longest=2999, shortest=1, softcap=30.0, window=1100, mix=6),
        # a beam search's step: four beams of each request go on from the beams that won
        dict(name="select_beams", kind="select", dtype="bf16", rows=64, pools=2, hk=8, dim=128, page=16,
             longest=1024, spare=256, die=0.4, grow=1, mix=7),
        # a large batch's turnover: forks of shared prompts, finished rows freed, new rows let in
        dict(name="select_turnover", kind="select", dtype="f16", rows=509, pools=4, hk=8, dim=128, page=64,
             longest=4096, spare=2001, die=0.5, grow=130, mix=8),
        # a small pool's compaction
        dict(name="compact_small", kind="compact", dtype="bf16", rows=12, pools=2, hk=8, dim=64, page=16,
             longest=500, total=601, move=77, mix=9),
        # a large pool's compaction, before half of it is given back
        dict(name="compact_large", kind="compact", dtype="bf16", rows=131, pools=4, hk=8, dim=128, page=32,
             longest=2048, total=7001, move=1703, mix=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "append", "attend", "attend", "select", "compact"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    dim = rng.choice([64, 72, 80, 96, 128, 128, 192, 256])
    hk = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 2, 4, 7, 8, 12])
    page = rng.choice([1, 8, 16, 24, 32, 64, 128])
    mix = rng.randrange(1 << 20)
    order = rng.choice(["slots", "heads"])
    layout = rng.choice(["half", "interleaved"])
    rot = rng.choice([dim, dim // 2])
    es = BYTES[dtype]
    if kind == "rope":
        hq, most = hk * group, 160e6
        seq = _log(rng, 1, 8192)
        batch = max(1, min(_log(rng, 1, 16), int(most / (seq * (hq + hk) * dim * es))))
        seq = max(1, min(seq, int(most / (batch * (hq + hk) * dim * es))))
        return dict(kind="rope", dtype=dtype, batch=batch, seq=seq, hq=hq, hk=hk, dim=dim, rot=rot, layout=layout,
                    backward=rng.random() < 0.5, start=_log(rng, 1, 1 << 20) - 1, base=rng.choice([1e4, 5e5]),
                    factor=rng.choice([1.0, 8.0]), scale=rng.choice([1.0, 1.25]))
    if kind == "append":
        rows = _log(rng, 1, 256)
        new = rng.choice([1, _log(rng, 2, 2048)])
        longest = new + _log(rng, 1, 2048)
        most = 5e8 / (hk * dim * es)  # tokens in the pool
        longest = max(new, min(longest, int(most / rows)))
        new = min(new, longest, max(1, int(1.5e8 / (rows * (group + 2) * hk * dim * es))))
        return dict(kind="append", dtype=dtype, rows=rows, new=new, hq=hk * group, hk=hk, dim=dim, rot=rot,
                    layout=layout, page=page, order=order, longest=max(longest, new), mix=mix)
    if kind == "attend":
        rows, longest = _log(rng, 1, 256), _log(rng, 1, 1 << 18)
        most = 6e8 / (2 * hk * dim * es * max(1, group / 8))
        longest = max(1, min(longest, int(most / rows)))
        return dict(kind="attend", dtype=dtype, rows=rows, hq=hk * group, hk=hk, dim=dim, page=page, order=order,
                    longest=longest, shortest=rng.choice([0, 1, longest]), softcap=rng.choice([0.0, 0.0, 25.0]),
                    window=rng.choice([0, 0, _log(rng, 1, 4096)]), mix=mix)
    page = max(page, 8)
    pools = rng.choice([1, 2, 4, 8])
    if kind == "select":
        rows, longest = _log(rng, 2, 512), _log(rng, 1, 4096)
        one = pools * page * hk * dim * es
        rows = max(2, min(rows, int(6e8 / one)))
        most = 1.2e9 / one  # pages in the pools
        longest = max(1, min(longest, int(max(1, most / rows / 2 - 2) * page)))
        grow = rng.choice([1, 1, 0, _log(rng, 2, 64)])
        return dict(kind="select", dtype=dtype, rows=rows, pools=pools, hk=hk, dim=dim, page=page, longest=longest,
                    spare=rows * (grow // page + 2) + _log(rng, 1, 64), die=rng.choice([0.0, 0.3, 0.8]), grow=grow, mix=mix)
    rows, longest = _log(rng, 1, 128), _log(rng, 1, 4096)
    most = int(1.2e9 / (pools * page * hk * dim * es))
    total = max(16, min(_log(rng, 16, 16384), most))
    rows = min(rows, total // 2)
    longest = min(longest, (total // 2 // rows) * page)
    return dict(kind="compact", dtype=dtype, rows=rows, pools=pools, hk=hk, dim=dim, page=page, longest=longest,
                total=total, move=rng.randrange(total // 4 + 1), mix=mix)


# ---- what a case fixes, whatever the seed ------------------------------------------------------------------------

def _lengths(c):
    """Sequence lengths over the case's range, evenly over their logarithm; the ends of the range come first."""
    rng = random.Random(c["mix"])
    lo, hi = c.get("shortest", 1), c["longest"]
    out = [hi, lo][: c["rows"]]
    while len(out) < c["rows"]:
        out.append(_log(rng, max(1, lo), max(1, hi)))
    return out


def _pages(length, page):
    return -(-length // page)


def _parents(c):
    """The rows that each row goes on from: survivors keep their place, dead rows' places go to forks of other
    rows, and a few to new sequences (-1)."""
    rng = random.Random(c["mix"] + 1)
    alive = [rng.random() >= c["die"] for _ in range(c["rows"])]
    alive[0] = True
    some = [i for i, a in enumerate(alive) if a]
    out = [i if a else (-1 if rng.random() < 0.2 else rng.choice(some)) for i, a in enumerate(alive)]
    if rng.random() < 0.5:
        rng.shuffle(out)
    return out


def _span(c, n):
    return min(n, c["window"]) if c["window"] else n


def work(case):
    c, es = case, BYTES[case["dtype"]]
    if c["kind"] == "rope":
        tokens = c["batch"] * c["seq"]
        n = tokens * (c["hq"] + c["hk"]) * c["dim"]
        return {"bytes": 2 * n * es + 4 * tokens + 4 * c["rot"], "flops": 3 * n * c["rot"] // c["dim"]}
    if c["kind"] == "append":
        tokens = c["rows"] * c["new"]
        moved = tokens * (c["hq"] + 2 * c["hk"]) * c["dim"]
        return {"bytes": 2 * moved * es + 12 * tokens + 4 * c["rot"],
                "flops": 3 * tokens * (c["hq"] + c["hk"]) * c["rot"]}
    lens = _lengths(c)
    if c["kind"] == "attend":
        keys = sum(_span(c, n) for n in lens)
        bytes_ = 2 * keys * c["hk"] * c["dim"] * es + 2 * c["rows"] * c["hq"] * c["dim"] * es
        return {"bytes": bytes_ + 4 * sum(_pages(_span(c, n), c["page"]) for n in lens) + 4 * c["rows"] * (c["hq"] + 1),
                "flops": 4 * keys * c["hq"] * c["dim"]}
    block = c["pools"] * c["page"] * c["hk"] * c["dim"] * es
    if c["kind"] == "select":
        wide = _width(c)
        parents, seen, copies = _parents(c), set(), 0
        for p in parents:
            if p >= 0:
                copies += p in seen and lens[p] % c["page"] != 0
                seen.add(p)
        used = sum(_pages(lens[p], c["page"]) for p in parents if p >= 0)
        return {"bytes": 2 * copies * block + 4 * (used + c["rows"] * wide + 5 * c["rows"] + 2 * _total(c)), "flops": 0}
    wide = _pages(c["longest"], c["page"])
    used = sum(_pages(n, c["page"]) for n in lens)
    return {"bytes": 2 * c["move"] * block + 4 * (used + c["rows"] * wide + c["rows"] + 3 * c["total"]), "flops": 0}


def _width(c):
    return _pages(c["longest"] + c["grow"], c["page"])


def _total(c):
    """Pages of a selection's pool: those in use, and spare ones."""
    return sum(_pages(n, c["page"]) for n in _lengths(c)) + c["spare"]


# ---- inputs -------------------------------------------------------------------------------------------------------

def _turns(c, device):
    """Turns per position of each rotated pair, as fractions of 2^64: base^(-2 i / rot) / (2 pi factor)."""
    i = torch.arange(c["rot"] // 2, dtype=torch.float64)
    f = torch.exp(-2.0 * i / c["rot"] * math.log(c.get("base", 10000.0))) / (2.0 * math.pi * c.get("factor", 1.0))
    return (f * 2.0 ** 64).to(torch.int64).to(device)


def _tables(lens, page, wide, numbers):
    """Table rows: each sequence takes the next of `numbers`, and -1 where it has no page."""
    t, at = np.full((len(lens), wide), -1, dtype=np.int32), 0
    for i, n in enumerate(lens):
        k = _pages(n, page)
        t[i, :k] = numbers[at:at + k]
        at += k
    return t, at


def _pool(gen, c, pages, dtype):
    """A pool of pages, logically [pages, slots, heads, dim], with the slots or the heads outermost in a page."""
    shape = (pages, c["page"], c["hk"], c["dim"])
    if c.get("order", "slots") == "heads":
        return torch.randn(shape[0], shape[2], shape[1], shape[3], generator=gen, device="cuda", dtype=dtype).transpose(1, 2)
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pick = np.random.RandomState(seed % (1 << 32))
    dtype = TYPES[c["dtype"]]
    s = {"case": c}

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)

    if c["kind"] == "rope":
        s["q"] = rand(c["batch"], c["seq"], c["hq"], c["dim"])
        s["k"] = rand(c["batch"], c["seq"], c["hk"], c["dim"])
        s["positions"] = (torch.arange(c["seq"], device="cuda", dtype=torch.int32) + c["start"]).expand(c["batch"], c["seq"])
        s["turns"] = _turns(c, "cuda")
        return s
    if c["kind"] == "append":
        rng = random.Random(c["mix"])
        lens = [rng.randint(c["new"], c["longest"]) for _ in range(c["rows"])]
        wide = _pages(c["longest"], c["page"])
        total = sum(_pages(n, c["page"]) for n in lens)
        t, _ = _tables(lens, c["page"], wide, pick.permutation(total))
        tokens = c["rows"] * c["new"]
        s["tables"] = _i32(t)
        s["positions"] = _i32([n - c["new"] + j for n in lens for j in range(c["new"])])
        s["rows"] = _i32([i for i in range(c["rows"]) for _ in range(c["new"])])
        s["q"], s["k"], s["v"] = rand(tokens, c["hq"], c["dim"]), rand(tokens, c["hk"], c["dim"]), rand(tokens, c["hk"], c["dim"])
        s["turns"] = _turns(c, "cuda")
        s["k_cache"], s["v_cache"] = (_pool(gen, c, total, dtype) for _ in range(2))
        return s
    lens = _lengths(c)
    if c["kind"] == "attend":
        wide = max(1, _pages(c["longest"], c["page"]))
        total = sum(_pages(n, c["page"]) for n in lens) + 1
        t, _ = _tables(lens, c["page"], wide, pick.permutation(total))
        s["tables"], s["lengths"] = _i32(t), _i32(lens)
        # queries twice as wide as the keys, so that the softmax has some weights well above the others
        s["q"] = 2 * rand(c["rows"], c["hq"], c["dim"])
        s["k_cache"], s["v_cache"] = (_pool(gen, c, total, dtype) for _ in range(2))
        return s
    refs = None
    if c["kind"] == "select":
        total = _total(c)
        t, _ = _tables(lens, c["page"], _width(c), pick.permutation(total))
        s["parents"], s["grow"] = _i32(_parents(c)), _i32([c["grow"]] * c["rows"])
    else:
        total = c["total"]
        # pages that no row lists are held outside the tables (a kept prefix, say): at most half of the pool is
        # free, and exactly `move` of the pages in use lie past the number of pages in use
        live, move = max(sum(_pages(n, c["page"]) for n in lens), total // 2), c["move"]
        assert move <= min(live, total - live)
        low, high = pick.permutation(live), live + pick.permutation(total - live)
        numbers = pick.permutation(np.concatenate([low[: live - move], high[:move]]))
        t, _ = _tables(lens, c["page"], _pages(c["longest"], c["page"]), numbers)
        refs = np.zeros(total, dtype=np.int32)
        refs[numbers] = 1
    if refs is None:
        refs = np.zeros(total, dtype=np.int32)
        refs[t[t >= 0]] = 1
    s["tables"], s["lengths"], s["refs"] = _i32(t), _i32(lens), _i32(refs)
    s["pools"] = [_pool(gen, c, total, dtype) for _ in range(c["pools"])]
    return s


# ---- the plain forms ----------------------------------------------------------------------------------------------

def _rotate(x, positions, turns, c, backward=False):
    phase = positions.to(torch.int64)[..., None] * turns  # modulo 2^64: a whole number of turns drops out
    angle = phase.to(torch.float32) * (math.pi / 2.0 ** 63)
    scale = c.get("scale", 1.0)
    cos, sin = (torch.cos(angle) * scale)[..., None, :], (torch.sin(angle) * (-scale if backward else scale))[..., None, :]
    w, rot = x.to(torch.float32), c["rot"]
    if c["layout"] == "half":
        a, b = w[..., : rot // 2], w[..., rot // 2: rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = w[..., 0:rot:2], w[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([y, w[..., rot:]], dim=-1).to(x.dtype)


def _attend(s):
    c, q = s["case"], s["q"].to(torch.float32)
    rows, dim, page = c["rows"], c["dim"], c["page"]
    at = s["tables"].clamp(min=0).to(torch.int64)
    k = s["k_cache"][at].flatten(1, 2).to(torch.float32)  # [rows, tokens, heads, dim]
    v = s["v_cache"][at].flatten(1, 2).to(torch.float32)
    token = torch.arange(k.shape[1], device=q.device)
    n = s["lengths"][:, None]
    seen = token < n
    if c["window"]:
        seen = seen & (token >= n - c["window"])
    q = q.reshape(rows, c["hk"], -1, dim)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)) * (dim ** -0.5)
    if c["softcap"]:
        scores = c["softcap"] * torch.tanh(scores / c["softcap"])
    scores = torch.where(seen[:, None, None], scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, torch.where(seen[:, :, None, None], v, 0.0).transpose(1, 2))
    o = torch.where(total == 0, 0.0, o / total)
    lse = (top + torch.log(total)).reshape(rows, -1)
    return {"out": o.reshape(rows, -1, dim).to(s["q"].dtype), "lse": lse}


def _append(s):
    c = s["case"]
    q, k = _rotate(s["q"], s["positions"], s["turns"], c), _rotate(s["k"], s["positions"], s["turns"], c)
    position = s["positions"].to(torch.int64)
    at = s["tables"].to(torch.int64)[s["rows"].to(torch.int64), position // c["page"]]
    s["k_cache"][at, position % c["page"]] = k
    s["v_cache"][at, position % c["page"]] = s["v"]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _select(s):
    page, tables, lengths, refs, parents = s["case"]["page"], s["tables"].long(), s["lengths"].long(), s["refs"], s["parents"].long()
    wide, rows = tables.shape[1], parents.shape[0]
    has, parent = parents >= 0, parents.clamp(min=0)
    j = torch.arange(wide, device="cuda")
    length = torch.where(has, lengths[parent], 0)
    old, total = (length + page - 1) // page, (length + s["grow"] + page - 1) // page
    fits = total <= wide
    earlier = torch.tril((parents[:, None] == parents[None, :]) & fits, diagonal=-1).any(1)
    split = has & earlier & (length % page != 0)  # a later child of a page in progress gets a copy of it
    keep = old - split.long()
    need = torch.where(fits, total - keep, 0)
    base = torch.cumsum(need, 0) - need
    # pages that nothing holds once the old rows are gone and the new ones hold what they keep
    was, stays = j < ((lengths + page - 1) // page)[:, None], (j < keep[:, None]) & fits[:, None]
    kept = tables[parent]
    count = refs.long().scatter_add(0, tables.clamp(min=0).flatten(), -was.long().flatten())
    count = count.scatter_add(0, kept.clamp(min=0).flatten(), stays.long().flatten())
    free = torch.sort((count != 0).to(torch.int8), stable=True).indices
    fits = fits & ((need == 0) | (base + need <= (count == 0).sum()))
    takes = (j >= keep[:, None]) & (j < total[:, None]) & fits[:, None]
    fresh = free[(base[:, None] + j - keep[:, None]).clamp(0, free.shape[0] - 1)]
    out = torch.where(takes, fresh, torch.where(stays & fits[:, None], kept, -1))
    count = count.scatter_add(0, kept.clamp(min=0).flatten(), -(stays & ~fits[:, None]).long().flatten())
    count = count.scatter_add(0, fresh.flatten(), takes.long().flatten())
    copy = (split & fits).nonzero().flatten()
    to, of = out[copy, keep[copy]], kept[copy, keep[copy]]
    for pool in s["pools"]:
        pool[to] = pool[of]
    return {"tables": out.int(), "lengths": torch.where(fits, length + s["grow"], 0).int(), "refs": count.int(),
            "pools": [_bits(p) for p in s["pools"]]}


def _compact(s):
    page, refs = s["case"]["page"], s["refs"]
    index = torch.arange(refs.shape[0], device="cuda")
    live = refs > 0
    n = live.sum()
    of, to = (live & (index >= n)).nonzero().flatten(), (~live & (index < n)).nonzero().flatten()
    where = torch.where(live, index, -1)
    where[of] = to
    held = torch.where(live & (index < n), refs, 0)
    held[to] = refs[of]
    used = torch.arange(s["tables"].shape[1], device="cuda") < ((s["lengths"] + page - 1) // page)[:, None]
    tables = torch.where(used, where[s["tables"].clamp(min=0).long()], -1)
    for pool in s["pools"]:
        pool[to] = pool[of]
    return {"tables": tables.int(), "refs": held, "page_map": where.int(), "pools": [_bits(p) for p in s["pools"]]}


def _bits(pool):
    """A pool's values as whole numbers: pages are moved, not computed."""
    return pool.view(torch.int32 if pool.dtype == torch.float32 else torch.int16)


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["kind"] == "rope":
        return [_rotate(s[x], s["positions"], s["turns"], c, c["backward"]) for x in ("q", "k")]
    return {"append": _append, "attend": _attend, "select": _select, "compact": _compact}[c["kind"]](s)


# ---- the framework's operators ------------------------------------------------------------------------------------

def _run_own(s, c):
    import tensor_command_execution_gb300 as T

    if c["kind"] == "rope":
        f = T.rope_backward if c["backward"] else T.rope
        return list(f(s["q"], s["k"], s["positions"], s["turns"], layout=c["layout"], scale=c["scale"]))
    if c["kind"] == "append":
        q = T.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["tables"], s["positions"], rows=s["rows"],
                           q=s["q"], turns=s["turns"], layout=c["layout"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["kind"] == "attend":
        out, lse = T.attention_decode(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lengths"],
                                      softcap=c["softcap"], window=c["window"], return_lse=True)
        return {"out": out, "lse": lse}
    if c["kind"] == "select":
        tables, lengths, refs = T.cache_select(s["tables"], s["lengths"], s["refs"], s["parents"], s["pools"],
                                               page_size=c["page"], grow=s["grow"])
        return {"tables": tables, "lengths": lengths, "refs": refs, "pools": [_bits(p) for p in s["pools"]]}
    tables, refs, page_map = T.cache_compact(s["tables"], s["lengths"], s["refs"], s["pools"], page_size=c["page"])
    return {"tables": tables, "refs": refs, "page_map": page_map, "pools": [_bits(p) for p in s["pools"]]}


# ---- the definitions in 64 bits -----------------------------------------------------------------------------------

def _rotated(x, positions, turns, rot, layout, scale):
    """x as pairs (u, v), each turned as the complex number u + iv by its position's angle, in binary64."""
    part = (positions.long().unsqueeze(-1) * turns).double() * 2.0 ** -64
    turn = torch.polar(torch.full_like(part, abs(scale)), (2 * math.pi if scale > 0 else -2 * math.pi) * part).unsqueeze(-2)
    y = x.double().clone()
    if layout == "half":
        z = torch.complex(y[..., : rot // 2], y[..., rot // 2: rot]) * turn
        y[..., : rot // 2], y[..., rot // 2: rot] = z.real, z.imag
    else:
        z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * turn
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    return y


def exact(case, seed):
    c = case
    if c["kind"] in ("select", "compact"):
        return None  # whole numbers only
    s = prepare(c, seed)
    if c["kind"] == "rope":
        scale = -c["scale"] if c["backward"] else c["scale"]
        return [_rotated(s[x], s["positions"], s["turns"], c["rot"], c["layout"], scale) for x in ("q", "k")]
    if c["kind"] == "append":
        q, k = (_rotated(s[x], s["positions"], s["turns"], c["rot"], c["layout"], 1.0) for x in ("q", "k"))
        page, slot = s["positions"] // c["page"], (s["positions"] % c["page"]).long()
        page = s["tables"][s["rows"].long(), page.long()].long()
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        k_cache[page, slot], v_cache[page, slot] = k, s["v"].double()
        return {"q": q, "k_cache": k_cache, "v_cache": v_cache}
    outs, sums = [], []
    for i, n in enumerate(_lengths(c)):
        lo = n - _span(c, n)
        if n == 0:
            outs.append(torch.zeros(c["hq"], c["dim"], dtype=torch.float64, device="cuda"))
            sums.append(torch.full((c["hq"],), -math.inf, dtype=torch.float64, device="cuda"))
            continue
        page = s["tables"][i, : _pages(n, c["page"])].long()
        k, v = (s[x][page].reshape(-1, c["hk"], c["dim"])[lo:n].double() for x in ("k_cache", "v_cache"))
        q = s["q"][i].double().reshape(c["hk"], -1, c["dim"])
        z = torch.einsum("hgd,thd->hgt", q, k) / math.sqrt(c["dim"])
        if c["softcap"]:
            z = c["softcap"] * torch.tanh(z / c["softcap"])
        outs.append(torch.einsum("hgt,thd->hgd", torch.softmax(z, -1), v).reshape(c["hq"], c["dim"]))
        sums.append(torch.logsumexp(z, -1).reshape(-1))
    return {"out": torch.stack(outs), "lse": torch.stack(sums)}
