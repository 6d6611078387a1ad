"""Drafted tokens and budgets on a paged key-value cache, as cases that can be measured.

A program that drafts guesses several tokens ahead, as a tree, stores their keys and values behind a sequence's tokens,
attends to all of them in one pass (`tree`), walks the tree along the model's own choices (`path`), and keeps the
accepted branch's slots (`accept`). One that has a budget adds up the attention that each cached token gets (`weigh`:
the same attention, of one token of each sequence or of the last tokens of a prompt, with its weights added to a running sum) and
now and then drops the tokens that got least (`evict`). All on the cache of the other operators: pools of pages,
logically [pages, page slots, key-value heads, head dim], with a table row of pages for each sequence.

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
        # a single conversation with a small tree of guesses: the smallest call
        dict(name="tree_one", kind="tree", dtype="bf16", rows=1, drafts=8, tree=True, hq=32, hk=8, dim=128, page=16,
             order="slots", longest=700, shortest=700, softcap=0.0, window=0, mix=1),
        # a serving batch, ragged lengths from none to 8192, rows with fewer guesses than others and an idle one
        dict(name="tree_batch", kind="tree", dtype="bf16", rows=16, drafts=24, tree=True, hq=32, hk=8, dim=128, page=16,
             order="slots", longest=8192, shortest=0, softcap=0.0, window=0, mix=2),
        # wide trees over long documents: 512 queries to each key head, bound by arithmetic
        dict(name="tree_wide", kind="tree", dtype="f16", rows=4, drafts=64, tree=True, hq=64, hk=8, dim=128, page=64,
             order="heads", longest=16384, shortest=9001, softcap=0.0, window=0, mix=3),
        # 32-bit numbers, one key head for each query head, an uncommon head dim, page size and number of guesses (a
        # chain), capped scores within a sliding window
        dict(name="tree_f32", kind="tree", dtype="f32", rows=12, drafts=13, tree=False, hq=16, hk=16, dim=80, page=24,
             order="slots", longest=2999, shortest=1, softcap=30.0, window=1100, mix=4),
        # a decode step of a batch whose cache has a budget: each token's weights are added up
        dict(name="weigh_decode", kind="weigh", dtype="bf16", rows=32, drafts=1, tree=False, hq=32, hk=8, dim=128, page=32,
             order="slots", longest=8192, shortest=500, softcap=0.0, window=0, mix=5),
        # the last 32 tokens of two long prompts, whose attention says what of the prompts is worth keeping
        dict(name="weigh_prompts", kind="weigh", dtype="bf16", rows=2, drafts=32, tree=False, hq=32, hk=8, dim=64, page=16,
             order="slots", longest=65536, shortest=30011, softcap=0.0, window=0, mix=6),
        # which guesses of a batch hold: a few small trees, and many of the largest size
        dict(name="path_batch", kind="path", rows=16, drafts=24, mix=7),
        dict(name="path_many", kind="path", rows=512, drafts=256, mix=8),
        # the accepted guesses' keys and values of one layer, and of a model's 16
        dict(name="accept_layer", kind="accept", dtype="bf16", rows=16, drafts=24, pools=2, hk=8, dim=128, page=16,
             order="slots", longest=2048, mix=9),
        dict(name="accept_model", kind="accept", dtype="bf16", rows=61, drafts=64, pools=32, hk=8, dim=128, page=16,
             order="slots", longest=512, mix=10),
        # a batch of generations that have grown past their budget by a page or two, one layer
        dict(name="evict_layer", kind="evict", dtype="bf16", rows=32, layers=1, hk=8, dim=128, page=32, order="slots",
             longest=2176, shortest=1500, budget=2048, recent=128, mix=11),
        # long prompts cut to an eighth before the generation begins, eight layers at once
        dict(name="evict_prompts", kind="evict", dtype="f16", rows=4, layers=8, hk=8, dim=128, page=64, order="heads",
             longest=32768, shortest=20011, budget=4096, recent=512, mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["tree", "tree", "tree", "weigh", "weigh", "path", "accept", "evict", "evict"])
    dtype = rng.choice(["bf16", "f16", "bf16", "f16", "f32"])
    dim = rng.choice([64, 72, 80, 96, 128, 128, 192, 256])
    hk = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 2, 4, 7, 8, 12])
    page = rng.choice([1, 8, 16, 24, 32, 64, 128])
    mix = rng.randrange(1 << 20)
    order = rng.choice(["slots", "heads"])
    drafts = rng.choice([1, 2, _log(rng, 3, 32), _log(rng, 16, 128), _log(rng, 16, 256)])
    es = BYTES[dtype]
    if kind in ("tree", "weigh"):
        if kind == "weigh":
            drafts = rng.choice([1, 1, min(drafts, 64)])
        rows, longest = _log(rng, 1, 128), _log(rng, 1, 1 << 17)
        # tokens in all, by bytes and by products (f32 rows take several times as long)
        most = min(4e8 / (2 * hk * dim * es), (1e11 if es == 2 else 1e10) / (4 * hk * group * dim * drafts))
        rows = max(1, min(rows, int(most / drafts)))
        longest = max(1, min(longest, int(most / rows) - drafts))
        return dict(kind=kind, dtype=dtype, rows=rows, drafts=drafts, tree=rng.random() < 0.7, hq=hk * group, hk=hk, dim=dim,
                    page=page, order=order, longest=longest, shortest=rng.choice([0, 1, longest]),
                    softcap=rng.choice([0.0, 0.0, 25.0]), window=rng.choice([0, 0, _log(rng, 1, 4096)]), mix=mix)
    if kind == "path":
        return dict(kind="path", rows=_log(rng, 1, 512), drafts=drafts, mix=mix)
    page = max(page, 8)
    if kind == "accept":
        rows, pools, longest = _log(rng, 1, 64), rng.choice([2, 2, 4, 16, 32]), _log(rng, 1, 2048)
        most = 2e9 / (pools * hk * dim * es)  # tokens in the pools
        rows = max(1, min(rows, int(most / (drafts + page))))
        longest = max(1, min(longest, int(most / rows) - drafts - page))
        return dict(kind="accept", dtype=dtype, rows=rows, drafts=drafts, pools=pools, hk=hk, dim=dim, page=page,
                    order=order, longest=longest, mix=mix)
    rows, layers, longest = _log(rng, 1, 64), rng.choice([1, 1, 2, 4, 8]), _log(rng, 16, 1 << 16)
    most = 1e9 / (2 * layers * hk * dim * es)  # tokens in the pools
    rows = max(1, min(rows, int(most / (4 * page))))
    longest = max(2, min(longest, int(most / rows) - page))
    budget = rng.randint(1, longest)
    return dict(kind="evict", dtype=dtype, rows=rows, layers=layers, hk=hk, dim=dim, page=page, order=order, longest=longest,
                shortest=rng.choice([0, 1, max(1, longest // 2)]), budget=budget, recent=rng.choice([0, 1, budget // 8, budget]), mix=mix)


# ---- what a case fixes, whatever the seed ------------------------------------------------------------------------

def _lengths(c):
    """Sequence lengths over the case's range, evenly over their logarithm; the ends of the range come first. Of cases
    with drafts these are the tokens before them; -1 marks a row that idles."""
    rng = random.Random(c["mix"])
    lo, hi = c.get("shortest", 1), c["longest"]
    out = [hi, lo][: c["rows"]]
    while len(out) < c["rows"]:
        out.append(_log(rng, max(1, lo), max(1, hi)))
    if c["kind"] == "tree" and c["rows"] > 4:
        out[3] = -1
    return out


def _totals(c):
    """Tokens of each row in the cache, drafts included."""
    return [n + c["drafts"] if n >= 0 else 0 for n in _lengths(c)]


def _parents(c):
    """The trees, i32 [rows, drafts]: each guess goes on from one of the few before it (or from the one before: a
    chain); rows have fewer guesses than others now and then, the rest is padding (-2)."""
    rng, d = random.Random(c["mix"] + 1), c["drafts"]
    out = np.full((c["rows"], d), -2, dtype=np.int32)
    for r in range(c["rows"]):
        used = d if r == 0 or rng.random() < 0.7 else rng.randint(1, d)
        for i in range(used):
            out[r, i] = i - 1 if i < 2 else rng.randint(max(0, i - rng.choice([1, 2, 6, 16])), i - 1)
    return out


def _seen(parents):
    """Which drafts each sees, [rows, drafts, drafts], and their depths, [rows, drafts] (-1: padding)."""
    rows, d = parents.shape
    seen, depth = np.zeros((rows, d, d), dtype=bool), np.full((rows, d), -1, dtype=np.int64)
    for i in range(d):
        p = parents[:, i]
        for r in np.nonzero(p == -1)[0]:
            seen[r, i, i], depth[r, i] = True, 0
        for r in np.nonzero((p >= 0) & (p < i))[0]:
            if depth[r, p[r]] >= 0:
                seen[r, i] = seen[r, p[r]]
                seen[r, i, i], depth[r, i] = True, depth[r, p[r]] + 1
    return seen, depth


def _tree(c):
    if c["tree"]:
        return _parents(c)
    return np.tile(np.arange(-1, c["drafts"] - 1, dtype=np.int32), (c["rows"], 1))


def _pages(length, page):
    return -(-length // page)


def work(case):
    c = case
    if c["kind"] == "path":
        return {"bytes": 4 * c["rows"] * (4 * c["drafts"] + 2), "flops": 0}
    es, one = BYTES[c["dtype"]], c["hk"] * c["dim"] * BYTES[c["dtype"]]
    if c["kind"] in ("tree", "weigh"):
        seen, depth = _seen(_tree(c))
        w, keys, pairs = c["window"], 0, 0
        for r, n in enumerate(_lengths(c)):
            if n < 0:
                continue
            at = depth[r][depth[r] >= 0]
            span = np.minimum(n, np.maximum(0, w - 1 - at)) if w else np.full(at.shape, n)
            near = seen[r] & ((depth[r][:, None] - depth[r][None, :] < w) if w else True)
            keys += int(span.max(initial=0)) + int(near.any(0).sum())
            pairs += int(span.sum()) + int(near.sum())
        q = c["rows"] * c["drafts"] * c["hq"]
        bytes_ = 2 * keys * one + 2 * q * c["dim"] * es + 4 * q + 4 * (keys // c["page"] + c["rows"] * (c["drafts"] + 1))
        return {"bytes": bytes_ + (8 * keys * c["hk"] if c["kind"] == "weigh" else 0), "flops": 4 * pairs * c["hq"] * c["dim"]}
    pages = sum(_pages(n, c["page"]) for n in (_totals(c) if c["kind"] == "accept" else _lengths(c)))
    if c["kind"] == "accept":
        path, counts = _paths(c)
        moved = sum(int((p[:n] != np.arange(n)).sum()) for p, n in zip(path, counts))
        return {"bytes": 2 * moved * c["pools"] * one + 4 * (3 * pages + 3 * c["rows"] + int(counts.sum())), "flops": 0}
    over = [n for n in _lengths(c) if n > c["budget"]]
    kept = len(over) * c["budget"]
    return {"bytes": c["layers"] * (2 * kept * (2 * one + 4 * c["hk"]) + 4 * c["hk"] * sum(over)) + 4 * (3 * pages + 2 * c["rows"]),
            "flops": 0}


def _paths(c):
    """Accepted branches, [rows, drafts] and their lengths: short ones mostly, sometimes none."""
    rng, d = random.Random(c["mix"] + 2), c["drafts"]
    path, counts = np.full((c["rows"], d), -1, dtype=np.int32), np.zeros(c["rows"], dtype=np.int32)
    for r in range(c["rows"]):
        n = min(d, int(rng.expovariate(0.25)) + (rng.random() < 0.9))
        path[r, :n] = sorted(rng.sample(range(d), n))
        counts[r] = n
    return path, counts


# ---- inputs -------------------------------------------------------------------------------------------------------

def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def _tables(totals, page, pick, spare=2):
    """A shuffled page table with room for the longest row, and the number of pages."""
    wide = max(1, _pages(max(totals), page))
    pages = sum(_pages(n, page) for n in totals) + spare
    t, numbers, at = np.full((len(totals), wide), -1, dtype=np.int32), pick.permutation(pages), 0
    for r, n in enumerate(totals):
        k = _pages(n, page)
        t[r, :k] = numbers[at:at + k]
        at += k
    return t, pages


def _pool(gen, c, pages, dtype):
    """A pool of pages, logically [pages, slots, heads, dim], with the slots or the heads outermost in a page."""
    shape = (pages, c["page"], c["hk"], c["dim"])
    if c["order"] == "heads":
        return torch.randn(shape[0], shape[2], shape[1], shape[3], generator=gen, device="cuda", dtype=dtype).transpose(1, 2)
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pick = np.random.RandomState(seed % (1 << 32))
    s = {"case": c}
    if c["kind"] == "path":
        parents = _parents(c)
        tokens = pick.randint(0, 32000, parents.shape)
        # the model's choice after a guess is one of the guesses that follow it, four times in five
        choices = pick.randint(0, 32000, parents.shape)
        hit = pick.random_sample(parents.shape) < 0.8
        for r in range(c["rows"]):
            for i in np.nonzero((parents[r] >= 0) & hit[r])[0]:
                choices[r, parents[r, i]] = tokens[r, i]
        s["tokens"], s["parents"], s["choices"] = _i32(tokens), _i32(parents), _i32(choices)
        return s
    dtype = TYPES[c["dtype"]]
    totals = _lengths(c) if c["kind"] == "evict" else _totals(c)
    t, pages = _tables(totals, c["page"], pick)
    s["tables"], s["lengths"] = _i32(t), _i32(totals)
    if c["kind"] in ("tree", "weigh"):
        # queries twice as wide as the keys, so that the softmax has some weights well above the others
        s["q"] = 2 * torch.randn(c["rows"], c["drafts"], c["hq"], c["dim"], generator=gen, device="cuda", dtype=dtype)
        s["parents"] = _i32(_parents(c)) if c["tree"] else None
        s["k_cache"], s["v_cache"] = (_pool(gen, c, pages, dtype) for _ in range(2))
        if c["kind"] == "weigh":
            s["weights"] = torch.rand(c["rows"], c["hk"], t.shape[1] * c["page"], generator=gen, device="cuda")
        return s
    refs = np.zeros(pages, dtype=np.int32)
    refs[t[t >= 0]] = 1
    s["refs"] = _i32(refs)
    if c["kind"] == "accept":
        path, counts = _paths(c)
        s["path"], s["counts"] = _i32(path), _i32(counts)
        s["pools"] = [_pool(gen, c, pages, dtype) for _ in range(c["pools"])]
        return s
    # a few tokens get most of the attention
    s["layers"] = [(_pool(gen, c, pages, dtype), _pool(gen, c, pages, dtype),
                    torch.exp(2 * torch.randn(c["rows"], c["hk"], t.shape[1] * c["page"], generator=gen, device="cuda")))
                   for _ in range(c["layers"])]
    return s


# ---- the plain forms ----------------------------------------------------------------------------------------------

def _ancestors(s):
    """Which drafts each sees, and depths (-1: padding), from the parents on the device."""
    c, q = s["case"], s["q"]
    rows, d = c["rows"], c["drafts"]
    if s["parents"] is None:
        seen = torch.ones(d, d, dtype=torch.bool, device=q.device).tril()
        return seen.expand(rows, d, d), torch.arange(d, device=q.device).expand(rows, d)
    parent, index = s["parents"].long(), torch.arange(d, device=q.device)
    ok = (parent >= -1) & (parent < index)
    step = torch.zeros(rows, d, d, device=q.device)
    step.scatter_(2, parent.clamp(min=0)[..., None], ((parent >= 0) & ok).float()[..., None])
    # a matrix that leads from each draft to its parent: its powers lead to all ancestors
    reach = torch.eye(d, device=q.device) + step
    for _ in range(max(1, (d - 1).bit_length())):
        reach = (torch.matmul(reach, reach) > 0).float()
    reach = reach > 0
    ok = (reach <= ok[:, None, :]).all(-1)
    reach = reach & ok[..., None]
    return reach, reach.sum(-1) - 1


def _attend(s):
    c, q = s["case"], s["q"].to(torch.float32)
    rows, dim, d = c["rows"], c["dim"], c["drafts"]
    at = s["tables"].clamp(min=0).to(torch.int64)
    k = s["k_cache"][at].flatten(1, 2).to(torch.float32)  # [rows, tokens, heads, dim]
    v = s["v_cache"][at].flatten(1, 2).to(torch.float32)
    token = torch.arange(k.shape[1], device=q.device)
    base = (s["lengths"] - d)[:, None, None]
    near, depth = _ancestors(s)
    idle = (depth < 0) | (base[..., 0] < 0)
    behind = token - base  # which draft a token is
    drafted = near.gather(2, behind.clamp(0, d - 1).expand(rows, d, -1)) & (behind >= 0) & (behind < d)
    seen = (behind < 0) | drafted
    if c["window"]:
        place = torch.where(behind < 0, behind, depth.gather(1, behind[:, 0].clamp(0, d - 1))[:, None])
        seen = seen & (depth[..., None] - place < c["window"])
    seen = (seen & ~idle[..., None])[:, None, :, None]  # [rows, 1, drafts, 1, tokens]
    q = q.reshape(rows, d, c["hk"], -1, dim).permute(0, 2, 1, 3, 4)
    scores = torch.matmul(q.flatten(2, 3), k.permute(0, 2, 3, 1)).unflatten(2, (d, -1)) * (dim ** -0.5)
    if c["softcap"]:
        scores = c["softcap"] * torch.tanh(scores / c["softcap"])
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    p = torch.where(total == 0, 0.0, p / total)
    o = torch.matmul(p.flatten(2, 3), v.transpose(1, 2)).unflatten(2, (d, -1))
    lse = (top + torch.log(total))[..., 0]
    got = {"out": o.permute(0, 2, 1, 3, 4).reshape(rows, d, -1, dim).to(s["q"].dtype),
           "lse": lse.permute(0, 2, 1, 3).reshape(rows, d, -1)}
    if c["kind"] == "weigh":
        s["weights"] += p.sum((2, 3))
        got["weights"] = s["weights"]
    return got


def _path(s):
    tokens, parents, choices = s["tokens"], s["parents"].long(), s["choices"]
    rows, d = tokens.shape
    j = torch.arange(d, device="cuda")
    alive = parents[:, 0] == -1
    at = torch.zeros(rows, dtype=torch.long, device="cuda")
    path = torch.full((rows, d), -1, dtype=torch.int32, device="cuda")
    last = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    for step in range(d):
        path[:, step] = torch.where(alive, at, -1)
        choice = choices.gather(1, at[:, None])
        last = torch.where(alive, choice[:, 0], last)
        follows = (parents == at[:, None]) & (j > at[:, None]) & (tokens == choice)
        first = torch.where(follows, j, d).amin(1)
        alive = alive & (first < d)
        at = torch.where(alive, first, at)
    return {"path": path, "counts": (path >= 0).sum(1).int(), "last": last}


def _bits(x):
    """Values as whole numbers: they are moved, not computed."""
    return x.view(torch.int32 if x.element_size() == 4 else torch.int16)


def _released(s, lengths):
    """The counts once rows hold the pages of `lengths` tokens only."""
    page, j = s["case"]["page"], torch.arange(s["tables"].shape[1], device="cuda")
    gone = (j >= ((lengths + page - 1) // page)[:, None]) & (j < ((s["lengths"] + page - 1) // page)[:, None])
    return s["refs"].scatter_add(0, s["tables"].clamp(min=0).long().flatten(), -gone.int().flatten())


def _accept(s):
    c = s["case"]
    base = s["lengths"] - c["drafts"]
    row, j = (torch.arange(c["drafts"], device="cuda") < s["counts"][:, None]).nonzero().unbind(1)
    of, to = (base[row] + s["path"][row, j]).long(), (base[row] + j).long()
    of_page, to_page = s["tables"][row, of // c["page"]].long(), s["tables"][row, to // c["page"]].long()
    for pool in s["pools"]:
        pool[to_page, to % c["page"]] = pool[of_page, of % c["page"]]
    lengths = torch.where(base < 0, s["lengths"], base + s["counts"])
    return {"lengths": lengths, "refs": _released(s, lengths), "pools": [_bits(p) for p in s["pools"]]}


def _evict(s):
    c, n = s["case"], s["lengths"].long()
    page, budget, recent = c["page"], c["budget"], c["recent"]
    token = torch.arange(s["tables"].shape[1] * page, device="cuda")
    over = n > budget
    rows = over.nonzero().flatten()
    lengths = torch.where(over, budget, n).int()
    if len(rows):
        n = n[rows][:, None, None]
        to = torch.arange(budget, device="cuda")
        to_page = s["tables"][rows].long()[:, to // page]
        heads = torch.arange(c["hk"], device="cuda")
        for k, v, weights in s["layers"]:
            w = weights[rows][..., : len(token)]
            w = torch.where(token < n - recent, w, torch.where(token < n, math.inf, -math.inf))  # the recent ones stay
            of = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget].sort(-1).values
            of_page = s["tables"][rows].long().gather(1, (of // page).flatten(1)).view(of.shape)
            for pool in (k, v):  # [rows, heads, budget, dim]
                pool[to_page[:, None], to % page, heads[:, None]] = pool[of_page, of % page, heads[:, None]]
            kept = weights[rows].gather(2, of)
            weights[rows] = torch.where(token < n, 0.0, weights[rows])
            weights[rows[:, None, None], heads[:, None], to] = kept
    return {"lengths": lengths, "refs": _released(s, lengths), "layers": [[_bits(x) for x in layer] for layer in s["layers"]]}


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    return {"tree": _attend, "weigh": _attend, "path": _path, "accept": _accept, "evict": _evict}[c["kind"]](s)


# ---- the framework's operators ------------------------------------------------------------------------------------

def _run_own(s, c):
    import tensor_command_execution_gb300 as T

    if c["kind"] in ("tree", "weigh"):
        weights = s.get("weights")
        out, lse = T.attention_drafts(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lengths"], parents=s["parents"],
                                      softcap=c["softcap"], window=c["window"], weights=weights, return_lse=True)
        return {"out": out, "lse": lse} if weights is None else {"out": out, "lse": lse, "weights": weights}
    if c["kind"] == "path":
        path, counts, last = T.draft_path(s["tokens"], s["choices"], parents=s["parents"])
        return {"path": path, "counts": counts, "last": last}
    if c["kind"] == "accept":
        lengths, refs = T.cache_accept(s["tables"], s["lengths"], s["refs"], s["path"], s["counts"], s["pools"],
                                       drafts=c["drafts"])
        return {"lengths": lengths, "refs": refs, "pools": [_bits(p) for p in s["pools"]]}
    lengths, refs = T.cache_evict(s["tables"], s["lengths"], s["refs"], s["layers"], budget=c["budget"], recent=c["recent"])
    return {"lengths": lengths, "refs": refs, "layers": [[_bits(x) for x in layer] for layer in s["layers"]]}


# ---- the definitions in 64 bits -----------------------------------------------------------------------------------

def exact(case, seed):
    c = case
    if c["kind"] not in ("tree", "weigh"):
        return None  # whole numbers only
    s = prepare(c, seed)
    seen, depth = _seen(_tree(c))
    d, hk, w = c["drafts"], c["hk"], c["window"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if c["kind"] == "weigh" else None
    for r, base in enumerate(_lengths(c)):
        if base < 0:
            continue
        n, live = base + d, np.nonzero(depth[r] >= 0)[0]
        at = np.concatenate([np.arange(base), base + depth[r]])  # every token's position, drafts at their depths
        mask = np.concatenate([np.ones((len(live), base), dtype=bool), seen[r][live]], axis=1)
        if w:
            mask &= at[None, :] > (base + depth[r][live])[:, None] - w
        mask = torch.as_tensor(mask).cuda()
        page = s["tables"][r, : _pages(n, c["page"])].long()
        for h in range(hk):  # (a head at a time: the scores are large)
            k, v = (s[x][page][:, :, h].reshape(-1, c["dim"])[:n].double() for x in ("k_cache", "v_cache"))
            heads = slice(h * c["hq"] // hk, (h + 1) * c["hq"] // hk)
            q = s["q"][r][live][:, heads].double()
            z = torch.einsum("igd,td->igt", q, k) / math.sqrt(c["dim"])
            if c["softcap"]:
                z = c["softcap"] * torch.tanh(z / c["softcap"])
            z = z.masked_fill(~mask[:, None], -math.inf)
            total = torch.logsumexp(z, -1)
            p = torch.exp(z - total[..., None])
            out[r, live, heads] = torch.einsum("igt,td->igd", p, v)
            lse[r, live, heads] = total
            if weights is not None:
                weights[r, h, :n] += p.sum((0, 1))
    got = {"out": out, "lse": lse}
    return got if weights is None else {**got, "weights": weights}
