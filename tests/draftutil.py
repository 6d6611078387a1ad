"""Plain 64-bit forms of the operators for drafted tokens and budgets, and trees to test them on."""
from __future__ import annotations

import math
import random

import torch

import cacheutil as U


def trees(rows, drafts, kind, seed=0):
    """Parents [rows][drafts]: chains, random trees, forests (several roots), stars, or trees with padding and invalid
    entries among them."""
    rng, out = random.Random(seed), []
    for r in range(rows):
        p = []
        for i in range(drafts):
            x = i - 1
            if kind == "tree" and i > 1:
                x = rng.randint(max(0, i - rng.choice([1, 3, 9])), i - 1)
            if kind == "forest":
                x = rng.randint(-1, i - 1)
            if kind == "star":
                x = min(i - 1, 0)
            if kind == "padded":
                x = rng.choice([rng.randint(-1, i - 1), rng.randint(-1, i - 1), i - 1, -2, -2 ** 31])
            p.append(x)
        out.append(p)
    return out


def seen_by(parents):
    """Each draft's ancestors and itself (None: padding), in order from the root."""
    out = []
    for i, p in enumerate(parents):
        if p == -1:
            out.append([i])
        elif 0 <= p < i and out[p] is not None:
            out.append(out[p] + [i])
        else:
            out.append(None)
    return out


def drafted(q, cache, lengths, parents, scale, softcap=0.0, window=0):
    """(out, lse, weights, and a bound on each) in binary64: what the attention of drafts gives, and how far arithmetic
    in 32 bits may be from it. lengths include the drafts; weights is a list of [kv heads, tokens]."""
    rows, drafts, heads, dim = q.shape
    out = torch.zeros(rows, drafts, heads, dim, dtype=torch.float64)
    lse = torch.full((rows, drafts, heads), -math.inf, dtype=torch.float64)
    bound, lse_bound = torch.zeros_like(out), torch.zeros_like(lse)
    weights, weight_bounds = [], []
    for r, n in enumerate(lengths):
        hk = cache.k.shape[2]
        weights.append(torch.zeros(hk, n, dtype=torch.float64))
        weight_bounds.append(torch.zeros(hk, n, dtype=torch.float64))
        base = n - drafts
        if base < 0:
            continue
        k, v = cache.rows(r, n)
        for i, path in enumerate(seen_by(parents[r])):
            if path is None:
                continue
            at = [(t, t) for t in range(base)] + [(base + j, base + d) for d, j in enumerate(path)]  # token, position
            mine = base + len(path) - 1
            t = torch.tensor([t for t, x in at if not window or x > mine - window])
            x = q[r, i].cpu().double().reshape(hk, -1, dim)
            kk, vv = k[t], v[t]
            s = torch.einsum("hgd,thd->hgt", x, kk) * scale
            # a dot product of dim terms in binary32, and four roundings of the score: of |q| . |k|
            err = (dim + 4) * 2.0 ** -24 * torch.einsum("hgd,thd->hgt", x.abs(), kk.abs()).amax(-1) * scale
            if softcap:
                s = softcap * torch.tanh(s / softcap)
                err = err + 4 * 2.0 ** -24 * softcap
            w = torch.softmax(s, -1)
            out[r, i] = torch.einsum("hgt,thd->hgd", w, vv).reshape(heads, dim)
            lse[r, i] = torch.logsumexp(s, -1).reshape(heads)
            # a weight is off by twice its score's error, the scores' distance to the maximum rounds, sums of n terms round
            each = 2 * err + (s.abs().amax(-1) * 4 + n + 8) * 2.0 ** -24
            bound[r, i] = (each[..., None] * torch.einsum("hgt,thd->hgd", w, vv.abs())).reshape(heads, dim)
            lse_bound[r, i] = (each + 4 * 2.0 ** -24).reshape(heads)
            weights[r][:, t] += w.sum(1)
            # (... and the sum over the rows, and the hardware's 2^x, good to 2^-22)
            weight_bounds[r][:, t] += ((each[..., None] + (drafts * heads + 8) * 2.0 ** -24) * w).sum(1)
    return out, lse, weights, bound, lse_bound, weight_bounds


def split_error(kind):
    """What holding a weight as two 16-bit numbers may leave of it."""
    return {"f32": 0.0, "f16": 2.0 ** -21, "bf16": 2.0 ** -16}[kind]


def walked(tokens, choices, parents):
    """The accepted branch of one row, in Python: (path, last)."""
    if parents[0] != -1:
        return [], -1
    path = [0]
    while True:
        at = path[-1]
        nxt = [j for j in range(at + 1, len(tokens)) if parents[j] == at and tokens[j] == choices[at]]
        if not nxt:
            return path, choices[at]
        path.append(nxt[0])


def slots(cache, r, n):
    """The page and slot of each of row r's first n tokens."""
    t = torch.arange(n, device=cache.tables.device)
    return cache.tables[r].long()[t // cache.page], t % cache.page



def evicted(weights, n, budget, recent):
    """Which of a row's n tokens one head keeps, ascending."""
    before = sorted(range(n - recent), key=lambda t: (0, -weights[t], t) if not math.isnan(weights[t]) else (1, 0.0, t))
    return sorted(before[: budget - recent]) + list(range(n - recent, n))


def counts(cache):
    refs = torch.zeros(cache.pages, dtype=torch.int32, device="cuda")
    for r, n in enumerate(cache.need):
        refs[cache.tables[r, :n].long()] += 1
    return refs
