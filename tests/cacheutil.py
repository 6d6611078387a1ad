"""Plain 64-bit forms of the cache operators, and caches to test them on."""
from __future__ import annotations

import math

import numpy as np
import torch

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROUND = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}   # one rounding (bf16: 8 bits)
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half of the smallest step


def angles(positions, turns):
    """Angle of each position and pair in binary64, from Python integers."""
    t = [int(x) % (1 << 64) for x in turns.tolist()]
    flat = [[2 * math.pi * ((int(p) * w) % (1 << 64)) / 2.0 ** 64 for w in t] for p in positions.flatten().tolist()]
    return torch.tensor(flat, dtype=torch.float64).reshape(*positions.shape, len(t))


def rotated(x, positions, turns, layout, scale, backward=False):
    """x [..., heads, dim] rotated in binary64 (on the CPU)."""
    x = x.detach().cpu().double()
    a = angles(positions.cpu(), turns.cpu())
    c, s = (scale * torch.cos(a))[..., None, :], (scale * torch.sin(-a if backward else a))[..., None, :]
    n = a.shape[-1]
    y = x.clone()
    i, j = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return y


def rope_bound(x, want, n_pairs, layout, scale, kind):
    """The error a rotation may have: the angle is the 64-bit phase's upper 32 bits rounded to 24 (2^-24 of half a
    turn, relative), its sine and cosine are good to 2 ulp, two products and a sum round: under 8 * 2^-24 of the
    pair's magnitudes; and one rounding to the type."""
    x = x.detach().cpu().double().abs()
    pair = torch.zeros_like(x)
    n = n_pairs
    i, j = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    pair[..., i] = pair[..., j] = x[..., i] + x[..., j]
    return 8 * 2.0 ** -24 * abs(scale) * pair + ROUND[kind] * want.abs() * (1 + 2.0 ** -20) + TINY[kind]


class Cache:
    """Pools of random values with a shuffled page table. order: "slots" or "heads" outermost in a page, or "both":
    keys and values interleaved in one tensor."""

    def __init__(self, kind, lengths, heads, dim, page, order="slots", spare=3, columns=None, seed=0, junk=None, pad=0):
        rng = np.random.RandomState(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        need = [-(-n // page) for n in lengths]
        pages, rows = sum(need) + spare, len(lengths)
        columns = max(need + [1]) if columns is None else columns
        numbers = rng.permutation(pages)
        t = np.full((rows, columns), 0x7ffffff0, dtype=np.int32)  # (never to be read)
        at = 0
        for r, n in enumerate(need):
            t[r, :n] = numbers[at:at + n]
            at += n
        self.tables = torch.from_numpy(t).cuda()
        self.lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        dt = TYPES[kind]

        def make(*shape):
            return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)
        wide = dim + pad  # (rows padded past the head dim)
        if order == "slots":
            self.k, self.v = make(pages, page, heads, wide)[..., :dim], make(pages, page, heads, wide)[..., :dim]
        elif order == "heads":
            self.k, self.v = (make(pages, heads, page, wide)[..., :dim].transpose(1, 2) for _ in range(2))
        else:
            both = make(pages, 2, page, heads, wide)
            self.k, self.v = both[:, 0, ..., :dim], both[:, 1, ..., :dim]
        self.page, self.pages, self.need = page, pages, need
        if junk is not None:  # what no row's tokens occupy
            used = torch.zeros(pages, page, dtype=torch.bool)
            for r, n in enumerate(lengths):
                for i in range(n):
                    used[t[r, i // page], i % page] = True
            self.k[~used.cuda()] = junk
            self.v[~used.cuda()] = junk

    def rows(self, r, n):
        """Row r's first n keys and values, [n, heads, dim], binary64 on the CPU."""
        page = self.tables[r, : -(-n // self.page)].long()
        return tuple(x[page].reshape(-1, x.shape[2], x.shape[3])[:n].cpu().double() for x in (self.k, self.v))


def attended(q, cache, lengths, scale, softcap=0.0, window=0):
    """(out, lse, bound) in binary64: what attention gives, and how far arithmetic in 32 bits may be from it."""
    rows, heads, dim = q.shape
    out = torch.zeros(rows, heads, dim, dtype=torch.float64)
    lse = torch.full((rows, heads), -math.inf, dtype=torch.float64)
    bound = torch.zeros_like(out)
    lse_bound = torch.zeros_like(lse)
    for r, n in enumerate(lengths):
        lo = max(0, n - window) if window else 0
        if n <= lo:
            continue
        k, v = (x[lo:] for x in cache.rows(r, n))
        h = k.shape[1]
        x = q[r].cpu().double().reshape(h, -1, dim)
        s = torch.einsum("hgd,thd->hgt", x, k) * scale
        # a dot product of dim terms in binary32, and four roundings of the score: of |q| . |k|
        err = (dim + 4) * 2.0 ** -24 * torch.einsum("hgd,thd->hgt", x.abs(), k.abs()).amax(-1) * scale
        if softcap:
            s = softcap * torch.tanh(s / softcap)
            err = err + 4 * 2.0 ** -24 * softcap
        w = torch.softmax(s, -1)
        out[r] = torch.einsum("hgt,thd->hgd", w, v).reshape(heads, dim)
        lse[r] = torch.logsumexp(s, -1).reshape(heads)
        # a weight is off by twice its score's error, the scores' distance to the maximum rounds, sums of n terms round
        each = 2 * err + (s.abs().amax(-1) * 4 + n + 8) * 2.0 ** -24
        bound[r] = (each[..., None] * torch.einsum("hgt,thd->hgd", w, v.abs())).reshape(heads, dim)
        lse_bound[r] = (each + 4 * 2.0 ** -24).reshape(heads)
    return out, lse, bound, lse_bound


def select_reference(tables, lengths, refs, parents, grow, page):
    """The selection row by row, in Python; returns (tables, lengths, refs, copies)."""
    columns = tables.shape[1]
    pages_of = lambda n: -(-n // page)  # noqa: E731
    count = [int(x) for x in refs]
    for r, n in enumerate(lengths):
        for j in range(pages_of(n)):
            count[tables[r][j]] -= 1
    seen, plan = set(), []
    for p, g in zip(parents, grow):
        n = int(lengths[p]) if p >= 0 else 0
        total = pages_of(n + g)
        if total > columns:
            plan.append(None)
            continue
        own_copy = p in seen and n % page != 0
        seen.add(p)
        shared = [int(x) for x in tables[p][:pages_of(n)]] if p >= 0 else []
        keep = shared[:-1] if own_copy else shared
        for x in keep:
            count[x] += 1
        plan.append((n + g, keep, total, shared[-1] if own_copy else None))
    free = [i for i, c in enumerate(count) if c == 0]
    out = np.full((len(parents), columns), -1, dtype=np.int32)
    lens, copies, at = np.zeros(len(parents), dtype=np.int32), [], 0
    for i, x in enumerate(plan):
        if x is None:
            continue
        n, keep, total, source = x
        want = total - len(keep)
        mine = free[at:at + want]
        at += want
        if len(mine) < want:
            for y in keep:
                count[y] -= 1
            continue
        if source is not None:
            copies.append((source, mine[0]))
        for y in mine:
            count[y] = 1
        out[i, :total] = keep + mine
        lens[i] = n
    return out, lens, np.array(count, dtype=np.int32), copies
