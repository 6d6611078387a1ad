"""Operators of a paged key-value cache: Python binding of ``include/cmd_cache.h``.

Rotary positions (``rope``, ``rope_backward``), the append of new tokens' keys and values (``cache_append``),
attention of one new token per sequence (``attention_decode``), the selection of the sequences that go on
(``cache_select``: fork, free, grow) and compaction (``cache_compact``); attention of a tree of drafted tokens
(``attention_drafts``, which also adds up the weight that each cached token gets), the branch that the model agrees with
(``draft_path``) and its slots (``cache_accept``); eviction by weight (``cache_evict``). The header says what each computes.

A cache is a pair of tensors [pages, page_size, kv_heads, dim] of any strides with a unit stride along dim: pages
stored with their heads outermost are passed as ``pool.transpose(1, 2)``. Tables, lengths, positions and counts are
int32. Outputs are allocated where none are given. ``stream`` is a torch.cuda.Stream, a raw handle, or None for
torch's current stream; inputs must be ready on it, and outputs and workspaces are allocated for it. Tensors of other
streams may be dropped as soon as a call returns.

The rotation is part of autograd. The operators on a cache are for serving: their results carry no gradient, whatever
their inputs require. Autograd is told of every tensor that an operator writes.

Tensors are described to the library by a small native module (csrc/cache_torch.cpp), built with it; the ``cmd_*``
functions and structures here mirror the C entry points for callers with raw pointers.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util

from . import CmdError, _build, _check, _P, lib

CMD_CACHE_MAX_DIM, CMD_CACHE_MAX_POOLS, CMD_CACHE_MAX_LAYERS, CMD_CACHE_MAX_DRAFTS = 256, 64, 32, 256
BAD_PAGE, BAD_INDEX, FULL_TABLE, NO_PAGES, SHARED_PAGE, TIMEOUT = 1, 2, 4, 8, 16, 32  # bits of the status word
LAYOUTS = {"half": 0, "interleaved": 1}
SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}

_I = ctypes.c_int
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_F32 = ctypes.c_float


# ---- one-to-one structures and wrappers of the C entry points ----------------------------------------------------

class cmd_operand(ctypes.Structure):
    _fields_ = [("ptr", _P), ("dtype", _I32), ("rank", _I32), ("sizes", _I64 * 4), ("strides", _I64 * 4)]


class cmd_rope_spec(ctypes.Structure):
    _fields_ = [("turns", _P), ("n_pairs", _I32), ("layout", _I32), ("scale", _F32), ("backward", _I32)]


class cmd_append_args(ctypes.Structure):
    _fields_ = [(n, cmd_operand) for n in ("k", "v", "k_cache", "v_cache", "tables", "positions", "rows", "q", "q_out")] + [
        ("rope", cmd_rope_spec), ("status", _P)]


class cmd_attention_args(ctypes.Structure):
    _fields_ = [(n, cmd_operand) for n in ("q", "out", "lse", "k_cache", "v_cache", "tables", "lengths")] + [
        ("scale", _F32), ("softcap", _F32), ("window", _I32), ("reserved", _I32), ("workspace", _P),
        ("workspace_bytes", _I64), ("status", _P)]


class cmd_pool(ctypes.Structure):
    _fields_ = [("ptr", _P), ("page_bytes", _I64), ("page_stride", _I64)]


_POOL_FIELDS = [("pools", ctypes.POINTER(cmd_pool)), ("n_pools", _I32), ("page_size", _I32), ("workspace", _P),
                ("workspace_bytes", _I64), ("status", _P)]


class cmd_select_args(ctypes.Structure):
    _fields_ = [(n, cmd_operand) for n in ("tables", "lengths", "refs", "parents", "grow", "tables_out", "lengths_out",
                                           "refs_out")] + _POOL_FIELDS


class cmd_compact_args(ctypes.Structure):
    _fields_ = [(n, cmd_operand) for n in ("tables", "lengths", "refs", "tables_out", "refs_out",
                                           "page_map_out")] + _POOL_FIELDS


_OP = ctypes.POINTER(cmd_operand)


class cmd_drafts_args(ctypes.Structure):
    _fields_ = [(n, cmd_operand) for n in ("q", "out", "lse", "k_cache", "v_cache", "tables", "lengths", "parents",
                                           "weights")] + [
        ("scale", _F32), ("softcap", _F32), ("window", _I32), ("reserved", _I32), ("workspace", _P),
        ("workspace_bytes", _I64), ("status", _P)]


class cmd_path_args(ctypes.Structure):
    _fields_ = [(n, cmd_operand) for n in ("tokens", "choices", "parents", "path", "counts", "last")] + [("status", _P)]


class cmd_accept_args(ctypes.Structure):
    _fields_ = [(n, cmd_operand) for n in ("tables", "lengths", "refs", "path", "counts", "lengths_out", "refs_out")] + [
        ("pools", _OP), ("n_pools", _I32), ("reserved", _I32), ("status", _P)]


class cmd_evict_args(ctypes.Structure):
    _fields_ = [(n, cmd_operand) for n in ("tables", "lengths", "refs", "lengths_out", "refs_out")] + [
        ("k_caches", _OP), ("v_caches", _OP), ("weights", _OP), ("n_layers", _I32), ("budget", _I32), ("recent", _I32),
        ("reserved", _I32), ("workspace", _P), ("workspace_bytes", _I64), ("status", _P)]


# Every symbol include/cmd_cache.h declares, with (restype, argtypes).
SIGNATURES = {
    "cmd_rope_turns": (_I, [_I32, ctypes.c_double, _I32] + [ctypes.c_double] * 4 + [ctypes.POINTER(ctypes.c_uint64)]),
    "cmd_rope": (_I, [_OP] * 5 + [ctypes.POINTER(cmd_rope_spec), _P]),
    "cmd_cache_append": (_I, [ctypes.POINTER(cmd_append_args), _P]),
    "cmd_attention_workspace": (_I, [_I32, _I32, _I32, ctypes.POINTER(_I64)]),
    "cmd_attention_decode": (_I, [ctypes.POINTER(cmd_attention_args), _P]),
    "cmd_select_workspace": (_I, [_I64, _I64, _I64, ctypes.POINTER(_I64)]),
    "cmd_cache_select": (_I, [ctypes.POINTER(cmd_select_args), _P]),
    "cmd_compact_workspace": (_I, [_I64, ctypes.POINTER(_I64)]),
    "cmd_cache_compact": (_I, [ctypes.POINTER(cmd_compact_args), _P]),
    "cmd_drafts_workspace": (_I, [_I64] + [_I32] * 4 + [_I64, ctypes.POINTER(_I64)]),
    "cmd_attention_drafts": (_I, [ctypes.POINTER(cmd_drafts_args), _P]),
    "cmd_attention_drafts_workspace": (_I, [ctypes.POINTER(cmd_drafts_args), ctypes.POINTER(_I64)]),
    "cmd_draft_path": (_I, [ctypes.POINTER(cmd_path_args), _P]),
    "cmd_cache_accept": (_I, [ctypes.POINTER(cmd_accept_args), _P]),
    "cmd_evict_workspace": (_I, [_I64] + [_I32] * 3 + [ctypes.POINTER(_I64)]),
    "cmd_cache_evict": (_I, [ctypes.POINTER(cmd_evict_args), _P]),
    "cmd_cache_status": (_I, [_P, ctypes.POINTER(_I32), _P]),
}

_entry: dict = {}


def entry(name: str):
    """The library's entry point of that name, with its signature set."""
    f = _entry.get(name)
    if f is None:
        f = getattr(lib(), name)
        f.restype, f.argtypes = SIGNATURES[name]
        _entry[name] = f
    return f


def cmd_rope_turns(n_pairs: int, base: float, scaling: int, factor: float, original_length: float, beta_fast: float,
                   beta_slow: float) -> list:
    out = (ctypes.c_uint64 * max(1, n_pairs))()
    _check(entry("cmd_rope_turns")(n_pairs, base, scaling, factor, original_length, beta_fast, beta_slow, out),
           "cmd_rope_turns")
    return list(out)[:n_pairs]


def cmd_attention_workspace(q_heads: int, kv_heads: int, dim: int) -> int:
    n = _I64()
    _check(entry("cmd_attention_workspace")(q_heads, kv_heads, dim, ctypes.byref(n)), "cmd_attention_workspace")
    return n.value


def cmd_select_workspace(old_rows: int, new_rows: int, pages: int) -> int:
    n = _I64()
    _check(entry("cmd_select_workspace")(old_rows, new_rows, pages, ctypes.byref(n)), "cmd_select_workspace")
    return n.value


def cmd_compact_workspace(pages: int) -> int:
    n = _I64()
    _check(entry("cmd_compact_workspace")(pages, ctypes.byref(n)), "cmd_compact_workspace")
    return n.value


def cmd_drafts_workspace(rows: int, drafts: int, q_heads: int, kv_heads: int, dim: int, tokens: int = 0) -> int:
    n = _I64()
    _check(entry("cmd_drafts_workspace")(rows, drafts, q_heads, kv_heads, dim, tokens, ctypes.byref(n)),
           "cmd_drafts_workspace")
    return n.value


def cmd_evict_workspace(rows: int, layers: int, kv_heads: int, budget: int) -> int:
    n = _I64()
    _check(entry("cmd_evict_workspace")(rows, layers, kv_heads, budget, ctypes.byref(n)), "cmd_evict_workspace")
    return n.value


# ---- the operators -----------------------------------------------------------------------------------------------

_module = None


def _native():
    """The native module, loaded on first use (with the library; both are built when missing or stale)."""
    global _module
    if _module is None:
        import torch  # noqa: F401  (its libraries come first)
        lib()
        loader = importlib.machinery.ExtensionFileLoader("_cache_torch", _build.module_path())
        m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_cache_torch", loader))
        loader.exec_module(m)
        m.set_error(CmdError)
        _module = m
    return _module


class _On:
    """`stream` as the current stream of `like`'s device while a call is made. Tensors that it uses and that belong to
    another stream stay allocated until the work is done, however soon the caller drops them."""

    def __init__(self, stream, like, *used):
        import torch
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), like.device)
        self.stream, self.current, self.used = stream, torch.cuda.stream(stream), (like, *used)

    def __enter__(self):
        self.current.__enter__()

    def __exit__(self, kind, error, trace):
        if kind is None:
            for x in self.used:
                if getattr(x, "is_cuda", False):
                    x.record_stream(self.stream)
        return self.current.__exit__(kind, error, trace)


def _layout(layout):
    code = LAYOUTS.get(layout)
    if code is None:
        raise ValueError(f"unknown layout {layout!r}: half or interleaved")
    return code


def rope_turns(rotated: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
               original_length: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """Turns per position of each of the ``rotated`` / 2 pairs, as 64-bit fractions of a turn (an int64 tensor whose
    bits the operators read as unsigned): the ``turns`` of ``rope`` and ``cache_append``. scaling: none, linear, base
    or parts (cmd_rope_scaling in the header)."""
    import torch
    if rotated % 2:
        raise ValueError("an odd number of rotated elements")
    if scaling not in SCALINGS:
        raise ValueError(f"unknown scaling {scaling!r}: one of {', '.join(SCALINGS)}")
    w = cmd_rope_turns(rotated // 2, base, SCALINGS[scaling], factor, original_length, beta_fast, beta_slow)
    return torch.tensor([x - (1 << 64) if x >> 63 else x for x in w], dtype=torch.int64).to(device)


_function = None


def _recorded():
    """The rotation as a function of autograd: linear, so that its gradient is the transposed rotation."""
    global _function
    if _function is None:
        import torch

        class Rope(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, positions, turns, layout, scale, backward):
                ctx.save_for_backward(positions, turns)
                ctx.call = layout, scale, backward
                ctx.set_materialize_grads(False)
                got = (_module or _native()).rope(q, k, positions, turns, _layout(layout), scale, None, None, backward)
                ctx.mark_non_differentiable(*(y for y, needed in zip(got, ctx.needs_input_grad) if y is not None and not needed))
                return got

            @staticmethod
            def backward(ctx, *grads):
                # (the kernels read rows of unit stride: a sum's gradient has none)
                grads = [g.resolve_neg() if g is not None and needed else None for g, needed in zip(grads, ctx.needs_input_grad)]
                grads = [g if g is None or g.stride(-1) == 1 or g.shape[-1] < 2 else g.contiguous() for g in grads]
                if all(g is None for g in grads):
                    return (None,) * 7
                positions, turns = ctx.saved_tensors
                layout, scale, backward = ctx.call
                return (*_rope(*grads, positions, turns, layout, scale, None, None, not backward), *(None,) * 5)
        _function = Rope
    return _function


def _rope(q, k, positions, turns, layout, scale, out, stream, backward):
    q_out, k_out = (None, None) if out is None else out
    if stream is not None:
        with _On(stream, q if q is not None else k, k, positions, turns, q_out, k_out):
            return _rope(q, k, positions, turns, layout, scale, out, None, backward)
    if getattr(q, "requires_grad", False) or getattr(k, "requires_grad", False):
        import torch
        if torch.is_grad_enabled():
            if out is not None:
                raise ValueError("out= records no gradient: q or k requires one")
            return _recorded().apply(q, k, positions, turns, layout, scale, backward)
    return (_module or _native()).rope(q, k, positions, turns, _layout(layout), scale, q_out, k_out, backward)


def rope(q, k, positions, turns, *, layout: str = "half", scale: float = 1.0, out=None, stream=None):
    """q and k ([batch,] tokens, heads, dim; either may be None) rotated by their positions, as (q, k). out: the pair
    of outputs (the inputs themselves: in place). Autograd records the call where an input requires a gradient (out= is
    refused then)."""
    return _rope(q, k, positions, turns, layout, scale, out, stream, False)


def rope_backward(dq, dk, positions, turns, *, layout: str = "half", scale: float = 1.0, out=None, stream=None):
    """The gradients of rope's inputs from those of its outputs (for programs that keep their own graph; recorded by
    autograd as rope is)."""
    return _rope(dq, dk, positions, turns, layout, scale, out, stream, True)


def cache_append(k, v, k_cache, v_cache, tables, positions, *, rows=None, q=None, q_out=None, turns=None,
                 layout: str = "half", scale: float = 1.0, status=None, stream=None):
    """Store each token's key, rotated where turns is given, and value in its page; returns q rotated (None without
    q). rows: each token's table row (None: token t has row t)."""
    if stream is not None:
        with _On(stream, k, v, k_cache, v_cache, tables, positions, rows, q, q_out, turns, status):
            return cache_append(k, v, k_cache, v_cache, tables, positions, rows=rows, q=q, q_out=q_out, turns=turns,
                                layout=layout, scale=scale, status=status)
    return (_module or _native()).cache_append(k, v, k_cache, v_cache, tables, positions, rows, q, q_out, turns,
                                               _layout(layout), scale, status)


def attention_decode(q, k_cache, v_cache, tables, lengths, *, scale: float | None = None, softcap: float = 0.0,
                     window: int = 0, out=None, lse=None, return_lse: bool = False, workspace=None, status=None,
                     stream=None):
    """Attention of one new token per row: q [rows, q_heads, dim] over the first lengths[r] tokens of row r. Returns
    out, or (out, lse) with return_lse. scale: dim ** -0.5 unless given. workspace: cmd_attention_workspace bytes
    (allocated where None)."""
    if stream is not None:
        with _On(stream, q, k_cache, v_cache, tables, lengths, out, lse, workspace, status):
            return attention_decode(q, k_cache, v_cache, tables, lengths, scale=scale, softcap=softcap, window=window,
                                    out=out, lse=lse, return_lse=return_lse, workspace=workspace, status=status)
    return (_module or _native()).attention_decode(q, k_cache, v_cache, tables, lengths, scale, softcap, window, out, lse,
                                                   return_lse, workspace, status)


def cache_select(tables, lengths, refs, parents, pools, *, page_size: int, grow=None, out=None, status=None,
                 stream=None):
    """New row i goes on from row parents[i] (-1: an empty row) with room for grow[i] more tokens; pages in progress
    are copied in every pool for later children. pools: up to 64 tensors [pages, ...] whose pages are dense (for more,
    a call for each 64, with the same inputs). Returns (tables, lengths, refs); out: those three, to write to. When the
    pool runs out, the first row that gets no page is dropped, and every later one that needs any."""
    if stream is not None:
        with _On(stream, tables, lengths, refs, parents, *pools, grow, *(out or ()), status):
            return cache_select(tables, lengths, refs, parents, pools, page_size=page_size, grow=grow, out=out, status=status)
    return (_module or _native()).cache_select(tables, lengths, refs, parents, pools, page_size, grow, out, status)


def cache_compact(tables, lengths, refs, pools, *, page_size: int, out=None, status=None, stream=None):
    """The pages in use moved to the front of every pool (up to 64; for more, a call for each 64 with the same inputs).
    Returns (tables, refs, page_map); out: those three."""
    if stream is not None:
        with _On(stream, tables, lengths, refs, *pools, *(out or ()), status):
            return cache_compact(tables, lengths, refs, pools, page_size=page_size, out=out, status=status)
    return (_module or _native()).cache_compact(tables, lengths, refs, pools, page_size, out, status)


def attention_drafts(q, k_cache, v_cache, tables, lengths, *, parents=None, scale: float | None = None,
                     softcap: float = 0.0, window: int = 0, weights=None, out=None, lse=None, return_lse: bool = False,
                     workspace=None, status=None, stream=None):
    """Attention of each row's last drafts, a tree: q [rows, drafts, q_heads, dim], whose keys and values are the last
    of the first lengths[r] tokens of row r. parents [rows, drafts]: the draft that each goes on from (below its own
    index; -1: the tokens before the drafts; less: padding); None: each goes on from the one before. A draft sees the
    tokens before the drafts, its ancestors and itself. weights [rows, kv_heads, tokens], float32: the attention that
    each token got is added to it. Returns out, or (out, lse) with return_lse. scale: dim ** -0.5 unless given.
    workspace: at most cmd_drafts_workspace bytes (allocated where None)."""
    if stream is not None:
        with _On(stream, q, k_cache, v_cache, tables, lengths, parents, weights, out, lse, workspace, status):
            return attention_drafts(q, k_cache, v_cache, tables, lengths, parents=parents, scale=scale, softcap=softcap,
                                    window=window, weights=weights, out=out, lse=lse, return_lse=return_lse,
                                    workspace=workspace, status=status)
    return (_module or _native()).attention_drafts(q, k_cache, v_cache, tables, lengths, parents, scale, softcap, window,
                                                   weights, out, lse, return_lse, workspace, status)


def draft_path(tokens, choices, *, parents=None, out=None, status=None, stream=None):
    """The branch of each row's tree of drafts that agrees with the model: from draft 0 to the first draft that goes on
    from it with the token choices[r][0], which the model chooses after draft 0, and so on. tokens, choices, parents:
    [rows, drafts] (parents as in attention_drafts). Returns (path, counts, last): the drafts passed (then -1), their
    number, and the choice after the last of them; out: those three, to write to."""
    if stream is not None:
        with _On(stream, tokens, choices, parents, *(out or ()), status):
            return draft_path(tokens, choices, parents=parents, out=out, status=status)
    return (_module or _native()).draft_path(tokens, choices, parents, out, status)


def cache_accept(tables, lengths, refs, path, counts, pools, *, drafts: int | None = None, out=None, status=None,
                 stream=None):
    """Of each row's last drafts (as many as path has columns; drafts, where given, has to say the same) keeps the
    first counts[r] of path[r]: their keys and values move together behind the tokens before the drafts, and pages past
    them are released. pools: up to 64 tensors [pages, page_size, kv_heads, dim] (for more, a call for each 64, with
    the same inputs). Returns (lengths, refs); out: those two, to write to."""
    if stream is not None:
        with _On(stream, tables, lengths, refs, path, counts, *pools, *(out or ()), status):
            return cache_accept(tables, lengths, refs, path, counts, pools, drafts=drafts, out=out, status=status)
    return (_module or _native()).cache_accept(tables, lengths, refs, path, counts, pools, drafts, out, status)


def cache_evict(tables, lengths, refs, layers, *, budget: int, recent: int = 0, out=None, status=None, stream=None):
    """Holds rows to a budget: in each layer, a (k_cache, v_cache, weights) triple, each kv head of a longer row keeps
    the last `recent` tokens and the others of the largest weights, moved together in their order, weights too; pages
    past them are released. Up to 32 layers (for more, a call for each 32, with the same inputs). Returns (lengths,
    refs); out: those two, to write to."""
    if stream is not None:
        with _On(stream, tables, lengths, refs, *(x for layer in layers for x in layer), *(out or ()), status):
            return cache_evict(tables, lengths, refs, layers, budget=budget, recent=recent, out=out, status=status)
    return (_module or _native()).cache_evict(tables, lengths, refs, layers, budget, recent, out, status)


def cache_status(status, stream=None) -> None:
    """Wait for the stream and raise CmdError if an operator given this status word met an invalid table or index, or
    had no room; the word is cleared."""
    if stream is not None:
        with _On(stream, status):
            return cache_status(status)
    (_module or _native()).cache_status(status)
