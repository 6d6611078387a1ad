"""Operators of a paged key-value cache: Python binding of ``include/cmd_cache.h``.

Rotary positions (``rope``, ``rope_backward``), the append of new tokens' keys and values (``cache_append``),
attention of one new token per sequence (``attention_decode``), the selection of the sequences that go on
(``cache_select``: fork, free, grow) and compaction (``cache_compact``). The header says what each computes; here
torch tensors are checked to lie on a GPU, described to the library, and outputs are allocated where none are given.

A cache is a pair of tensors [pages, page_size, kv_heads, dim] of any strides with a unit stride along dim: pages
stored with their heads outermost are passed as ``pool.transpose(1, 2)``. Tables, lengths, positions and counts are
int32. ``stream`` is a torch.cuda.Stream, a raw handle, or None for torch's current stream; inputs must be ready on
it, and outputs and workspaces are allocated for it.
"""
from __future__ import annotations

import ctypes
import math
import struct

from . import _check, _P, lib

LAYOUTS = {"half": 0, "interleaved": 1}
SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}
BAD_PAGE, BAD_INDEX, FULL_TABLE, NO_PAGES = 1, 2, 4, 8

_I = ctypes.c_int
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_BYTES = ctypes.c_char_p  # (a packed argument structure)

# Every symbol include/cmd_cache.h declares, with (restype, argtypes).
SIGNATURES = {
    "cmd_rope_turns": (_I, [_I32, ctypes.c_double, _I32] + [ctypes.c_double] * 4 + [_P]),
    "cmd_rope": (_I, [_BYTES] * 6 + [_P]),
    "cmd_cache_append": (_I, [_BYTES, _P]),
    "cmd_attention_workspace": (_I, [_I32, _I32, _I32, ctypes.POINTER(_I64)]),
    "cmd_attention_decode": (_I, [_BYTES, _P]),
    "cmd_select_workspace": (_I, [_I64, _I64, _I64, ctypes.POINTER(_I64)]),
    "cmd_cache_select": (_I, [_BYTES, _P]),
    "cmd_compact_workspace": (_I, [_I64, ctypes.POINTER(_I64)]),
    "cmd_cache_compact": (_I, [_BYTES, _P]),
    "cmd_cache_status": (_I, [_P, ctypes.POINTER(_I32), _P]),
}

_entry = {}


def _call(name):
    """The library's entry point of that name, with its signature set."""
    f = _entry.get(name)
    if f is None:
        f = getattr(lib(), name)
        f.restype, f.argtypes = SIGNATURES[name]
        _entry[name] = f
    return f


# ---- argument marshalling --------------------------------------------------------------------------------------

_OPERAND = "Pii8q"  # cmd_operand
_ROPE = "Piifi"     # cmd_rope_spec
_pack_operand = struct.Struct("@" + _OPERAND).pack
_pack_rope = struct.Struct("@" + _ROPE).pack
_append_args = struct.Struct("@" + _OPERAND * 9 + _ROPE + "P")
_attention_args = struct.Struct("@" + _OPERAND * 7 + "ffiiPqP")
_select_args = struct.Struct("@" + _OPERAND * 8 + "PiiPqP")
_compact_args = struct.Struct("@" + _OPERAND * 6 + "PiiPqP")

_ABSENT = (0, 0, 0) + (0,) * 8
_dtype_codes = {}


def _code(dtype):
    if not _dtype_codes:
        import torch
        _dtype_codes.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.int32: 3})
    c = _dtype_codes.get(dtype)
    if c is None:
        raise TypeError(f"the operators take float32, float16, bfloat16 and int32 tensors, not {dtype}")
    return c


_ZEROS = ((), (0,), (0, 0), (0, 0, 0), (0, 0, 0, 0))


def _operand(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} is not on a GPU")
    shape = t.shape
    n = len(shape)
    if n > 4:
        raise ValueError(f"{name} has rank {n}: at most 4")
    pad = _ZEROS[4 - n]
    return (t.data_ptr(), _code(t.dtype), n) + tuple(shape) + pad + t.stride() + pad


def _optional(t, name):
    return _ABSENT if t is None else _operand(t, name)


def _status(status):
    if status is None:
        return 0
    if not status.is_cuda or status.numel() != 1 or _code(status.dtype) != 3:
        raise ValueError("status is one int32 on a GPU")
    return status.data_ptr()


class _Stream:
    """The stream of a call: its handle, and torch allocations made for it."""

    def __init__(self, stream, like):
        import torch
        self.device = like.device
        if stream is None:
            self.handle = torch._C._cuda_getCurrentRawStream(like.device.index)
            self.other = None
        else:
            self.handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
            self.other = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(self.handle, self.device)

    def empty(self, shape, dtype, zero=False):
        import torch
        make = torch.zeros if zero else torch.empty
        if self.other is None:
            return make(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.other):
            return make(shape, dtype=dtype, device=self.device)


# ---- rotary positions --------------------------------------------------------------------------------------------

def cmd_rope_turns(n_pairs: int, base: float, scaling: int, factor: float, original_length: float, beta_fast: float,
                   beta_slow: float) -> list:
    out = (ctypes.c_uint64 * max(1, n_pairs))()
    _check(_call("cmd_rope_turns")(n_pairs, base, scaling, factor, original_length, beta_fast, beta_slow, out),
           "cmd_rope_turns")
    return list(out)[:n_pairs]


def rope_turns(rotated: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
               original_length: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """Turns per position of each of the ``rotated`` / 2 pairs, as 64-bit fractions of a turn (an int64 tensor whose
    bits the operators read as unsigned): the ``turns`` of ``rope`` and ``cache_append``."""
    import torch
    if rotated % 2:
        raise ValueError("an odd number of rotated elements")
    if scaling not in SCALINGS:
        raise ValueError(f"unknown scaling {scaling!r}: one of {', '.join(SCALINGS)}")
    w = cmd_rope_turns(rotated // 2, base, SCALINGS[scaling], factor, original_length, beta_fast, beta_slow)
    return torch.tensor([x - (1 << 64) if x >> 63 else x for x in w], dtype=torch.int64).to(device)


def _spec(turns, layout, scale, backward):
    if layout not in LAYOUTS:
        raise ValueError(f"unknown layout {layout!r}: half or interleaved")
    if turns is None:
        return (0, 0, LAYOUTS[layout], scale, 0)
    import torch
    if not turns.is_cuda or turns.dtype != torch.int64 or turns.dim() != 1 or not turns.is_contiguous():
        raise ValueError("turns is a contiguous int64 vector on a GPU (see rope_turns)")
    return (turns.data_ptr(), turns.shape[0], LAYOUTS[layout], scale, backward)


def _rope(q, k, positions, turns, layout, scale, out, stream, backward):
    like = q if q is not None else k
    if like is None:
        raise ValueError("q and k are both absent")
    s = _Stream(stream, like)
    q_out, k_out = out if out is not None else (None, None)
    if q is not None and q_out is None:
        q_out = s.empty(q.shape, q.dtype)
    if k is not None and k_out is None:
        k_out = s.empty(k.shape, k.dtype)
    packed = [None if t is None else _pack_operand(*_operand(t, n))
              for t, n in ((q, "q"), (q_out if q is not None else None, "q_out"), (k, "k"),
                           (k_out if k is not None else None, "k_out"), (positions, "positions"))]
    _check(_call("cmd_rope")(*packed, _pack_rope(*_spec(turns, layout, scale, backward)), s.handle), "cmd_rope")
    return q_out, k_out


def rope(q, k, positions, turns, *, layout: str = "half", scale: float = 1.0, out=None, stream=None):
    """q and k ([batch,] tokens, heads, dim; either may be None) rotated by their positions, as (q, k). out: the pair
    of outputs (the inputs themselves: in place)."""
    return _rope(q, k, positions, turns, layout, scale, out, stream, 0)


def rope_backward(dq, dk, positions, turns, *, layout: str = "half", scale: float = 1.0, out=None, stream=None):
    """The gradients of rope's inputs from those of its outputs."""
    return _rope(dq, dk, positions, turns, layout, scale, out, stream, 1)


# ---- append ------------------------------------------------------------------------------------------------------

def cache_append(k, v, k_cache, v_cache, tables, positions, *, rows=None, q=None, q_out=None, turns=None,
                 layout: str = "half", scale: float = 1.0, status=None, stream=None):
    """Store each token's key, rotated where turns is given, and value in its page; returns q rotated (None without
    q). rows: each token's table row (None: token t has row t)."""
    s = _Stream(stream, k)
    if q is not None and q_out is None:
        q_out = s.empty(q.shape, q.dtype)
    args = _append_args.pack(*_operand(k, "k"), *_operand(v, "v"), *_operand(k_cache, "k_cache"),
                             *_operand(v_cache, "v_cache"), *_operand(tables, "tables"),
                             *_operand(positions, "positions"), *_optional(rows, "rows"), *_optional(q, "q"),
                             *(_ABSENT if q is None else _operand(q_out, "q_out")), *_spec(turns, layout, scale, 0),
                             _status(status))
    _check(_call("cmd_cache_append")(args, s.handle), "cmd_cache_append")
    return None if q is None else q_out


# ---- attention ---------------------------------------------------------------------------------------------------

def cmd_attention_workspace(q_heads: int, kv_heads: int, dim: int) -> int:
    n = _I64()
    _check(_call("cmd_attention_workspace")(q_heads, kv_heads, dim, ctypes.byref(n)), "cmd_attention_workspace")
    return n.value


def attention_decode(q, k_cache, v_cache, tables, lengths, *, scale: float | None = None, softcap: float = 0.0,
                     window: int = 0, out=None, lse=None, return_lse: bool = False, workspace=None, status=None,
                     stream=None):
    """Attention of one new token per row: q [rows, q_heads, dim] over the first lengths[r] tokens of row r. Returns
    out, or (out, lse) with return_lse. scale: dim ** -0.5 unless given. workspace: cmd_attention_workspace bytes
    (allocated where None)."""
    s = _Stream(stream, q)
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q has rank 3 and the caches have rank 4")
    rows, heads, dim = q.shape
    if out is None:
        out = s.empty((rows, heads, dim), q.dtype)
    if return_lse and lse is None:
        import torch
        lse = s.empty((rows, heads), torch.float32)
    kv = k_cache.shape[2]
    n = cmd_attention_workspace(heads, kv, dim) if rows and heads and kv and heads % kv == 0 else 0
    if workspace is None and n:
        import torch
        workspace = s.empty(n, torch.uint8)
    w = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    args = _attention_args.pack(*_operand(q, "q"), *_operand(out, "out"), *_optional(lse, "lse"),
                                *_operand(k_cache, "k_cache"), *_operand(v_cache, "v_cache"),
                                *_operand(tables, "tables"), *_operand(lengths, "lengths"),
                                1.0 / math.sqrt(dim) if scale is None and dim else scale or 1.0, softcap, window, 0,
                                *w, _status(status))
    _check(_call("cmd_attention_decode")(args, s.handle), "cmd_attention_decode")
    return (out, lse) if return_lse else out


# ---- pages -------------------------------------------------------------------------------------------------------

def _pools(pools, pages):
    """The pools as cmd_pool records (kept alive by the caller)."""
    rec = []
    for i, t in enumerate(pools):
        if not t.is_cuda:
            raise ValueError(f"pool {i} is not on a GPU")
        if t.dim() < 1 or t.shape[0] != pages:
            raise ValueError(f"pool {i} does not have {pages} pages in its first dim")
        es = t.element_size()
        block = t.numel() // pages if pages else 0
        stride = t.stride(0)
        if not t.is_contiguous():  # a page's elements must be dense, in any order
            reach = 1
            for st, n in sorted((st, n) for n, st in zip(t.shape[1:], t.stride()[1:]) if n != 1):
                if st != reach:
                    raise ValueError(f"a page of pool {i} is not dense")
                reach *= n
        if pages == 1:
            stride = max(stride, block)
        rec += [t.data_ptr(), block * es, stride * es]
    return struct.pack(f"@{len(rec)}q", *rec)


def cache_select(tables, lengths, refs, parents, pools, *, page_size: int, grow=None, out=None, status=None,
                 stream=None):
    """New row i goes on from row parents[i] (-1: an empty row) with room for grow[i] more tokens; pages in progress
    are copied in every pool for later children. Returns (tables, lengths, refs); out: those three, to write to."""
    import torch
    s = _Stream(stream, tables)
    pages = refs.shape[0]
    if out is None:
        rows = parents.shape[0]
        out = tuple(s.empty(n, torch.int32) for n in ((rows, tables.shape[1]), (rows,), (pages,)))
    n = _I64()
    _check(_call("cmd_select_workspace")(tables.shape[0], parents.shape[0], pages, ctypes.byref(n)), "cmd_select_workspace")
    w = s.empty(n.value, torch.uint8)
    rec = _pools(pools, pages)
    args = _select_args.pack(*_operand(tables, "tables"), *_operand(lengths, "lengths"), *_operand(refs, "refs"),
                             *_operand(parents, "parents"), *_optional(grow, "grow"), *_operand(out[0], "tables_out"),
                             *_operand(out[1], "lengths_out"), *_operand(out[2], "refs_out"), _address(rec), len(pools),
                             page_size, w.data_ptr(), n.value, _status(status))
    _check(_call("cmd_cache_select")(args, s.handle), "cmd_cache_select")
    return out


def cache_compact(tables, lengths, refs, pools, *, page_size: int, out=None, status=None, stream=None):
    """The pages in use moved to the front of every pool. Returns (tables, refs, page_map); out: those three."""
    import torch
    s = _Stream(stream, tables)
    pages = refs.shape[0]
    if out is None:
        out = s.empty(tables.shape, torch.int32), s.empty((pages,), torch.int32), s.empty((pages,), torch.int32)
    n = _I64()
    _check(_call("cmd_compact_workspace")(pages, ctypes.byref(n)), "cmd_compact_workspace")
    w = s.empty(n.value, torch.uint8)
    rec = _pools(pools, pages)
    args = _compact_args.pack(*_operand(tables, "tables"), *_operand(lengths, "lengths"), *_operand(refs, "refs"),
                              *_operand(out[0], "tables_out"), *_operand(out[1], "refs_out"),
                              *_operand(out[2], "page_map_out"), _address(rec), len(pools), page_size, w.data_ptr(),
                              n.value, _status(status))
    _check(_call("cmd_cache_compact")(args, s.handle), "cmd_cache_compact")
    return out


def _address(rec):
    """The address of a bytes object's contents, while it lives."""
    return ctypes.cast(ctypes.c_char_p(rec), _P).value or 0


def cache_status(status, stream=None) -> None:
    """Wait for the stream and raise CmdError if an operator given this status word met an invalid table, index or a
    lack of room; the word is cleared."""
    s = _Stream(stream, status)
    bits = _I32()
    _check(_call("cmd_cache_status")(_status(status), ctypes.byref(bits), s.handle), "cmd_cache_status")
