"""Frequencies scaled by parts, from how often each pair turns over the original length; no GPU."""
from __future__ import annotations

import math
from decimal import ROUND_CEILING, ROUND_FLOOR, Decimal, getcontext

import pytest

import tensor_command_execution_gb300 as T
from tensor_command_execution_gb300 import cache as C

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
PARTS = 3


def _by_parts(n, base, factor, length, fast, slow):
    """Turns of each pair in 60 digits. Pair x makes length * base^(-x / n) / (2 pi) turns; the ramp runs from the index
    that makes `fast` of them, rounded down and at least 0, to that which makes `slow`, rounded up and at most the
    rotated elements less one, 2 n - 1."""
    base, length, factor = Decimal(base), Decimal(length), Decimal(factor)

    def index(beta):
        return n * (length / (Decimal(beta) * 2 * PI)).ln() / base.ln()
    lo = max(index(fast).to_integral_value(ROUND_FLOOR), Decimal(0))
    hi = min(index(slow).to_integral_value(ROUND_CEILING), Decimal(2 * n - 1))
    out = []
    for i in range(n):
        ramp = Decimal(i > lo) if hi <= lo else min(max((i - lo) / (hi - lo), Decimal(0)), Decimal(1))
        f = (-(base.ln() * i / n)).exp()
        out.append((f * (1 - ramp) + f / factor * ramp) / (2 * PI) * 2 ** 64)
    return out


@pytest.mark.parametrize("n,base,factor,length,fast,slow", [
    (64, 1e4, 16.0, 4096.0, 32.0, 1.0),      # the ramp lies within the pairs
    (64, 1e4, 8.0, 131072.0, 32.0, 1.0),     # ends past the last pair (which makes 2.4 turns)
    (64, 1e4, 4.0, 262144.0, 32.0, 1.0), (48, 5e5, 40.0, 8e6, 16.0, 0.5),
    (64, 1e4, 8.0, 3e6, 32.0, 1.0),          # begins past it: nothing is scaled
    (16, 100.0, 4.0, 131072.0, 64.0, 2.0),   # ends past the rotated elements
    (64, 1e4, 8.0, 100.0, 32.0, 1.0),        # begins before the first
    (5, 2.5, 2.0, 40.0, 4.0, 1.0),
])
def test_turns_by_parts_wherever_the_ramp_lies(n, base, factor, length, fast, slow):
    got = C.cmd_rope_turns(n, base, PARTS, factor, length, fast, slow)
    for i, (g, w) in enumerate(zip(got, _by_parts(n, base, factor, length, fast, slow))):
        # binary64: a power, two divisions, the ramp and two products, a few 2^-53 each, and the integer's rounding
        assert abs(Decimal(g) - w) <= w * Decimal(2) ** -48 + 1, (i, g, w)


def test_every_pair_goes_by_its_own_number_of_turns():
    """Pairs that make beta_fast turns and more are kept, those that make beta_slow and fewer divided by the factor, those
    between neither."""
    n, base, factor, length, fast, slow = 64, 1e4, 8.0, 131072.0, 32.0, 1.0
    plain = C.cmd_rope_turns(n, base, 0, 0, 0, 0, 0)
    got = C.cmd_rope_turns(n, base, PARTS, factor, length, fast, slow)
    for i in range(n):
        turns, part = length * base ** (-i / n) / (2 * math.pi), got[i] / plain[i]
        assert part == 1.0 if turns >= fast else abs(part - 1 / factor) < 1e-12 if turns <= slow else 1 / factor < part <= 1.0, i
    assert got[-1] / plain[-1] == pytest.approx(0.28 + 0.72 / factor, abs=1e-9)  # (18 of the ramp's 25 steps)


def test_a_base_of_one_has_no_parts():
    """With base 1 every index turns alike: the ramp has no place."""
    assert len(C.cmd_rope_turns(1, 1.0, 0, 0, 0, 0, 0)) == 1
    for length in (1.0, 4096.0):
        with pytest.raises(T.CmdError, match="base") as e:
            C.cmd_rope_turns(1, 1.0, PARTS, 2.0, length, 32.0, 1.0)
        assert e.value.name == "CMD_ERR_ARG"
    assert C.cmd_rope_turns(0, 1.0, PARTS, 2.0, 1.0, 32.0, 1.0) == []
