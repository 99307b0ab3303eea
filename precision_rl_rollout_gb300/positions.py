"""Frequencies of rotary positions for ``binding.fp8rl_rope_table``, plain and scaled
to contexts longer than the trained one.  Pure arithmetic in 64 bits; the table
itself is made on the GPU.

Pair i of R/2 turns by ``base ** (-2 i / R)`` radians a position.  To reach
``factor`` times the trained context:

- ``linear``: every frequency divided by the factor;
- ``base``: the base raised so that the slowest pair turns ``factor`` times slower
  and the fastest keeps its frequency;
- ``bands``: pairs that make more than ``fast`` turns within the trained context
  keep their frequency, pairs that make fewer than ``slow`` are divided by the
  factor, those between are blended linearly in their number of turns; cosines and
  sines are multiplied by ``0.1 ln(factor) + 1``, which sharpens the attention over
  the longer context.
"""
from __future__ import annotations

import math


def rope_frequencies(R: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     trained: int = 0, slow: float = 1.0, fast: float = 32.0):
    """-> (R/2 frequencies in radians a position, magnitude)."""
    if R <= 0 or R % 2:
        raise ValueError("R must be a positive even number")
    if base <= 0 or factor < 1:
        raise ValueError("base must be positive and factor at least 1")
    if scaling not in (None, "linear", "base", "bands"):
        raise ValueError(f"scaling {scaling!r}: linear, base, bands or None")
    if scaling == "base" and R > 2:
        base *= factor ** (R / (R - 2))
    freq = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if scaling == "linear":
        return [f / factor for f in freq], 1.0
    if scaling == "bands":
        if trained <= 0 or not 0 <= slow < fast:
            raise ValueError("bands need the trained context and 0 <= slow < fast")
        keep = [min(max((trained * f / (2 * math.pi) - slow) / (fast - slow), 0.0), 1.0) for f in freq]
        return [f * (k + (1 - k) / factor) for f, k in zip(freq, keep)], 0.1 * math.log(factor) + 1.0
    return freq, 1.0
