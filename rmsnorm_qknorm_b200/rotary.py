"""Frequencies of rotary positions, plain or scaled for longer contexts.

Pair i of r / 2 turns by ``base ** (-2 i / r)`` radians per position.  A model
trained to ``original`` positions reaches ``factor`` times as far with

* ``"linear"``: every frequency divided by the factor (positions interpolated);
* ``"ntk"``: the base raised to ``base * factor ** (r / (r - 2))``, which leaves
  the fastest pair as it is and divides the slowest one by the factor;
* ``"yarn"``: pairs that turn more than ``fast`` times over the original length
  keep their frequency, pairs that turn less than ``slow`` times are divided by
  the factor, a linear ramp between them; cos and sin are multiplied by
  ``0.1 ln(factor) + 1``.

Any other scheme is a tensor of frequencies of the caller's own.
"""
from __future__ import annotations

import math

import torch

__all__ = ["rotary_inv_freq"]


def rotary_inv_freq(rotary_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                    original: int | None = None, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """``(inv_freq, mscale)`` for the rotary calls: float64 [rotary_dim / 2] and a float.

    Made once per model (and again when a call needs another ``factor``).
    """
    r = int(rotary_dim)
    if r < 2 or r % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    if not base > 1.0 or not math.isfinite(base):
        raise ValueError("base must be finite and greater than 1")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if not factor >= 1.0 or not math.isfinite(factor):
        raise ValueError("factor must be finite and at least 1")
    if scaling == "ntk":
        if r == 2:
            raise ValueError("ntk scaling needs rotary_dim of at least 4")
        base = base * factor ** (r / (r - 2))
    inv = base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    mscale = 1.0
    if scaling == "linear":
        inv = inv / factor
    elif scaling == "yarn":
        if original is None or original < 1:
            raise ValueError("yarn scaling needs the original length")
        if not fast > slow > 0:
            raise ValueError("yarn scaling needs fast > slow > 0")
        if original < slow * 2 * math.pi:
            raise ValueError("yarn scaling needs an original length over which the fastest pair turns `slow` times")
        # the (fractional) pair that turns n times over the original length
        low, high = (r * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (fast, slow))
        low, high = max(math.floor(low), 0), min(math.ceil(high), r - 1)
        ramp = ((torch.arange(r // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
        inv = inv / factor * ramp + inv * (1 - ramp)
        mscale = 0.1 * math.log(factor) + 1.0
    return inv.to(device), mscale
