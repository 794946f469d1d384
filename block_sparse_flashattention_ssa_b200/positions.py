"""Positions and frequencies for ``rotary``: small host-side tables.

``grid_positions`` numbers the tokens of packed video sequences (frame, row,
column; row-major, column fastest); ``frequencies`` gives each pair's radians
per position, with the usual ways to serve sequences longer than the ones a
model was trained on. Frequencies are float64: the kernel forms angles in
double, so far positions keep their phase.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence, Tuple

METHODS = ("linear", "base", "by_parts")


def sections(pairs: int, axes: int) -> Tuple[int, ...]:
    """Pairs per axis: the axes after the first get pairs // axes each, the
    first (frames) what is left."""
    if pairs < 0 or axes < 1:
        raise ValueError("pairs must be >= 0 and axes >= 1")
    rest = pairs // axes
    return (pairs - rest * (axes - 1),) + (rest,) * (axes - 1)


def grid_positions(grids: Sequence[Tuple[int, int, int]], device=None):
    """int32 [total_tokens, 3]: frame, row and column of every token of packed
    sequences of ``grids`` = (frames, rows, columns) tokens."""
    import torch

    parts = []
    for t, h, w in grids:
        if min(t, h, w) < 0:
            raise ValueError("grid sizes must be >= 0")
        i = torch.arange(t * h * w, dtype=torch.int32, device=device)
        hw, w1 = max(h * w, 1), max(w, 1)
        parts.append(torch.stack([i // hw, i % hw // w1, i % w1], 1))
    if not parts:
        return torch.empty((0, 3), dtype=torch.int32, device=device)
    return torch.cat(parts)


def frequencies(pairs_per_axis: Sequence[int], base: float = 10000.0, stretch: float = 1.0, method: str = "linear",
                original_length: Optional[int] = None, turns: Tuple[float, float] = (1.0, 32.0), device=None):
    """(inv_freq float64 [sum of pairs], scale) for ``rotary``. Pair i of an
    axis with n pairs turns base^(-i / n) radians per position. ``stretch`` > 1
    serves sequences that many times longer:
      linear    every frequency is divided by it;
      base      the base is raised to base * stretch^(n / (n - 1)): the fastest
                pair keeps its frequency, the slowest is divided by stretch;
      by_parts  pairs that turn more than ``turns[1]`` times over
                ``original_length`` positions keep their frequency, those below
                ``turns[0]`` turns are divided by stretch, with a linear ramp
                between; scale = 0.1 ln(stretch) + 1 (else it is 1)."""
    import torch

    if method not in METHODS:
        raise ValueError(f"method must be one of {METHODS}")
    if not (base > 1.0 and math.isfinite(base)) or not (stretch >= 1.0 and math.isfinite(stretch)):
        raise ValueError("base must be > 1 and stretch >= 1")
    if method == "by_parts" and (not original_length or original_length < 1 or not turns[1] > turns[0]):
        raise ValueError("by_parts needs original_length >= 1 and turns[1] > turns[0]")
    out = []
    for n in pairs_per_axis:
        if n < 0:
            raise ValueError("pairs must be >= 0")
        b = base
        if method == "base" and n > 1:
            b = base * stretch ** (n / (n - 1))
        f = b ** (-torch.arange(n, dtype=torch.float64) / max(n, 1))
        if method == "linear":
            f = f / stretch
        elif method == "by_parts":
            keep = ((original_length * f / (2 * math.pi) - turns[0]) / (turns[1] - turns[0])).clamp(0.0, 1.0)
            f = f * keep + f / stretch * (1 - keep)
        out.append(f)
    inv = torch.cat(out) if out else torch.empty(0, dtype=torch.float64)
    return inv.to(device), (0.1 * math.log(stretch) + 1.0 if method == "by_parts" and stretch > 1.0 else 1.0)
