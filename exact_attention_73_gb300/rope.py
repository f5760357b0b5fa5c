"""Frequencies of rotary positions, with the usual scalings for long contexts.

``inv_freq`` gives the float64 frequencies that ``attn_rope_tables`` turns into
its float32 tables. A few dozen numbers, computed once per model on the host;
the tables and the rotation are the library's kernels.
"""
from __future__ import annotations

import math

import torch


def inv_freq(rot_dim, base=10000.0, scaling=None, factor=1.0, trained=None, fast=32.0, slow=1.0):
    """base^(-2i/rot_dim), i < rot_dim/2, as a float64 CPU tensor [rot_dim/2].

    scaling (``factor``: the new context length over the trained one):
      None       no change;
      "linear"   every frequency divided by factor (positions interpolated);
      "base"     base times factor^(rot_dim / (rot_dim - 2)): the slowest
                 frequency is divided by factor, the fastest kept;
      "parts"    by the turns a frequency makes over ``trained`` positions: at
                 least ``fast`` kept, at most ``slow`` divided by factor, in
                 between a linear mix.
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and positive, got {rot_dim}")
    if not factor > 0:
        raise ValueError(f"factor must be positive, got {factor}")
    if scaling == "base" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = float(base) ** (-2.0 * torch.arange(rot_dim // 2, dtype=torch.float64) / rot_dim)
    if scaling in (None, "base"):
        return f
    if scaling == "linear":
        return f / factor
    if scaling == "parts":
        if trained is None or not fast > slow:
            raise ValueError('scaling "parts" needs the trained length, and fast > slow')
        keep = ((trained * f / (2.0 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        return f * keep + f / factor * (1.0 - keep)
    raise ValueError(f"unknown scaling {scaling!r}")
