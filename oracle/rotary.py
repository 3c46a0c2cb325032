"""Rotary positions in float64 (TEST INFRASTRUCTURE ONLY, see the package docstring).

Pair i of the first rot_dim elements of a head turns by theta = t f_i at position t (Su et al.,
"RoFormer"): (a, b) -> A (a cos - b sin, b cos + a sin).  Pairs are (i, i + rot_dim / 2) in the half
layout and (2i, 2i + 1) in the interleaved one.  f_i = base^(-2i / rot_dim), divided by a factor
(linear), or by parts (Peng et al., "YaRN"): a pair that makes r turns over the trained context
keeps its frequency from r = beta_fast on, is divided up to r = beta_slow, with a ramp between,
and A = 0.1 ln(factor) + 1.
"""
from __future__ import annotations

import math

import numpy as np

HALF, INTERLEAVED = 0, 1
PLAIN, LINEAR, BY_PARTS = 0, 1, 2


def frequencies(rot_dim, base, scaling=PLAIN, factor=1.0, orig_ctx=0, beta_fast=32.0,
                beta_slow=1.0):
    """(f [rot_dim / 2], amplitude)."""
    f = base ** (-2.0 * np.arange(rot_dim // 2, dtype=np.float64) / rot_dim)
    if scaling == LINEAR:
        return f / factor, 1.0
    if scaling == BY_PARTS:
        turns = orig_ctx * f / (2 * math.pi)
        g = np.clip((turns - beta_slow) / (beta_fast - beta_slow), 0.0, 1.0)
        return f * (g + (1 - g) / factor), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rotate(x, pos, f, amplitude=1.0, layout=HALF):
    """x [rows, heads, D] turned by pos [rows]."""
    x = np.asarray(x, np.float64)
    n = len(f)
    th = np.asarray(pos, np.float64)[:, None, None] * f
    c, s = amplitude * np.cos(th), amplitude * np.sin(th)
    out = x.copy()
    ia = np.arange(n) if layout == HALF else 2 * np.arange(n)
    ib = ia + (n if layout == HALF else 1)
    a, b = x[..., ia], x[..., ib]
    out[..., ia] = a * c - b * s
    out[..., ib] = b * c + a * s
    return out
