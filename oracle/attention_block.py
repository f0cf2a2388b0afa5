"""CPU oracle of the attention block's operators around the projections, the
norm and the cache: numpy, fp64 (and IEEE fp32 where the definition itself is
fp32).  TEST INFRASTRUCTURE ONLY, like the rest of this package; written from
the formulas in include/tern.h and sharing no code with the CUDA library.

Parity status: pinned by tests/test_oracle_attention_block.py (closed forms,
brute force, invariants).
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np


def frequencies(rotary, base, scaling="none", factor=1.0, trained=0.0, low=1.0, high=4.0):
    """(theta [rotary / 2] in radians a token, magnitude)."""
    magnitude = 1.0
    if scaling == "base":
        base = base * factor ** (rotary / (rotary - 2))
    theta = np.array([base ** (-2 * i / rotary) for i in range(rotary // 2)])
    if scaling == "linear":
        theta = theta / factor
    elif scaling == "bands":
        turns = trained * theta / (2 * math.pi)
        s = np.clip((turns - low) / (high - low), 0, 1)
        theta = theta * (s + (1 - s) / factor)
    elif scaling == "ramp":
        def pair(turns):  # trained * base^(-2 i / rotary) = 2 pi turns
            return rotary / 2 * math.log(trained / (2 * math.pi * turns)) / math.log(base)
        a = max(math.floor(pair(high)), 0)
        b = min(math.ceil(pair(low)), rotary - 1)
        s = 1 - np.clip((np.arange(rotary // 2) - a) / max(b - a, 0.001), 0, 1)
        theta = theta * (s + (1 - s) / factor)
        magnitude = 0.1 * math.log(factor) + 1
    return theta, magnitude


def angles(freq, positions):
    """[len(positions), len(freq)] radians in [0, 2 pi): position * freq / 2^64
    turns, the product and its remainder exact (Python integers)."""
    return np.array([[float(Fraction((int(p) * int(f)) % 2 ** 64, 2 ** 64)) * 2 * math.pi
                      for f in freq] for p in positions]).reshape(len(positions), len(freq))


def rope(x, positions, freq, interleaved, magnitude):
    """(turned x in fp64, |u| + |v| of each element's pair, 0 where none turns)."""
    x = np.asarray(x, dtype=np.float64)
    rot = 2 * len(freq)
    a = angles(freq, positions)[:, None]
    c, s = np.cos(a) * magnitude, np.sin(a) * magnitude
    at = ((np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved
          else (np.arange(rot // 2), np.arange(rot // 2, rot)))
    out, size = x.copy(), np.zeros_like(x)
    u, v = x[..., at[0]], x[..., at[1]]
    out[..., at[0]] = u * c - v * s
    out[..., at[1]] = u * s + v * c
    size[..., at[0]] = size[..., at[1]] = np.abs(u) + np.abs(v)
    return out, size


def norm_add_norm(x, post, gate, branch_scale, residual, residual_scale, eps):
    """(r before its rounding, sum of its terms' magnitudes) in fp64."""
    n = np.asarray(x, dtype=np.float64)
    if post is not None:
        n = n * np.asarray(post, dtype=np.float64) / np.sqrt((n * n).mean(1, keepdims=True) + eps)
    if gate is not None:
        n = n * np.asarray(gate, dtype=np.float64)
    n = n * branch_scale
    res = residual_scale * np.asarray(residual, dtype=np.float64)
    return res + n, np.abs(res) + np.abs(n)


def norm(r, weight, eps):
    """(y, x_scale, y / x_scale) in fp64."""
    r, w = np.asarray(r, dtype=np.float64), np.asarray(weight, dtype=np.float64)
    y = r * w / np.sqrt((r * r).mean(axis=1, keepdims=True) + eps)
    scale = np.abs(y).max(axis=1) / 127
    with np.errstate(invalid="ignore", divide="ignore"):
        return y, scale, np.where(scale[:, None] > 0, y / scale[:, None], 0.0)
