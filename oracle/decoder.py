"""CPU oracle of the decoder operators beside the linear layer: numpy, fp64
(and IEEE fp32 where the definition itself is fp32).  TEST INFRASTRUCTURE ONLY,
like the rest of this package; written from the formulas in include/tern.h and
sharing no code with the CUDA library.

Parity status: pinned by tests/test_oracle_decoder.py (closed forms, brute
force on tiny inputs, invariants).
"""
from __future__ import annotations

import numpy as np

BLOCK = 64


def add_rmsnorm(x, residual, weight, eps, round_residual):
    """(r, y, x_scale, y / x_scale) of token rows in fp64.

    x, residual, weight: arrays of the stored values; round_residual maps the
    fp32 sum to the residual's type's values (or None: r = x)."""
    if residual is None:
        r = np.asarray(x, dtype=np.float64)
    else:
        s = np.asarray(x, dtype=np.float32) + np.asarray(residual, dtype=np.float32)
        r = np.asarray(round_residual(s), dtype=np.float64)
    w = np.asarray(weight, dtype=np.float64)
    y = r * w / np.sqrt((r * r).mean(axis=1, keepdims=True) + eps)
    scale = np.abs(y).max(axis=1) / 127
    with np.errstate(invalid="ignore", divide="ignore"):
        ratio = np.where(scale[:, None] > 0, y / scale[:, None], 0.0)
    return r, y, scale, ratio


def kv8_append(codes, scales, page_table, row_start, seq_lens, k, v):
    """The cache after the append: (codes, scales), new arrays.  fp32 IEEE
    arithmetic, which the definition names: the result is exact."""
    codes, scales = codes.copy(), scales.copy()
    f = np.float32
    for b, n in enumerate(seq_lens):
        r0, m = int(row_start[b]), int(row_start[b + 1] - row_start[b])
        done = n - m
        while done < n:
            j, off = divmod(int(done), BLOCK)
            take = int(min(BLOCK - off, n - done))
            page = int(page_table[b, j])
            for which, src in enumerate((k, v)):
                for h in range(codes.shape[2]):
                    x = np.asarray(src[r0 + done - (n - m):r0 + done - (n - m) + take, h],
                                   dtype=f)
                    big = np.abs(x).max()
                    fresh = f(big) / f(127) if np.isfinite(x).all() else f(np.nan)
                    old = scales[page, which, h] if off else f(0)
                    if np.isnan(old) or np.isnan(fresh):
                        s = f(np.nan)
                    else:
                        s = max(old, fresh)
                    c = codes[page, which, h]
                    if off and s > old:
                        c[:off] = np.rint(c[:off].astype(f) * (old / s)).astype(np.int8)
                    if s > 0:
                        c[off:off + take] = np.clip(np.rint(x / s), -127, 127).astype(np.int8)
                    elif not np.isnan(s):
                        c[off:off + take] = 0
                    scales[page, which, h] = s
            done += take
    return codes, scales


def visible(p, n, window, sinks):
    """Truth values over tokens 0..n-1: what the row at position p sees."""
    j = np.arange(n)
    ok = j <= p
    if window > 0:
        ok &= (j > p - window) | (j < sinks)
    return ok


def kv8_attention(q, codes, scales, page_table, row_start, seq_lens, window, sinks, scale):
    """(out, lse, sum_j p_j |v_j|) in fp64; rows outside every sequence are 0.

    A page number outside the pool masks its tokens."""
    rows, heads, dim = q.shape
    hkv = codes.shape[2]
    group = heads // hkv
    out = np.zeros((rows, heads, dim))
    absum = np.zeros((rows, heads, dim))
    lse = np.full((rows, heads), -np.inf)
    for b, n in enumerate(seq_lens):
        n = int(n)
        r0, m = int(row_start[b]), int(row_start[b + 1] - row_start[b])
        if m == 0:
            continue
        used = page_table[b, :(n + BLOCK - 1) // BLOCK]
        good = (used >= 0) & (used < codes.shape[0])
        at = np.where(good, used, 0)
        there = np.repeat(good, BLOCK)[:n]
        for h in range(hkv):
            c = codes[at][:, :, h].astype(np.float64)
            s = scales[at][:, :, h].astype(np.float64)
            kv = c * s[:, :, None, None]
            kk = kv[:, 0].reshape(-1, dim)[:n]
            vv = kv[:, 1].reshape(-1, dim)[:n]
            for i in range(m):
                see = visible(n - m + i, n, window, sinks) & there
                if not see.any():
                    continue
                for g in range(h * group, (h + 1) * group):
                    z = scale * (kk[see] @ q[r0 + i, g].astype(np.float64))
                    big = z.max()
                    p = np.exp(z - big)
                    lse[r0 + i, g] = big + np.log(p.sum())
                    p /= p.sum()
                    out[r0 + i, g] = p @ vv[see]
                    absum[r0 + i, g] = p @ np.abs(vv[see])
    return out, lse, absum
