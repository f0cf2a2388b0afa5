"""What repeated growth of a block's scale costs the codes already in it, on the
append's definition (oracle/decoder.py; the kernel is pinned to it bit for bit).

A token's code is rounded when it is written and at every growth after that, each
time by at most half a step of the scale then reached: its error is at most half
the sum of those scales.
"""
import numpy as np
import pytest

from oracle import decoder as od


def _appended(x, at_once):
    """Codes and scale of one block of x [64, dim], and the scale after each token."""
    n, dim = x.shape
    x = x[:, None]
    codes, scales = np.zeros((1, 2, 1, 64, dim), np.int8), np.zeros((1, 2, 1), np.float32)
    table, seen = np.zeros((1, 1), np.int32), []
    for i in range(0, n, at_once):
        codes, scales = od.kv8_append(codes, scales, table, np.array([0, at_once]),
                                      np.array([i + at_once]), x[i:i + at_once],
                                      x[i:i + at_once])
        seen.append(float(scales[0, 0, 0]))
    return codes[0, 0, 0].astype(np.float64) * seen[-1], seen


def _block(seed, grow):
    rng = np.random.default_rng(seed)
    by = grow ** (np.arange(64) / 63.0)
    return (rng.standard_normal((64, 128)) * by[:, None]).astype(np.float32)


@pytest.mark.parametrize("grow", [1, 4, 100])
@pytest.mark.parametrize("seed", range(5))
def test_error_is_at_most_half_the_scales_that_a_code_has_had(seed, grow):
    x = _block(seed, grow)
    got, seen = _appended(x, 1)
    for i in range(64):
        had = [seen[i]] + [b for a, b in zip(seen[i:], seen[i + 1:]) if b > a]
        # (2^-20: the quotients' and the products' own fp32 roundings)
        assert np.abs(got[i] - x[i]).max() <= 0.5 * sum(had) * (1 + 2.0 ** -20)


@pytest.mark.parametrize("grow,lo,hi", [(1, 1.3, 2.0), (4, 2.0, 3.0)])
def test_size_beside_codes_rounded_once(grow, lo, hi):
    """Root mean square error of the first sixteen of 64 tokens appended one by
    one, over that of the same tokens appended together: the header's figures."""
    ratio = []
    for seed in range(20):
        x = _block(seed, grow)
        one, all_ = (np.square(_appended(x, n)[0] - x)[:16].mean() for n in (1, 64))
        ratio.append((one / all_) ** 0.5)
    assert lo < np.mean(ratio) < hi
