"""Pins of oracle/attention_block.py (CPU)."""
import math

import numpy as np
import pytest

import ternary_weight_linear_gb300 as tl
from oracle import attention_block as ab

SCALINGS = [("none", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
            ("bands", dict(factor=8.0, trained=8192.0, low=1.0, high=4.0)),
            ("ramp", dict(factor=4.0, trained=4096.0, low=1.0, high=32.0))]


def test_frequencies_closed_forms():
    theta, m = ab.frequencies(64, 1e4)
    assert m == 1 and theta[0] == 1 and math.isclose(theta[16], 0.01)
    assert np.allclose(ab.frequencies(64, 1e4, "linear", 4.0)[0], theta / 4, rtol=1e-15)
    # the slowest pair of the larger base is slowed by just the factor, the fastest not
    base, _ = ab.frequencies(64, 1e4, "base", 8.0)
    assert base[0] == 1 and math.isclose(base[31], theta[31] / 8, rel_tol=1e-12)
    bands, _ = ab.frequencies(64, 1e4, "bands", 8.0, 8192, 1, 4)
    turns = 8192 * theta / (2 * math.pi)
    assert np.array_equal(bands[turns >= 4], theta[turns >= 4])
    assert np.allclose(bands[turns <= 1], theta[turns <= 1] / 8, rtol=1e-15)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and np.all((bands[mid] < theta[mid]) & (bands[mid] > theta[mid] / 8))
    ramp, m = ab.frequencies(64, 1e4, "ramp", 4.0, 4096, 1, 32)
    assert math.isclose(m, 0.1 * math.log(4) + 1)
    assert np.array_equal(ramp[:4], theta[:4]) and np.allclose(ramp[-2:], theta[-2:] / 4)
    assert np.all(np.diff(ramp / theta) <= 1e-15)


def test_rotation_closed_forms():
    quarter = 2 ** 62
    freq = [quarter] * 8  # a quarter turn a token
    x = np.arange(1.0, 33).reshape(1, 1, 32)
    out, size = ab.rope(x, [1], freq, False, 1.0)
    assert np.allclose(out[0, 0, :8], -x[0, 0, 8:16]) and np.allclose(out[0, 0, 8:16], x[0, 0, :8])
    assert np.array_equal(out[..., 16:], x[..., 16:]) and not size[..., 16:].any()
    out, _ = ab.rope(x, [1], freq, True, 2.0)
    assert np.allclose(out[0, 0, 0:16:2], -2 * x[0, 0, 1:16:2])
    assert np.allclose(out[0, 0, 1:16:2], 2 * x[0, 0, 0:16:2])
    # whole turns, and back again
    assert np.allclose(ab.rope(x, [4 * 10 ** 6], freq, False, 1.0)[0], x, atol=1e-12)
    theta, _ = ab.frequencies(32, 1e4)
    turns = [int(t / (2 * math.pi) * 2 ** 64) for t in theta]
    there, _ = ab.rope(x, [123457], turns, True, 1.0)
    assert np.allclose(ab.rope(there, [-123457], turns, True, 1.0)[0], x, atol=1e-12)
    assert np.allclose(np.linalg.norm(there), np.linalg.norm(x))


def test_rotation_depends_on_distances_alone():
    rng = np.random.default_rng(0)
    theta, _ = ab.frequencies(64, 1e4)
    turns = [int(t / (2 * math.pi) * 2 ** 64) for t in theta]
    q, k = rng.standard_normal((2, 1, 1, 64))
    dots = [np.sum(ab.rope(q, [p + 7], turns, False, 1.0)[0] * ab.rope(k, [p], turns, False, 1.0)[0])
            for p in (0, 5, 900000)]
    assert np.allclose(dots, dots[0], rtol=1e-9)


def test_norms_closed_forms():
    x = np.array([[3.0, 4.0, 0, 0]])
    res = np.array([[1.0, 1, 1, 1]])
    r, mag = ab.norm_add_norm(x, np.ones(4), None, 2.0, res, 0.5, 0.0)
    assert np.allclose(r, 0.5 + 2 * x / 2.5) and np.allclose(mag, r)
    r, _ = ab.norm_add_norm(x, None, np.array([1.0, 0, 0, 0]), 1.0, res, 1.0, 0.0)
    assert np.allclose(r, [[4, 1, 1, 1]])
    y, s, ratio = ab.norm(np.array([[1.0, -1, 1, 1], [0, 0, 0, 0]]), np.array([1.0, 2, 1, 1]), 0.0 + 1e-30)
    assert np.allclose(y[0], [1, -2, 1, 1]) and np.allclose(s, [2 / 127, 0])
    assert np.allclose(ratio[0], [63.5, -127, 63.5, 63.5]) and not ratio[1].any()


# ------------------------------------------------- the library's host function

@pytest.fixture(scope="module", autouse=True)
def built():
    tl.build()
    tl.load()


@pytest.mark.parametrize("rotary", [16, 64, 128, 1024])
@pytest.mark.parametrize("base", [1.5, 1e4, 1e6])
@pytest.mark.parametrize("scaling,args", SCALINGS)
def test_library_frequencies(rotary, base, scaling, args):
    freq, m = tl.tern_rope_frequencies(rotary, base=base, scaling=scaling, device="cpu", **args)
    theta, want_m = ab.frequencies(rotary, base, scaling, **args)
    assert freq.dtype.itemsize == 8 and freq.shape == (rotary // 2,)
    assert m == np.float32(want_m)
    got = np.array([int(f) % 2 ** 64 for f in freq.tolist()], dtype=np.float64)
    want = theta / (2 * math.pi) * 2.0 ** 64
    # a dozen roundings of 2^-53, some of a logarithm times 1024
    assert np.all(np.abs(got - want) <= 2.0 ** -40 * want + 1)


def test_library_frequencies_refusals():
    f = lambda *a, **k: tl.tern_rope_frequencies(*a, device="cpu", **k)  # noqa: E731
    bad = [dict(rotary_dim=0), dict(rotary_dim=8), dict(rotary_dim=24), dict(rotary_dim=1040),
           dict(rotary_dim=-16), dict(rotary_dim=64, base=1.0), dict(rotary_dim=64, base=float("nan")),
           dict(rotary_dim=64, base=float("inf")),
           dict(rotary_dim=64, scaling="linear", factor=0.5),
           dict(rotary_dim=64, scaling="base", factor=float("inf")),
           dict(rotary_dim=64, scaling="bands", factor=2.0),
           dict(rotary_dim=64, scaling="ramp", factor=2.0, trained=4096, low=4.0, high=2.0),
           dict(rotary_dim=64, scaling="ramp", factor=2.0, trained=-1.0)]
    for args in bad:
        with pytest.raises(tl.TernError):
            f(**args)
    with pytest.raises(ValueError):
        f(64, scaling="cubic")
