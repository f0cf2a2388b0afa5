"""GPU parity of tern_norm_add_norm_s8 against the fp64 oracle.

Bars: the first norm's factor has a relative error below 2^-18 (the bound of
test_gpu_decoder.py's norm: a mean of at most 32768 fp32 squares, its root, and
a few roundings), and the branch's product four roundings more; r before its
rounding is so within 2^-17.9 < 2^-17 of its terms' magnitudes, and r itself is
the rounding of some value in that range.  What follows takes r as it was
stored, so x_scale, the codes and y are held to that test's bars on it.
"""
import numpy as np
import pytest

from oracle import attention_block as ab

pytestmark = pytest.mark.gpu

REL = 2.0 ** -18


@pytest.fixture(scope="module")
def tl():
    import torch
    import ternary_weight_linear_gb300 as tl
    tl.build()
    tl.load()
    torch.cuda.init()
    return tl


def _np(t):
    return t.double().cpu().numpy()


def _round(a, like):
    import torch
    return _np(torch.from_numpy(np.ascontiguousarray(a)).to(like.dtype))


def check(tl, T, K, xt="float32", rt="bfloat16", wt="bfloat16", post="bfloat16", gate=None,
          gate_rows=False, rs=1.0, bs=1.0, with_y=False, ld=None, in_place=False, scale=1.0, seed=0,
          x=None):
    import torch
    rng = np.random.default_rng([seed, T, K])
    up = lambda a, t: torch.from_numpy(a.astype(np.float32)).cuda().to(getattr(torch, t))  # noqa: E731
    if x is None:
        x = up(rng.standard_normal((T, ld or K)) * scale, xt)[:, :K]
    r0 = rng.standard_normal((T, K)) * scale
    r0[:, rng.integers(0, K, max(1, K // 100))] *= 20
    res = up(r0, rt)
    w = up(1 + 0.2 * rng.standard_normal(K), wt)
    p = up(1 + 0.2 * rng.standard_normal(K), post) if post else None
    g = None
    if gate:
        g = up(0.5 + rng.standard_normal((T, K) if gate_rows else K), gate)
    res64 = _np(res)
    y = torch.empty(T, K, dtype=torch.bfloat16, device="cuda") if with_y else None
    q, xs, r = tl.tern_norm_add_norm_s8(x, p, res, w, gate=g, residual_scale=rs, branch_scale=bs,
                                        eps=1e-6, y=y, residual_out=res if in_place else None)
    torch.cuda.synchronize()
    assert (r is res) == in_place
    f32 = lambda v: float(np.float32(v))  # noqa: E731
    want, mag = ab.norm_add_norm(_np(x), _np(p) if post else None, _np(g) if gate else None, f32(bs),
                                 res64, f32(rs), f32(1e-6))
    lo, hi = _round(want - 2.0 ** -17 * mag, res), _round(want + 2.0 ** -17 * mag, res)
    got = _np(r)
    assert np.all((got >= lo) & (got <= hi))
    y_ref, s_ref, ratio = ab.norm(got, _np(w), f32(1e-6))
    assert np.all(np.abs(_np(xs) - s_ref) <= REL * s_ref)
    c = _np(q)
    assert np.all(np.abs(c) <= 127)
    assert np.all(np.abs(c - ratio) <= 0.5 + 127 * 2.0 ** -17)
    assert np.all(np.abs(c).max(1)[s_ref > 0] == 127)
    if with_y:
        a, b = _round(y_ref * (1 - 2 * REL), y), _round(y_ref * (1 + 2 * REL), y)
        assert np.all((_np(y) >= np.minimum(a, b)) & (_np(y) <= np.maximum(a, b)))
    return q, xs, r, y


# one vector, an odd count of warps, the model's width, two and four vectors
@pytest.mark.parametrize("T,K", [(1, 16), (3, 272), (1, 5120), (37, 5120), (5, 9984), (2, 17408),
                                 (3, 32768)])
@pytest.mark.parametrize("gate", [None, "bfloat16"])
def test_widths(tl, T, K, gate):
    check(tl, T, K, gate=gate, rs=0.9, bs=1.25, with_y=True)


@pytest.mark.parametrize("xt", ["float32", "bfloat16"])
@pytest.mark.parametrize("rt", ["float32", "bfloat16"])
@pytest.mark.parametrize("wt", ["float32", "bfloat16"])
@pytest.mark.parametrize("post", [None, "float32", "bfloat16"])
def test_types(tl, xt, rt, wt, post):
    check(tl, 9, 1040, xt, rt, wt, post, gate=wt, gate_rows=True, rs=-0.5, bs=2.0, ld=1072,
          with_y=True, seed=3)


# two vectors a thread from 8208 on, four from 16400
@pytest.mark.parametrize("K", [8208, 16384, 16400, 30000])
@pytest.mark.parametrize("xt,rt,wt,post,gate", [
    ("float32", "float32", "float32", "bfloat16", None),
    ("bfloat16", "float32", "bfloat16", "bfloat16", "bfloat16"),
    ("float32", "bfloat16", "float32", None, "float32"),
    ("bfloat16", "bfloat16", "bfloat16", "float32", "float32")])
def test_types_of_long_rows_in_place(tl, K, xt, rt, wt, post, gate):
    check(tl, 3, K, xt, rt, wt, post, gate=gate, gate_rows=True, rs=0.9, bs=-1.25, with_y=True,
          in_place=True, seed=5)


def test_gates(tl):
    """A row for all tokens, rows of their own, expanded and strided ones."""
    import torch
    check(tl, 6, 256, gate="float32")
    check(tl, 6, 256, gate="float32", gate_rows=True)
    x = torch.randn(6, 256, device="cuda")
    res = torch.randn(6, 256, device="cuda").bfloat16()
    w = torch.ones(256, device="cuda")
    g = torch.randn(256, device="cuda")
    a = tl.tern_norm_add_norm_s8(x, w, res, w, gate=g)
    b = tl.tern_norm_add_norm_s8(x, w, res, w, gate=g.expand(6, 256))
    wide = torch.zeros(6, 512, device="cuda")
    wide[:, 256:] = g
    c = tl.tern_norm_add_norm_s8(x, w, res, w, gate=wide[:, 256:])
    for i in range(3):
        assert torch.equal(a[i], b[i]) and torch.equal(a[i], c[i])


def test_in_place_and_small_and_large_values(tl):
    check(tl, 4, 512, in_place=True)
    check(tl, 4, 512, rt="float32", scale=1e-12)
    check(tl, 4, 512, rt="float32", post=None, scale=1e12)


def test_without_the_first_norm_it_is_the_residual_norm(tl):
    """Scales of 1, no gate: r is tern_add_rmsnorm_s8's, bit for bit."""
    import torch
    x = torch.randn(5, 768, device="cuda")
    res = torch.randn(5, 768, device="cuda").bfloat16()
    w = (1 + torch.randn(768, device="cuda") / 5).bfloat16()
    a = tl.tern_norm_add_norm_s8(x, None, res, w)
    b = tl.tern_add_rmsnorm_s8(x, w, res)
    for i in range(3):
        assert torch.equal(a[i], b[i])


def test_zero_rows_and_scales(tl):
    import torch
    x = torch.zeros(3, 256, device="cuda")
    x[1] = 1.0
    res = torch.zeros(3, 256, device="cuda")
    res[2] = 2.0
    w = torch.ones(256, device="cuda")
    q, s, r = tl.tern_norm_add_norm_s8(x, w, res, w)
    assert s.tolist()[0] == 0 and not q[0].any() and not r[0].any()
    assert (q[1:] == 127).all() and (r[2] == 2).all()
    # a branch of scale 0 leaves the scaled residual
    q, s, r = tl.tern_norm_add_norm_s8(x, w, res, w, branch_scale=0.0, residual_scale=0.5)
    assert torch.equal(r, res * 0.5)


def test_not_finite_stays_in_its_row(tl):
    import torch
    x = torch.ones(3, 256, device="cuda")
    x[1, 7] = float("nan")
    res = torch.ones(3, 256, device="cuda")
    w = torch.ones(256, device="cuda")
    _, s, r = tl.tern_norm_add_norm_s8(x, w, res, w)
    assert torch.isnan(s[1]) and torch.isnan(r[1]).all()
    assert torch.isfinite(r[0]).all() and torch.isfinite(s[0]) and torch.isfinite(s[2])


def test_y_alone_and_refusals_of_the_binding(tl):
    import torch
    x = torch.randn(3, 256, device="cuda")
    w = torch.ones(256, device="cuda")
    y = torch.empty(3, 256, dtype=torch.bfloat16, device="cuda")
    q, s, r = tl.tern_norm_add_norm_s8(x, w, x, w, y=y, quantise=False)
    assert q is None and s is None
    y2 = torch.empty_like(y)
    tl.tern_norm_add_norm_s8(x, w, x, w, y=y2)
    assert torch.equal(y, y2)
    for bad in (dict(gate=w[:16]), dict(gate=torch.ones(2, 256, device="cuda")),
                dict(gate=w.half()), dict(post_weight=w.half()), dict(residual=x[:2]),
                dict(quantise=False), dict(gate=w.double())):
        args = dict(x=x, post_weight=w, residual=x, weight=w)
        args.update(bad)
        with pytest.raises(ValueError):
            tl.tern_norm_add_norm_s8(**args)
