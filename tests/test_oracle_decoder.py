"""CPU pins of oracle/decoder.py (closed forms, brute force, invariants) and
host-side refusals of the decoder operators' entry points."""
import ctypes

import numpy as np
import pytest

import ternary_weight_linear_gb300 as tl
from oracle import decoder as od


def _cache(rng, pages, heads, dim):
    codes = rng.integers(-127, 128, size=(pages, 2, heads, od.BLOCK, dim)).astype(np.int8)
    scales = (0.01 + 0.02 * rng.random((pages, 2, heads))).astype(np.float32)
    return codes, scales


def test_norm_of_a_constant_row():
    # r = 3 everywhere: mean(r^2) = 9, y = weight, the largest weight gets 127
    x = np.full((1, 16), 3.0)
    w = np.linspace(0.5, 2.0, 16)
    r, y, scale, ratio = od.add_rmsnorm(x, None, w, 0.0, None)
    assert np.array_equal(r, x) and np.allclose(y[0], w, rtol=1e-15)
    assert scale[0] == pytest.approx(2.0 / 127) and ratio[0, -1] == pytest.approx(127)


def test_norm_rounds_the_residual_sum():
    x = np.array([[1.0, 2.0 ** -12]], dtype=np.float32)
    res = np.array([[2.0 ** -12, 1.0]], dtype=np.float32)
    r, *_ = od.add_rmsnorm(x, res, np.ones(2), 0.0, lambda s: np.round(s * 256) / 256)
    assert np.array_equal(r, [[1.0, 1.0]])


def test_norm_of_zeros_has_scale_zero():
    *_, scale, ratio = od.add_rmsnorm(np.zeros((2, 16)), None, np.ones(16), 1e-6, None)
    assert not scale.any() and not ratio.any()


def test_append_fresh_page_and_growth():
    codes = np.full((2, 2, 1, od.BLOCK, 64), 99, dtype=np.int8)
    scales = np.full((2, 2, 1), 7.0, dtype=np.float32)  # stale
    table = np.array([[1]], dtype=np.int32)
    x = np.zeros((1, 1, 64), dtype=np.float32)
    x[0, 0, :3] = [1.27, -0.635, 0.01]
    c, s = od.kv8_append(codes, scales, table, [0, 1], [1], x, 2 * x)
    assert s[1, 0, 0] == np.float32(1.27) / np.float32(127) and s[0, 0, 0] == 7.0
    assert list(c[1, 0, 0, 0, :4]) == [127, -64, 1, 0]  # -63.5 rounds to even
    assert (c[1, 0, 0, 1:] == 99).all()  # other slots untouched
    # twice the magnitude: older codes halve (ties to even), the scale doubles
    c2, s2 = od.kv8_append(c, s, table, [0, 1], [2], 2 * x, x)
    assert s2[1, 0, 0] == 2 * s[1, 0, 0] and s2[1, 1, 0] == s[1, 1, 0]
    assert list(c2[1, 0, 0, 0, :4]) == [64, -32, 0, 0]
    assert np.array_equal(c2[1, 1, 0, 0], c[1, 1, 0, 0])


def test_append_nan_stays_in_its_block():
    rng = np.random.default_rng(0)
    codes, scales = _cache(rng, 4, 2, 64)
    x = rng.standard_normal((1, 2, 64)).astype(np.float32)
    x[0, 1, 5] = np.inf
    c, s = od.kv8_append(codes, scales, np.array([[2, 3]]), [0, 1], [70], x, np.zeros_like(x))
    bad = np.isnan(s)
    assert bad.sum() == 1 and bad[3, 0, 1]


def test_attention_uniform_and_single():
    rng = np.random.default_rng(1)
    codes, scales = _cache(rng, 3, 1, 64)
    table = np.array([[2, 0]], dtype=np.int32)
    # zero queries: the mean of the visible values
    q = np.zeros((1, 2, 64))
    out, lse, _ = od.kv8_attention(q, codes, scales, table, [0, 1], [70], 0, 0, 0.125)
    v = np.concatenate([codes[2, 1, 0] * scales[2, 1, 0].astype(float),
                        codes[0, 1, 0] * scales[0, 1, 0].astype(float)])[:70]
    assert np.allclose(out[0], v.mean(0)) and np.allclose(lse, np.log(70))
    # one visible token: its value, whatever the query
    q = rng.standard_normal((1, 2, 64))
    out, *_ = od.kv8_attention(q, codes, scales, table, [0, 1], [70], 1, 0, 0.125)
    assert np.allclose(out[0], v[69])


@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (3, 2), (1, 4)])
def test_attention_against_a_loop(window, sinks):
    rng = np.random.default_rng(window * 10 + sinks)
    codes, scales = _cache(rng, 2, 2, 64)
    n, m = 9, 4
    q = rng.standard_normal((m, 4, 64))
    out, lse, _ = od.kv8_attention(q, codes, scales, np.array([[1]]), [0, m], [n], window, sinks,
                                   0.3)
    for i in range(m):
        p = n - m + i
        for h in range(4):
            top, bottom = 0.0, 0.0
            for j in range(n):
                if j > p or (window and not (j > p - window or j < sinks)):
                    continue
                k = codes[1, 0, h // 2, j] * float(scales[1, 0, h // 2])
                v = codes[1, 1, h // 2, j] * float(scales[1, 1, h // 2])
                w = np.exp(0.3 * float(np.dot(q[i, h], k)))
                top, bottom = top + w * v, bottom + w
            assert np.allclose(out[i, h], top / bottom) and np.isclose(lse[i, h], np.log(bottom))


# ------------------------------------------------------------------ refusals

P = 4096  # a 16-byte aligned fake address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    tl.build()
    return tl.load()


def test_linear_s8_refusals(lib, monkeypatch):
    ok = [P, P, P, P, P, 1, 128, 8, None, 0, None]

    def call(**at):
        a = list(ok)
        for i, v in at.items():
            a[int(i[1:])] = v
        return lib.tern_linear_s8(*a)

    for i in range(5):
        assert call(**{f"a{i}": None}) == -1
        assert call(**{f"a{i}": P + 4}) == -2
    assert call(a5=0) == -1 and call(a6=120) == -1 and call(a6=0) == -1 and call(a7=0) == -1
    monkeypatch.setenv("TERN_RUNG", "bf16")
    tl.tern_reload_env()
    try:
        assert call() == -1  # no int8 form
    finally:
        monkeypatch.delenv("TERN_RUNG")
        tl.tern_reload_env()


def test_norm_refusals(lib):
    #     x  xt ld  res out rt w  wt eps   q  xs y  T  K
    ok = [P, 0, 64, P, P, 1, P, 1, 1e-6, P, P, P, 2, 64, None]

    def call(**at):
        a = list(ok)
        for i, v in at.items():
            a[int(i[1:])] = v
        return lib.tern_add_rmsnorm_s8(*a)

    assert call(a0=None) == -1 and call(a6=None) == -1
    assert call(a1=2) == -1 and call(a5=2) == -1 and call(a7=-1) == -1  # types
    assert call(a2=63) == -1 and call(a13=56) == -1 and call(a12=0) == -1
    assert call(a13=65536, a2=65536) == -1
    assert call(a8=-1.0) == -1 and call(a8=float("nan")) == -1
    assert call(a9=None) == -1 and call(a10=None) == -1  # codes without scales and back
    assert call(a9=None, a10=None, a11=None) == -1       # nothing to write
    assert call(a3=None) == -1                           # residual_out without residual
    for i in (0, 3, 4, 6, 9, 10, 11):
        assert call(**{f"a{i}": P + 8}) == -2
    assert call(a2=66) == -2  # rows of 264 bytes


def _fake_cache(**kw):
    d = dict(codes=P, scales=P, page_table=P, seq_lens=P, row_start=P, pages=4, seqs=1,
             table_width=4, kv_heads=2, head_dim=64)
    d.update(kw)
    return tl._KV8Cache(**d)


BAD_CACHES = [
    (dict(codes=None), -1), (dict(scales=None), -1), (dict(page_table=None), -1),
    (dict(seq_lens=None), -1), (dict(row_start=None), -1), (dict(pages=0), -1),
    (dict(seqs=0), -1), (dict(table_width=0), -1), (dict(kv_heads=0), -1),
    (dict(head_dim=96), -1), (dict(pages=1 << 24), -1), (dict(table_width=1 << 26), -1),
    (dict(codes=P + 8), -2), (dict(scales=P + 4), -2), (dict(page_table=P + 4), -2),
]


def test_append_refusals(lib):
    def call(cache=None, k=P, v=P, type=0, ld=128, hd=64, rows=3, new=1):
        c = _fake_cache() if cache is None else cache
        return lib.tern_kv8_append(ctypes.byref(c), k, v, type, ld, hd, rows, new, None)

    for kw, want in BAD_CACHES:
        assert call(_fake_cache(**kw)) == want, kw
    assert call(k=None) == -1 and call(v=None) == -1 and call(type=3) == -1
    assert call(rows=-1) == -1 and call(new=0) == -1 and call(ld=63) == -1 and call(hd=0) == -1
    assert call(ld=1 << 40) == -1
    assert call(k=P + 8) == -2 and call(v=P + 2) == -2 and call(ld=130) == -2
    assert call(type=1, hd=68) == -2
    assert call(rows=0, k=None, v=None) == 0  # no rows: nothing to do


def test_attention_refusals(lib):
    def call(cache=None, q=P, type=1, ld=256, hd=64, rows=3, heads=4, new=1, window=0, sinks=0,
             scale=0.1, out=P, lse=None, ws=P, nws=1 << 30):
        c = _fake_cache() if cache is None else cache
        return lib.tern_kv8_attention(ctypes.byref(c), q, type, ld, hd, rows, heads, new, window,
                                      sinks, scale, out, lse, ws, nws, None)

    for kw, want in BAD_CACHES:
        assert call(_fake_cache(**kw)) == want, kw
    assert call(q=None) == -1 and call(out=None) == -1
    assert call(type=0) == -1 and call(heads=3) == -1 and call(heads=0) == -1
    assert call(heads=2 * 65) == -1 and call(new=0) == -1 and call(rows=-1) == -1
    assert call(window=-1) == -1 and call(sinks=-1) == -1
    assert call(scale=0.0) == -1 and call(scale=float("nan")) == -1
    assert call(scale=float("inf")) == -1
    assert call(q=P + 8) == -2 and call(out=P + 8) == -2 and call(lse=P + 4) == -2
    assert call(ld=260) == -2 and call(hd=68) == -2
    need = lib.tern_kv8_attention_workspace_bytes(1, 3, 4, 2, 64)
    assert call(nws=need - 1) == -3 and call(ws=None) == -3 and call(ws=P + 8) == -2
    assert call(rows=0, q=None, out=None, ws=None, nws=0) == 0


def test_attention_workspace_bytes():
    f = tl.tern_kv8_attention_workspace_bytes
    assert f(1, 1, 4, 4, 64) > tl.SYNC_BYTES
    assert f(0, 1, 4, 4, 64) == 0 and f(1, 0, 4, 4, 64) == 0 and f(1, 1, 5, 4, 64) == 0
    assert f(1, 1, 4, 4, 80) == 0


def test_status_text():
    assert "out of range" in tl.tern_status_string(-7)
