"""GPU parity of the decoder operators beside the linear layer (norm with int8
codes, the layer on such codes, the int8 cache's append) against the fp64 /
IEEE-fp32 oracle in oracle/decoder.py.

Bars, derived from the formulas:
- norm: r bit-exact.  The mean square is an fp32 sum of K <= 32768 terms over
  at least 32 lanes, 32 sequential additions and 10 tree levels at most per
  value, so its relative error is below 64 * 2^-24 and its root's half that;
  with the square root, the divisions and the products (2^-24 each, below 10
  of them) y and x_scale are within 2^-18 of the exact values.  A code is
  within 0.5 + 127 * 2^-17 of the exact quotient.
- append: codes and scales bit-exact (every step is one IEEE fp32 operation).
- linear on codes: the s8 rung's bar.
"""
import numpy as np
import pytest

import oracle
import synth
from helpers import assert_s8_parity, to_device
from oracle import decoder as od

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
    return t.float().cpu().numpy()


def _bf16(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).bfloat16().float().numpy()


# ------------------------------------------------------------------ norm

def _norm_check(tl, T, K, xt, rt, wt, with_y=True, ld=None, in_place=False, seed=0, scale=1.0):
    import torch
    rng = np.random.default_rng([seed, T, K])
    x = torch.from_numpy((rng.standard_normal((T, ld or K)) * scale).astype(np.float32)).cuda()
    x = x.to(xt)[:, :K]
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(K)).astype(np.float32)).cuda().to(wt)
    res = None
    if rt is not None:
        r0 = rng.standard_normal((T, K)) * scale
        r0[:, rng.integers(0, K, max(1, K // 100))] *= 20
        res = torch.from_numpy(r0.astype(np.float32)).cuda().to(rt)
    xn, wn = _np(x), _np(w)
    rn = _np(res) if res is not None else None
    y = torch.empty(T, K, dtype=torch.bfloat16, device="cuda") if with_y else None
    q, xs, r = tl.tern_add_rmsnorm_s8(x, w, res, 1e-6, y=y,
                                      residual_out=res if in_place else None)
    torch.cuda.synchronize()
    rnd = None if rt is None else (_bf16 if rt == torch.bfloat16 else (lambda s: s))
    r_ref, y_ref, s_ref, ratio = od.add_rmsnorm(xn, rn, wn, 1e-6, rnd)
    if res is not None:
        assert np.array_equal(_np(r).astype(np.float64), r_ref)
        assert (r is res) == in_place
    else:
        assert r is None
    s = xs.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(s - s_ref) <= REL * s_ref)
    c = q.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(c) <= 127)
    assert np.all(np.abs(c - ratio) <= 0.5 + 127 * 2.0 ** -17)
    assert np.all(np.abs(c).max(1)[s_ref > 0] == 127)
    if with_y:
        # the bf16 rounding of some value within 2 REL of the exact one
        # (rounding is monotonic)
        lo, hi = _bf16(y_ref * (1 - 2 * REL)), _bf16(y_ref * (1 + 2 * REL))
        got = _np(y)
        assert np.all((got >= np.minimum(lo, hi)) & (got <= np.maximum(lo, hi)))


# one vector, an odd count of warps, the model's width, two and four vectors
# per thread (the last with a partial warp)
@pytest.mark.parametrize("T,K", [(1, 16), (3, 272), (1, 5120), (37, 5120), (5, 9984),
                                 (2, 17408), (3, 32768)])
def test_norm_widths(tl, T, K):
    import torch
    _norm_check(tl, T, K, torch.float32, torch.bfloat16, torch.bfloat16)


@pytest.mark.parametrize("xt", ["float32", "bfloat16"])
@pytest.mark.parametrize("rt", ["float32", "bfloat16", None])
@pytest.mark.parametrize("wt", ["float32", "bfloat16"])
def test_norm_types(tl, xt, rt, wt):
    import torch
    f = lambda n: None if n is None else getattr(torch, n)  # noqa: E731
    _norm_check(tl, 9, 1040, f(xt), f(rt), f(wt), with_y=rt is None, ld=1072, seed=3)


def test_norm_in_place_and_small_and_large_values(tl):
    import torch
    _norm_check(tl, 4, 512, torch.float32, torch.bfloat16, torch.float32, in_place=True)
    _norm_check(tl, 4, 512, torch.float32, torch.float32, torch.bfloat16, scale=1e-12)
    _norm_check(tl, 4, 512, torch.float32, torch.float32, torch.bfloat16, scale=1e12)


def test_norm_zero_rows_and_y_alone(tl):
    import torch
    x = torch.zeros(3, 256, device="cuda")
    x[1] = 1.0
    w = torch.ones(256, device="cuda")
    q, s, _ = tl.tern_add_rmsnorm_s8(x, w)
    assert s.tolist()[0] == 0 and s.tolist()[2] == 0 and not q[0].any() and not q[2].any()
    assert (q[1] == 127).all()
    y = torch.empty(3, 256, dtype=torch.bfloat16, device="cuda")
    q, s, r = tl.tern_add_rmsnorm_s8(x, w, y=y, quantise=False)
    assert q is None and s is None and r is None and (y[1] == 1).all() and not y[0].any()


def test_norm_nonfinite_row_keeps_to_itself(tl):
    import torch
    x = torch.randn(3, 256, device="cuda")
    w = torch.ones(256, device="cuda")
    q0, s0, _ = tl.tern_add_rmsnorm_s8(x, w)
    x[1, 7] = float("nan")
    q1, s1, _ = tl.tern_add_rmsnorm_s8(x, w)
    for t in (0, 2):
        assert torch.equal(q0[t], q1[t]) and s0[t] == s1[t]


def test_norm_argument_errors(tl):
    import torch
    x = torch.zeros(2, 256, device="cuda")
    w = torch.ones(256, device="cuda")
    with pytest.raises(ValueError):
        tl.tern_add_rmsnorm_s8(x.half(), w)
    with pytest.raises(ValueError):
        tl.tern_add_rmsnorm_s8(x, w[:128])
    with pytest.raises(ValueError):
        tl.tern_add_rmsnorm_s8(x, w, residual=x[:1])
    with pytest.raises(ValueError):
        tl.tern_add_rmsnorm_s8(x, w, residual_out=x)
    with pytest.raises(ValueError):
        tl.tern_add_rmsnorm_s8(x, w, quantise=False)
    with pytest.raises(ValueError):
        tl.tern_add_rmsnorm_s8(x.t(), w)
    with pytest.raises(ValueError):
        tl.tern_add_rmsnorm_s8(x.cpu(), w)
    with pytest.raises(tl.TernError):
        tl.tern_add_rmsnorm_s8(x[:, :250].contiguous(), w[:250].contiguous())


# ------------------------------------------------------------------ linear on codes

# every token tile and rung, ragged row blocks, one and several stages of K
@pytest.mark.parametrize("T,K,N", [(1, 128, 8), (1, 2048, 1000), (3, 5120, 300), (4, 1152, 129),
                                   (8, 1024, 512), (13, 5120, 257), (16, 640, 128),
                                   (17, 256, 100), (31, 1280, 640), (33, 512, 130),
                                   (130, 5120, 1000), (277, 1024, 384)])
def test_linear_s8_parity(tl, T, K, N):
    import torch
    c = synth.case("tiny", T, K=K, N=N, seed=T + N)
    W, s, _ = to_device(c)
    Wp = tl.tern_pack(W)
    rng = np.random.default_rng([T, K, N])
    q = rng.integers(-128, 128, size=(T, K)).astype(np.int8)
    xs = (rng.random(T) * 0.1).astype(np.float32)
    xs[T // 2] *= -1  # the codes' sign may sit in the scale
    if T > 2:
        xs[-1] = -0.0
        q[0] = 0
    y = tl.tern_linear_s8(Wp, s, torch.from_numpy(q).cuda(), torch.from_numpy(xs).cuda())
    torch.cuda.synchronize()
    assert tl.tern_device_status() == 0
    assert tl.tern_last_rung() == tl.tern_rung_name(tl.tern_select_rung(T))
    wp, _ = oracle.pack(c.W)
    y_ref, m, _ = oracle.linear_s8(wp, c.scales, q, np.abs(xs), T, K, N)
    assert_s8_parity(y.cpu().numpy(), y_ref * np.where(np.signbit(xs), -1, 1)[:, None], m,
                     f"codes T={T} K={K} N={N}")


@pytest.mark.parametrize("T", [40, 2])
def test_linear_s8_is_the_layer_on_its_own_codes(tl, T, monkeypatch):
    """The codes of tern_quant_act_s8 give tern_linear's s8 rung bit for bit
    (and its int8-activation form on the small-T rungs)."""
    import torch
    monkeypatch.setenv("TERN_DECODE_ACT", "int8")
    tl.tern_reload_env()
    try:
        c = synth.case("tiny", T, K=1024, N=600, seed=5, outliers=True)
        W, s, x = to_device(c)
        Wp = tl.tern_pack(W)
        q, xs = tl.tern_quant_act_s8(x)
        assert torch.equal(tl.tern_linear_s8(Wp, s, q, xs), tl.tern_linear(Wp, s, x))
    finally:
        monkeypatch.delenv("TERN_DECODE_ACT")
        tl.tern_reload_env()


def test_linear_s8_every_rung_forced(tl, monkeypatch):
    import torch
    T, K, N = 19, 640, 260
    c = synth.case("tiny", T, K=K, N=N, seed=8)
    W, s, _ = to_device(c)
    Wp = tl.tern_pack(W)
    rng = np.random.default_rng(8)
    q = rng.integers(-127, 128, size=(T, K)).astype(np.int8)
    xs = (rng.random(T) * 0.1).astype(np.float32)
    wp, _ = oracle.pack(c.W)
    y_ref, m, _ = oracle.linear_s8(wp, c.scales, q, xs, T, K, N)
    ws = torch.zeros(tl.tern_linear_workspace_bytes(T, K, N), dtype=torch.uint8, device="cuda")
    for rung in ("gemv", "small_t", "small_t_tiled", "s8"):
        monkeypatch.setenv("TERN_RUNG", rung)
        tl.tern_reload_env()
        try:
            for _ in range(2):  # the kept workspace stays valid
                y = tl.tern_linear_s8(Wp, s, torch.from_numpy(q).cuda(),
                                      torch.from_numpy(xs).cuda(), workspace=ws)
                assert tl.tern_last_rung() == rung
                assert_s8_parity(y.cpu().numpy(), y_ref, m, rung)
        finally:
            monkeypatch.delenv("TERN_RUNG")
            tl.tern_reload_env()


def test_linear_s8_argument_errors(tl):
    import torch
    q = torch.zeros(2, 256, dtype=torch.int8, device="cuda")
    xs = torch.zeros(2, device="cuda")
    Wp = torch.zeros(8, 16, dtype=torch.int32, device="cuda")
    s = torch.zeros(8, 2, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        tl.tern_linear_s8(Wp, s, q.float(), xs)
    with pytest.raises(ValueError):
        tl.tern_linear_s8(Wp, s, q, xs[:1])
    with pytest.raises(ValueError):
        tl.tern_linear_s8(Wp, s[:, :1].contiguous(), q, xs)
    with pytest.raises(tl.TernError):
        tl.tern_linear_s8(Wp, s, q, xs, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------ append

def _append_case(lens, new, heads, dim, seed, width=None, extra=2):
    rng = np.random.default_rng(seed)
    each = [(n + 63) // 64 for n in lens]
    width = width or max(1, max(each))
    pages = sum(each) + extra
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), width), 2 ** 30, dtype=np.int32)  # unused entries: rubbish
    at = 0
    for b, e in enumerate(each):
        table[b, :e] = order[at:at + e]
        at += e
    codes = rng.integers(-127, 128, size=(pages, 2, heads, 64, dim)).astype(np.int8)
    scales = (0.005 + 0.02 * rng.random((pages, 2, heads))).astype(np.float32)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return rng, table, codes, scales, start, np.asarray(lens, dtype=np.int32)


def _append_check(tl, lens, new, heads, dim, dtype, seed=0, strided=False, tweak=None,
                  max_new=None):
    import torch
    rng, table, codes, scales, start, lens = _append_case(lens, new, heads, dim, seed)
    rows = int(start[-1])
    kv = rng.standard_normal((rows, 2 * heads + 1, dim)).astype(np.float32)
    kv *= np.exp(rng.standard_normal((rows, 1, 1))).astype(np.float32)
    if tweak:
        tweak(kv, scales)
    dev = torch.from_numpy(kv).cuda().to(getattr(torch, dtype))
    k, v = dev[:, :heads], dev[:, heads:2 * heads]
    if not strided:
        k, v = k.contiguous(), v.contiguous()
    c, s = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    args = (torch.from_numpy(table).cuda(), torch.from_numpy(start).cuda(),
            torch.from_numpy(lens).cuda())
    tl.tern_kv8_append(k, v, c, s, *args, max_new=max_new)
    torch.cuda.synchronize()
    assert tl.tern_device_status() == 0
    c_ref, s_ref = od.kv8_append(codes, scales, table, start, lens, _np(k), _np(v))
    sn = s.cpu().numpy()
    assert np.array_equal(sn, s_ref, equal_nan=True)
    good = ~np.isnan(s_ref)
    assert np.array_equal(c.cpu().numpy()[good], c_ref[good])
    return c, s, (k, v, args)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("heads,dim", [(8, 128), (1, 64), (3, 128), (5, 64)])
def test_append_bit_exact(tl, dtype, heads, dim):
    # page starts and ends inside, at and across the new tokens; nothing new;
    # nothing at all; one token into a page of one, of 63 and a fresh one
    lens = [1, 64, 65, 200, 128, 77, 0, 130, 64, 2]
    new = [1, 64, 65, 66, 1, 0, 0, 129, 1, 1]
    _append_check(tl, lens, new, heads, dim, dtype, seed=heads, strided=True)


def test_append_decode_steps_many_sequences(tl):
    lens = [1 + (37 * i) % 500 for i in range(300)]
    _append_check(tl, lens, [1] * 300, 2, 64, "bfloat16", seed=1, max_new=1)


def test_append_long_prompt(tl):
    _append_check(tl, [1500, 901], [1333, 901], 4, 128, "bfloat16", seed=2)


def test_append_twice_is_append_once(tl):
    """Appending the same tokens again changes nothing: the scale has grown."""
    import torch
    c, s, (k, v, args) = _append_check(tl, [100, 70], [3, 6], 2, 128, "bfloat16", seed=3)
    c0, s0 = c.clone(), s.clone()
    tl.tern_kv8_append(k, v, c, s, *args)
    assert torch.equal(c, c0) and torch.equal(s, s0)


def test_append_zeros_nan_and_extremes(tl):
    def tweak(kv, scales):
        kv[0] = 0                  # all-zero block
        kv[1, 0, 3] = np.inf       # a block with an infinity
        kv[2, 1, 5] = np.nan       # and one with a NaN
        kv[3] *= 1e-38             # subnormal scales
        kv[4] *= 1e37
        scales[0] = np.nan         # (stale scale of whichever page is first)
    _append_check(tl, [1, 65, 129, 193, 257], [1, 1, 1, 1, 1], 1, 64, "float32", seed=4,
                  tweak=tweak)


def test_append_skips_what_is_out_of_range(tl):
    import torch
    rng, table, codes, scales, start, lens = _append_case([70, 10, 20, 30], [2, 3, 4, 5], 2, 64, 9)
    kv = torch.randn(14, 2, 64, device="cuda")
    c, s = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    table[0, 1] = len(codes)      # a page past the pool
    table[1, 0] = -1
    lens[2] = 64 * table.shape[1] + 1  # does not fit the table
    tl.tern_kv8_append(kv, kv, c, s, torch.from_numpy(table).cuda(),
                       torch.from_numpy(start).cuda(), torch.from_numpy(lens).cuda())
    assert tl.tern_device_status() == -7
    assert tl.tern_device_status() == 0
    # the one good sequence is written, nothing else is
    kn = kv.cpu().numpy()
    c_ref, s_ref = od.kv8_append(codes, scales, table[3:], start[3:], lens[3:], kn, kn)
    assert np.array_equal(c.cpu().numpy(), c_ref) and np.array_equal(s.cpu().numpy(), s_ref)
    # more new tokens than max_new, than tokens, rows past the end, descending rows
    for st, ln, most in (([0, 5], [5], 4), ([0, 6], [5], 14), ([10, 15], [9], 14),
                         ([9, 5], [9], 14), ([-2, 1], [9], 14), ([0, 1], [-1], 14)):
        c1, s1 = c.clone(), s.clone()
        tl.tern_kv8_append(kv, kv, c1, s1, torch.from_numpy(table[3:].copy()).cuda(),
                           torch.tensor(st, dtype=torch.int32).cuda(),
                           torch.tensor(ln, dtype=torch.int32).cuda(), max_new=most)
        assert tl.tern_device_status() == -7, (st, ln)
        assert torch.equal(c1, c) and torch.equal(s1, s)


def test_append_argument_errors(tl):
    import torch
    rng, table, codes, scales, start, lens = _append_case([70], [2], 2, 64, 9)
    c, s, t, st, ln = (torch.from_numpy(a).cuda() for a in (codes, scales, table, start, lens))
    kv = torch.randn(2, 2, 64, device="cuda")
    tl.tern_kv8_append(kv[:0], kv[:0], c, s, t, st, ln)  # no rows: nothing is done
    assert np.array_equal(c.cpu().numpy(), codes)
    for bad in ((kv[:, :1], kv[:, :1], c, s, t, st, ln), (kv, kv[:1], c, s, t, st, ln),
                (kv, kv.half(), c, s, t, st, ln), (kv, kv, c[:, :1], s, t, st, ln),
                (kv, kv, c, s[:1], t, st, ln), (kv, kv, c, s, t.long(), st, ln),
                (kv, kv, c, s, t, st[:1], ln), (kv, kv, c, s, t, st, ln.cpu()),
                (kv.double(), kv.double(), c, s, t, st, ln)):
        with pytest.raises(ValueError):
            tl.tern_kv8_append(*bad)
    with pytest.raises(tl.TernError):  # rows of every token the same: strides too small
        tl.tern_kv8_append(kv[:1].expand(2, 2, 64), kv[:1].expand(2, 2, 64), c, s, t, st, ln)
