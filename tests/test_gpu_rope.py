"""GPU parity of tern_rope and tern_kv8_append_rope.

tern_rope against the fp64 oracle.  Bar, in units of u = 2^-24: the turn is
cut at 2^-32 (2^-29 radians) and its rest x <= pi / 4 rounded three times to
fp32 (2.4 u); the series' roundings and the terms left out are below 1.6 u, so
sine and cosine are within 4 u; the magnitude's product, the pair's two products
and their sum add a u each.  So an element is within 8 u m (|u| + |v|) = 2^-21 m
(|u| + |v|), and half a step of the output's type (2^-8, 2^-11, 2^-24 of the
value, 2^-25 for fp16's subnormals).

tern_kv8_append_rope bit for bit: its queries are what tern_rope writes into
their type, and its cache what the IEEE-fp32 oracle of the append makes of the
keys that tern_rope writes in fp32.
"""
import numpy as np
import pytest

from oracle import attention_block as ab
from oracle import decoder as od

pytestmark = pytest.mark.gpu

HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}


@pytest.fixture(scope="module")
def tl():
    import torch
    import ternary_weight_linear_gb300 as tl
    tl.build()
    tl.load()
    torch.cuda.init()
    return tl


def _rand(shape, dtype, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(getattr(torch, dtype))


def _f64(t):
    return t.double().cpu().numpy()


def _table(tl, rotary, **kw):
    freq, m = tl.tern_rope_frequencies(rotary, **kw)
    return freq, m, [f % 2 ** 64 for f in freq.cpu().tolist()]


def check(tl, x, pos, rotary, interleaved, out_dtype="float32", out=None, **table):
    import torch
    freq, m, turns = _table(tl, rotary, **table)
    want, size = ab.rope(_f64(x), pos, turns, interleaved, np.float32(m).astype(np.float64))
    where = torch.tensor(pos, dtype=torch.int32, device="cuda")
    if out is None:
        out = torch.empty(x.shape, dtype=getattr(torch, out_dtype), device="cuda")
    got = tl.tern_rope(x, where, freq, interleaved=interleaved, magnitude=m, out=out)
    assert got is out
    torch.cuda.synchronize()
    name = str(out.dtype).split(".")[1]
    bound = 2.0 ** -21 * m * size
    bound = bound + HALF[name] * (np.abs(want) + bound) + (2.0 ** -25 if name == "float16" else 0)
    err = np.abs(_f64(out) - want)
    assert np.all(err <= bound), float(np.max(err / np.maximum(bound, 1e-30)))
    return out


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,heads,dim,rotary", [
    (1, 1, 16, 16), (1, 48, 128, 128), (3, 7, 96, 32), (70, 5, 64, 48), (33, 56, 128, 16),
    (2, 3, 1024, 1024), (130, 1, 256, 64), (1, 300, 64, 64)])
def test_rope_shapes(tl, T, heads, dim, rotary, interleaved):
    pos = (np.arange(T) * 37 + 5).tolist()
    check(tl, _rand((T, heads, dim), "float32", T), pos, rotary, interleaved)


@pytest.mark.parametrize("xt", list(HALF))
@pytest.mark.parametrize("ot", list(HALF))
def test_rope_types(tl, xt, ot):
    check(tl, _rand((9, 6, 128), xt, 1), list(range(9)), 64, True, ot)


def test_rope_positions(tl):
    """Zero, far, negative, the ends of int32."""
    pos = [0, 1, -1, 999999, -999999, 2 ** 31 - 1, -2 ** 31, 12345678]
    for interleaved in (False, True):
        check(tl, _rand((8, 3, 64), "float32", 2), pos, 64, interleaved, base=5e5)


@pytest.mark.parametrize("table", [dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
                                   dict(scaling="bands", factor=8.0, trained=8192),
                                   dict(scaling="ramp", factor=16.0, trained=4096)])
def test_rope_scalings(tl, table):
    check(tl, _rand((5, 4, 128), "bfloat16", 3), [0, 7, 8191, 70000, 131071], 128, False, "bfloat16",
          **table)


def test_rope_many_tokens(tl):
    """Several heads a thread, a last block of fewer tokens."""
    T = 4099
    x = _rand((T, 24, 64), "bfloat16", 4)
    pick = np.r_[0:3, 2047:2050, T - 3:T]
    pos = np.arange(T, dtype=np.int64) + 100
    import torch
    freq, m, turns = _table(tl, 32)
    got = tl.tern_rope(x, torch.from_numpy(pos).int().cuda(), freq, out=torch.empty_like(x).float())
    want, size = ab.rope(_f64(x)[pick], pos[pick], turns, False, 1.0)
    assert np.all(np.abs(_f64(got)[pick] - want) <= 2.0 ** -21 * size + 2.0 ** -23 * np.abs(want))
    assert torch.equal(got[..., 32:], x[..., 32:].float())
    # every row, against the same row alone
    for t in range(0, T, 511):
        alone = tl.tern_rope(x[t:t + 1], torch.tensor([pos[t]], dtype=torch.int32, device="cuda"),
                             freq, out=torch.empty(1, 24, 64, device="cuda"))
        assert torch.equal(alone, got[t:t + 1])


def test_rope_in_place_and_strided(tl):
    """The queries and keys of a projection's rows, turned where they are."""
    import torch
    y = _rand((6, 20, 64), "float32", 5)
    before = y.clone()
    part = y[:, 3:15]
    pos = [4, 0, 9, 2, 77, 1000]
    freq, m, turns = _table(tl, 64)
    want, size = ab.rope(_f64(part), pos, turns, False, 1.0)
    where = torch.tensor(pos, dtype=torch.int32, device="cuda")
    tl.tern_rope(part, where, freq, out=part)
    err = np.abs(_f64(part) - want)
    assert np.all(err <= 2.0 ** -21 * size + 2.0 ** -23 * np.abs(want))
    assert torch.equal(y[:, :3], before[:, :3]) and torch.equal(y[:, 15:], before[:, 15:])
    # out of place the same bits, through other strides
    out = torch.zeros(12, 6, 80, device="cuda").transpose(0, 1)[..., :64]
    tl.tern_rope(before[:, 3:15], where, freq, out=out)
    assert torch.equal(out, part)


def test_rope_gradient_is_the_turn_back(tl):
    """<g, R x> = <R^T g, x>, and against a difference quotient."""
    import torch
    x, g = _rand((5, 2, 64), "float32", 6), _rand((5, 2, 64), "float32", 7)
    pos = torch.tensor([1, 50, 999, 123456, 0], dtype=torch.int32, device="cuda")
    freq, _, _ = _table(tl, 32)
    back = tl.tern_rope(g, -pos, freq)
    lhs = (g.double() * tl.tern_rope(x, pos, freq).double()).sum((1, 2))
    rhs = (back.double() * x.double()).sum((1, 2))
    # each side's elements are off by 2^-21 of their pairs
    size = (g.abs().double() * x.abs().double()).sum((1, 2)) + (g.norm() * x.norm()).double()
    assert torch.all((lhs - rhs).abs() <= 2.0 ** -20 * size)
    # the map is linear: the quotient has no error of its own
    e = torch.zeros_like(x)
    e[3, 1, 5] = 1.0
    quotient = (g.double() * (tl.tern_rope(x + e, pos, freq).double()
                              - tl.tern_rope(x, pos, freq).double())).sum()
    assert abs(float(quotient) - float(back[3, 1, 5])) <= 2.0 ** -20 * float(size.sum())


def test_rope_keeps_what_is_not_finite_to_its_pair(tl):
    import torch
    x = torch.ones(1, 2, 64, device="cuda")
    x[0, 1, 3] = float("nan")
    x[0, 1, 60] = float("inf")
    out = tl.tern_rope(x, torch.tensor([3], dtype=torch.int32, device="cuda"), _table(tl, 32)[0])
    bad = ~torch.isfinite(out)
    assert bad.nonzero()[:, 2].tolist() == [3, 19, 60] and not bad[0, 0].any()


def test_rope_refusals_of_the_binding(tl):
    import torch
    x = torch.zeros(2, 3, 64, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    freq, _ = tl.tern_rope_frequencies(64)
    for bad in (dict(x=x.cpu()), dict(x=x.double()), dict(positions=pos.long()),
                dict(positions=pos[:1]), dict(freq=freq.int()), dict(out=x[:1]),
                dict(x=x.transpose(1, 2))):
        args = dict(x=x, positions=pos, freq=freq)
        args.update(bad)
        with pytest.raises(ValueError):
            tl.tern_rope(**args)
    with pytest.raises(tl.TernError):
        tl.tern_rope(x, pos, torch.cat((freq, freq)))
    assert tl.tern_rope(x[:0], pos[:0], freq).shape == (0, 3, 64)


# ------------------------------------------------------------------ append

class Cache:
    """Pages in a shuffled order, older tokens of random codes."""

    def __init__(self, lens, new, kv, dim, seed=0, scale=0.02):
        import torch
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, np.int32)
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        each = [(n + 63) // 64 for n in lens]
        pages = sum(each) + 2
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.full((len(lens), max(1, max(each)) + 1), -7, np.int32)
        at = 0
        for b, e in enumerate(each):
            self.table[b, :e] = order[at:at + e]
            at += e
        self.codes = rng.integers(-127, 128, (pages, 2, kv, 64, dim)).astype(np.int8)
        self.scales = (scale * rng.random((pages, 2, kv))).astype(np.float32)
        self.dev = [torch.from_numpy(a).cuda() for a in
                    (self.codes, self.scales, self.table, self.start, self.lens)]

    def positions(self):
        return np.concatenate([np.arange(n - m, n) for n, m in
                               zip(self.lens, np.diff(self.start))] + [[]]).astype(np.int32)


def append_check(tl, lens, new, heads, kv, dim, rotary, interleaved, xt="float32", qt="bfloat16",
                 positions=None, max_new=True, q=True, seed=0, **table):
    import torch
    c = Cache(lens, new, kv, dim, seed)
    rows = int(c.start[-1])
    y = _rand((rows, heads + 2 * kv, dim), xt, seed + 1)
    yq, yk, yv = y.split((heads, kv, kv), 1)
    freq, m, _ = _table(tl, rotary, **table)
    pos = torch.from_numpy(c.positions() if positions is None else positions).cuda()
    k32 = torch.empty(rows, kv, dim, device="cuda")
    q_want = torch.empty(rows, heads, dim, dtype=getattr(torch, qt), device="cuda")
    if rows:
        tl.tern_rope(yk, pos, freq, interleaved=interleaved, magnitude=m, out=k32)
        tl.tern_rope(yq, pos, freq, interleaved=interleaved, magnitude=m, out=q_want)
    want = od.kv8_append(c.codes, c.scales, c.table, c.start, c.lens, k32.cpu().numpy(),
                         yv.float().cpu().numpy())
    out = torch.full((rows, heads, dim), 7.0, dtype=getattr(torch, qt), device="cuda")
    got = tl.tern_kv8_append_rope(
        yq if q else None, yk, yv, *c.dev, freq, interleaved=interleaved, magnitude=m,
        positions=None if positions is None else pos, max_new=max(new) if max_new else None,
        q_out=out if q else None)
    torch.cuda.synchronize()
    assert tl.tern_device_status() == 0
    assert got is (out if q else None)
    if q:
        assert torch.equal(out, q_want)
    assert np.array_equal(c.dev[1].cpu().numpy(), want[1])
    assert np.array_equal(c.dev[0].cpu().numpy(), want[0])


LENS = [1, 63, 64, 65, 0, 200, 130, 77]


@pytest.mark.parametrize("dim,rotary", [(128, 128), (128, 32), (64, 64), (64, 48), (64, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_one_token(tl, dim, rotary, interleaved):
    new = [min(1, n) for n in LENS]
    new[-1] = 0
    append_check(tl, LENS, new, 12, 2, dim, rotary, interleaved, seed=dim + rotary)


@pytest.mark.parametrize("xt", list(HALF))
@pytest.mark.parametrize("qt", ["bfloat16", "float16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_append_prompts(tl, xt, qt, dim):
    append_check(tl, [300, 129, 64, 70], [200, 129, 1, 6], 10, 2, dim, dim // 2, dim == 64, xt, qt,
                 base=1e6, scaling="ramp", factor=4.0, trained=4096)


def test_append_all_rows_as_max_new_and_many_heads(tl):
    append_check(tl, [90, 20], [17, 20], 70, 5, 128, 64, False, max_new=False)
    append_check(tl, [5], [5], 3, 3, 64, 64, True)  # query heads no multiple of the others


def test_append_positions_of_the_caller(tl):
    rng = np.random.default_rng(3)
    append_check(tl, [100, 40], [30, 40], 4, 2, 128, 128, False,
                 positions=rng.integers(-10 ** 6, 10 ** 6, 70).astype(np.int32))


def test_append_without_queries(tl):
    append_check(tl, [100, 40], [30, 2], 4, 2, 128, 128, False, q=False)


def test_append_without_turning_values_matches_the_plain_append(tl):
    """Positions of 0 turn nothing."""
    import torch
    a, b = (Cache([150, 30], [40, 30], 2, 64, seed=5) for _ in range(2))
    k, v = _rand((70, 2, 64), "bfloat16", 8), _rand((70, 2, 64), "bfloat16", 9)
    tl.tern_kv8_append(k, v, *a.dev, max_new=40)
    tl.tern_kv8_append_rope(None, k, v, *b.dev, _table(tl, 64)[0], max_new=40,
                            positions=torch.zeros(70, dtype=torch.int32, device="cuda"))
    assert torch.equal(a.dev[0], b.dev[0]) and torch.equal(a.dev[1], b.dev[1])


def test_append_skips_what_is_inconsistent(tl):
    """A sequence that does not fit its table, a page out of range, rows of no
    sequence: skipped, reported, the others unaffected."""
    import torch
    c = Cache([100, 70, 30], [3, 2, 4], 2, 64, seed=6)
    c.lens[1] = 5000
    c.table[2, 0] = 999
    c.dev[4].copy_(torch.from_numpy(c.lens))
    c.dev[2].copy_(torch.from_numpy(c.table))
    rows = 12  # three behind the last sequence
    y = _rand((rows, 8, 64), "float32", 10)
    out = torch.full((rows, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    freq = _table(tl, 64)[0]
    tl.tern_kv8_append_rope(y[:, :4], y[:, 4:6], y[:, 6:], *c.dev, freq, max_new=4, q_out=out)
    assert tl.tern_device_status() == -7
    pos = torch.tensor([97, 98, 99, 0, 0, 26, 27, 28, 29, 0, 0, 0], dtype=torch.int32, device="cuda")
    want = tl.tern_rope(y[:, :4], pos, freq, out=torch.empty_like(out))
    assert torch.equal(out[:3], want[:3]) and torch.equal(out[5:9], want[5:9])
    assert (out[3:5] == 7).all() and (out[9:] == 7).all()
    k = tl.tern_rope(y[:, 4:6], pos, freq)
    ref = od.kv8_append(c.codes, c.scales, c.table[:1], c.start[:2], c.lens[:1],
                        k.cpu().numpy(), y[:, 6:].cpu().numpy())
    assert np.array_equal(c.dev[0].cpu().numpy(), ref[0])
    assert np.array_equal(c.dev[1].cpu().numpy(), ref[1])


def test_append_not_finite(tl):
    """A key that is not finite makes its block's scale NaN, and no other's."""
    import torch
    c = Cache([70, 64], [70, 64], 2, 64, seed=7)
    k, v = _rand((134, 2, 64), "float32", 11), _rand((134, 2, 64), "float32", 12)
    k[66, 1, 3] = float("inf")
    tl.tern_kv8_append_rope(None, k, v, *c.dev, _table(tl, 32)[0], max_new=70)
    bad = torch.isnan(c.dev[1]).nonzero().tolist()
    assert bad == [[int(c.table[0, 1]), 0, 1]]
    assert tl.tern_device_status() == 0


def test_append_refusals_of_the_binding(tl):
    import torch
    c = Cache([5], [2], 2, 64)
    k = torch.zeros(2, 2, 64, device="cuda")
    q = torch.zeros(2, 4, 64, device="cuda")
    freq = _table(tl, 64)[0]
    call = lambda q=q, k=k, v=k, freq=freq, **kw: tl.tern_kv8_append_rope(  # noqa: E731
        q, k, v, *c.dev, freq, **kw)
    with pytest.raises(ValueError):
        call(q=q.bfloat16())
    with pytest.raises(ValueError):
        call(q=q[:1])
    with pytest.raises(ValueError):
        call(q_out=torch.zeros_like(q))
    with pytest.raises(ValueError):
        call(q=None, q_out=q.bfloat16())
    with pytest.raises(ValueError):
        call(v=k.half())
    with pytest.raises(ValueError):
        call(positions=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(tl.TernError):
        call(freq=_table(tl, 128)[0])


def test_as_many_tokens_as_a_call_can_name(tl):
    """2^31 - 1 of one head of 16, in place: tokens, units and bytes past 31 bits."""
    import torch
    T = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 78 GB")
    x = torch.zeros(T, 1, 16, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    at = [0, 1, 2 ** 30 + 5, T - 64, T - 2, T - 1]
    rows = torch.randn(len(at), 1, 16, device="cuda").bfloat16()
    places = torch.arange(7, 7 + len(at), dtype=torch.int32, device="cuda") * 1000
    for i, row, place in zip(at, rows, places):
        x[i], pos[i] = row, place
    freq, _ = tl.tern_rope_frequencies(16)
    tl.tern_rope(x, pos, freq, out=x)
    assert torch.equal(torch.stack([x[i] for i in at]), tl.tern_rope(rows, places, freq))
    assert not x[2:2000].any() and not x[T - 63:T - 2].any()
    del x, pos
    torch.cuda.empty_cache()
