"""GPU parity of tern_kv8_attention against the fp64 oracle (oracle/decoder.py).

Bar, from what the kernels round (u16 = 2^-11, fp16's unit roundoff):
- the weights are rounded to fp16 for their products with the values:
  u16 * A, A = sum_j p_j |v_j|;
- a score is an fp32 sum of at most 128 exact products times fp32 factors:
  its error is below 2^-16 * sum|q k| scale, at most 2^-16 * 40 here, which
  moves every weight, and the sum that divides them, by that factor:
  2 * 40 * 2^-16 < 2.5 u16 together with the exponential's 2^-22;
- the sums over n <= 8192 tokens in fp32: below n * 2^-24 = u16;
- the output's rounding: 2^-8 |o| in bf16, half of it here beside the first
  term (A >= |o|, which is 8 u16 of the two together at A = |o|); 2^-11 |o| (and
  half the smallest subnormal, 2^-25) in fp16.
So |o - o_ref| <= 5 * 2^-11 * A + 2^-9 |o| + 2^-25, and the log-sum-exp, which
has only the scores' errors, is within 2.5 * 2^-11 of the oracle's.
"""
import numpy as np
import pytest

from oracle import decoder as od

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tl():
    import torch
    import ternary_weight_linear_gb300 as tl
    tl.build()
    tl.load()
    torch.cuda.init()
    return tl


class Case:
    """A batch: tables with rubbish in unused entries, stale codes past the
    last token, stale scales (NaN) in unused pages."""

    def __init__(self, lens, new, heads, kv_heads, dim, dtype="bfloat16", seed=0, spread=0.3,
                 q_scale=1.0):
        import torch
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, dtype=np.int32)
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        each = [(n + 63) // 64 for n in lens]
        pages = sum(each) + 2
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.full((len(lens), max(1, max(each)) + 1), -5, dtype=np.int32)
        at = 0
        for b, e in enumerate(each):
            self.table[b, :e] = order[at:at + e]
            at += e
        self.codes = np.clip(np.rint(rng.standard_normal((pages, 2, kv_heads, 64, dim)) * 40), -127,
                             127).astype(np.int8)
        # block scales that differ by their spread
        self.scales = (0.02 * np.exp(spread * rng.standard_normal((pages, 2, kv_heads)))).astype(
            np.float32)
        self.scales[order[at:]] = np.nan
        rows = int(self.start[-1])
        self.q_dev = (torch.from_numpy(rng.standard_normal((rows, heads, dim)).astype(np.float32))
                      * q_scale).cuda().to(getattr(torch, dtype))
        self.heads, self.dim = heads, dim
        self.max_new = int(max(new))

    def run(self, tl, window=0, sinks=0, scale=None, q=None, **kw):
        import torch
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        kw.setdefault("max_new", self.max_new)
        return tl.tern_kv8_attention(
            self.q_dev if q is None else q, up(self.codes), up(self.scales), up(self.table),
            up(self.start), up(self.lens), window=window, sinks=sinks, softmax_scale=scale, **kw)

    def check(self, tl, window=0, sinks=0, scale=None, status=0, **kw):
        import torch
        rows = self.q_dev.shape[0]
        lse = torch.full((rows, self.heads), 7.0, device="cuda")
        out = self.run(tl, window, sinks, scale, lse=lse, **kw)
        torch.cuda.synchronize()
        assert tl.tern_device_status() == status
        q = self.q_dev.float().cpu().numpy().astype(np.float64)
        ref, ref_lse, absum = od.kv8_attention(q, self.codes, self.scales, self.table, self.start,
                                               self.lens, window, sinks,
                                               self.dim ** -0.5 if scale is None else scale)
        got = out.float().cpu().numpy().astype(np.float64)
        bound = 5 * 2.0 ** -11 * absum + 2.0 ** -9 * np.abs(ref) + 2.0 ** -25
        err = np.abs(got - ref)
        bad = ~(err <= bound)
        assert not bad.any(), (int(bad.sum()), float(np.max(err / bound)),
                               np.argwhere(bad)[:4].tolist())
        ll = lse.cpu().numpy()
        none = np.isneginf(ref_lse)
        assert np.array_equal(np.isneginf(ll), none)
        assert np.all(np.abs(ll[~none] - ref_lse[~none]) <= 2.5 * 2.0 ** -11)
        return out


# new rows x group: one tile's corner, a full tile, one row more, two tiles,
# several; sequences of one token, page ends, nothing new, nothing at all
LENS = [1, 63, 64, 65, 0, 200, 130, 77]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv", [(4, 4), (6, 1), (8, 2), (20, 1)])
@pytest.mark.parametrize("m", [1, 3])
def test_few_rows(tl, dim, heads, kv, m):
    new = [min(m, n) for n in LENS]
    new[-1] = 0
    Case(LENS, new, heads, kv, dim, seed=heads + m).check(tl)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv,lens,new", [
    (6, 1, [40], [40]),                     # a prompt from nothing, not a whole tile
    (2, 1, [64, 129], [64, 65]),
    (4, 4, [300, 1, 0, 171], [130, 1, 0, 33]),  # mixed with decode and empty
    (12, 2, [260], [150]),
    (1, 1, [700, 513], [257, 513]),
    (64, 1, [90], [11]),                    # the largest group
])
def test_many_rows(tl, dim, heads, kv, lens, new):
    Case(lens, new, heads, kv, dim, seed=heads + len(lens)).check(tl)


@pytest.mark.parametrize("dim,heads,kv", [(128, 6, 2), (64, 4, 4)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 2), (64, 0), (64, 64), (100, 70),
                                          (1000, 10), (31, 300), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_windows_and_sinks(tl, dim, heads, kv, window, sinks):
    Case([400, 333, 64, 5], [3, 1, 2, 5], heads, kv, dim, seed=window % 97).check(
        tl, window, sinks)
    Case([400, 333], [140, 333], heads, kv, dim, seed=window % 89).check(tl, window, sinks)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_types_and_scale(tl, dtype):
    Case([200, 90], [2, 70], 8, 2, 128, dtype=dtype, seed=11).check(tl, scale=0.05)


@pytest.mark.parametrize("m", [1, 60])
def test_long_context_is_split_and_reproducible(tl, m):
    """One sequence over many CTAs: joined in a fixed order."""
    import torch
    c = Case([8000], [m], 4, 1, 128, seed=21)
    a = c.check(tl)
    ws = torch.zeros(tl.tern_kv8_attention_workspace_bytes(1, m, 4, 1, 128), dtype=torch.uint8,
                     device="cuda")
    for _ in range(3):
        assert torch.equal(a, c.run(tl, workspace=ws))
    assert not ws[:tl.SYNC_BYTES].any()


@pytest.mark.parametrize("m", [1, 5, 10])
def test_long_batch_on_shared_pages(tl, m):
    """A batch long enough that CTAs take further ranges as they finish (the
    sequences share pages, as after a common prefix): the same bits each time,
    and a workspace that is left as it was found."""
    import torch
    seqs, rng = 30, np.random.default_rng(61)
    c = Case([8192], [m], 32, 16, 64, seed=62)
    lens = [8192 - 37 * b for b in range(seqs)]
    c.table = np.stack([rng.permutation(c.table[0, :128]) for _ in range(seqs)]).astype(np.int32)
    c.lens = np.asarray(lens, dtype=np.int32)
    c.start = (np.arange(seqs + 1) * m).astype(np.int32)
    c.q_dev = torch.randn(seqs * m, 32, 64, device="cuda").bfloat16()
    a = c.check(tl)
    ws = torch.zeros(tl.tern_kv8_attention_workspace_bytes(seqs, seqs * m, 32, 16, 64),
                     dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(a, c.run(tl, workspace=ws))
    assert not ws[:tl.SYNC_BYTES].any()


@pytest.mark.parametrize("dim,heads,kv,m", [(128, 6, 1, 4), (64, 40, 8, 5), (64, 32, 8, 5),
                                               (128, 34, 2, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (3000, 70)])
def test_three_tiles_of_rows(tl, dim, heads, kv, m, window, sinks):
    """17 to 25 rows per key-value head of a long batch, on shared pages."""
    import torch
    seqs, rng = -(-7000 // (46 * kv)), np.random.default_rng(66)
    c = Case([3200], [m], heads, kv, dim, seed=67)
    c.table = np.stack([rng.permutation(c.table[0, :50]) for _ in range(seqs)]).astype(np.int32)
    c.lens = (3200 - rng.integers(0, 300, seqs)).astype(np.int32)
    c.lens[1] = 0
    new = np.minimum(m, c.lens)
    new[2] = min(1, m - 1)
    c.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    c.q_dev = torch.randn(int(c.start[-1]), heads, dim, device="cuda").bfloat16()
    c.check(tl, window, sinks)
    # (25 rows: the kernel for more rows, beside the one for sequences of few)
    assert tl.tern_last_launches() == -(-seqs // 128) + (m * heads // kv > 24)


@pytest.mark.parametrize("m", [20, 70])
def test_last_wave_in_parts(tl, m):
    """Blocks of rows that outnumber the SMs by a few: the last ones are cut."""
    import torch
    c = Case([2500, 2400, 2300, 2200, 2100], [m] * 5, 32, 32, 64, seed=63)
    a = c.check(tl)
    ws = torch.zeros(tl.tern_kv8_attention_workspace_bytes(5, 5 * m, 32, 32, 64),
                     dtype=torch.uint8, device="cuda")
    for _ in range(2):
        assert torch.equal(a, c.run(tl, workspace=ws))
    assert not ws[:tl.SYNC_BYTES].any()


@pytest.mark.parametrize("m", [20, 70])
def test_blocks_of_more_pages_than_records(tl, m):
    """More than 512 pages for a block of rows that is not cut into parts (the
    sequences share pages); the sums' error grows with the n tokens, n * 2^-24
    of A beside the others'."""
    import torch
    seqs, n, rng = 20, 33500, np.random.default_rng(64)
    c = Case([3200], [m], 8, 8, 64, seed=65)
    c.table = rng.permuted(np.tile(c.table[0, :50], (seqs, 11)), axis=1)[:, :530]
    c.lens = (n - 64 * np.arange(seqs)).astype(np.int32)
    c.start = (np.arange(seqs + 1) * m).astype(np.int32)
    c.q_dev = torch.randn(seqs * m, 8, 64, device="cuda").bfloat16()
    out = c.run(tl)
    torch.cuda.synchronize()
    assert tl.tern_device_status() == 0
    assert torch.equal(out, c.run(tl))
    for b in (0, seqs - 1):
        rows = slice(b * m, (b + 1) * m)
        q = c.q_dev[rows].float().cpu().numpy().astype(np.float64)
        ref, _, absum = od.kv8_attention(q, c.codes, c.scales, c.table[b:b + 1],
                                         np.asarray([0, m], np.int32), c.lens[b:b + 1], 0, 0,
                                         64 ** -0.5)
        err = np.abs(out[rows].float().cpu().numpy() - ref)
        assert np.all(err <= (5 * 2.0 ** -11 + n * 2.0 ** -24) * absum + 2.0 ** -9 * np.abs(ref)
                      + 2.0 ** -25)


def test_more_sequences_than_one_launch_takes(tl):
    lens = [(31 * i) % 190 for i in range(300)]
    Case(lens, [min(1 + i % 2, n) for i, n in enumerate(lens)], 2, 1, 64, seed=31).check(tl)


@pytest.mark.parametrize("new", [[2, 3], [80, 3]])
def test_strided_queries(tl, new):
    """Queries as a slice of a fused projection's output."""
    import torch
    c = Case([150, 40], new, 4, 2, 64, seed=41)
    wide = torch.randn(c.q_dev.shape[0], 9, 64, device="cuda").bfloat16()
    wide[:, 2:6] = c.q_dev
    want = c.check(tl)
    assert torch.equal(want, c.run(tl, q=wide[:, 2:6]))
    by_head = c.q_dev.transpose(0, 1).contiguous().transpose(0, 1)  # [heads][rows] in memory
    assert torch.equal(want, c.run(tl, q=by_head))


@pytest.mark.parametrize("new", [[2, 1, 4], [1, 1, 9], [100, 1, 90]])
def test_value_scales_of_the_whole_range(tl, new):
    """Value blocks of 2^-100, 1 and 2^100 times the usual scale in one sequence."""
    c = Case([400, 300, 90], new, 4, 2, 128, seed=53)
    rng = np.random.default_rng(54)
    c.scales[:, 1] *= (2.0 ** rng.choice([-100, 0, 100], c.scales[:, 1].shape)).astype(np.float32)
    c.check(tl)


@pytest.mark.parametrize("new", [[2, 1, 4], [100, 1, 90]])
def test_value_scales_far_apart(tl, new):
    """Blocks whose scales differ by up to 2^40, with zero blocks among them."""
    c = Case([400, 300, 90], new, 4, 2, 128, seed=51)
    rng = np.random.default_rng(52)
    c.scales = (0.02 * 2.0 ** rng.uniform(-14, 6, c.scales.shape)).astype(np.float32)
    c.scales[:, 0] = 0.02
    zero = rng.random(c.scales.shape) < 0.2
    c.scales[zero] = 0
    c.codes[zero] = 0
    c.check(tl)


@pytest.mark.parametrize("new", [[2, 3], [70, 40]])
def test_query_magnitudes(tl, new):
    """Rows of very large and small queries: the scores stay in range by the
    softmax scale, the row's own power of two keeps the codes' products exact."""
    import torch
    c = Case([150, 90], new, 4, 2, 64, seed=61)
    f = torch.full((c.q_dev.shape[0], 1, 1), 2.0 ** -20, device="cuda")
    f[::2] = 2.0 ** -60
    f[1] = 1.0
    c.q_dev = (c.q_dev.float() * f).bfloat16()
    c.q_dev[0, 0] = 0
    c.check(tl)


@pytest.mark.parametrize("new", [[2, 3, 1], [70, 40, 65]])
def test_nan_stays_with_the_rows_that_see_it(tl, new):
    import torch
    c = Case([200, 150, 100], new, 4, 2, 128, seed=71)
    clean = c.run(tl)
    c.scales[c.table[1, 0], 1, 1] = np.nan  # sequence 1, value block 0, head 1
    got = c.run(tl)
    torch.cuda.synchronize()
    a, b = c.start[1], c.start[2]
    assert torch.isnan(got[a:b, 2:].float()).all()
    assert torch.equal(got[:a], clean[:a]) and torch.equal(got[b:], clean[b:])
    assert torch.equal(got[a:b, :2], clean[a:b, :2])
    # outside the window it is not seen
    w = c.run(tl, window=20)
    late = 150 - new[1] >= 64 + 20
    if late:
        assert not torch.isnan(w.float()).any()
    c.q_dev[0, 1, 3] = float("inf")
    got = c.run(tl)
    assert torch.isnan(got[0, 1].float()).all() and torch.equal(got[0, 0], clean[0, 0])


def test_windowed_rows_of_one_tile_see_different_pages(tl):
    """A NaN block seen by the first rows of a tile only."""
    import torch
    c = Case([300], [100], 2, 1, 64, seed=73)
    clean = c.run(tl, window=30)
    c.scales[c.table[0, 3], 1, 0] = np.nan  # tokens 192..255
    got = c.run(tl, window=30)
    p = torch.arange(200, 300, device="cuda")
    sees = p - 29 <= 255
    assert torch.isnan(got[sees].float()).all()
    assert torch.equal(got[~sees], clean[~sees])


@pytest.mark.parametrize("new", [[1, 2, 3], [90, 40, 3]])
def test_pages_out_of_range_read_as_masked(tl, new):
    c = Case([200, 150, 3], new, 4, 2, 64, seed=81)
    c.table[0, 1] = 10 ** 6
    c.table[2, 0] = -1  # a whole sequence: its rows are empty
    out = c.check(tl, status=-7)
    import torch
    assert not out[c.start[2]:].any() and tl.tern_device_status() == 0
    del torch


def test_inconsistent_sequences_are_skipped(tl):
    import torch
    for field, value in (("lens", -1), ("lens", 10 ** 6), ("lens", 1), ("start", -3),
                         ("start", 10 ** 6)):
        c = Case([200, 150, 90], [2, 3, 1], 4, 2, 64, seed=83)
        want = c.run(tl)
        getattr(c, field)[1] = value
        out = torch.full_like(want, 5.0)
        c.run(tl, out=out)
        assert tl.tern_device_status() == -7
        first = 0 if field == "start" else 2  # rows 0.. are also sequence 0's end
        if field == "lens":
            assert torch.equal(out[:2], want[:2]) and torch.equal(out[5:], want[5:])
        else:
            assert torch.equal(out[5:], want[5:])
        assert (out[max(first, 2):5] == 5.0).all()
    # more new tokens than max_new
    c = Case([200, 150], [2, 3], 4, 2, 64, seed=84)
    want = c.run(tl)
    out = torch.full_like(want, 5.0)
    c.run(tl, out=out, max_new=2)
    assert tl.tern_device_status() == -7
    assert torch.equal(out[:2], want[:2]) and (out[2:] == 5.0).all()


def test_pool_past_four_gigabytes(tl):
    """Pages whose bytes start past 2^32."""
    import torch
    heads, kv, dim = 16, 8, 128
    small = Case([150, 70], [2, 70], heads, kv, dim, seed=91)
    pages, per = small.codes.shape[0], 2 * kv * 64 * dim
    shift = (1 << 32) // per + 5
    codes = torch.empty(shift + pages, 2, kv, 64, dim, dtype=torch.int8, device="cuda")
    scales = torch.empty(shift + pages, 2, kv, device="cuda")
    codes[shift:] = torch.from_numpy(small.codes).cuda()
    scales[shift:] = torch.from_numpy(small.scales).cuda()
    table = torch.from_numpy(np.where(small.table >= 0, small.table + shift, -5)).int().cuda()
    start, lens = (torch.from_numpy(a).cuda() for a in (small.start, small.lens))
    got = tl.tern_kv8_attention(small.q_dev, codes, scales, table, start, lens,
                                max_new=small.max_new)
    assert torch.equal(got, small.check(tl))
    k = torch.randn(72, kv, dim, device="cuda")
    c2, s2 = torch.from_numpy(small.codes).cuda(), torch.from_numpy(small.scales).cuda()
    tl.tern_kv8_append(k, k, codes, scales, table, start, lens)
    tl.tern_kv8_append(k, k, c2, s2, torch.from_numpy(small.table).cuda(), start, lens)
    assert torch.equal(codes[shift:], c2)
    assert torch.equal(scales[shift:].nan_to_num(-1), s2.nan_to_num(-1))


@pytest.mark.parametrize("new", [[1, 1], [60, 1]])
def test_captured_call_follows_the_index_arrays(tl, new):
    """A captured call replays with other lengths, tables and queries."""
    import torch
    c = Case([130, 100], new, 4, 2, 64, seed=101)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    q, codes, scales = c.q_dev.clone(), up(c.codes), up(c.scales)
    table, start, lens = up(c.table), up(c.start), up(c.lens)
    ws = torch.zeros(tl.tern_kv8_attention_workspace_bytes(2, q.shape[0], 4, 2, 64),
                     dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)

    def call():
        tl.tern_kv8_attention(q, codes, scales, table, start, lens, max_new=max(new), out=out,
                              workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    lens[0] = 99
    q.mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    c.lens[0] = 99
    c.q_dev = q
    assert torch.equal(out, c.run(tl))


def test_another_stream(tl):
    import torch
    c = Case([130, 100], [2, 40], 4, 2, 64, seed=111)
    want = c.run(tl)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = c.run(tl, stream=s)
        s.synchronize()
        assert torch.equal(got, want)
    got = c.run(tl, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want)


def test_argument_errors(tl):
    import torch
    c = Case([130], [2], 4, 2, 64, seed=121)
    assert c.run(tl, q=c.q_dev[:0]).shape == (0, 4, 64)
    for bad in (c.q_dev.float(), c.q_dev[..., :32], c.q_dev[0], c.q_dev.cpu(),
                c.q_dev.transpose(1, 2)):
        with pytest.raises(ValueError):
            c.run(tl, q=bad)
    for kw in (dict(window=-1), dict(sinks=-1), dict(scale=0.0), dict(max_new=0),
               dict(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda")),
               dict(q=c.q_dev[:, :3].contiguous())):
        with pytest.raises(tl.TernError):
            c.run(tl, **kw)
    with pytest.raises(ValueError):
        c.run(tl, out=torch.empty(2, 4, 64, device="cuda"))
    with pytest.raises(ValueError):
        c.run(tl, lse=torch.empty(2, 4, dtype=torch.float16, device="cuda"))
