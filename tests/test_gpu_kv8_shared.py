"""GPU parity of tern_kv8_attention_shared against the fp64 oracle of the
attention over each sequence's whole table (oracle/decoder.py).

Bar: that of test_gpu_kv8_attention.py.  The join of the prefix's and the own
tokens' parts adds to it only what fp32 log-sum-exps round: at most 3 * 2^-24 of
a log-sum-exp below 64 in size, 2^-16 of a part's weight, which the 5 * 2^-11
there (4.5 of them in use) covers.

One more term, for rows whose weight lies on tokens of small codes, where that
bar is small: the values enter as code + 128 and -128 times the weights.  Within
half a page's products the sums are at most 255 sum_j p_j v_scale_j in size and
pass four tensor instructions (two of codes, two of the bias), each of which may
cut 2^-23 of them: 4 * 255 * 2^-23 < 2^-13 times sum_j p_j v_scale_j over all
tokens, beside sums of the size of the codes that are counted above.
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
    """A batch whose sequences begin with the same pages.  own, new: tokens of
    each sequence behind the shared ones, and how many of them are new (own None:
    an empty sequence).  Rubbish in unused table entries, stale codes past the
    last token, NaN scales in unused pages; `gap` rows of no sequence before the
    first and behind the last."""

    def __init__(self, shared, own, new, heads, kv_heads, dim, dtype="bfloat16", seed=0, spread=0.3,
                 q_scale=1.0, gap=0):
        import torch
        rng = np.random.default_rng(seed)
        self.shared, self.heads, self.dim = shared, heads, dim
        self.lens = np.array([0 if n is None else shared + n for n in own], np.int32)
        self.start = (gap + np.concatenate([[0], np.cumsum(new)])).astype(np.int32)
        common = shared // 64
        each = [0 if n is None else (n + 63) // 64 for n in own]
        pages = common + sum(each) + 2
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.full((len(own), common + max(1, max(each)) + 1), -5, np.int32)
        self.table[:, :common] = order[:common]
        at = common
        for b, e in enumerate(each):
            self.table[b, common:common + e] = order[at:at + e]
            at += e
        self.codes = np.clip(np.rint(rng.standard_normal((pages, 2, kv_heads, 64, dim)) * 40), -127,
                             127).astype(np.int8)
        self.scales = (0.02 * np.exp(spread * rng.standard_normal((pages, 2, kv_heads)))).astype(
            np.float32)
        self.scales[order[at:]] = np.nan
        self.rows = int(self.start[-1]) + gap
        self.q_dev = (torch.from_numpy(rng.standard_normal((self.rows, heads, dim)).astype(
            np.float32)) * q_scale).cuda().to(getattr(torch, dtype))
        self.max_new = int(max(new))

    def args(self):
        import torch
        return [torch.from_numpy(np.ascontiguousarray(a)).cuda()
                for a in (self.codes, self.scales, self.table, self.start, self.lens)]

    def run(self, tl, window=0, sinks=0, scale=None, q=None, **kw):
        kw.setdefault("max_new", self.max_new)
        return tl.tern_kv8_attention_shared(self.q_dev if q is None else q, *self.args(),
                                            self.shared, window=window, sinks=sinks,
                                            softmax_scale=scale, **kw)

    def check(self, tl, window=0, sinks=0, scale=None, status=0, skipped=(), **kw):
        import torch
        lse = torch.full((self.rows, self.heads), 7.0, device="cuda")
        out = torch.full((self.rows, self.heads, self.dim), 9.0, dtype=self.q_dev.dtype,
                         device="cuda")
        self.run(tl, window, sinks, scale, lse=lse, out=out, **kw)
        torch.cuda.synchronize()
        assert tl.tern_device_status() == status
        lens, start = self.lens.copy(), self.start
        live = np.zeros(self.rows, bool)
        for b in range(len(lens)):
            if b not in skipped:
                live[start[b]:start[b + 1]] = True
        q = self.q_dev.double().cpu().numpy()
        ref, ref_lse, absum = od.kv8_attention(q, self.codes, self.scales, self.table, start,
                                               np.where(np.isin(np.arange(len(lens)), skipped),
                                                        np.maximum(np.diff(start), 1), lens),
                                               window, sinks,
                                               self.dim ** -0.5 if scale is None else scale)
        ones = self.codes.copy()
        ones[:, 1] = 1  # sum_j p_j v_scale_j
        scales = od.kv8_attention(q, ones, self.scales, self.table, start,
                                  np.where(np.isin(np.arange(len(lens)), skipped),
                                           np.maximum(np.diff(start), 1), lens), window, sinks,
                                  self.dim ** -0.5 if scale is None else scale)[2]
        got = out.double().cpu().numpy()
        assert np.all(got[~live] == 9) and np.all(lse.cpu().numpy()[~live] == 7)
        bound = 5 * 2.0 ** -11 * absum + 2.0 ** -9 * np.abs(ref) + 2.0 ** -25
        bound = bound + 2.0 ** -13 * scales
        err = np.abs(got - ref)
        bad = ~(err <= bound) & live[:, None, None]
        assert not bad.any(), (int(bad.sum()), float(np.max((err / bound)[live])),
                               np.argwhere(bad)[:4].tolist())
        ll = lse.cpu().numpy()[live]
        ref_lse = ref_lse[live]
        none = np.isneginf(ref_lse)
        assert np.array_equal(np.isneginf(ll), none)
        assert np.all(np.abs(ll[~none] - ref_lse[~none]) <= 2.5 * 2.0 ** -11)
        return out, lse


OWN = [1, 63, 64, 65, None, 200, 130, 77]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv", [(4, 4), (6, 1), (16, 2), (20, 1)])
@pytest.mark.parametrize("m", [1, 3])
@pytest.mark.parametrize("shared", [64, 1088])
def test_few_rows(tl, dim, heads, kv, m, shared):
    new = [0 if n is None else min(m, n) for n in OWN]
    new[-1] = 0
    Case(shared, OWN, new, heads, kv, dim, seed=heads + m).check(tl)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("seqs,m,group", [(2, 1, 1), (9, 1, 7), (11, 1, 6), (21, 1, 6), (22, 2, 6),
                                          (43, 1, 6), (130, 1, 4), (300, 1, 2)])
def test_rows_of_the_batch(tl, dim, seqs, m, group):
    """Rows per key-value head on both sides of 64, 128 and 256, several blocks
    of them, more sequences than a launch of the few-row kernel takes."""
    own = [m + (17 * b) % 90 for b in range(seqs)]
    Case(704, own, [m] * seqs, 2 * group, 2, dim, seed=seqs).check(tl)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("shared", [64 * 7, 64 * 8, 64 * 33, 64 * 150])
def test_lengths_of_the_prefix(tl, dim, shared):
    """Too short to be cut, cut in parts of different lengths, long."""
    Case(shared, [5, 70, 9], [1, 1, 2], 12, 2, dim, seed=shared).check(tl)
    Case(shared, [30] * 20, [2] * 20, 8, 1, dim, seed=shared).check(tl)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [[6, 4, 1], [20, 1, 0], [100, 7, 1], [300, 280, 1]])
def test_verify_steps_and_prompt_chunks(tl, dim, new):
    """Rows of a sequence for the few-row kernel, the split and the plain form of
    the one on the tensor cores, and mixed."""
    Case(640, [m + 90 for m in new], new, 12, 2, dim, seed=new[0]).check(tl)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("shared,new,launches", [
    (640, [100] + [1] * 20, 3), (640, [11] + [1] * 9 + [0, 2], 3), (64 * 90, [300, 40] + [1] * 14, 4),
    (64 * 90, [1] * 30 + [64], 4), (640, [2] * 6, 2), (64 * 90, [2] * 40, 3), (640, [60, 50, 1], 2),
    (64, [3], 1)])
def test_mixed_batches_and_which_launches(tl, dim, shared, new, launches):
    """Prompt chunks among decode steps: shared where those are many, each for
    itself otherwise; a launch for the prefix where it is long for the rows, one
    for the spans, one for the chunks' own tokens, the join."""
    c = Case(shared, [m + 70 for m in new], new, 12, 2, dim, seed=len(new))
    c.check(tl)
    c.run(tl)
    assert tl.tern_last_launches() == launches
    if launches > 2:
        c.check(tl, window=shared - 30, sinks=70)


# (shared tokens, sequences, new tokens, columns of the table behind the shared pages)
@pytest.mark.parametrize("shared,seqs,m,columns,shares", [
    (64, 32, 1, 2000, True), (64, 5, 2, 128, True), (64, 5, 2, 129, False), (512, 5, 2, 300, True),
    (64, 5, 4, 72, True), (64, 5, 4, 73, False), (512, 5, 4, 128, True), (512, 5, 4, 129, False),
    (512, 5, 5, 16, True), (512, 5, 5, 17, False), (512, 5, 8, 8, True), (512, 5, 8, 9, False),
    (512, 5, 10, 4, True), (512, 5, 10, 5, False), (64, 2, 10, 320, False),
    (64, 704, 1, 2, True), (64, 705, 1, 2, False), (64, 448, 2, 2, True), (64, 449, 2, 2, False),
    (0, 3, 1, 2, False), (64, 1, 1, 2, False)])
def test_what_does_not_gain_reads_each_for_itself(tl, shared, seqs, m, columns, shares):
    """Where the table is too wide for the rows and the prefix, or the sequences too
    many for it, the ordinary kernels run, with their very bits; 6 query heads."""
    import torch
    c = Case(shared, [m + 7 * (b % 9) for b in range(seqs)], [m] * seqs, 6, 1, 64, seed=columns)
    wide = np.full((seqs, shared // 64 + columns), -7, np.int32)
    n = min(wide.shape[1], c.table.shape[1])
    wide[:, :n] = c.table[:, :n]
    c.table = wide
    out, lse = c.check(tl)
    c.run(tl)
    launches = tl.tern_last_launches()
    lse2 = torch.full_like(lse, 7.0)
    whole = tl.tern_kv8_attention(c.q_dev, *c.args(), max_new=c.max_new, lse=lse2)
    assert (torch.equal(out, whole) and torch.equal(lse, lse2)) == (not shares)
    if not shares:
        assert launches == tl.tern_last_launches()


@pytest.mark.parametrize("seqs,columns,shares", [(128, 3, True), (129, 3, False), (40, 128, True),
                                                 (40, 129, False)])
def test_a_chunk_among_too_many_or_in_too_wide_a_table(tl, seqs, columns, shares):
    """66 rows of one sequence, 6 of the others, behind a page: 16 * (1 + 7) sequences and
    own pages at most."""
    import torch
    new = [11] + [1] * (seqs - 1)
    c = Case(64, [m + 7 * (b % 9) for b, m in enumerate(new)], new, 6, 1, 64, seed=columns)
    wide = np.full((seqs, 1 + columns), -7, np.int32)
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    out, lse = c.check(tl)
    lse2 = torch.full_like(lse, 7.0)
    whole = tl.tern_kv8_attention(c.q_dev, *c.args(), max_new=c.max_new, lse=lse2)
    assert (torch.equal(out, whole) and torch.equal(lse, lse2)) == (not shares)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 0), (130, 7), (400, 64), (600, 100),
                                          (900, 65), (100, 2000), (5000, 3)])
def test_windows(tl, dim, window, sinks):
    """From windows within the own tokens (no prefix token seen, or its sinks
    alone) to ones that reach over all of it."""
    Case(640, [40, 3, 150, 300], [2, 1, 3, 1], 12, 2, dim, seed=window).check(tl, window, sinks)
    own = [200 + 9 * b for b in range(25)]
    Case(640, own, [2] * 25, 12, 2, dim, seed=window).check(tl, window, sinks)


def test_windows_over_a_cut_prefix(tl):
    Case(64 * 60, [40, 800, 70], [1, 2, 1], 12, 2, 128, seed=1).check(tl, 2000, 70)
    Case(64 * 60, [40 + b for b in range(40)], [2] * 40, 12, 2, 64, seed=2).check(tl, 1500, 129)


@pytest.mark.parametrize("seqs,m,group,longest", [(40, 4, 5, 200), (30, 1, 6, 1500),
                                                  (36, 1, 2, 900), (9, 2, 12, 2000)])
def test_spans_beside_the_prefix(tl, seqs, m, group, longest):
    """More sequences and heads than the SMs beside the prefix hold spans, and own
    tokens of very different lengths, a few of them cut."""
    own = [m + (b * b * 37) % longest if b % 3 else m for b in range(seqs)]
    c = Case(64 * 40, own, [m] * seqs, 8 * group, 8, 64, seed=longest)
    c.check(tl)
    c.check(tl, window=1700, sinks=40)


def check_twice(tl, c, launches, **kw):
    """Against the oracle on a workspace that is kept, and again, bit for bit."""
    import torch
    kv = c.codes.shape[2]
    ws = torch.zeros(tl.tern_kv8_attention_shared_workspace_bytes(len(c.lens), c.rows, c.heads, kv,
                                                                  c.dim),
                     dtype=torch.uint8, device="cuda")
    first, _ = c.check(tl, workspace=ws, **kw)
    assert tl.tern_last_launches() == launches
    assert torch.equal(c.run(tl, workspace=ws, **kw), first)
    assert not ws[:tl.SYNC_BYTES].any()


@pytest.mark.parametrize("group,m,shared,tokens,launches", [
    (3, 1, 512, 11000, 2), (9, 1, 512, 8000, 2), (17, 1, 1280, 5500, 3), (5, 4, 1280, 5500, 3)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 10)])
def test_spans_of_more_pages_than_records(tl, group, m, shared, tokens, launches, window, sinks):
    """16 sequences of `tokens` and up to 1.4 times as many, 8 heads of them: 26000,
    19000 and 13000 pages for 608, 456 and 304 resident spans, 40 and more for each,
    whose records are held 32 at a time.  The window is nine tenths of them."""
    own = [tokens + tokens // 40 * b for b in range(16)]
    window, sinks = tokens * window // 10, 10 * sinks
    c = Case(shared, own, [m] * 16, 8 * group, 8, 64, seed=group)
    check_twice(tl, c, launches, window=window, sinks=sinks)


@pytest.mark.parametrize("long", [3000, 6100])
def test_more_parts_than_the_workspace_holds(tl, long):
    """300 rows of 48 heads leave room for 40960 / 14400 = 2 parts of own tokens; the
    long sequence's pages, 3 and 5 times the quota of all, go into those."""
    own = [20] * 300
    own[137] = long
    c = Case(64 * 10, own, [1] * 300, 48, 8, 64, seed=long)
    check_twice(tl, c, 3)
    check_twice(tl, c, 3, window=1700, sinks=10)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1400, 0), (1500, 700)])
def test_chunks_whose_own_tokens_are_cut(tl, dim, window, sinks):
    """Chunks of more than 64 rows over 25 to 60 pages of their own (cut from 16 on)
    among single tokens, whose parts of the own tokens are joined once more."""
    own = [1700] + [30] * 12 + [3800, 1530] + [70] * 15
    c = Case(640, own, [40] + [1] * 12 + [33, 11] + [1] * 15, 12, 2, dim, seed=window)
    check_twice(tl, c, 3, window=window, sinks=sinks)  # spans (the prefix's too), chunks, join


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_types_and_strides(tl, dtype):
    """Queries within a projection's rows."""
    import torch
    c = Case(256, [9, 30, 64], [3, 1, 2], 8, 2, 64, dtype, seed=3)
    wide = torch.zeros(c.rows, 12, 64, dtype=c.q_dev.dtype, device="cuda")
    wide[:, 2:10] = c.q_dev
    out, lse = c.check(tl)
    out2, lse2 = c.check(tl, q=wide[:, 2:10])
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("seqs", [4, 30])
def test_rows_of_no_sequence_are_left(tl, seqs):
    Case(320, [20] * seqs, [2] * seqs, 8, 1, 128, gap=5, seed=4).check(tl)
    Case(64 * 40, [20] * seqs, [2] * seqs, 8, 1, 64, gap=37, seed=4).check(tl)


@pytest.mark.parametrize("shared", [192, 64 * 40])
@pytest.mark.parametrize("seqs", [5, 30])
def test_inconsistent_sequences_are_skipped(tl, shared, seqs):
    """One whose new tokens reach into the prefix, one too long for its table."""
    c = Case(shared, [20] * seqs, [2] * seqs, 8, 1, 64, seed=5)
    c.lens[1] = shared + 1
    c.lens[3] = 10 ** 6
    c.check(tl, status=-7, skipped=[1, 3])
    c = Case(shared, [20] * seqs, [2] * seqs, 8, 1, 64, seed=5)
    c.lens[:] = 3
    c.check(tl, status=-7, skipped=list(range(seqs)))


def test_a_lone_sequence(tl):
    Case(256, [30], [2], 8, 2, 64, seed=6).check(tl)
    c = Case(256, [30], [2], 8, 2, 64, seed=6)
    c.lens[0] = 257
    c.check(tl, status=-7, skipped=[0])
    Case(0, [30, 5, 100], [2, 1, 1], 8, 2, 64, seed=6).check(tl)


@pytest.mark.parametrize("shared,new", [(0, [2, 1, 1]), (256, [2]), (256, [70])])
def test_the_ordinary_workspace_where_nothing_is_shared(tl, shared, new):
    import torch
    c = Case(shared, [m + 30 for m in new], new, 8, 2, 64, seed=6)
    need = tl.tern_kv8_attention_workspace_bytes(len(new), c.rows, 8, 2, 64)
    held = torch.zeros(need + 4096, dtype=torch.uint8, device="cuda")
    held[need:] = 77
    c.check(tl, workspace=held[:need])
    assert (held[need:] == 77).all()


def test_first_sequence_without_tokens(tl):
    """Its row of the table still names the shared pages."""
    Case(320, [None, 30, 5], [0, 2, 1], 8, 2, 64, seed=7).check(tl)


@pytest.mark.parametrize("seqs", [3, 40])
def test_bad_pages(tl, seqs):
    """Out of range: masked and reported."""
    c = Case(64 * 20, [20] * seqs, [2] * seqs, 8, 2, 64, seed=8)
    c.table[:, 3] = 10 ** 6
    c.table[:, 19] = -1
    c.table[2, 20] = 10 ** 6  # the third sequence's own tokens, all of them
    c.check(tl, status=-7)
    c.table[:, :20] = -1  # nothing left of the prefix
    c.check(tl, status=-7)


@pytest.mark.parametrize("seqs", [3, 40])
def test_scales_that_cannot_be_used(tl, seqs):
    """A NaN block of the prefix: its head's rows that see it, and only they."""
    import torch
    c = Case(64 * 20, [400 + b for b in range(seqs)], [1] * seqs, 8, 2, 64, seed=9)
    c.scales[c.table[0, 4], 1, 1] = np.nan
    out = c.run(tl)
    assert torch.isnan(out[:, 4:]).all() and torch.isfinite(out[:, :4]).all()
    out = c.run(tl, window=1370)  # (page 4 is seen by the shorter ones alone)
    low = torch.from_numpy(c.lens - 1370).cuda() < 320
    assert torch.isnan(out[low][:, 4:]).all() and torch.isfinite(out[~low]).all()
    assert torch.isfinite(out[:, :4]).all()
    # and one of a sequence's own
    c = Case(64 * 20, [40] * seqs, [1] * seqs, 8, 2, 64, seed=9)
    c.scales[c.table[1, 20], 0, 0] = -1.0
    out = c.run(tl)
    assert torch.isnan(out[1, :4]).all() and torch.isfinite(out[1, 4:]).all()
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[2:]).all()


@pytest.mark.parametrize("seqs", [3, 40])
@pytest.mark.parametrize("dim", [64, 128])
def test_value_scales_far_apart(tl, seqs, dim):
    c = Case(64 * 30, [90] * seqs, [1] * seqs, 12, 2, dim, seed=10)
    rng = np.random.default_rng(0)
    c.scales[:, 1] *= (2.0 ** rng.integers(-20, 20, c.scales[:, 1].shape)).astype(np.float32)
    c.check(tl)
    c.scales[c.table[0, 5], 1] = 1e-20
    c.scales[c.table[1, 30], 1] = 0
    c.scales[c.table[2, 30], 1] = 1e-20
    c.check(tl)


def test_parts_of_very_different_weight(tl):
    """All of the softmax in the prefix, or all of it in the own tokens."""
    for big in (0, 1):
        c = Case(64 * 20, [40, 70, 64], [1, 1, 1], 12, 2, 128, seed=11)
        common = c.table[0, :20]
        rest = np.setdiff1d(np.arange(len(c.scales)), common)
        c.scales[(common, rest)[big], 0] *= 8
        c.check(tl)


def test_same_bits_as_before_and_the_workspace(tl):
    """Call after call, with a workspace of its own or one kept, and after other
    shapes have used it."""
    import torch
    cases = [Case(64 * 40, [40 + b for b in range(n)], [2] * n, 12, 2, 128, seed=12)
             for n in (3, 40)]
    need = max(tl.tern_kv8_attention_shared_workspace_bytes(len(c.lens), c.rows, 12, 2, 128)
               for c in cases)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    first = [c.run(tl) for c in cases]
    for _ in range(3):
        for c, want in zip(cases, first):
            assert torch.equal(c.run(tl, workspace=ws), want)
    assert not ws[:tl.SYNC_BYTES].any()
    assert tl.tern_device_status() == 0


def test_max_new_left_out(tl):
    c = Case(64 * 20, [40, 70, 64], [3, 1, 1], 12, 2, 64, seed=13)
    c.check(tl, max_new=None)


def test_captured_and_replayed_with_other_contents(tl):
    """Two graphs with workspaces of their own, replayed side by side on two
    streams, their lengths, tables and queries changed in between."""
    import torch
    cs = [Case(64 * 24, [100 + b for b in range(n)], [1] * n, 12, 2, 128, seed=n) for n in (4, 30)]
    held, graphs = [], []
    for c in cs:
        args = c.args()
        ws = torch.zeros(tl.tern_kv8_attention_shared_workspace_bytes(len(c.lens), c.rows, 12, 2,
                                                                      128),
                         dtype=torch.uint8, device="cuda")
        out = torch.empty_like(c.q_dev)
        q = c.q_dev.clone()
        call = lambda a=args, q=q, o=out, w=ws, s=c.shared: tl.tern_kv8_attention_shared(  # noqa: E731
            q, *a, s, max_new=1, out=o, workspace=w)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        held.append((args, q, out, ws))  # (what the graph's launches point to lives as long)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cs]
    for step in range(4):
        wants = []
        for c, (args, q, _, _) in zip(cs, held):
            c.lens = (c.lens - 7 * (step > 0)).astype(np.int32)
            c.q_dev = torch.randn_like(c.q_dev)
            args[4].copy_(torch.from_numpy(c.lens))
            q.copy_(c.q_dev)
            wants.append(c.run(tl))
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        for want, (_, _, out, _) in zip(wants, held):
            assert torch.equal(out, want)
    assert tl.tern_device_status() == 0


def test_refusals_of_the_binding(tl):
    c = Case(128, [20, 30], [1, 1], 8, 2, 64, seed=14)
    for shared in (-64, 100, 64 * 1000, 2 ** 40):
        c.shared = shared
        with pytest.raises(tl.TernError):
            c.run(tl)
