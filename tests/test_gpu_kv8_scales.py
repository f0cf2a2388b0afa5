"""Value blocks of one sequence whose scales lie far apart: a row's result is
that of the blocks that it sees and weighs, whatever else its call reads.

Bar: that of test_gpu_kv8_attention.py without its absolute term (outputs are
bf16 and far above its smallest value): 5 * 2^-11 * A + 2^-9 |o|, and 2.5 * 2^-11
for the log-sum-exp.
"""
import numpy as np
import pytest

from oracle import decoder as od
from test_gpu_kv8_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tl():
    import torch
    import ternary_weight_linear_gb300 as tl
    tl.build()
    tl.load()
    torch.cuda.init()
    return tl


def attention(q, codes, scales, pages, n, scale, window, sinks):
    """(out, sum_j p_j |v_j|, log sum_j exp(s_j)) of the last rows of one
    sequence of n tokens and one key-value head, in fp64: q [m, group, dim],
    codes [pages, 2, 64, dim], scales [pages, 2]; oracle.decoder's arithmetic on all rows at once."""
    m, group, dim = q.shape
    k, v = ((codes[pages, i].astype(np.float64) * scales[pages, i].astype(np.float64)[:, None, None])
            .reshape(-1, dim)[:n] for i in (0, 1))
    z = scale * (q.reshape(-1, dim).astype(np.float64) @ k.T).reshape(m, group, n)
    for i in range(m):
        z[i, :, ~od.visible(n - m + i, n, window, sinks)] = -np.inf
    big = z.max(-1, keepdims=True)
    p = np.exp(z - big)
    lse = (big + np.log(p.sum(-1, keepdims=True)))[..., 0]
    p = (p / p.sum(-1, keepdims=True)).reshape(-1, n)
    return (p @ v).reshape(q.shape), (p @ np.abs(v)).reshape(q.shape), lse


class Batch(Case):
    """seqs sequences of one length, which share their pages (one table)."""

    def __init__(self, seqs, n, m, heads, kv_heads, dim, seed, pool=None):
        import torch
        pages = (n + 63) // 64
        super().__init__([64 * min(pages, pool or pages)], [1], heads, kv_heads, dim, seed=seed)
        held = self.table.shape[1] - 1
        row = self.table[0, np.arange(pages) % held]
        self.table = np.tile(row, (seqs, 1)).astype(np.int32)
        self.lens = np.full(seqs, n, dtype=np.int32)
        self.start = (np.arange(seqs + 1) * m).astype(np.int32)
        self.q_dev = torch.randn(seqs * m, heads, dim, device="cuda").bfloat16()
        self.max_new, self.m, self.kv = m, m, kv_heads
        # values of one sign: a part of them that is lost shows
        self.codes[:, 1] = np.maximum(np.abs(self.codes[:, 1]), 1)
        self.scales[:] = 0.02

    def own_page(self, at):
        """Gives page `at` of the sequences a place of its own in the pool."""
        new = len(self.codes)
        was = self.table[0, at]
        self.codes = np.concatenate([self.codes, self.codes[was:was + 1]])
        self.scales = np.concatenate([self.scales, self.scales[was:was + 1]])
        self.table[:, at] = new
        return new

    def check_all(self, tl, which, window=0, sinks=0):
        import torch
        lse = torch.empty(self.q_dev.shape[0], self.heads, device="cuda")
        out = self.run(tl, window, sinks, lse=lse)
        torch.cuda.synchronize()
        assert tl.tern_device_status() == 0 and not torch.isnan(lse).any()
        group = self.heads // self.kv
        for b in which:
            rows, n = slice(b * self.m, (b + 1) * self.m), int(self.lens[b])
            for h in range(self.kv):
                of = slice(h * group, (h + 1) * group)
                ref, absum, ref_lse = attention(
                    self.q_dev[rows, of].float().cpu().numpy(), self.codes[:, :, h],
                    self.scales[:, :, h], self.table[b], n, self.dim ** -0.5, window, sinks)
                err = np.abs(out[rows, of].float().cpu().numpy().astype(np.float64) - ref)
                long = max(0, n - 8192) * 2.0 ** -24  # (the sums')
                bound = (5 * 2.0 ** -11 + long) * absum + 2.0 ** -9 * np.abs(ref)
                assert np.all(err <= bound), (b, h, float(np.max(err / bound)),
                                              np.argwhere(err > bound)[:3].tolist())
                err = np.abs(lse[rows, of].cpu().numpy() - ref_lse)
                assert np.all(err <= 2.5 * 2.0 ** -11 + long), (b, h, float(np.max(err)))


# few rows (one to three tiles; enough sequences that a warp takes many pages),
# the prompt kernel's split form, and its other one
FORMS = [(40, 3, 8), (60, 3, 24), (60, 4, 40), (8, 30, 8), (6, 100, 16)]


@pytest.mark.parametrize("up", [10, 30, 100])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("seqs,m,heads", FORMS)
def test_a_block_that_only_later_rows_see(tl, seqs, m, heads, dim, up):
    """The last page's value scale is 2^up times the others'; the first rows
    stand before it."""
    c = Batch(seqs, 41 * 64 + m // 2, m, heads, 8, dim, seed=up + m)
    page = c.own_page(41)
    c.scales[page, 1] *= np.float32(2.0 ** up)
    c.check_all(tl, (0, seqs - 1))


@pytest.mark.parametrize("up", [30, 100])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("seqs,m,heads", FORMS)
def test_a_block_that_leaves_the_window(tl, seqs, m, heads, dim, up):
    """The first rows' window ends in a page whose value scale is 2^up times
    the others', the last rows' past it."""
    c = Batch(seqs, 43 * 64 + 7, m, heads, 8, dim, seed=up + m)
    first = 43 * 64 + 7 - m  # position of the first row
    window = first - (3 * 64 - 1 - m // 2)  # its first token: the page's last but m // 2
    page = c.own_page(2)
    c.scales[page, 1] *= np.float32(2.0 ** up)
    c.check_all(tl, (0, seqs - 1), window)
    c.check_all(tl, (0, seqs - 1), window, sinks=5)


@pytest.mark.parametrize("up", [-100, -30, 30, 40, 100])
@pytest.mark.parametrize("seqs,m,heads", FORMS)
def test_a_block_of_small_weights(tl, seqs, m, heads, up):
    """A block whose tokens weigh 2^-46 of the others': it counts where its
    values are that much larger, and takes nothing from the others where not."""
    import torch
    c = Batch(seqs, 40 * 64, m, heads, 8, 64, seed=up + 200)
    page = c.own_page(17)
    c.scales[page, 1] *= np.float32(2.0 ** up)
    c.codes[:, 0] = np.abs(c.codes[:, 0] % 21) + 80
    c.codes[page, 0] = -c.codes[page, 0]  # scores 64 / 8 * 0.02 * 90 (1 + 1) = 29 apart
    c.q_dev = torch.full_like(c.q_dev, 1.0) + 0.1 * torch.rand_like(c.q_dev)
    c.check_all(tl, (0, seqs - 1))


@pytest.mark.parametrize("up", [6, 12, 18, 24])
@pytest.mark.parametrize("seqs,m,heads", FORMS)
def test_a_block_whose_weights_fp16_cannot_hold(tl, seqs, m, heads, up):
    """One token has nearly all the weight, those of a block 2^-35 to 2^-36 of
    it: they are a part of the result where their values are 2^up times as
    large."""
    import torch
    c = Batch(seqs, 40 * 64, m, heads, 8, 64, seed=up + 300)
    first, page = c.own_page(5), c.own_page(17)
    c.scales[page, 1] *= np.float32(2.0 ** up)
    c.codes[:, 0] = -127
    c.codes[first, 0, :, 9] = 100
    c.codes[page, 0] = -50  # 150 codes below: 64 / 8 * 0.02 * 150 = 24 = 34.6 ln 2
    c.q_dev = torch.full_like(c.q_dev, 1.0) + 0.05 * torch.rand_like(c.q_dev)
    c.check_all(tl, (0, seqs - 1))


@pytest.mark.parametrize("up", [4, 30, 100])
@pytest.mark.parametrize("m,heads", [(3, 8), (30, 8), (70, 8)])
def test_a_rise_beyond_the_first_records(tl, m, heads, up):
    """Blocks of more than 512 pages, the last of which only the last rows
    see; more than 256 pages a CTA of the few-row kernel."""
    c = Batch(20, 514 * 64 + 2 * (m // 3), m, heads, 8, 64, seed=up + m, pool=40)
    page = c.own_page(514)
    c.scales[page, 1] *= np.float32(2.0 ** up)
    c.check_all(tl, (0, 9, 19))


@pytest.mark.parametrize("scale", [0.02, 2.0 ** -20, 2.0 ** -37, 2.0 ** -60, 2.0 ** 30, 2.0 ** 60])
@pytest.mark.parametrize("seqs,m,heads", FORMS)
def test_blocks_of_zero_scale(tl, seqs, m, heads, scale):
    """A value scale of 0 makes its block's values 0 whatever its codes are."""
    c = Batch(seqs, 40 * 64 + 5, m, heads, 8, 64, seed=seqs + m)
    c.scales[:, 1] = scale
    for at in (0, 3, 11, 40):
        page = c.own_page(at)
        c.scales[page, 1] = 0
    c.check_all(tl, (0, seqs - 1))


@pytest.mark.parametrize("seqs,m,heads", FORMS)
@pytest.mark.parametrize("which", [0, 1])
def test_a_negative_scale_reads_as_nan(tl, seqs, m, heads, which):
    """The append writes none: the rows that see such a block, and only they,
    become NaN, as with a scale that is not finite."""
    import torch
    c = Batch(seqs, 43 * 64 + 7, m, heads, 8, 64, seed=m)
    window = 20 * 64
    clean = c.run(tl, window=window)
    page = c.own_page(43)
    c.scales[page, which, 1] *= -1
    got = c.run(tl, window=window).view(seqs, m, 8, -1)
    clean = clean.view(got.shape)
    torch.cuda.synchronize()
    sees = (torch.arange(m, device="cuda") + 43 * 64 + 7 - m) >= 43 * 64
    assert torch.isnan(got[:, sees, 1].float()).all()
    assert torch.equal(got[:, ~sees], clean[:, ~sees])
    rest = [h for h in range(8) if h != 1]
    assert torch.equal(got[:, :, rest], clean[:, :, rest])


@pytest.mark.parametrize("m,heads", [(1, 8), (2, 64)])
@pytest.mark.parametrize("dim", [64, 128])
def test_many_short_sequences_with_far_blocks(tl, m, heads, dim):
    """Several whole segments a CTA, one after the other, each with a block that
    is left to the plain path: the oracle's result, and the same bits each time."""
    import torch
    c = Batch(100, 4 * 64 + 9, m, heads, 8, dim, seed=m)
    for at, up in ((1, 90), (3, -80)):
        page = c.own_page(at)
        c.scales[page, 1] *= np.float32(2.0 ** up)
    c.check_all(tl, (0, 50, 99))
    first = c.run(tl)
    for _ in range(5):
        assert torch.equal(c.run(tl), first)
