"""Blocks of query rows over more pages than the prompt kernel holds records of
(512): the exponent that their products with the values share may rise from one
set of records to the next.

Bar: the one of test_gpu_kv8_attention.py, and the fp32 sums' n * 2^-24 of A
where n passes the 8192 tokens that it counts with.
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


def shared_pages(seqs, pages, last, heads, kv_heads, dim, m, seed):
    """seqs sequences of `pages` pages on a pool of 40, all ending in a page of
    their own that holds `last` tokens; values of one sign, so that a part of
    them that is scaled wrongly shows."""
    import torch
    rng = np.random.default_rng(seed)
    c = Case([41 * 64], [1], heads, kv_heads, dim, seed=seed)
    pool = c.table[0, :41]
    c.table = np.empty((seqs, pages), dtype=np.int32)
    c.table[:, :-1] = pool[rng.integers(0, 40, (seqs, pages - 1))]
    c.table[:, -1] = pool[40]
    c.codes[:, 1] = np.maximum(np.abs(c.codes[:, 1]), 1)
    c.lens = np.full(seqs, (pages - 1) * 64 + last, dtype=np.int32)
    c.start = (np.arange(seqs + 1) * m).astype(np.int32)
    c.q_dev = torch.randn(seqs * m, heads, dim, device="cuda").bfloat16()
    c.max_new = m
    c.last_page = int(pool[40])
    return c


def attention(q, codes, scales, pages, n, scale):
    """(out, sum_j p_j |v_j|) of the last rows of one sequence of n tokens and
    one key-value head, in fp64: q [m, group, dim], codes [pages, 2, 64, dim],
    scales [pages, 2]; oracle.decoder's arithmetic on all rows at once."""
    m, group, dim = q.shape
    k, v = ((codes[pages, i].astype(np.float64) * scales[pages, i].astype(np.float64)[:, None, None])
            .reshape(-1, dim)[:n] for i in (0, 1))
    z = scale * (q.reshape(-1, dim).astype(np.float64) @ k.T).reshape(m, group, n)
    for i in range(m):
        z[i, :, ~od.visible(n - m + i, n, 0, 0)] = -np.inf
    p = np.exp(z - z.max(-1, keepdims=True))
    p = (p / p.sum(-1, keepdims=True)).reshape(-1, n)
    return (p @ v).reshape(q.shape), (p @ np.abs(v)).reshape(q.shape)


def check_sequences(c, tl, out, which, m):
    kv = c.codes.shape[2]
    group = c.heads // kv
    for b in which:
        rows = slice(b * m, (b + 1) * m)
        n = int(c.lens[b])
        pages = c.table[b, :(n + 63) // 64]
        for h in range(kv):
            of = slice(h * group, (h + 1) * group)
            ref, absum = attention(c.q_dev[rows, of].float().cpu().numpy(), c.codes[:, :, h],
                                   c.scales[:, :, h], pages, n, c.dim ** -0.5)
            err = np.abs(out[rows, of].float().cpu().numpy() - ref)
            bound = ((5 * 2.0 ** -11 + max(0, n - 8192) * 2.0 ** -24) * absum
                     + 2.0 ** -9 * np.abs(ref) + 2.0 ** -25)
            assert np.all(err <= bound), (b, h, float(np.max(err / bound)))


# 32 rows a head take the split form (two query tiles on alternate pages, the
# second of which has no page in a set of records of one), 96 the other
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("pages", [513, 514, 1025])
@pytest.mark.parametrize("m", [4, 12])
def test_value_exponent_rises_with_the_last_records(tl, dim, pages, m):
    """The last page's value scales are 8 times the others'."""
    import torch
    seqs = 20  # of 8 heads: all but the last sequence's blocks are whole
    c = shared_pages(seqs, pages, 37, 64, 8, dim, m, seed=dim + pages + m)
    c.scales[:, 1] = 0.02
    c.scales[c.last_page, 1] = 0.16
    out = c.run(tl)
    torch.cuda.synchronize()
    assert tl.tern_device_status() == 0 and tl.tern_last_launches() == 2
    check_sequences(c, tl, out, (0, 18, 19), m)


# What only the split form of the prompt kernel does (25 to 64 rows a head; up
# to 24 a long batch of few rows goes to the other kernel, which would be one
# launch).

@pytest.mark.parametrize("m", [30, 64])
def test_split_blocks_of_more_pages_than_records(tl, m):
    import torch
    seqs, kv, dim = 20, 8, 64
    c = shared_pages(seqs, 531, 1, kv, kv, dim, m, seed=m)
    c.lens = (530 * 64 + 1 - 64 * np.arange(seqs)).astype(np.int32)  # 531 pages to 512
    out = c.run(tl)
    torch.cuda.synchronize()
    assert tl.tern_device_status() == 0 and tl.tern_last_launches() == 2
    assert torch.equal(out, c.run(tl))
    check_sequences(c, tl, out, (0, 7, 18, 19), m)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,m", [(32, 30), (64, 32), (96, 9)])
def test_split_blocks_of_the_last_wave_in_parts(tl, heads, m, dim):
    """160 blocks of rows: the last ones are cut along the keys."""
    import torch
    c = Case([2500, 2400, 2300, 2200, 2100], [m] * 5, heads, 32, dim, seed=heads + m)
    a = c.check(tl)
    ws = torch.zeros(tl.tern_kv8_attention_workspace_bytes(5, 5 * m, heads, 32, dim),
                     dtype=torch.uint8, device="cuda")
    for _ in range(2):
        assert torch.equal(a, c.run(tl, workspace=ws))
        assert tl.tern_last_launches() == 2
    assert not ws[:tl.SYNC_BYTES].any()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,new,heads", [([600], [512], 48), ([2000], [512], 48),
                                            ([300, 900], [60, 500], 16)])
def test_a_wide_table_leaves_short_blocks_whole(tl, lens, new, heads, dim):
    """A table of the longest context that a program allows gives what a tight
    one does: blocks of few pages are not cut for its width."""
    import torch
    c = Case(lens, new, heads, 8, dim, seed=heads + dim)
    # (the oracle takes its time over long prompts)
    tight = c.check(tl) if max(lens) < 1000 else c.run(tl)
    wide = np.full((len(lens), 512), -7, dtype=np.int32)
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    assert torch.equal(c.run(tl), tight) and tl.tern_device_status() == 0
