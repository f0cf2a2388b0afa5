"""Corners of the norm's and the append's arguments."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tl():
    import torch
    import ternary_weight_linear_gb300 as tl
    tl.build()
    tl.load()
    torch.cuda.init()
    return tl


def test_append_takes_one_row_or_head_of_any_stride(tl):
    """The stride of a dimension of one element does not matter: keys from a
    fused projection, values of their own."""
    import torch
    for rows, heads in ((1, 4), (3, 1), (1, 1)):
        wide = torch.randn(rows, 3 * heads + 1, 64, device="cuda")
        k, v = wide[:, heads:2 * heads], torch.randn(rows, heads, 64, device="cuda")
        if heads == 1 and rows > 1:
            v = torch.randn(rows, 4, 64, device="cuda")[:, 2:3]  # rows apart as k's
        got = []
        for a, b in ((k, v), (k.contiguous(), v.contiguous())):
            codes = torch.zeros(2, 2, heads, 64, 64, dtype=torch.int8, device="cuda")
            scales = torch.zeros(2, 2, heads, device="cuda")
            table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
            start = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
            tl.tern_kv8_append(a, b, codes, scales, table, start, start[1:].clone())
            got.append((codes, scales))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        assert tl.tern_device_status() == 0
    k, v = (torch.randn(2, 4, 64, device="cuda"), torch.randn(2, 6, 64, device="cuda")[:, :4])
    codes = torch.zeros(2, 2, 4, 64, 64, dtype=torch.int8, device="cuda")
    with pytest.raises(ValueError):  # two rows: their strides have to agree
        tl.tern_kv8_append(k, v, codes, torch.zeros(2, 2, 4, device="cuda"), table, start,
                           start[1:].clone())


@pytest.mark.parametrize("width", [256, 9984, 32768])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_norm_weight_that_is_not_finite(tl, width, bad):
    """Such a y reaches the scale: max|y| / 127 is not finite."""
    import torch
    x = torch.randn(3, width, device="cuda")
    x[1, 8] = 0  # 0 * inf
    w = torch.ones(width, device="cuda")
    w[8] = float(bad)
    y = torch.empty(3, width, dtype=torch.bfloat16, device="cuda")
    q, s, _ = tl.tern_add_rmsnorm_s8(x, w, y=y)
    torch.cuda.synchronize()
    assert not torch.isfinite(s).any()
    assert torch.isnan(s[1]) and torch.isnan(y[1, 8].float())
    assert torch.isfinite(y[:, 9:].float()).all()


def test_bounds_past_32_bits_are_no_bounds(tl):
    """A window, sinks or max_new of any size: not their low 32 bits."""
    import torch
    from test_gpu_kv8_attention import Case
    c = Case([200, 130], [3, 70], 4, 2, 64, seed=7)
    want = c.run(tl)
    assert torch.equal(c.run(tl, window=2 ** 32 + 5), want)
    some = c.run(tl, window=20, sinks=10 ** 6)
    assert torch.equal(c.run(tl, window=20, sinks=2 ** 33 + 1), some)
    assert torch.equal(some, want) and not torch.equal(c.run(tl, window=20), want)
    assert torch.equal(c.run(tl, max_new=2 ** 32 + 70), c.run(tl, max_new=73))
    for kw in (dict(window=-2 ** 40), dict(sinks=-2 ** 33), dict(max_new=-2 ** 32)):
        with pytest.raises(tl.TernError):
            c.run(tl, **kw)
    kv = torch.randn(2, 2, 64, device="cuda")
    codes = torch.zeros(2, 2, 2, 64, 64, dtype=torch.int8, device="cuda")
    scales = torch.zeros(2, 2, 2, device="cuda")
    ix = (torch.tensor([[1]], dtype=torch.int32, device="cuda"),
          torch.tensor([0, 2], dtype=torch.int32, device="cuda"),
          torch.tensor([2], dtype=torch.int32, device="cuda"))
    tl.tern_kv8_append(kv, kv, codes, scales, *ix, max_new=2 ** 32 + 1)
    assert tl.tern_device_status() == 0 and scales[1].all()
