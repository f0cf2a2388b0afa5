"""What the C entries of the attention block's operators refuse before any
device work (no GPU needed)."""
import ctypes

import pytest

import ternary_weight_linear_gb300 as tl

EINVAL, EALIGN = -1, -2
P = 4096  # a 16-byte aligned fake address; never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    tl.build()
    tl.load()


def rotation(freq=P, rotary=64, interleaved=0, magnitude=1.0):
    return ctypes.byref(tl._Rotation(freq, rotary, interleaved, magnitude))


def rope(x=P, t=0, ld=1024, hd=128, out=2 * P, ot=1, old=1024, ohd=128, pos=P, rot=None, T=1, heads=8,
         dim=128):
    return tl.load().tern_rope(x, t, ld, hd, out, ot, old, ohd, pos, rot or rotation(), T, heads,
                               dim, None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(out=None), dict(pos=None), dict(T=0), dict(T=-1), dict(heads=0),
    dict(dim=120), dict(dim=1040, ld=1040 * 8, hd=1040, old=1040 * 8, ohd=1040), dict(t=3),
    dict(ot=-1), dict(ld=64), dict(hd=64), dict(old=64), dict(ohd=-128), dict(hd=1 << 29)])
def test_rope_refuses(bad):
    assert rope(**bad) == EINVAL


@pytest.mark.parametrize("bad", [dict(freq=None), dict(rotary=0), dict(rotary=24),
                                 dict(rotary=144), dict(rotary=-16), dict(magnitude=NAN),
                                 dict(magnitude=INF)])
def test_rotations_that_are_refused(bad):
    assert rope(rot=rotation(**bad)) == EINVAL
    assert append(rot=rotation(**bad)) == EINVAL


def test_rope_in_place_keeps_type_and_strides():
    Q = 8192
    for bad in (dict(ot=1), dict(t=1, ot=0), dict(ot=0, old=2048, T=2), dict(ot=0, ohd=256)):
        assert rope(out=P, **bad) == EINVAL
    # (of one token, or apart, the next check is the alignment's)
    assert rope(ot=0, old=2048, pos=P + 4) == EALIGN and rope(out=Q, pos=P + 4) == EALIGN


def test_rope_alignment():
    for bad in (dict(x=P + 4), dict(out=P + 8), dict(pos=P + 4), dict(ld=1026), dict(ohd=132),
                dict(rot=rotation(freq=P + 8))):
        assert rope(**bad) == EALIGN


def cache(pages=8, seqs=2, width=4, kv_heads=8, dim=128):
    return ctypes.byref(tl._KV8Cache(P, P, P, P, P, pages, seqs, width, kv_heads, dim))


def append(c=None, q=P, k=P, v=P, t=0, qld=6144, qhd=128, heads=48, ld=1024, hd=128, pos=None,
           rot=None, out=P, qt=1, rows=2, max_new=1):
    return tl.load().tern_kv8_append_rope(c or cache(), q, k, v, t, qld, qhd, heads, ld, hd, pos,
                                          rot or rotation(), out, qt, rows, max_new, None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(out=None), dict(k=None), dict(v=None), dict(t=3), dict(qt=0), dict(heads=0),
    dict(heads=513), dict(qld=64), dict(qhd=64), dict(ld=64), dict(hd=64), dict(rows=-1),
    dict(max_new=0), dict(max_new=-1), dict(c=cache(dim=96)), dict(c=cache(pages=0)),
    dict(rot=rotation(rotary=128), c=cache(dim=64), qhd=64, hd=64)])
def test_append_refuses(bad):
    assert append(**bad) == EINVAL


def test_append_alignment_and_no_rows():
    for bad in (dict(q=P + 8), dict(k=P + 4), dict(out=P + 2), dict(pos=P + 4), dict(ld=1026),
                dict(qhd=130)):
        assert append(**bad) == EALIGN
    assert append(rows=0, max_new=0, k=None, v=None, q=None, out=None) == 0


def norms(x=P, xt=0, ld=256, post=P, pt=1, gate=P, gt=1, gld=0, bs=1.0, res=P, rout=P, rt=1, rs=1.0,
          w=P, wt=1, eps=1e-6, q=P, s=P, y=None, T=2, K=256):
    return tl.load().tern_norm_add_norm_s8(x, xt, ld, post, pt, gate, gt, gld, bs, res, rout, rt, rs,
                                           w, wt, eps, q, s, y, T, K, None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(res=None), dict(w=None), dict(q=None), dict(s=None), dict(q=None, s=None),
    dict(T=0), dict(K=0), dict(K=264, ld=264), dict(K=1 << 16, ld=1 << 16), dict(ld=240), dict(xt=2),
    dict(pt=2), dict(gt=3), dict(rt=2), dict(wt=2), dict(gld=128), dict(gld=-256), dict(eps=-1.0),
    dict(eps=NAN), dict(bs=NAN), dict(rs=INF)])
def test_norms_refuse(bad):
    assert norms(**bad) == EINVAL


def test_norms_alignment():
    for bad in (dict(x=P + 8), dict(post=P + 2), dict(gate=P + 4), dict(res=P + 8), dict(rout=P + 8),
                dict(w=P + 8), dict(q=P + 8), dict(s=P + 4), dict(y=P + 8), dict(ld=258),
                dict(gld=260)):
        assert norms(**bad) == EALIGN


def shared(n=64, c=None, rows=2, heads=8, max_new=1, ws=1 << 40, scale=0.125, q=P, out=P, ld=1024):
    return tl.load().tern_kv8_attention_shared(c or cache(), q, 1, ld, 128, rows, heads, n, max_new,
                                               0, 0, scale, out, None, P, ws, None)


@pytest.mark.parametrize("bad", [dict(n=-64), dict(n=1), dict(n=63), dict(n=320), dict(heads=12),
                                 dict(rows=-1), dict(max_new=0), dict(scale=NAN), dict(q=None),
                                 dict(out=None), dict(ld=64), dict(c=cache(dim=96)),
                                 dict(c=cache(kv_heads=16384, width=64), rows=1 << 25,
                                      heads=16384)])
def test_shared_attention_refuses(bad):
    assert shared(**bad) == EINVAL


def test_shared_attention_workspace():
    need = tl.tern_kv8_attention_shared_workspace_bytes(2, 2, 8, 8, 128)
    plain = tl.tern_kv8_attention_workspace_bytes(2, 2, 8, 8, 128)
    assert need > plain + 2 * 8 * 129 * 4
    assert shared(ws=need - 1) == -3 and shared(ws=plain) == -3
    assert shared(rows=0, max_new=0, ws=0) == 0 and shared(q=P + 2) == EALIGN
    for bad in ((0, 1, 8, 8, 128), (1, 0, 8, 8, 128), (1, 1, 12, 8, 128), (1, 1, 8, 8, 96)):
        assert tl.tern_kv8_attention_shared_workspace_bytes(*bad) == 0


def test_rope_refuses_more_heads_than_it_counts():
    for heads in ((1 << 30) + 1, 2 ** 31 - 4, 2 ** 31 - 1):
        assert rope(heads=heads, pos=P + 4) == EINVAL
    assert rope(heads=1 << 30, pos=P + 4) == EALIGN


def test_nothing_to_share_needs_the_ordinary_workspace():
    """Refused for its alignment, the check behind the size's."""
    for n, seqs in ((0, 2), (64, 1), (0, 1)):
        plain = tl.tern_kv8_attention_workspace_bytes(seqs, 2, 8, 8, 128)
        call = lambda ws, at: tl.load().tern_kv8_attention_shared(  # noqa: E731
            cache(seqs=seqs), P, 1, 1024, 128, 2, 8, n, 1, 0, 0, 0.125, P, None, at, ws, None)
        assert call(plain - 1, P) == -3 and call(plain, P + 4) == EALIGN
