"""Host-side checks of the decoder operators' C entries that need no GPU: what
is refused before any device work."""
import ctypes

import pytest

import ternary_weight_linear_gb300 as tl

EINVAL = -1
P = 4096  # a 16-byte aligned fake address; never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built():
    tl.build()
    tl.load()


def test_layer_on_codes_has_no_rotated_form(monkeypatch):
    lib = tl.load()
    monkeypatch.setenv("TERN_ROTATE", "1")
    tl.tern_reload_env()
    try:
        for T in (1, 40):
            assert lib.tern_linear_s8(P, P, P, P, P, T, 1024, 8, None, 0, None) == EINVAL
    finally:
        monkeypatch.delenv("TERN_ROTATE")
        tl.tern_reload_env()


def cache(pages=8, seqs=2, width=4, kv_heads=8, dim=64):
    return ctypes.byref(tl._KV8Cache(P, P, P, P, P, pages, seqs, width, kv_heads, dim))


def attention(c, rows, max_new, heads=8, ws=1 << 40, scale=0.125):
    return tl.load().tern_kv8_attention(c, P, 1, heads * 64, 64, rows, heads, max_new, 0, 0, scale,
                                        P, None, P, ws, None)


def test_no_rows_need_no_max_new():
    lib = tl.load()
    assert attention(cache(), 0, 0) == 0
    assert lib.tern_kv8_append(cache(), None, None, 1, 512, 64, 0, 0, None) == 0
    for max_new in (-1, 0):
        assert attention(cache(), 1, max_new) == EINVAL
        assert lib.tern_kv8_append(cache(), P, P, 1, 512, 64, 1, max_new, None) == EINVAL
    assert attention(cache(), 0, -1) == EINVAL


def test_a_sequence_of_too_many_pages_and_heads_is_refused():
    """The pages of a sequence's heads are counted in 32 bits."""
    wide = cache(pages=64, seqs=1, width=1 << 20, kv_heads=4096)
    assert attention(wide, 1, 1, heads=4096, ws=0) == EINVAL
    assert tl.load().tern_kv8_append(wide, P, P, 1, 4096 * 64, 64, 0, 1, None) == EINVAL
    # (the next check is the workspace's)
    assert attention(cache(64, 1, (1 << 19) - 1, 4096), 1, 1, heads=4096, ws=0) == -3


def test_a_grid_of_too_many_blocks_is_refused_before_any_launch():
    """2^17 sequences of at most 2^20 new tokens, 8 heads: 2^32 blocks of rows."""
    many = cache(seqs=1 << 17)
    assert attention(many, 1 << 20, 1 << 20, ws=0) == EINVAL
    assert attention(many, 1 << 20, 1, ws=0) == -3  # (the next check is the workspace's)


def test_a_scale_that_overflows_is_refused():
    """In base 2 it is 1.44 times as large."""
    for scale in (2.5e38, float("inf"), float("nan"), 0.0, -1.0):
        assert attention(cache(), 1, 1, scale=scale, ws=0) == EINVAL
    assert attention(cache(), 1, 1, scale=2.3e38, ws=0) == -3
