"""Host-side checks of the decoder operators' C entries that need no GPU: what
is refused before any device work."""
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
