"""Room for own FP8 pages in the decode over shared prefixes: sizes and refusals on
the host."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    from mla_decode_attention_05_gb300 import build
    build.build()
    import mla_decode_attention_05_gb300 as m
    return m.lib()


def _call(L, **k):
    a = dict(fmt=1, width=2, own=2, pages=-1, G=1, B=2, T=1, H=4)
    a.update(k)
    p = ctypes.c_void_p(256)
    return L.mla_decode_shared_bounded(p, p, a["fmt"], 4, 64, p, a["width"], p, None, a["G"], p, a["own"], p, a["pages"], p, 0.1, 0,
                                       p, 0, p, p, a["B"], a["T"], a["H"], None)


def test_refusals(L):
    assert _call(L, pages=-2) == -1 and b"own_pages" in L.mla_last_error_string()
    assert _call(L, pages=-2 ** 31) == -1
    assert _call(L, B=0) == -1 and _call(L, fmt=7) == -1
    # more pages in the tables' width than are counted
    assert _call(L, width=1 << 29, own=1 << 20, pages=2 ** 31 - 1) == -2 and _call(L, own=1 << 29, pages=4) == -2
    assert L.mla_decode_shared_bounded_workspace_bytes(2, 1, 4, 1, 1, 2, 2, -2) == 0


def test_binding():
    import mla_decode_attention_05_gb300 as m
    assert m._bound(0) == 0 and m._bound(7) == 7 and m._bound(2 ** 40) == 2 ** 31 - 1
    with pytest.raises(ValueError, match="own_pages"):
        m._bound(-1)
    with pytest.raises(TypeError):
        m._bound(1.5)
