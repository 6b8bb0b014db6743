"""Refusals of the decode over shared prefixes, the attention weights and the
eviction (on the host, before anything is launched), and their oracle's own checks."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import long_context as O


@pytest.fixture(scope="module")
def L():
    from mla_decode_attention_05_gb300 import build
    build.build()
    import mla_decode_attention_05_gb300 as m
    return m.lib()


def v(x):
    return None if x is None else ctypes.c_void_p(x)


@pytest.mark.parametrize("args,code", [
    (dict(B=0), -1), (dict(T=0), -1), (dict(T=17), -1), (dict(H=0), -1), (dict(H=129), -1), (dict(G=0), -1), (dict(width=0), -1),
    (dict(own=0), -1), (dict(fmt=3), -1), (dict(fmt=-1), -1), (dict(B=9000), -2), (dict(G=8192), -2),
    (dict(G=1 << 12, width=1 << 20), -2), (dict(own=1 << 30), -2), (dict(B=64, T=16, H=128, own=1 << 20), -2), (dict(q=None), -1), (dict(cache=None), -1), (dict(pt=None), -1), (dict(pl=None), -1),
    (dict(bt=None), -1), (dict(sk=None), -1), (dict(out=None), -1), (dict(lse=None), -1), (dict(off=None, G=2), -1), (dict(q=8), -1),
    (dict(cache=264), -1), (dict(out=264), -1), (dict(pt=258), -1), (dict(off=258), -1), (dict(lse=258), -1), (dict(fmt=1, sc=None), -1),
    (dict(fmt=1, sc=264), -1), (dict(fmt=2, sc=258), -1), (dict(page=32), -2), (dict(pages=0), -1), (dict(causal=2), -1),
    (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
])
def test_shared_arguments(L, args, code):
    a = dict(q=256, cache=256, fmt=0, pages=4, page=64, pt=256, width=2, pl=256, off=256, G=1, bt=256, own=2, sk=256, sc=256,
             scale=0.1, causal=0, ws=256, ws_bytes=1 << 40, out=256, lse=256, B=2, T=1, H=4)
    a.update(args)
    rc = L.mla_decode_shared(v(a["q"]), v(a["cache"]), a["fmt"], a["pages"], a["page"], v(a["pt"]), a["width"], v(a["pl"]),
                             v(a["off"]), a["G"], v(a["bt"]), a["own"], v(a["sk"]), v(a["sc"]), a["scale"], a["causal"],
                             v(a["ws"]), a["ws_bytes"], v(a["out"]), v(a["lse"]), a["B"], a["T"], a["H"], None)
    assert rc == code and L.mla_last_error_string()


@pytest.mark.parametrize("args,code", [
    (dict(B=0), -1), (dict(B=8193), -1), (dict(T=0), -1), (dict(H=0), -1), (dict(H=129), -1), (dict(cap=0), -1),
    (dict(cap=(1 << 24) + 1), -2), (dict(B=8192, T=1 << 13, H=128), -2), (dict(T=1 << 30, H=128), -2), (dict(fmt=3), -1), (dict(q=None), -1), (dict(cache=None), -1),
    (dict(bt=None), -1), (dict(sk=None), -1), (dict(lse=None), -1), (dict(mass=None), -1), (dict(q=264), -1), (dict(cache=8), -1),
    (dict(lse=258), -1), (dict(mass=257), -1), (dict(fmt=1, sc=None), -1), (dict(fmt=2, sc=258), -1), (dict(page=16), -2),
    (dict(pages=0), -1), (dict(own=0), -1), (dict(causal=-1), -1), (dict(scale=-1.0), -1), (dict(decay=-0.5), -1),
    (dict(decay=float("inf")), -1), (dict(decay=float("nan")), -1), (dict(T=100, ws=None), -3), (dict(T=100, ws_bytes=256), -3),
    (dict(T=100, ws=272), -1),
])
def test_mass_arguments(L, args, code):
    a = dict(q=256, cache=256, fmt=0, pages=4, page=64, bt=256, own=2, sk=256, sc=256, lse=256, scale=0.1, causal=0, decay=1.0,
             mass=256, cap=128, ws=256, ws_bytes=1 << 40, B=2, T=1, H=4)
    a.update(args)
    rc = L.mla_attention_mass(v(a["q"]), v(a["cache"]), a["fmt"], a["pages"], a["page"], v(a["bt"]), a["own"], v(a["sk"]),
                              v(a["sc"]), v(a["lse"]), a["scale"], a["causal"], a["decay"], v(a["mass"]), a["cap"], v(a["ws"]),
                              a["ws_bytes"], a["B"], a["T"], a["H"], None)
    assert rc == code and L.mla_last_error_string()


@pytest.mark.parametrize("args,code", [
    (dict(B=0), -1), (dict(B=8193), -1), (dict(cap=0), -1), (dict(cap=(1 << 24) + 1), -2), (dict(keep=0), -1), (dict(sinks=-1), -1),
    (dict(recent=-1), -1), (dict(sinks=60, recent=41), -1), (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), -1), (dict(cache=None), -1),
    (dict(bt=None), -1), (dict(sk=None), -1), (dict(mass=None), -1), (dict(pos=None), -1), (dict(out=None), -1), (dict(cache=264), -1),
    (dict(mass=258), -1), (dict(pos=257), -1), (dict(out=258), -1), (dict(fmt=9), -1), (dict(fmt=1, sc=None), -1),
    (dict(fmt=1, sc=264), -1), (dict(page=128), -2), (dict(pages=0), -1), (dict(own=0), -1), (dict(ws=None), -3),
    (dict(ws_bytes=64), -3), (dict(ws=272), -1),
])
def test_evict_arguments(L, args, code):
    a = dict(cache=256, fmt=0, pages=4, page=64, bt=256, own=2, sk=256, sc=256, mass=256, pos=256, cap=128, keep=100, sinks=4,
             recent=10, out=256, ws=256, ws_bytes=1 << 40, B=2)
    a.update(args)
    rc = L.mla_evict(v(a["cache"]), a["fmt"], a["pages"], a["page"], v(a["bt"]), a["own"], v(a["sk"]), v(a["sc"]), v(a["mass"]),
                     v(a["pos"]), a["cap"], a["keep"], a["sinks"], a["recent"], v(a["out"]), v(a["ws"]), a["ws_bytes"], a["B"],
                     None)
    assert rc == code and L.mla_last_error_string()


def test_workspace_sizes(L):
    import mla_decode_attention_05_gb300 as m
    assert m.attention_mass_workspace_bytes(4, 1, 128, 1000) == 0     # one tile of query rows, whatever the format
    assert m.attention_mass_workspace_bytes(4, 2, 128, 1000) > 0      # (FP8 rows with scales: two)
    assert m.attention_mass_workspace_bytes(4, 3, 128, 1000) > 0
    assert L.mla_attention_mass_workspace_bytes(0, 1, 1, 1) == 0
    assert m.evict_workspace_bytes(3, 1000, 400) >= 3 * 4 + 2 * 3 * 400 * 4
    assert m.evict_workspace_bytes(3, 1000, 900) >= 3 * 4 + 2 * 3 * 100 * 4
    assert m.evict_workspace_bytes(3, 100, 900) > 0
    with pytest.raises(m.MlaError):
        m.evict_workspace_bytes(3, 100, 0)


def test_binding_refuses_wrong_types_and_places():
    import mla_decode_attention_05_gb300 as m
    b, i32 = lambda *s: torch.zeros(s, dtype=torch.bfloat16), lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(TypeError, match="q must be"):
        m.decode_shared(torch.zeros(1, 1, 2, 576), b(2, 64, 576), i32(1, 1), i32(1), i32(1, 1), i32(1), softmax_scale=0.1)
    with pytest.raises(ValueError, match="CUDA"):
        m.decode_shared(b(1, 1, 2, 576), b(2, 64, 576), i32(1, 1), i32(1), i32(1, 1), i32(1), softmax_scale=0.1)
    with pytest.raises(ValueError, match="CUDA"):
        m.attention_mass(b(1, 1, 2, 576), b(2, 64, 576), i32(1, 1), i32(1), torch.zeros(1, 2, 1), torch.zeros(1, 64), softmax_scale=0.1)
    with pytest.raises(TypeError, match="kv_cache"):
        m.evict(torch.zeros(2, 64, 576), i32(1, 2), i32(1), torch.zeros(1, 128), i32(1, 128), keep=64)
    with pytest.raises(TypeError):
        m.evict(None, i32(1, 2), i32(1), torch.zeros(1, 128), i32(1, 128), keep=64)
    with pytest.raises(ValueError, match="CUDA"):
        m.evict(b(2, 64, 576), i32(1, 2), i32(1), torch.zeros(1, 128), i32(1, 128), keep=64)


@pytest.mark.parametrize("causal", [False, True])
def test_oracle_attention_and_mass(causal):
    """Against one softmax over prefix and own tokens together, with a mask."""
    rng = np.random.default_rng(1)
    T, H, P, n = 3, 2, 5, 4
    q, pre, own = rng.standard_normal((T, H, 576)), rng.standard_normal((P, 576)), rng.standard_normal((n, 576))
    r = O.attention(q, pre, own, 0.05, causal)
    k = torch.from_numpy(np.concatenate([pre, own]))
    s = torch.from_numpy(q) @ k.T * 0.05
    if causal:
        i, j = torch.arange(T)[:, None], torch.arange(P + n)[None]
        s.masked_fill_((j > P + n - T + i)[:, None, :], -np.inf)
    w = torch.softmax(s, -1)
    # (sums that cancel: nine weighted values of at most 5, and scores off by 576 steps of 2^-53)
    np.testing.assert_allclose(r["out"], (w @ k[:, :512]).numpy(), rtol=0, atol=1e-11)
    np.testing.assert_allclose(r["lse"], torch.logsumexp(s, -1).numpy(), rtol=1e-12)
    m, bound = O.mass(q, own, r["lse"], 0.05, causal)
    np.testing.assert_allclose(m, w.sum((0, 1))[P:].numpy(), rtol=1e-11)
    assert np.all(bound > 0) and np.all(bound < 0.1 * m)
    # without a prefix every row's weights sum to one
    r = O.attention(q, np.zeros((0, 576)), own, 0.05, False)
    assert abs(O.mass(q, own, r["lse"], 0.05, False)[0].sum() - T * H) < 1e-9


def test_oracle_rows_without_keys():
    rng = np.random.default_rng(2)
    q, none = rng.standard_normal((4, 1, 576)), np.zeros((0, 576))
    r = O.attention(q, none, rng.standard_normal((2, 576)), 0.1, True)   # tokens 0 and 1 of 4 see nothing
    assert np.isneginf(r["lse"][:2]).all() and not r["out"][:2].any() and np.isfinite(r["lse"][2:]).all()
    m, _ = O.mass(q, rng.standard_normal((2, 576)), r["lse"], 0.1, True)
    assert np.isfinite(m).all()


def test_oracle_eviction():
    m = np.array([5, 1, 3, 3, 9, 2, 0, 7], dtype=np.float32)
    pos = np.arange(8)
    assert O.evict(m, pos, 8, 8, 0, 0) == ([], [])
    # 5, 9, 7 and the first of the two threes stay
    assert O.evict(m, pos, 8, 4, 0, 0) == ([1, 3], [4, 7])
    # slot 1 as the second position, and the latest two; the heaviest of the others is 9
    assert O.evict(m, pos, 8, 5, 2, 2) == ([2, 3], [6, 7])
    # positions, not slots, tell what is late
    assert O.evict(m, pos[::-1].copy(), 8, 2, 0, 2) == ([], [])
    # nan is lighter than everything, -0 equal to 0
    assert O.evict(np.array([np.nan, -np.inf, 0, -0.0, 1], np.float32), pos, 5, 3, 0, 0) == ([0, 1], [3, 4])


def test_planted_mistakes_are_seen():
    """What the oracle is compared with would show: a slot off by one, a tie the
    wrong way, a row that sees one key too many."""
    rng = np.random.default_rng(3)
    q, own = rng.standard_normal((2, 1, 576)), rng.standard_normal((6, 576))
    none = np.zeros((0, 576))
    right, wrong = O.attention(q, none, own, 0.1, True), O.attention(q, none, own, 0.1, False)
    assert np.abs(right["out"][0] - wrong["out"][0]).max() > 1e-2 and np.array_equal(right["out"][1], wrong["out"][1])
    m = np.array([1, 1, 1, 1], np.float32)
    assert O.evict(m, np.arange(4), 4, 2, 0, 0) != ([0, 1], [2, 3])
