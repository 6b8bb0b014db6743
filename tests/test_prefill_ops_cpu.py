"""Refusals of the operators around the decode (checked on the host before
anything is launched, so they need no GPU), and the oracle's own checks."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import prefill as O
from oracle.kv_insert import bf16_bits_to_f64, f64_to_bf16_bits


@pytest.fixture(scope="module")
def L():
    from mla_decode_attention_05_gb300 import build
    build.build()
    import mla_decode_attention_05_gb300 as m
    return m.lib()


def v(x):
    return None if x is None else ctypes.c_void_p(x)


@pytest.mark.parametrize("args,code", [
    (dict(N=-1), -1), (dict(max_pos=0), -1), (dict(interleaved=2), -1), (dict(q=None), -1), (dict(qo=None), -1),
    (dict(H=0), -1), (dict(H=129), -1), (dict(q_tok=12), -1), (dict(o_head=68), -1), (dict(o_head=32), -1),
    (dict(q=264), -1), (dict(qo=8), -1), (dict(pos=None), -1), (dict(pos=260), -1), (dict(cs=None), -1),
    (dict(cs=264), -1), (dict(kv_c=None), -1), (dict(ld_kv=500), -1), (dict(kv_format=5), -1),
    (dict(kv_format=1, scales=None), -1), (dict(kv_format=2, ksi=None), -1), (dict(eps=float("inf")), -1),
    (dict(N=0, kv_c=None, slots=None, kv=None, pos=None), 0),
])
def test_insert_rope_arguments(L, args, code):
    a = dict(kv_c=256, ld_kv=2112, k_pe=256, ld_pe=2112, w=256, eps=1e-6, slots=256, pos=256, cs=256, max_pos=10,
             interleaved=1, N=4, kv=256, kv_format=0, num_pages=4, page_size=64, scales=256, ksi=256, q=256,
             q_tok=8 * 576, q_head=576, qo=256, o_tok=8 * 576, o_head=576, H=8)
    a.update(args)
    rc = L.mla_kv_insert_rope(v(a["kv_c"]), a["ld_kv"], v(a["k_pe"]), a["ld_pe"], v(a["w"]), a["eps"], v(a["slots"]),
                              v(a["pos"]), v(a["cs"]), a["max_pos"], a["interleaved"], a["N"], v(a["kv"]),
                              a["kv_format"], a["num_pages"], a["page_size"], v(a["scales"]), v(a["ksi"]), v(a["q"]),
                              a["q_tok"], a["q_head"], v(a["qo"]), a["o_tok"], a["o_head"], a["H"], None)
    assert rc == code
    assert bool(L.mla_last_error_string()) == (code != 0)


@pytest.mark.parametrize("args,code", [
    (dict(B=-1), -1), (dict(total=-1), -1), (dict(total=(1 << 30) + 1), -2), (dict(H=0), -1), (dict(H=129), -1),
    (dict(fmt=3), -1), (dict(page=32), -2), (dict(pages=0), -1), (dict(max_pages=0), -1), (dict(uk_row=500), -1),
    (dict(uk_row=516), -1), (dict(uv_head=60), -1), (dict(uv_row=8), -1), (dict(kv=None), -1), (dict(kv=8), -1),
    (dict(uk=None), -1), (dict(uv=264), -1), (dict(pe=264), -1), (dict(bt=258), -1), (dict(cu=257), -1),
    (dict(fmt=1, sc=None), -1), (dict(fmt=1, sc=264), -1), (dict(fmt=2, sc=258), -1), (dict(pages=1 << 25), -2), (dict(cache=264), -1),
    (dict(total=0, kv=None, pe=None), 0), (dict(B=0), 0),
])
def test_expand_arguments(L, args, code):
    a = dict(cache=256, fmt=0, pages=4, page=64, bt=256, max_pages=2, cu=256, B=2, total=100, sc=256, uk=256,
             uk_row=512, uk_head=65536, uv=256, uv_row=512, uv_head=65536, H=4, kv=256, pe=256)
    a.update(args)
    rc = L.mla_kv_expand(v(a["cache"]), a["fmt"], a["pages"], a["page"], v(a["bt"]), a["max_pages"], v(a["cu"]),
                         a["B"], a["total"], v(a["sc"]), v(a["uk"]), a["uk_row"], a["uk_head"], v(a["uv"]),
                         a["uv_row"], a["uv_head"], a["H"], v(a["kv"]), v(a["pe"]), None)
    assert rc == code
    assert bool(L.mla_last_error_string()) == (code != 0)


@pytest.mark.parametrize("args,code", [
    (dict(B=-1), -1), (dict(B=(1 << 20) + 1), -2), (dict(Nq=-1), -1), (dict(Nk=-1), -1), (dict(Nq=(1 << 30) + 1), -2),
    (dict(Nk=(1 << 26) + 1), -2),
    (dict(H=0), -1), (dict(H=129), -1), (dict(causal=2), -1), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1), (dict(scale=2.5e38), -1), (dict(q_tok=100), -1), (dict(q_head=188), -1), (dict(k_tok=64), -1),
    (dict(v_head=132), -1), (dict(pe_tok=32), -1), (dict(q=None), -1), (dict(q=264), -1), (dict(out=8), -1),
    (dict(lse=2), -1), (dict(cq=None), -1), (dict(ck=257), -1), (dict(kn=None), -1), (dict(vv=264), -1),
    (dict(Nq=0, q=None, out=None, lse=None), 0), (dict(B=0), 0),
    (dict(B=1, Nk=9000, ws=None), -3), (dict(B=1, Nk=9000, ws_bytes=1000), -3), (dict(B=1, Nk=9000, ws=128), -1),
])
def test_prefill_arguments(L, args, code):
    a = dict(q=256, q_tok=768, q_head=192, kn=256, k_tok=1024, k_head=256, pe=256, pe_tok=64, vv=256, v_tok=1024,
             v_head=256, cq=256, ck=256, B=2, H=4, Nq=10, Nk=20, scale=0.07, causal=1, out=256, lse=256, ws=256,
             ws_bytes=1 << 30)
    a.update(args)
    rc = L.mla_prefill(v(a["q"]), a["q_tok"], a["q_head"], v(a["kn"]), a["k_tok"], a["k_head"], v(a["pe"]), a["pe_tok"],
                       v(a["vv"]), a["v_tok"], a["v_head"], v(a["cq"]), v(a["ck"]), a["B"], a["H"], a["Nq"], a["Nk"],
                       a["scale"], a["causal"], v(a["ws"]), a["ws_bytes"], v(a["out"]), v(a["lse"]), None)
    assert rc == code
    assert bool(L.mla_last_error_string()) == (code != 0)


def test_prefill_workspace(L):
    """Few query tiles over long keys are split over the keys, others not."""
    import mla_decode_attention_05_gb300 as m
    assert m.prefill_workspace_bytes(1, 128, 256, 9000) == 0        # 128 tiles on 152 SMs
    assert m.prefill_workspace_bytes(1, 128, 2000, 100000) == 0     # 1024
    assert m.prefill_workspace_bytes(8, 20, 16, 24000) > 0          # 160: two rounds, the second one almost empty
    assert m.prefill_workspace_bytes(1, 8, 200, 500) == 0           # short keys
    n = m.prefill_workspace_bytes(1, 8, 200, 12200)
    assert n == 16 * 200 * 8 * 129 * 4 + (-(16 * 200 * 8 * 4) % 256)
    assert m.prefill_workspace_bytes(1, 1, 1, 1 << 26) == 32 * 128 * 4 + 256
    assert m.prefill_workspace_bytes(0, 8, 0, 0) == 0 and m.prefill_workspace_bytes(1, 0, 5, 5) == 0


@pytest.mark.parametrize("args,code", [
    (dict(N=-1), -1), (dict(H=0), -1), (dict(H=129), -1), (dict(ld_t=516), -1), (dict(ld_t=256), -1),
    (dict(ld_h=500), -1), (dict(w_row=256), -1), (dict(w_head=4), -1), (dict(attn=None), -1), (dict(attn=264), -1),
    (dict(w=8), -1), (dict(out=264), -1), (dict(N=0, attn=None, out=None), 0),
])
def test_value_project_arguments(L, args, code):
    a = dict(attn=256, ld_t=2048, ld_h=512, w=256, w_row=512, w_head=65536, N=3, H=4, out=256)
    a.update(args)
    rc = L.mla_value_project(v(a["attn"]), a["ld_t"], a["ld_h"], v(a["w"]), a["w_row"], a["w_head"], a["N"], a["H"],
                             v(a["out"]), None)
    assert rc == code
    assert bool(L.mla_last_error_string()) == (code != 0)


def test_binding_refuses_wrong_types_and_places():
    """The binding's checks: types, shapes, strides and devices."""
    import mla_decode_attention_05_gb300 as m
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError, match="q must be"):
        m.prefill(torch.zeros(4, 2, 192), b(4, 2, 128), b(4, 64), b(4, 2, 128), i32, i32, softmax_scale=0.1)
    with pytest.raises(ValueError, match="q must be"):
        m.prefill(b(4, 2, 128), b(4, 2, 128), b(4, 64), b(4, 2, 128), i32, i32, softmax_scale=0.1)
    with pytest.raises(ValueError, match="CUDA"):
        m.prefill(b(4, 2, 192), b(4, 2, 128), b(4, 64), b(4, 2, 128), i32, i32, softmax_scale=0.1)
    with pytest.raises(ValueError, match="CUDA"):
        m.value_project(b(4, 2, 512), b(2, 128, 512))
    with pytest.raises(TypeError):
        m.value_project(None, b(2, 128, 512))
    with pytest.raises(TypeError):
        m.kv_expand(torch.zeros(2, 64, 576), i32, i32, b(2, 128, 512), b(2, 128, 512), total=4)
    with pytest.raises(TypeError):
        m.kv_insert_rope(torch.zeros(4, 512), b(4, 64), b(512), i32, b(1, 64, 576), eps=1e-6, positions=i32, cos_sin=i32)


@pytest.mark.parametrize("shape,stride,good", [
    ((4, 8, 64), (512, 64, 1), True), ((4, 8, 64), (4608, 576, 1), True), ((8, 4, 64), (64, 512, 1), True),
    ((4, 8, 64), (0, 64, 1), False), ((4, 8, 64), (512, 0, 1), False), ((4, 8, 64), (448, 64, 1), False),
    ((1, 8, 64), (0, 64, 1), True), ((4, 1, 64), (64, 0, 1), True), ((4, 8, 64), (64, 64, 1), False),
])
def test_written_rows_must_not_overlap(shape, stride, good):
    import mla_decode_attention_05_gb300 as m
    if good:
        m.check_rows_apart(shape, stride, "q_out")
    else:
        with pytest.raises(ValueError, match="overlap"):
            m.check_rows_apart(shape, stride, "q_out")


@pytest.mark.parametrize("interleaved", [True, False])
def test_oracle_rotation(interleaved):
    """A rotation keeps a pair's length, by 0 it is the identity, and its pairs
    are the complex product with e^(i angle)."""
    rng = np.random.default_rng(1)
    x = f64_to_bf16_bits(rng.standard_normal((5, 64)))
    t = O.angle_table(1000)
    assert np.array_equal(O.rotate(x, t[[0] * 5], interleaved), x)
    pos = np.array([0, 1, 17, 400, 999])
    y = bf16_bits_to_f64(O.rotate(x, t[pos], interleaved))
    z = bf16_bits_to_f64(x)
    z = z[:, 0::2] + 1j * z[:, 1::2] if interleaved else z[:, :32] + 1j * z[:, 32:]
    w = z * np.exp(1j * pos[:, None] * 10000.0 ** (-np.arange(32) / 32))
    got = y[:, 0::2] + 1j * y[:, 1::2] if interleaved else y[:, :32] + 1j * y[:, 32:]
    assert np.all(np.abs(got - w) <= 2.0 ** -8 * np.abs(w) + 1e-6)


def test_oracle_attention():
    """Against one plain softmax over the whole masked matrix; rows without keys."""
    rng = np.random.default_rng(2)
    q, kn, kp, vv = (rng.standard_normal(s) for s in ((6, 2, 192), (4, 2, 128), (4, 64), (4, 2, 128)))
    r = O.attention(q, kn, kp, vv, 0.1, True)
    for h in range(2):
        s = 0.1 * (q[:, h, :128] @ kn[:, h].T + q[:, h, 128:] @ kp.T)
        for i in range(6):
            n = max(0, 4 - 6 + i + 1)
            if n == 0:
                assert np.isneginf(r["lse"][i, h]) and not r["out"][i, h].any()
                continue
            e = np.exp(s[i, :n])
            np.testing.assert_allclose(r["out"][i, h], e @ vv[:n, h] / e.sum(), rtol=1e-12)
            np.testing.assert_allclose(r["lse"][i, h], np.log(e.sum()), rtol=1e-12)
    vv[3] = np.nan  # a key that only the last row sees
    r2 = O.attention(q, kn, kp, vv, 0.1, True)
    assert np.array_equal(r2["out"][:5], r["out"][:5]) and np.isnan(r2["out"][5]).all()
