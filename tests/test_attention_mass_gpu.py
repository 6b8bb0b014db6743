"""The attention weight of cached tokens (GPU) against the float64 oracle."""
import numpy as np
import pytest
import torch

from _long import Cache, i32, table
from _ops import STEP_F32, bf16, f64
from oracle import long_context as O

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


def _make(seed, fmt, T, H, lens, causal, spoil=True):
    rng = np.random.default_rng(seed)
    c = Cache(rng, sum(-(-n // 64) for n in lens) + 2, fmt)
    pages = [c.take(n) for n in lens]
    if spoil:
        c.spoil(list(zip(pages, lens)))
    q = bf16(rng, (len(lens), T, H, 576), 1.3)
    lse = torch.empty(len(lens), H, T)
    for b, n in enumerate(lens):
        ref = O.attention(q[b].double().numpy(), np.zeros((0, 576)), c.exact_rows(pages[b], n), SCALE, causal)
        lse[b] = torch.from_numpy(ref["lse"]).t()
    return c, pages, q, lse


def _check(c, pages, q, lse, lens, causal, before, decay, got):
    T, H = q.shape[1], q.shape[2]
    for b, n in enumerate(lens):
        want, bound = O.mass(q[b].double().numpy(), c.exact_rows(pages[b], n), lse[b].t().double().numpy(), SCALE, causal)
        old = decay * f64(before[b, :n]) if decay else np.zeros(n)
        err = np.abs(f64(got[b, :n]) - (want + old))
        # the weights' own bounds, a step for each addition of the T * H, and the two roundings of the update
        tol = bound + (T * H + 2) * STEP_F32 * (want + bound) + 2 * STEP_F32 * (np.abs(old) + want) + 1e-37
        assert np.all(err <= tol), (b, float(err.max()), float(tol[err.argmax()]))
        assert torch.equal(got[b, n:].cpu(), before[b, n:])


CASES = [
    # fmt, T, H, lens, causal, decay
    ("bf16", 1, 128, [1000], False, 0.0),
    ("bf16", 1, 128, [1, 63, 64, 65, 128, 129, 0, 500], False, 1.0),
    ("bf16", 1, 16, [300, 17], False, 0.9),
    ("bf16", 1, 1, [130], False, 1.0),
    ("bf16", 4, 20, [3, 200, 0, 4], True, 1.0),
    ("bf16", 4, 64, [2, 200, 257], True, 0.5),         # two tiles of query rows
    ("bf16", 3, 128, [400], False, 0.0),
    ("bf16", 64, 20, [333], True, 1.0),                 # sums in parts
    ("bf16", 40, 16, [30, 100], True, 0.9),             # tokens before the first key
    ("fp8", 1, 128, [300, 64, 1], False, 1.0),
    ("fp8", 2, 100, [129, 70], True, 0.0),
    ("fp8_tensor", 1, 40, [200, 0, 65], False, 0.9),
    ("fp8_tensor", 5, 64, [190], True, 1.0),
    ("fp8", 1, 8, [20000, 4097], False, 0.5),           # many key tiles one after the other
    ("fp8", 2, 128, [5000, 64 * 39 + 1], True, 1.0),    # and two tiles of query rows
    ("fp8", 3, 100, [5000], True, 1.0),
    ("fp8_tensor", 1, 8, [20000, 4097], False, 0.5),
    ("fp8_tensor", 64, 10, [2500], True, 1.0),
    ("fp8", 64, 10, [2500, 20], True, 1.0),
    ("fp8", 1, 1, [30000], False, 0.0),                 # few query rows: more codes on their way
    ("fp8_tensor", 1, 24, [30000, 64, 0, 200], False, 1.0),
    ("fp8_tensor", 1, 128, [20000, 100], False, 1.0),
    ("fp8_tensor", 2, 128, [9000], True, 1.0),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_the_oracle(case):
    import mla_decode_attention_05_gb300 as mla
    fmt, T, H, lens, causal, decay = CASES[case]
    mla.device_status()
    c, pages, q, lse = _make(400 + case, fmt, T, H, lens, causal)
    cap = max(64, -(-max(lens) // 64) * 64) + 3
    before = torch.rand(len(lens), cap) * 3
    if decay == 0:
        before[:] = float("nan")   # not read
        for b, n in enumerate(lens):
            before[b, n:] = 7.0
    data, scales = c.cuda()
    args = (q.cuda(), data, table(pages), i32(lens), lse.cuda())
    mass = before.cuda()
    ret = mla.attention_mass(*args, mass, softmax_scale=SCALE, causal=causal, decay=decay, kv_scales=scales)
    assert ret is mass
    _check(c, pages, q, lse, lens, causal, before, decay, mass)
    again = before.cuda()
    mla.attention_mass(*args, again, softmax_scale=SCALE, causal=causal, decay=decay, kv_scales=scales)
    assert torch.equal(again.nan_to_num(), mass.nan_to_num())
    assert mla.device_status() == 0


def test_many_tiles_over_all_sms():
    """Several sequences, and parts of sequences, in one block."""
    rng = np.random.default_rng(430)
    lens = [int(x) for x in rng.integers(0, 3000, 40)]
    c, pages, q, lse = _make(431, "bf16", 1, 4, lens, False)
    before = torch.zeros(40, 3008)
    data, _ = c.cuda()
    mass = mla_mass(q, data, pages, lens, lse, before.cuda())
    _check(c, pages, q, lse, lens, False, before, 1.0, mass)
    # every query row gives a weight of one in all
    total = mass.double().sum(1).cpu()
    assert all(abs(float(total[b]) - (4 if n else 0)) < 4e-3 for b, n in enumerate(lens))


def mla_mass(q, data, pages, lens, lse, mass, **kw):
    import mla_decode_attention_05_gb300 as mla
    return mla.attention_mass(q.cuda(), data, table(pages), i32(lens), lse.cuda(), mass, softmax_scale=SCALE, **kw)


def test_rows_without_weight_and_bad_pages():
    import mla_decode_attention_05_gb300 as mla
    lens = [100, 70]
    c, pages, q, lse = _make(432, "bf16", 1, 8, lens, False)
    lse[0, 3] = -float("inf")     # says that it saw no key
    q[1, 0, 2] = float("nan")
    before = torch.zeros(2, 128)
    data, _ = c.cuda()
    mla.device_status()
    got = mla_mass(q, data, pages, lens, lse, before.cuda())
    want, _ = O.mass(q[0].double().numpy(), c.exact_rows(pages[0], 100), lse[0].t().double().numpy(), SCALE, False)
    assert np.allclose(f64(got[0, :100]), want, rtol=1e-4, atol=1e-7)
    assert got[1, :70].isnan().all() and (got[1, 70:] == 0).all()  # a row of nan reaches what it sees, and nothing else
    bt = table(pages)
    bt[0, 1] = -5
    got = mla.attention_mass(q.cuda(), data, bt, i32(lens), lse.cuda(), torch.ones(2, 128, device="cuda"), softmax_scale=SCALE)
    assert mla.device_status() == mla.STATUS_BAD_PAGE
    assert (got[0, 64:100] == 1).all() and np.allclose(f64(got[0, :64]), want[:64] + 1, rtol=1e-4)
    mla.attention_mass(q.cuda(), data, table(pages), i32([-1, 1000]), lse.cuda(), torch.ones(2, 90, device="cuda"),
                       softmax_scale=SCALE)
    assert mla.device_status() & mla.STATUS_BAD_SEQLEN


def test_another_stream_and_a_graph():
    import mla_decode_attention_05_gb300 as mla
    lens = [400, 90]
    for T in (1, 30):
        c, pages, q, lse = _make(433, "bf16", T, 16, lens, False)
        data, _ = c.cuda()
        q, bt, sk, l = q.cuda(), table(pages), i32(lens), lse.cuda()
        cap = 448
        ws = torch.full((max(256, mla.attention_mass_workspace_bytes(2, T, 16, cap)),), 0xFF, dtype=torch.uint8, device="cuda")
        mass = torch.zeros(2, cap, device="cuda")
        call = lambda: mla.attention_mass(q, data, bt, sk, l, mass, softmax_scale=SCALE, decay=0.5, workspace=ws)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            call()
        s.synchronize()
        first = mass.clone()
        want = mla.attention_mass(q, data, bt, sk, l, torch.zeros(2, cap, device="cuda"), softmax_scale=SCALE, decay=0.5)
        assert torch.equal(first, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        sk.copy_(i32([10, 64]))
        eager = mla.attention_mass(q, data, bt, sk, l, first.clone(), softmax_scale=SCALE, decay=0.5)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(mass, eager)
