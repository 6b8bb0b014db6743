"""Eviction (GPU) against the rule token by token: every slot, row, scale, sum and
position exact."""
import numpy as np
import pytest
import torch

from _long import Cache, i32, table
from oracle import long_context as O

pytestmark = pytest.mark.gpu


def _expect(c, pages, lens, mass, pos, keep, sinks, recent):
    data, scales = c.data.clone(), None if c.scales is None else c.scales.clone()
    mass, pos, new = mass.clone(), pos.clone(), []
    for b, n in enumerate(lens):
        new.append(min(n, keep))
        if n <= keep:
            continue
        holes, movers = O.evict(mass[b].numpy(), pos[b].numpy(), n, keep, sinks, recent)
        for h, m in zip(holes, movers):
            a, z = (pages[b][h // 64], h % 64), (pages[b][m // 64], m % 64)
            data[a] = data[z]
            if c.fmt == "fp8":
                scales[a] = scales[z]
            mass[b, h], pos[b, h] = mass[b, m].clone(), pos[b, m].clone()
        mass[b, keep:n], pos[b, keep:n] = 0, -1
    return data, scales, mass, pos, new


def _same(got, want):
    return torch.equal(got.cpu().contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))


def _run_and_check(c, pages, lens, mass, pos, keep, sinks, recent, in_place=False):
    import mla_decode_attention_05_gb300 as mla
    data, scales = c.cuda()
    m, p, sk = mass.cuda(), pos.cuda(), i32(lens)
    new = mla.evict(data, table(pages), sk, m, p, keep=keep, sinks=sinks, recent=recent, kv_scales=scales,
                    out_seqlens=sk if in_place else None)
    w_data, w_scales, w_mass, w_pos, w_new = _expect(c, pages, lens, mass, pos, keep, sinks, recent)
    assert new.tolist() == w_new
    assert _same(p, w_pos)
    assert _same(m, w_mass)
    assert _same(data, w_data)
    if c.fmt == "fp8":
        assert _same(scales, w_scales)
    assert mla.device_status() == 0
    if not in_place:
        assert sk.tolist() == lens


def _make(seed, fmt, lens, keep, kind="lognormal", aged=True):
    rng = np.random.default_rng(seed)
    c = Cache(rng, sum(-(-n // 64) for n in lens) + 2, fmt)
    pages = [c.take(n) for n in lens]
    cap = max(1, max(lens)) + 5
    mass = np.exp(2 * rng.standard_normal((len(lens), cap))).astype(np.float32)
    if kind == "ties":
        mass = np.floor(mass).astype(np.float32)
    if kind == "odd":
        mass.reshape(-1)[::3] = np.nan
        mass.reshape(-1)[1::7] = np.inf
        mass.reshape(-1)[2::5] = -0.0
        mass.reshape(-1)[4::5] = 0.0
        mass.reshape(-1)[5::11] = -np.inf
        mass.reshape(-1)[6::13] = -1.5
    pos = np.tile(np.arange(cap, dtype=np.int32), (len(lens), 1))
    if aged:
        for b in range(len(lens)):
            pos[b] = np.sort(rng.choice(4 * cap, cap, replace=False)).astype(np.int32)
            k = min(keep, cap)
            pos[b, :k] = rng.permutation(pos[b, :k])
    return c, pages, torch.from_numpy(mass), torch.from_numpy(pos)


CASES = [
    # fmt, lens, keep, sinks, recent, kind, aged
    ("bf16", [200], 100, 4, 16, "lognormal", False),
    ("bf16", [200, 100, 101, 0, 1, 64, 300], 100, 0, 0, "lognormal", True),
    ("bf16", [130, 129], 128, 1, 127, "lognormal", True),      # nothing but what is forced
    ("bf16", [5, 2, 1], 1, 0, 1, "lognormal", False),
    ("bf16", [700], 650, 3, 20, "ties", True),
    ("bf16", [1000, 900], 64, 4, 8, "ties", False),
    ("bf16", [500, 333], 200, 2, 10, "odd", True),
    ("fp8", [200, 350, 90], 128, 4, 30, "lognormal", True),
    ("fp8_tensor", [200, 350, 90], 128, 4, 30, "ties", True),
    ("bf16", [6000, 4097, 300], 1000, 4, 100, "lognormal", True),   # a cluster to a sequence
    ("fp8", [9001], 8192, 0, 512, "ties", True),
    ("bf16", [4500], 4096, 4096, 0, "lognormal", True),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_every_slot_is_right(case):
    fmt, lens, keep, sinks, recent, kind, aged = CASES[case]
    c, pages, mass, pos = _make(500 + case, fmt, lens, keep, kind, aged)
    _run_and_check(c, pages, lens, mass, pos, keep, sinks, recent, in_place=case % 2 == 1)


def test_more_tokens_than_the_key_cache():
    """A long sequence whose sort keys do not all fit into shared memory."""
    n = 140_000
    rng = np.random.default_rng(530)
    c = Cache(rng, -(-n // 64), "fp8_tensor")
    pages = [c.take(n)]
    mass = torch.from_numpy(rng.integers(0, 1000, (1, n)).astype(np.float32))
    pos = torch.from_numpy(rng.permutation(n).astype(np.int32))[None]
    _run_and_check(c, pages, [n], mass, pos, 100_000, 100, 1000)


def test_many_sequences():
    rng = np.random.default_rng(531)
    lens = [int(x) for x in rng.integers(0, 200, 300)]
    c, pages, mass, pos = _make(532, "fp8", lens, 90)
    _run_and_check(c, pages, lens, mass, pos, 90, 2, 20)


def test_positions_that_repeat_break_nothing_but_their_order():
    c, pages, mass, pos = _make(533, "bf16", [300], 50, aged=False)
    pos[:] = 9   # all of them are the latest: the lower slots stay
    _run_and_check(c, pages, [300], mass, pos, 50, 0, 10)


def test_bad_pages_and_lengths_are_told():
    import mla_decode_attention_05_gb300 as mla
    c, pages, mass, pos = _make(534, "bf16", [300, 200], 100)
    data, _ = c.cuda()
    bt = table(pages)
    bt[0, 3] = 10 ** 6
    mla.device_status()
    m, p = mass.cuda(), pos.cuda()
    new = mla.evict(data, bt, i32([300, 200]), m, p, keep=100, recent=60)
    assert mla.device_status() == mla.STATUS_BAD_PAGE and new.tolist() == [100, 100]
    _, _, w_mass, w_pos, _ = _expect(c, pages, [300, 200], mass, pos, 100, 0, 60)
    assert _same(m, w_mass) and _same(p, w_pos)
    before = data.clone()
    new = mla.evict(data, table(pages), i32([-4, 90]), mass.cuda(), pos.cuda(), keep=100)
    assert mla.device_status() == mla.STATUS_BAD_SEQLEN and new.tolist() == [0, 90] and torch.equal(data, before)


def test_another_stream_and_a_graph():
    import mla_decode_attention_05_gb300 as mla
    lens = [300, 5000]
    c, pages, mass, pos = _make(535, "bf16", lens, 200)
    data, _ = c.cuda()
    bt, sk, m, p, new = table(pages), i32(lens), mass.cuda(), pos.cuda(), i32([0, 0])
    ws = torch.full((mla.evict_workspace_bytes(2, m.shape[1], 200),), 0xFF, dtype=torch.uint8, device="cuda")
    call = lambda: mla.evict(data, bt, sk, m, p, keep=200, sinks=4, recent=50, out_seqlens=new, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    w_data, _, w_mass, w_pos, w_new = _expect(c, pages, lens, mass, pos, 200, 4, 50)
    assert _same(data, w_data) and _same(m, w_mass) and _same(p, w_pos) and new.tolist() == w_new
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    data.copy_(c.data)
    m.copy_(mass)
    p.copy_(pos)
    sk.copy_(i32([250, 199]))
    ws.fill_(0xFF)
    g.replay()
    torch.cuda.synchronize()
    w_data, _, w_mass, w_pos, w_new = _expect(c, pages, [250, 199], mass, pos, 200, 4, 50)
    assert _same(data, w_data) and _same(m, w_mass) and _same(p, w_pos) and new.tolist() == w_new
