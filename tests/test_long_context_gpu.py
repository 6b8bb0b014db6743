"""The operators for long contexts together, as a serving program runs them; their
short way past the interpreter; rows of garbage; waits that run out."""
import numpy as np
import pytest
import torch

from _long import Cache, check_rows, i32, table
from _ops import HALF_BF16, bf16
from oracle import long_context as O
from oracle import prefill as OP
from test_fastcall_gpu import _taken, both  # noqa: F401

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


def _batch(seed, fmt, T, H, prefixes, own, spoil=False, std=1.3):
    rng = np.random.default_rng(seed)
    c = Cache(rng, sum(-(-n // 64) for n in prefixes + own) + 2, fmt)
    pre, mine = [c.take(n) for n in prefixes], [c.take(n) for n in own]
    if spoil:
        c.spoil(list(zip(pre, prefixes)) + list(zip(mine, own)))
    return c, pre, mine, bf16(rng, (len(own), T, H, 576), std)


@pytest.mark.parametrize("fmt,width", [("bf16", None), ("fp8", None), ("fp8", 1500), ("fp8_tensor", None), ("fp8_tensor", 1500)])
def test_what_lies_behind_the_last_token_does_not_count(fmt, width):
    """nan and inf in every row that no token holds."""
    import mla_decode_attention_05_gb300 as mla
    prefixes, own, offsets = [70, 200], [5, 0, 65, 130], [0, 2, 4]
    c, pre, mine, q = _batch(600, fmt, 2, 40, prefixes, own, spoil=True)
    data, scales = c.cuda()
    out, lse = mla.decode_shared(q.cuda(), data, table(pre), i32(prefixes), table(mine, width), i32(own), softmax_scale=SCALE,
                                 group_offsets=i32(offsets), causal=True, kv_scales=scales)
    for b, g in enumerate([0, 0, 1, 1]):
        rows = (c.rows if width else c.exact_rows)(mine[b], own[b])  # (a wide table's own rows go through the decode kernel)
        ref = O.attention(q[b].double().numpy(), c.exact_rows(pre[g], prefixes[g]), rows, SCALE, True)
        check_rows(out[b], lse[b].t(), ref, prefixes[g] + own[b], fmt)


def test_scores_that_grow_a_lot():
    """A row's later keys outweigh its first ones by more than 2^32: the running
    reference moves, and what was summed before is scaled down."""
    import mla_decode_attention_05_gb300 as mla
    rng = np.random.default_rng(601)
    c = Cache(rng, 12, "bf16")
    c.data[:] *= 0.25
    n = 640
    pages = c.take(n)
    for i, j in enumerate((3, 5, 9)):   # three pages ever larger
        c.data[pages[j]] *= 4 * 3 ** i
    c.exact = c.data.double()
    q = bf16(rng, (3, 1, 16, 576), 2.0)
    out, lse = mla.decode_shared(q.cuda(), c.data.cuda(), table([pages]), i32([n]), table([[]] * 3, 1), i32([0, 0, 0]),
                                 softmax_scale=SCALE)
    for b in range(3):
        ref = O.attention(q[b].double().numpy(), c.exact_rows(pages, n), np.zeros((0, 576)), SCALE, False)
        assert (ref["top"] > 60).any()
        check_rows(out[b], lse[b].t(), ref, n)


def test_the_short_way_gives_the_same(both):  # noqa: F811
    import mla_decode_attention_05_gb300 as mla
    for fmt in ("bf16", "fp8", "fp8_tensor"):
        prefixes, own = [100], [70, 9]
        c, pre, mine, q = _batch(602, fmt, 2, 8, prefixes, own)
        data, sc = c.cuda()
        q, pt, pl, bt, sk = q.cuda(), table(pre), i32(prefixes), table(mine), i32(own)
        f = lambda **k: mla.decode_shared(q, data, pt, pl, bt, sk, softmax_scale=SCALE, causal=True, kv_scales=sc, **k)
        a, b = both(f)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and _taken(f)
        out, lse = torch.empty_like(a[0]), torch.empty_like(a[1])
        a2, b2 = both(lambda: f(out=out, lse=lse, group_offsets=i32([0, 2])))
        assert a2[0].data_ptr() == out.data_ptr() == b2[0].data_ptr() and torch.equal(out, a[0])
        mass = lambda: mla.attention_mass(q, data, bt, sk, a[1], torch.ones(2, 130, device="cuda"), softmax_scale=SCALE,
                                          causal=True, decay=0.5, kv_scales=sc)
        sums, y = both(mass)
        assert torch.equal(sums, y) and _taken(mass)
        pos = torch.arange(130, dtype=torch.int32, device="cuda").repeat(2, 1)

        def evict():
            d, m, p, s = data.clone(), sums.clone(), pos.clone(), None if sc is None else sc.clone()
            n = mla.evict(d, bt, sk, m, p, keep=40, sinks=2, recent=10, kv_scales=s)
            return [d.view(torch.uint8), m, p, n] + ([s] if s is not None else [])
        x, y = both(evict)
        assert all(torch.equal(i, j) for i, j in zip(x, y)) and _taken(evict)


def test_refusals_are_pythons():
    import mla_decode_attention_05_gb300 as mla
    c, pre, mine, q = _batch(603, "bf16", 1, 8, [100], [70, 9])
    data, _ = c.cuda()
    q, pt, pl, bt, sk = q.cuda(), table(pre), i32([100]), table(mine), i32([70, 9])
    call = lambda **k: mla.decode_shared(**{**dict(q=q, kv_cache=data, prefix_table=pt, prefix_lens=pl, block_table=bt,
                                                   cache_seqlens=sk, softmax_scale=SCALE), **k})
    with pytest.raises(ValueError, match="q must be"):
        call(q=q[..., :512].contiguous())
    with pytest.raises(ValueError, match="prefix_lens"):
        call(prefix_lens=i32([1, 2]))
    with pytest.raises(ValueError, match="group_offsets"):
        call(group_offsets=i32([0, 1, 2]))
    with pytest.raises(ValueError, match="group_offsets"):
        call(prefix_table=pt.repeat(2, 1), prefix_lens=i32([1, 2]))
    with pytest.raises(ValueError, match="batch"):
        call(cache_seqlens=i32([1]))
    with pytest.raises(ValueError, match="contiguous"):
        call(q=q.repeat(1, 1, 1, 2)[..., :576])
    with pytest.raises(mla.MlaError, match="workspace"):
        call(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(mla.MlaError, match="softmax_scale"):
        call(softmax_scale=0.0)
    lse, mass, pos = torch.zeros(2, 8, 1, device="cuda"), torch.zeros(2, 128, device="cuda"), torch.zeros(2, 128, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="lse"):
        mla.attention_mass(q, data, bt, sk, lse[:, :4].contiguous(), mass, softmax_scale=SCALE)
    with pytest.raises(ValueError, match="mass"):
        mla.attention_mass(q, data, bt, sk, lse, mass[:1], softmax_scale=SCALE)
    with pytest.raises(mla.MlaError, match="decay"):
        mla.attention_mass(q, data, bt, sk, lse, mass, softmax_scale=SCALE, decay=-1.0)
    with pytest.raises(ValueError, match="positions"):
        mla.evict(data, bt, sk, mass, pos[:, :100].contiguous(), keep=10)
    with pytest.raises(TypeError, match="positions"):
        mla.evict(data, bt, sk, mass, pos.long(), keep=10)
    with pytest.raises(mla.MlaError, match="sinks"):
        mla.evict(data, bt, sk, mass, pos, keep=10, sinks=6, recent=5)
    with pytest.raises(mla.MlaError):
        mla.evict(data, bt, sk, mass, pos, keep=0)
    assert mla.device_status() == 0


def test_a_cache_that_stays_small():
    """Samples of one prompt: decode behind the shared prefix, the weights of the own
    tokens from that decode's log-sum-exp, an eviction every eight steps, the next
    tokens appended by the rotating insert.  What the operators kept is what a plain
    program keeps, and attention over it agrees."""
    import mla_decode_attention_05_gb300 as mla
    rng = np.random.default_rng(610)
    B, H, P, keep, cap = 3, 8, 150, 32, 64
    c = Cache(rng, 12, "bf16")
    pre, mine = c.take(P), [c.take(cap) for _ in range(B)]
    data, _ = c.cuda()
    pt, pl, bt = table([pre]), i32([P]), table(mine)
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    angles = torch.from_numpy(OP.angle_table(1000)).cuda()
    mass, pos = torch.zeros(B, cap, device="cuda"), torch.full((B, cap), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    # the plain program: rows, sums and positions of each slot
    rows, sums, where = [[] for _ in range(B)], [[] for _ in range(B)], [[] for _ in range(B)]
    for step in range(70):
        kv, q = bf16(rng, (B, 576)).cuda(), bf16(rng, (B, 1, H, 576), 1.3).cuda()
        n = len(rows[0])
        slots = torch.tensor([mine[b][n // 64] * 64 + n % 64 for b in range(B)], device="cuda")
        at = torch.full((B,), P + step, dtype=torch.int64, device="cuda")
        mla.kv_insert_rope(kv[:, :512], kv[:, 512:], w, slots, data, eps=1e-6, positions=at, cos_sin=angles, q_pe=q[:, 0, :, 512:])
        pos[:, n] = P + step
        lens += 1
        out, lse = mla.decode_shared(q, data, pt, pl, bt, lens, softmax_scale=SCALE)
        mla.attention_mass(q, data, bt, lens, lse, mass, softmax_scale=SCALE)
        flat = data.view(-1, 576)[slots].double().cpu().numpy()
        for b in range(B):
            rows[b].append(flat[b])
            sums[b].append(0.0)
            where[b].append(P + step)
            own, qb = np.array(rows[b]), q[b].double().cpu().numpy()
            ref = O.attention(qb, c.exact_rows(pre, P), own, SCALE, False)
            check_rows(out[b], lse[b].t(), ref, P + len(own))
            weights, _ = O.mass(qb, own, lse[b].t().double().cpu().numpy(), SCALE, False)
            sums[b] = list(np.array(sums[b]) + weights)
        got = mass.double().cpu().numpy()
        for b in range(B):
            np.testing.assert_allclose(got[b, :n + 1], sums[b], rtol=2e-4)
            sums[b] = list(got[b, :n + 1])     # so that near ties fall as they fell there
        if step % 8 == 7:
            lens = mla.evict(data, bt, lens, mass, pos, keep=keep, recent=8)
            for b in range(B):
                holes, movers = O.evict(np.array(sums[b], np.float32), np.array(where[b]), n + 1, keep, 0, 8)
                for h, m in zip(holes, movers):
                    rows[b][h], sums[b][h], where[b][h] = rows[b][m], sums[b][m], where[b][m]
                rows[b], sums[b], where[b] = rows[b][:keep], sums[b][:keep], where[b][:keep]
            assert lens.tolist() == [len(rows[0])] * B
            assert [p[:len(rows[0])] for p in pos.tolist()] == where
    assert len(rows[0]) < 50 and mla.device_status() == 0


def _shared(mla, fmt="bf16", width=None):
    prefixes, own = [3000], [400, 130, 700]
    c, pre, mine, q = _batch(620, fmt, 1, 64, prefixes, own)
    data, sc = c.cuda()
    args = (q.cuda(), data, table(pre), i32(prefixes), table(mine, width), i32(own))
    return lambda: mla.decode_shared(*args, softmax_scale=SCALE, kv_scales=sc)


def _mass(mla, T, fmt="bf16"):
    lens = [3000, 400, 1700]
    c, _, pages, q = _batch(621, fmt, T, 64, [], lens)
    data, sc = c.cuda()
    args = (q.cuda(), data, table(pages), i32(lens), torch.full((3, 64, T), 9.0, device="cuda"))
    return lambda: (mla.attention_mass(*args, torch.zeros(3, 3008, device="cuda"), softmax_scale=SCALE, kv_scales=sc),)


CASES = {
    "shared": lambda m: _shared(m), "shared_fp8": lambda m: _shared(m, "fp8"), "shared_fp8_wide": lambda m: _shared(m, "fp8", 1500),
    "mass": lambda m: _mass(m, 1), "mass_many_rows": lambda m: _mass(m, 12), "mass_fp8": lambda m: _mass(m, 1, "fp8"),
    "mass_fp8_many_rows": lambda m: _mass(m, 12, "fp8_tensor"),
}


@pytest.mark.parametrize("case", CASES)
def test_waits_run_out_then_next_call_is_correct(case):
    """Ordinary calls with the limit of every wait shortened to a microsecond: the
    status word tells, and the calls behind are right."""
    import mla_decode_attention_05_gb300 as mla
    call = CASES[case](mla)
    mla.device_status()
    want = call()
    assert mla.device_status() == 0
    mla.set_wait_limit_ns(1000)
    try:
        call()
    finally:
        mla.set_wait_limit_ns(0)
    behind = call()
    assert mla.device_status() == mla.STATUS_WAIT_TIMEOUT, "no wait ran out"
    after = call()
    assert mla.device_status() == 0
    assert all(torch.equal(a, b) for got in (behind, after) for a, b in zip(got, want))


def test_two_graphs_with_a_workspace_each():
    """Captured calls on two streams at once, each with its own workspace."""
    import mla_decode_attention_05_gb300 as mla
    prefixes, own = [700], [90, 300]
    c, pre, mine, q = _batch(630, "bf16", 1, 32, prefixes, own)
    data, _ = c.cuda()
    q, pt, pl, bt, sk = q.cuda(), table(pre), i32(prefixes), table(mine), i32(own)
    want = mla.decode_shared(q, data, pt, pl, bt, sk, softmax_scale=SCALE)
    size = mla.decode_shared_workspace_bytes(2, 1, 32, 1, mla.KV_BF16, pt.shape[1], bt.shape[1])
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mla.decode_shared(q, data, pt, pl, bt, sk, softmax_scale=SCALE, workspace=ws, out=out, lse=lse)
        graphs.append((g, ws))
        outs.append((out, lse))
    for _ in range(5):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(l, want[1]) for o, l in outs)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_many_small_groups_and_sequences(fmt):
    """More groups than the schedule keeps at hand, more sequences than it has
    threads, groups without sequences and prefixes of no tokens among them."""
    import mla_decode_attention_05_gb300 as mla
    rng = np.random.default_rng(620)
    G, B = 700, 1300
    prefixes = [int(x) for x in rng.integers(0, 3, G)]
    own = [int(x) for x in rng.integers(0, 3, B)]
    cuts = np.sort(rng.integers(0, B + 1, G + 1))
    prefixes[5], own[7], own[B - 1] = 130, 70, 66
    c = Cache(rng, sum(-(-n // 64) for n in prefixes + own), fmt)
    pre, mine = [c.take(n) for n in prefixes], [c.take(n) for n in own]
    q = bf16(rng, (B, 1, 2, 576), 1.3)
    data, scales = c.cuda()
    mla.device_status()
    out, lse = mla.decode_shared(q.cuda(), data, table(pre), i32(prefixes), table(mine), i32(own), softmax_scale=SCALE,
                                 group_offsets=i32([int(x) for x in cuts]), kv_scales=scales)
    assert mla.device_status() == 0
    group = {}
    for g in range(G):
        for b in range(cuts[g], cuts[g + 1]):
            group[b] = g
    out, lse = out.cpu(), lse.cpu()
    for b in list(range(0, B, 13)) + [7, B - 1, cuts[5], min(B - 1, cuts[6])]:
        prefix = c.exact_rows(pre[group[b]], prefixes[group[b]]) if b in group else np.zeros((0, 576))
        rounded = B * table(mine).shape[1] > 2048 and fmt != "bf16"
        ref = O.attention(q[b].double().numpy(), prefix, (c.rows if rounded else c.exact_rows)(mine[b], own[b]), SCALE, False)
        check_rows(out[b], lse[b].t(), ref, len(prefix) + own[b], fmt)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_tensor"])
def test_weights_and_eviction_of_many_sequences(fmt):
    import mla_decode_attention_05_gb300 as mla
    rng = np.random.default_rng(621)
    B, cap = 3001, 64
    own = [int(x) for x in rng.integers(0, 4, B)]
    own[0] = own[B - 1] = 64
    c = Cache(rng, sum(-(-n // 64) for n in own), fmt)
    mine = [c.take(n) for n in own]
    q = bf16(rng, (B, 1, 2, 576), 1.0)
    data, scales = c.cuda()
    bt, sk = table(mine), i32(own)
    lse = torch.full((B, 2, 1), 3.0, device="cuda")
    mass = mla.attention_mass(q.cuda(), data, bt, sk, lse, torch.zeros(B, cap, device="cuda"), softmax_scale=SCALE, kv_scales=scales)
    got = mass.cpu()
    for b in list(range(0, B, 29)) + [B - 1]:
        want, bound = O.mass(q[b].double().numpy(), c.exact_rows(mine[b], own[b]), lse[b].t().double().cpu().numpy(), SCALE, False)
        # a step for each of the two additions beside the weights' own bounds
        assert np.all(np.abs(got[b, :own[b]].double().numpy() - want) <= bound + 4 * 2.0 ** -24 * (want + bound))
        assert (got[b, own[b]:] == 0).all()
    pos = torch.arange(cap, dtype=torch.int32, device="cuda").repeat(B, 1)
    before, plain = data.clone(), mass.clone()
    n = mla.evict(data, bt, sk, mass, pos, keep=2, recent=1, kv_scales=scales)
    assert n.tolist() == [min(x, 2) for x in own] and mla.device_status() == 0
    for b in list(range(0, B, 31)) + [B - 1]:
        holes, movers = O.evict(plain[b].cpu().numpy(), np.arange(cap), own[b], 2, 0, 1)
        for h, m in zip(holes, movers):
            assert torch.equal(data[mine[b][0], h], before[mine[b][0], m]) and int(pos[b, h]) == m
            assert mass[b, h] == plain[b, m]


def test_two_calls_at_once():
    """On two streams, with workspaces of their own."""
    import mla_decode_attention_05_gb300 as mla
    own, prefixes = [300, 700, 90, 5], [3000]
    c, pre, mine, q = _batch(622, "fp8", 2, 64, prefixes, own)
    data, scales = c.cuda()
    q, pt, pl, bt, sk = q.cuda(), table(pre), i32(prefixes), table(mine), i32(own)
    shared = lambda: mla.decode_shared(q, data, pt, pl, bt, sk, softmax_scale=SCALE, causal=True, kv_scales=scales)
    want = shared()
    weigh = lambda: mla.attention_mass(q, data, bt, sk, want[1], torch.zeros(4, 704, device="cuda"), softmax_scale=SCALE, causal=True,
                                       kv_scales=scales)
    sums = weigh()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(4)], []
    for k in range(12):
        with torch.cuda.stream(streams[k % 4]):
            got.append(shared() if k % 2 else weigh())
    torch.cuda.synchronize()
    for k, r in enumerate(got):
        if k % 2:
            assert torch.equal(r[0], want[0]) and torch.equal(r[1], want[1])
        else:
            assert torch.equal(r[:, :90], sums[:, :90])
    assert mla.device_status() == 0
