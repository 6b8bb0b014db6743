"""The operators together, as a serving program runs them: a prompt into the
cache, its attention, and decode steps behind it; on another stream; captured
into CUDA graphs."""
import numpy as np
import pytest
import torch

from _ops import bf16, cu, f64
from oracle import prefill as O

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5
EPS = 1e-6


class Layer:
    """Random weights of one attention layer and a paged cache."""

    def __init__(self, H, pages, seed, fmt="bf16"):
        rng = np.random.default_rng(seed)
        self.H, self.fmt = H, fmt
        self.w_qa = (torch.ones(1536) + 0.1 * bf16(rng, (1536,)).float()).to(torch.bfloat16).cuda()
        self.w_kva = (torch.ones(512) + 0.1 * bf16(rng, (512,)).float()).to(torch.bfloat16).cuda()
        self.w_qb = bf16(rng, (H * 192, 1536), 1536 ** -0.5).cuda()
        self.w_kvb = bf16(rng, (H, 256, 512), 512 ** -0.5).cuda()
        self.w_uk = self.w_kvb[:, :128].contiguous()
        self.table = torch.from_numpy(O.angle_table(2048)).cuda()
        self.cache = torch.zeros((pages, 64, 576), dtype=torch.bfloat16, device="cuda")


def _expanded_queries(layer, q_a):
    """The prompt's 192-wide queries by plain matrix products."""
    x = q_a.float()
    x = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * layer.w_qa.float()
    return (x.to(torch.bfloat16).float() @ layer.w_qb.float().T).to(torch.bfloat16).view(len(q_a), layer.H, 192)


@pytest.mark.parametrize("H", [8, 64])
def test_prompt_and_decode_agree(H):
    """The last tokens of prompts, once as prefill rows and once as decode
    steps (absorbed form): the same values up to the roundings of bf16."""
    import mla_decode_attention_05_gb300 as mla
    lens = [130, 77, 300]
    n = sum(lens)
    layer = Layer(H, 12, 20)
    rng = np.random.default_rng(21)
    qkv = bf16(rng, (n, 2112)).cuda()
    per = [-(-m // 64) for m in lens]
    bt = torch.full((3, max(per)), -1, dtype=torch.int32)
    ids = torch.from_numpy(rng.permutation(12).astype(np.int32))
    at = 0
    for b, m in enumerate(per):
        bt[b, :m] = ids[at:at + m]
        at += m
    pos = torch.cat([torch.arange(m) for m in lens])
    seq = torch.cat([torch.full((m,), b) for b, m in enumerate(lens)])
    slots = bt[seq, pos // 64].long() * 64 + pos % 64
    bt, pos_d, slots = bt.cuda(), pos.cuda(), slots.cuda()
    q = _expanded_queries(layer, qkv[:, :1536])
    mla.device_status()
    mla.kv_insert_rope(qkv[:, 1536:2048], qkv[:, 2048:], layer.w_kva, slots, layer.cache, eps=EPS, positions=pos_d,
                       cos_sin=layer.table, q_pe=q[..., 128:])
    kv, pe = mla.kv_expand(layer.cache, bt, cu(lens), layer.w_uk, layer.w_kvb[:, 128:], total=n)
    out, lse = mla.prefill(q, kv[..., :128], pe, kv[..., 128:], cu(lens), cu(lens), softmax_scale=SCALE)

    last = torch.tensor(np.cumsum(lens) - 1, device="cuda")
    qd = mla.query_absorb(qkv[last, :1536], layer.w_qa, layer.w_qb, layer.w_uk, eps=EPS)
    # the tokens are in the cache already: rotate the queries alone (no slots)
    mla.kv_insert_rope(qkv[last, 1536:2048], qkv[last, 2048:], layer.w_kva, torch.full((3,), -1, device="cuda"),
                       layer.cache, eps=EPS, positions=pos_d[last], cos_sin=layer.table, q_pe=qd[..., 512:])
    sk = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, l = mla.decode(qd.view(3, 1, H, 576), layer.cache, bt, sk, softmax_scale=SCALE)
    vals = mla.value_project(o.view(3, H, 512), layer.w_kvb[:, 128:])
    assert mla.device_status() == 0
    # Relative to the largest value.  Per path a handful of bf16 roundings (2^-8 each) lie between inputs and
    # output: Q_B, W_UK or the expanded key, the probabilities, the expanded value or the decode's output, the
    # result.  Scores of order one carry the first three into the weights, so six half steps on each side.
    a, b = f64(out[last]), f64(vals)
    assert np.abs(a - b).max() <= 12 * 2.0 ** -8 * np.abs(a).max()
    assert np.abs(f64(lse[:, last].T) - f64(l[:, :, 0])).max() <= 12 * 2.0 ** -8 * max(1.0, np.abs(f64(l)).max())


def _chunk_state(seed, H=4, lens=(200, 90)):
    rng = np.random.default_rng(seed)
    layer = Layer(H, 8, seed)
    n = sum(lens)
    pos = torch.cat([torch.arange(m) for m in lens]).cuda()
    bt = torch.tensor([[0, 1, 2, 3], [4, 5, -1, -1]], dtype=torch.int32, device="cuda")
    seq = torch.cat([torch.full((m,), b) for b, m in enumerate(lens)]).cuda()
    return dict(layer=layer, qkv=bf16(rng, (n, 2112)).cuda(), q=bf16(rng, (n, H, 192), 1.5).cuda(), pos=pos, bt=bt,
                slots=bt[seq, pos // 64].long() * 64 + pos % 64, cu=cu(lens), n=n,
                q_out=torch.empty((n, H, 64), dtype=torch.bfloat16, device="cuda"))


def _chunk(s):
    import mla_decode_attention_05_gb300 as mla
    L = s["layer"]
    mla.kv_insert_rope(s["qkv"][:, 1536:2048], s["qkv"][:, 2048:], L.w_kva, s["slots"], L.cache, eps=EPS,
                       positions=s["pos"], cos_sin=L.table, q_pe=s["q"][..., 128:], q_out=s["q_out"])
    kv, pe = mla.kv_expand(L.cache, s["bt"], s["cu"], L.w_uk, L.w_kvb[:, 128:], total=s["n"])
    out, lse = mla.prefill(s["q"], kv[..., :128], pe, kv[..., 128:], s["cu"], s["cu"], softmax_scale=SCALE)
    vals = mla.value_project(kv.view(s["n"], -1, 512), L.w_kvb[:kv.shape[1] // 2, 128:])
    return s["q_out"], kv, pe, out, lse, vals


def test_other_stream_and_graph_replay():
    """The same bits on a side stream and from replayed graphs, two of which
    alternate, after their inputs have changed."""
    a, b = _chunk_state(31), _chunk_state(32)
    want = [[t.clone() for t in _chunk(s)] for s in (a, b)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = _chunk(a)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want[0]))
    graphs, outs = [], []
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_chunk(s))
        graphs.append(g)
    for _ in range(2):
        for o in outs:
            for t in o:
                t.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(x, y) for x, y in zip(o, w))
    a["qkv"].copy_(b["qkv"]), a["q"].copy_(b["q"])  # a graph reads its inputs at replay
    a["layer"].w_kva.copy_(b["layer"].w_kva), a["layer"].w_uk.copy_(b["layer"].w_uk)
    a["layer"].w_kvb.copy_(b["layer"].w_kvb)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs[0], want[1]))


def test_runs_give_the_same_bits():
    s = _chunk_state(33)
    first = [t.clone() for t in _chunk(s)]
    for _ in range(5):
        assert all(torch.equal(x, y) for x, y in zip(_chunk(s), first))


@pytest.mark.parametrize("H,lens", [(16, [40] * 64), (128, [500, 64, 3000])])
def test_a_projection_right_behind_its_decode(H, lens):
    """Sequences of one part and of several: the projection starts while the
    decode's last kernel ends, and reads what the decode itself wrote.  Eager and
    replayed without a pause, the bits of calls that wait for one another."""
    import mla_decode_attention_05_gb300 as mla
    rng = np.random.default_rng(41)
    B = len(lens)
    per = [-(-m // 64) for m in lens]
    bt = torch.zeros((B, max(per)), dtype=torch.int32)
    for b, m in enumerate(per):
        bt[b, :m] = torch.arange(sum(per[:b]), sum(per[:b + 1]))
    bt, sk = bt.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    cache = bf16(rng, (sum(per), 64, 576)).cuda()
    w_uv = bf16(rng, (H, 128, 512), 512 ** -0.5).cuda()
    qs = [bf16(rng, (B, 1, H, 576), 0.3).cuda() for _ in range(4)]
    q = torch.empty_like(qs[0])

    def step(x, wait=False):
        q.copy_(x)
        o, _ = mla.decode(q, cache, bt, sk, softmax_scale=SCALE)
        if wait:
            torch.cuda.synchronize()
        return mla.value_project(o.view(B, H, 512), w_uv)
    mla.device_status()
    want = [step(x, True).clone() for x in qs]
    for _ in range(5):
        got = [step(x) for x in qs]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = [step(x) for x in qs]
    for _ in range(5):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert mla.device_status() == 0
