"""Decode over shared prefixes of FP8 caches: what becomes of own rows goes by the
tokens there are, not by how wide the tables that name their pages are."""
import numpy as np
import pytest
import torch

from _long import Cache, check_rows, i32, table
from _odd_scale import odd_scale
from _ops import bf16
from oracle import long_context as O

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


class Batch:
    def __init__(self, seed, fmt, prefixes, offsets, own, T=1, H=40):
        rng = np.random.default_rng(seed)
        self.c = Cache(rng, sum(-(-n // 64) for n in prefixes + own) + 1, fmt)
        if fmt == "fp8_tensor":   # a product of a code and this scale takes more than bf16's bits
            odd_scale(self.c)
        self.prefixes, self.offsets, self.own = prefixes, offsets, own
        self.pre, self.mine = [self.c.take(n) for n in prefixes], [self.c.take(n) for n in own]
        self.pages = sum(len(p) for p in self.mine)
        self.q = bf16(rng, (len(own), T, H, 576), 1.3)
        self.dev = (self.q.cuda(), *self.c.cuda())

    def run(self, width=None, prefix_width=None, **kw):
        import mla_decode_attention_05_gb300 as mla
        q, data, scales = self.dev
        mla.device_status()
        r = mla.decode_shared(q, data, table(self.pre, prefix_width), i32(self.prefixes), table(self.mine, width), i32(self.own),
                              softmax_scale=SCALE, group_offsets=i32(self.offsets), causal=True, kv_scales=scales, **kw)
        assert mla.device_status() == 0
        return r

    def check(self, out, lse, rounded=False, seqs=None):
        for b in range(len(self.own)) if seqs is None else seqs:
            g = [g for g in range(len(self.prefixes)) if self.offsets[g] <= b < self.offsets[g + 1]]
            prefix = self.c.exact_rows(self.pre[g[0]], self.prefixes[g[0]]) if g else np.zeros((0, 576))
            rows = (self.c.rows if rounded else self.c.exact_rows)(self.mine[b], self.own[b])
            ref = O.attention(self.q[b].double().numpy(), prefix, rows, SCALE, True)
            check_rows(out[b], lse[b].t(), ref, len(prefix) + self.own[b], self.c.fmt)


def same(a, b):
    return torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


SHAPES = {
    "few": dict(prefixes=[130, 64], offsets=[0, 1, 3], own=[9, 0, 70], T=4, H=48),
    "one token": dict(prefixes=[70], offsets=[0, 2], own=[1, 64, 65, 300, 0], T=1, H=128),
    "no prefix": dict(prefixes=[0], offsets=[0, 0], own=[5, 700, 64], T=2, H=16),
}


@pytest.mark.parametrize("shape", SHAPES)
def test_one_scale_exact_behind_a_table_of_any_width(shape):
    x = Batch(800, "fp8_tensor", **SHAPES[shape])
    narrow = x.run()
    x.check(*narrow)
    for width in (700, 1500, 5000):
        assert same(x.run(width), narrow)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("fmt", ["fp8", "fp8_tensor"])
def test_bounded_own_pages_give_equal_bits_for_any_width(fmt, shape):
    x = Batch(801, fmt, **SHAPES[shape])
    narrow = x.run()
    x.check(*narrow)
    for width in (None, 700, 1500, 5000):
        for bound in (x.pages, x.pages + 3, 2048, 2 ** 40):
            if bound <= 2048 or width in (None, 700):   # (room for all that a table could name)
                assert same(x.run(width, own_pages=bound), narrow)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("fmt", ["fp8", "fp8_tensor"])
def test_more_pages_in_use_than_the_bound(fmt, shape):
    """Own rows are rounded then, and the pages that there is room for hold nothing."""
    x = Batch(802, fmt, **SHAPES[shape])
    for bound in (0, x.pages - 1):
        for width in (None, 1500):
            x.check(*x.run(width, own_pages=bound), rounded=True)


@pytest.mark.parametrize("fmt", ["fp8", "fp8_tensor"])
def test_wide_prefix_tables(fmt):
    x = Batch(803, fmt, [130, 0, 600], [0, 1, 2, 4], [9, 30, 0, 70], T=2)
    narrow = x.run()
    x.check(*narrow)
    for width in (11, 300):
        assert same(x.run(prefix_width=width), narrow)


def test_more_than_2048_pages_of_one_scale():
    """As many as there is room for without a bound, and one more."""
    own = [64 * 1000, 64 * 1000 - 5, 64 * 48 - 63]
    x = Batch(804, "fp8_tensor", [100], [0, 3], own, T=1, H=4)
    assert x.pages == 2048
    x.check(*x.run(), seqs=[2])
    assert same(x.run(), x.run(own_pages=2048)) and same(x.run(), x.run(3000))
    x.own[2] += 63
    x.check(*x.run(), seqs=[2])
    x = Batch(804, "fp8_tensor", [100], [0, 3], own[:2] + [64 * 48 + 1], T=1, H=4)
    assert x.pages == 2049
    over = x.run()
    x.check(*over, rounded=True, seqs=[2])
    x.check(*x.run(own_pages=2049), seqs=[2])


@pytest.mark.parametrize("fmt", ["fp8", "fp8_tensor"])
def test_a_graph_goes_the_way_of_each_replay(fmt):
    import mla_decode_attention_05_gb300 as mla
    x = Batch(805, fmt, [130], [0, 3], [200, 130, 300], T=2)   # (pages for the longest of the replays)
    q, data, scales = x.dev
    pt, pl, bt, sk, off = table(x.pre), i32(x.prefixes), table(x.mine, 1500), i32(x.own), i32(x.offsets)
    ws = torch.full((mla.decode_shared_workspace_bytes(3, 2, 40, 1, mla.KV_FP8_E4M3 if fmt == "fp8" else mla.KV_FP8_E4M3_TENSOR,
                                                       pt.shape[1], 1500, own_pages=5),), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty((3, 2, 40, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((3, 40, 2), device="cuda")
    call = lambda **k: mla.decode_shared(q, data, pt, pl, bt, sk, softmax_scale=SCALE, group_offsets=off, kv_scales=scales,
                                         causal=True, own_pages=5, **k)
    call(workspace=ws, out=out, lse=lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(workspace=ws, out=out, lse=lse)
    for own in ([200, 130, 64], [64, 65, 128], [1, 0, 300], [0, 0, 0], [193, 64, 64]):   # 8, 5, 6, 0 and 6 pages
        x.own = own
        sk.copy_(i32(own))
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        x.check(out, lse, rounded=sum(-(-n // 64) for n in own) > 5)
        assert same(call(), (out, lse))
    assert mla.device_status() == 0


def test_the_short_way_and_refusals():
    import mla_decode_attention_05_gb300 as mla
    x = Batch(806, "fp8", [130], [0, 2], [200, 130], T=2)
    a = x.run(1500, own_pages=6)
    fast, mla._fast = mla._fast, None
    try:
        b = x.run(1500, own_pages=6)
    finally:
        mla._fast = fast
    assert same(a, b)
    with pytest.raises(ValueError, match="own_pages"):
        x.run(own_pages=-1)
    with pytest.raises(TypeError):
        x.run(own_pages=2.5)
    with pytest.raises(mla.MlaError, match="workspace"):
        ws = torch.empty(mla.decode_shared_workspace_bytes(2, 2, 40, 1, mla.KV_FP8_E4M3, 3, 1500, own_pages=6), dtype=torch.uint8, device="cuda")
        x.run(1500, own_pages=60, workspace=ws)
    assert mla.device_status() == 0


def test_a_bad_page_and_lengths_outside():
    """Of own tokens behind a wide table: skipped and told, as behind a narrow one."""
    import mla_decode_attention_05_gb300 as mla
    x = Batch(807, "fp8_tensor", [100], [0, 2], [200, 130])
    q, data, scales = x.dev
    got = []
    for width in (4, 1500):
        bt = table(x.mine, width)
        bt[0, 1] = x.c.pages
        mla.device_status()
        got.append(mla.decode_shared(q, data, table(x.pre), i32([100]), bt, i32([200, 130]), softmax_scale=SCALE, kv_scales=scales))
        assert mla.device_status() == mla.STATUS_BAD_PAGE
    assert same(*got)
    kept = np.delete(x.c.exact_rows(x.mine[0], 200), np.arange(64, 128), 0)
    ref = O.attention(x.q[0].double().numpy(), x.c.exact_rows(x.pre[0], 100), kept, SCALE, False)
    check_rows(got[1][0][0], got[1][1][0].t(), ref, 300, "fp8_tensor")
    bt = table(x.mine, 1500)
    mla.decode_shared(q, data, table(x.pre), i32([100]), bt, i32([-5, 130]), softmax_scale=SCALE, kv_scales=scales)
    assert mla.device_status() == mla.STATUS_BAD_SEQLEN
