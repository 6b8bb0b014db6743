"""Queries of nan or inf, and products that overflow: what the softmax makes of
them comes out, and is not taken for a row without keys."""
import numpy as np
import pytest
import torch

from _long import Cache, i32, table
from _ops import bf16

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5
NAN, INF = float("nan"), float("inf")
DIM = 570          # of the rotated part, so that no value holds it
HUGE = 2.0 ** 120  # its square is beyond fp32, it is not


class Batch:
    """Two sequences behind a prefix each (tokens of 0: none).  No query has anything in DIM, so
    what the cache holds there counts for nobody until one has."""

    def __init__(self, seed, fmt, prefixes, own, T=2, H=40, width=None):
        rng = np.random.default_rng(seed)
        self.c = Cache(rng, sum(-(-n // 64) for n in prefixes + own) + 1, fmt)
        self.prefixes, self.own, self.width = prefixes, own, width
        self.pre, self.mine = [self.c.take(n) for n in prefixes], [self.c.take(n) for n in own]
        self.q = bf16(rng, (len(own), T, H, 576), 1.3)
        self.q[..., DIM] = 0
        for pages, n in list(zip(self.pre, prefixes)) + list(zip(self.mine, own)):
            self.set_dim(pages, n, 0)

    def seen(self, b):
        """The keys of sequence b, without DIM."""
        return np.concatenate([self.c.exact_rows(self.pre[b], self.prefixes[b]), self.c.exact_rows(self.mine[b], self.own[b])])

    def set_dim(self, pages, n, value):
        """DIM of the first n tokens behind a page list (not 0: bf16 rotated parts)."""
        flat = self.c.data.view(self.c.pages * 64, -1)
        for i in range(n):
            row = flat[pages[i // 64] * 64 + i % 64]
            if self.c.fmt != "fp8":
                row[DIM] = value
            else:
                row[512:].view(torch.bfloat16)[DIM - 512] = value

    def run(self, q=None, causal=False):
        import mla_decode_attention_05_gb300 as mla
        data, scales = self.c.cuda()
        q = (self.q if q is None else q).cuda()
        bt, sk = table(self.mine, self.width), i32(self.own)
        out, lse = mla.decode_shared(q, data, table(self.pre), i32(self.prefixes), bt, sk, softmax_scale=SCALE,
                                     group_offsets=i32(list(range(len(self.own) + 1))), causal=causal, kv_scales=scales)
        mass = mla.attention_mass(q, data, bt, sk, lse, torch.zeros(len(self.own), bt.shape[1] * 64, device="cuda"),
                                  softmax_scale=SCALE, causal=causal, kv_scales=scales)
        assert mla.device_status() == 0
        return out.cpu(), lse.cpu(), mass.cpu()


def _only_this_row(base, got, row):
    """Every other row is what it was, bit by bit."""
    (out, lse, _), (b, t, h) = got, row
    rest = torch.ones(out.shape[:3], dtype=torch.bool)
    rest[row] = False
    assert torch.equal(out[rest], base[0][rest])
    assert torch.equal(lse.transpose(1, 2)[rest], base[1].transpose(1, 2)[rest])
    return out[b, t, h], lse[b, h, t]


SHAPES = {  # prefixes, own
    "one worker": ([0, 0], [50, 3]),
    "a prefix": ([70, 0], [50, 64]),
    "only a prefix": ([200, 130], [0, 5]),
    "many workers": ([4000, 100], [300, 3000]),
    "many workers, no prefix": ([0, 0], [3000, 90]),
}


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_tensor"])
def test_a_query_of_nan_or_inf(fmt, shape, bad):
    prefixes, own = SHAPES[shape]
    x = Batch(700, fmt, prefixes, own)
    base = x.run()
    assert torch.isfinite(base[0].float()).all() and torch.isfinite(base[1]).all()
    for row in ((0, 1, 7), (1, 0, 39)):
        q = x.q.clone()
        q[row][17] = bad
        got = x.run(q)
        out, lse = _only_this_row(base, got, row)
        with np.errstate(invalid="ignore"):
            scores = bad * x.seen(row[0])[:, 17]
        all_low = bool((scores == -INF).all())   # (of few keys all may be on one side)
        assert out.isnan().all() and (lse == -INF if all_low else lse.isnan())
        n = own[row[0]]   # and it reaches the sums of the tokens that the row sees
        assert all_low or got[2][row[0], :n].isnan().all()
        assert torch.equal(got[2][1 - row[0]], base[2][1 - row[0]])


@pytest.mark.parametrize("where", ["prefix", "own"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_scores_that_overflow_in_one_part(fmt, sign, where):
    """+inf beside finite scores: 0 * inf in the softmax.  -inf beside them: no weight."""
    prefixes, own = [200, 0], [90, 3]
    x = Batch(701, fmt, prefixes, own)
    x.set_dim(*((x.pre[0], 200) if where == "prefix" else (x.mine[0], 90)), sign * HUGE)
    base, row = x.run(), (0, 1, 30)
    q = x.q.clone()
    q[row][DIM] = HUGE
    out, lse = _only_this_row(base, x.run(q), row)
    if sign > 0:
        assert out.isnan().all() and lse.isnan()
        return
    only = Batch(701, fmt, prefixes, own)   # the same without the tokens of that part
    (only.prefixes if where == "prefix" else only.own)[0] = 0
    want = only.run()
    # Scores of 576 products whose sizes sum to about 35, off by 576 * 2^-23 * 35 in each call: 2.4e-3.  Weights by
    # three times that and half a bf16 step, values of 0.8 on average.
    assert abs(lse - want[1][0, 30, 1]) < 5e-3
    assert (out.float() - want[0][row].float()).abs().max() < 2 * 0.8 * (2 * 2.0 ** -8 + 3 * 2.4e-3)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_scores_that_are_all_minus_inf(fmt, shape):
    """0 / 0, as the prefill gives it; a causal row without keys beside it is still 0."""
    prefixes, own = SHAPES[shape]
    x = Batch(702, fmt, prefixes, own)
    for pages, n in list(zip(x.pre, prefixes)) + list(zip(x.mine, own)):
        x.set_dim(pages, n, -HUGE)
    base = x.run()
    for row in ((0, 1, 7), (1, 0, 39)):
        q = x.q.clone()
        q[row][DIM] = HUGE
        out, lse = _only_this_row(base, x.run(q), row)
        assert out.isnan().all() and lse == -INF


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_tensor"])
def test_a_row_that_sees_no_key_stays_empty_whatever_its_query(fmt):
    x = Batch(703, fmt, [0, 0], [1, 130], T=2)
    q = x.q.clone()
    q[0, 0, 5] = NAN     # causal: token 0 of 2 sees nothing of one key
    q[0, 0, 6, 3] = INF
    out, lse, mass = x.run(q, causal=True)
    assert not out[0, 0].any() and (lse[0, :, 0] == -INF).all()
    assert torch.isfinite(out[0, 1].float()).all() and torch.isfinite(mass).all()


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("fmt", ["fp8", "fp8_tensor"])
def test_behind_a_wide_page_table(fmt, bad):
    x = Batch(704, fmt, [130, 0], [70, 1500], width=1500)
    base = x.run()
    for row in ((0, 1, 7), (1, 0, 39)):
        q = x.q.clone()
        q[row][17] = bad
        out, lse = _only_this_row(base, x.run(q), row)
        assert out.isnan().all() and lse.isnan()
    if fmt == "fp8":
        for pages, n in list(zip(x.pre, x.prefixes)) + list(zip(x.mine, x.own)):
            x.set_dim(pages, n, -HUGE)
        base, q = x.run(), x.q.clone()
        q[1, 0, 39, DIM] = HUGE
        out, lse = _only_this_row(base, x.run(q), (1, 0, 39))
        assert out.isnan().all() and lse == -INF


def _decode(x, q, parts, causal=False, topk=None):
    import mla_decode_attention_05_gb300 as mla
    data, scales = x.c.cuda()
    sk, T, H = i32(x.own), q.shape[1], q.shape[2]
    md, ns = mla.metadata(sk, H, T, topk=0 if topk is None else topk.shape[2], causal=causal, num_parts=parts)
    out, lse = mla.decode(q.cuda(), data, table(x.mine), sk, softmax_scale=SCALE, causal=causal, kv_scales=scales,
                          topk_indices=topk, tile_md=md, num_splits=ns)
    assert mla.device_status() == 0
    return out.cpu(), lse.cpu(), ns.cpu()


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("parts", [1, 3, 76])
@pytest.mark.parametrize("fmt,way", [("bf16", "dense"), ("bf16", "causal"), ("bf16", "topk"), ("bf16", "dual"), ("fp8", "dense"),
                                     ("fp8", "topk"), ("fp8_tensor", "causal")])
def test_decode_whole_and_in_parts(fmt, way, parts, bad):
    import mla_decode_attention_05_gb300 as mla
    x = Batch(705, fmt, [0, 0], [3000, 90], T=2, H=32 if way == "dual" else 40)
    topk = None
    if way == "topk":
        rng = np.random.default_rng(706)
        topk = i32([[rng.permutation(n)[:64].tolist() for _ in range(2)] for n in x.own])
    call = lambda q: _decode(x, q, parts, way == "causal", topk)
    mla.set_dual_gemm(way == "dual")
    try:
        base = call(x.q)
        if parts == 3 and topk is None:
            assert (base[2].diff() > 1).any()
        for row in ((0, 1, 7), (1, 0, 31)):
            q = x.q.clone()
            q[row][17] = bad
            out, lse = _only_this_row(base, call(q), row)
            assert out.isnan().all() and lse.isnan()
        if fmt == "fp8_tensor":
            return
        for sign in (-1, 1):
            for pages, n in zip(x.mine, x.own):
                x.set_dim(pages, n, sign * HUGE)
            base = call(x.q)
            for row in ((0, 1, 7), (1, 0, 31)):
                q = x.q.clone()
                q[row][DIM] = HUGE
                out, lse = _only_this_row(base, call(q), row)
                assert out.isnan().all() and (lse.isnan() if sign > 0 else lse == -INF)
    finally:
        mla.set_dual_gemm(False)


@pytest.mark.parametrize("parts", [1, 4])
def test_decode_of_rows_without_keys_whatever_their_queries(parts):
    x = Batch(707, "bf16", [0, 0], [1, 400], T=2)
    q = x.q.clone()
    q[0, 0, 5] = NAN
    out, lse, _ = _decode(x, q, parts, causal=True)
    assert not out[0, 0].any() and (lse[0, :, 0] == -INF).all() and torch.isfinite(out[0, 1].float()).all()
