"""Decode of a batch behind shared prefixes (GPU) against the float64 oracle."""
import numpy as np
import pytest
import torch

from _long import Cache, check_rows, i32, table
from _ops import bf16
from oracle import long_context as O

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


def _make(seed, fmt, T, H, prefixes, groups, own, spoil=False):
    """groups: sequences of each group in turn; own: own tokens of each sequence."""
    rng = np.random.default_rng(seed)
    pages = sum(-(-n // 64) for n in prefixes + own) + 2
    c = Cache(rng, pages, fmt)
    pre = [c.take(n) for n in prefixes]
    mine = [c.take(n) for n in own]
    if spoil:
        c.spoil(list(zip(pre, prefixes)) + list(zip(mine, own)))
    q = bf16(rng, (len(own), T, H, 576), 1.3)
    return c, pre, mine, q


def _run(c, pre, mine, q, prefixes, offsets, own, causal, **kw):
    import mla_decode_attention_05_gb300 as mla
    data, scales = c.cuda()
    return mla.decode_shared(q.cuda(), data, table(pre), i32(prefixes), table(mine), i32(own), softmax_scale=SCALE,
                             group_offsets=None if offsets is None else i32(offsets), causal=causal, kv_scales=scales, **kw)


def _check(c, pre, mine, q, prefixes, offsets, own, causal, out, lse, seqs=None, rounded=False):
    """rounded: own tokens go through the decode kernel."""
    group = {}
    for g in range(len(prefixes)):
        for b in range(offsets[g] if offsets else 0, offsets[g + 1] if offsets else len(own)):
            group[b] = g
    for b in seqs if seqs is not None else range(len(own)):
        g = group.get(b)
        prefix = np.zeros((0, 576)) if g is None else c.exact_rows(pre[g], prefixes[g])
        rows = (c.rows if rounded else c.exact_rows)(mine[b], own[b])
        ref = O.attention(q[b].double().numpy(), prefix, rows, SCALE, causal)
        check_rows(out[b], lse[b].t(), ref, len(prefix) + own[b], c.fmt)


CASES = [
    # fmt, T, H, prefixes, offsets, own tokens, causal
    ("bf16", 1, 16, [200], None, [37, 12], False),
    ("bf16", 1, 128, [1000], None, [64, 0, 1, 200, 63], False),
    ("bf16", 1, 128, [64], None, [1], False),
    ("bf16", 1, 1, [65], None, [3, 130, 0], False),
    ("bf16", 2, 64, [500, 1], [0, 2, 5], [10, 70, 2, 1, 129], True),
    ("bf16", 4, 20, [129, 0, 640], [0, 1, 3, 7], [5, 4, 3, 0, 1, 200, 64], True),
    ("bf16", 3, 20, [129, 640], [1, 3, 4], [5, 4, 90, 70, 0, 11], False),   # sequences of no group at both ends
    ("bf16", 7, 128, [321], [0, 2], [20, 9, 5], True),
    ("bf16", 16, 8, [100], None, [16, 40, 7], True),
    ("bf16", 1, 40, [0], None, [0, 5], False),
    ("fp8", 1, 128, [300, 64], [0, 3, 4], [5, 64, 100, 1], False),
    ("fp8", 4, 64, [200, 31], [0, 1, 4], [4, 2, 150, 0], True),
    ("fp8_tensor", 1, 16, [130], None, [9, 0, 70], False),
    ("fp8_tensor", 2, 48, [65, 400], [0, 2, 3], [1, 128, 66], True),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_the_oracle(case):
    import mla_decode_attention_05_gb300 as mla
    fmt, T, H, prefixes, offsets, own, causal = CASES[case]
    mla.device_status()
    c, pre, mine, q = _make(300 + case, fmt, T, H, prefixes, offsets, own)
    out, lse = _run(c, pre, mine, q, prefixes, offsets, own, causal)
    _check(c, pre, mine, q, prefixes, offsets, own, causal, out, lse)
    assert mla.device_status() == 0


def _log2_sizes(rng, n, spread):
    return torch.from_numpy(2.0 ** rng.integers(-spread, spread + 1, n).astype(np.float32))


@pytest.mark.parametrize("fmt", ["fp8", "fp8_tensor"])
@pytest.mark.parametrize("size", [2.0 ** -90, 2.0 ** 60])
def test_fp8_rows_and_queries_of_any_size(fmt, size):
    """Very small and very large keys, and queries that undo it; rows of other sizes
    side by side; a page whose latent or whose rotated part is all zeros."""
    T, H, prefixes, own = 1, 40, [150], [70, 64, 3]
    c, pre, mine, q = _make(336, fmt, T, H, prefixes, None, own)
    rng = np.random.default_rng(337)
    c.scales *= size
    if fmt == "fp8":
        tiles = _log2_sizes(rng, (c.pages, 64, 4), 6)
        c.scales *= tiles
        pe = c.data[..., 512:].contiguous().view(torch.bfloat16)
        pe *= size
        c.data[pre[0][0], :, :512] = 0
        pe[pre[0][1]] = 0
        c.data[..., 512:] = pe.view(torch.uint8)
        codes = c.data[..., :512].contiguous().view(torch.float8_e4m3fn).double().reshape(c.pages, 64, 4, 128)
        c.exact = torch.cat([(codes * c.scales[..., None].double()).reshape(c.pages, 64, 512), pe.double()], -1)
    else:
        c.exact = c.data.view(torch.float8_e4m3fn).double() * c.scales.double()
    q = (q.float() * _log2_sizes(rng, (3, T, H, 1), 5) / 64 / size).to(torch.bfloat16)
    out, lse = _run(c, pre, mine, q, prefixes, None, own, False)
    if size < 1:  # the test's bounds hold relative to the output's size: bf16 has its smallest numbers at 2^-126
        assert (out != 0).any()
    _check(c, pre, mine, q, prefixes, None, own, False, out, lse)


@pytest.mark.parametrize("fmt", ["fp8", "fp8_tensor"])
def test_fp8_scales_of_zero(fmt):
    """Cached rows that are all zeros, as an empty model's: every key counts alike."""
    c, pre, mine, q = _make(338, fmt, 1, 16, [70], None, [5, 0])
    c.scales[...] = 0
    if fmt == "fp8":
        c.data[..., 512:] = 0
    out, lse = _run(c, pre, mine, q, [70], None, [5, 0], False)
    assert (out == 0).all()
    assert torch.allclose(lse[:, :, 0].cpu(), torch.log(torch.tensor([[75.0], [70.0]])), atol=1e-6)


@pytest.mark.parametrize("fmt", ["fp8", "fp8_tensor"])
def test_fp8_own_tokens_behind_a_wide_page_table(fmt):
    """A page table too wide for its pages to be widened ahead."""
    import mla_decode_attention_05_gb300 as mla
    prefixes, offsets, own = [130, 64], [0, 1, 3], [9, 0, 70]
    c, pre, mine, q = _make(335, fmt, 4, 48, prefixes, offsets, own)
    data, scales = c.cuda()
    out, lse = mla.decode_shared(q.cuda(), data, table(pre), i32(prefixes), table(mine, 1400), i32(own), softmax_scale=SCALE,
                                 group_offsets=i32(offsets), causal=True, kv_scales=scales)
    _check(c, pre, mine, q, prefixes, offsets, own, True, out, lse, rounded=True)


def test_many_sequences_and_a_long_prefix():
    """Prefix tiles split over many workers, and own caches of all lengths."""
    rng = np.random.default_rng(330)
    own = [int(x) for x in rng.integers(0, 500, 70)]
    prefixes, offsets = [5000, 333, 2000], [0, 33, 34, 70]
    c, pre, mine, q = _make(331, "bf16", 1, 16, prefixes, offsets, own)
    out, lse = _run(c, pre, mine, q, prefixes, offsets, own, False)
    _check(c, pre, mine, q, prefixes, offsets, own, False, out, lse, seqs=[0, 1, 20, 32, 33, 34, 50, 69])


def test_equal_calls_give_equal_bits_and_joined_is_whole():
    """The same tokens as one sequence's cache of its own (decode) agree."""
    import mla_decode_attention_05_gb300 as mla
    own, prefixes = [70, 130, 5], [640]
    c, pre, mine, q = _make(332, "bf16", 1, 32, prefixes, None, own)
    a = _run(c, pre, mine, q, prefixes, None, own, False)
    b = _run(c, pre, mine, q, prefixes, None, own, False)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    data, _ = c.cuda()
    out, lse = mla.decode(q.cuda(), data, table([pre[0] + m for m in mine]), i32([640 + n for n in own]), softmax_scale=SCALE)
    assert (out.float() - a[0].float()).abs().max() <= 2.0 ** -6 * out.float().abs().max()
    assert (lse - a[1]).abs().max() <= 1e-3


def test_bad_pages_lengths_and_offsets_are_told():
    import mla_decode_attention_05_gb300 as mla
    own, prefixes = [70, 10], [200]
    c, pre, mine, q = _make(333, "bf16", 1, 8, prefixes, None, own)
    data, _ = c.cuda()
    mla.device_status()
    call = lambda pt, pl, off, bt, sk: mla.decode_shared(q.cuda(), data, pt, i32(pl), bt, i32(sk), softmax_scale=SCALE,
                                                          group_offsets=None if off is None else i32(off))
    pt, bt = table(pre), table(mine)
    good = call(pt, prefixes, None, bt, own)
    assert mla.device_status() == 0
    bad = pt.clone()
    bad[0, 1] = c.pages
    got = call(bad, prefixes, None, bt, own)
    assert mla.device_status() == mla.STATUS_BAD_PAGE
    for b in range(2):  # tokens of that page are left out
        kept = np.delete(c.rows(pre[0], 200), np.arange(64, 128), 0)
        check_rows(got[0][b], got[1][b].t(), O.attention(q[b].double().numpy(), kept, c.rows(mine[b], own[b]), SCALE, False), 300)
    call(pt, [-3], None, bt, own)
    assert mla.device_status() == mla.STATUS_BAD_SEQLEN
    got = call(pt, [100000], None, bt, own)   # clamped to its pages
    assert mla.device_status() == mla.STATUS_BAD_SEQLEN and torch.isfinite(got[1]).all()
    for off in ([0, 5], [2, 1], [-1, 2]):
        call(pt, prefixes, off, bt, own)
        assert mla.device_status() == mla.STATUS_BAD_SEQLEN
    call(pt, prefixes, None, bt, [-1, 10])
    assert mla.device_status() == mla.STATUS_BAD_SEQLEN
    again = call(pt, prefixes, None, bt, own)
    assert mla.device_status() == 0 and torch.equal(again[0], good[0])


def test_given_buffers_another_stream_and_a_graph():
    import mla_decode_attention_05_gb300 as mla
    own, prefixes = [70, 10, 200], [300]
    c, pre, mine, q = _make(334, "bf16", 2, 16, prefixes, None, own)
    data, _ = c.cuda()
    q, pt, pl, bt, sk = q.cuda(), table(pre), i32(prefixes), table(mine), i32(own)
    want = mla.decode_shared(q, data, pt, pl, bt, sk, softmax_scale=SCALE, causal=True)
    ws = torch.full((mla.decode_shared_workspace_bytes(3, 2, 16, 1, mla.KV_BF16, pt.shape[1], bt.shape[1]),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((3, 2, 16, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, 16, 2), float("nan"), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call = lambda: mla.decode_shared(q, data, pt, pl, bt, sk, softmax_scale=SCALE, causal=True, workspace=ws, out=out, lse=lse)
    with torch.cuda.stream(s):
        got = call()
    s.synchronize()
    assert got[0] is out and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    sk.copy_(i32([10, 64, 1]))
    pl.fill_(77)
    eager = mla.decode_shared(q, data, pt, pl, bt, sk, softmax_scale=SCALE, causal=True)
    ws.fill_(0xFF)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
