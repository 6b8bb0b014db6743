"""GPU parity of the prefill attention (mla_prefill) against float64, row by
row, within the bounds derived in _ops.check_attention."""
import numpy as np
import pytest
import torch

from _ops import bf16, check_attention, cu, f64
from oracle import prefill as O

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


def _inputs(nq, nk, H, seed, q_std=1.5):
    rng = np.random.default_rng(seed)
    kv = bf16(rng, (sum(nk), H, 256)).cuda()
    return bf16(rng, (sum(nq), H, 192), q_std).cuda(), kv[..., :128], bf16(rng, (sum(nk), 64)).cuda(), kv[..., 128:]


def _check(out, lse, ins, nq, nk, causal, scale=SCALE):
    q, kn, kp, v = (f64(t) for t in ins)
    at, kt = np.cumsum([0] + nq), np.cumsum([0] + nk)
    for b in range(len(nq)):
        s, k = slice(at[b], at[b + 1]), slice(kt[b], kt[b + 1])
        ref = O.attention(q[s], kn[k], kp[k], v[k], scale, causal)
        check_attention(out[s], lse[:, s].T, ref, nk[b])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,H", [
    ([1], [1], 1), ([1], [300], 2), ([5], [3], 2), ([128], [128], 1), ([129], [129], 2), ([256], [256], 1),
    ([257], [257], 1), ([300], [700], 1), ([64, 0, 1, 200], [64, 10, 1, 333], 3), ([33, 260], [0, 129], 2),
    ([130], [128], 1), ([17, 3, 400], [900, 2, 380], 2), ([1] * 40, list(range(1, 41)), 2)])
def test_prefill(nq, nk, H, causal):
    import mla_decode_attention_05_gb300 as mla
    ins = _inputs(nq, nk, H, 100 + sum(nq) + sum(nk))
    mla.device_status()
    out, lse = mla.prefill(*ins, cu(nq), cu(nk), softmax_scale=SCALE, causal=causal)
    _check(out, lse, ins, nq, nk, causal)
    assert mla.device_status() == 0


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,H", [([200], [2200], 2), ([1], [5000], 1), ([3, 130], [40, 4100], 2), ([260], [4099], 1),
                                     ([300, 5], [100, 6000], 3), ([9, 0, 2], [1, 2, 9000], 1),
                                     ([2] * 8, [3000] * 8, 20)])
def test_few_queries_over_long_keys(nq, nk, H, causal):
    """These are split over the keys; parts without keys of a row among them."""
    import mla_decode_attention_05_gb300 as mla
    assert mla.prefill_workspace_bytes(len(nq), H, sum(nq), sum(nk)) > 0
    ins = _inputs(nq, nk, H, 300 + sum(nq) + sum(nk))
    mla.device_status()
    out, lse = mla.prefill(*ins, cu(nq), cu(nk), softmax_scale=SCALE, causal=causal)
    _check(out, lse, ins, nq, nk, causal)
    assert mla.device_status() == 0
    # values that are not finite, in and behind what rows see; rows of no sequence
    ins[3][-2, 0, 5] = float("inf")
    ins[3][3, 0, 7] = float("nan")
    o2 = torch.full((sum(nq) + 3, H, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    l2 = torch.full((H, sum(nq) + 3), 9.0, device="cuda")
    q2 = torch.cat([ins[0], ins[0].new_ones((3, H, 192))])
    mla.prefill(q2, *ins[1:], cu(nq), cu(nk), softmax_scale=SCALE, causal=causal, out=o2, lse=l2)
    assert bool((o2[sum(nq):] == 9).all()) and bool((l2[:, sum(nq):] == 9).all())
    assert torch.equal(l2[:, :sum(nq)], lse)
    hit = torch.zeros_like(out, dtype=torch.bool)
    at, kt = np.cumsum([0] + nq), np.cumsum([0] + nk)
    for key, d in ((sum(nk) - 2, 5), (3, 7)):
        b = int(np.searchsorted(kt, key, side="right")) - 1
        first = max(0, key - int(kt[b]) - nk[b] + nq[b]) if causal else 0
        hit[at[b] + first:at[b + 1], 0, d] = True
    assert not bool(o2[:sum(nq)][hit].isfinite().any()) and torch.equal(o2[:sum(nq)][~hit], out[~hit])


def test_many_units_of_work():
    """More tiles than SMs, so that a block takes over the work of others; a
    given workspace."""
    import mla_decode_attention_05_gb300 as mla
    nq, nk, H = [513, 40, 0, 300, 257, 1, 700] * 3, [513, 100, 5, 290, 600, 1, 900] * 3, 12
    ins = _inputs(nq, nk, H, 18, 1.0)
    mla.device_status()
    out, lse = mla.prefill(*ins, cu(nq), cu(nk), softmax_scale=SCALE, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert mla.device_status() == 0
    at, kt = np.cumsum([0] + nq), np.cumsum([0] + nk)
    for b, heads in ((0, (0, 11)), (8, (5,)), (10, (7,)), (20, (3, 8)), (18, (9,)), (19, (0,))):
        s, k = slice(at[b], at[b + 1]), slice(kt[b], kt[b + 1])
        h = list(heads)
        part = [ins[0][s, h], ins[1][k, h], ins[2][k], ins[3][k, h]]
        _check(out[s, h], lse[h, s], part, [nq[b]], [nk[b]], True)
    again = mla.prefill(*ins, cu(nq), cu(nk), softmax_scale=SCALE)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("q_std,scale", [(0.01, SCALE), (30.0, SCALE), (1.0, 1.5)])
def test_flat_and_sharp_scores(q_std, scale):
    """Scores that grow along the keys move the reference many times."""
    import mla_decode_attention_05_gb300 as mla
    nq, nk, H = [200], [900], 2
    q, kn, kp, v = _inputs(nq, nk, H, 11, q_std)
    kn *= torch.linspace(0.01, 1.5, 900, device="cuda").to(torch.bfloat16)[:, None, None]
    out, lse = mla.prefill(q, kn, kp, v, cu(nq), cu(nk), softmax_scale=scale)
    _check(out, lse, (q, kn, kp, v), nq, nk, True, scale)


def test_layouts():
    """Contiguous keys and values, heads before tokens, queries in wider rows,
    a given output: the same bits as the views of one tensor."""
    import mla_decode_attention_05_gb300 as mla
    nq, nk, H = [150, 40], [150, 200], 3
    q, kn, kp, v = _inputs(nq, nk, H, 12)
    a, b = cu(nq), cu(nk)
    out, lse = mla.prefill(q, kn, kp, v, a, b, softmax_scale=SCALE)
    _check(out, lse, (q, kn, kp, v), nq, nk, True)
    swap = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.zeros((190, H, 576), dtype=torch.bfloat16, device="cuda")
    wide[..., 384:] = q
    pe = torch.zeros((350, 640), dtype=torch.bfloat16, device="cuda")
    pe[:, 576:] = kp
    for args in ((q, kn.contiguous(), kp, v.contiguous()), (swap(q), swap(kn), kp, swap(v)),
                 (wide[..., 384:], kn, pe[:, 576:], v)):
        o, l = mla.prefill(*args, a, b, softmax_scale=SCALE)
        assert torch.equal(o, out) and torch.equal(l, lse)
    o, l = torch.empty_like(out), torch.empty_like(lse)
    r = mla.prefill(q, kn, kp, v, a, b, softmax_scale=SCALE, out=o, lse=l)
    assert r[0] is o and r[1] is l and torch.equal(o, out) and torch.equal(l, lse)


def test_rows_of_no_sequence_stay():
    import mla_decode_attention_05_gb300 as mla
    nq, nk, H = [70, 130], [100, 140], 2
    ins = _inputs([70, 130, 50], [100, 140, 60], H, 13)
    out = torch.full((250, H, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, 250), 9.0, device="cuda")
    mla.prefill(*ins, cu(nq), cu(nk), softmax_scale=SCALE, out=out, lse=lse)
    _check(out, lse, ins, nq, nk, True)
    assert bool((out[200:] == 9).all()) and bool((lse[:, 200:] == 9).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("causal", [True, False])
def test_what_a_row_does_not_see_does_not_reach_it(bad, causal):
    """Keys and values of later tokens, of other sequences and of rows behind
    the last hold what is not finite."""
    import mla_decode_attention_05_gb300 as mla
    nq, nk, H = [300, 90], [310, 95], 2
    ins = _inputs(nq, nk + [70], H, 14)
    q, kn, kp, v = ins
    base, bl = mla.prefill(*ins, cu(nq), cu(nk), softmax_scale=SCALE, causal=causal)
    base, bl = base.clone(), bl.clone()
    # the key that only queries from 200 on see (causal), the first of the second sequence, the rows behind the last
    for at in (210, 310, 405, 440):
        kn[at], kp[at], v[at] = bad, bad, bad
    out, lse = mla.prefill(*ins, cu(nq), cu(nk), softmax_scale=SCALE, causal=causal)
    if causal:
        assert torch.equal(out[:200], base[:200]) and torch.equal(lse[:, :200], bl[:, :200])
        assert not bool(out[200:].isfinite().any())
    else:
        assert not bool(out.isfinite().any())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_value_that_is_not_finite_reaches_the_rows_that_see_it(bad):
    """Values alone: the other dimensions of a row that sees the key, and all of
    a row that does not, keep their results."""
    import mla_decode_attention_05_gb300 as mla
    nq, nk, H = [290], [300], 2
    ins = _inputs(nq, nk, H, 15)
    v = ins[3]
    clean = v.clone()
    spots = [(5, 0, 3), (150, 1, 64), (260, 0, 127), (299, 1, 0)]
    for j, h, d in spots:
        v[j, h, d] = bad
    out, lse = mla.prefill(*ins, cu(nq), cu(nk), softmax_scale=SCALE)
    hit = torch.zeros_like(out, dtype=torch.bool)
    for j, h, d in spots:
        hit[max(0, j - 10):, h, d] = True
    assert not bool(out[hit].isfinite().any()) and bool(out[~hit].isfinite().all())
    for j, h, d in spots:
        clean[j, h, d] = 0
    want, wl = mla.prefill(*ins[:3], clean, cu(nq), cu(nk), softmax_scale=SCALE)
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse, wl)


@pytest.mark.parametrize("nq,nk", [([70], [200]), ([3], [4000])])
def test_scores_of_minus_infinity(nq, nk):
    """Keys whose scores are -inf: of weight 0 beside others, as if they
    were not there, and 0 / 0 where a row sees no
    other key.  In one part and in several."""
    import mla_decode_attention_05_gb300 as mla
    H = 2
    q, kn, kp, v = _inputs(nq, nk, H, 31)
    q[:, :, 128] = 1.0
    gone = kp.clone()
    gone[:, 0] = -float("inf")
    out, lse = mla.prefill(q, kn, gone, v, cu(nq), cu(nk), softmax_scale=SCALE)
    assert bool(out.isnan().all()) and bool(lse.isneginf().all())
    some = gone.clone()
    keep = [5, 130, nk[0] - 100]
    some[keep] = kp[keep]
    out, lse = mla.prefill(q, kn, some, v, cu(nq), cu(nk), softmax_scale=SCALE, causal=False)
    few = (q, kn[keep], kp[keep], v[keep])
    _check(out, lse, few, nq, [3], False)


def test_many_short_sequences():
    """Thousands of sequences, empty ones among them, some of several tiles."""
    import mla_decode_attention_05_gb300 as mla
    rng = np.random.default_rng(23)
    nq = [int(x) for x in rng.integers(0, 5, 3000)]
    for b in (0, 700, 1500, 2999):
        nq[b] = 300
    nk = [q + int(c) for q, c in zip(nq, rng.integers(0, 4, 3000))]
    ins = _inputs(nq, nk, 2, 24)
    mla.device_status()
    out, lse = mla.prefill(*ins, cu(nq), cu(nk), softmax_scale=SCALE)
    assert mla.device_status() == 0
    at, kt = np.cumsum([0] + nq), np.cumsum([0] + nk)
    for b in [0, 1, 2, 31, 32, 33, 699, 700, 701, 1024, 1499, 1500, 2000, 2998, 2999]:
        s, k = slice(at[b], at[b + 1]), slice(kt[b], kt[b + 1])
        _check(out[s], lse[:, s], [ins[0][s], ins[1][k], ins[2][k], ins[3][k]], [nq[b]], [nk[b]], True)
    # a row's result does not depend on the sequences around its own
    for a, z in ((0, 40), (1480, 1530), (2950, 3000)):
        s, k = slice(at[a], at[z]), slice(kt[a], kt[z])
        o, l = mla.prefill(ins[0][s], ins[1][k], ins[2][k], ins[3][k], cu(nq[a:z]), cu(nk[a:z]), softmax_scale=SCALE)
        assert torch.equal(o, out[s]) and torch.equal(l, lse[:, s])


def test_many_units_of_work_are_done_again():
    """Every unit of work holds a value that its earlier rows do not see and
    that is not finite: more than wait to be done again at a time."""
    import mla_decode_attention_05_gb300 as mla
    B, H = 60, 128
    nq = [3] * B
    ins = _inputs(nq, nq, H, 19)
    base, bl = mla.prefill(*ins, cu(nq), cu(nq), softmax_scale=SCALE)
    ins[3][2::3] = float("nan")
    out, lse = mla.prefill(*ins, cu(nq), cu(nq), softmax_scale=SCALE)
    last = torch.arange(3 * B, device="cuda") % 3 == 2
    assert torch.equal(out[~last], base[~last]) and torch.equal(lse, bl)
    assert bool(out[last].isnan().all()) and mla.device_status() == 0


def test_lengths_out_of_order_are_clamped():
    """cu_seqlens that leave the rows there are, or go back: a status bit, no
    access outside, and the sequences before them as they are."""
    import mla_decode_attention_05_gb300 as mla
    nq, nk, H = [40, 60], [50, 70], 2
    ins = _inputs(nq, nk, H, 16)
    out, lse = mla.prefill(*ins, cu(nq), cu(nk), softmax_scale=SCALE)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    for a, b in ((i32(0, 40, 500), cu(nk)), (i32(0, 40, 20), cu(nk)), (cu(nq), i32(0, 50, 1 << 30)),
                 (cu(nq), i32(0, 50, -7)), (i32(0, 40, -1), cu(nk))):
        mla.device_status()
        o, l = mla.prefill(*ins, a, b, softmax_scale=SCALE)
        assert mla.device_status() == mla.STATUS_BAD_SEQLEN
        assert torch.equal(o[:40], out[:40]) and torch.equal(l[:, :40], lse[:, :40])


def test_empty_calls():
    import mla_decode_attention_05_gb300 as mla
    ins = _inputs([3], [4], 2, 17)
    q, kn, kp, v = ins
    o, l = mla.prefill(q[:0], kn, kp, v, cu([0]), cu([4]), softmax_scale=SCALE)
    assert o.shape == (0, 2, 128) and l.shape == (2, 0)
    o, l = mla.prefill(q, kn[:0], kp[:0], v[:0], cu([3]), cu([0]), softmax_scale=SCALE)
    assert not bool(o.any()) and bool(l.isneginf().all())
    o, l = mla.prefill(q[:0], kn[:0], kp[:0], v[:0], cu([]), cu([]), softmax_scale=SCALE)
    assert o.shape == (0, 2, 128)


@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_end_inside_a_warp(causal):
    """Tiles whose last row is at every place of a warp, one after the other in
    the same CTAs: lanes without a row take no part in the output, but in every
    load from tensor memory."""
    import mla_decode_attention_05_gb300 as mla
    nq = list(range(1, 34)) + [95, 97, 127, 129, 161, 191, 193, 225, 255, 257, 289]
    nk = [n + 7 * (i % 3) for i, n in enumerate(nq)]
    H = 6
    ins = _inputs(nq, nk, H, 51)
    mla.device_status()
    out, lse = mla.prefill(*ins, cu(nq), cu(nk), softmax_scale=SCALE, causal=causal)
    _check(out, lse, ins, nq, nk, causal)
    assert mla.device_status() == 0
