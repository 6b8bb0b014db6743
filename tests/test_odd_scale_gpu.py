"""FP8 caches whose one scale takes all of fp32's bits: exact codes against the float64
oracle of exact rows.  Calls that overlap, compared in full."""
import numpy as np
import pytest
import torch

from _long import Cache, check_rows, i32, table
from _odd_scale import odd_scale
from _ops import STEP_F32, bf16, f64
from oracle import long_context as O

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


def _make(seed, T, H, lens, fmt="fp8_tensor"):
    rng = np.random.default_rng(seed)
    c = Cache(rng, sum(-(-n // 64) for n in lens) + 2, fmt)
    if fmt == "fp8_tensor":
        odd_scale(c)
    return c, [c.take(n) for n in lens], bf16(rng, (len(lens), T, H, 576), 1.3)


@pytest.mark.parametrize("T,H,prefixes,offsets,own,causal", [
    (1, 16, [130], [0, 3], [9, 0, 70], False), (2, 48, [65, 400], [0, 2, 3], [1, 128, 66], True),
    (1, 128, [1000], [0, 2], [64, 3], False), (1, 1, [0], [0, 1], [1], False), (4, 64, [3000], [0, 3], [5, 700, 64], True),
])
def test_decode_shared(T, H, prefixes, offsets, own, causal):
    import mla_decode_attention_05_gb300 as mla
    mla.device_status()
    c, pages, q = _make(820, T, H, prefixes + own)
    q = q[:len(own)].contiguous()
    pre, mine = pages[:len(prefixes)], pages[len(prefixes):]
    data, scales = c.cuda()
    out, lse = mla.decode_shared(q.cuda(), data, table(pre), i32(prefixes), table(mine), i32(own), softmax_scale=SCALE,
                                 group_offsets=i32(offsets), causal=causal, kv_scales=scales)
    for b in range(len(own)):
        g = next(g for g in range(len(prefixes)) if offsets[g] <= b < offsets[g + 1])
        ref = O.attention(q[b].double().numpy(), c.exact_rows(pre[g], prefixes[g]), c.exact_rows(mine[b], own[b]), SCALE, causal)
        check_rows(out[b], lse[b].t(), ref, prefixes[g] + own[b], "fp8_tensor")
    assert mla.device_status() == 0


@pytest.mark.parametrize("T,H,lens,causal,decay", [
    (1, 40, [200, 0, 65], False, 0.9), (5, 64, [190], True, 1.0), (1, 8, [20000, 4097], False, 0.5), (64, 10, [2500], True, 0.0),
    (1, 1, [1], False, 0.0), (2, 128, [9000], True, 1.0),
])
def test_attention_mass(T, H, lens, causal, decay):
    import mla_decode_attention_05_gb300 as mla
    mla.device_status()
    c, pages, q = _make(821, T, H, lens)
    lse = torch.empty(len(lens), H, T)
    for b, n in enumerate(lens):
        ref = O.attention(q[b].double().numpy(), np.zeros((0, 576)), c.exact_rows(pages[b], n), SCALE, causal)
        lse[b] = torch.from_numpy(ref["lse"]).t()
    cap = -(-max(lens) // 64) * 64
    before = torch.rand(len(lens), cap) * 3
    data, scales = c.cuda()
    got = mla.attention_mass(q.cuda(), data, table(pages), i32(lens), lse.cuda(), before.cuda(), softmax_scale=SCALE, causal=causal,
                             decay=decay, kv_scales=scales)
    for b, n in enumerate(lens):
        want, bound = O.mass(q[b].double().numpy(), c.exact_rows(pages[b], n), lse[b].t().double().numpy(), SCALE, causal)
        # (the weights' own bounds, which have no part for rounded rows; a step for each addition of the T * H; two roundings of
        # the update; and two more of each score, the scale's product with the softmax scale and that with the sum)
        old = decay * f64(before[b, :n])
        s = SCALE * np.abs(c.exact_rows(pages[b], n)) @ np.abs(q[b].double().numpy()).reshape(-1, 576).T if n else np.zeros((0, 1))
        tol = bound + ((T * H + 2) * STEP_F32 + 2 * STEP_F32 * s.max(1)) * (want + bound) + 2 * STEP_F32 * (old + want) + 1e-37
        err = np.abs(f64(got[b, :n]) - (want + old))
        assert np.all(err <= tol), (b, float((err - tol).max()))
        assert torch.equal(got[b, n:].cpu(), before[b, n:])
    assert mla.device_status() == 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_tensor"])
@pytest.mark.parametrize("T,H", [(1, 64), (4, 64)])
def test_calls_that_overlap_whole(fmt, T, H):
    """Streams with workspaces of their own; with 256 query rows and more, partial sums of the weights are in them."""
    import mla_decode_attention_05_gb300 as mla
    mla.device_status()
    lens = [3000, 300, 700, 90, 5]
    c, pages, q = _make(822, T, H, lens, fmt)
    pre, mine, own = pages[:1], pages[1:], lens[1:]
    q = q[1:].contiguous().cuda()
    data, scales = c.cuda()
    pt, pl, bt, sk = table(pre), i32(lens[:1]), table(mine), i32(own)
    shared = lambda **k: mla.decode_shared(q, data, pt, pl, bt, sk, softmax_scale=SCALE, causal=T > 1, kv_scales=scales, **k)
    want = shared()
    weigh = lambda **k: mla.attention_mass(q, data, bt, sk, want[1], torch.full((4, 704), 0.5, device="cuda"), softmax_scale=SCALE,
                                           causal=T > 1, kv_scales=scales, **k)
    sums = weigh()
    size = mla.attention_mass_workspace_bytes(4, T, H, 704)
    assert (size > 0) == (T * H > 128)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(4)], []
    room = [torch.full((max(256, size),), 0xFF, dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for k in range(24):
        with torch.cuda.stream(streams[k % 4]):
            got.append(shared() if k % 3 == 0 else weigh(workspace=room[k % 4]))
    torch.cuda.synchronize()
    for k, r in enumerate(got):
        if k % 3 == 0:
            assert torch.equal(r[0], want[0]) and torch.equal(r[1], want[1])
        else:
            assert torch.equal(r, sums)
    for b, n in enumerate(own):   # nothing behind the last token
        assert (sums[b, n:] == 0.5).all()
    assert mla.device_status() == 0
