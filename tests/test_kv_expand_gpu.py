"""GPU parity of the expansion of cached rows (mla_kv_expand) against float64:
each value within half a bf16 step and the bound of an fp32 sum of 512
products; the rotated keys bit for bit."""
import numpy as np
import pytest
import torch

import workloads as W
from _ops import bf16, bits, check_sum, cu, f64
from oracle import prefill as O
from oracle.kv_insert import f64_to_bf16_bits

pytestmark = pytest.mark.gpu
FMTS = ["bf16", "fp8", "fp8_tensor"]


def _cache(lens, fmt, seed):
    return W.make_workload("expand", len(lens), 1, 1, lens, seed=seed, fp8=fmt == "fp8", fp8_tensor=fmt == "fp8_tensor")


def _rows(w, fmt):
    """Latent rows as the MMA's operand holds them (float64), the factor left
    to the sum, and k_pe bits, packed."""
    lat, pe = [], []
    for b in range(w.B):
        n = int(w.cache_seqlens[b])
        at = np.arange(n)
        rows = w.kv[w.block_table[b, at // 64], at % 64]
        if fmt == "bf16":
            lat.append(f64(torch.from_numpy(rows[:, :512].view(np.int16).copy()).view(torch.bfloat16)))
            pe.append(rows[:, 512:])
            continue
        codes = f64(torch.from_numpy(rows[:, :512].copy()).view(torch.float8_e4m3fn))
        if fmt == "fp8":
            sc = w.kv_scales[w.block_table[b, at // 64], at % 64].astype(np.float64)
            x = (codes.reshape(n, 4, 128) * sc[..., None]).reshape(n, 512).astype(np.float32)
            lat.append(f64(torch.from_numpy(x).to(torch.bfloat16)))
            pe.append(rows[:, 512:].copy().view(np.uint16))
        else:
            lat.append(codes)
            k = f64(torch.from_numpy(rows[:, 512:].copy()).view(torch.float8_e4m3fn)).astype(np.float32)
            pe.append(f64_to_bf16_bits((k * w.kv_scales[0]).astype(np.float64)))
    return np.concatenate(lat), (float(w.kv_scales[0]) if fmt == "fp8_tensor" else 1.0), np.concatenate(pe)


def _dev(w, fmt):
    kv = torch.from_numpy(w.kv.view(np.int16)).view(torch.bfloat16) if fmt == "bf16" else torch.from_numpy(w.kv)
    return kv.cuda(), torch.from_numpy(w.block_table).cuda(), None if fmt == "bf16" else torch.from_numpy(w.kv_scales).cuda()


def _check(kv, pe, w, fmt, w_uk, w_uv):
    lat, factor, pe_bits = _rows(w, fmt)
    want, mag = O.expand(lat, f64(w_uk), f64(w_uv))
    n = len(lat)
    check_sum(kv[:n], want * factor, mag * abs(factor), 513)
    np.testing.assert_array_equal(bits(pe[:n]), pe_bits)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,H", [([1], 1), ([64], 2), ([130, 1, 63, 65], 3), ([127, 129, 0, 300], 8), ([517], 20)])
def test_expand(fmt, lens, H):
    import mla_decode_attention_05_gb300 as mla
    w = _cache(lens, fmt, 300 + sum(lens))
    rng = np.random.default_rng(1)
    w_uk, w_uv = bf16(rng, (H, 128, 512), 0.05).cuda(), bf16(rng, (H, 128, 512), 0.05).cuda()
    cache, bt, sc = _dev(w, fmt)
    mla.device_status()
    kv, pe = mla.kv_expand(cache, bt, cu(lens), w_uk, w_uv, total=sum(lens), kv_scales=sc)
    _check(kv, pe, w, fmt, w_uk, w_uv)
    assert mla.device_status() == 0


def test_fused_weight_views_and_rows_behind_the_last():
    """W_UK and W_UV as halves of one tensor give the same bits; rows of no
    sequence stay as they were."""
    import mla_decode_attention_05_gb300 as mla
    lens, H = [70, 200], 4
    w = _cache(lens, "bf16", 7)
    rng = np.random.default_rng(2)
    w_kv = bf16(rng, (H, 256, 512), 0.05).cuda()
    cache, bt, _ = _dev(w, "bf16")
    kv, pe = mla.kv_expand(cache, bt, cu(lens), w_kv[:, :128].contiguous(), w_kv[:, 128:].contiguous(), total=270)
    _check(kv, pe, w, "bf16", w_kv[:, :128], w_kv[:, 128:])
    kv2 = torch.full((400, H, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    pe2 = torch.full((400, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    mla.kv_expand(cache, bt, cu(lens), w_kv[:, :128], w_kv[:, 128:], kv=kv2, k_pe=pe2)
    assert torch.equal(kv2[:270], kv) and torch.equal(pe2[:270], pe)
    assert bool((kv2[270:] == 5).all()) and bool((pe2[270:] == 5).all())


@pytest.mark.parametrize("fmt", FMTS)
def test_pages_and_lengths_that_cannot_be_read(fmt):
    """A page outside the pool, and a sequence longer than its pages: zeros and
    a status bit, and the rows around them unharmed."""
    import mla_decode_attention_05_gb300 as mla
    lens, H = [150, 128], 2
    w = _cache(lens, fmt, 8)
    rng = np.random.default_rng(3)
    w_uk, w_uv = bf16(rng, (H, 128, 512), 0.05).cuda(), bf16(rng, (H, 128, 512), 0.05).cuda()
    cache, bt, sc = _dev(w, fmt)
    good, gpe = mla.kv_expand(cache, bt, cu(lens), w_uk, w_uv, total=278, kv_scales=sc)
    for page in (-1, w.num_pages, 1 << 30):
        b2 = bt.clone()
        b2[0, 1] = page
        mla.device_status()
        kv, pe = mla.kv_expand(cache, b2, cu(lens), w_uk, w_uv, total=278, kv_scales=sc)
        assert mla.device_status() == mla.STATUS_BAD_PAGE
        assert not bool(kv[64:128].any()) and not bool(pe[64:128].any())
        assert torch.equal(kv[:64], good[:64]) and torch.equal(kv[128:], good[128:])
        assert torch.equal(pe[:64], gpe[:64]) and torch.equal(pe[128:], gpe[128:])
    short = bt[:, :2].contiguous()  # 150 tokens need three pages
    mla.device_status()
    kv, pe = mla.kv_expand(cache, short, cu(lens), w_uk, w_uv, total=278, kv_scales=sc)
    assert mla.device_status() == mla.STATUS_BAD_SEQLEN
    assert torch.equal(kv[:128], good[:128]) and not bool(kv[128:150].any()) and torch.equal(kv[150:], good[150:])
    # more tokens than rows: the rows there are, and the bit
    mla.device_status()
    kv, pe = mla.kv_expand(cache, bt, cu(lens), w_uk, w_uv, total=200, kv_scales=sc)
    assert mla.device_status() == mla.STATUS_BAD_SEQLEN
    assert torch.equal(kv, good[:200])


def test_many_short_sequences():
    import mla_decode_attention_05_gb300 as mla
    lens, H = [int(x) for x in np.random.default_rng(11).integers(0, 4, 1500)], 2
    lens[700] = 400
    w = _cache(lens, "fp8", 12)
    rng = np.random.default_rng(13)
    w_uk, w_uv = bf16(rng, (H, 128, 512), 0.05).cuda(), bf16(rng, (H, 128, 512), 0.05).cuda()
    cache, bt, sc = _dev(w, "fp8")
    mla.device_status()
    kv, pe = mla.kv_expand(cache, bt, cu(lens), w_uk, w_uv, total=sum(lens), kv_scales=sc)
    _check(kv, pe, w, "fp8", w_uk, w_uv)
    assert mla.device_status() == 0


def test_more_row_blocks_than_pairs():
    """Pairs of CTAs that come by several blocks of rows: the same rows as in
    calls of their own, bit for bit."""
    import mla_decode_attention_05_gb300 as mla
    lens, H = [9000, 70, 11000], 7
    w = _cache(lens, "bf16", 14)
    rng = np.random.default_rng(15)
    w_uk, w_uv = bf16(rng, (H, 128, 512), 0.05).cuda(), bf16(rng, (H, 128, 512), 0.05).cuda()
    cache, bt, _ = _dev(w, "bf16")
    mla.device_status()
    kv, pe = mla.kv_expand(cache, bt, cu(lens), w_uk, w_uv, total=sum(lens))
    at = np.cumsum([0] + lens)
    for b in range(3):
        k, e = mla.kv_expand(cache, bt[b:b + 1].contiguous(), cu(lens[b:b + 1]), w_uk, w_uv, total=lens[b])
        assert torch.equal(kv[at[b]:at[b + 1]], k) and torch.equal(pe[at[b]:at[b + 1]], e)
    lat, _, _ = _rows(w, "bf16")
    some = rng.integers(0, sum(lens), 200)
    want, mag = O.expand(lat[some], f64(w_uk), f64(w_uv))
    check_sum(kv[torch.from_numpy(some).cuda()], want, mag, 513)
    assert mla.device_status() == 0


@pytest.mark.parametrize("H,n", [(2, 300), (4, 16000), (8, 16383), (8, 12000)])
def test_few_heads_over_many_rows(H, n):
    """Few heads: a block of rows for each pair of CTAs, or an equal share.  Each
    head alone, which is shared out differently, has the same bits."""
    import mla_decode_attention_05_gb300 as mla
    w = _cache([n], "fp8", 16)
    rng = np.random.default_rng(17)
    w_uk, w_uv = bf16(rng, (H, 128, 512), 0.05).cuda(), bf16(rng, (H, 128, 512), 0.05).cuda()
    cache, bt, sc = _dev(w, "fp8")
    mla.device_status()
    kv, pe = mla.kv_expand(cache, bt, cu([n]), w_uk, w_uv, total=n, kv_scales=sc)
    for h in range(H):
        k, e = mla.kv_expand(cache, bt, cu([n]), w_uk[h:h + 1], w_uv[h:h + 1], total=n, kv_scales=sc)
        assert torch.equal(kv[:, h], k[:, 0]) and torch.equal(pe, e)
    lat, _, _ = _rows(w, "fp8")
    some = rng.integers(0, n, 100)
    want, mag = O.expand(lat[some], f64(w_uk), f64(w_uv))
    check_sum(kv[torch.from_numpy(some).cuda()], want, mag, 513)
    assert mla.device_status() == 0


def test_a_row_that_is_not_finite_stays_alone():
    import mla_decode_attention_05_gb300 as mla
    lens, H = [140], 3
    w = _cache(lens, "bf16", 9)
    rng = np.random.default_rng(4)
    w_uk, w_uv = bf16(rng, (H, 128, 512), 0.05).cuda(), bf16(rng, (H, 128, 512), 0.05).cuda()
    cache, bt, _ = _dev(w, "bf16")
    good, _ = mla.kv_expand(cache, bt, cu(lens), w_uk, w_uv, total=140)
    cache[bt[0, 1].long(), 3, 100] = float("nan")
    kv, _ = mla.kv_expand(cache, bt, cu(lens), w_uk, w_uv, total=140)
    assert bool(kv[67].isnan().all())
    keep = torch.arange(140, device="cuda") != 67
    assert torch.equal(kv[keep], good[keep])


def test_empty_calls():
    import mla_decode_attention_05_gb300 as mla
    w = _cache([5], "bf16", 10)
    cache, bt, _ = _dev(w, "bf16")
    z = torch.zeros((2, 128, 512), dtype=torch.bfloat16, device="cuda")
    kv, pe = mla.kv_expand(cache, bt, cu([0]), z, z, total=0)
    assert kv.shape == (0, 2, 256) and pe.shape == (0, 64)
    kv, pe = mla.kv_expand(cache, bt[:0], cu([]), z, z, total=0)
    out = torch.full((9, 2, 256), 2.0, dtype=torch.bfloat16, device="cuda")
    mla.kv_expand(cache, bt, cu([0]), z, z, kv=out)
    assert bool((out == 2).all())
    with pytest.raises(ValueError, match="total"):
        mla.kv_expand(cache, bt, cu([5]), z, z)


@pytest.mark.parametrize("lens,H", [([33], 2), ([290, 7], 40), ([2000, 61], 64)])
def test_rows_of_no_sequence_inside_a_warp(lens, H):
    """Rows of no sequence in front of the first and behind the last one, which
    share warps with rows that are written, in few and in many units of work:
    the written rows' bits are those of a call without them, the others stay."""
    import mla_decode_attention_05_gb300 as mla
    w = _cache(lens, "bf16", 90 + H)
    rng = np.random.default_rng(5)
    w_uk, w_uv = bf16(rng, (H, 128, 512), 0.05).cuda(), bf16(rng, (H, 128, 512), 0.05).cuda()
    cache, bt, _ = _dev(w, "bf16")
    n = sum(lens)
    kv, pe = mla.kv_expand(cache, bt, cu(lens), w_uk, w_uv, total=n)
    for front, back in ((5, 0), (45, 19), (0, 70)):
        total = front + n + back
        mla.device_status()
        kv2 = torch.full((total, H, 256), 5.0, dtype=torch.bfloat16, device="cuda")
        pe2 = torch.full((total, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        mla.kv_expand(cache, bt, cu(lens) + front, w_uk, w_uv, kv=kv2, k_pe=pe2)
        assert torch.equal(kv2[front:front + n], kv) and torch.equal(pe2[front:front + n], pe)
        rest = torch.cat([kv2[:front], kv2[front + n:]])
        assert bool((rest == 5).all()) and bool((pe2[:front] == 5).all()) and bool((pe2[front + n:] == 5).all())
        assert mla.device_status() == 0
