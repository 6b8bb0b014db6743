"""GPU parity of the KV insert with rotation (mla_kv_insert_rope): every cache
byte, scale and rotated query bit for bit against the oracle."""
import numpy as np
import pytest
import torch

import workloads as W
from _ops import bf16, bits
from oracle import kv_insert as K
from oracle import prefill as O

pytestmark = pytest.mark.gpu
MAX_POS = 777
FMTS = [K.FMT_BF16, K.FMT_FP8_TILE, K.FMT_FP8_TENSOR]


def _setup(N, pages, H, seed, width=192, page_size=64):
    inp = W.make_insert_inputs(N, pages, page_size, seed=seed)
    rng = np.random.default_rng(seed)
    pos = rng.integers(0, MAX_POS, N).astype(np.int64)
    pos[0], pos[-1] = 0, MAX_POS - 1
    return inp, pos, bf16(rng, (N, H, width))


def _want(inp, fmt, pos, q, interleaved, slots=None):
    table = O.angle_table(MAX_POS)
    ok = (pos >= 0) & (pos < MAX_POS)
    cs = table[np.where(ok, pos, 0)]
    pe = O.rotate(inp.qkv[:, W.K_PE_COL:], cs, interleaved)
    qr = bits(q[..., -64:]).copy()
    qr[ok] = O.rotate(qr, cs[:, None], interleaved)[ok]
    sl = np.where(ok, inp.slots if slots is None else slots, -1)
    cache = np.full((inp.num_pages, inp.page_size, K.ROW_BYTES[fmt]), 0xAB, np.uint8)
    scales = np.full((inp.num_pages, inp.page_size, 4), -1.0, np.float32)
    K.kv_insert(fmt, inp.qkv[:, W.KV_C_COL:], pe, inp.w_kva, inp.eps, sl, cache, scales, inp.k_scale_inv)
    return cache, scales, qr


def _args(inp, fmt, pos, slots=None):
    qkv = torch.from_numpy(inp.qkv.view(np.int16)).view(torch.bfloat16).cuda()
    raw = torch.full((inp.num_pages, inp.page_size, K.ROW_BYTES[fmt]), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((inp.num_pages, inp.page_size, 4), -1.0, dtype=torch.float32, device="cuda")
    cache = raw.view(torch.bfloat16) if fmt == K.FMT_BF16 else raw
    a = (qkv[:, W.KV_C_COL:W.KV_C_COL + 512], qkv[:, W.K_PE_COL:],
         torch.from_numpy(inp.w_kva.view(np.int16)).view(torch.bfloat16).cuda(),
         torch.from_numpy(inp.slots if slots is None else slots).cuda(), cache)
    kw = dict(eps=inp.eps, positions=torch.from_numpy(pos).cuda(), cos_sin=torch.from_numpy(O.angle_table(MAX_POS)).cuda(),
              kv_scales=scales, k_scale_inv=torch.tensor([inp.k_scale_inv], device="cuda"),
              fp8_per_tensor=fmt == K.FMT_FP8_TENSOR)
    return a, kw, raw, scales


def _same(raw, scales, q, want, fmt):
    cache, sc, qr = want
    np.testing.assert_array_equal(raw.cpu().numpy(), cache)
    if fmt == K.FMT_FP8_TILE:
        np.testing.assert_array_equal(scales.cpu().numpy().view(np.uint32), sc.view(np.uint32))
    if q is not None:
        np.testing.assert_array_equal(bits(q), qr)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("N,pages,H,width,page_size", [(1, 1, 1, 192, 64), (7, 2, 5, 576, 64), (203, 8, 8, 192, 64),
                                                       (300, 40, 3, 576, 16), (33, 1, 128, 576, 64)])
def test_bit_exact(fmt, interleaved, N, pages, H, width, page_size):
    import mla_decode_attention_05_gb300 as mla
    inp, pos, q = _setup(N, pages, H, 200 + N, width, page_size)
    want = _want(inp, fmt, pos, q, interleaved)
    a, kw, raw, scales = _args(inp, fmt, pos)
    qd = q.cuda()
    out = torch.full((N, H, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    mla.device_status()
    c, qo = mla.kv_insert_rope(*a, **kw, interleaved=interleaved, q_pe=qd[..., -64:], q_out=out)
    assert c is a[4] and qo is out
    _same(raw, scales, out, want, fmt)
    assert torch.equal(qd.cpu(), q)
    # in place, and without queries
    raw.fill_(0xAB), scales.fill_(-1.0)
    mla.kv_insert_rope(*a, **kw, interleaved=interleaved, q_pe=qd[..., -64:])
    _same(raw, scales, qd[..., -64:], want, fmt)
    assert torch.equal(qd[..., :-64].cpu(), q[..., :-64])
    raw.fill_(0xAB), scales.fill_(-1.0)
    mla.kv_insert_rope(*a, **kw, interleaved=interleaved)
    _same(raw, scales, None, want, fmt)
    assert mla.device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_position_zero_is_the_plain_insert(fmt):
    import mla_decode_attention_05_gb300 as mla
    inp, pos, _ = _setup(65, 3, 1, 5)
    a, kw, raw, scales = _args(inp, fmt, np.zeros_like(pos))
    mla.kv_insert_rope(*a, **kw)
    b, kb, raw2, scales2 = _args(inp, fmt, pos)
    del kb["positions"], kb["cos_sin"]
    mla.kv_insert(*b, **kb)
    assert torch.equal(raw, raw2) and torch.equal(scales, scales2)


def test_padded_batch_and_bad_positions():
    """-1 skips a token silently; a position outside the table skips it and
    sets the status bit; a token without a slot still gets its queries."""
    import mla_decode_attention_05_gb300 as mla
    inp, pos, q = _setup(40, 2, 4, 6)
    pos[5], pos[6] = -1, -1
    slots = inp.slots.copy()
    slots[6], slots[7] = -1, -1
    for bad, status in ((None, 0), ((11, MAX_POS), mla.STATUS_BAD_POSITION), ((12, -2), mla.STATUS_BAD_POSITION),
                        ((13, 1 << 40), mla.STATUS_BAD_POSITION)):
        if bad:
            pos[bad[0]] = bad[1]
        want = _want(inp, K.FMT_FP8_TILE, pos, q, True, slots)
        a, kw, raw, scales = _args(inp, K.FMT_FP8_TILE, pos, slots)
        out = q[..., -64:].contiguous().cuda()  # skipped rows keep these
        mla.device_status()
        mla.kv_insert_rope(*a, **kw, q_pe=q.cuda()[..., -64:], q_out=out)
        assert mla.device_status() == status
        _same(raw, scales, out, want, K.FMT_FP8_TILE)


def test_query_layouts():
    """Heads before tokens, and an output inside wider rows."""
    import mla_decode_attention_05_gb300 as mla
    inp, pos, q = _setup(50, 2, 6, 8)
    want = _want(inp, K.FMT_BF16, pos, q, False)
    a, kw, raw, scales = _args(inp, K.FMT_BF16, pos)
    qt = q.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((6, 50, 200), 3.0, dtype=torch.bfloat16, device="cuda")
    out = wide[..., 8:72].transpose(0, 1)
    mla.kv_insert_rope(*a, **kw, interleaved=False, q_pe=qt[..., 128:], q_out=out)
    _same(raw, scales, out, want, K.FMT_BF16)
    assert bool((wide[..., :8] == 3).all()) and bool((wide[..., 72:] == 3).all())
    with pytest.raises(ValueError, match="overlap"):
        mla.kv_insert_rope(*a, **kw, q_pe=qt[..., 128:], q_out=wide[0, 0, :64].expand(50, 6, 64))


def test_empty_call():
    import mla_decode_attention_05_gb300 as mla
    inp, pos, q = _setup(4, 1, 2, 9)
    a, kw, raw, _ = _args(inp, K.FMT_BF16, pos)
    kw["positions"] = kw["positions"][:0]
    c, qo = mla.kv_insert_rope(a[0][:0], a[1][:0], a[2], a[3][:0], a[4], **kw, q_pe=q.cuda()[:0, :, 128:])
    assert qo.shape == (0, 2, 64)
    torch.cuda.synchronize()
    assert bool((raw == 0xAB).all())
