"""GPU parity of the value projection (mla_value_project) against float64: each
value within half a bf16 step and the bound of an fp32 sum of 512 products."""
import numpy as np
import pytest
import torch

from _ops import bf16, check_sum, f64
from oracle import prefill as O

pytestmark = pytest.mark.gpu


def _check(out, attn, w):
    want, mag = O.value_project(f64(attn), f64(w))
    check_sum(out, want, mag, 512)


@pytest.mark.parametrize("N,H", [(1, 1), (1, 128), (15, 2), (16, 3), (17, 1), (48, 2), (63, 4), (64, 5), (65, 2),
                                 (129, 8), (200, 20), (700, 1)])
def test_value_project(N, H):
    import mla_decode_attention_05_gb300 as mla
    rng = np.random.default_rng(N * 1000 + H)
    attn, w = bf16(rng, (N, H, 512), 0.5).cuda(), bf16(rng, (H, 128, 512), 0.05).cuda()
    mla.device_status()
    out = mla.value_project(attn, w)
    _check(out, attn, w)
    assert mla.device_status() == 0


def test_layouts_and_rows_behind_the_last():
    """Heads before tokens, wider rows, a weight that is half of a larger one,
    a given output whose other rows stay."""
    import mla_decode_attention_05_gb300 as mla
    rng = np.random.default_rng(5)
    N, H = 70, 6
    attn, w = bf16(rng, (N, H, 512), 0.5).cuda(), bf16(rng, (H, 256, 512), 0.05).cuda()
    base = mla.value_project(attn, w[:, 128:].contiguous())
    _check(base, attn, w[:, 128:])
    assert torch.equal(mla.value_project(attn, w[:, 128:]), base)
    assert torch.equal(mla.value_project(attn.transpose(0, 1).contiguous().transpose(0, 1), w[:, 128:]), base)
    wide = torch.zeros((N, H, 576), dtype=torch.bfloat16, device="cuda")
    wide[..., :512] = attn
    big = torch.full((N + 30, H, 128), 4.0, dtype=torch.bfloat16, device="cuda")
    mla.value_project(wide[..., :512], w[:, 128:], out=big[:N])
    assert torch.equal(big[:N], base) and bool((big[N:] == 4).all())
    with pytest.raises(ValueError, match="stride"):
        mla.value_project(attn.transpose(0, 2).contiguous().transpose(0, 2), w[:, 128:])


def test_a_row_that_is_not_finite_stays_alone():
    import mla_decode_attention_05_gb300 as mla
    rng = np.random.default_rng(6)
    attn, w = bf16(rng, (90, 3, 512), 0.5).cuda(), bf16(rng, (3, 128, 512), 0.05).cuda()
    base = mla.value_project(attn, w)
    attn[66, 1, 7] = float("inf")
    out = mla.value_project(attn, w)
    assert not bool(out[66, 1].isfinite().any())
    out[66, 1] = base[66, 1]
    assert torch.equal(out, base)


def test_empty_call():
    import mla_decode_attention_05_gb300 as mla
    z = torch.zeros((2, 128, 512), dtype=torch.bfloat16, device="cuda")
    assert mla.value_project(z[:0, :2].reshape(0, 2, 512), z).shape == (0, 2, 128)


@pytest.mark.parametrize("N,H", [(3000, 8), (10000, 1), (33, 128)])
def test_many_tiles_in_one_block(N, H):
    """More tiles than SMs, with and without a change of the head in a block's
    share: a row's bits are those it has in a call of its own tile."""
    import mla_decode_attention_05_gb300 as mla
    rng = np.random.default_rng(N)
    attn, w = bf16(rng, (N, H, 512), 0.5).cuda(), bf16(rng, (H, 128, 512), 0.05).cuda()
    mla.device_status()
    out = mla.value_project(attn, w)
    for a in (0, 64 * (N // 128), 64 * (N // 64) - (64 if N % 64 == 0 else 0)):
        assert torch.equal(out[a:a + 64], mla.value_project(attn[a:a + 64], w))
    _check(out[-70:], attn[-70:], w)
    assert mla.device_status() == 0
