"""The failure path of the prefill attention, the expansion and the value
projection, as test_failure_gpu.py has it for the decode: ordinary calls with
the limit of every wait shortened to a microsecond, so that real waits run
out; the status word tells, the kernels return, and the next calls, right
behind in the stream and after a look at the status, are right."""
import numpy as np
import pytest
import torch

import workloads as W
from _ops import bf16, cu

pytestmark = pytest.mark.gpu


def _prefill(mla, nq, nk, H, bad=None):
    rng = np.random.default_rng(61)
    kv = bf16(rng, (sum(nk), H, 256)).cuda()
    if bad is not None:
        kv[bad, :, 128:] = float("nan")  # values are looked through
    args = (bf16(rng, (sum(nq), H, 192)).cuda(), kv[..., :128], bf16(rng, (sum(nk), 64)).cuda(), kv[..., 128:], cu(nq), cu(nk))
    return lambda: mla.prefill(*args, softmax_scale=192 ** -0.5)


def _expand(mla, lens, H, fmt):
    w = W.make_workload("expand", len(lens), 1, 1, lens, seed=62, fp8=fmt == "fp8", fp8_tensor=fmt == "fp8_tensor")
    rng = np.random.default_rng(63)
    w_kv = bf16(rng, (H, 256, 512), 0.05).cuda()
    cache = (torch.from_numpy(w.kv.view(np.int16)).view(torch.bfloat16) if fmt == "bf16" else torch.from_numpy(w.kv)).cuda()
    sc = None if fmt == "bf16" else torch.from_numpy(w.kv_scales).cuda()
    bt, ends = torch.from_numpy(w.block_table).cuda(), cu(lens)
    return lambda: mla.kv_expand(cache, bt, ends, w_kv[:, :128], w_kv[:, 128:], total=sum(lens), kv_scales=sc)


def _value(mla, N, H):
    rng = np.random.default_rng(64)
    attn, w = bf16(rng, (N, H, 512), 0.5).cuda(), bf16(rng, (H, 128, 512), 0.05).cuda()
    return lambda: (mla.value_project(attn, w),)


CASES = {
    "prefill": lambda m: _prefill(m, [600, 130], [600, 300], 4),
    "prefill_takes_over_blocks": lambda m: _prefill(m, [700] * 8, [700] * 8, 16),
    "prefill_split": lambda m: _prefill(m, [200], [2200], 2),
    "prefill_done_again": lambda m: _prefill(m, [300] * 3, [300] * 3, 3, bad=slice(250, 260)),
    "expand_few": lambda m: _expand(m, [300], 8, "bf16"),
    "expand_many": lambda m: _expand(m, [2000, 301], 64, "bf16"),
    "expand_fp8": lambda m: _expand(m, [700, 90], 8, "fp8"),
    "expand_fp8_tensor": lambda m: _expand(m, [100], 64, "fp8_tensor"),
    "value_few": lambda m: _value(m, 64, 128),
    "value_many": lambda m: _value(m, 3000, 8),
}


@pytest.mark.parametrize("case", CASES)
def test_waits_run_out_then_next_call_is_correct(case):
    import mla_decode_attention_05_gb300 as mla
    call = CASES[case](mla)
    mla.device_status()
    want = call()
    assert mla.device_status() == 0
    mla.set_wait_limit_ns(1000)  # 1 us: the kernels' ordinary waits are longer
    try:
        call()
    finally:
        mla.set_wait_limit_ns(0)
    behind = call()  # launched as a dependent of the one that gives up
    assert mla.device_status() == mla.STATUS_WAIT_TIMEOUT, "no wait ran out"
    after = call()
    assert mla.device_status() == 0
    same = lambda a, b: torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())
    assert all(same(a, b) for got in (behind, after) for a, b in zip(got, want))


def test_a_long_limit_changes_nothing():
    """Limits above what the prefill's 32-bit clock holds."""
    import mla_decode_attention_05_gb300 as mla
    calls = [CASES[c](mla) for c in ("prefill", "expand_few", "value_few")]
    want = [c() for c in calls]
    for ns in (3_000_000, 5_000_000_000, 1 << 62):
        mla.set_wait_limit_ns(ns)
        try:
            got = [c() for c in calls]
        finally:
            mla.set_wait_limit_ns(0)
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    assert mla.device_status() == 0
