"""Helpers of the tests of the operators around the decode.

Bounds (derived, not fitted).  Half a step of a bf16 rounding is 2^-8 of the
value.  A sum of K products in fp32 whose every addition is off by at most one
step (2^-23) of a partial sum is off by at most K * 2^-23 * sum |products|."""
import numpy as np
import torch

HALF_BF16 = 2.0 ** -8
STEP_F32 = 2.0 ** -23


def bf16(rng, shape, std=1.0):
    """N(0, std) rounded to bf16 on the CPU."""
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * np.float32(std)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def check_sum(got, want, mag, K):
    """got: bf16 of an fp32 sum of K products; want, mag in float64."""
    tol = HALF_BF16 * np.abs(want) * (1 + 2.0 ** -7) + 2 * K * STEP_F32 * mag + 1e-38
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), float(np.max(err - tol))


def cu(lens, device="cuda"):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=device)


def check_attention(got, lse, ref, n_keys, scale=None):
    """One sequence's out [nq, H, 128] and lse [nq, H] against oracle.prefill.attention's.

    score error d: 192 products in fp32, and the rounding of score and reference
    in the exponent (|s| log2 e * 2^-23 each).  p: relative error d + 2^-21 (the
    exponential), then half a bf16 step.  l: the same without the bf16 step, and
    n additions.  out: the weighted sum of |v| times these, n additions, half a
    bf16 step of the result."""
    d = 192 * STEP_F32 * ref["mag"] + 4 * STEP_F32 * ref["top"] + 2.0 ** -21
    n = max(1, n_keys) * STEP_F32
    got, lse = f64(got), f64(lse)
    empty = np.isneginf(ref["lse"])
    assert np.array_equal(np.isneginf(lse), empty)
    assert np.all(got[empty] == 0)
    live = ~empty
    err = np.abs(lse[live] - ref["lse"][live])
    tol = (d + n)[live] + 4 * STEP_F32 * np.abs(ref["lse"][live])
    assert np.all(err <= tol), f"lse off by {err.max()}, bound {tol[err.argmax()]}"
    rel = (HALF_BF16 + 2 * d + 2 * n)[..., None]
    tol = ref["spread"] * rel + HALF_BF16 * (np.abs(ref["out"]) + ref["spread"] * rel) + 1e-38
    err = np.abs(got - ref["out"])[live]
    assert np.all(err <= tol[live]), f"out off by {err.max()}"
