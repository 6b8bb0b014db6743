"""Helpers of the tests of the operators for long contexts: paged caches in the
three formats, with what the kernels read of them in float64."""
import numpy as np
import torch

from _ops import HALF_BF16, STEP_F32, f64


class Cache:
    """A pool of pages.  `exact_rows(pages, n)` gives the first n tokens behind a
    page list, FP8 rows as code times scale; `rows` has these rounded to bf16, as
    the decode kernel sees them."""

    def __init__(self, rng, pages, fmt, std=1.0):
        self.fmt, self.pages = fmt, pages
        x = torch.from_numpy(rng.standard_normal((pages, 64, 576)).astype(np.float32) * np.float32(std))
        self.scales = None
        if fmt == "bf16":
            self.data = x.to(torch.bfloat16)
            self.seen = self.exact = self.data.double()
        elif fmt == "fp8_tensor":
            self.scales = torch.tensor([2.0 ** -6 * 1.25])
            codes = (x / self.scales).clamp(-448, 448).to(torch.float8_e4m3fn)
            self.data = codes.view(torch.uint8)
            self.seen = (codes.float() * self.scales).to(torch.bfloat16).double()
            self.exact = codes.double() * self.scales.double()
        else:
            tiles = x[..., :512].reshape(pages, 64, 4, 128)
            self.scales = (tiles.abs().amax(-1) / 448).contiguous()
            codes = (tiles / self.scales[..., None]).to(torch.float8_e4m3fn)
            pe = x[..., 512:].to(torch.bfloat16)
            self.data = torch.cat([codes.view(torch.uint8).reshape(pages, 64, 512), pe.view(torch.uint8)], -1).contiguous()
            latent = (codes.float() * self.scales[..., None]).to(torch.bfloat16).reshape(pages, 64, 512)
            self.seen = torch.cat([latent, pe], -1).double()
            latent = (codes.double() * self.scales[..., None].double()).reshape(pages, 64, 512)
            self.exact = torch.cat([latent, pe.double()], -1)
        self.order = [int(i) for i in rng.permutation(pages)]

    def take(self, n):
        """Pages for n tokens."""
        k = -(-n // 64)
        got, self.order = self.order[:k], self.order[k:]
        assert len(got) == k
        return got

    def spoil(self, used):
        """nan and inf into every row that is not among `used` [(pages, tokens)]."""
        free = torch.ones(self.pages * 64, dtype=torch.bool)
        for pages, n in used:
            for i in range(n):
                free[pages[i // 64] * 64 + i % 64] = False
        flat = self.data.view(self.pages * 64, -1)
        if self.fmt == "bf16":
            flat[free] = float("nan")
            flat[free, ::2] = float("inf")
        else:
            flat[free] = 0x7F
            if self.fmt == "fp8":
                self.scales.view(-1, 4)[free] = float("inf")

    def rows(self, pages, n):
        if n == 0:
            return np.zeros((0, 576))
        return self.seen[pages].reshape(-1, 576)[:n].numpy()

    def exact_rows(self, pages, n):
        if n == 0:
            return np.zeros((0, 576))
        return self.exact[pages].reshape(-1, 576)[:n].numpy()

    def cuda(self):
        return self.data.cuda(), None if self.scales is None else self.scales.cuda()


def table(lists, width=None):
    """Page lists as a table, -1 behind the last page of each."""
    w = width or max(1, max(len(p) for p in lists))
    t = torch.full((len(lists), w), -1, dtype=torch.int32)
    for b, p in enumerate(lists):
        t[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    return t.cuda()


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def check_rows(got, lse, ref, n_keys, fmt="bf16"):
    """One sequence's out [T, H, 512] and lse [T, H] against oracle.long_context's.

    Score error d: 576 products in fp32, and the rounding of score and reference
    in the exponent.  p: relative error d + 2^-21 (the exponential), then half a
    bf16 step.  The sum: the same without that step, and n additions.  out: the
    weighted sum of |v| times these, n additions, the join's weights (d again),
    and half a bf16 step of the result.

    FP8 with one scale: codes are exact, two more roundings of scores and output in
    fp32.  With a scale for each 128 values: each product of code and scale is the
    sum of two bf16 values as a key (half a step of half a step, 512 products more),
    and rounded to bf16 as a value (half a step)."""
    d = 576 * STEP_F32 * ref["mag"] + 4 * STEP_F32 * ref["top"] + 2.0 ** -20
    v = 0.0
    if fmt == "fp8_tensor":
        d, v = d + 2 * STEP_F32 * ref["top"], 2 * STEP_F32
    elif fmt == "fp8":
        d, v = d + (512 * STEP_F32 + HALF_BF16 ** 2) * ref["mag"], HALF_BF16 + STEP_F32
    n = max(1, n_keys) * STEP_F32
    got, lse = f64(got), f64(lse)
    empty = np.isneginf(ref["lse"])
    assert np.array_equal(np.isneginf(lse), empty)
    assert np.all(got[empty] == 0)
    live = ~empty
    err = np.abs(lse[live] - ref["lse"][live])
    tol = (d + n)[live] + 4 * STEP_F32 * np.abs(ref["lse"][live]) + 4 * STEP_F32 * ref["top"][live]
    assert np.all(err <= tol), f"lse off by {err.max()}, bound {tol[err.argmax()]}"
    rel = (HALF_BF16 + v + 3 * d + 2 * n)[..., None]
    tol = ref["spread"] * rel + HALF_BF16 * (np.abs(ref["out"]) + ref["spread"] * rel) + 1e-38
    err = np.abs(got - ref["out"])[live]
    assert np.all(err <= tol[live]), f"out off by {err.max()}"
