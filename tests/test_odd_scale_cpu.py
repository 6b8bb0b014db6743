"""What the tests of FP8 caches with one scale compare with: exact rows, which rounded
ones differ from."""
import numpy as np

from _long import Cache
from _odd_scale import odd_scale
from oracle import long_context as O


def test_rounded_and_exact_rows_differ():
    c = odd_scale(Cache(np.random.default_rng(1), 2, "fp8_tensor"))
    pages = c.take(100)
    seen, exact = c.rows(pages, 100), c.exact_rows(pages, 100)
    live = exact != 0
    assert (seen[live] != exact[live]).mean() > 0.9
    assert np.abs(seen / np.where(live, exact, 1) - live).max() <= 2.0 ** -8 + 2.0 ** -23


def test_the_difference_shows_in_sums_and_weights():
    """An oracle of rounded rows in the place of one of exact rows would be seen."""
    rng = np.random.default_rng(2)
    c = odd_scale(Cache(rng, 2, "fp8_tensor"))
    pages = c.take(60)
    q = 1.3 * rng.standard_normal((1, 8, 576))
    exact = O.attention(q, np.zeros((0, 576)), c.exact_rows(pages, 60), 192 ** -0.5, False)
    rounded = O.attention(q, np.zeros((0, 576)), c.rows(pages, 60), 192 ** -0.5, False)
    assert np.abs(exact["lse"] - rounded["lse"]).max() > 1e-3
    m, _ = O.mass(q, c.exact_rows(pages, 60), exact["lse"], 192 ** -0.5, False)
    r, _ = O.mass(q, c.rows(pages, 60), exact["lse"], 192 ** -0.5, False)
    assert np.abs(m / r - 1).max() > 1e-3
