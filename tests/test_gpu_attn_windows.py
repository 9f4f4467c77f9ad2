"""Paged attention under windows of every size the entry takes, beside sequences with more new
tokens than cached ones (their first queries stand before the first key), against 64-bit
softmax attention."""
import pytest

from test_gpu_attn import Batch, q  # noqa: F401 (fixture)
from test_gpu_kv_cache import FMTS

pytestmark = pytest.mark.gpu

WINDOWS = [1, 2, 40, 1 << 20, 1 << 30, 2 ** 31 - 1]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [
    [(5, 2), (1, 300), (3, 0)],                    # few rows
    [(8, 3), (8, 8), (6, 500)],
    [(200, 150), (90, 1), (1, 300), (130, 0)],     # chunks, with and without single tokens
    [(300, 3), (300, 700)],
])
def test_windows_with_queries_before_the_first_key(q, fmt, D, lens):  # noqa: F811
    b = Batch(q, fmt, 4, 2, D, 16, lens, seed=31)
    for window in WINDOWS:
        b.check(q, window=window)


@pytest.mark.parametrize("lens", [[(5, 2), (1, 300)], [(200, 150), (90, 1), (1, 300)]])
def test_a_window_of_the_whole_cache_is_none(q, lens):  # noqa: F811
    b = Batch(q, "fp8", 8, 2, 128, 16, lens, seed=32)
    want, lse = b.run(q)
    for window in (300, 1 << 25, 2 ** 31 - 1):
        got, gl = b.run(q, window=window)
        assert (got == want).all() and (gl == lse).all()
