"""Limits of the cache's and its attention's arguments, checked on the host."""
import ctypes

import pytest

from test_kv_abi import desc


@pytest.fixture(scope="module")
def q():
    import block_quantized_weight_fly_gb300 as q
    return q


@pytest.mark.parametrize("fmt", [1, 2, 3, 4])
@pytest.mark.parametrize("dim", [64, 256])
def test_sizes_past_63_bits_are_refused(q, fmt, dim):
    """Never a size that wrapped: 2^28 + 1 pages of 1024 tokens x 65536 heads are 2^64 bytes and
    a little for D = 256 in bf16."""
    row = {1: 2 * dim, 2: dim + dim // 16, 3: dim, 4: dim // 2 + dim // 16}[fmt]
    for pages in (1, 1 << 20, (1 << 27) + 1, (1 << 28) + 1, (1 << 30) + 5, (1 << 31) - 1):
        c = desc(q, fmt=fmt, page=1024, heads=65536, dim=dim, pages=pages)
        true = pages * 65536 * 1024 * 2 * row
        size = q._kv_size(ctypes.byref(c))
        assert size == (true if true < 1 << 48 else 0), (pages, true)
        if size == 0:                                  # the calls refuse it too
            P = ctypes.c_void_p(256)
            assert q._kv_read(ctypes.byref(c), P, 4, P, P, 1, None) == 3
            assert q._kv_write(ctypes.byref(c), P, P, 1, 128, 64, 128, 64, P, 4, None) == 3
            assert q._attn_ws(ctypes.byref(c), 65536) == 0


def test_nvfp4_scales_whose_six_fold_leaves_fp32_are_refused(q):
    """b = amax / (6 s): with 6 s = inf every block would be stored as zeros."""
    for s, served in ((5.6e37, True), (5.7e37, False), (1e38, False), (2.9e38, False)):
        for kw in (dict(ks=s), dict(vs=s)):
            assert (q._kv_size(ctypes.byref(desc(q, fmt=4, **kw))) > 0) == served, (s, kw)
            assert q._kv_size(ctypes.byref(desc(q, fmt=3, **kw))) > 0
