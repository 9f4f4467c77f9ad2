"""The chunk kernel's rings while copies arrive late and out of order: long rings of tiles per SM over
pages in a new random order each time, out of a cache that other writes have pushed out of L2.
No wait may run out, and every call gives the same bits."""
import pytest
import torch

from test_gpu_attn import q  # noqa: F401 (fixture)
from test_gpu_kv_cache import FMTS, SCALE

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_late_copies(q, fmt, D, page):  # noqa: F811
    n, c, G = 65536, 60, 4
    g = torch.Generator(device="cuda").manual_seed(61)
    k = torch.randn((n, 1, D), generator=g, device="cuda").bfloat16()
    v = torch.randn((n, 1, D), generator=g, device="cuda").bfloat16()
    qq = torch.randn((c, G, D), generator=g, device="cuda").bfloat16()
    cache = q.kv_cache(fmt, n // page, page, 1, D, *SCALE[fmt])
    ws = q.attn_workspace(cache, G)
    length = torch.tensor([n], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, c], dtype=torch.int32, device="cuda")
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    j = torch.arange(n, device="cuda")
    first = None
    for i in range(24):
        table = torch.randperm(n // page, generator=g, device="cuda").to(torch.int32)
        q.qmv_kv_write(cache, k, v, table.long()[j // page] * page + j % page)
        if i % 3:
            flush.fill_(i)
        if i % 3 == 1:
            q.qmv_kv_read(cache, j[: n // 2])                   # half of it back in L2
        out = q.qmv_attn_paged(cache, qq, table[None], length, start, c, ws, causal=i % 2 == 0)
        assert q.qmv_device_status() == 0, i
        if i < 2:
            first = [out] if first is None else first + [out]
        assert torch.equal(out, first[i % 2]), i
