"""Blocks with one and with two row tiles in turn on every SM, with NaN among the values: the rows
that see one show it, whatever the SM goes on to, and no others."""
import pytest
import torch

from test_gpu_attn import Batch, q  # noqa: F401 (fixture)
from test_gpu_kv_cache import FMTS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H", [1, 2])
def test_nan_rows_of_blocks_in_turn(q, fmt, D, H):  # noqa: F811
    # rows per KV head: 200 (two tiles, the second not full), then 40 to 120 (one) three times over
    lens = []
    for i in range(120):
        lens += [(50, 50 + 3 * i), (30, 30 + i), (10, 10 + 2 * i), (25, 400)]
    bad = list(range(0, len(lens), 4)) + list(range(3, len(lens), 8))

    def edit(b, k, v):
        for s in bad:
            c, n = b.lens[s]
            v[b.slots[s][n - 2], 0, 3] = torch.nan                     # seen by the last two tokens
    b = Batch(q, fmt, 4 * H, H, D, 16, lens, seed=81, edit=edit)
    out, lse = b.run(q)
    clean, cl = Batch(q, fmt, 4 * H, H, D, 16, lens, seed=81).run(q)
    start = torch.cumsum(torch.tensor([0] + [c for c, _ in lens]), 0)
    sees = torch.zeros(out.shape[:2], dtype=torch.bool)
    for s in bad:
        sees[start[s + 1] - 2:start[s + 1], :4] = True
    sees = sees.cuda()
    assert torch.equal(lse, cl)
    assert torch.isnan(out[sees][:, 3]).all()
    assert torch.equal(out[~sees], clean[~sees])
