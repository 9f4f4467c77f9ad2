"""Batches of single tokens and chunks in a q with rows of no sequence behind them, as a captured
graph's fixed buffers have it: the same bits as without them, and those rows left alone."""
import pytest
import torch

from test_gpu_attn import Batch, q  # noqa: F401 (fixture)
from test_gpu_kv_cache import FMTS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,Hq,H", [(64, 4, 4), (128, 8, 2), (256, 12, 2)])
@pytest.mark.parametrize("lens", [[(1, 900), (60, 333), (1, 17), (2, 40)], [(1, 50), (1, 4000)]])
def test_rows_of_no_sequence_change_nothing(q, fmt, D, Hq, H, lens):  # noqa: F811
    b = Batch(q, fmt, Hq, H, D, 16, lens, seed=91)
    b.max_q = 60
    want, wl = b.run(q)
    for rows in (60 * len(lens), 60 * len(lens) + 7):
        qq = torch.zeros((rows, Hq, D), dtype=torch.bfloat16, device="cuda")
        qq[:b.T] = b.q
        out = torch.full_like(qq, 5.0)
        lse = torch.full((rows, Hq), 5.0, device="cuda")
        q.qmv_attn_paged(b.cache, qq, b.table, b.kv_len, b.q_start, 60, b.ws, out=out, lse=lse)
        assert q.qmv_device_status() == 0
        assert torch.equal(out[:b.T], want) and torch.equal(lse[:b.T], wl)
        assert (out[b.T:] == 5).all() and (lse[b.T:] == 5).all()
