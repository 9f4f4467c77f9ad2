"""Batches of single tokens and chunks in a q with rows of no sequence behind them, as a captured
graph's fixed buffers have it: the same bits as without them, and those rows left alone."""
import pytest
import torch

import attn_bounds
import kv_ref
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


@pytest.mark.parametrize("D,Hq,H", [(64, 4, 4), (128, 8, 2), (256, 12, 2)])
@pytest.mark.parametrize("rows", [90, 120])
def test_a_captured_call_serves_any_mix(q, D, Hq, H, rows):  # noqa: F811
    """Fixed buffers of `rows` rows (below and at B max_q), lengths and starts new at every replay."""
    b = Batch(q, "fp8", Hq, H, D, 16, [(30, 400), (30, 90), (20, 333), (1, 64)], seed=92)
    b.max_q = 30
    b.q = torch.cat([b.q, torch.zeros((rows - b.T, Hq, D), dtype=torch.bfloat16, device="cuda")])
    out = torch.zeros_like(b.q)
    args = (b.cache, b.q, b.table, b.kv_len, b.q_start, 30, b.ws)
    q.qmv_attn_paged(*args, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qmv_attn_paged(*args, out=out)
    for cs, ns in (((30, 30, 20, 1), (400, 90, 333, 64)), ((1, 1, 1, 1), (390, 3, 300, 64)), ((30, 1, 1, 30), (200, 1, 30, 40)),
                   ((0, 0, 5, 0), (0, 7, 320, 0)), ((30, 30, 30, 0), (390, 80, 301, 10))):
        b.kv_len.copy_(torch.tensor(ns, dtype=torch.int32))
        b.q_start.copy_(torch.cumsum(torch.tensor((0,) + cs), 0).int())
        out.fill_(3.0)
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        got, used = out.clone(), sum(cs)
        out.fill_(3.0)
        q.qmv_attn_paged(*args, out=out)
        assert q.qmv_device_status() == 0
        assert torch.equal(got, out) and (got[used:] == 3).all() and torch.isfinite(got).all()
        ref, rl, mag, dots = kv_ref.attention(b.q[:used].double(), [k[:n] for k, n in zip(b.keys, ns)],
                                              [v[:n] for v, n in zip(b.values, ns)], list(zip(cs, ns)),
                                              float(torch.tensor(D ** -0.5)), True, 0)
        bound, _ = attn_bounds.tight("fp8", ref, rl, mag, dots, 400, 4.2)
        assert ((got[:used].double() - ref).abs() <= bound).all()
