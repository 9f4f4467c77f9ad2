"""One NaN value per sequence, at every place of it: exactly the rows that see its token show it,
whatever tile, half of a tile or cut by the mask it lies in; all other outputs keep their bits."""
import pytest
import torch

import kv_ref
from test_gpu_attn import Batch, q  # noqa: F401 (fixture)
from test_gpu_kv_cache import FMTS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("c,n,causal,window", [
    (60, 160, True, 0), (60, 250, True, 0), (100, 230, True, 0), (50, 420, True, 200), (70, 500, True, 130),
    (60, 200, False, 0), (1, 100, True, 0), (3, 150, True, 70), (2, 90, False, 0),
])
def test_a_nan_anywhere(q, fmt, D, c, n, causal, window):  # noqa: F811
    step = 3
    places = list(range(0, n, step)) + [n - 1]
    lens = [(c, n)] * len(places)

    def edit(b, k, v):
        for s, t in enumerate(places):
            v[b.slots[s][t], 0, 5] = torch.nan
    b = Batch(q, fmt, 6, 2, D, 16, lens, seed=101, edit=edit)
    out, lse = b.run(q, causal=causal, window=window)
    clean, cl = Batch(q, fmt, 6, 2, D, 16, lens, seed=101).run(q, causal=causal, window=window)
    see = kv_ref.visible(c, n, causal, window)                           # [c, n]
    sees = torch.zeros((len(places), c, 6), dtype=torch.bool)
    for s, t in enumerate(places):
        sees[s, :, :3] = see[:, t, None]
    sees = sees.view(-1, 6).cuda()
    assert torch.equal(lse, cl)
    assert torch.equal(out[~sees], clean[~sees])
    lost = sees & ~torch.isnan(out[..., 5])
    assert not lost.any(), sorted({places[i // c] for i in lost.any(1).nonzero().flatten().tolist()})
