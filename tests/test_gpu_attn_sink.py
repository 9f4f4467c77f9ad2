"""A key that outweighs all others by far and whose value is zero (an attention sink): the output
is then made of the small probabilities alone, which 16-bit probabilities must still hold."""
import pytest
import torch

import attn_bounds
import kv_ref
from test_gpu_attn import q  # noqa: F401 (fixture)
from test_gpu_kv_cache import FMTS, SCALE

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,n,c", [(170, 4096, 1), (170, 4096, 60), (1, 65536, 1), (1, 65536, 60)])
def test_small_probabilities_beside_a_sink(q, fmt, D, B, n, c):  # noqa: F811
    """B sequences over the same pages (170: no unit is cut, one warp or thread carries a row through
    all its keys), the sink at their start, logits of the others around 0."""
    G, page = 4, 64
    g = torch.Generator(device="cuda").manual_seed(51)
    for gap in (12.0, 16.0, 18.0, 20.0):
        k = 0.5 * torch.randn((n, 1, D), generator=g, device="cuda")
        k[:, :, 0] = 0
        k[0] = 0
        k[0, :, 0] = gap / 4
        v = 1 + 0.25 * torch.randn((n, 1, D), generator=g, device="cuda")
        v[0] = 0
        cache = q.kv_cache(fmt, n // page, page, 1, D, *SCALE[fmt])
        slots = torch.arange(n, device="cuda")
        q.qmv_kv_write(cache, k, v, slots)
        rk, rv = (t.double() for t in q.qmv_kv_read(cache, slots, torch.float32))
        qq = 0.1 * torch.randn((B * c, G, D), generator=g, device="cuda")
        qq[:, :, 0] = 4
        qq = qq.bfloat16()
        lse = torch.zeros((B * c, G), device="cuda")
        # not causal: all queries see all keys, and all sequences are alike
        out = q.qmv_attn_paged(cache, qq, torch.arange(n // page, dtype=torch.int32, device="cuda").repeat(B, 1),
                               torch.full((B,), n, dtype=torch.int32, device="cuda"),
                               torch.arange(0, B * c + 1, c, dtype=torch.int32, device="cuda"), c,
                               q.attn_workspace(cache, G), scale=1.0, causal=False, lse=lse)
        assert q.qmv_device_status() == 0
        ref, rl, mag, dots = kv_ref.attention(qq.double(), [rk], [rv], [(B * c, n)], 1.0, False, 0)
        b, bl = attn_bounds.tight(fmt, ref, rl, mag, dots, n, float(rv.abs().max()))
        err = (out.double() - ref).abs()
        assert (err <= b).all(), (gap, float((err / b).max()), float(out.float().mean()), float(ref.mean()))
        assert ((lse.double() - rl).abs() <= bl).all(), gap
