"""The bounds that long contexts are held to see a part of the sequence that is lost, counted
twice or misweighted; computed on the host with 64-bit attention."""
import pytest
import torch

import attn_bounds
import kv_ref
from test_gpu_kv_cache import SCALE


@pytest.mark.parametrize("fmt", ["bf16", "q8_0", "fp8", "nvfp4"])
@pytest.mark.parametrize("n,part", [(40000, 264), (20011, 132), (9000, 64), (5000, 32)])
def test_a_part_that_is_lost_exceeds_the_bound(fmt, n, part):
    """part: the tokens of one of 152 SMs, or a tile. Q8_0's bound, twice the others' because its
    keys enter the products as f16(d q), sees half the weight gone over two of them."""
    D = 64
    g = torch.Generator().manual_seed(71)
    k = torch.randn((n, 1, D), generator=g)
    v = 0.5 * torch.randn((n, 1, D), generator=g) + attn_bounds.drift(n, 1, D, g)
    k, v = (torch.from_numpy(kv_ref.stored(fmt, t.bfloat16().float().numpy(), s)) for t, s in zip((k, v), SCALE[fmt]))
    qq = torch.randn((1, 2, D), generator=g).bfloat16().double()
    full = lambda vv: kv_ref.attention(qq, [k], [vv], [(1, n)], D ** -0.5, True, 0)
    ref, rl, mag, dots = full(v)
    b, _ = attn_bounds.tight(fmt, ref, rl, mag, dots, n, float(v.abs().max()))
    assert (b < 0.03).all()
    for at in (0, n // 3, n - part):
        for weight in (0.0, 2.0, 0.5):
            long = 2 * part if fmt == "q8_0" and weight == 0.5 else part
            w = v.clone()
            w[min(at, n - long):][:long] *= weight
            off = (full(w)[0] - ref).abs()
            assert (off > b).any(), (at, weight, float((off / b).max()))
