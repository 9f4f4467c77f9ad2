"""Paged attention over long contexts, held to bounds that see a lost part, and over contexts near
the longest it takes."""
import math

import pytest
import torch

import attn_bounds
import kv_ref
from test_gpu_attn import Batch, q  # noqa: F401 (fixture)
from test_gpu_kv_cache import FMTS, SCALE

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [2 ** 31 - 16, 2 ** 31 - 17, 2 ** 31 - 40])
@pytest.mark.parametrize("c,causal", [(1, True), (40, False)])
def test_contexts_up_to_2_31(q, n, c, causal):  # noqa: F811
    """One page of 16 tokens, 2^27 times: each of its keys has its softmax weight n / 16 times over
    (exactly so but for the last page's missing tokens, 2^-27 of it). The sums' errors are at most the
    additions to one fp32 number times 2^-24: 16 per 128 keys on one of 152 or more SMs."""
    D, page = 64, 16
    g = torch.Generator(device="cuda").manual_seed(41)
    cache = q.kv_cache("nvfp4", 2, page, 1, D, *SCALE["nvfp4"])
    k = torch.randn((page, 1, D), generator=g, device="cuda").bfloat16()
    v = torch.randn((page, 1, D), generator=g, device="cuda").bfloat16()
    q.qmv_kv_write(cache, k, v, torch.arange(page, device="cuda"))
    rk, rv = (t.double() for t in q.qmv_kv_read(cache, torch.arange(page, device="cuda"), torch.float32))
    qq = torch.randn((c, 4, D), generator=g, device="cuda").bfloat16()
    table = torch.zeros((1, 2 ** 27 - 1), dtype=torch.int32, device="cuda")
    lse = torch.zeros((c, 4), device="cuda")
    out = q.qmv_attn_paged(cache, qq, table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                           torch.tensor([0, c], dtype=torch.int32, device="cuda"), c, q.attn_workspace(cache, 4),
                           causal=causal, lse=lse)
    assert q.qmv_device_status() == 0
    ref, rl, mag, _ = kv_ref.attention(qq.double(), [rk], [rv], [(c, page)], D ** -0.5, False, 0)
    sums = 16 * (2 ** 24 / 152) * 2.0 ** -24 + 2.0 ** -9
    assert ((out.double() - ref).abs() <= sums * mag + 2.0 ** -7 * (mag + ref.abs())).all()
    assert ((lse.double() - rl - math.log(n / page)).abs() <= 2 * sums).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [[(1, 40000), (1, 3)], [(8, 20011)], [(4, 30011), (3, 9000)], [(130, 9000), (1, 20000)],
                                  [(64, 60000)]])
def test_no_part_of_a_long_context_is_lost(q, fmt, D, lens):  # noqa: F811
    def edit(b, k, v):
        g = torch.Generator(device="cuda").manual_seed(43)
        for s, (_, n) in zip(b.slots, b.lens):
            v[s.cuda()] = (0.5 * v[s.cuda()] + attn_bounds.drift(n, 1, D, g, "cuda")).bfloat16()
    b = Batch(q, fmt, 4, 1, D, 64, lens, seed=42, edit=edit)
    out, lse = b.run(q)
    sc = float(torch.tensor(D ** -0.5))
    t = 0
    for (c, n), k, v in zip(lens, b.keys, b.values):
        rows = slice(t, t + c)
        ref, rl, mag, dots = kv_ref.attention(b.q[rows].double(), [k], [v], [(c, n)], sc, True, 0)
        bo, bl = attn_bounds.tight(fmt, ref, rl, mag, dots, n, float(v.abs().max()))
        assert ((out[rows].double() - ref).abs() <= bo).all()
        assert ((lse[rows].double() - rl).abs() <= bl).all()
        t += c
