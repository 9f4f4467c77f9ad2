"""Outputs that a call allocates for a stream other than the current one: the current stream may still be
writing to memory that was freed there, and the allocator would hand it out."""
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import block_quantized_weight_fly_gb300 as q
    torch.cuda.set_device(0)
    q.qmv_device_status(reset=True)
    return q


def busy(shape, dtype, count):
    """Tensors that the current stream will fill later, given up at once."""
    x = [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(count)]
    torch.cuda._sleep(300_000_000)                                       # some 0.15 s
    for t in x:
        t.fill_(7)


def test_cache_and_attention(q):
    T, H, D = 4096, 4, 128
    g = torch.Generator(device="cuda").manual_seed(95)
    cache = q.kv_cache("bf16", T // 16, 16, H, D)
    k = torch.randn((T, H, D), generator=g, device="cuda").bfloat16()
    slots = torch.arange(T, device="cuda")
    q.qmv_kv_write(cache, k, k, slots)
    args = (cache, k, torch.arange(T // 16, dtype=torch.int32, device="cuda")[None],
            torch.tensor([T], dtype=torch.int32, device="cuda"), torch.tensor([0, T], dtype=torch.int32, device="cuda"),
            T, q.attn_workspace(cache, H))
    want = q.qmv_attn_paged(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    busy((T, H, D), torch.bfloat16, 3)
    rk, rv = q.qmv_kv_read(cache, slots, stream=s)
    out = q.qmv_attn_paged(*args, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(rk, k) and torch.equal(rv, k) and torch.equal(out, want)


def test_gemv(q):
    N, K = 1 << 16, 256
    W = q.qmv_pack("q8_0", q.qmv_quantize("q8_0", synth.weights(3, N, K, device="cuda")), N, K)
    x = synth.activations(4, 8, K).cuda()
    ws = q.workspace(q.QMV_ENTRY_GEMV, "q8_0", 8, N, K)
    want = q.qmv_gemv("q8_0", W, x, N, K, ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    busy((8, N), torch.float32, 1)
    got = q.qmv_gemv("q8_0", W, x, N, K, ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
