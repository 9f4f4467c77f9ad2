"""The cache's and its attention's binding on a machine without a GPU: what it refuses before it
calls the library. A stand-in cache on device -1, where CPU tensors are, passes the device
checks of the tensors."""
import ctypes
import types

import pytest
import torch


@pytest.fixture
def q(monkeypatch):
    import block_quantized_weight_fly_gb300 as q
    monkeypatch.setattr(q, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(q, "_current_device", lambda: -1)
    for name in ("_kv_write", "_kv_read", "_attn", "_attn_ws"):          # nothing reaches the library
        monkeypatch.setattr(q, name, lambda *a: 0)
    return q


def stand_in(q):
    c = q.KvCache.__new__(q.KvCache)
    c.desc = q.KvDesc(1, 16, 2, 64, 4, 1.0, 1.0, 256)
    c.ref = ctypes.byref(c.desc)
    c.heads, c.head_dim, c.index, c.device = 2, 64, -1, torch.device("cpu")
    c.data = torch.zeros(8, dtype=torch.uint8)
    return c


def calls(q, c, **kw):
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    a = dict(q=torch.zeros((3, 4, 64), dtype=torch.bfloat16), page_table=torch.zeros((1, 4), dtype=torch.int32),
             kv_len=torch.zeros(1, dtype=torch.int32), q_start=torch.zeros(2, dtype=torch.int32), max_q=3,
             ws=torch.zeros(64, dtype=torch.uint8))
    a.update({k: v for k, v in kw.items() if k != "stream"})
    s = {"stream": kw["stream"]} if "stream" in kw else {}
    return [lambda: q.qmv_kv_write(c, x, x, slots, **s), lambda: q.qmv_kv_read(c, slots, **s),
            lambda: q.qmv_attn_paged(c, **a, **s)]


def test_the_stand_in_passes(q):
    for call in calls(q, stand_in(q)):
        call()


def test_a_cache_that_is_not_on_the_current_device(q, monkeypatch):
    c = stand_in(q)
    monkeypatch.setattr(q, "_current_device", lambda: 0)
    for call in calls(q, c) + [lambda: q.qmv_attn_workspace_size(c, 4)]:
        with pytest.raises(ValueError, match="current device"):
            call()


def test_a_stream_of_another_device(q):
    other = types.SimpleNamespace(device_index=1, cuda_stream=0)
    for call in calls(q, stand_in(q), stream=other):
        with pytest.raises(ValueError, match="stream"):
            call()


def test_outputs_are_allocated_on_the_stream_that_writes_them(q, monkeypatch):
    """... whose earlier work may not be done with a block of the current stream's."""
    import contextlib
    mine = types.SimpleNamespace(device_index=-1, cuda_stream=0)
    on, took = [None], []

    @contextlib.contextmanager
    def stream(s):
        on.append(s)
        yield
        on.pop()

    empty = torch.empty
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: (took.append(on[-1]), empty(*a, **kw))[1])
    for call in calls(q, stand_in(q), stream=mine):
        call()
    assert took == [mine] * 3                                            # k, v and the attention's out
    took.clear()
    assert q._out(None, (2, 3), "cpu", "y", mine).shape == (2, 3) and took == [mine]
    for call in calls(q, stand_in(q)):
        call()
    assert took[1:] == [None] * 3


def test_a_workspace_that_is_not_contiguous(q):
    """numel() of an expanded or strided tensor says nothing about the memory behind it."""
    c = stand_in(q)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 30), torch.zeros(64, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="ws"):
            calls(q, c, ws=ws)[2]()


def test_integers_that_do_not_fit(q):
    """2^32 + 5 is not 5."""
    c = stand_in(q)
    for name in ("max_q", "window"):
        for value in ((1 << 32) + 5, 1 << 31, -(1 << 31) - 1):
            with pytest.raises(ValueError, match=name):
                calls(q, c, **{name: value})[2]()
    with pytest.raises(ValueError, match="q_heads"):
        q.qmv_attn_workspace_size(c, (1 << 32) + 4)
    good = dict(pages=4, page_size=16, heads=2, head_dim=64)
    for name, value in (("page_size", (1 << 32) + 16), ("heads", (1 << 32) + 2), ("head_dim", (1 << 32) + 64),
                        ("pages", (1 << 64) + 4)):
        with pytest.raises(ValueError, match=name):
            q.KvCache("bf16", **{**good, name: value})
