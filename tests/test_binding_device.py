"""Tensors of a device that is not the current one are refused before a kernel is launched."""
import pytest
import torch


class Elsewhere:
    """What the binding asks of a contiguous tensor on device 1."""
    is_cuda, dtype, shape, device = True, torch.bfloat16, (1, 256), "cuda:1"
    dim = lambda self: 2
    is_contiguous = lambda self: True
    get_device = lambda self: 1
    data_ptr = lambda self: 256
    numel = lambda self: 256
    element_size = lambda self: 2


def test_tensors_elsewhere_are_refused(monkeypatch):
    import block_quantized_weight_fly_gb300 as q
    monkeypatch.setattr(q, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        q._ptr(Elsewhere())
    with pytest.raises(ValueError, match="current device"):
        q.qmv_quant_act_nvfp4(Elsewhere(), 1.0, *[type("Bytes", (Elsewhere,), {"dtype": torch.uint8})()] * 2)
    monkeypatch.setattr(q, "_current_device", lambda: 1)
    assert q._ptr(Elsewhere()).value == 256
    assert q._ptr(None) is None
