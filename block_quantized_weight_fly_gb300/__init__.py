"""Python binding of libqmv: block-quantized weight GEMV on GB300 (sm_103a).

Argument marshalling only. Every function has the name of the C entry point it
calls (include/qmv.h), takes torch tensors for device buffers, passes their raw
pointers and the current CUDA stream, and raises QmvError on a non-zero status.
All arithmetic runs in the CUDA kernels of libqmv.so; there is no fallback: if
the library has not been built, importing this package raises.
"""
from __future__ import annotations

import ctypes
import operator
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqmv.so")

QMV_Q8_0, QMV_Q4_K, QMV_Q6_K, QMV_NVFP4, QMV_FP8_ROW, QMV_Q5_K = 1, 2, 3, 4, 5, 6
QMV_IQ4_XS, QMV_IQ3_S, QMV_IQ2_S = 7, 8, 9
FORMATS = {"q8_0": QMV_Q8_0, "q4_k": QMV_Q4_K, "q6_k": QMV_Q6_K, "nvfp4": QMV_NVFP4,
           "fp8_row": QMV_FP8_ROW, "q5_k": QMV_Q5_K, "iq4_xs": QMV_IQ4_XS, "iq3_s": QMV_IQ3_S,
           "iq2_s": QMV_IQ2_S}
GRID_BYTES = {"iq3_s": 512 * 4, "iq2_s": 1024 * 8}
QMV_ENTRY_GEMV, QMV_ENTRY_GROUPED, QMV_ENTRY_W4A4, QMV_ENTRY_SWIGLU = 1, 2, 3, 4
QMV_ENTRY_GROUPED_SWIGLU, QMV_ENTRY_KQUANT, QMV_ENTRY_MLP_LAYER, QMV_ENTRY_INT8DOT = 5, 6, 7, 8
QMV_MAX_M = 8
QMV_KV_BF16, QMV_KV_Q8_0, QMV_KV_FP8, QMV_KV_NVFP4 = 1, 2, 3, 4
KV_FORMATS = {"bf16": QMV_KV_BF16, "q8_0": QMV_KV_Q8_0, "fp8": QMV_KV_FP8, "nvfp4": QMV_KV_NVFP4}
QMV_TYPE_BF16, QMV_TYPE_F32 = 1, 2

STATUS = {0: "QMV_OK", 1: "QMV_EINVAL", 2: "QMV_EALIGN", 3: "QMV_EUNSUPPORTED", 4: "QMV_ECUDA",
          5: "QMV_EHEADER", 6: "QMV_ETIMEOUT", 7: "QMV_ERANGE", 8: "QMV_EWORKSPACE"}


class QmvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({qmv_status_str(status)})")


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      f"`python block_quantized_weight_fly_gb300/build.py` (no CPU fallback exists)")

_lib = ctypes.CDLL(LIB_PATH)
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_F = ctypes.c_float


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


_canon_size = _sig("qmv_canon_size", _SZ, [_I, _I64, _I64, _I64])
_pack_size = _sig("qmv_pack_size", _SZ, [_I, _I64, _I64, _I64])
_pack = _sig("qmv_pack", _I, [_I, _P, _I64, _I64, _I64, _P, _P])
_quantize = _sig("qmv_quantize", _I, [_I, _P, _I64, _I64, _F, _P, _P])
_quantize_cb = _sig("qmv_quantize_codebook", _I, [_I, _P, _I64, _I64, _P, _P, _P])
_dequant = _sig("qmv_dequant", _I, [_I, _P, _I64, _I64, _I64, _I64, _I64, _P, _P])
_ws_size = _sig("qmv_workspace_size", _SZ, [_I, _I, _I, _I64, _I64, _I64, _I])
_gemv = _sig("qmv_gemv", _I, [_I, _P, _P, _P, _I, _I64, _I64, _P, _SZ, _P])
_gemv_swiglu = _sig("qmv_gemv_swiglu", _I, [_I, _P, _P, _P, _I, _I64, _I64, _P, _SZ, _P])
_gemv_noalloc = _sig("qmv_gemv_noalloc", _I, [_I, _P, _P, _P, _I, _I64, _I64, _P])
_grouped = _sig("qmv_grouped", _I, [_I, _P, _P, _P, _I, _P, _I, _I, _I64, _I64, _I64, _P, _SZ, _P])
_mlp_layer = _sig("qmv_mlp_layer", _I, [_I, _P, _P, _P, _P, _I, _I64, _I64, _P, _SZ, _P])
_grouped_swiglu = _sig("qmv_grouped_swiglu", _I, [_I, _P, _P, _P, _P, _I, _I, _I64, _I64, _I64, _P, _SZ, _P])
_quant_act = _sig("qmv_quant_act_nvfp4", _I, [_P, _F, _P, _P, _I, _I64, _P])
_w4a4 = _sig("qmv_gemm_nvfp4_w4a4", _I, [_P, _P, _F, _P, _I, _I64, _I64, _P, _SZ, _P])
_kquant = _sig("qmv_gemm_kquant", _I, [_I, _P, _P, _P, _I, _I64, _I64, _P, _SZ, _P])
_int8dot = _sig("qmv_gemv_int8dot", _I, [_I, _P, _P, _P, _I, _I64, _I64, _P, _SZ, _P])


class KvDesc(ctypes.Structure):
    """qmv_kv_cache of include/qmv.h."""
    _fields_ = [("fmt", _I), ("page_size", _I), ("heads", _I), ("head_dim", _I), ("pages", _I64),
                ("k_scale", _F), ("v_scale", _F), ("data", _P)]


_DESC = ctypes.POINTER(KvDesc)
_kv_size = _sig("qmv_kv_cache_size", _SZ, [_DESC])
_kv_write = _sig("qmv_kv_write", _I, [_DESC, _P, _P, _I, _I64, _I64, _I64, _I64, _P, _I64, _P])
_kv_read = _sig("qmv_kv_read", _I, [_DESC, _P, _I64, _P, _P, _I, _P])
_attn_ws = _sig("qmv_attn_workspace_size", _SZ, [_DESC, _I])
_attn = _sig("qmv_attn_paged", _I, [_DESC, _P, _I64, _P, _I64, _P, _P, _I, _I64, _I, _I, _F, _I, _I, _P, _I64, _P,
                                    _P, _SZ, _P])
_status_str = _sig("qmv_status_str", ctypes.c_char_p, [_I])
_last_route = _sig("qmv_last_route", _I, [])
_dev_status = _sig("qmv_device_status", _I, [_I])
_split_fault = _sig("qmv_debug_split_k_fault", None, [_I, ctypes.c_uint64])

EXPORTED = ["qmv_canon_size", "qmv_pack_size", "qmv_pack", "qmv_quantize", "qmv_dequant",
            "qmv_workspace_size", "qmv_gemv", "qmv_grouped", "qmv_quant_act_nvfp4",
            "qmv_gemm_nvfp4_w4a4", "qmv_status_str", "qmv_last_route", "qmv_device_status",
            "qmv_gemv_noalloc", "qmv_gemv_swiglu", "qmv_grouped_swiglu", "qmv_gemm_kquant",
            "qmv_debug_split_k_fault", "qmv_quantize_codebook", "qmv_mlp_layer", "qmv_gemv_int8dot",
            "qmv_kv_cache_size", "qmv_kv_write", "qmv_kv_read", "qmv_attn_workspace_size", "qmv_attn_paged"]


_current_device = torch._C._cuda_getDevice


def _fmt(fmt) -> int:
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    if t.is_cuda and t.get_device() != _current_device():       # the library launches on the current device
        raise ValueError(f"tensor on device {t.get_device()}, which is not the current device")
    return ctypes.c_void_p(t.data_ptr())


def _dev(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(st: int, what: str):
    if st != 0:
        raise QmvError(st, what)


def _bits16(x: torch.Tensor) -> torch.Tensor:
    if x.dtype == torch.bfloat16:
        return x
    if x.dtype in (torch.int16, torch.uint16):
        return x
    raise ValueError("x must be bf16 (or its raw 16-bit patterns)")


def _act(x: torch.Tensor, K: int, rows: int | None = None) -> tuple[torch.Tensor, int]:
    """Check an activation tensor [M, K] (or [K]) and return it with its row count.
    The library reads M * K values through a raw pointer, so a short or strided x
    is refused here rather than read out of bounds on the device."""
    x = _bits16(x)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if x.dim() == 1:
        M = 1
        if x.shape[0] != K:
            raise ValueError(f"x has {x.shape[0]} values, K = {K}")
    elif x.dim() == 2:
        M = x.shape[0]
        if x.shape[1] != K:
            raise ValueError(f"x has rows of {x.shape[1]} values, K = {K}")
    else:
        raise ValueError("x must be [M, K] or [K]")
    if rows is not None and M != rows:
        raise ValueError(f"x has {M} rows, {rows} expected")
    return x, M


def _empty(shape, dtype, dev, stream) -> torch.Tensor:
    """Memory for an output, taken on the stream that will write it: the allocator may hand out a
    block that earlier work of the stream it belongs to has yet to finish with. The current
    stream, where the caller goes on, is noted as a user of it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    if t.is_cuda:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _out(y: torch.Tensor | None, shape, dev, name: str, stream=None) -> torch.Tensor:
    """An fp32 output of `shape`: allocated if None, else checked (float32, contiguous,
    on x's device, at least as many values as the library writes)."""
    if y is None:
        return _empty(shape, torch.float32, dev, stream)
    if not y.is_cuda or y.device != torch.device(dev):
        raise ValueError(f"{name} must be a CUDA tensor on {dev}")
    if y.dtype != torch.float32:
        raise ValueError(f"{name} must be float32")
    if not y.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    need = 1
    for d in shape:
        need *= int(d)
    if y.numel() < need:
        raise ValueError(f"{name} holds {y.numel()} values, {need} needed")
    return y


# ---- entry points -------------------------------------------------------------
def qmv_status_str(status: int) -> str:
    return _status_str(int(status)).decode()


def qmv_last_route() -> int:
    return int(_last_route())


def qmv_device_status(reset: bool = True) -> int:
    return int(_dev_status(1 if reset else 0))


def qmv_debug_split_k_fault(mode: int, wait_limit_ns: int = 0) -> None:
    """Test hook of the split-K reduction (include/qmv.h): mode 1, peers publish
    nothing and reducers time out after wait_limit_ns; mode 2, reducers give up at
    once and leave their peers' partial sums behind; mode 0, normal operation."""
    _split_fault(int(mode), int(wait_limit_ns))


def qmv_canon_size(fmt, N: int, K: int, E: int = 1) -> int:
    return int(_canon_size(_fmt(fmt), N, K, E))


def qmv_pack_size(fmt, N: int, K: int, E: int = 1) -> int:
    return int(_pack_size(_fmt(fmt), N, K, E))


def qmv_workspace_size(entry: int, fmt, M: int, N: int, K: int, E: int = 1, topk: int = 1) -> int:
    return int(_ws_size(int(entry), _fmt(fmt), M, N, K, E, topk))


def qmv_pack(fmt, canon: torch.Tensor, N: int, K: int, E: int = 1, dst: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
    _dev(canon, "canon")
    size = qmv_pack_size(fmt, N, K, E)
    if size == 0:
        raise QmvError(3, "qmv_pack_size")
    if canon.numel() * canon.element_size() < qmv_canon_size(fmt, N, K, E):
        raise ValueError("canon is shorter than qmv_canon_size")
    if dst is None:
        dst = _empty(size, torch.uint8, canon.device, stream)
    elif not dst.is_cuda or not dst.is_contiguous() or dst.numel() * dst.element_size() < size:
        raise ValueError(f"dst must be a contiguous CUDA tensor of at least {size} bytes")
    _check(_pack(_fmt(fmt), _ptr(canon), N, K, E, _ptr(dst), _stream(stream)), "qmv_pack")
    return dst


def qmv_quantize(fmt, W: torch.Tensor, tensor_scale: float = 0.0, canon: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    _dev(W, "W")
    if W.dtype != torch.float32 or W.dim() != 2:
        raise ValueError("W must be a 2-D float32 tensor")
    rows, K = W.shape
    size = qmv_canon_size(fmt, rows, K, 1)
    if not W.is_contiguous():
        raise ValueError("W must be contiguous")
    if canon is None:
        canon = _empty(size, torch.uint8, W.device, stream)
    elif not canon.is_cuda or not canon.is_contiguous() or canon.numel() * canon.element_size() < size:
        raise ValueError(f"canon must be a contiguous CUDA tensor of at least {size} bytes")
    _check(_quantize(_fmt(fmt), _ptr(W), rows, K, float(tensor_scale), _ptr(canon), _stream(stream)),
           "qmv_quantize")
    return canon


def qmv_quantize_codebook(fmt, W: torch.Tensor, codebook, canon: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """The codebook formats' encoder: IQ4_XS takes 16 int8 values, IQ3_S / IQ2_S the
    grid (uint8 magnitudes, 512 x 4 / 1024 x 8) -- host sequences."""
    _dev(W, "W")
    if W.dtype != torch.float32 or W.dim() != 2 or not W.is_contiguous():
        raise ValueError("W must be a contiguous 2-D float32 tensor")
    name = fmt if isinstance(fmt, str) else next(k for k, v in FORMATS.items() if v == int(fmt))
    vals = [int(v) for v in (codebook.reshape(-1) if hasattr(codebook, "reshape") else codebook)]
    n = GRID_BYTES.get(name, 16)
    if len(vals) != n:
        raise ValueError(f"the {name} table holds {n} values")
    cb = (ctypes.c_int8 * 16)(*vals) if n == 16 else (ctypes.c_uint8 * n)(*vals)
    rows, K = W.shape
    size = qmv_canon_size(fmt, rows, K, 1)
    if canon is None:
        canon = _empty(size, torch.uint8, W.device, stream)
    elif not canon.is_cuda or not canon.is_contiguous() or canon.numel() * canon.element_size() < size:
        raise ValueError(f"canon must be a contiguous CUDA tensor of at least {size} bytes")
    _check(_quantize_cb(_fmt(fmt), _ptr(W), rows, K, ctypes.cast(cb, ctypes.c_void_p), _ptr(canon),
                        _stream(stream)), "qmv_quantize_codebook")
    return canon


def qmv_dequant(fmt, packed: torch.Tensor, N: int, K: int, E: int = 1, row0: int = 0,
                rows: int | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _dev(packed, "packed")
    rows = N * E - row0 if rows is None else rows
    out = _out(out, (rows, K), packed.device, "out", stream)
    _check(_dequant(_fmt(fmt), _ptr(packed), N, K, E, row0, rows, _ptr(out), _stream(stream)),
           "qmv_dequant")
    return out


def workspace(entry: int, fmt, M: int, N: int, K: int, E: int = 1, topk: int = 1,
              device="cuda") -> torch.Tensor:
    """A zero-filled workspace of the size the entry point needs."""
    size = qmv_workspace_size(entry, fmt, M, N, K, E, topk)
    if size == 0:
        raise QmvError(1, "qmv_workspace_size")
    return torch.zeros(size, dtype=torch.uint8, device=device)


def qmv_gemv(fmt, packed_W: torch.Tensor, x: torch.Tensor, N: int, K: int,
             ws: torch.Tensor, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _dev(packed_W, "packed_W"); _dev(x, "x"); _dev(ws, "ws")
    x, M = _act(x, K)
    y = _out(y, (M, N), x.device, "y", stream)
    _check(_gemv(_fmt(fmt), _ptr(packed_W), _ptr(x), _ptr(y), M, N, K, _ptr(ws), ws.numel(),
                 _stream(stream)), "qmv_gemv")
    return y


def qmv_gemv_swiglu(fmt, tower: torch.Tensor, x: torch.Tensor, N: int, K: int, ws: torch.Tensor,
                    h: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h = silu(gate . x) * (up . x) over a 2-expert tower (gate = expert 0, up = expert 1)."""
    _dev(tower, "tower"); _dev(x, "x"); _dev(ws, "ws")
    x, M = _act(x, K)
    h = _out(h, (M, N), x.device, "h", stream)
    _check(_gemv_swiglu(_fmt(fmt), _ptr(tower), _ptr(x), _ptr(h), M, N, K, _ptr(ws), ws.numel(),
                        _stream(stream)), "qmv_gemv_swiglu")
    return h


def qmv_mlp_layer(fmt, gateup: torch.Tensor, down: torch.Tensor, x: torch.Tensor, N_ff: int, K_h: int,
                  ws: torch.Tensor, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = bf16(silu(x Wg^T) * (x Wu^T)) Wd^T in one launch: gateup = the 2-matrix
    [N_ff, K_h] tower (gate, up), down = the [K_h, N_ff] matrix."""
    _dev(gateup, "gateup"); _dev(down, "down"); _dev(x, "x"); _dev(ws, "ws")
    x, M = _act(x, K_h)
    y = _out(y, (M, K_h), x.device, "y", stream)
    _check(_mlp_layer(_fmt(fmt), _ptr(gateup), _ptr(down), _ptr(x), _ptr(y), M, N_ff, K_h, _ptr(ws), ws.numel(),
                      _stream(stream)), "qmv_mlp_layer")
    return y


def qmv_gemv_noalloc(fmt, packed_W: torch.Tensor, x: torch.Tensor, N: int, K: int,
                     y: torch.Tensor, stream=None) -> torch.Tensor:
    """qmv_gemv with the library's built-in scratch instead of a workspace. y is
    required (the caller owns every buffer); nothing is allocated."""
    _dev(packed_W, "packed_W"); _dev(x, "x"); _dev(y, "y")
    x, M = _act(x, K)
    y = _out(y, (M, N), x.device, "y", stream)
    _check(_gemv_noalloc(_fmt(fmt), _ptr(packed_W), _ptr(x), _ptr(y), M, N, K, _stream(stream)),
           "qmv_gemv_noalloc")
    return y


def qmv_grouped(fmt, tower: torch.Tensor, expert_ids: torch.Tensor, x: torch.Tensor, N: int, K: int,
                E: int, ws: torch.Tensor, x_per_pair: bool = False, y: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    _dev(tower, "tower"); _dev(expert_ids, "expert_ids"); _dev(x, "x"); _dev(ws, "ws")
    if expert_ids.dtype != torch.int32 or expert_ids.dim() != 2:
        raise ValueError("expert_ids must be int32 [M, topk]")
    if not expert_ids.is_contiguous():
        raise ValueError("expert_ids must be contiguous")
    M, topk = expert_ids.shape
    x, _ = _act(x, K, M * topk if x_per_pair else M)
    y = _out(y, (M, topk, N), x.device, "y", stream)
    _check(_grouped(_fmt(fmt), _ptr(tower), _ptr(expert_ids), _ptr(x), 1 if x_per_pair else 0, _ptr(y),
                    M, topk, N, K, E, _ptr(ws), ws.numel(), _stream(stream)), "qmv_grouped")
    return y


def qmv_grouped_swiglu(fmt, tower: torch.Tensor, expert_ids: torch.Tensor, x: torch.Tensor, N: int,
                       K: int, E: int, ws: torch.Tensor, h: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """h[t, j] = silu(gate_e . x[t]) * (up_e . x[t]), e = expert_ids[t, j], over a
    2E-expert tower (gate matrices 0..E-1, then up matrices E..2E-1)."""
    _dev(tower, "tower"); _dev(expert_ids, "expert_ids"); _dev(x, "x"); _dev(ws, "ws")
    if expert_ids.dtype != torch.int32 or expert_ids.dim() != 2:
        raise ValueError("expert_ids must be int32 [M, topk]")
    if not expert_ids.is_contiguous():
        raise ValueError("expert_ids must be contiguous")
    M, topk = expert_ids.shape
    x, _ = _act(x, K, M)
    h = _out(h, (M, topk, N), x.device, "h", stream)
    _check(_grouped_swiglu(_fmt(fmt), _ptr(tower), _ptr(expert_ids), _ptr(x), _ptr(h), M, topk, N, K, E,
                           _ptr(ws), ws.numel(), _stream(stream)), "qmv_grouped_swiglu")
    return h


def qmv_quant_act_nvfp4(x: torch.Tensor, x_scale: float, codes: torch.Tensor | None = None,
                        scales: torch.Tensor | None = None, stream=None):
    _dev(x, "x")
    x = _bits16(x)
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous [M, K] tensor")
    M, K = x.shape
    for t, n, name in ((codes, M * (K // 2), "codes"), (scales, M * (K // 16), "scales")):
        if t is not None and (t.dtype != torch.uint8 or not t.is_contiguous() or t.numel() < n or not t.is_cuda):
            raise ValueError(f"{name} must be a contiguous CUDA uint8 tensor of at least {n} bytes")
    if codes is None:
        codes = _empty((M, K // 2), torch.uint8, x.device, stream)
    if scales is None:
        scales = _empty((M, K // 16), torch.uint8, x.device, stream)
    _check(_quant_act(_ptr(x), float(x_scale), _ptr(codes), _ptr(scales), M, K, _stream(stream)),
           "qmv_quant_act_nvfp4")
    return codes, scales


def qmv_gemm_nvfp4_w4a4(packed_W: torch.Tensor, x: torch.Tensor, x_scale: float, N: int, K: int,
                        ws: torch.Tensor, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _dev(packed_W, "packed_W"); _dev(x, "x"); _dev(ws, "ws")
    x, M = _act(x, K)
    y = _out(y, (M, N), x.device, "y", stream)
    _check(_w4a4(_ptr(packed_W), _ptr(x), float(x_scale), _ptr(y), M, N, K, _ptr(ws), ws.numel(),
                 _stream(stream)), "qmv_gemm_nvfp4_w4a4")
    return y


def qmv_gemm_kquant(fmt, packed_W: torch.Tensor, x: torch.Tensor, N: int, K: int, ws: torch.Tensor,
                    y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = x . W^T for a K-quant W at prefill sizes (tensor cores, each weight read once)."""
    _dev(packed_W, "packed_W"); _dev(x, "x"); _dev(ws, "ws")
    x, M = _act(x, K)
    y = _out(y, (M, N), x.device, "y", stream)
    _check(_kquant(_fmt(fmt), _ptr(packed_W), _ptr(x), _ptr(y), M, N, K, _ptr(ws), ws.numel(), _stream(stream)),
           "qmv_gemm_kquant")
    return y


def qmv_gemv_int8dot(fmt, packed_W: torch.Tensor, x: torch.Tensor, N: int, K: int, ws: torch.Tensor,
                     y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = q8(x) . W^T: x quantized to int8 per 32 values, integer dots (Q8_0, Q4_K; M <= 8)."""
    _dev(packed_W, "packed_W"); _dev(x, "x"); _dev(ws, "ws")
    x, M = _act(x, K)
    y = _out(y, (M, N), x.device, "y", stream)
    _check(_int8dot(_fmt(fmt), _ptr(packed_W), _ptr(x), _ptr(y), M, N, K, _ptr(ws), ws.numel(), _stream(stream)),
           "qmv_gemv_int8dot")
    return y


# ---- the paged KV cache and its attention ---------------------------------------
# These calls take single-digit microseconds on the device, so their checks are kept
# lean: plain integers to ctypes, one stream look-up, one descriptor reference per cache.
_raw_stream = torch._C._cuda_getCurrentRawStream
_KV_TYPES = {torch.bfloat16: QMV_TYPE_BF16, torch.float32: QMV_TYPE_F32}


def _int32(x, name: str) -> int:
    """ctypes passes the low 32 bits of a larger number without a word."""
    x = operator.index(x)
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError(f"{name} = {x} does not fit 32 bits")
    return x


class KvCache:
    """One layer's paged cache: its device buffer (`data`, uint8) and its descriptor (`desc`)."""

    def __init__(self, fmt, pages: int, page_size: int, heads: int, head_dim: int, k_scale: float = 1.0,
                 v_scale: float = 1.0, device="cuda", data: torch.Tensor | None = None):
        f = KV_FORMATS[fmt] if isinstance(fmt, str) else int(fmt)
        if not -(1 << 63) <= operator.index(pages) < 1 << 63:
            raise ValueError(f"pages = {pages} does not fit 64 bits")
        self.desc = KvDesc(_int32(f, "fmt"), _int32(page_size, "page_size"), _int32(heads, "heads"),
                           _int32(head_dim, "head_dim"), pages, k_scale, v_scale, None)
        self.ref = ctypes.byref(self.desc)
        self.heads, self.head_dim = heads, head_dim
        size = qmv_kv_cache_size(self)
        if size == 0:
            raise QmvError(3, "qmv_kv_cache_size")
        if data is None:
            data = torch.zeros(size, dtype=torch.uint8, device=device)
        elif not data.is_cuda or not data.is_contiguous() or data.numel() * data.element_size() < size:
            raise ValueError(f"data must be a contiguous CUDA tensor of at least {size} bytes")
        self.data = data
        self.index, self.device = data.get_device(), data.device
        self.desc.data = data.data_ptr()

    def _check_device(self) -> None:
        """The library launches, and counts SMs, on the current device."""
        if _current_device() != self.index:
            raise ValueError(f"the cache is on device {self.index}, which is not the current device")

    def _stream(self, stream) -> int:
        self._check_device()
        if stream is None:
            return _raw_stream(self.index)
        if stream.device_index != self.index:
            raise ValueError("stream must be on the cache's device")
        return stream.cuda_stream


def kv_cache(fmt, pages: int, page_size: int, heads: int, head_dim: int, k_scale: float = 1.0,
             v_scale: float = 1.0, device="cuda") -> KvCache:
    """A zero-filled cache of `pages` pages of page_size tokens for `heads` heads of head_dim values."""
    return KvCache(fmt, pages, page_size, heads, head_dim, k_scale, v_scale, device)


def attn_workspace(cache: KvCache, q_heads: int) -> torch.Tensor:
    """A zero-filled workspace of the size qmv_attn_paged needs."""
    size = qmv_attn_workspace_size(cache, q_heads)
    if size == 0:
        raise QmvError(1, "qmv_attn_workspace_size")
    return torch.zeros(size, dtype=torch.uint8, device=cache.data.device)


def _kv_rows(x: torch.Tensor, cache: KvCache, name: str):
    """Check rows [T, heads, head_dim] of any token and head strides; (T, token stride, head stride)."""
    if x.dim() != 3:
        raise ValueError(f"{name} must be [T, {cache.heads}, {cache.head_dim}]")
    T, H, D = x.shape
    st, sh, sd = x.stride()
    if H != cache.heads or D != cache.head_dim:
        raise ValueError(f"{name} must be [T, {cache.heads}, {cache.head_dim}]")
    if x.dtype not in _KV_TYPES:
        raise ValueError(f"{name} must be bfloat16 or float32")
    if x.get_device() != cache.index:
        raise ValueError(f"{name} must be on the cache's device")
    if sd != 1:
        raise ValueError(f"the values of {name}'s rows must be contiguous")
    return T, st, sh


def _index(t: torch.Tensor, shape: tuple, dtype, cache: KvCache, name: str) -> int:
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != cache.index:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on the cache's device")
    return t.data_ptr()


def qmv_kv_cache_size(cache: KvCache) -> int:
    return int(_kv_size(cache.ref))


def qmv_attn_workspace_size(cache: KvCache, q_heads: int) -> int:
    cache._check_device()
    return int(_attn_ws(cache.ref, _int32(q_heads, "q_heads")))


def qmv_kv_write(cache: KvCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
    """Quantize K and V rows [T, heads, head_dim] (bf16 or fp32, strided) into slots [T] (int64;
    page * page_size + offset, negative: skip)."""
    T, kt, kh = _kv_rows(k, cache, "k")
    Tv, vt, vh = _kv_rows(v, cache, "v")
    if k.dtype != v.dtype or T != Tv:
        raise ValueError("k and v must have the same type and number of tokens")
    st = _kv_write(cache.ref, k.data_ptr(), v.data_ptr(), _KV_TYPES[k.dtype], kt, kh, vt, vh,
                   _index(slots, (T,), torch.int64, cache, "slots"), T, cache._stream(stream))
    if st:
        raise QmvError(st, "qmv_kv_write")


def qmv_kv_read(cache: KvCache, slots: torch.Tensor, dtype=torch.bfloat16, k: torch.Tensor | None = None,
                v: torch.Tensor | None = None, stream=None):
    """The K and V values [T, heads, head_dim] that slots [T] hold, as bf16 or fp32."""
    if dtype not in _KV_TYPES:
        raise ValueError("dtype must be bfloat16 or float32")
    T = slots.shape[0]
    ps = _index(slots, (T,), torch.int64, cache, "slots")
    shape = (T, cache.heads, cache.head_dim)
    pk = _index(k, shape, dtype, cache, "k") if k is not None else 0
    pv = _index(v, shape, dtype, cache, "v") if v is not None else 0
    if not pk:
        k = _empty(shape, dtype, cache.device, stream)
        pk = k.data_ptr()
    if not pv:
        v = _empty(shape, dtype, cache.device, stream)
        pv = v.data_ptr()
    st = _kv_read(cache.ref, ps, T, pk, pv, _KV_TYPES[dtype], cache._stream(stream))
    if st:
        raise QmvError(st, "qmv_kv_read")
    return k, v


def qmv_attn_paged(cache: KvCache, q: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor,
                   q_start: torch.Tensor, max_q: int, ws: torch.Tensor, scale: float | None = None,
                   causal: bool = True, window: int = 0, out: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of q [T, q_heads, head_dim] (bf16; sequence b's queries are rows q_start[b] ..
    q_start[b+1]-1, its last new tokens) over the cached keys and values of page_table [B, max_pages],
    kv_len [B] (int32). scale: 1 / sqrt(head_dim) if None. lse: fp32 [T, q_heads] or None."""
    D = cache.head_dim
    if q.dim() != 3 or q.shape[2] != D or q.dtype != torch.bfloat16 or q.get_device() != cache.index:
        raise ValueError(f"q must be a bfloat16 tensor [T, q_heads, {D}] on the cache's device")
    T, H, _ = q.shape
    if out is None:
        out = _empty((T, H, D), torch.bfloat16, cache.device, stream)
    elif out.dtype != torch.bfloat16 or out.shape != q.shape or out.get_device() != cache.index:
        raise ValueError("out must be bfloat16, of q's shape, on its device")
    qs, os = q.stride(), out.stride()
    if qs[2] != 1 or os[2] != 1 or (H > 1 and (qs[1] != D or os[1] != D)):
        raise ValueError("the heads of a token of q and of out must be contiguous")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B, P = page_table.shape
    if ws.get_device() != cache.index or not ws.is_contiguous():
        raise ValueError("ws must be contiguous and on the cache's device")
    st = _attn(cache.ref, q.data_ptr(), qs[0], _index(page_table, (B, P), torch.int32, cache, "page_table"), P,
               _index(kv_len, (B,), torch.int32, cache, "kv_len"),
               _index(q_start, (B + 1,), torch.int32, cache, "q_start"), B, T, _int32(max_q, "max_q"), H,
               D ** -0.5 if scale is None else scale, 1 if causal else 0, _int32(window, "window"), out.data_ptr(), os[0],
               None if lse is None else _index(lse, (T, H), torch.float32, cache, "lse"), ws.data_ptr(),
               ws.numel() * ws.element_size(), cache._stream(stream))
    if st:
        raise QmvError(st, "qmv_attn_paged")
    return out
