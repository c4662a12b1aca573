"""Python binding of the mxmoe C ABI (include/mxmoe.h): MXFP4 weight-streaming MoE layer,
dense MXFP4 linear layer and dense feed-forward operators with their gradients for MI355X
(gfx950).

Argument marshalling only: every step of the computation runs in the HIP kernels of
libmxmoe.so.  PyTorch provides device memory and the current stream.  If the library is
not built, importing this package raises: there is no fallback path.

bf16 tensors are passed as their bit patterns; MXFP4 weights are uint8 code tensors
[..., rows, K/2] (element 2i in the low nibble) plus uint8 E8M0 scale tensors
[..., rows, K/32].
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxmoe.so")

MX_OK = 0
MX_MAX_TOKENS = 256
MX_MAX_EXPERTS = 1024
MX_MAX_TOPK = 32

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run `python mxfp4_weight_moe_amd/build.py` (hipcc, gfx950) first")

_lib = ctypes.CDLL(LIB_PATH)
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_lib.mx_version.restype = ctypes.c_int
_lib.mx_status_string.restype = ctypes.c_char_p
_lib.mx_status_string.argtypes = [ctypes.c_int]
_lib.mx_linear.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, _P]
_lib.mxfp4_dequantize.argtypes = [_P, _P, _I64, _I64, _P, _P]
_lib.moe_route_topk.argtypes = [_P, _I64, _I64, _I64, _P, _P, _P]
_lib.moe_sort_by_expert.argtypes = [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P]
_lib.moe_route_sort.argtypes = [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P]
_lib.moe_gate_up_swiglu.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _P,
                                    ctypes.c_size_t, _P]
_lib.moe_gate_up_swiglu_from_ids.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _P,
                                             ctypes.c_size_t, _P]
_lib.moe_down_combine.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _P,
                                  ctypes.c_size_t, _P]
_lib.moe_expert_gemms_from_ids.argtypes = [_P, _P, _P, _P, _P, _P, _P, ctypes.c_int, _P, _I64, _I64, _I64, _I64,
                                           _I64, _P, ctypes.c_size_t, _P]
_lib.moe_combine.argtypes = [_P, _P, _P, _I64, _I64, _I64, _P]
_lib.moe_mxfp4_workspace_size.restype = ctypes.c_size_t
_lib.moe_mxfp4_workspace_size.argtypes = [_I64, _I64, _I64, _I64, _I64]
_lib.moe_mxfp4_forward.argtypes = [_P, _P, _I64, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P, ctypes.c_size_t, _P]
_lib.moe_mxfp4_forward_persistent.argtypes = list(_lib.moe_mxfp4_forward.argtypes)
_lib.moe_mxfp4_forward_shared.argtypes = [_P, _P, _I64, _I64, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P,
                                          ctypes.c_size_t, _P]
_lib.moe_mxfp4_forward_a8.argtypes = list(_lib.moe_mxfp4_forward_shared.argtypes)
_lib.mx_linear_a8.argtypes = list(_lib.mx_linear.argtypes)
_lib.mxfp8_quantize.argtypes = [_P, _I64, _I64, _P, _P, _P]
_lib.moe_mxfp4_forward_noalloc.argtypes = [_P, _P, _I64, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P]
_lib.mx_hbm_read.argtypes = [_P, ctypes.c_size_t, _P, _P]
_lib.mx_hbm_copy.argtypes = [_P, _P, ctypes.c_size_t, _P]
_SZ = ctypes.c_size_t
_F = ctypes.c_float
_INT = ctypes.c_int
_lib.mx_linear_fused.argtypes = [_P, _P, _P, _P, _P, _F, _INT, _P, _P, _I64, _I64, _I64, _P, _SZ, _P]
_lib.mx_linear_fused_backward.argtypes = [_P, _P, _P, _P, _F, _INT, _P, _P, _I64, _I64, _I64, _P, _SZ, _P]
_lib.mx_gate_up.argtypes = [_P, _P, _P, _P, _INT, _P, _P, _I64, _I64, _I64, _P, _SZ, _P]
_lib.mx_gate_up_backward.argtypes = [_P, _P, _P, _P, _INT, _P, _P, _I64, _I64, _I64, _P, _SZ, _P]
_lib.mx_norm_residual.argtypes = [_P, _P, _P, _P, _INT, _F, _P, _F, _P, _P, _I64, _I64, _P]
_lib.mx_norm_residual_backward.argtypes = [_P, _P, _P, _P, _P, _P, _INT, _F, _P, _F, _P, _P, _P, _P, _P, _I64, _I64,
                                           _P, _SZ, _P]
_lib.mx_ffn_block.argtypes = [_P, _P, _P, _P, _P, _INT, _P, _P, _P, _P, _P, _INT, _F, _F, _P, _I64, _I64, _I64, _P,
                              _SZ, _P]
_FFN_SIZES = ("mx_linear_fused_workspace_size", "mx_linear_fused_backward_workspace_size",
              "mx_gate_up_workspace_size", "mx_gate_up_backward_workspace_size", "mx_ffn_block_workspace_size",
              "mx_norm_residual_backward_workspace_size")
_FFN_CALLS = ("mx_linear_fused", "mx_linear_fused_backward", "mx_gate_up", "mx_gate_up_backward", "mx_norm_residual",
              "mx_norm_residual_backward", "mx_ffn_block")
for _n in _FFN_SIZES:
    getattr(_lib, _n).restype = _SZ
    getattr(_lib, _n).argtypes = [_I64] * (2 if "norm" in _n else 3)
for _n in _FFN_CALLS:
    getattr(_lib, _n).restype = ctypes.c_int
for _n in ("mx_linear", "mxfp4_dequantize", "moe_route_topk", "moe_sort_by_expert", "moe_route_sort",
           "moe_gate_up_swiglu", "moe_down_combine", "moe_mxfp4_forward", "moe_mxfp4_forward_persistent",
           "moe_mxfp4_forward_shared", "moe_mxfp4_forward_a8", "mx_linear_a8", "mxfp8_quantize", "mx_hbm_read",
           "mx_hbm_copy", "moe_mxfp4_forward_noalloc", "moe_gate_up_swiglu_from_ids", "moe_expert_gemms_from_ids",
           "moe_combine"):
    getattr(_lib, _n).restype = ctypes.c_int

EXPORTED = ("mx_version", "mx_status_string", "mx_linear", "mxfp4_dequantize", "moe_route_topk",
            "moe_sort_by_expert", "moe_route_sort", "moe_gate_up_swiglu", "moe_down_combine",
            "moe_mxfp4_workspace_size", "moe_mxfp4_forward", "moe_mxfp4_forward_persistent",
            "moe_mxfp4_forward_shared", "moe_mxfp4_forward_a8", "mx_linear_a8", "mxfp8_quantize", "mx_hbm_read",
            "mx_hbm_copy", "moe_mxfp4_forward_noalloc", "moe_gate_up_swiglu_from_ids", "moe_expert_gemms_from_ids",
            "moe_combine") + _FFN_CALLS + _FFN_SIZES
MX_ERR_SCRATCH = -6
MX_NOALLOC_SCRATCH_BYTES = 40 << 20


class MxError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call} failed: {status_string(status)} (status {status})")


def version() -> int:
    return _lib.mx_version()


def status_string(status: int) -> str:
    return _lib.mx_status_string(int(status)).decode()


def raw():
    """The ctypes handle of libmxmoe.so (for tests that call the C ABI directly)."""
    return _lib


def _ptr(t: torch.Tensor):
    return ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(t: torch.Tensor, name: str, dtype, ndim=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def _raise(status: int, call: str):
    if status != MX_OK:
        if status in (-2, -7):  # MX_ERR_SHAPE, MX_ERR_ARG
            raise ValueError(f"{call}: {status_string(status)}")
        raise MxError(status, call)


def mx_linear(x: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
              out: torch.Tensor | None = None, act8: bool = False) -> torch.Tensor:
    """y[T,N] = bf16(x[T,K] @ dequant(w)[N,K]^T), fp32 accumulation.
    act8=True: x quantized to MXFP8 first, scaled MFMA (mx_linear_a8)."""
    _check(x, "x", torch.bfloat16, 2)
    dev = x.device
    _check(w_codes, "w_codes", torch.uint8, 2, dev)
    _check(w_scales, "w_scales", torch.uint8, 2, dev)
    T, K = x.shape
    N = w_codes.shape[0]
    if w_codes.shape != (N, K // 2) or w_scales.shape != (N, K // 32) or K % 32:
        raise ValueError(f"weight shapes {tuple(w_codes.shape)}, {tuple(w_scales.shape)} do not match K={K}")
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
    _check(out, "out", torch.bfloat16, 2, dev)
    if out.shape != (T, N):
        raise ValueError("out has the wrong shape")
    name = "mx_linear_a8" if act8 else "mx_linear"
    st = getattr(_lib, name)(_ptr(x), _ptr(w_codes), _ptr(w_scales), _ptr(out), T, K, N, _stream(dev))
    _raise(st, name)
    return out


def hbm_read(src: torch.Tensor, xor_out: torch.Tensor | None = None, clear: bool = True) -> torch.Tensor:
    """HBM reference read of a contiguous device tensor (size a multiple of 16 bytes):
    returns int32 [4], word c = XOR of 32-bit word c of every 16-byte piece (XORed into
    xor_out, which is zeroed first unless clear=False)."""
    if not src.is_cuda or not src.is_contiguous():
        raise ValueError("src must be a contiguous device tensor")
    dev = src.device
    if xor_out is None:
        xor_out = torch.zeros(4, dtype=torch.int32, device=dev)
    else:
        _check(xor_out, "xor_out", torch.int32, 1, dev)
        if clear:
            xor_out.zero_()
    nbytes = src.numel() * src.element_size()
    st = _lib.mx_hbm_read(_ptr(src), nbytes, _ptr(xor_out), _stream(dev))
    _raise(st, "mx_hbm_read")
    return xor_out


def hbm_copy(dst: torch.Tensor, src: torch.Tensor) -> torch.Tensor:
    """HBM reference copy between two contiguous device tensors of the same byte size."""
    for t, n in ((dst, "dst"), (src, "src")):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous device tensor")
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes or dst.device != src.device:
        raise ValueError("dst and src must have the same byte size and device")
    st = _lib.mx_hbm_copy(_ptr(dst), _ptr(src), nbytes, _stream(src.device))
    _raise(st, "mx_hbm_copy")
    return dst


def mxfp8_quantize(x: torch.Tensor):
    """MXFP8 (E4M3 codes, E8M0 scales per 32) of bf16 rows: (codes uint8 [R, K], scales uint8 [R, K/32])."""
    _check(x, "x", torch.bfloat16, 2)
    dev = x.device
    R, K = x.shape
    if K % 32:
        raise ValueError("K must be a multiple of 32")
    codes = torch.empty((R, K), dtype=torch.uint8, device=dev)
    scales = torch.empty((R, K // 32), dtype=torch.uint8, device=dev)
    st = _lib.mxfp8_quantize(_ptr(x), R, K, _ptr(codes), _ptr(scales), _stream(dev))
    _raise(st, "mxfp8_quantize")
    return codes, scales


def mxfp4_dequantize(w_codes: torch.Tensor, w_scales: torch.Tensor) -> torch.Tensor:
    """bf16 [rows, K] = E2M1(code) * 2^(s - 127), exact."""
    _check(w_codes, "w_codes", torch.uint8)
    dev = w_codes.device
    _check(w_scales, "w_scales", torch.uint8, None, dev)
    K = w_codes.shape[-1] * 2
    rows = w_codes.numel() // (K // 2)
    if w_scales.numel() != rows * (K // 32) or w_scales.shape[:-1] != w_codes.shape[:-1]:
        raise ValueError("scale tensor does not match the code tensor")
    out = torch.empty((*w_codes.shape[:-1], K), dtype=torch.bfloat16, device=dev)
    st = _lib.mxfp4_dequantize(_ptr(w_codes), _ptr(w_scales), rows, K, _ptr(out), _stream(dev))
    _raise(st, "mxfp4_dequantize")
    return out


def moe_route_topk(logits: torch.Tensor, top_k: int, ids: torch.Tensor | None = None,
                   gates: torch.Tensor | None = None):
    """(ids int32 [T,k], gates fp32 [T,k]): top-k logits (ties to lower id), softmax over them."""
    _check(logits, "router_logits", torch.float32, 2)
    dev = logits.device
    T, E = logits.shape
    if ids is None:
        ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    if gates is None:
        gates = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    _check(ids, "ids", torch.int32, 2, dev)
    _check(gates, "gates", torch.float32, 2, dev)
    if ids.shape != (T, top_k) or gates.shape != (T, top_k):
        raise ValueError("ids / gates must be [T, top_k]")
    st = _lib.moe_route_topk(_ptr(logits), T, E, top_k, _ptr(ids), _ptr(gates), _stream(dev))
    _raise(st, "moe_route_topk")
    return ids, gates


_SORT_KEYS = ("counts", "offsets", "sorted_slots", "active", "num_active")


def _sort_ptrs(sort: dict, dev):
    for key in _SORT_KEYS:
        _check(sort[key], key, torch.int32, 1, dev)
    return [_ptr(sort[key]) for key in _SORT_KEYS]


def _sort_out(out: dict | None, T: int, k: int, E: int, dev) -> dict:
    if out is not None:
        _sort_ptrs(out, dev)
        if (out["counts"].numel() != E or out["offsets"].numel() != E + 1 or out["sorted_slots"].numel() != T * k
                or out["active"].numel() != E or out["num_active"].numel() != 2):
            raise ValueError("sort output tensors have the wrong sizes")
        return out
    return dict(
        counts=torch.empty(E, dtype=torch.int32, device=dev),
        offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
        sorted_slots=torch.empty(T * k, dtype=torch.int32, device=dev),
        active=torch.empty(E, dtype=torch.int32, device=dev),
        num_active=torch.empty(2, dtype=torch.int32, device=dev),
    )


def moe_sort_by_expert(ids: torch.Tensor, num_experts: int, out: dict | None = None) -> dict:
    """Counting sort of the flat slots by expert (experts ascending, slot ascending)."""
    _check(ids, "ids", torch.int32, 2)
    dev = ids.device
    T, k = ids.shape
    E = int(num_experts)
    out = _sort_out(out, T, k, E, dev)
    st = _lib.moe_sort_by_expert(_ptr(ids), T, k, E, _ptr(out["counts"]), _ptr(out["offsets"]),
                                 _ptr(out["sorted_slots"]), _ptr(out["active"]), _ptr(out["num_active"]),
                                 _stream(dev))
    _raise(st, "moe_sort_by_expert")
    return out


def moe_route_sort(logits: torch.Tensor, top_k: int, ids: torch.Tensor | None = None,
                   gates: torch.Tensor | None = None, out: dict | None = None):
    """moe_route_topk then moe_sort_by_expert in one launch: (ids, gates, sort dict)."""
    _check(logits, "router_logits", torch.float32, 2)
    dev = logits.device
    T, E = logits.shape
    if ids is None:
        ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    if gates is None:
        gates = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    _check(ids, "ids", torch.int32, 2, dev)
    _check(gates, "gates", torch.float32, 2, dev)
    if ids.shape != (T, top_k) or gates.shape != (T, top_k):
        raise ValueError("ids / gates must be [T, top_k]")
    out = _sort_out(out, T, top_k, E, dev)
    st = _lib.moe_route_sort(_ptr(logits), T, E, top_k, _ptr(ids), _ptr(gates), *[_ptr(out[key]) for key in _SORT_KEYS],
                             _stream(dev))
    _raise(st, "moe_route_sort")
    return ids, gates, out


def moe_gate_up_swiglu(x: torch.Tensor, W_gate_up: torch.Tensor, S_gate_up: torch.Tensor, sort: dict, top_k: int,
                       h: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Stage hook: h [T*k, I] bf16 (rows in sorted-slot order) from a moe_sort_by_expert result."""
    _check(x, "x", torch.bfloat16, 2)
    dev = x.device
    _check(W_gate_up, "W_gate_up", torch.uint8, 3, dev)
    _check(S_gate_up, "S_gate_up", torch.uint8, 3, dev)
    T, H = x.shape
    E, two_i, _ = W_gate_up.shape
    I = two_i // 2
    if W_gate_up.shape != (E, 2 * I, H // 2) or S_gate_up.shape != (E, 2 * I, H // 32):
        raise ValueError("W_gate_up / S_gate_up shapes do not match [E, 2I, H/2] / [E, 2I, H/32]")
    if h is None:
        h = torch.empty((T * top_k, I), dtype=torch.bfloat16, device=dev)
    _check(h, "h", torch.bfloat16, 2, dev)
    if ws is None:
        ws = workspace(T, H, I, E, top_k, dev)
    _check(ws, "workspace", torch.uint8, 1, dev)
    st = _lib.moe_gate_up_swiglu(_ptr(x), _ptr(W_gate_up), _ptr(S_gate_up), *_sort_ptrs(sort, dev), _ptr(h), T, H, I,
                                 E, top_k, _ptr(ws), ws.numel(), _stream(dev))
    _raise(st, "moe_gate_up_swiglu")
    return h


def moe_gate_up_swiglu_from_ids(x: torch.Tensor, ids: torch.Tensor, W_gate_up: torch.Tensor, S_gate_up: torch.Tensor,
                                h: torch.Tensor | None = None, sort: dict | None = None,
                                ws: torch.Tensor | None = None):
    """Stage hook for T <= 32: (h [T*k, I] bf16, sort dict) from the routed ids, the slots
    sorted inside the gate_up launch (the sort equals moe_sort_by_expert's)."""
    _check(x, "x", torch.bfloat16, 2)
    dev = x.device
    _check(ids, "ids", torch.int32, 2, dev)
    _check(W_gate_up, "W_gate_up", torch.uint8, 3, dev)
    _check(S_gate_up, "S_gate_up", torch.uint8, 3, dev)
    T, H = x.shape
    top_k = ids.shape[1]
    E, two_i, _ = W_gate_up.shape
    I = two_i // 2
    if ids.shape[0] != T:
        raise ValueError("ids must be [T, top_k]")
    if W_gate_up.shape != (E, 2 * I, H // 2) or S_gate_up.shape != (E, 2 * I, H // 32):
        raise ValueError("W_gate_up / S_gate_up shapes do not match [E, 2I, H/2] / [E, 2I, H/32]")
    sort = _sort_out(sort, T, top_k, E, dev)
    if h is None:
        h = torch.empty((T * top_k, I), dtype=torch.bfloat16, device=dev)
    _check(h, "h", torch.bfloat16, 2, dev)
    if ws is None:
        ws = workspace(T, H, I, E, top_k, dev)
    _check(ws, "workspace", torch.uint8, 1, dev)
    st = _lib.moe_gate_up_swiglu_from_ids(_ptr(x), _ptr(ids), _ptr(W_gate_up), _ptr(S_gate_up),
                                          *[_ptr(sort[key]) for key in _SORT_KEYS], _ptr(h), T, H, I, E, top_k,
                                          _ptr(ws), ws.numel(), _stream(dev))
    _raise(st, "moe_gate_up_swiglu_from_ids")
    return h, sort


def moe_expert_gemms_from_ids(x: torch.Tensor, ids: torch.Tensor, W_gate_up: torch.Tensor, S_gate_up: torch.Tensor,
                              W_down: torch.Tensor, S_down: torch.Tensor, h: torch.Tensor | None = None,
                              d: torch.Tensor | None = None, ws: torch.Tensor | None = None, fill_h: bool = True):
    """Stage hook for T <= 32: both expert GEMMs in one launch from the routed ids:
    (h [T*k, I] bf16 in sorted-slot order, d [T*k, H] fp32 down outputs by flat slot).
    The launch needs every element of h at 0xFFFF when it starts: fill_h=True has the call
    fill it first (one more launch); with fill_h=False the caller has done so on this stream."""
    _check(x, "x", torch.bfloat16, 2)
    dev = x.device
    _check(ids, "ids", torch.int32, 2, dev)
    for t, n in ((W_gate_up, "W_gate_up"), (S_gate_up, "S_gate_up"), (W_down, "W_down"), (S_down, "S_down")):
        _check(t, n, torch.uint8, 3, dev)
    T, H = x.shape
    top_k = ids.shape[1]
    E = W_gate_up.shape[0]
    I = W_down.shape[2] * 2
    if ids.shape[0] != T:
        raise ValueError("ids must be [T, top_k]")
    if (W_gate_up.shape != (E, 2 * I, H // 2) or S_gate_up.shape != (E, 2 * I, H // 32)
            or W_down.shape != (E, H, I // 2) or S_down.shape != (E, H, I // 32)):
        raise ValueError("expert weight shapes do not match [E, 2I, H/2], [E, 2I, H/32], [E, H, I/2], [E, H, I/32]")
    if h is None:
        h = torch.empty((T * top_k, I), dtype=torch.bfloat16, device=dev)
    if d is None:
        d = torch.empty((T * top_k, H), dtype=torch.float32, device=dev)
    _check(h, "h", torch.bfloat16, 2, dev)
    _check(d, "d", torch.float32, 2, dev)
    if h.shape != (T * top_k, I) or d.shape != (T * top_k, H):
        raise ValueError("h must be [T*top_k, I] and d [T*top_k, H]")
    if ws is None:
        ws = workspace(T, H, I, E, top_k, dev)
    _check(ws, "workspace", torch.uint8, 1, dev)
    st = _lib.moe_expert_gemms_from_ids(_ptr(x), _ptr(ids), _ptr(W_gate_up), _ptr(S_gate_up), _ptr(W_down),
                                        _ptr(S_down), _ptr(h), 0 if fill_h else 1, _ptr(d), T, H, I, E, top_k,
                                        _ptr(ws), ws.numel(), _stream(dev))
    _raise(st, "moe_expert_gemms_from_ids")
    return h, d


def moe_combine(d: torch.Tensor, gates: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Stage hook: y [T, H] bf16 = sum_j gates[t, j] d[t*k + j] (fp32, j ascending)."""
    _check(d, "d", torch.float32, 2)
    dev = d.device
    _check(gates, "gates", torch.float32, 2, dev)
    T, top_k = gates.shape
    H = d.shape[1]
    if d.shape[0] != T * top_k:
        raise ValueError("d must be [T*top_k, H] for gates [T, top_k]")
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    _check(out, "out", torch.bfloat16, 2, dev)
    if out.shape != (T, H):
        raise ValueError("out must be [T, H]")
    _raise(_lib.moe_combine(_ptr(d), _ptr(gates), _ptr(out), T, H, top_k, _stream(dev)), "moe_combine")
    return out


def moe_down_combine(h: torch.Tensor, gates: torch.Tensor, W_down: torch.Tensor, S_down: torch.Tensor, sort: dict,
                     T: int, top_k: int, out: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """Stage hook: y [T, H] bf16 from gate_up's h, the gates and the sort result."""
    _check(h, "h", torch.bfloat16, 2)
    dev = h.device
    _check(gates, "gates", torch.float32, 2, dev)
    _check(W_down, "W_down", torch.uint8, 3, dev)
    _check(S_down, "S_down", torch.uint8, 3, dev)
    E, H, half_i = W_down.shape
    I = half_i * 2
    if S_down.shape != (E, H, I // 32) or h.shape != (T * top_k, I) or gates.shape != (T, top_k):
        raise ValueError("shapes do not match h [T*k, I], gates [T, k], W_down [E, H, I/2], S_down [E, H, I/32]")
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    _check(out, "out", torch.bfloat16, 2, dev)
    if ws is None:
        ws = workspace(T, H, I, E, top_k, dev)
    st = _lib.moe_down_combine(_ptr(h), _ptr(gates), _ptr(W_down), _ptr(S_down), *_sort_ptrs(sort, dev), _ptr(out),
                               T, H, I, E, top_k, _ptr(ws), ws.numel(), _stream(dev))
    _raise(st, "moe_down_combine")
    return out


def workspace_size(T: int, H: int, I: int, E: int, top_k: int) -> int:
    return int(_lib.moe_mxfp4_workspace_size(T, H, I, E, top_k))


_ws_cache: dict = {}


def workspace(T: int, H: int, I: int, E: int, top_k: int, device, stream=None) -> torch.Tensor:
    """A cached uint8 workspace tensor large enough for these sizes, one per (device,
    stream) -- by default the device's current stream.  Calls that share a workspace must
    not overlap in time: calls on one stream run one after another, and calls on two
    streams get two workspaces.  Allocated zero-filled: its leading control words must start
    at zero, and every call leaves them so."""
    need = workspace_size(T, H, I, E, top_k)
    dev = torch.device(device)
    if dev.index is None:
        dev = torch.device(dev.type, torch.cuda.current_device())
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    key = (dev, int(stream.cuda_stream))
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < need:
        buf = torch.zeros(need, dtype=torch.uint8, device=dev)
        _ws_cache[key] = buf
    return buf


# moe_mxfp4_forward_persistent: byte offset of the int32 word its bounded waits set to 1
# when they give up (sticky until cleared)
PERSISTENT_ERROR_OFFSET = 8


class MxWaitError(RuntimeError):
    """A single-launch layer's cross-workgroup wait gave up; its output is undefined."""


def take_persistent_error(ws: torch.Tensor) -> int:
    """Read and clear the single-launch layer's sticky error word in `ws` (synchronizes
    with the stream that used it)."""
    word = ws[PERSISTENT_ERROR_OFFSET:PERSISTENT_ERROR_OFFSET + 4].view(torch.int32)
    v = int(word.item())
    if v:
        word.zero_()
    return v


def raise_for_persistent_error(word: int) -> None:
    if word:
        raise MxWaitError("moe_mxfp4_forward_persistent: a cross-workgroup wait gave up (are other kernels "
                          "occupying the GPU?); the output is undefined")


def moe_mxfp4_forward(x: torch.Tensor, router_logits: torch.Tensor, top_k: int, W_gate_up: torch.Tensor,
                      S_gate_up: torch.Tensor, W_down: torch.Tensor, S_down: torch.Tensor,
                      out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                      persistent: bool = False, n_shared: int = 0, act8: bool = False,
                      check: bool = True) -> torch.Tensor:
    """y[T,H] of the MXFP4 SwiGLU MoE layer (see include/mxmoe.h for the definition).
    persistent=True runs it as one persistent launch (moe_mxfp4_forward_persistent; T <= 16);
    with check=True (and outside graph capture) the call then waits for it, reads and clears
    its sticky error word and raises MxWaitError when a wait gave up.
    n_shared > 0: the weights hold E routed + n_shared shared experts, router_logits [T, E]
    (moe_mxfp4_forward_shared).  act8=True: MXFP8 activations for both expert GEMMs
    (moe_mxfp4_forward_a8, with or without shared experts)."""
    _check(x, "x", torch.bfloat16, 2)
    dev = x.device
    _check(router_logits, "router_logits", torch.float32, 2, dev)
    for t, n in ((W_gate_up, "W_gate_up"), (S_gate_up, "S_gate_up"), (W_down, "W_down"), (S_down, "S_down")):
        _check(t, n, torch.uint8, 3, dev)
    T, H = x.shape
    E = router_logits.shape[1]
    Ew = E + n_shared
    I = W_down.shape[2] * 2
    if router_logits.shape[0] != T:
        raise ValueError("router_logits must be [T, E]")
    if (W_gate_up.shape != (Ew, 2 * I, H // 2) or S_gate_up.shape != (Ew, 2 * I, H // 32)
            or W_down.shape != (Ew, H, I // 2) or S_down.shape != (Ew, H, I // 32)):
        raise ValueError("expert weight shapes do not match [E, 2I, H/2], [E, 2I, H/32], [E, H, I/2], [E, H, I/32] "
                         "with E routed + n_shared shared experts")
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    _check(out, "out", torch.bfloat16, 2, dev)
    if ws is None:
        ws = workspace(T, H, I, Ew, top_k + n_shared, dev)
    _check(ws, "workspace", torch.uint8, 1, dev)
    if persistent and (n_shared or act8):
        raise ValueError("the single-launch layer has neither shared experts nor MXFP8 activations")
    if n_shared or act8:
        name = "moe_mxfp4_forward_a8" if act8 else "moe_mxfp4_forward_shared"
        st = getattr(_lib, name)(_ptr(x), _ptr(router_logits), top_k, n_shared, _ptr(W_gate_up), _ptr(S_gate_up),
                                 _ptr(W_down), _ptr(S_down), _ptr(out), T, H, I, E, _ptr(ws), ws.numel(),
                                 _stream(dev))
    else:
        name = "moe_mxfp4_forward_persistent" if persistent else "moe_mxfp4_forward"
        st = getattr(_lib, name)(_ptr(x), _ptr(router_logits), top_k, _ptr(W_gate_up), _ptr(S_gate_up),
                                 _ptr(W_down), _ptr(S_down), _ptr(out), T, H, I, E, _ptr(ws), ws.numel(),
                                 _stream(dev))
    _raise(st, name)
    if persistent and check and not torch.cuda.is_current_stream_capturing():
        raise_for_persistent_error(take_persistent_error(ws))
    return out


# ------------------------------------------------------------------ dense feed-forward operators
#
# Autograd does not record these calls: their results have no history, also where an input
# requires grad.  The gradients come from the *_backward calls, e.g. inside a
# torch.autograd.Function.

_ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "sigmoid": 5}
_GATE_NONE, _GATE_TOKEN, _GATE_CHANNEL, _GATE_FULL = 0, 1, 2, 3
MX_NORM_MAX_H = 16384
_BF16, _U8, _F32 = torch.bfloat16, torch.uint8, torch.float32


def _act_code(act: str) -> int:
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(_ACTS)}, got {act!r}")
    return code


# A decode step's call is a few microseconds of GPU time, so the checks below take their fast
# way in one expression and leave naming what is wrong to _check; the raw stream handle saves
# building a Stream object (2 us of the 12 that a call took).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _tensor(t, name: str, dtype, shape, dev):
    """_check with the whole shape at once."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.shape == shape and t.device == dev
            and t.is_contiguous()):
        _check(t, name, dtype, None, dev)
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _opt(t) -> int | None:
    return None if t is None else t.data_ptr()


def _scratch(nbytes: int, dev, ws):
    """(tensor, pointer, bytes) of a call's workspace: the caller's, or a fresh one from the
    allocator, which keeps it for this stream (and, under graph capture, for this graph)."""
    if ws is not None:
        _check(ws, "workspace", _U8, 1, dev)
        return ws, ws.data_ptr(), ws.numel()
    if nbytes == 0:
        return None, None, 0
    ws = torch.empty(nbytes, dtype=_U8, device=dev)
    return ws, ws.data_ptr(), nbytes


def _call(fn, dev, *args):
    """The C call `fn` on dev's current stream, which is its last argument."""
    index = dev.index
    stream = _raw_stream(index)
    if _current_device() == index:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st != MX_OK:
        _raise(st, fn.__name__)


def _bf16_rows(t, name: str):
    if not (isinstance(t, torch.Tensor) and t.dtype is _BF16 and t.is_cuda and t.dim() == 2 and t.is_contiguous()):
        _check(t, name, _BF16, 2)
    if t.numel() == 0:
        raise ValueError(f"{name} is empty: {list(t.shape)}")
    return t.shape


def _apart(out, t, name: str, itself: bool = False):
    """Refuses an output over an input that other workgroups still read while it is written;
    `itself`: over exactly the same elements it is fine, each is read before it is written."""
    o, i = out.data_ptr(), t.data_ptr()
    if o < i + 2 * t.numel() and i < o + 2 * out.numel() and not (itself and o == i):
        raise ValueError(f"out must not overlap {name}" + (" except as the same tensor" if itself else ""))


def _weights(codes, scales, name: str, rows: int | None, K: int, dev) -> int:
    if rows is None:
        if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
            raise ValueError(f"{name} codes must be a 2-d tensor")
        rows = codes.shape[0]
    if K % 32:
        raise ValueError(f"the reduction length {K} must be a multiple of 32")
    _tensor(codes, f"{name} codes", _U8, (rows, K // 2), dev)
    _tensor(scales, f"{name} scales", _U8, (rows, K // 32), dev)
    return rows


def mx_linear_fused(x: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor, bias: torch.Tensor | None = None,
                    residual: torch.Tensor | None = None, scale: float = 1.0, act: str = "none",
                    save_z: bool = False, out: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """y[T,N] = residual + scale * act(x W^T + bias), all in fp32, rounded once to bf16.
    act: none, relu, silu, gelu, gelu_tanh or sigmoid.  out may be the residual itself,
    not x.  save_z=True: (y, z), z = x W^T + bias in bf16 for mx_linear_fused_backward.  Autograd
    records nothing: the gradients are that call's."""
    T, K = _bf16_rows(x, "x")
    dev = x.device
    N = _weights(w_codes, w_scales, "weight", None, K, dev)
    if bias is not None:
        _tensor(bias, "bias", _BF16, (N,), dev)
    if residual is not None:
        _tensor(residual, "residual", _BF16, (T, N), dev)
    code = _act_code(act)
    if out is None:
        out = x.new_empty((T, N)) if residual is None else torch.empty_like(residual)
    else:
        _tensor(out, "out", _BF16, (T, N), dev)
        _apart(out, x, "x")
        if residual is not None:
            _apart(out, residual, "residual", itself=True)
    z = torch.empty((T, N), dtype=_BF16, device=dev) if save_z else None
    ws, wp, wn = _scratch(_lib.mx_linear_fused_workspace_size(T, K, N), dev, ws)
    _call(_lib.mx_linear_fused, dev, x.data_ptr(), w_codes.data_ptr(), w_scales.data_ptr(), _opt(bias), _opt(residual),
          scale, code, out.data_ptr(), _opt(z), T, K, N, wp, wn)
    return (out, z) if save_z else out


def mx_linear_fused_backward(dy: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
                             z: torch.Tensor | None = None, scale: float = 1.0, act: str = "none",
                             need_dx: bool = True, need_dbias: bool = True, ws: torch.Tensor | None = None):
    """(dx bf16 [T,K], dbias fp32 [N]) of mx_linear_fused from dy and its saved z (not needed
    for act "none"); None for what is not asked for.  The residual's gradient is dy."""
    T, N = _bf16_rows(dy, "dy")
    dev = dy.device
    if not isinstance(w_codes, torch.Tensor) or w_codes.dim() != 2:
        raise ValueError("w_codes must be a 2-d tensor")
    K = w_codes.shape[1] * 2
    _weights(w_codes, w_scales, "weight", N, K, dev)
    code = _act_code(act)
    if code and z is None:
        raise ValueError(f"act {act!r} needs z, the pre-activations of the forward call")
    if z is not None:
        _tensor(z, "z", _BF16, (T, N), dev)
    if not need_dx and not need_dbias:
        raise ValueError("neither dx nor dbias is asked for")
    dx = torch.empty((T, K), dtype=_BF16, device=dev) if need_dx else None
    dbias = torch.empty(N, dtype=_F32, device=dev) if need_dbias else None
    ws, wp, wn = _scratch(_lib.mx_linear_fused_backward_workspace_size(T, K, N), dev, ws)
    _call(_lib.mx_linear_fused_backward, dev, dy.data_ptr(), _opt(z), w_codes.data_ptr(), w_scales.data_ptr(), scale, code,
          _opt(dx), _opt(dbias), T, K, N, wp, wn)
    return dx, dbias


def mx_gate_up(x: torch.Tensor, W_gate_up: torch.Tensor, S_gate_up: torch.Tensor, bias: torch.Tensor | None = None,
               act: str = "silu", save_z: bool = False, out: torch.Tensor | None = None,
               ws: torch.Tensor | None = None):
    """h[T,I] = act(x Wg^T + bg) * (x Wu^T + bu) with W_gate_up [2I, H/2] (gate rows, then up
    rows), all in fp32, rounded once to bf16.  save_z=True: (h, z), z bf16 [T, 2I] the two
    pre-activations for mx_gate_up_backward.  Autograd records nothing: the gradients are that
    call's."""
    T, H = _bf16_rows(x, "x")
    dev = x.device
    two_i = _weights(W_gate_up, S_gate_up, "W_gate_up", None, H, dev)
    if two_i % 2:
        raise ValueError("W_gate_up must have an even number of rows")
    I = two_i // 2
    if bias is not None:
        _tensor(bias, "bias", _BF16, (two_i,), dev)
    code = _act_code(act)
    if out is None:
        out = x.new_empty((T, I))
    else:
        _tensor(out, "out", _BF16, (T, I), dev)
        _apart(out, x, "x")
    z = torch.empty((T, two_i), dtype=_BF16, device=dev) if save_z else None
    ws, wp, wn = _scratch(_lib.mx_gate_up_workspace_size(T, H, I), dev, ws)
    _call(_lib.mx_gate_up, dev, x.data_ptr(), W_gate_up.data_ptr(), S_gate_up.data_ptr(), _opt(bias), code, out.data_ptr(),
          _opt(z), T, H, I, wp, wn)
    return (out, z) if save_z else out


def mx_gate_up_backward(dh: torch.Tensor, z: torch.Tensor, W_gate_up: torch.Tensor, S_gate_up: torch.Tensor,
                        act: str = "silu", need_dx: bool = True, need_dbias: bool = True,
                        ws: torch.Tensor | None = None):
    """(dx bf16 [T,H], dbias fp32 [2I]) of mx_gate_up from dh and its saved z; None for what is
    not asked for."""
    T, I = _bf16_rows(dh, "dh")
    dev = dh.device
    if not isinstance(W_gate_up, torch.Tensor) or W_gate_up.dim() != 2:
        raise ValueError("W_gate_up must be a 2-d tensor")
    H = W_gate_up.shape[1] * 2
    _weights(W_gate_up, S_gate_up, "W_gate_up", 2 * I, H, dev)
    _tensor(z, "z", _BF16, (T, 2 * I), dev)
    code = _act_code(act)
    if not need_dx and not need_dbias:
        raise ValueError("neither dx nor dbias is asked for")
    dx = torch.empty((T, H), dtype=_BF16, device=dev) if need_dx else None
    dbias = torch.empty(2 * I, dtype=_F32, device=dev) if need_dbias else None
    ws, wp, wn = _scratch(_lib.mx_gate_up_backward_workspace_size(T, H, I), dev, ws)
    _call(_lib.mx_gate_up_backward, dev, dh.data_ptr(), z.data_ptr(), W_gate_up.data_ptr(), S_gate_up.data_ptr(), code,
          _opt(dx), _opt(dbias), T, H, I, wp, wn)
    return dx, dbias


def _gate_mode(gate, T: int, H: int, dev) -> int:
    if gate is None:
        return _GATE_NONE
    shape = gate.shape if isinstance(gate, torch.Tensor) else None
    mode = {(H,): _GATE_CHANNEL, (T, H): _GATE_FULL, (T, 1): _GATE_TOKEN}.get(shape)
    if mode is None:
        raise ValueError(f"gate must be a tensor of shape [T, 1], [H] or [T, H] with T={T}, H={H}")
    _tensor(gate, "gate", _BF16, shape, dev)
    return mode


def mx_norm_residual(x: torch.Tensor, b: torch.Tensor | None = None, w_post: torch.Tensor | None = None,
                     gate: torch.Tensor | None = None, scale: float = 1.0, w_pre: torch.Tensor | None = None,
                     eps: float = 1e-6, out: torch.Tensor | None = None):
    """(y, xn): y = x + scale * gate * rms_norm(b) * w_post, the residual stream after a block
    with output b, and xn = rms_norm(y) * w_pre, the next block's input; each norm where its
    weight is given, xn None without w_pre.  gate: [T, 1] per token, [H] per channel or [T, H].
    Without b: (x, rms_norm(x) * w_pre).  out, for y, may be x itself.  Autograd records nothing:
    the gradients are mx_norm_residual_backward's."""
    T, H = _bf16_rows(x, "x")
    dev = x.device
    for t, n in ((w_post, "w_post"), (w_pre, "w_pre")):
        if t is not None:
            _tensor(t, n, _BF16, (H,), dev)
    mode = _gate_mode(gate, T, H, dev)
    if b is None:
        if w_post is not None or gate is not None or out is not None or w_pre is None:
            raise ValueError("without b the call takes w_pre alone")
        y = None
    else:
        _tensor(b, "b", _BF16, (T, H), dev)
        y = out
        if y is None:
            y = torch.empty_like(x)
        else:
            _tensor(y, "out", _BF16, (T, H), dev)
            _apart(y, x, "x", itself=True)
            _apart(y, b, "b", itself=True)
    xn = torch.empty_like(x) if w_pre is not None else None
    _call(_lib.mx_norm_residual, dev, x.data_ptr(), _opt(b), _opt(w_post), _opt(gate), mode, scale, _opt(w_pre), eps,
          _opt(y), _opt(xn), T, H)
    return (x if y is None else y), xn


def mx_norm_residual_backward(dy: torch.Tensor | None, dxn: torch.Tensor | None, y: torch.Tensor | None,
                              b: torch.Tensor | None = None, w_post: torch.Tensor | None = None,
                              gate: torch.Tensor | None = None, scale: float = 1.0,
                              w_pre: torch.Tensor | None = None, eps: float = 1e-6,
                              ws: torch.Tensor | None = None, *, need_db: bool = True, need_dgate: bool = True,
                              need_dw_post: bool = True, need_dw_pre: bool = True) -> dict:
    """The gradients of mx_norm_residual from those of y and xn: a dict of dx, db (bf16 [T, H]),
    dgate (fp32 [T, 1] or [H], bf16 [T, H]), dw_post and dw_pre (fp32 [H]), None for what the
    forward did not have or is not asked for.  y is the forward's y (its x without b); dy may be
    None with w_pre."""
    first = dy if dy is not None else dxn
    T, H = _bf16_rows(first, "dy" if dy is not None else "dxn")
    dev = first.device
    for t, n in ((dy, "dy"), (dxn, "dxn"), (y, "y"), (b, "b")):
        if t is not None:
            _tensor(t, n, _BF16, (T, H), dev)
    for t, n in ((w_post, "w_post"), (w_pre, "w_pre")):
        if t is not None:
            _tensor(t, n, _BF16, (H,), dev)
    mode = _gate_mode(gate, T, H, dev)
    if (w_pre is None) != (dxn is None) or (w_pre is not None and y is None):
        raise ValueError("w_pre, dxn and y go together")
    if b is None and (w_post is not None or gate is not None):
        raise ValueError("w_post and gate need b")
    dx = torch.empty_like(first)
    db = torch.empty_like(first) if b is not None and need_db else None
    dgate = None
    if gate is not None and need_dgate:
        dgate = torch.empty(tuple(gate.shape), dtype=_BF16 if mode == _GATE_FULL else _F32, device=dev)
    dw_post = torch.empty(H, dtype=_F32, device=dev) if w_post is not None and need_dw_post else None
    dw_pre = torch.empty(H, dtype=_F32, device=dev) if w_pre is not None and need_dw_pre else None
    ws, wp, wn = _scratch(_lib.mx_norm_residual_backward_workspace_size(T, H), dev, ws)
    _call(_lib.mx_norm_residual_backward, dev, _opt(dy), _opt(dxn), _opt(y), _opt(b), _opt(w_post), _opt(gate), mode,
          scale, _opt(w_pre), eps, dx.data_ptr(), _opt(db), _opt(dgate), _opt(dw_post), _opt(dw_pre), T, H, wp, wn)
    return dict(dx=dx, db=db, dgate=dgate, dw_post=dw_post, dw_pre=dw_pre)


def mx_ffn_block(x: torch.Tensor, W_gate_up: torch.Tensor, S_gate_up: torch.Tensor, W_down: torch.Tensor,
                 S_down: torch.Tensor, w_pre: torch.Tensor | None = None, bias_gate_up: torch.Tensor | None = None,
                 bias_down: torch.Tensor | None = None, act: str = "silu", w_post: torch.Tensor | None = None,
                 gate: torch.Tensor | None = None, scale: float = 1.0, eps: float = 1e-6,
                 out: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """A dense feed-forward block of a transformer: y = x + scale * gate * rms_norm(b) * w_post
    with b = mx_gate_up(rms_norm(x) * w_pre) W_down^T + bias_down; each norm where its weight is
    given, gate as for mx_norm_residual.  out may be x itself.  For inference: it saves nothing for
    a backward pass and autograd records nothing; a training step makes the separate calls."""
    T, H = _bf16_rows(x, "x")
    dev = x.device
    two_i = _weights(W_gate_up, S_gate_up, "W_gate_up", None, H, dev)
    if two_i % 2:
        raise ValueError("W_gate_up must have an even number of rows")
    I = two_i // 2
    _weights(W_down, S_down, "W_down", H, I, dev)
    for t, n, size in ((w_pre, "w_pre", H), (w_post, "w_post", H), (bias_gate_up, "bias_gate_up", two_i),
                       (bias_down, "bias_down", H)):
        if t is not None:
            _tensor(t, n, _BF16, (size,), dev)
    mode = _gate_mode(gate, T, H, dev)
    code = _act_code(act)
    if out is None:
        out = torch.empty_like(x)
    else:
        _tensor(out, "out", _BF16, (T, H), dev)
        _apart(out, x, "x", itself=True)
    ws, wp, wn = _scratch(_lib.mx_ffn_block_workspace_size(T, H, I), dev, ws)
    _call(_lib.mx_ffn_block, dev, x.data_ptr(), _opt(w_pre), W_gate_up.data_ptr(), S_gate_up.data_ptr(),
          _opt(bias_gate_up), code, W_down.data_ptr(), S_down.data_ptr(), _opt(bias_down), _opt(w_post), _opt(gate), mode,
          scale, eps, out.data_ptr(), T, H, I, wp, wn)
    return out
