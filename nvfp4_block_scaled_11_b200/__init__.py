"""nvfp4_block_scaled_11_b200 -- Python binding of libnvfp4 (NVFP4 ScaleSearch quantization, sm_100a).

Argument marshalling only: every function checks that its tensors are contiguous CUDA tensors,
allocates outputs with torch when the caller did not pass them, and calls the C ABI declared in
``include/nvfp4.h`` with raw device pointers and the current CUDA stream.  All computation happens
in the library's CUDA kernels; there is no CPU path.  A missing ``libnvfp4.so`` raises.

Element types: torch.float32, torch.bfloat16, torch.float16.
"""
from __future__ import annotations

import array
import ctypes
import math
import numbers
import os
import struct

import torch

__all__ = [
    "NVFP4Error", "lib", "status_str", "tensor_amax", "global_scale", "quantize", "quantize_ex",
    "dequantize", "quantize_dequantize", "hadamard16", "kv_mixed", "kv_mixed_dequantize", "DTYPE_CODE", "sf_mma_bytes", "quantize_mma", "quantize_mma_t", "kv_mixed_mma",
    "gemm_nt", "gemm_sf_offsets", "kv_gscale", "kv_append", "mxfp4_quantize", "mxfp4_dequantize",
    "msda_forward", "softmax_quantize_mma", "rows_divide", "attention_fp4", "search_policy", "kv_append_batch", "KvAppendBatch",
    "KvStore", "kv_attention", "rope", "rope_frequencies", "copy_pages",
]

_SO = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnvfp4.so")
_lib = None

DTYPE_CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
DTYPE_OF = {v: k for k, v in DTYPE_CODE.items()}

# C-ABI entry points and their argument types (include/nvfp4.h)
_P, _I64, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
_SIGS = {
    "nvfp4_status_str": (ctypes.c_char_p, [_I]),
    "nvfp4_version": (_I, []),
    "nvfp4_search_policy": (_I, [_I64, _I64, _P, _P]),
    "nvfp4_tensor_amax": (_I, [_P, _I64, _I, _P, _P]),
    "nvfp4_global_scale": (_I, [_P, _P, _P]),
    "nvfp4_quantize": (_I, [_P, _I64, _I, _I, _I, _I, _P, _P, _P, _P]),
    "nvfp4_quantize_ex": (_I, [_P, _I64, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P]),
    "nvfp4_dequantize": (_I, [_P, _P, _P, _I64, _I, _P, _P]),
    "nvfp4_dequantize_ex": (_I, [_P, _P, _P, _I64, _I, _P, _I, _P]),
    "nvfp4_quantize_dequantize": (_I, [_P, _I64, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "nvfp4_hadamard16": (_I, [_P, _I64, _I, _P, _I, _P]),
    "nvfp4_hadamard16_ex": (_I, [_P, _I64, _I, _P, _I, ctypes.c_uint32, _I, _P]),
    "nvfp4_kv_mixed": (_I, [_P, _I64, _I64, _I64, _I64, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "nvfp4_kv_mixed_dequantize": (_I, [_P, _I64, _I64, _I64, _I64, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P]),
    "nvfp4_msda_forward_nvfp4": (_I, [_P, _P, _P, _I64, _I64, _I64, _I64, _P, _I, _I, _I64, _P, _P, _P, _P]),
    "nvfp4_msda_forward": (_I, [_P, _I, _I64, _I64, _I64, _I64, _P, _I, _I, _I64, _P, _P, _P, _P]),
    "nvfp4_mxfp4_quantize": (_I, [_P, _I64, _I, _P, _P, _P]),
    "nvfp4_mxfp4_dequantize": (_I, [_P, _P, _I64, _I, _P, _P]),
    "nvfp4_kv_gscale": (_I, [_P, _I64, _I64, _I64, _I64, _I, _I, _I, _P, _P]),
    "nvfp4_kv_append": (_I, [_P, _I64, _I64, _I64, _I64, _I64, _I, _I, _I, _P, _P, _P, _I64, _I64, _I, _P]),
    "nvfp4_kv_append_batch": (_I, [_P, _I, _I, _I, _P]),
    "nvfp4_sf_mma_bytes": (_I64, [_I64, _I64, _I64]),
    "nvfp4_quantize_mma": (_I, [_P, _I64, _I64, _I64, _I, _I, _I, _P, _P, _P, _P, _P]),
    "nvfp4_quantize_mma_t": (_I, [_P, _I64, _I64, _I64, _I, _I, _I, _P, _P, _P, _P, _P]),
    "nvfp4_kv_mixed_mma": (_I, [_P, _I64, _I64, _I64, _I64, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "nvfp4_gemm_nt": (_I, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, ctypes.c_float, _P, _I, _P, _P]),
    "nvfp4_gemm_nt_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, ctypes.c_float, _P, _I, _P]),
    "nvfp4_softmax_quantize_mma": (_I, [_P, _I64, _I64, _I64, _I, _I64, _I, _I, _P, _P, _P, _P, _P, _P]),
    "nvfp4_rows_divide": (_I, [_P, _P, _I64, _I64, _P]),
    "nvfp4_attention_fused": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, ctypes.c_float, _I,
                                   _I64, _I, _I, _I, _P, ctypes.c_size_t, _P, _P, _P, _P, _P, _P, _P, _P]),
    "nvfp4_attention_fused_splits": (_I, [_I64, _I64, _I64, _P]),
    "nvfp4_attention_fused_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64, _I]),
    "nvfp4_kv_attention": (_I, [_P, _I, _P, ctypes.c_size_t, _P]),
    "nvfp4_kv_attention_splits": (_I, [_I64, _I64, _I64, _I64, _I64, _P]),
    "nvfp4_kv_attention_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I]),
    "nvfp4_rope": (_I, [_P, _I, _I64, _I64, _I64, _I64, _I, _I, _P, _I, _I64, _I64, _P, ctypes.c_float, _I, _P]),
    "nvfp4_copy_pages": (_I, [_P, _I, _P, _P, _I64, _P]),
    "nvfp4_gemm_sf_offsets": (_I, [_I64, _I64, _I64, _P]),
}


class NVFP4Error(RuntimeError):
    def __init__(self, status: int):
        super().__init__(status_str(status))
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded libnvfp4 (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_SO):
            raise RuntimeError(
                f"libnvfp4.so is not built ({_SO}); run `python -m nvfp4_block_scaled_11_b200.build`"
            )
        L = ctypes.CDLL(_SO)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def library_path() -> str:
    """Path of the loaded libnvfp4.so (for C programs that link it)."""
    lib()
    return _SO


def status_str(status: int) -> str:
    return lib().nvfp4_status_str(status).decode()


def _check(rc: int) -> None:
    if rc != 0:
        raise NVFP4Error(rc)


def search_policy(lane1_max: int | None = None, lanes_max: int | None = None) -> tuple[int, int]:
    """Launch policy of the ScaleSearch quantizers (windows of at most 32 offsets), bounds in threads
    (blocks x lanes per block): up to `lane1_max`, one offset per lane (16 or 32 lanes per block); up to
    `lanes_max`, a few offsets per lane (4 or 8 lanes per block); beyond, a thread per block.  All write
    the same bytes.  None keeps a bound; returns the previous bounds."""
    a, b = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().nvfp4_search_policy(-1 if lane1_max is None else int(lane1_max),
                                     -1 if lanes_max is None else int(lanes_max), ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def _cuda(t: torch.Tensor, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _out(t: torch.Tensor, name: str, dtype, need: int) -> torch.Tensor:
    """A caller-provided buffer that a kernel reads or writes by size: a contiguous CUDA tensor of `dtype`
    (None: any dtype) with at least `need` elements, so that no launch reaches past its end."""
    _cuda(t, name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() < need:
        raise ValueError(f"{name} holds {t.numel()} elements, {need} needed")
    return t


def _one_device(dev: torch.device, **tensors) -> None:
    """Every tensor of a launch is on the device that it runs on: a kernel given another device's memory faults."""
    for name, t in tensors.items():
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the call runs on {dev}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _dt(t: torch.Tensor) -> int:
    try:
        return DTYPE_CODE[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def tensor_amax(x: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """max |x| as a 1-element float32 device tensor (NaN / Inf propagate)."""
    _cuda(x, "x")
    out = torch.empty(1, dtype=torch.float32, device=x.device) if out is None else _out(out, "out", torch.float32, 1)
    _check(lib().nvfp4_tensor_amax(_ptr(x), x.numel(), _dt(x), _ptr(out), _stream(x)))
    return out


def global_scale(amax: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """g = amax / 2688 on the device."""
    _out(amax, "amax", torch.float32, 1)
    out = torch.empty(1, dtype=torch.float32, device=amax.device) if out is None else _out(out, "out", torch.float32, 1)
    _check(lib().nvfp4_global_scale(_ptr(amax), _ptr(out), _stream(amax)))
    return out


def _alloc_q(x, codes, scales, gscale):
    n = x.numel()
    dev = x.device
    codes = torch.empty(n // 2, dtype=torch.uint8, device=dev) if codes is None else _out(codes, "codes", torch.uint8, n // 2)
    scales = (torch.empty(n // 16, dtype=torch.uint8, device=dev) if scales is None
              else _out(scales, "scales", torch.uint8, n // 16))
    gscale = (torch.empty(1, dtype=torch.float32, device=dev) if gscale is None
              else _out(gscale, "gscale", torch.float32, 1))
    return codes, scales, gscale


def quantize(x: torch.Tensor, f_lo: int = -2, f_hi: int = 6, block: int = 16, codes=None, scales=None, gscale=None):
    """ScaleSearch quantize of x (blocks of 16 along the contiguous order).

    Returns (codes uint8[n/2], scales uint8[n/16], gscale float32[1])."""
    _cuda(x, "x")
    codes, scales, gscale = _alloc_q(x, codes, scales, gscale)
    _check(lib().nvfp4_quantize(_ptr(x), x.numel(), _dt(x), block, f_lo, f_hi, _ptr(codes), _ptr(scales),
                                _ptr(gscale), _stream(x)))
    return codes, scales, gscale


def quantize_ex(x: torch.Tensor, f_lo: int = -2, f_hi: int = 6, gscale_in: torch.Tensor | None = None,
                want_f: bool = True, want_sse: bool = True, block: int = 16, codes=None, scales=None, gscale=None,
                block_f=None, block_sse=None):
    """Quantize with optional external tensor scale and per-block outputs.

    Returns (codes, scales, gscale, block_f int8[n/16] or None, block_sse float32[n/16] or None)."""
    _cuda(x, "x")
    n = x.numel()
    keep = gscale
    if gscale_in is not None:
        _out(gscale_in, "gscale_in", torch.float32, 1)
    codes, scales, gscale = _alloc_q(x, codes, scales, gscale)
    if gscale_in is not None and keep is None:
        gscale = None  # g comes from gscale_in; no copy requested
    if want_f and block_f is None:
        block_f = torch.empty(n // 16, dtype=torch.int8, device=x.device)
    elif block_f is not None:
        _out(block_f, "block_f", torch.int8, n // 16)
    if want_sse and block_sse is None:
        block_sse = torch.empty(n // 16, dtype=torch.float32, device=x.device)
    elif block_sse is not None:
        _out(block_sse, "block_sse", torch.float32, n // 16)
    _check(lib().nvfp4_quantize_ex(_ptr(x), n, _dt(x), block, f_lo, f_hi, _ptr(gscale_in), _ptr(codes),
                                   _ptr(scales), _ptr(gscale), _ptr(block_f), _ptr(block_sse), _stream(x)))
    return codes, scales, gscale, block_f, block_sse


def quantize_dequantize(x: torch.Tensor, f_lo: int = -2, f_hi: int = 6, gscale_in: torch.Tensor | None = None,
                        codes=None, scales=None, gscale=None, out: torch.Tensor | None = None):
    """Fused round trip: quantize x with ScaleSearch and write its dequantized values (x's dtype) in the same
    pass.  Returns (out, codes, scales, gscale); out equals dequantize(codes, scales, g, x.dtype) bit for bit.
    out may be x itself (in-place simulated quantization)."""
    _cuda(x, "x")
    n = x.numel()
    if gscale_in is not None:
        _out(gscale_in, "gscale_in", torch.float32, 1)
    keep = gscale
    codes, scales, gscale = _alloc_q(x, codes, scales, gscale)
    if gscale_in is not None and keep is None:
        gscale = None
    out = torch.empty_like(x) if out is None else out
    _cuda(out, "out")
    if out.dtype != x.dtype or out.numel() != n:
        raise ValueError("out must have x's dtype and size")
    _check(lib().nvfp4_quantize_dequantize(_ptr(x), n, _dt(x), f_lo, f_hi, _ptr(gscale_in), _ptr(codes), _ptr(scales),
                                           _ptr(gscale), _ptr(out), _stream(x)))
    return out, codes, scales, gscale


def dequantize(codes: torch.Tensor, scales: torch.Tensor, gscale: torch.Tensor, out_dtype=torch.float32,
               out: torch.Tensor | None = None, ctas_per_sm: int = 0) -> torch.Tensor:
    """Dequantize n = 16 * scales.numel() elements to out_dtype.  ctas_per_sm > 0 bounds the launch
    footprint (to run beside another kernel on a second stream); 0 = default."""
    _cuda(scales, "scales")
    n = scales.numel() * 16
    _out(codes, "codes", torch.uint8, n // 2), _out(gscale, "gscale", torch.float32, 1)
    out = torch.empty(n, dtype=out_dtype, device=codes.device) if out is None else _out(out, "out", None, n)
    _check(lib().nvfp4_dequantize_ex(_ptr(codes), _ptr(scales), _ptr(gscale), n, DTYPE_CODE[out.dtype], _ptr(out),
                                     ctas_per_sm, _stream(codes)))
    return out


def hadamard16(x: torch.Tensor, out_dtype=None, out: torch.Tensor | None = None, signs: int = 0,
               inverse: bool = False) -> torch.Tensor:
    """FWHT-16 / 4 on every contiguous group of 16 elements; with `signs` (16-bit mask) the sign diagonal
    D goes first, (H/4) D x, or last for the inverse, D (H/4) x."""
    _cuda(x, "x")
    out_dtype = x.dtype if out_dtype is None else out_dtype
    out = torch.empty(x.shape, dtype=out_dtype, device=x.device) if out is None else _out(out, "out", None, x.numel())
    if signs == 0 and not inverse:
        _check(lib().nvfp4_hadamard16(_ptr(x), x.numel(), _dt(x), _ptr(out), DTYPE_CODE[out.dtype], _stream(x)))
    else:
        _check(lib().nvfp4_hadamard16_ex(_ptr(x), x.numel(), _dt(x), _ptr(out), DTYPE_CODE[out.dtype], signs,
                                         int(inverse), _stream(x)))
    return out


def kv_mixed(k: torch.Tensor, sink: int = 16, recent: int = 16, rotate: bool = True, f_lo: int = -2, f_hi: int = 6):
    """Mixed-precision KV layout of K[B,H,T,D] (BF16).

    Returns (sink bf16[B,H,sink,D], recent bf16[B,H,recent,D], codes uint8[B,H,Tm,D/2],
    scales uint8[B,H,Tm,D/16], gscale float32[1])."""
    _cuda(k, "k")
    if k.dtype != torch.bfloat16 or k.dim() != 4:
        raise TypeError("k must be a 4-D bfloat16 tensor [B,H,T,D]")
    B, H, T, D = k.shape
    Tm = T - sink - recent
    dev = k.device
    so = torch.empty((B, H, sink, D), dtype=torch.bfloat16, device=dev)
    ro = torch.empty((B, H, recent, D), dtype=torch.bfloat16, device=dev)
    codes = torch.empty((B, H, max(Tm, 0), D // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((B, H, max(Tm, 0), D // 16), dtype=torch.uint8, device=dev)
    gscale = torch.empty(1, dtype=torch.float32, device=dev)
    _check(lib().nvfp4_kv_mixed(_ptr(k), B, H, T, D, sink, recent, int(bool(rotate)), f_lo, f_hi, _ptr(so),
                                _ptr(ro), _ptr(codes), _ptr(scales), _ptr(gscale), _stream(k)))
    return so, ro, codes, scales, gscale


# ---- tensor-core consumer: scales in the MMA tile layout, NVFP4 x NVFP4 product ----
def sf_mma_bytes(rows: int, cols: int, batch: int = 1) -> int:
    """Bytes of the tile-layout scales of `batch` [rows, cols] matrices (padded to 128 rows x 4 blocks)."""
    nb = lib().nvfp4_sf_mma_bytes(rows, cols, batch)
    if nb < 0:
        raise NVFP4Error(int(nb))
    return int(nb)


def kv_mixed_dequantize(k: torch.Tensor, sink: int = 16, recent: int = 16, rotate: bool = True, f_lo: int = -2,
                        f_hi: int = 6, mid_out: torch.Tensor | None = None):
    """kv_mixed plus the middle's dequantized values (BF16 [B,H,Tm,D], rotated when `rotate`) in the same
    pass.  Returns (sink, recent, codes, scales, gscale, mid)."""
    _cuda(k, "k")
    if k.dtype != torch.bfloat16 or k.dim() != 4:
        raise TypeError("k must be a 4-D bfloat16 tensor [B,H,T,D]")
    B, H, T, D = k.shape
    Tm = T - sink - recent
    if Tm < 0:
        raise ValueError("T < sink + recent")
    dev = k.device
    so = torch.empty((B, H, sink, D), dtype=torch.bfloat16, device=dev)
    ro = torch.empty((B, H, recent, D), dtype=torch.bfloat16, device=dev)
    codes = torch.empty((B, H, Tm, D // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((B, H, Tm, D // 16), dtype=torch.uint8, device=dev)
    gscale = torch.empty(1, dtype=torch.float32, device=dev)
    mid = torch.empty((B, H, Tm, D), dtype=torch.bfloat16, device=dev) if mid_out is None else mid_out
    _cuda(mid, "mid_out")
    if mid.dtype != torch.bfloat16 or mid.numel() != B * H * Tm * D:
        raise ValueError("mid_out must be bfloat16 with B*H*Tm*D elements")
    _check(lib().nvfp4_kv_mixed_dequantize(_ptr(k), B, H, T, D, sink, recent, int(bool(rotate)), f_lo, f_hi, _ptr(so),
                                           _ptr(ro), _ptr(codes), _ptr(scales), _ptr(gscale), _ptr(mid), _stream(k)))
    return so, ro, codes, scales, gscale, mid


def quantize_mma(x: torch.Tensor, f_lo: int = -2, f_hi: int = 6, gscale_in: torch.Tensor | None = None,
                 codes: torch.Tensor | None = None, sf: torch.Tensor | None = None,
                 gscale: torch.Tensor | None = None):
    """Quantize x [rows, cols] or [batch, rows, cols] along cols with the scales in the tensor-core tile
    layout.  Returns (codes uint8[..., rows, cols/2] (x's rank), sf uint8[sf_mma_bytes], gscale float32[1])."""
    _cuda(x, "x")
    if x.dim() not in (2, 3):
        raise ValueError("x must be [rows, cols] or [batch, rows, cols]")
    batch, rows, cols = (1, *x.shape) if x.dim() == 2 else x.shape
    dev = x.device
    if codes is None:
        codes = torch.empty((*x.shape[:-1], cols // 2), dtype=torch.uint8, device=dev)
    if sf is None:
        sf = torch.empty(sf_mma_bytes(rows, cols, batch), dtype=torch.uint8, device=dev)
    if gscale is None:
        gscale = torch.empty(1, dtype=torch.float32, device=dev)
    _out(codes, "codes", torch.uint8, x.numel() // 2), _out(gscale, "gscale", torch.float32, 1)
    _out(sf, "sf", torch.uint8, sf_mma_bytes(rows, cols, batch))
    if gscale_in is not None:
        _out(gscale_in, "gscale_in", torch.float32, 1)
    _check(lib().nvfp4_quantize_mma(_ptr(x), batch, rows, cols, _dt(x), f_lo, f_hi, _ptr(gscale_in), _ptr(codes),
                                    _ptr(sf), _ptr(gscale), _stream(x)))
    return codes, sf, gscale


def quantize_mma_t(x: torch.Tensor, f_lo: int = -2, f_hi: int = 6, gscale_in: torch.Tensor | None = None,
                   codes: torch.Tensor | None = None, sf: torch.Tensor | None = None,
                   gscale: torch.Tensor | None = None):
    """Quantize x [rows, cols] or [batch, rows, cols] in blocks of 16 rows per column, written transposed:
    codes uint8[..., cols, rows/2], sf (tile layout of the [cols, rows] matrices), gscale float32[1]."""
    _cuda(x, "x")
    if x.dim() not in (2, 3):
        raise ValueError("x must be [rows, cols] or [batch, rows, cols]")
    batch, rows, cols = (1, *x.shape) if x.dim() == 2 else x.shape
    dev = x.device
    if codes is None:
        codes = torch.empty((*x.shape[:-2], cols, rows // 2), dtype=torch.uint8, device=dev)
    if sf is None:
        sf = torch.empty(sf_mma_bytes(cols, rows, batch), dtype=torch.uint8, device=dev)
    if gscale is None:
        gscale = torch.empty(1, dtype=torch.float32, device=dev)
    _out(codes, "codes", torch.uint8, x.numel() // 2), _out(gscale, "gscale", torch.float32, 1)
    _out(sf, "sf", torch.uint8, sf_mma_bytes(cols, rows, batch))
    if gscale_in is not None:
        _out(gscale_in, "gscale_in", torch.float32, 1)
    _check(lib().nvfp4_quantize_mma_t(_ptr(x), batch, rows, cols, _dt(x), f_lo, f_hi, _ptr(gscale_in), _ptr(codes),
                                      _ptr(sf), _ptr(gscale), _stream(x)))
    return codes, sf, gscale


def kv_mixed_mma(k: torch.Tensor, sink: int = 16, recent: int = 16, rotate: bool = True, f_lo: int = -2,
                 f_hi: int = 6, codes: torch.Tensor | None = None, sf: torch.Tensor | None = None,
                 gscale: torch.Tensor | None = None):
    """kv_mixed with the middle-token scales of every (batch, head) in the tensor-core tile layout.
    With sink = recent = 0 and rotate it is the rotated quantize of every token, fused (codes and scales
    as quantize_mma of the FWHT-16-rotated FP32 tensor).  codes / sf / gscale: optional preallocated outputs.

    Returns (sink, recent, codes uint8[B,H,Tm,D/2], sf uint8[sf_mma_bytes(Tm, D, B*H)], gscale)."""
    _cuda(k, "k")
    if k.dtype != torch.bfloat16 or k.dim() != 4:
        raise TypeError("k must be a 4-D bfloat16 tensor [B,H,T,D]")
    B, H, T, D = k.shape
    Tm = max(T - sink - recent, 0)
    dev = k.device
    so = torch.empty((B, H, sink, D), dtype=torch.bfloat16, device=dev)
    ro = torch.empty((B, H, recent, D), dtype=torch.bfloat16, device=dev)
    codes = torch.empty((B, H, Tm, D // 2), dtype=torch.uint8, device=dev) if codes is None else codes
    sf = torch.empty(max(sf_mma_bytes(Tm, D, B * H), 1), dtype=torch.uint8, device=dev) if sf is None else sf
    gscale = torch.empty(1, dtype=torch.float32, device=dev) if gscale is None else gscale
    for t, nm, need in ((codes, "codes", B * H * Tm * D // 2), (sf, "sf", sf_mma_bytes(Tm, D, B * H)),
                        (gscale, "gscale", 1)):
        _cuda(t, nm)
        if t.numel() < need:
            raise ValueError(f"{nm} holds {t.numel()} elements, {need} needed")
    _check(lib().nvfp4_kv_mixed_mma(_ptr(k), B, H, T, D, sink, recent, int(bool(rotate)), f_lo, f_hi, _ptr(so),
                                    _ptr(ro), _ptr(codes), _ptr(sf), _ptr(gscale), _stream(k)))
    return so, ro, codes, sf, gscale


def gemm_nt(a_codes: torch.Tensor, a_sf: torch.Tensor, a_gscale: torch.Tensor, b_codes: torch.Tensor,
            b_sf: torch.Tensor, b_gscale: torch.Tensor, alpha: float = 1.0, out_dtype=torch.float32,
            out: torch.Tensor | None = None, alpha_work: torch.Tensor | None = None) -> torch.Tensor:
    """D[l] = alpha * g_a * g_b * A[l] B[l]^T on the tensor cores (FP32 accumulation).

    a_codes: uint8 [M, K/2] or [batch, M, K/2] (quantize_mma output), b_codes: [.., N, K/2] likewise;
    returns D [M, N] or [batch, M, N] in out_dtype (float32 or bfloat16)."""
    for t, nm in ((a_codes, "a_codes"), (a_sf, "a_sf"), (a_gscale, "a_gscale"), (b_codes, "b_codes"),
                  (b_sf, "b_sf"), (b_gscale, "b_gscale")):
        _cuda(t, nm)
    squeeze = a_codes.dim() == 2
    a3 = a_codes if a_codes.dim() == 3 else a_codes.unsqueeze(0)
    b3 = b_codes if b_codes.dim() == 3 else b_codes.unsqueeze(0)
    batch, M, K2 = a3.shape
    if b3.shape[0] != batch or b3.shape[2] != K2:
        raise ValueError("a_codes and b_codes disagree on batch or K")
    N, K = b3.shape[1], 2 * K2
    dev = a_codes.device
    if a_codes.dtype != torch.uint8 or b_codes.dtype != torch.uint8:
        raise TypeError("a_codes and b_codes must be uint8")
    _out(a_sf, "a_sf", torch.uint8, sf_mma_bytes(M, K, batch) if M and K else 0)
    _out(b_sf, "b_sf", torch.uint8, sf_mma_bytes(N, K, batch) if N and K else 0)
    _out(a_gscale, "a_gscale", torch.float32, 1), _out(b_gscale, "b_gscale", torch.float32, 1)
    if out is None:
        out = torch.empty((batch, M, N), dtype=out_dtype, device=dev)
    _out(out, "out", None, batch * M * N)
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out must be float32 or bfloat16")
    if alpha_work is None:
        alpha_work = torch.empty(1, dtype=torch.float32, device=dev)
    _out(alpha_work, "alpha_work", torch.float32, 1)
    _check(lib().nvfp4_gemm_nt(_ptr(a_codes), _ptr(a_sf), _ptr(a_gscale), _ptr(b_codes), _ptr(b_sf), _ptr(b_gscale),
                               batch, M, N, K, float(alpha), _ptr(out), DTYPE_CODE[out.dtype], _ptr(alpha_work),
                               _stream(a_codes)))
    return out[0] if squeeze and out.dim() == 3 else out


def gemm_sf_offsets(rows: int, K: int, batch: int = 1):
    """Host-side: byte offsets at which gemm_nt reads scale (l, r, c), as a numpy int64 array."""
    import numpy as np
    out = np.empty(batch * rows * (K // 16), np.int64)
    _check(lib().nvfp4_gemm_sf_offsets(rows, K, batch, out.ctypes.data))
    return out


# ---- incremental KV cache (decode) ----
def kv_gscale(k: torch.Tensor, sink: int = 16, recent: int = 16, rotate: bool = True,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """Tensor scale over the (rotated) middle tokens of K[B,H,T,D] (BF16), as kv_mixed computes it."""
    _cuda(k, "k")
    if k.dtype != torch.bfloat16 or k.dim() != 4:
        raise TypeError("k must be a 4-D bfloat16 tensor [B,H,T,D]")
    B, H, T, D = k.shape
    out = torch.empty(1, dtype=torch.float32, device=k.device) if out is None else _out(out, "out", torch.float32, 1)
    _one_device(k.device, out=out)
    _launch(k.device, lib().nvfp4_kv_gscale, _ptr(k), B, H, T, D, sink, recent, int(bool(rotate)), _ptr(out))
    return out


def kv_append(k_rows: torch.Tensor, first: int, n: int, gscale: torch.Tensor, codes: torch.Tensor,
              scales: torch.Tensor, t0: int, rotate: bool = True, f_lo: int = -2, f_hi: int = 6,
              tile_layout: bool = False) -> None:
    """Quantize tokens [first, first+n) of k_rows [..., T, D] (BF16, contiguous; leading dims = batch x
    heads) with the tensor scale gscale into rows [t0, t0+n) of codes [..., cap, D/2] and scales
    ([..., cap, D/16], or the tile layout of the per-head [cap, D] matrices when tile_layout)."""
    for t, nm in ((k_rows, "k_rows"), (gscale, "gscale"), (codes, "codes"), (scales, "scales")):
        _cuda(t, nm)
    if k_rows.dtype != torch.bfloat16:
        raise TypeError("k_rows must be bfloat16")
    T, D = k_rows.shape[-2], k_rows.shape[-1]
    BH = k_rows.numel() // max(T * D, 1)
    cap = codes.shape[-2]
    _out(gscale, "gscale", torch.float32, 1), _out(codes, "codes", torch.uint8, BH * cap * (D // 2))
    _out(scales, "scales", torch.uint8, sf_mma_bytes(cap, D, BH) if tile_layout else BH * cap * (D // 16))
    _one_device(k_rows.device, gscale=gscale, codes=codes, scales=scales)
    _launch(k_rows.device, lib().nvfp4_kv_append, _ptr(k_rows), BH, T, first, n, D, int(bool(rotate)), f_lo, f_hi, _ptr(gscale),
            _ptr(codes), _ptr(scales), cap, t0, 1 if tile_layout else 0)


class _KvAppendDesc(ctypes.Structure):
    """nvfp4_kv_append_desc (include/nvfp4.h)."""
    _fields_ = [("k_bf16", _P), ("gscale", _P), ("codes", _P), ("scales", _P), ("BH", _I64), ("T", _I64),
                ("first", _I64), ("n", _I64), ("D", _I64), ("cap", _I64), ("t0", _I64),
                ("rotate", ctypes.c_int32), ("scale_layout", ctypes.c_int32)]


KV_APPEND_BATCH_MAX = 64


class KvAppendBatch:
    """A prepared nvfp4_kv_append_batch over fixed caches: `caches` is a sequence of tuples
    (k_rows, gscale, codes, scales, rotate, tile_layout) with kv_append's meanings, validated once (at most
    64, every tensor on one device; the tensors are kept alive).  Each call sets only the rows: first, n and t0 (an int for every item,
    or one value per item; n = 0 skips an item) and launches once.  Outputs of different items must not
    overlap."""

    def __init__(self, caches, f_lo: int = -2, f_hi: int = 6):
        caches = list(caches)
        if len(caches) > KV_APPEND_BATCH_MAX:
            raise ValueError(f"at most {KV_APPEND_BATCH_MAX} items per batch")
        self._keep, self.f_lo, self.f_hi = caches, f_lo, f_hi
        self._descs = (_KvAppendDesc * max(len(caches), 1))()
        self._device = None
        for i, (k_rows, gscale, codes, scales, rotate, tile_layout) in enumerate(caches):
            for t, nm in ((k_rows, "k_rows"), (gscale, "gscale"), (codes, "codes"), (scales, "scales")):
                _cuda(t, nm)
                # one launch on one device's stream reads and writes every item: all on that device
                self._device = self._device or t.device
                if t.device != self._device:
                    raise ValueError(f"item {i}: {nm} is on {t.device}, the batch runs on {self._device}")
            if k_rows.dtype != torch.bfloat16:
                raise TypeError("k_rows must be bfloat16")
            T, D = k_rows.shape[-2], k_rows.shape[-1]
            BH = k_rows.numel() // max(T * D, 1)
            cap = codes.shape[-2]
            _out(gscale, "gscale", torch.float32, 1), _out(codes, "codes", torch.uint8, BH * cap * (D // 2))
            _out(scales, "scales", torch.uint8, sf_mma_bytes(cap, D, BH) if tile_layout else BH * cap * (D // 16))
            self._descs[i] = _KvAppendDesc(k_rows.data_ptr(), gscale.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                                           BH, T, 0, 0, D, cap, 0, int(bool(rotate)), 1 if tile_layout else 0)
        self._count = len(caches)

    def __len__(self) -> int:
        return self._count

    def __call__(self, first, n, t0) -> None:
        if self._count == 0:
            return
        d = self._descs
        one = [isinstance(v, numbers.Integral) for v in (first, n, t0)]
        for i in range(self._count):
            d[i].first = int(first if one[0] else first[i])
            d[i].n = int(n if one[1] else n[i])
            d[i].t0 = int(t0 if one[2] else t0[i])
        _launch(self._device, lib().nvfp4_kv_append_batch, ctypes.cast(d, _P), self._count, self.f_lo, self.f_hi)


def kv_append_batch(items, f_lo: int = -2, f_hi: int = 6) -> None:
    """Several kv_append calls in one launch.  `items`: a sequence of tuples
    (k_rows, first, n, gscale, codes, scales, t0, rotate, tile_layout) with kv_append's meanings; all use
    the window [f_lo, f_hi] (at most 32 offsets).  Outputs of different items must not overlap."""
    items = list(items)
    if len(items) > KV_APPEND_BATCH_MAX:
        raise ValueError(f"at most {KV_APPEND_BATCH_MAX} items per batch")
    if not items:
        return
    b = KvAppendBatch([(it[0], it[3], it[4], it[5], it[7], it[8]) for it in items], f_lo, f_hi)
    b([it[1] for it in items], [it[2] for it in items], [it[6] for it in items])


# ---- MXFP4 (comparison format) ----
def mxfp4_quantize(x: torch.Tensor, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """MXFP4 (32-element blocks, E8M0 power-of-two scales).  Returns (codes uint8[n/2], scales uint8[n/32])."""
    _cuda(x, "x")
    n = x.numel()
    codes = torch.empty(n // 2, dtype=torch.uint8, device=x.device) if codes is None else _out(codes, "codes", torch.uint8, n // 2)
    scales = (torch.empty(n // 32, dtype=torch.uint8, device=x.device) if scales is None
              else _out(scales, "scales", torch.uint8, n // 32))
    _check(lib().nvfp4_mxfp4_quantize(_ptr(x), n, _dt(x), _ptr(codes), _ptr(scales), _stream(x)))
    return codes, scales


def mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, out_dtype=torch.float32,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    _cuda(scales, "scales")
    n = scales.numel() * 32
    _out(codes, "codes", torch.uint8, n // 2)
    out = torch.empty(n, dtype=out_dtype, device=codes.device) if out is None else _out(out, "out", None, n)
    _check(lib().nvfp4_mxfp4_dequantize(_ptr(codes), _ptr(scales), n, DTYPE_CODE[out.dtype], _ptr(out),
                                        _stream(codes)))
    return out


# ---- multi-scale deformable attention forward on NVFP4 (or full-precision) values ----
def msda_forward(value, shapes, loc: torch.Tensor, w: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """value: a tensor [bs, nkeys, heads, ch] (float32 / bfloat16 / float16), or the NVFP4 triple
    (codes uint8 [bs, nkeys, heads, ch/2], scales uint8 [bs, nkeys, heads, ch/16], gscale float32[1]);
    shapes: sequence of (H_l, W_l); loc [bs, nq, heads, L, P, 2] and w [bs, nq, heads, L, P] float32.
    Returns out [bs, nq, heads, ch] float32."""
    import numpy as np
    _cuda(loc, "loc"), _cuda(w, "w")
    sh = np.ascontiguousarray(np.asarray(shapes, np.int64).reshape(-1, 2))
    bs, nq, heads, L, P, _ = loc.shape
    if isinstance(value, (tuple, list)):
        codes, scales, gscale = value
        _, nkeys, _, ch2 = codes.shape
        ch = 2 * ch2
        _out(codes, "codes", torch.uint8, bs * nkeys * heads * ch2)
        _out(scales, "scales", torch.uint8, bs * nkeys * heads * (ch // 16)), _out(gscale, "gscale", torch.float32, 1)
    else:
        _cuda(value, "value")
        _, nkeys, _, ch = value.shape
        _out(value, "value", None, bs * nkeys * heads * ch)
    _out(loc, "loc", torch.float32, bs * nq * heads * L * P * 2), _out(w, "w", torch.float32, bs * nq * heads * L * P)
    if out is None:
        out = torch.empty((bs, nq, heads, ch), dtype=torch.float32, device=loc.device)
    _out(out, "out", torch.float32, bs * nq * heads * ch)
    shp = sh.ctypes.data
    if isinstance(value, (tuple, list)):
        _check(lib().nvfp4_msda_forward_nvfp4(_ptr(codes), _ptr(scales), _ptr(gscale), bs, nkeys, heads, ch, shp,
                                              L, P, nq, _ptr(loc), _ptr(w), _ptr(out), _stream(loc)))
    else:
        _check(lib().nvfp4_msda_forward(_ptr(value), _dt(value), bs, nkeys, heads, ch, shp, L, P, nq, _ptr(loc),
                                        _ptr(w), _ptr(out), _stream(loc)))
    return out


# ---- FP4 attention (ScaleSearchAttention numerics, unfused) ----
def softmax_quantize_mma(s: torch.Tensor, causal: bool = False, q_offset: int = 0, f_lo: int = -2, f_hi: int = 6,
                         codes=None, sf=None, g=None, m=None, l=None):
    """s float32 [batch, Tq, Tk] (or [Tq, Tk]).  Returns (codes [.., Tq, Tk/2], sf tile layout, gscale[1],
    row_max [batch*Tq], row_sum [batch*Tq]) for the softmax numerators P~ = exp(S - m); outputs may be given."""
    _cuda(s, "s")
    batch, Tq, Tk = (1, *s.shape) if s.dim() == 2 else s.shape
    dev = s.device
    if s.dtype != torch.float32:
        raise TypeError("s must be float32")
    codes = torch.empty((*s.shape[:-1], Tk // 2), dtype=torch.uint8, device=dev) if codes is None else codes
    sf = torch.empty(max(sf_mma_bytes(Tq, Tk, batch), 1), dtype=torch.uint8, device=dev) if sf is None else sf
    g = torch.empty(1, dtype=torch.float32, device=dev) if g is None else g
    m = torch.empty(batch * Tq, dtype=torch.float32, device=dev) if m is None else m
    l = torch.empty(batch * Tq, dtype=torch.float32, device=dev) if l is None else l
    _out(codes, "codes", torch.uint8, batch * Tq * (Tk // 2)), _out(sf, "sf", torch.uint8, sf_mma_bytes(Tq, Tk, batch))
    _out(g, "g", torch.float32, 1), _out(m, "m", torch.float32, batch * Tq), _out(l, "l", torch.float32, batch * Tq)
    _check(lib().nvfp4_softmax_quantize_mma(_ptr(s), batch, Tq, Tk, int(bool(causal)), q_offset, f_lo, f_hi,
                                            _ptr(codes), _ptr(sf), _ptr(g), _ptr(m), _ptr(l), _stream(s)))
    return codes, sf, g, m, l


def rows_divide(x: torch.Tensor, l: torch.Tensor) -> torch.Tensor:
    """In place: x[r, :] /= l[r] for x float32 [..., cols] viewed as rows."""
    _cuda(x, "x")
    if x.dtype != torch.float32:
        raise TypeError("x must be float32")
    cols = x.shape[-1]
    _out(l, "l", torch.float32, x.numel() // max(cols, 1))
    _check(lib().nvfp4_rows_divide(_ptr(x), _ptr(l), x.numel() // max(cols, 1), cols, _stream(x)))
    return x


def _prologue_operand(x: torch.Tensor, rotate: bool, signs: int, f_lo: int, f_hi: int):
    """Q or K [H, T, D] as an NVFP4 tensor-core operand, Hadamard-rotated along D when `rotate`.  BF16
    input without signs takes the fused path (rotation inside the amax and search kernels, no FP32 copy);
    the result is bit-identical to quantize_mma(hadamard16(x, float32))."""
    x = x.contiguous()
    if rotate and signs == 0 and x.dtype == torch.bfloat16:
        _, _, codes, sf, g = kv_mixed_mma(x[None], 0, 0, True, f_lo, f_hi)
        return codes[0], sf, g
    if rotate:
        x = hadamard16(x, out_dtype=torch.float32, signs=signs)
    return quantize_mma(x, f_lo, f_hi)


def attention_fused_splits(H: int, Tq: int, Tk: int) -> int:
    """The key-range count nvfp4_attention_fused_splits chooses for the current device."""
    s = ctypes.c_int(0)
    _check(lib().nvfp4_attention_fused_splits(H, Tq, Tk, ctypes.byref(s)))
    return s.value


def attention_fused_workspace(H: int, Tq: int, Tk: int, splits: int, device) -> torch.Tensor:
    """A workspace for nvfp4_attention_fused (uint8, nvfp4_attention_fused_workspace_bytes long)."""
    n = lib().nvfp4_attention_fused_workspace_bytes(H, Tq, Tk, splits)
    if n == 0:
        raise NVFP4Error(-2)
    return torch.empty(n, dtype=torch.uint8, device=device)


def attention_fused(qc, qsf, qg, kc, ksf, kg, vc_t, vsf_t, vg, causal: bool = False, q_offset: int = 0,
                    alpha: float = 1.0, f_lo: int = -2, f_hi: int = 6, verify: bool = False, out=None, m=None, l=None,
                    status=None, splits: int | None = None, workspace=None):
    """nvfp4_attention_fused on NVFP4 operands: q (codes [H, Tq, D/2], tile-layout scales, g), k likewise for
    [H, Tk, D], v transposed (codes [H, D, Tk/2] and the tile layout of [D, Tk] matrices, as quantize_mma_t
    gives them).  splits: key ranges per query tile (None: attention_fused_splits); workspace: a uint8 tensor
    of attention_fused_workspace's size (None: allocated here).  Returns (O [H, Tq, D] float32, row_max,
    row_sum), and with verify=True also the scores [H, Tq, Tk] and P~ (codes, tile-layout scales)."""
    for t_, nm in ((qc, "q codes"), (qsf, "q scales"), (qg, "q g"), (kc, "k codes"), (ksf, "k scales"), (kg, "k g"),
                   (vc_t, "v codes"), (vsf_t, "v scales"), (vg, "v g")):
        _cuda(t_, nm)
    H, Tq, D = qc.shape[0], qc.shape[1], 2 * qc.shape[2]
    Tk = kc.shape[1]
    dev = qc.device
    if splits is None:
        splits = attention_fused_splits(H, Tq, Tk)
    if workspace is None:
        workspace = attention_fused_workspace(H, Tq, Tk, splits, dev)
    _cuda(workspace, "workspace")
    out = torch.empty((H, Tq, D), dtype=torch.float32, device=dev) if out is None else out
    m = torch.empty(H * Tq, dtype=torch.float32, device=dev) if m is None else m
    l = torch.empty(H * Tq, dtype=torch.float32, device=dev) if l is None else l
    status = torch.zeros(1, dtype=torch.int32, device=dev) if status is None else status
    _out(out, "out", torch.float32, H * Tq * D), _out(m, "m", torch.float32, H * Tq)
    _out(l, "l", torch.float32, H * Tq), _out(status, "status", torch.int32, 1)
    s_out = p_codes = p_sf = None
    if verify:
        s_out = torch.zeros((H, Tq, Tk), dtype=torch.float32, device=dev)
        p_codes = torch.full((H, Tq, Tk // 2), 0xEE, dtype=torch.uint8, device=dev)   # every byte is written
        p_sf = torch.full((max(sf_mma_bytes(Tq, Tk, H), 1),), 0xEE, dtype=torch.uint8, device=dev)
    _check(lib().nvfp4_attention_fused(_ptr(qc), _ptr(qsf), _ptr(qg), _ptr(kc), _ptr(ksf), _ptr(kg), _ptr(vc_t),
                                       _ptr(vsf_t), _ptr(vg), H, Tq, Tk, D, float(alpha), int(bool(causal)), q_offset,
                                       f_lo, f_hi, int(splits), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                       _ptr(out), _ptr(m), _ptr(l), _ptr(s_out), _ptr(p_codes), _ptr(p_sf),
                                       _ptr(status), _stream(qc)))
    if verify:
        return out, m, l, s_out, p_codes, p_sf, status
    return out, m, l


def attention_fp4_fused(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False, rotate: bool = True,
                        scale: float | None = None, f_lo: int = -2, f_hi: int = 6, signs: int = 0):
    """attention_fp4 with the scores kept on chip: the same NVFP4 prologue (Q and K rotated and quantized into
    the tile layout, V quantized along the tokens), then nvfp4_attention_fused.  q [H, Tq, D], k and v
    [H, Tk, D] with D = 128, Tq % 128 == 0, Tk % 64 == 0.  Returns O [H, Tq, D] float32."""
    H, Tq, D = q.shape
    Tk = k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    qc, qsf, qg = _prologue_operand(q, rotate, signs, f_lo, f_hi)
    kc, ksf, kg = _prologue_operand(k, rotate, signs, f_lo, f_hi)
    vc, vsf, vg = quantize_mma_t(v.contiguous(), f_lo, f_hi)
    o, _, _ = attention_fused(qc.view(H, Tq, D // 2), qsf, qg, kc.view(H, Tk, D // 2), ksf, kg,
                              vc.view(H, D, Tk // 2), vsf, vg, causal, Tk - Tq, scale, f_lo, f_hi)
    return o


def attention_fp4(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False, rotate: bool = True,
                  scale: float | None = None, f_lo: int = -2, f_hi: int = 6, signs: int = 0):
    """Attention with every product in NVFP4 on the tensor cores ("Search your block floating-point
    scales!", ScaleSearchAttention; unfused): q [H, Tq, D], k and v [H, Tk, D].
      rotate: Hadamard-16 along D on q and k (Q K^T unchanged, outliers spread), after the sign
        diagonal given by the 16-bit mask `signs` (the same for both, so Q K^T is still unchanged);
      S = scale * Q K^T (NVFP4 x NVFP4, FP32 accumulation);  P~ = exp(S - rowmax) quantized with ScaleSearch;
      O = (P~ V) / rowsum with V quantized along the tokens.  Causal: query i sees keys <= i + Tk - Tq.
    Returns O [H, Tq, D] float32."""
    H, Tq, D = q.shape
    Tk = k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    qc, qsf, qg = _prologue_operand(q, rotate, signs, f_lo, f_hi)
    kc, ksf, kg = _prologue_operand(k, rotate, signs, f_lo, f_hi)
    s = gemm_nt(qc, qsf, qg, kc, ksf, kg, alpha=scale)
    pc, psf, pg, _, l = softmax_quantize_mma(s, causal, Tk - Tq, f_lo, f_hi)
    vc, vsf, vg = quantize_mma_t(v.contiguous(), f_lo, f_hi)
    o = gemm_nt(pc, psf, pg, vc, vsf, vg)
    return rows_divide(o, l)


# ---- decode: attention over the cache, rotary positions, cache pages ----
# the current stream's handle without a Stream object around it (5 us per call), where this torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _launch(device: torch.device, fn, *args) -> None:
    """fn(*args, stream) on `device` and its current stream: a kernel is launched on the current device, so
    that one is switched when the tensors live on another."""
    i = device.index
    if i == torch.cuda.current_device():
        rc = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _raw_stream(i))
    if rc:
        raise NVFP4Error(rc)


def _rows(t: torch.Tensor, name: str) -> torch.Tensor:
    """A CUDA tensor that is addressed by strides, its last dimension contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t


def _no_shared_elements(t: torch.Tensor, name: str) -> None:
    """An output's elements are written at the same time: none may be another's.  Every view that slicing, splitting and
    transposing give has strides that pass the reach of the smaller ones; others are taken as overlapping."""
    reach = 0
    for s, n in sorted((s, n) for n, s in zip(t.shape, t.stride()) if n > 1):
        if s <= reach and t.numel():
            raise ValueError(f"{name} must not be an expanded tensor or one whose rows overlap (it is written)")
        reach += (n - 1) * s


def _extent(t: torch.Tensor) -> tuple[int, int]:
    """First and past-the-last byte that t's elements occupy."""
    lo = hi = 0
    for n, s in zip(t.shape, t.stride()):
        if n == 0:
            return 0, 0
        if s < 0:
            lo += (n - 1) * s
        else:
            hi += (n - 1) * s
    e, p = t.element_size(), t.data_ptr()
    return p + lo * e, p + (hi + 1) * e


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two tensors may share elements.  Views of one buffer with the same strides (q, k and v side by side in
    a row) are told apart exactly; others by the bytes that they span."""
    (a0, a1), (b0, b1) = _extent(a), _extent(b)
    if not (a0 < b1 and b0 < a1):
        return False
    sizes = list(zip(a.shape, a.stride(), b.shape, b.stride()))
    e = a.element_size()
    off = b.data_ptr() - a.data_ptr()
    if a.dim() != b.dim() or e != b.element_size() or off % e or any(na > 1 and nb > 1 and sa != sb for na, sa, nb, sb in sizes):
        return True
    # b's element j is a's element i where sum (i_d - j_d) stride_d is the distance of their first ones
    dims = sorted(((sa if na > 1 else sb, 1 - nb, na - 1) for na, sa, nb, sb in sizes if (na > 1 or nb > 1) and (sa if na > 1 else sb)),
                  reverse=True)
    reach = [(0, 0)]
    for s, lo, hi in reversed(dims):
        reach.append((reach[-1][0] + lo * s, reach[-1][1] + hi * s))
    reach.reverse()

    def hits(d: int, left: int) -> bool:
        if d == len(dims):
            return left == 0
        s, lo, hi = dims[d]
        r_lo, r_hi = reach[d + 1]
        return any(hits(d + 1, left - i * s) for i in range(max(lo, -(-(left - r_hi) // s)), min(hi, (left - r_lo) // s) + 1))
    return hits(0, off // e)


class _KvStore(ctypes.Structure):
    """nvfp4_kv_store (include/nvfp4.h)."""
    _fields_ = [("sink", _P), ("window", _P), ("codes", _P), ("scales", _P), ("gscale", _P), ("gscale_stride", _I64),
                ("rotate", ctypes.c_int32), ("scale_layout", ctypes.c_int32)]


class _KvAttentionDesc(ctypes.Structure):
    """nvfp4_kv_attention_desc (include/nvfp4.h)."""
    _fields_ = [("q", _P), ("out", _P), ("lse", _P),
                *((n, _I64) for n in ("q_sb", "q_sh", "q_st", "out_sb", "out_sh", "out_st", "B", "Hq", "Hkv", "Tq", "D")),
                ("k", _KvStore), ("v", _KvStore),
                *((n, _I64) for n in ("slots", "sink_rows", "window_rows", "pages", "page_rows", "table_cols")),
                ("slot", _P), ("table", _P), ("lens", _P),
                *((n, ctypes.c_int32) for n in ("n_sink", "n_mid", "head", "n_window", "dtype", "causal")),
                ("scale", ctypes.c_float)]


# The same record packed in one go (setting its fields one by one takes 2.5 us of a call's 15).
_KV_ATTENTION = struct.Struct("@3Q11q%ds%ds6q3Q6if0q" % (2 * (ctypes.sizeof(_KvStore),)))
assert _KV_ATTENTION.size == ctypes.sizeof(_KvAttentionDesc)


class KvStore:
    """One side (K or V) of a mixed-precision cache as kv_attention reads it, checked once: sink [slots, H, s, D]
    and window [slots, H, w, D] (BF16; zero rows if there are none), codes uint8 [pages, H, rows, D/2], scales
    uint8 [pages, H, rows, D/16] (or the tile layout of the pages * H matrices [rows, D]), gscale float32 [1]
    or [slots].  The tensors are kept alive; their contents are read at each call."""

    def __init__(self, sink: torch.Tensor, window: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                 gscale: torch.Tensor, rotate: bool = True, tile_layout: bool = False):
        for t, nm in ((sink, "sink"), (window, "window"), (codes, "codes"), (scales, "scales"), (gscale, "gscale")):
            _cuda(t, nm)
            if t.device != codes.device:
                raise ValueError(f"{nm} is on {t.device}, codes on {codes.device}")
        if sink.dtype != torch.bfloat16 or window.dtype != torch.bfloat16:
            raise TypeError("sink and window must be bfloat16")
        if codes.dtype != torch.uint8 or codes.dim() != 4 or sink.dim() != 4 or window.dim() != 4:
            raise TypeError("codes must be 4-D uint8 [pages, H, rows, D/2], sink and window 4-D [slots, H, rows, D]")
        pages, H, rows, D = codes.shape[0], codes.shape[1], codes.shape[2], 2 * codes.shape[3]
        S = sink.shape[0]
        if sink.shape[1] != H or sink.shape[3] != D or window.shape[:2] != (S, H) or window.shape[3] != D:
            raise ValueError("sink, window and codes disagree on slots, heads or head_dim")
        if D % 16:
            raise ValueError("head_dim must be a multiple of 16")
        _out(scales, "scales", torch.uint8, sf_mma_bytes(rows, D, pages * H) if tile_layout else pages * H * rows * (D // 16))
        _out(gscale, "gscale", torch.float32, 1)
        if gscale.numel() not in (1, S):
            raise ValueError("gscale must hold one value, or one per slot")
        self.slots, self.H, self.D, self.pages, self.page_rows = S, H, D, pages, rows
        self.sink_rows, self.window_rows, self.device = sink.shape[2], window.shape[2], codes.device
        self.geometry = (S, H, D, pages, rows, self.sink_rows, self.window_rows, codes.device)
        self._keep = (sink, window, codes, scales, gscale)
        self._desc = bytes(_KvStore(*(t.data_ptr() for t in self._keep), 1 if gscale.numel() > 1 else 0, int(bool(rotate)),
                                    int(bool(tile_layout))))


_kv_splits_memo: dict = {}


def _kv_splits(device: torch.device, B: int, H: int, rows: int, D: int, max_mid: int) -> tuple[int, int]:
    """(splits, workspace bytes) that nvfp4_kv_attention_splits gives for these sizes (a pure function of them
    and the device, remembered)."""
    key = (device.index, B, H, rows, D, max_mid)
    got = _kv_splits_memo.get(key)
    if got is None:
        s = ctypes.c_int(0)
        with torch.cuda.device(device):
            _check(lib().nvfp4_kv_attention_splits(B, H, rows, D, max_mid, ctypes.byref(s)))
        if len(_kv_splits_memo) > 4096:
            _kv_splits_memo.clear()
        got = _kv_splits_memo[key] = (s.value, lib().nvfp4_kv_attention_workspace_bytes(rows, D, s.value))
    return got


def kv_attention(q: torch.Tensor, k: KvStore, v: KvStore, lens, table: torch.Tensor | None = None,
                 slots: torch.Tensor | None = None, causal: bool = True, scale: float | None = None,
                 max_mid: int | None = None, want_lse: bool = False, out: torch.Tensor | None = None,
                 lse: torch.Tensor | None = None, splits: int | None = None, workspace: torch.Tensor | None = None):
    """Attention of the newest Tq tokens of every sequence over its cached tokens (those Tq included), reading the
    NVFP4 middle where it lies.

    q: bfloat16 / float16 [B, Hq, Tq, D] (any strides, D contiguous), D 64, 128 or 256, Hq a multiple of the
    stores' H (query head h reads K/V head h // (Hq // H)).
    lens: (n_sink, n_mid, head, n_window) for every slot, or an int32 device tensor [slots, 4] read by the kernel.
    table: int32 [slots, cols], the page of each run of `rows` middle tokens (rows a multiple of 16); None: slot s
    owns page s.  slots: int32 [B], the slot of each batch row (outside [0, slots): an empty sequence); None: row
    b is slot b.  causal: query i of Tq sees positions <= length - Tq + i.
    max_mid: a bound on the middle's length that sizes the work split when lens is on the device (any value
    gives a correct result).  splits / workspace: nvfp4_kv_attention_splits' choice and an own allocation by default.
    out, lse and workspace share no memory with q or one another.  The result carries no gradient.
    Returns out [B, Hq, Tq, D] in q's dtype, or (out, lse float32 [B, Hq, Tq]) with want_lse."""
    _rows(q, "q")
    if q.dim() != 4:
        raise ValueError("q must be [B, Hq, Tq, D]")
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("q must be bfloat16 or float16")
    if not isinstance(k, KvStore) or not isinstance(v, KvStore):
        raise TypeError("k and v must be KvStore")
    if k.geometry != v.geometry:
        raise ValueError("k and v stores disagree on their sizes or device")
    B, Hq, Tq, D = q.shape
    if D not in (64, 128, 256):
        raise ValueError("head_dim must be 64, 128 or 256")
    dev = q.device
    if D != k.D or dev != k.device:
        raise ValueError("q and the stores disagree on head_dim or device")
    if k.H == 0 or Hq % k.H:
        raise ValueError("query heads must be a multiple of the K/V heads")
    rows = Hq // k.H * Tq
    most, cols, table_at, lens_at, slots_at, ends = k.page_rows, 0, 0, 0, 0, (0, 0, 0, 0)
    if table is not None:
        _cuda(table, "table")
        if table.dtype != torch.int32 or table.dim() != 2 or table.shape[0] != k.slots or table.device != dev:
            raise ValueError("table must be int32 [slots, cols] on q's device")
        table_at, cols = table.data_ptr(), table.shape[1]
        most *= cols
        if cols == 0:
            raise ValueError("table has no columns")
    elif k.pages < k.slots:
        raise ValueError("without a table every slot needs its own page")
    if isinstance(lens, torch.Tensor):
        _cuda(lens, "lens")
        if lens.dtype != torch.int32 or lens.shape != (k.slots, 4) or lens.device != dev:
            raise ValueError("lens must be int32 [slots, 4] on q's device")
        lens_at = lens.data_ptr()
        hint = most if max_mid is None else min(max(int(max_mid), 0), most)
    else:
        _, hint, _, _ = ends = tuple(lens)
        if min(ends) < 0 or max(ends) >> 31:
            raise ValueError("lengths are 32-bit and not negative")
    if slots is not None:
        _cuda(slots, "slots")
        if slots.dtype != torch.int32 or slots.shape != (B,) or slots.device != dev:
            raise ValueError("slots must be int32 [B] on q's device")
        slots_at = slots.data_ptr()
    elif B > k.slots:
        raise ValueError("more batch rows than slots")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _rows(out, "out")
        if out.shape != q.shape or out.dtype != q.dtype or out.device != dev:
            raise ValueError("out must have q's shape, dtype and device")
        _no_shared_elements(out, "out")
        if _overlap(out, q):
            raise ValueError("out must not overlap q")
    if lse is not None:
        _out(lse, "lse", torch.float32, B * Hq * Tq)
        if lse.device != dev:
            raise ValueError("lse must be on q's device")
        if _overlap(lse, q) or _overlap(lse, out):
            raise ValueError("lse must not overlap q or out")
    elif want_lse:
        lse = q.new_empty((B, Hq, Tq), dtype=torch.float32)
    if splits is None:
        splits, need = _kv_splits(dev, B, k.H, rows, D, max(hint, 0))
    else:
        splits = int(splits)
        need = lib().nvfp4_kv_attention_workspace_bytes(rows, D, splits)
    if workspace is None:
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _cuda(workspace, "workspace")
        if workspace.device != dev or workspace.numel() * workspace.element_size() < need:
            raise ValueError(f"workspace must hold {need} bytes on q's device")
        if any(_overlap(workspace, t) for t in (q, out, lse) if t is not None):
            raise ValueError("workspace must not overlap q, out or lse")
    q_sb, q_sh, q_st, _ = q.stride()
    o_sb, o_sh, o_st, _ = out.stride()
    desc = _KV_ATTENTION.pack(
        q.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(), q_sb, q_sh, q_st, o_sb, o_sh, o_st, B, Hq, k.H, Tq, D,
        k._desc, v._desc, k.slots, k.sink_rows, k.window_rows, k.pages, k.page_rows, cols, slots_at, table_at, lens_at, *ends,
        DTYPE_CODE[q.dtype], 1 if causal else 0, D ** -0.5 if scale is None else scale)
    _launch(dev, lib().nvfp4_kv_attention, desc, splits, None if workspace is None else workspace.data_ptr(),
            need if workspace is not None else 0)
    return (out, lse) if want_lse else out


def rope_frequencies(rot: int, base: float = 10000.0, scaling: dict | None = None, device="cuda") -> tuple[torch.Tensor, float]:
    """(freqs float64 [rot / 2] in radians per position, mscale) for rope: base^(-2 i / rot), stretched for contexts
    longer than the trained one by `scaling`:
      {"type": "linear", "factor"}: every angle divided by factor (arXiv 2306.15595);
      {"type": "ntk", "factor"}: base * factor^(rot / (rot - 2)), so that the lowest frequency is divided by factor;
      {"type": "yarn", "factor", "original", "fast": 32, "slow": 1}: pairs that turn more than `fast` times in
        `original` positions kept, fewer than `slow` divided by factor, a linear ramp over the pairs between;
        mscale = 0.1 ln(factor) + 1 (arXiv 2309.00071);
      {"type": "bands", "factor", "original", "low": 1, "high": 4}: the same idea with the ramp linear in the turns."""
    if rot < 0 or rot % 2:
        raise ValueError("rot must be even")
    i = torch.arange(rot // 2, dtype=torch.float64)
    s = dict(scaling or {})
    kind, factor = s.get("type"), float(s.get("factor", 1.0))
    if kind not in (None, "linear", "ntk", "yarn", "bands"):
        raise ValueError(f"unknown scaling type {kind!r}")
    if not base > 1.0 or not factor >= 1.0:
        raise ValueError("base must exceed 1 and factor be at least 1")
    if kind == "ntk":
        if rot <= 2:
            raise ValueError("ntk scaling needs rot > 2")
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / max(rot, 1))
    mscale = 1.0
    if kind == "linear":
        f = f / factor
    elif kind in ("yarn", "bands"):
        if not float(s.get("original", 0)) > 0:
            raise ValueError(f"{kind} scaling needs the original context length")
        n = float(s["original"])
        if kind == "yarn":
            def pair(turns):   # the (fractional) pair that turns so often in n positions
                return rot * math.log(n / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo = max(math.floor(pair(float(s.get("fast", 32.0)))), 0)
            hi = min(math.ceil(pair(float(s.get("slow", 1.0)))), rot - 1)
            cut = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
            mscale = 0.1 * math.log(factor) + 1.0
        else:
            low, high = float(s.get("low", 1.0)), float(s.get("high", 4.0))
            if not high > low:
                raise ValueError("bands scaling needs high > low")
            cut = 1 - ((n * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f / factor * cut + f * (1 - cut)
    return f.to(device), mscale


class _RopeTensor(ctypes.Structure):
    """nvfp4_rope_tensor (include/nvfp4.h)."""
    _fields_ = [("x", _P), ("out", _P), *((n, _I64) for n in ("heads", "x_sb", "x_sh", "x_st", "out_sb", "out_sh", "out_st"))]


_ROPE_TENSOR = struct.Struct("@2Q7q")     # the same, packed in one go
assert _ROPE_TENSOR.size == ctypes.sizeof(_RopeTensor)
ROPE_MAX = 8


def rope(x, positions, freqs: torch.Tensor, interleaved: bool = False, mscale: float = 1.0, inverse: bool = False,
         out=None):
    """Rotary positions for x [B, heads, T, D] (or [heads, T, D]; any strides, D contiguous), or for a sequence of up
    to 8 such tensors (q and k of a step) in one launch; float32 / bfloat16 / float16, one dtype per call.

    positions: int32 / int64 device tensor [T] or [B, T].  freqs: float64 device tensor [rot / 2], radians per
    position (rope_frequencies); channels from rot on pass unchanged.  Pairs are (i, i + rot/2), or (2i, 2i + 1) when
    interleaved.  inverse=True turns back: with the same mscale the adjoint, the gradient's pass.
    out: None (new contiguous tensors), or what x is, with the same shapes; x itself for in place.
    Gradients reach x (by the inverse), not positions or freqs; a call with out= records none and is refused where one is
    asked for.
    Returns a tensor, or a list for a sequence."""
    one = isinstance(x, torch.Tensor)
    xs = [x] if one else list(x)
    if not xs or len(xs) > ROPE_MAX:
        raise ValueError(f"1 to {ROPE_MAX} tensors per call")
    given = out is not None
    outs = ([out] if one else list(out)) if given else [None] * len(xs)
    if len(outs) != len(xs):
        raise ValueError("one output per tensor")
    x0 = _rows(xs[0], "x")
    dev, dtype, dt, nd = x0.device, x0.dtype, _dt(x0), x0.dim()
    if nd not in (3, 4):
        raise ValueError("x must be [B, heads, T, D] or [heads, T, D]")
    s0 = x0.shape
    B, T, D = s0[0] if nd == 4 else 1, s0[-2], s0[-1]
    _cuda(freqs, "freqs")
    if freqs.dtype != torch.float64 or freqs.dim() != 1 or freqs.device != dev:
        raise TypeError("freqs must be a 1-D float64 tensor on x's device")
    rot = 2 * freqs.shape[0]
    if rot > D:
        raise ValueError("freqs holds more pairs than x has channels")
    if not isinstance(positions, torch.Tensor) or positions.dtype not in (torch.int32, torch.int64) or not positions.is_cuda:
        raise TypeError("positions must be an int32 or int64 CUDA tensor")
    pos_shape, ps = positions.shape, positions.stride()
    if pos_shape not in ((T,), (B, T)) or positions.device != dev:
        raise ValueError("positions must be [T] or [B, T] on x's device")
    if torch.is_grad_enabled():
        if freqs.requires_grad:
            raise ValueError("freqs get no gradient: detach them")
        asked = [a for a in (xs + outs if given else xs) if a.requires_grad]
        if asked and given:
            raise ValueError("a call with out= records no gradient: call it under no_grad, or without out")
        if asked:
            outs = list(_Rope.apply(positions, freqs, interleaved, mscale, inverse, *xs))
            return outs[0] if one else outs
    descs = []
    for j, a in enumerate(xs):
        if j:
            _rows(a, "x")
            s = a.shape
            if len(s) != nd or s[-2] != T or s[-1] != D or (nd == 4 and s[0] != B) or a.dtype != dtype or a.device != dev:
                raise ValueError("the tensors of a call share batch, length, head_dim, dtype and device")
        else:
            s = s0
        sx = a.stride()
        if not given:
            o = outs[j] = torch.empty_like(a, memory_format=torch.contiguous_format)
        else:
            o = _rows(outs[j], "out")
            if o.shape != s or o.dtype != dtype or o.device != dev:
                raise ValueError("out must have x's shape, dtype and device")
            _no_shared_elements(o, "out")
            if any(_overlap(o, outs[i]) for i in range(j)):
                raise ValueError("two outputs share elements")
            same = o.data_ptr() == a.data_ptr() and o.stride() == sx
            if any(_overlap(o, b) for i, b in enumerate(xs) if not (same and i == j)):
                raise ValueError("out must be x itself or not overlap any x")
        x_st, o_st = (sx, o.stride()) if nd == 4 else ((0, *sx), (0, *o.stride()))
        descs.append(_ROPE_TENSOR.pack(a.data_ptr(), o.data_ptr(), s[-3], *x_st[:3], *o_st[:3]))
    _launch(dev, lib().nvfp4_rope, b"".join(descs), len(xs), B, T, D, rot, 1 if interleaved else 0, dt, positions.data_ptr(),
            1 if positions.dtype == torch.int64 else 0, ps[0] if len(ps) == 2 else 0, ps[-1], freqs.data_ptr(), mscale,
            1 if inverse else 0)
    return outs[0] if one else outs


class _Rope(torch.autograd.Function):
    """rope with its gradient: the map is linear in x and its adjoint is the inverse with the same mscale."""

    @staticmethod
    def forward(ctx, positions, freqs, interleaved, mscale, inverse, *xs):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(positions, freqs)
        ctx.how = (interleaved, mscale, not inverse)
        return tuple(rope(xs, positions, freqs, interleaved, mscale, inverse))

    @staticmethod
    def backward(ctx, *grads):
        need = [n and g is not None for n, g in zip(ctx.needs_input_grad[5:], grads)]
        gs = [g if g.shape[-1] < 2 or g.stride(-1) == 1 else g.contiguous() for g, n in zip(grads, need) if n]
        got = iter(rope(gs, *ctx.saved_tensors, *ctx.how) if gs else ())
        return (None,) * 5 + tuple(next(got) if n else None for n in need)


class _PagesArray(ctypes.Structure):
    """nvfp4_pages_array (include/nvfp4.h)."""
    _fields_ = [("base", _P), ("outer", _I64), ("stride", _I64), ("item", _I64), ("pages", _I64)]


PAGES_MAX = 16


def copy_pages(arrays, src, dst) -> None:
    """Copies page src[j] to page dst[j] in every array, in one launch per 1024 pairs.  arrays: up to 16 pairs
    (tensor, dim): a contiguous CUDA tensor of any dtype whose dimension `dim` counts pages.  src, dst: host
    integers (sequences); all pairs move at once, so every dst is distinct and none of them is a src."""
    arrays = list(arrays)
    if len(arrays) > PAGES_MAX:
        raise ValueError(f"at most {PAGES_MAX} arrays per call")
    if len(src) != len(dst):
        raise ValueError("src and dst differ in length")
    if not arrays or not len(src):
        return
    descs = (_PagesArray * len(arrays))()
    dev = arrays[0][0].device
    for j, (t, dim) in enumerate(arrays):
        _cuda(t, f"array {j}")
        if t.device != dev:
            raise ValueError(f"array {j} is on {t.device}, the call runs on {dev}")
        if not -t.dim() <= dim < t.dim():
            raise ValueError(f"array {j} has no dimension {dim}")
        dim %= t.dim()
        outer, pages = math.prod(t.shape[:dim]), t.shape[dim]
        item = math.prod(t.shape[dim + 1:]) * t.element_size()
        descs[j] = _PagesArray(t.data_ptr(), outer, pages * item, item, pages)
    spans = sorted((d.base, d.base + d.outer * d.stride) for d in descs if d.outer * d.stride)
    if any(b[0] < a[1] for a, b in zip(spans, spans[1:])):
        raise ValueError("two arrays overlap")
    s, d = (array.array("i", list(v)) for v in (src, dst))
    _launch(dev, lib().nvfp4_copy_pages, descs, len(arrays), s.buffer_info()[0], d.buffer_info()[0], len(s))
