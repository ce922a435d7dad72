"""KroQuant online activation quantizer for NVIDIA B200 (sm_100a).

Thin Python binding over the C ABI of ``include/kroquant.h`` (the shared
library ``libkroquant.so`` built in-tree by ``w4a4_mxfp4_post_b200.build``).
The functions below only marshal arguments: they check dtypes, devices and
shapes of torch tensors, allocate outputs when none are given, and pass raw
device pointers and the current CUDA stream to the library.  Every step of
the computation runs in the library's CUDA kernels; there is no fallback, and
every function raises if the library is missing or returns an error.

    codes, scales = kq_quantize(act, factors)            # [M, d/2], [M, d/32] uint8
    codes, scales = kq_quantize_shared(act, factors5)
    codes, scales = sq_quantize(act, mult)
    codes, scales = mx_quantize(act)
    W_folded      = kq_fold_weights(W, factors, shared=False)
    y             = kq_transform_f32(act, factors, shared=False)

W4A4 consumer (scales in the tensor core's scale-factor layout):

    codes, sf     = kq_quantize_sf(act, factors)         # [M, d/2], [kq_sf_bytes(M, d)] uint8
    wcodes, wsf   = mx_quantize_f32(W_folded, sf_layout=True)
    out           = mxf4_gemm(codes, sf, wcodes, wsf)    # bf16 [M, N] = X W^T, W4A4

A few tokens at a time (a 4-bit layer that answers):

    y   = mxf4_gemv(x, wcodes, wsf)                      # bf16 [M, N], M <= 32, x bf16 as it is
    mx_cache_write(k, v, *cache, table, cu, lens)        # cache: k and v codes and scales, in pages
    o   = mx_paged_attention(q, *cache, table, cu, lens) # bf16 [T, heads_q, head_dim]
    k, v = mx_cache_read(*cache, table, cu_k, rows)      # bf16 [rows, heads, head_dim]
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

__all__ = [
    "LIB_PATH", "KQ_OK", "KQ_ERR_NULL", "KQ_ERR_SHAPE", "KQ_ERR_ALIGN", "KQ_ERR_CUDA", "KQ_ERR_VARIANT",
    "KroQuantError", "lib", "kq_quantize", "kq_quantize_shared", "kq_quantize_variant", "sq_quantize",
    "mx_quantize", "kq_fold_weights", "kq_transform_f32", "kq_last_error", "kq_abi_version",
    "sq_quantize_variant", "mx_quantize_variant", "kq_wait_timeouts", "kq_selftest_bounded_wait",
    "kq_transform_f32_variant", "kq_quantize_lu", "fwht_quantize", "kq_inverse_f32", "mx_dequantize", "norm_kq_quantize",
    "KQ_SCALES_ROWMAJOR", "KQ_SCALES_SF", "kq_sf_bytes", "kq_quantize_sf", "mx_quantize_f32", "mx_scales_to_sf",
    "mxf4_gemm", "mxf4_gemm_variant", "norm_kq_quantize_sf", "norm_kq_quantize_variant",
    "mxf4_gemv", "mxf4_gemv_workspace", "mx_cache_write", "mx_cache_read", "mx_paged_attention", "mx_attention_workspace",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkroquant.so")

KQ_OK, KQ_ERR_NULL, KQ_ERR_SHAPE, KQ_ERR_ALIGN, KQ_ERR_CUDA, KQ_ERR_VARIANT = 0, -1, -2, -3, -4, -5
KQ_SCALES_ROWMAJOR, KQ_SCALES_SF = 0, 1

# Entry points and their argument types (p = pointer, i = int, q = int64, f = float).
_SIGS = {
    "kq_quantize": "ppppqqp",
    "kq_quantize_shared": "ppppqqp",
    "kq_quantize_variant": "ippippqqp",
    "sq_quantize_variant": "ippppqqp",
    "mx_quantize_variant": "ipppqqp",
    "kq_selftest_bounded_wait": "p",
    "sq_quantize": "ppppqqp",
    "mx_quantize": "pppqqp",
    "kq_fold_weights": "ppipqqp",
    "kq_transform_f32": "ppipqqp",
    "kq_transform_f32_variant": "ippipqqp",
    "kq_quantize_lu": "ppippqqp",
    "fwht_quantize": "pqppqqp",
    "kq_inverse_f32": "ppipqqp",
    "mx_dequantize": "pppqqp",
    "kq_quantize_sf": "ppippqqp",
    "mx_quantize_f32": "pppiqqp",
    "mx_scales_to_sf": "ppqqp",
    "mxf4_gemm": "pppppiqqqp",
    "mxf4_gemm_variant": "ipppppiqqqp",
    "mxf4_gemv": "pqpppiqqqpqp",
    "mx_cache_write": "pqqpqqippqp",
    "mx_cache_read": "pppppiqp",
    "mx_paged_attention": "pqqppfipqqqpqp",
}

_lib = None


class KroQuantError(RuntimeError):
    """A non-OK status from the library, with its status code and message."""

    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded C library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"KroQuant CUDA library not found at {LIB_PATH}; build it with "
                "`python -m w4a4_mxfp4_post_b200.build` (there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        kinds = {"p": ctypes.c_void_p, "i": ctypes.c_int, "q": ctypes.c_int64, "f": ctypes.c_float}
        for name, sig in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = [kinds[c] for c in sig]
            fn.restype = ctypes.c_int
        L.kq_last_error.argtypes = []
        L.kq_last_error.restype = ctypes.c_char_p
        L.kq_abi_version.argtypes = []
        L.kq_abi_version.restype = ctypes.c_int
        L.kq_wait_timeouts.argtypes = [ctypes.POINTER(ctypes.c_int), ctypes.c_int]
        L.kq_wait_timeouts.restype = ctypes.c_int
        L.norm_kq_quantize.argtypes = [ctypes.c_void_p] * 3 + [ctypes.c_int64, ctypes.c_float, ctypes.c_void_p,
                                                                ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                                                ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p]
        L.norm_kq_quantize.restype = ctypes.c_int
        L.norm_kq_quantize_sf.argtypes = L.norm_kq_quantize.argtypes
        L.norm_kq_quantize_sf.restype = ctypes.c_int
        L.norm_kq_quantize_variant.argtypes = [ctypes.c_int] + L.norm_kq_quantize.argtypes
        L.norm_kq_quantize_variant.restype = ctypes.c_int
        L.kq_sf_bytes.argtypes = [ctypes.c_int64, ctypes.c_int64]
        L.kq_sf_bytes.restype = ctypes.c_int64
        L.mxf4_gemv_workspace.argtypes = [ctypes.c_int64] * 3
        L.mxf4_gemv_workspace.restype = ctypes.c_int64
        L.mx_attention_workspace.argtypes = [ctypes.c_int64] * 5
        L.mx_attention_workspace.restype = ctypes.c_int64
        _lib = L
    return _lib


def kq_last_error() -> str:
    return lib().kq_last_error().decode()


def kq_abi_version() -> int:
    return lib().kq_abi_version()


def _call(name: str, device, *args) -> None:
    """Call entry point `name` with `device` (the tensors' device; None = the
    current one) as the current CUDA device: the library launches on the
    current device and caches its properties per device."""
    fn = getattr(lib(), name)
    if device is not None and device.index is not None and device.index != _torch().cuda.current_device():
        with _torch().cuda.device(device):
            rc = fn(*args)
    else:
        rc = fn(*args)
    if rc != KQ_OK:
        raise KroQuantError(name, rc, kq_last_error())


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


def _stream(stream, device):
    """The raw handle of `stream`, default the current stream of `device`; a
    torch stream must belong to `device`."""
    torch = _torch()
    if stream is None:
        raw = getattr(getattr(torch, "_C", None), "_cuda_getCurrentRawStream", None)
        if raw is not None and device is not None and device.index is not None:
            return ctypes.c_void_p(raw(device.index))        # without making a Stream object
        stream = torch.cuda.current_stream(device)
    elif isinstance(stream, torch.cuda.Stream) and device is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t) -> int:
    return t.data_ptr() if t is not None and t.numel() > 0 else 0


@functools.lru_cache(maxsize=1024)
def _sizes(name, *args) -> int:
    """What a size query of the library says (a function of its arguments alone)."""
    return getattr(lib(), name)(*args)


def _need(t, name, dtype, device=None, shape=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    # what calls give almost always, in as few steps as it takes
    if t.dtype is dtype and t.is_cuda and t.is_contiguous() and (device is None or t.device == device) and \
            (shape is None or t.shape == shape):
        return t
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _act(act):
    torch = _torch()
    _need(act, "act", torch.bfloat16)
    if act.dim() != 2:
        raise ValueError("act must be 2-D [M, d]")
    return act.shape


def _outs(act, out_codes, out_scales):
    torch = _torch()
    M, d = act.shape
    if out_codes is None:
        out_codes = torch.empty((M, d // 2), dtype=torch.uint8, device=act.device)
    if out_scales is None:
        out_scales = torch.empty((M, d // 32), dtype=torch.uint8, device=act.device)
    _need(out_codes, "out_codes", torch.uint8, act.device, (M, d // 2))
    _need(out_scales, "out_scales", torch.uint8, act.device, (M, d // 32))
    return out_codes, out_scales


def _factors(factors, d, shared, device):
    torch = _torch()
    _need(factors, "factors", torch.float32, device)
    n = 1 if shared else d // 32
    if factors.numel() != n * 20:
        raise ValueError(f"factors must hold {n} x 5 x 2 x 2 floats, got {tuple(factors.shape)}")
    return factors


def kq_quantize(act, factors, out_codes=None, out_scales=None, stream=None):
    """KroQuant quantizer with one factor set per 32-column block ([d/32, 5, 2, 2])."""
    M, d = _act(act)
    _factors(factors, d, False, act.device)
    out_codes, out_scales = _outs(act, out_codes, out_scales)
    _call("kq_quantize", act.device, _ptr(act), _ptr(factors), _ptr(out_codes), _ptr(out_scales), M, d,
          _stream(stream, act.device))
    return out_codes, out_scales


def kq_quantize_shared(act, factors, out_codes=None, out_scales=None, stream=None):
    """KroQuant quantizer with one factor set ([5, 2, 2]) for every block."""
    M, d = _act(act)
    _factors(factors, d, True, act.device)
    out_codes, out_scales = _outs(act, out_codes, out_scales)
    _call("kq_quantize_shared", act.device, _ptr(act), _ptr(factors), _ptr(out_codes), _ptr(out_scales), M, d,
          _stream(stream, act.device))
    return out_codes, out_scales


def kq_quantize_variant(variant, act, factors, shared=False, out_codes=None, out_scales=None, stream=None):
    """The KroQuant quantizer through a chosen kernel variant (0 = the default)."""
    M, d = _act(act)
    _factors(factors, d, shared, act.device)
    out_codes, out_scales = _outs(act, out_codes, out_scales)
    _call("kq_quantize_variant", act.device, int(variant), _ptr(act), _ptr(factors), int(bool(shared)), _ptr(out_codes),
          _ptr(out_scales), M, d, _stream(stream, act.device))
    return out_codes, out_scales


def sq_quantize(act, mult, out_codes=None, out_scales=None, stream=None):
    """SmoothQuant baseline: fp32(x * mult[c]) per channel, then MXFP4."""
    torch = _torch()
    M, d = _act(act)
    _need(mult, "mult", torch.float32, act.device, (d,))
    out_codes, out_scales = _outs(act, out_codes, out_scales)
    _call("sq_quantize", act.device, _ptr(act), _ptr(mult), _ptr(out_codes), _ptr(out_scales), M, d,
          _stream(stream, act.device))
    return out_codes, out_scales


def mx_quantize(act, out_codes=None, out_scales=None, stream=None):
    """Plain MXFP4 baseline (no transform)."""
    M, d = _act(act)
    out_codes, out_scales = _outs(act, out_codes, out_scales)
    _call("mx_quantize", act.device, _ptr(act), _ptr(out_codes), _ptr(out_scales), M, d, _stream(stream, act.device))
    return out_codes, out_scales


def kq_quantize_lu(act, lu_params, shared=False, out_codes=None, out_scales=None, stream=None):
    """KroQuant quantizer from 15 LU scalars per block ([d/32, 5, 3] or [5, 3] if shared)."""
    torch = _torch()
    M, d = _act(act)
    _need(lu_params, "lu_params", torch.float32, act.device)
    n = 1 if shared else d // 32
    if lu_params.numel() != n * 15:
        raise ValueError(f"lu_params must hold {n} x 5 x 3 floats, got {tuple(lu_params.shape)}")
    out_codes, out_scales = _outs(act, out_codes, out_scales)
    _call("kq_quantize_lu", act.device, _ptr(act), _ptr(lu_params), int(bool(shared)), _ptr(out_codes),
          _ptr(out_scales), M, d, _stream(stream, act.device))
    return out_codes, out_scales


def fwht_quantize(act, H, out_codes=None, out_scales=None, stream=None):
    """Fixed-Hadamard (block size H) baseline quantizer."""
    M, d = _act(act)
    out_codes, out_scales = _outs(act, out_codes, out_scales)
    _call("fwht_quantize", act.device, _ptr(act), int(H), _ptr(out_codes), _ptr(out_scales), M, d,
          _stream(stream, act.device))
    return out_codes, out_scales


def norm_kq_quantize(h, gamma, beta, factors, eps=1e-6, shared=False, out_codes=None, out_scales=None,
                     stream=None):
    """LayerNorm + AdaLN modulation (gamma, beta: [nsamples, d]) fused with kq_quantize."""
    return norm_kq_quantize_variant(0, h, gamma, beta, factors, eps, shared, out_codes, out_scales, stream)


def norm_kq_quantize_variant(variant, h, gamma, beta, factors, eps=1e-6, shared=False, out_codes=None,
                             out_scales=None, stream=None):
    """norm_kq_quantize through a chosen kernel (0 = the default)."""
    torch = _torch()
    M, d = _act(h)
    _need(gamma, "gamma", torch.float32, h.device)
    _need(beta, "beta", torch.float32, h.device, tuple(gamma.shape))
    if gamma.dim() != 2 or gamma.shape[1] != d:
        raise ValueError("gamma and beta must be [nsamples, d]")
    _factors(factors, d, shared, h.device)
    out_codes, out_scales = _outs(h, out_codes, out_scales)
    args = (_ptr(h), _ptr(gamma), _ptr(beta), int(gamma.shape[0]), float(eps), _ptr(factors), int(bool(shared)),
            _ptr(out_codes), _ptr(out_scales), M, d, _stream(stream, h.device))
    if variant == 0:
        _call("norm_kq_quantize", h.device, *args)
    else:
        _call("norm_kq_quantize_variant", h.device, int(variant), *args)
    return out_codes, out_scales


def kq_inverse_f32(y, factors, shared=False, out=None, stream=None):
    """x = T^-1 y per 32-block (fp32 [M, d])."""
    torch = _torch()
    _need(y, "y", torch.float32)
    if y.dim() != 2:
        raise ValueError("y must be 2-D [M, d]")
    M, d = y.shape
    _factors(factors, d, shared, y.device)
    if out is None:
        out = torch.empty_like(y)
    _need(out, "out", torch.float32, y.device, (M, d))
    _call("kq_inverse_f32", y.device, _ptr(y), _ptr(factors), int(bool(shared)), _ptr(out), M, d,
          _stream(stream, y.device))
    return out


def mx_dequantize(codes, scales, out=None, stream=None):
    """MXFP4 decode of codes [M, d/2] and scales [M, d/32] to fp32 [M, d]."""
    torch = _torch()
    _need(codes, "codes", torch.uint8)
    if codes.dim() != 2:
        raise ValueError("codes must be 2-D [M, d/2]")
    M, d = codes.shape[0], codes.shape[1] * 2
    _need(scales, "scales", torch.uint8, codes.device, (M, d // 32))
    if out is None:
        out = torch.empty((M, d), dtype=torch.float32, device=codes.device)
    _need(out, "out", torch.float32, codes.device, (M, d))
    _call("mx_dequantize", codes.device, _ptr(codes), _ptr(scales), _ptr(out), M, d, _stream(stream, codes.device))
    return out


def sq_quantize_variant(variant, act, mult, out_codes=None, out_scales=None, stream=None):
    """The SmoothQuant quantizer through a chosen kernel variant (0 = the default)."""
    torch = _torch()
    M, d = _act(act)
    _need(mult, "mult", torch.float32, act.device, (d,))
    out_codes, out_scales = _outs(act, out_codes, out_scales)
    _call("sq_quantize_variant", act.device, int(variant), _ptr(act), _ptr(mult), _ptr(out_codes), _ptr(out_scales), M,
          d, _stream(stream, act.device))
    return out_codes, out_scales


def mx_quantize_variant(variant, act, out_codes=None, out_scales=None, stream=None):
    """The plain MXFP4 quantizer through a chosen kernel variant (0 = the default)."""
    M, d = _act(act)
    out_codes, out_scales = _outs(act, out_codes, out_scales)
    _call("mx_quantize_variant", act.device, int(variant), _ptr(act), _ptr(out_codes), _ptr(out_scales), M, d,
          _stream(stream, act.device))
    return out_codes, out_scales


def kq_wait_timeouts(reset: bool = False) -> int:
    """Number of bounded waits that gave up in the staged kernels (synchronises the device)."""
    v = ctypes.c_int(0)
    rc = lib().kq_wait_timeouts(ctypes.byref(v), int(bool(reset)))
    if rc != KQ_OK:
        raise KroQuantError("kq_wait_timeouts", rc, kq_last_error())
    return v.value


def kq_selftest_bounded_wait(stream=None) -> None:
    """Launch one staged CTA whose waits run out (no copies issued); see the C header."""
    _call("kq_selftest_bounded_wait", None, _stream(stream, None))


def kq_fold_weights(W, factors, shared=False, out=None, stream=None):
    """W T^-1 per 32-column block (fp32 [N, d])."""
    torch = _torch()
    _need(W, "W", torch.float32)
    if W.dim() != 2:
        raise ValueError("W must be 2-D [N, d]")
    N, d = W.shape
    _factors(factors, d, shared, W.device)
    if out is None:
        out = torch.empty_like(W)
    _need(out, "out", torch.float32, W.device, (N, d))
    _call("kq_fold_weights", W.device, _ptr(W), _ptr(factors), int(bool(shared)), _ptr(out), N, d,
          _stream(stream, W.device))
    return out


def kq_transform_f32_variant(variant, act, factors, shared=False, out=None, stream=None):
    """The fp32 transform through a chosen kernel variant (test export)."""
    torch = _torch()
    M, d = _act(act)
    _factors(factors, d, shared, act.device)
    if out is None:
        out = torch.empty((M, d), dtype=torch.float32, device=act.device)
    _need(out, "out", torch.float32, act.device, (M, d))
    _call("kq_transform_f32_variant", act.device, int(variant), _ptr(act), _ptr(factors), int(bool(shared)), _ptr(out),
          M, d, _stream(stream, act.device))
    return out


def kq_transform_f32(act, factors, shared=False, out=None, stream=None):
    """The fp32 transform y = T x that the quantizer computes (test export)."""
    torch = _torch()
    M, d = _act(act)
    _factors(factors, d, shared, act.device)
    if out is None:
        out = torch.empty((M, d), dtype=torch.float32, device=act.device)
    _need(out, "out", torch.float32, act.device, (M, d))
    _call("kq_transform_f32", act.device, _ptr(act), _ptr(factors), int(bool(shared)), _ptr(out), M, d,
          _stream(stream, act.device))
    return out


def kq_sf_bytes(rows: int, d: int) -> int:
    """Bytes of a scale-factor-layout buffer for a [rows, d] MXFP4 matrix."""
    n = lib().kq_sf_bytes(int(rows), int(d))
    if n < 0:
        raise ValueError(f"kq_sf_bytes: bad shape rows={rows}, d={d}")
    return n


def _sf_out(out_sf, rows, d, device):
    torch = _torch()
    n = kq_sf_bytes(rows, d)
    if out_sf is None:
        out_sf = torch.empty((n,), dtype=torch.uint8, device=device)
    _need(out_sf, "out_sf", torch.uint8, device, (n,))
    return out_sf


def kq_quantize_sf(act, factors, shared=False, out_codes=None, out_sf=None, stream=None):
    """kq_quantize with the scales in the tensor core's scale-factor layout (1-D uint8)."""
    torch = _torch()
    M, d = _act(act)
    _factors(factors, d, shared, act.device)
    if out_codes is None:
        out_codes = torch.empty((M, d // 2), dtype=torch.uint8, device=act.device)
    _need(out_codes, "out_codes", torch.uint8, act.device, (M, d // 2))
    out_sf = _sf_out(out_sf, M, d, act.device)
    _call("kq_quantize_sf", act.device, _ptr(act), _ptr(factors), int(bool(shared)), _ptr(out_codes), _ptr(out_sf), M,
          d, _stream(stream, act.device))
    return out_codes, out_sf


def mx_quantize_f32(x, sf_layout=False, out_codes=None, out_scales=None, stream=None):
    """Plain MXFP4 quantizer on fp32 input [M, d] (the folded weights).

    Scales row-major [M, d/32], or with sf_layout=True in the scale-factor layout (1-D).
    """
    torch = _torch()
    _need(x, "x", torch.float32)
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, d]")
    M, d = x.shape
    if out_codes is None:
        out_codes = torch.empty((M, d // 2), dtype=torch.uint8, device=x.device)
    _need(out_codes, "out_codes", torch.uint8, x.device, (M, d // 2))
    if sf_layout:
        out_scales = _sf_out(out_scales, M, d, x.device)
    else:
        if out_scales is None:
            out_scales = torch.empty((M, d // 32), dtype=torch.uint8, device=x.device)
        _need(out_scales, "out_scales", torch.uint8, x.device, (M, d // 32))
    _call("mx_quantize_f32", x.device, _ptr(x), _ptr(out_codes), _ptr(out_scales),
          KQ_SCALES_SF if sf_layout else KQ_SCALES_ROWMAJOR, M, d, _stream(stream, x.device))
    return out_codes, out_scales


def mx_scales_to_sf(scales, out_sf=None, stream=None):
    """Row-major scales [M, d/32] -> the scale-factor layout (1-D uint8)."""
    torch = _torch()
    _need(scales, "scales", torch.uint8)
    if scales.dim() != 2:
        raise ValueError("scales must be 2-D [M, d/32]")
    M, d = scales.shape[0], scales.shape[1] * 32
    out_sf = _sf_out(out_sf, M, d, scales.device)
    _call("mx_scales_to_sf", scales.device, _ptr(scales), _ptr(out_sf), M, d, _stream(stream, scales.device))
    return out_sf


def mxf4_gemm(a_codes, a_sf, b_codes, b_sf, out=None, out_dtype=None, stream=None):
    """W4A4 linear layer: out[m, n] = sum_k a[m, k] b[n, k] over decoded MXFP4 operands.

    a_codes [M, K/2], b_codes [N, K/2] uint8; a_sf, b_sf their scales in the
    scale-factor layout; out bf16 (default) or float32 [M, N].
    """
    return mxf4_gemm_variant(0, a_codes, a_sf, b_codes, b_sf, out, out_dtype, stream)


def mxf4_gemm_variant(variant, a_codes, a_sf, b_codes, b_sf, out=None, out_dtype=None, stream=None):
    """mxf4_gemm through a chosen tile configuration (0 = the default; test export)."""
    torch = _torch()
    _need(a_codes, "a_codes", torch.uint8)
    if a_codes.dim() != 2 or b_codes.dim() != 2:
        raise ValueError("a_codes and b_codes must be 2-D")
    M, K = a_codes.shape[0], a_codes.shape[1] * 2
    dev = a_codes.device
    _need(b_codes, "b_codes", torch.uint8, dev)
    N = b_codes.shape[0]
    if b_codes.shape[1] * 2 != K:
        raise ValueError(f"b_codes must be [N, {K // 2}], got {tuple(b_codes.shape)}")
    _need(a_sf, "a_sf", torch.uint8, dev, (kq_sf_bytes(M, K),))
    _need(b_sf, "b_sf", torch.uint8, dev, (kq_sf_bytes(N, K),))
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype or torch.bfloat16, device=dev)
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out must be bfloat16 or float32")
    _need(out, "out", out.dtype, dev, (M, N))
    _call("mxf4_gemm_variant", dev, int(variant), _ptr(a_codes), _ptr(a_sf), _ptr(b_codes), _ptr(b_sf), _ptr(out),
          int(out.dtype == torch.float32), M, N, K, _stream(stream, dev))
    return out


def norm_kq_quantize_sf(h, gamma, beta, factors, eps=1e-6, shared=False, out_codes=None, out_sf=None, stream=None):
    """norm_kq_quantize with the scales in the tensor core's scale-factor layout (1-D uint8)."""
    torch = _torch()
    M, d = _act(h)
    _need(gamma, "gamma", torch.float32, h.device)
    _need(beta, "beta", torch.float32, h.device, tuple(gamma.shape))
    if gamma.dim() != 2 or gamma.shape[1] != d:
        raise ValueError("gamma and beta must be [nsamples, d]")
    _factors(factors, d, shared, h.device)
    if out_codes is None:
        out_codes = torch.empty((M, d // 2), dtype=torch.uint8, device=h.device)
    _need(out_codes, "out_codes", torch.uint8, h.device, (M, d // 2))
    out_sf = _sf_out(out_sf, M, d, h.device)
    _call("norm_kq_quantize_sf", h.device, _ptr(h), _ptr(gamma), _ptr(beta), int(gamma.shape[0]), float(eps),
          _ptr(factors), int(bool(shared)), _ptr(out_codes), _ptr(out_sf), M, d, _stream(stream, h.device))
    return out_codes, out_sf


def mxf4_gemv_workspace(M: int, N: int, K: int) -> int:
    """Bytes of workspace that mxf4_gemv needs for calls of these sizes."""
    n = _sizes("mxf4_gemv_workspace", int(M), int(N), int(K))
    if n < 0:
        raise ValueError(f"mxf4_gemv_workspace: bad sizes {M}, {N}, {K}")
    return n


def mxf4_gemv(x, b_codes, b_sf, out=None, out_dtype=None, workspace=None, stream=None):
    """A few rows times MXFP4 weights: out[m, n] = sum_k x[m, k] b[n, k], M <= 32.

    x bf16 [M, K] (rows may be strided), not quantized; b_codes [N, K/2] and b_sf the
    weight operand of mxf4_gemm; out bf16 (default) or float32 [M, N].  workspace: uint8
    tensor of mxf4_gemv_workspace(M, N, K) bytes for this call alone; allocated if None.
    stream: default the current one; what a call on another allocates (results, too) is that
    stream's, as under torch.cuda.stream(stream).
    """
    torch = _torch()
    if out is None and workspace is None and stream is None and (out_dtype is None or out_dtype in (torch.bfloat16, torch.float32)):
        native = _native()
        done = native.gemv(x, b_codes, b_sf, out_dtype is torch.float32) if native else None
        if done is not None:
            return _done("mxf4_gemv", done)
    u8 = torch.uint8
    M, N = _gemv_sizes(x, b_codes, b_sf)
    K = x.shape[1]
    dev = x.device
    if out is None:
        out = _new((M, N), out_dtype or torch.bfloat16, dev, stream)
    else:
        _need(out, "out", out.dtype, dev, (M, N))
    f32 = out.dtype is torch.float32
    if not (f32 or out.dtype is torch.bfloat16) or (out_dtype is not None and out.dtype != out_dtype):
        raise TypeError(f"out must be {out_dtype or 'bfloat16 or float32'}, got {out.dtype}")
    need = _sizes("mxf4_gemv_workspace", M, N, K)            # -1: sizes that the call refuses
    if workspace is not None:
        _need(workspace, "workspace", u8, dev)
    elif need > 0:
        workspace = _new((need,), u8, dev, stream)
    _call("mxf4_gemv", dev, x.data_ptr(), x.stride(0) if M > 1 else K, b_codes.data_ptr(), b_sf.data_ptr(), out.data_ptr(),
          f32, M, N, K,
          _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(stream, dev))
    return out


_native_module = None


def _native():
    """The binding's native part (csrc/binding.cpp), which does ordinary calls of the few-token
    operators in one step and answers None to the others; False where it was not built or does not load."""
    global _native_module
    if _native_module is None:
        import importlib.machinery
        import importlib.util
        import warnings

        from .build import binding_path

        L = lib()
        _native_module = False
        try:
            path = binding_path()
            if not os.path.exists(path):
                return False
            loader = importlib.machinery.ExtensionFileLoader("kq_binding", path)
            module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("kq_binding", path, loader=loader))
            loader.exec_module(module)
        except (ImportError, OSError) as e:                  # (no metadata of torch, a file of another torch or Python)
            warnings.warn(f"the binding's native part does not load, calls take longer: {e}")
            return False
        module.init(*(ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in (
            "mxf4_gemv", "mxf4_gemv_workspace", "kq_sf_bytes", "mx_cache_write", "mx_cache_read", "mx_paged_attention",
            "mx_attention_workspace")))
        _native_module = module
    return _native_module


def _done(name, result):
    """What a native call returned, or its error."""
    if type(result) is int:
        raise KroQuantError(name, result, kq_last_error())
    return result


def _gemv_sizes(x, b_codes, b_sf):
    """M and N of mxf4_gemv's operands, checked (as in _cache: at once, and one by one to say what is wrong)."""
    torch = _torch()
    u8 = torch.uint8
    try:
        M, K = x.shape
        N, half = b_codes.shape
        dev = x.device
        if x.dtype is torch.bfloat16 and b_codes.dtype is u8 and b_sf.dtype is u8 and x.is_cuda and b_codes.device == dev \
                and b_sf.device == dev and 2 * half == K and x.stride(1) == 1 and b_codes.is_contiguous() \
                and b_sf.shape == (_sizes("kq_sf_bytes", N, K),) and b_sf.is_contiguous():
            return M, N
    except (AttributeError, TypeError, ValueError):
        pass
    _need_rows(x, "x", (torch.bfloat16,), 2)
    M, K = x.shape
    _need(b_codes, "b_codes", u8, x.device)
    if b_codes.dim() != 2 or b_codes.shape[1] * 2 != K:
        raise ValueError(f"b_codes must be [N, {K // 2}], got {tuple(b_codes.shape)}")
    _need(b_sf, "b_sf", u8, x.device, (kq_sf_bytes(b_codes.shape[0], K),))
    return M, b_codes.shape[0]


# mx_cache and mx_batch of the C header, passed as bytes.
_CACHE = struct.Struct("4P4q")
_BATCH = struct.Struct("PqqPPq")

def _need_rows(t, name, dtypes, dim, device=None, shape=None):
    """An operand whose last dimension is contiguous and whose others may be strided."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype in dtypes and t.is_cuda and (device is None or t.device == device) and t.dim() == dim and \
            (shape is None or t.shape == shape) and t.stride(-1) == 1:
        return t
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dim() != dim:
        raise ValueError(f"{name} must be {dim}-D, got {tuple(t.shape)}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.numel() > 0 and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t


def _cache(k_codes, k_scales, v_codes, v_scales):
    """(packed mx_cache, device, heads, head_dim) of a cache's four arrays."""
    torch = _torch()
    u8 = torch.uint8
    try:
        # these calls are made once per layer and token: all of it at once, and one by one only to say what is wrong
        shape = k_codes.shape
        P, H, S, half = shape
        scales = (P, H, S, half // 16)
        dev = k_codes.device
        if k_codes.dtype is u8 and v_codes.dtype is u8 and k_scales.dtype is u8 and v_scales.dtype is u8 and k_codes.is_cuda \
                and v_codes.device == dev and k_scales.device == dev and v_scales.device == dev \
                and v_codes.shape == shape and k_scales.shape == scales and v_scales.shape == scales \
                and k_codes.is_contiguous() and v_codes.is_contiguous() and k_scales.is_contiguous() and v_scales.is_contiguous():
            return _CACHE.pack(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(), P, H, S,
                               2 * half), dev, H, 2 * half
    except (AttributeError, TypeError, ValueError):
        pass
    _need(k_codes, "k_codes", u8)
    if k_codes.dim() != 4:
        raise ValueError("k_codes must be [num_pages, heads, page_size, head_dim / 2]")
    _need(v_codes, "v_codes", u8, dev, shape)
    _need(k_scales, "k_scales", u8, dev, scales)
    _need(v_scales, "v_scales", u8, dev, scales)
    raise ValueError("the cache's arrays do not fit together")


def _batch(block_table, cu_seqlens, seq_lens, device):
    """(packed mx_batch, sequences) of a call's sequences; seq_lens None where the call reads none."""
    i32 = _torch().int32
    try:
        B, pages = block_table.shape
        stride, inner = block_table.stride()
        if B <= 1:
            stride = pages                   # (not used, whatever the tensor says)
        if block_table.dtype is i32 and cu_seqlens.dtype is i32 and block_table.device == device \
                and cu_seqlens.device == device and stride >= pages and (inner == 1 or pages <= 1) \
                and cu_seqlens.shape == (B + 1,) and cu_seqlens.is_contiguous():
            if seq_lens is None:
                return _BATCH.pack(block_table.data_ptr(), stride, pages, cu_seqlens.data_ptr(), 0, B), B
            if seq_lens.dtype is i32 and seq_lens.device == device and seq_lens.shape == (B,) and seq_lens.is_contiguous():
                return _BATCH.pack(block_table.data_ptr(), stride, pages, cu_seqlens.data_ptr(), seq_lens.data_ptr(), B), B
    except (AttributeError, TypeError, ValueError):
        pass
    _need_rows(block_table, "block_table", (i32,), 2, device)
    B, pages = block_table.shape
    if B > 1 and block_table.stride(0) < pages:
        raise ValueError(f"block_table's rows overlap (stride {block_table.stride(0)}, {pages} entries); make it contiguous")
    _need(cu_seqlens, "cu_seqlens", i32, device, (B + 1,))
    _need(seq_lens, "seq_lens", i32, device, (B,))
    raise ValueError("block_table, cu_seqlens and seq_lens do not fit together")


def mx_cache_write(k, v, k_codes, k_scales, v_codes, v_scales, block_table, cu_seqlens, seq_lens, stream=None):
    """Quantize new tokens' keys and values into a paged MXFP4 cache.

    k, v: bf16 or float32 [T, heads, head_dim], tokens and heads may be strided (slices of a
    fused projection).  The cache: codes uint8 [pages, heads, page_size, head_dim/2] and
    scales uint8 [pages, heads, page_size, head_dim/32] of keys and of values.  Sequences:
    block_table int32 [B, max_pages] (its rows may be strided, but not overlap: an expanded
    table is refused, .contiguous() does), cu_seqlens int32 [B+1] (rows of each sequence),
    seq_lens int32 [B] (lengths with the new tokens, which are the last ones).
    """
    torch = _torch()
    if stream is None:
        native = _native()
        done = native.write(k, v, k_codes, k_scales, v_codes, v_scales, block_table, cu_seqlens, seq_lens) if native else None
        if done is not None:
            _done("mx_cache_write", None if done is True else done)
            return
    c, dev, H, D = _cache(k_codes, k_scales, v_codes, v_scales)
    if seq_lens is None:
        raise TypeError("seq_lens must be a torch.Tensor")
    b, _ = _batch(block_table, cu_seqlens, seq_lens, dev)
    _need_rows(k, "k", (torch.bfloat16, torch.float32), 3, dev)
    shape = k.shape
    T = shape[0]
    if shape[1] != H or shape[2] != D:
        raise ValueError(f"k must be [T, {H}, {D}], got {tuple(shape)}")
    _need_rows(v, "v", (k.dtype,), 3, dev, shape)
    kst, ksh, _ = k.stride()
    vst, vsh, _ = v.stride()
    _call("mx_cache_write", dev, k.data_ptr(), kst, ksh, v.data_ptr(), vst, vsh, k.dtype is torch.float32, c, b, T, _stream(stream, dev))


def mx_cache_read(k_codes, k_scales, v_codes, v_scales, block_table, cu_seqlens, rows, starts=None, out_k=None,
                  out_v=None, out_dtype=None, stream=None):
    """Positions of a paged MXFP4 cache back as bf16 (default) or float32, keys and values.

    Row cu_seqlens[b] + i of the [rows, heads, head_dim] outputs is position starts[b] + i
    (starts int32 [B], default zeros) of sequence b.  Rows of no sequence keep their values
    (undefined ones where the call allocates the outputs).  stream as in mxf4_gemv.
    """
    torch = _torch()
    if out_k is None and out_v is None and stream is None and (out_dtype is None or out_dtype in (torch.bfloat16, torch.float32)):
        native = _native()
        done = native.read(k_codes, k_scales, v_codes, v_scales, block_table, cu_seqlens, rows, starts,
                           out_dtype is torch.float32) if native else None
        if done is not None:
            return _done("mx_cache_read", done)
    c, dev, H, D = _cache(k_codes, k_scales, v_codes, v_scales)
    b, B = _batch(block_table, cu_seqlens, None, dev)
    if starts is not None:
        _need(starts, "starts", torch.int32, dev, (B,))
    shape = (int(rows), H, D)
    dtype = out_dtype or (out_k.dtype if out_k is not None else torch.bfloat16)
    f32 = dtype is torch.float32
    if not f32 and dtype is not torch.bfloat16:
        raise TypeError(f"out_k and out_v must be bfloat16 or float32, got {dtype}")
    if out_k is None:
        out_k = _new(shape, dtype, dev, stream)
    else:
        _need(out_k, "out_k", dtype, dev, shape)
    if out_v is None:
        out_v = _new(shape, dtype, dev, stream)
    else:
        _need(out_v, "out_v", dtype, dev, shape)
    _call("mx_cache_read", dev, c, b, _ptr(starts), out_k.data_ptr(), out_v.data_ptr(), f32, shape[0], _stream(stream, dev))
    return out_k, out_v


def mx_attention_workspace(rows: int, heads_q: int, heads: int, head_dim: int, max_new: int) -> int:
    """Bytes of workspace that mx_paged_attention needs for calls of these sizes."""
    n = _sizes("mx_attention_workspace", int(rows), int(heads_q), int(heads), int(head_dim), int(max_new))
    if n < 0:
        raise ValueError(f"mx_attention_workspace: bad sizes {rows}, {heads_q}, {heads}, {head_dim}, {max_new}")
    return n


def mx_paged_attention(q, k_codes, k_scales, v_codes, v_scales, block_table, cu_seqlens, seq_lens, max_new=None,
                       scale=None, causal=True, out=None, workspace=None, stream=None):
    """Attention of each sequence's new tokens over its positions in a paged MXFP4 cache.

    q bf16 [T, heads_q, head_dim] (tokens and heads may be strided); heads_q a multiple of the
    cache's heads.  The new tokens' keys and values have been written (mx_cache_write).
    causal: a token sees the positions up to its own, otherwise all seq_lens[b].  scale:
    default head_dim ** -0.5.  max_new: the most new tokens of any one sequence; T if left out,
    which costs a batch of single tokens: with more than 48 rows per kv head (T times heads_q /
    heads) the kernels for chunks are launched, too, for nothing.
    out bf16 [T, heads_q, head_dim]; rows of no sequence keep their values (undefined ones
    where the call allocates it).  workspace: uint8 tensor of mx_attention_workspace(...) bytes
    for this call alone; allocated if None.  stream as in mxf4_gemv.
    """
    torch = _torch()
    if out is None and workspace is None and stream is None:
        native = _native()
        done = native.attention(q, k_codes, k_scales, v_codes, v_scales, block_table, cu_seqlens, seq_lens, max_new, scale,
                                bool(causal)) if native else None
        if done is not None:
            return _done("mx_paged_attention", done)
    c, dev, H, D = _cache(k_codes, k_scales, v_codes, v_scales)
    if seq_lens is None:
        raise TypeError("seq_lens must be a torch.Tensor")
    b, _ = _batch(block_table, cu_seqlens, seq_lens, dev)
    _need_rows(q, "q", (torch.bfloat16,), 3, dev)
    T, hq, d = shape = q.shape
    if d != D or hq == 0 or H == 0 or hq % H:
        raise ValueError(f"q must be [T, a multiple of {H}, {D}], got {tuple(shape)}")
    max_new = T if max_new is None else int(max_new)
    scale = d ** -0.5 if scale is None else float(scale)
    if out is None:
        out = _new(shape, torch.bfloat16, dev, stream)
    else:
        _need(out, "out", torch.bfloat16, dev, shape)
    if workspace is None:
        need = mx_attention_workspace(T, hq, H, d, max_new)
        workspace = _new((need,), torch.uint8, dev, stream)
    else:
        _need(workspace, "workspace", torch.uint8, dev)
        need = workspace.numel()
    qst, qsh, _ = q.stride()
    _call("mx_paged_attention", dev, q.data_ptr(), qst, qsh, c, b, scale, bool(causal), out.data_ptr(), T, hq, max_new,
          workspace.data_ptr(), need, _stream(stream, dev))
    return out


def _new(shape, dtype, device, stream):
    """Memory for a call: of the pool of the stream that the call runs on, so that what used it
    before and what uses it afterwards is in that stream's order."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)
