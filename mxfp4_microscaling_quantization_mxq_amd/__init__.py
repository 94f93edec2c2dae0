"""MXFP4 / NVFP4 microscaling on AMD MI355X (gfx950): Python binding.

Thin ctypes layer over ``libmxq.so`` (the C ABI in ``include/mxq.h``).  It
only checks shapes/dtypes, allocates outputs with ``torch.empty`` and passes
raw device pointers plus the current HIP stream; every step of the
computation runs in the library's HIP kernels.  There is no fallback: if the
library is not built, or the device is not gfx950, calls raise.

    q, s = quantize(x)                  # MXFP4: x [rows, k] bf16/fp32, k % 32 == 0
    y = dequantize(q, s, torch.float32)
    y = gemv_w4a16(wq, ws, x)           # y[m, n] = x @ deq(W)^T, x bf16
    c = gemm_w4a4(aq, as_, bq, bs)      # c[m, n] = deq(A) @ deq(B)^T
    q, s, g = nvq.quantize(x)           # NVFP4: k % 16 == 0, g = fp32 tensor scale
    y = nvq.dequantize(q, s, g)         # (also nv_quantize / nv_dequantize / nv_gemm)
    y = nvq.gemm(wq, ws, g, x)

and, between the products of a served model's decode step:

    q, s, r = rmsnorm_quantize_fp8(x, w, residual)   # r = x + residual, MXFP8 of its norm
    cache = kv_cache(pages, 64, kv_heads, 128)       # paged MXFP8 (or "mxfp4") keys and values
    kv_append(cache, k, v, slots)                    # quantize new tokens into their slots
    o = paged_attention(q, cache, table, lens)       # one new token per sequence
    k, v = kv_read(cache, slots)                     # read slots back

or, for tokens with positions and for drafted tokens that one step checks:

    q = rope_append(cache, q, k, v, slots, positions, freqs)   # rotate, quantize new tokens into their slots
    o = tree_attention(q, cache, table, context, mask)         # several drafted tokens per sequence
    tokens, shares = sample(logits, u, temperature=0.8, top_p=0.95)   # draw a token of each row

Every tensor argument is checked before anything is enqueued: dtype, shape
(scales and caller-supplied outputs must match the operands exactly),
contiguity, and that it lives on the operands' device; the NVFP4 tensor
scale must be a 1-element fp32 device tensor.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import NamedTuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxq.so")

MXQ_F32 = 0
MXQ_BF16 = 1
MXQ_MXFP8 = 0
MXQ_MXFP4 = 1
STATUS = {
    0: "MXQ_SUCCESS",
    1: "MXQ_ERROR_INVALID_VALUE",
    2: "MXQ_ERROR_MISALIGNED",
    3: "MXQ_ERROR_NOT_SUPPORTED",
    4: "MXQ_ERROR_LAUNCH_FAILURE",
}
API = (
    "mxq_status_string", "mxq_version", "mxq_quantize", "mxq_quantize_hadamard", "mxq_quantize_fp8",
    "mxq_dequantize", "mxq_gemv_w4a16", "mxq_gemm_w4a4", "mxq_gemm_w4a4_quant", "mxq_gemm_w4a4_dynamic",
    "mxq_gemm_w4a8", "mxq_gemm_w4a8_dynamic", "nvq_quantize", "nvq_dequantize", "nvq_gemm", "mxq_transfp4_quantize", "mxq_transfp4_dequantize",
    "mxq_rmsnorm_quantize_fp8", "mxq_kv_append", "mxq_kv_read", "mxq_paged_attention_workspace", "mxq_paged_attention",
    "mxq_rope_append", "mxq_tree_attention_workspace", "mxq_tree_attention",
    "mxq_sample_workspace", "mxq_sample",
)


class MXQError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)} ({status_string(code)})")


_lib = None


def capi() -> ctypes.CDLL:
    """The loaded C library with argument types set (raises if not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with "
            "`python -m mxfp4_microscaling_quantization_mxq_amd.build` (hipcc, gfx950)"
        )
    lib = ctypes.CDLL(LIB_PATH)
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.mxq_status_string.argtypes = [I]
    lib.mxq_status_string.restype = ctypes.c_char_p
    lib.mxq_version.argtypes = []
    lib.mxq_version.restype = I
    lib.mxq_quantize.argtypes = [P, I, I64, I64, P, P, P]
    lib.mxq_quantize_hadamard.argtypes = [P, I, I64, I64, I, P, P, P]
    lib.mxq_quantize_fp8.argtypes = [P, I, I64, I64, P, P, P]
    lib.mxq_gemm_w4a8.argtypes = [P, P, P, P, I64, I64, I64, P, I, P]
    lib.mxq_dequantize.argtypes = [P, P, I64, I64, P, I, P]
    lib.mxq_gemv_w4a16.argtypes = [P, P, I64, I64, P, I64, P, I, P]
    lib.mxq_gemm_w4a4.argtypes = [P, P, P, P, I64, I64, I64, P, I, P]
    lib.mxq_gemm_w4a4_quant.argtypes = [P, P, P, P, I64, I64, I64, P, P, P]
    lib.mxq_gemm_w4a4_dynamic.argtypes = [P, P, P, I64, I64, I64, P, I, P]
    lib.mxq_gemm_w4a8_dynamic.argtypes = [P, P, P, I64, I64, I64, P, I, P]
    lib.nvq_quantize.argtypes = [P, I, I64, I64, P, I, P, P, P]
    lib.nvq_dequantize.argtypes = [P, P, P, I64, I64, P, I, P]
    lib.nvq_gemm.argtypes = [P, P, P, I64, I64, P, I64, P, I, P]
    lib.mxq_transfp4_quantize.argtypes = [P, I, I64, I64, P, I, P, P, P, P, P]
    lib.mxq_transfp4_dequantize.argtypes = [P, P, P, P, P, I64, I64, P, I, P]
    F = ctypes.c_float
    lib.mxq_rmsnorm_quantize_fp8.argtypes = [P, P, P, I, I64, I64, F, P, P, P, P]
    lib.mxq_kv_append.argtypes = [P, I64, P, I64, I, P, I64, I64, I64, I64, I64, I, P, P, P, P, P]
    lib.mxq_kv_read.argtypes = [P, P, P, P, P, I64, I64, I64, I64, I64, I, P, P, I, P]
    lib.mxq_paged_attention_workspace.argtypes = [I64, I64, I64, I64, I64, I64, I64, ctypes.POINTER(I64)]
    lib.mxq_paged_attention.argtypes = [P, I64, P, P, P, P, P, I64, I64, P, P, I64, I64, I64, I64, I64, I64, I, F,
                                        I64, P, I64, P, I, P]
    lib.mxq_rope_append.argtypes = [P, I64, P, I64, P, I64, I, P, I64, P, P, I64, I, P, I64, I64, I64, I64, I64, I64, I,
                                    P, P, P, P, P, P]
    lib.mxq_tree_attention_workspace.argtypes = [I64, I64, I64, I64, I64, I64, I64, I64, I64, ctypes.POINTER(I64)]
    lib.mxq_tree_attention.argtypes = [P, I64, P, P, P, P, P, I64, I64, P, P, P, I64, I64, I64, I64, I64, I64, I64, I, F,
                                       I64, I64, P, I64, P, I, P]
    lib.mxq_sample_workspace.argtypes = [I64, I64, ctypes.POINTER(I64)]
    lib.mxq_sample.argtypes = [P, I, I64, I64, I64, P, P, F, P, I64, P, F, P, F, P, I64, P, P, P]
    for name in API[2:]:
        getattr(lib, name).restype = I
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return capi().mxq_status_string(code).decode()


def _check(code: int, what: str):
    if code != 0:
        raise MXQError(code, what)


# ------------------------------------------------------------------ helpers

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


def _stream(dev=None):
    """The current stream of the current device as a raw handle; with `dev`, the
    operands have to be on that device.  (The Stream object of
    torch.cuda.current_stream() costs 3 us to build, as much as a launch.)"""
    c = _torch()._C
    current = c._cuda_getDevice()
    if dev is not None and dev != current:
        raise ValueError(f"the operands are on device {dev}, the current device is {current}")
    return c._cuda_getCurrentRawStream(current)


def _dtype_code(dt) -> int:
    torch = _torch()
    if dt == torch.float32:
        return MXQ_F32
    if dt == torch.bfloat16:
        return MXQ_BF16
    raise TypeError(f"unsupported dtype {dt}: use torch.float32 or torch.bfloat16")


def _p(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr())


def _need(t, name, dtype=None, shape=None, ndim=2, device=None):
    """Validate one tensor argument's type, dtype, shape and contiguity
    (where it lives is checked by _on_device, after every shape check).
    Raises TypeError / ValueError; `device` is accepted for symmetry only."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if dtype is not None and t.dtype is not dtype:
        allowed = dtype if isinstance(dtype, tuple) else (dtype,)
        if t.dtype not in allowed:
            raise TypeError(f"{name} must be {' or '.join(str(d) for d in allowed)}, got {t.dtype}")
    if shape is not None:
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    elif t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_device(**tensors):
    """Every tensor of the call on one and the same device (cuda/hip)."""
    dev = None
    for name, t in tensors.items():
        d = t.get_device()
        if d < 0 or not t.is_cuda:
            raise ValueError(f"{name} must be a device (cuda/hip) tensor")
        if dev is None:
            dev = d
        elif d != dev:
            raise ValueError(f"{name} is on {t.device}, the other operands on device {dev}")
    return dev


def _floats():
    torch = _torch()
    return (torch.float32, torch.bfloat16)


def _out(t, name, shape, dtype, device, real=False):
    """An output tensor: allocated if None, else validated like an input.
    `real` outputs (unquantized values) must be float32 or bfloat16."""
    torch = _torch()
    if real and dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, got {dtype}")
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(t, name, dtype, shape, device=device)
    return t


def _gscale(g, name, device):
    """The NVFP4 tensor scale: a 1-element fp32 device tensor."""
    torch = _torch()
    _need(g, name, torch.float32, (1,), device=device)
    return g


# ------------------------------------------------------------------ MXFP4

def _k_blocks(k, blk, what):
    if k % blk != 0:
        raise ValueError(f"{what}: k = {k} is not a multiple of {blk}")


def quantize(x, q=None, s=None):
    """MXFP4 quantize x[rows, k] (bf16 or fp32) -> (q[rows, k/2] u8, s[rows, k/32] u8)."""
    torch = _torch()
    _need(x, "x", _floats())
    rows, k = x.shape
    _k_blocks(k, 32, "quantize")
    q = _out(q, "q", (rows, k // 2), torch.uint8, x.device)
    s = _out(s, "s", (rows, k // 32), torch.uint8, x.device)
    _on_device(x=x, q=q, s=s)
    _check(capi().mxq_quantize(_p(x), _dtype_code(x.dtype), rows, k, _p(q), _p(s), _stream()), "mxq_quantize")
    return q, s


def quantize_hadamard(x, hk=32, q=None, s=None):
    """Rotated MXFP4: quantize x[rows, k] after the orthonormal block Hadamard
    H_hk along k (hk in 16, 32, 64, 128) -> (q[rows, k/2] u8, s[rows, k/32] u8)."""
    torch = _torch()
    _need(x, "x", _floats())
    rows, k = x.shape
    _k_blocks(k, 32, "quantize_hadamard")
    q = _out(q, "q", (rows, k // 2), torch.uint8, x.device)
    s = _out(s, "s", (rows, k // 32), torch.uint8, x.device)
    _on_device(x=x, q=q, s=s)
    _check(capi().mxq_quantize_hadamard(_p(x), _dtype_code(x.dtype), rows, k, int(hk), _p(q), _p(s), _stream()),
           "mxq_quantize_hadamard")
    return q, s


def quantize_fp8(x, q=None, s=None):
    """MXFP8 quantize x[rows, k] -> (q[rows, k] E4M3 codes u8, s[rows, k/32] E8M0 u8)."""
    torch = _torch()
    _need(x, "x", _floats())
    rows, k = x.shape
    _k_blocks(k, 32, "quantize_fp8")
    q = _out(q, "q", (rows, k), torch.uint8, x.device)
    s = _out(s, "s", (rows, k // 32), torch.uint8, x.device)
    _on_device(x=x, q=q, s=s)
    _check(capi().mxq_quantize_fp8(_p(x), _dtype_code(x.dtype), rows, k, _p(q), _p(s), _stream()), "mxq_quantize_fp8")
    return q, s


def dequantize(q, s, dtype=None, y=None):
    """(q[rows, k/2], s[rows, k/32]) -> y[rows, k] in dtype (default bf16; y's dtype if y is given)."""
    torch = _torch()
    _need(q, "q", torch.uint8)
    rows, k = q.shape[0], q.shape[1] * 2
    _k_blocks(k, 32, "dequantize")
    _need(s, "s", torch.uint8, (rows, k // 32), device=q.device)
    dtype = dtype or (y.dtype if y is not None else torch.bfloat16)
    y = _out(y, "y", (rows, k), dtype, q.device, real=True)
    _on_device(q=q, s=s, y=y)
    _check(capi().mxq_dequantize(_p(q), _p(s), rows, k, _p(y), _dtype_code(y.dtype), _stream()), "mxq_dequantize")
    return y


def _weight(wq, ws, blk, what):
    """An MXFP4 (blk 32) or NVFP4 (blk 16) weight: (n, k) after validation."""
    torch = _torch()
    _need(wq, "wq", torch.uint8)
    n, k = wq.shape[0], wq.shape[1] * 2
    _k_blocks(k, blk, what)
    _need(ws, "ws", torch.uint8, (n, k // blk), device=wq.device)
    return n, k


def _activations(x, k, dev):
    torch = _torch()
    _need(x, "x", torch.bfloat16, device=dev)
    if x.shape[1] != k:
        raise ValueError(f"x has k={x.shape[1]}, weight has k={k}")
    return x.shape[0]


def gemv_w4a16(wq, ws, x, out_dtype=None, y=None):
    """y[m, n] = x[m, k] @ deq(W)^T with W = (wq[n, k/2], ws[n, k/32]); x bf16."""
    torch = _torch()
    n, k = _weight(wq, ws, 32, "gemv_w4a16")
    m = _activations(x, k, wq.device)
    out_dtype = out_dtype or (y.dtype if y is not None else torch.bfloat16)
    y = _out(y, "y", (m, n), out_dtype, wq.device, real=True)
    _on_device(wq=wq, ws=ws, x=x, y=y)
    _check(capi().mxq_gemv_w4a16(_p(wq), _p(ws), n, k, _p(x), m, _p(y), _dtype_code(y.dtype), _stream()),
           "mxq_gemv_w4a16")
    return y


def _ab(aq, as_, bq, bs, a_bytes_per_k, what):
    """Block-scaled operands A (aq[m, k * a_bytes_per_k], as_[m, k/32]) and
    B (bq[n, k/2], bs[n, k/32]): (m, n, k) after validation."""
    torch = _torch()
    _need(aq, "aq", torch.uint8)
    m = aq.shape[0]
    k = int(aq.shape[1] / a_bytes_per_k)
    _k_blocks(k, 32, what)
    dev = aq.device
    _need(as_, "as", torch.uint8, (m, k // 32), device=dev)
    _need(bq, "bq", torch.uint8, device=dev)
    if bq.shape[1] * 2 != k:
        raise ValueError(f"{what}: A has k={k}, B has k={bq.shape[1] * 2}")
    n = bq.shape[0]
    _need(bs, "bs", torch.uint8, (n, k // 32), device=dev)
    return m, n, k


def gemm_w4a4(aq, as_, bq, bs, out_dtype=None, c=None):
    """c[m, n] = deq(A)[m, k] @ deq(B)[n, k]^T, both MXFP4."""
    torch = _torch()
    m, n, k = _ab(aq, as_, bq, bs, 0.5, "gemm_w4a4")
    out_dtype = out_dtype or (c.dtype if c is not None else torch.bfloat16)
    c = _out(c, "c", (m, n), out_dtype, aq.device, real=True)
    _on_device(aq=aq, as_=as_, bq=bq, bs=bs, c=c)
    _check(capi().mxq_gemm_w4a4(_p(aq), _p(as_), _p(bq), _p(bs), m, n, k, _p(c), _dtype_code(c.dtype), _stream()),
           "mxq_gemm_w4a4")
    return c


def _gemm_dynamic(entry, x, bq, bs, out_dtype, c):
    torch = _torch()
    n, k = _weight(bq, bs, 32, entry)
    m = _activations(x, k, bq.device)
    out_dtype = out_dtype or (c.dtype if c is not None else torch.bfloat16)
    c = _out(c, "c", (m, n), out_dtype, bq.device, real=True)
    _on_device(x=x, bq=bq, bs=bs, c=c)
    _check(getattr(capi(), entry)(_p(x), _p(bq), _p(bs), m, n, k, _p(c), _dtype_code(c.dtype), _stream()), entry)
    return c


def gemm_w4a4_dynamic(x, bq, bs, out_dtype=None, c=None):
    """c[m, n] = MXFP4(x)[m, k] @ deq(B)[n, k]^T with bf16 x quantized inside
    the kernel (bit-identical to gemm_w4a4(*quantize(x), bq, bs)); m <= 16,
    k % 512 == 0."""
    return _gemm_dynamic("mxq_gemm_w4a4_dynamic", x, bq, bs, out_dtype, c)


def gemm_w4a8_dynamic(x, bq, bs, out_dtype=None, c=None):
    """c[m, n] = MXFP8(x)[m, k] @ deq(B)[n, k]^T with bf16 x quantized to MXFP8
    inside the kernel (bit-identical to gemm_w4a8(*quantize_fp8(x), bq, bs));
    m <= 16, k % 512 == 0."""
    return _gemm_dynamic("mxq_gemm_w4a8_dynamic", x, bq, bs, out_dtype, c)


def gemm_w4a8(aq8, as_, bq, bs, out_dtype=None, c=None):
    """c[m, n] = deq8(A)[m, k] @ deq4(B)[n, k]^T: MXFP8 activations, MXFP4 weights."""
    torch = _torch()
    m, n, k = _ab(aq8, as_, bq, bs, 1, "gemm_w4a8")
    out_dtype = out_dtype or (c.dtype if c is not None else torch.bfloat16)
    c = _out(c, "c", (m, n), out_dtype, aq8.device, real=True)
    _on_device(aq8=aq8, as_=as_, bq=bq, bs=bs, c=c)
    _check(capi().mxq_gemm_w4a8(_p(aq8), _p(as_), _p(bq), _p(bs), m, n, k, _p(c), _dtype_code(c.dtype), _stream()),
           "mxq_gemm_w4a8")
    return c


def gemm_w4a4_quant(aq, as_, bq, bs, cq=None, cs=None):
    """W4A4 with MXFP4 output: (cq[m, n/2], cs[m, n/32]) = MXFP4 of the
    bf16-rounded deq(A) @ deq(B)^T, quantized in the GEMM epilogue."""
    torch = _torch()
    m, n, k = _ab(aq, as_, bq, bs, 0.5, "gemm_w4a4_quant")
    if n % 32 != 0:
        raise ValueError(f"gemm_w4a4_quant: n = {n} is not a multiple of 32")
    cq = _out(cq, "cq", (m, n // 2), torch.uint8, aq.device)
    cs = _out(cs, "cs", (m, n // 32), torch.uint8, aq.device)
    _on_device(aq=aq, as_=as_, bq=bq, bs=bs, cq=cq, cs=cs)
    _check(capi().mxq_gemm_w4a4_quant(_p(aq), _p(as_), _p(bq), _p(bs), m, n, k, _p(cq), _p(cs), _stream()),
           "mxq_gemm_w4a4_quant")
    return cq, cs


# ------------------------------------------------------------------ NVFP4

def _tensor_scale_arg(gscale, g, device):
    """(compute, g): gscale None -> computed on the device into g (allocated
    if None); a float -> a new device tensor; a tensor -> used as given."""
    torch = _torch()
    if gscale is None:
        if g is None:
            g = torch.empty(1, dtype=torch.float32, device=device)
        return True, _gscale(g, "g", device)
    if isinstance(gscale, (float, int)):
        return False, torch.tensor([float(gscale)], dtype=torch.float32, device=device)
    return False, _gscale(gscale, "gscale", device)


def nv_quantize(x, gscale=None, q=None, s=None, g=None):
    """NVFP4 quantize x[rows, k] -> (q[rows, k/2], s[rows, k/16] E4M3, g[1] fp32 tensor scale).

    gscale=None computes the tensor scale on the device (into g if given); a
    float or a 1-element fp32 tensor is used as given."""
    torch = _torch()
    _need(x, "x", _floats())
    rows, k = x.shape
    _k_blocks(k, 16, "nv_quantize")
    compute, g = _tensor_scale_arg(gscale, g, x.device)
    q = _out(q, "q", (rows, k // 2), torch.uint8, x.device)
    s = _out(s, "s", (rows, k // 16), torch.uint8, x.device)
    _on_device(x=x, g=g, q=q, s=s)
    _check(capi().nvq_quantize(_p(x), _dtype_code(x.dtype), rows, k, _p(g), int(compute), _p(q), _p(s),
                               _stream()), "nvq_quantize")
    return q, s, g


def nv_dequantize(q, s, g, dtype=None, y=None):
    """(q[rows, k/2], s[rows, k/16], g[1]) -> y[rows, k] = g * E4M3(s) * E2M1(q), rounded once to dtype."""
    torch = _torch()
    _need(q, "q", torch.uint8)
    rows, k = q.shape[0], q.shape[1] * 2
    _k_blocks(k, 16, "nv_dequantize")
    _need(s, "s", torch.uint8, (rows, k // 16), device=q.device)
    _gscale(g, "g", q.device)
    dtype = dtype or (y.dtype if y is not None else torch.bfloat16)
    y = _out(y, "y", (rows, k), dtype, q.device, real=True)
    _on_device(q=q, s=s, g=g, y=y)
    _check(capi().nvq_dequantize(_p(q), _p(s), _p(g), rows, k, _p(y), _dtype_code(y.dtype), _stream()),
           "nvq_dequantize")
    return y


def nv_gemm(wq, ws, g, x, out_dtype=None, y=None):
    """y[m, n] = s_t * x[m, k] @ (s_b * q)[n, k]^T with an NVFP4 weight; x bf16."""
    torch = _torch()
    n, k = _weight(wq, ws, 16, "nv_gemm")
    _gscale(g, "g", wq.device)
    m = _activations(x, k, wq.device)
    out_dtype = out_dtype or (y.dtype if y is not None else torch.bfloat16)
    y = _out(y, "y", (m, n), out_dtype, wq.device, real=True)
    _on_device(wq=wq, ws=ws, g=g, x=x, y=y)
    _check(capi().nvq_gemm(_p(wq), _p(ws), _p(g), n, k, _p(x), m, _p(y), _dtype_code(y.dtype), _stream()),
           "nvq_gemm")
    return y


# ------------------------------------------------------------------ TransFP4 blocks

def transfp4_quantize(x, gscale=None, q=None, s=None, meta=None, res=None, g=None):
    """TransFP4 quantize x[rows, k] -> (q[rows, k/2], s[rows, k/16] E4M3,
    meta[rows, k/32] (bit 7 INT4 tag, bits 0-4 residual position),
    res[rows, k/32] bf16 residuals, g[1] fp32 tensor scale).  gscale as in
    nv_quantize."""
    torch = _torch()
    _need(x, "x", _floats())
    rows, k = x.shape
    _k_blocks(k, 32, "transfp4_quantize")
    dev = x.device
    compute, g = _tensor_scale_arg(gscale, g, dev)
    q = _out(q, "q", (rows, k // 2), torch.uint8, dev)
    s = _out(s, "s", (rows, k // 16), torch.uint8, dev)
    meta = _out(meta, "meta", (rows, k // 32), torch.uint8, dev)
    res = _out(res, "res", (rows, k // 32), torch.bfloat16, dev)
    _on_device(x=x, g=g, q=q, s=s, meta=meta, res=res)
    _check(capi().mxq_transfp4_quantize(_p(x), _dtype_code(x.dtype), rows, k, _p(g), int(compute), _p(q), _p(s),
                                        _p(meta), _p(res), _stream()), "mxq_transfp4_quantize")
    return q, s, meta, res, g


def transfp4_dequantize(q, s, meta, res, g, dtype=None, y=None):
    """x_hat[rows, k] (fp32 or bf16) from the TransFP4 arrays."""
    torch = _torch()
    _need(q, "q", torch.uint8)
    rows, k = q.shape[0], q.shape[1] * 2
    _k_blocks(k, 32, "transfp4_dequantize")
    dev = q.device
    _need(s, "s", torch.uint8, (rows, k // 16), device=dev)
    _need(meta, "meta", torch.uint8, (rows, k // 32), device=dev)
    _need(res, "res", torch.bfloat16, (rows, k // 32), device=dev)
    _gscale(g, "g", dev)
    dtype = dtype or (y.dtype if y is not None else torch.float32)
    y = _out(y, "y", (rows, k), dtype, dev, real=True)
    _on_device(q=q, s=s, meta=meta, res=res, g=g, y=y)
    _check(capi().mxq_transfp4_dequantize(_p(q), _p(s), _p(meta), _p(res), _p(g), rows, k, _p(y),
                                          _dtype_code(y.dtype), _stream()), "mxq_transfp4_dequantize")
    return y


# ------------------------------------------------------------------ norm, paged cache, attention

# These run between the products of a decode step, where a call's host time is
# its cost: one pass of plain comparisons accepts a good call, and only a call
# that fails it goes through the named checks (which then raise).

def rmsnorm_quantize_fp8(x, weight, residual=None, eps=1e-6, q=None, s=None, r=None):
    """r = x + residual (rounded to x's dtype), y = r / sqrt(mean r^2 + eps) * weight
    along rows, MXFP8 of y: (q[rows, k] E4M3 codes u8, s[rows, k/32] E8M0 u8, r).

    x, residual [rows, k] and weight [k], all bf16 or all fp32; k % 32 == 0.
    Without a residual r is x itself.  Pass r=residual (or r=x) to update the
    residual stream in place."""
    torch = _torch()
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        _need(x, "x", _floats())
    rows, k = x.shape
    dt, dev = x.dtype, x.get_device()
    code = MXQ_BF16 if dt is torch.bfloat16 else MXQ_F32
    good = ((code == MXQ_BF16 or dt is torch.float32) and dev >= 0 and k % 32 == 0 and eps > 0 and x.is_contiguous()
            and _same(weight, dt, (k,), dev) and (r is None or residual is not None or r is x)
            and (residual is None or _same(residual, dt, x.shape, dev))
            and (q is None or _same(q, torch.uint8, x.shape, dev))
            and (s is None or _same(s, torch.uint8, (rows, k // 32), dev))
            and (r is None or _same(r, dt, x.shape, dev)))
    if not good:
        _need(x, "x", _floats())
        _k_blocks(k, 32, "rmsnorm_quantize_fp8")
        _need(weight, "weight", x.dtype, (k,))
        if not eps > 0:
            raise ValueError(f"eps must be > 0, got {eps}")
        on = {"x": x, "weight": weight, "q": _out(q, "q", (rows, k), torch.uint8, x.device),
              "s": _out(s, "s", (rows, k // 32), torch.uint8, x.device)}
        if residual is None:
            if r is not None and r is not x:
                raise ValueError("r is only written with a residual")
        else:
            _need(residual, "residual", x.dtype, (rows, k))
            on["residual"], on["r"] = residual, _out(r, "r", (rows, k), x.dtype, x.device)
        _on_device(**on)
    if q is None:
        q = torch.empty_like(x, dtype=torch.uint8)
    if s is None:
        s = x.new_empty((rows, k // 32), dtype=torch.uint8)
    if residual is None:
        rp, op, r = None, None, x
    else:
        if r is None:
            r = torch.empty_like(x)
        rp, op = residual.data_ptr(), r.data_ptr()
    _check(capi().mxq_rmsnorm_quantize_fp8(x.data_ptr(), rp, weight.data_ptr(), code, rows, k, eps, op, q.data_ptr(),
                                           s.data_ptr(), _stream(dev)), "mxq_rmsnorm_quantize_fp8")
    return q, s, r


def _same(t, dtype, shape, dev):
    """A contiguous tensor of this dtype, shape and device (an index)."""
    return (isinstance(t, _torch_module.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev
            and t.is_contiguous())


class KVCache(NamedTuple):
    """A paged MXFP8 or MXFP4 cache: kq, vq [pages, kv_heads, page_size, D] E4M3
    codes (or [..., D/2] packed E2M1), ks [pages, kv_heads, page_size, D/32] and
    vs [pages, kv_heads, D/32, page_size] E8M0 codes, all uint8 and contiguous.
    A token's slot is page * page_size + its position in the page."""
    kq: object
    ks: object
    vq: object
    vs: object


def kv_cache(pages, page_size, kv_heads, head_dim, fmt="mxfp8", device="cuda"):
    """A new zero-filled KVCache; fmt "mxfp8" or "mxfp4", page_size a power of
    two from 16 to 1024, head_dim a multiple of 32 (64, 128 or 256 for
    paged_attention)."""
    torch = _torch()
    if fmt not in ("mxfp8", "mxfp4"):
        raise ValueError(f"fmt must be 'mxfp8' or 'mxfp4', got {fmt!r}")
    _k_blocks(head_dim, 32, "kv_cache")
    code = head_dim if fmt == "mxfp8" else head_dim // 2
    shapes = ((pages, kv_heads, page_size, code), (pages, kv_heads, page_size, head_dim // 32),
              (pages, kv_heads, page_size, code), (pages, kv_heads, head_dim // 32, page_size))
    return KVCache(*(torch.zeros(sh, dtype=torch.uint8, device=device) for sh in shapes))


def _cache(cache, dev):
    """(pages, kv_heads, page_size, head_dim, format) of a KVCache after
    validation; its tensors are on device `dev` (an index) or the call is
    refused by the caller's _on_device."""
    torch = _torch()
    kq, ks, vq, vs = cache
    if isinstance(kq, torch.Tensor) and isinstance(ks, torch.Tensor) and kq.dim() == 4 and ks.dim() == 4:
        u8 = torch.uint8
        pages, heads, page, w = kq.shape
        n = ks.shape[3]
        d = 32 * n
        if ((w == d or 2 * w == d) and _same(kq, u8, kq.shape, dev) and _same(ks, u8, (pages, heads, page, n), dev)
                and _same(vq, u8, kq.shape, dev) and _same(vs, u8, (pages, heads, n, page), dev)):
            return pages, heads, page, d, MXQ_MXFP8 if w == d else MXQ_MXFP4
    _need(kq, "kq", torch.uint8, ndim=4)
    _need(ks, "ks", torch.uint8, ndim=4)
    pages, heads, page, w = kq.shape
    d = ks.shape[3] * 32
    if w != d and 2 * w != d:
        raise ValueError(f"kq has {w} bytes a row, ks names head_dim {d}: MXFP8 has {d}, MXFP4 {d // 2}")
    _need(ks, "ks", torch.uint8, (pages, heads, page, d // 32))
    _need(vq, "vq", torch.uint8, (pages, heads, page, w))
    _need(vs, "vs", torch.uint8, (pages, heads, d // 32, page))
    _on_device(kq=kq, ks=ks, vq=vq, vs=vs)
    raise ValueError("the cache and the other operands are on different devices")


def _index(t):
    """The device index of a tensor (-1: host); other things fail their own check later."""
    return t.get_device() if isinstance(t, _torch().Tensor) else -1


def _rows(t, name, dtype, heads, dim):
    """[n, heads, dim] whose rows are contiguous inside (a slice of a fused
    projection's output): the row stride in elements."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in dtype:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtype)}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must have shape [n, {heads or 'heads'}, {dim}], got {tuple(shape)}")
    row, inner, one = t.stride()
    if one != 1 or (inner != dim and shape[1] > 1):
        raise ValueError(f"{name} must be contiguous in its last two dims")
    return row if shape[0] > 1 else shape[1] * dim


def kv_append(cache, k, v, slots):
    """Quantize new tokens k, v [tokens, kv_heads, head_dim] (bf16 or fp32, row
    stride free) into their slots (int64 [tokens]; outside the cache, e.g. -1:
    skipped).  The cache is updated in place."""
    torch = _torch()
    dev = _index(cache[0])
    pages, heads, page, d, fmt = _cache(cache, dev)
    k_stride = _rows(k, "k", _floats(), heads, d)
    v_stride = _rows(v, "v", (k.dtype,), heads, d)
    n = k.shape[0]
    if v.shape[0] != n:
        raise ValueError(f"k has {n} tokens, v {v.shape[0]}")
    kq, ks, vq, vs = cache
    if dev < 0 or not _same(slots, torch.int64, (n,), dev) or k.get_device() != dev or v.get_device() != dev:
        _need(slots, "slots", torch.int64, (n,))
        _on_device(kq=kq, k=k, v=v, slots=slots)
    _check(capi().mxq_kv_append(k.data_ptr(), k_stride, v.data_ptr(), v_stride, _dtype_code(k.dtype),
                                slots.data_ptr(), n, pages, heads, page, d, fmt, kq.data_ptr(), ks.data_ptr(),
                                vq.data_ptr(), vs.data_ptr(), _stream(dev)), "mxq_kv_append")


def rope_append(cache, q, k, v, slots, positions, freqs, axes=None, interleaved=False, out=None):
    """Rotate new queries and keys by their positions and quantize keys and
    values into their slots (as kv_append, from the rotated keys, rounded once).
    Returns the rotated queries, bf16 [tokens, q_heads, head_dim].

    q [tokens, q_heads, head_dim], k, v [tokens, kv_heads, head_dim], all bf16 or
    all fp32, row strides free; slots int64 [tokens] (outside the cache, e.g. -1:
    not written); positions int64 [tokens]; freqs fp32 [n], radians a position: a
    head's first 2 n elements turn in pairs (i, n + i), or (2 i, 2 i + 1) if
    interleaved; n % 8 == 0.  With several position axes (time, height, width),
    positions is [axes, tokens] and axes uint8 [n] names the axis of each pair.
    out must not overlap q, k or v."""
    torch = _torch()
    dev = _index(cache[0])
    pages, heads, page, d, fmt = _cache(cache, dev)
    q_stride = _rows(q, "q", _floats(), None, d)
    k_stride = _rows(k, "k", (q.dtype,), heads, d)
    v_stride = _rows(v, "v", (q.dtype,), heads, d)
    n, q_heads, _ = q.shape
    if k.shape[0] != n or v.shape[0] != n:
        raise ValueError(f"q has {n} tokens, k {k.shape[0]}, v {v.shape[0]}")
    if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1 or not _same(freqs, torch.float32, freqs.shape, dev):
        _need(freqs, "freqs", torch.float32, ndim=1)
    pairs = freqs.shape[0]
    if axes is None:
        count = 1
        if not _same(positions, torch.int64, (n,), dev):
            _need(positions, "positions", torch.int64, (n,))
    else:
        if not isinstance(positions, torch.Tensor) or positions.dim() != 2 or positions.shape[0] < 2:
            raise ValueError("with axes, positions must have shape [2 or more axes, tokens]")
        count = positions.shape[0]
        if not _same(positions, torch.int64, (count, n), dev) or not _same(axes, torch.uint8, (pairs,), dev):
            _need(positions, "positions", torch.int64, (count, n))
            _need(axes, "axes", torch.uint8, (pairs,))
    if not _same(slots, torch.int64, (n,), dev):
        _need(slots, "slots", torch.int64, (n,))
    if out is None:
        out = q.new_empty((n, q_heads, d), dtype=torch.bfloat16)
    else:
        _need(out, "out", torch.bfloat16, (n, q_heads, d))
    on = (q, k, v, slots, positions, freqs, out) if axes is None else (q, k, v, slots, positions, freqs, out, axes)
    if dev < 0 or any(t.get_device() != dev for t in on):
        names = ("q", "k", "v", "slots", "positions", "freqs", "out", "axes")
        _on_device(kq=cache[0], **dict(zip(names, on)))
    kq, ks, vq, vs = cache
    _check(capi().mxq_rope_append(q.data_ptr(), q_stride, k.data_ptr(), k_stride, v.data_ptr(), v_stride,
                                  _dtype_code(q.dtype), positions.data_ptr(), count,
                                  None if axes is None else axes.data_ptr(), freqs.data_ptr(), pairs,
                                  int(bool(interleaved)), slots.data_ptr(), n, q_heads, pages, heads, page, d, fmt,
                                  kq.data_ptr(), ks.data_ptr(), vq.data_ptr(), vs.data_ptr(), out.data_ptr(),
                                  _stream(dev)), "mxq_rope_append")
    return out


def kv_read(cache, slots, dtype=None, k=None, v=None):
    """The slots' keys and values, (k, v) [tokens, kv_heads, head_dim] in dtype
    (default bf16); a slot outside the cache reads as zeros."""
    torch = _torch()
    dev = _index(cache[0])
    pages, heads, page, d, fmt = _cache(cache, dev)
    kq, ks, vq, vs = cache
    _need(slots, "slots", torch.int64, ndim=1)
    n = slots.shape[0]
    dtype = dtype or (k.dtype if k is not None else torch.bfloat16)
    k = _out(k, "k", (n, heads, d), dtype, kq.device, real=True)
    v = _out(v, "v", (n, heads, d), dtype, kq.device, real=True)
    if dev < 0 or slots.get_device() != dev or k.get_device() != dev or v.get_device() != dev:
        _on_device(kq=kq, slots=slots, k=k, v=v)
    _check(capi().mxq_kv_read(kq.data_ptr(), ks.data_ptr(), vq.data_ptr(), vs.data_ptr(), slots.data_ptr(), n, pages,
                              heads, page, d, fmt, k.data_ptr(), v.data_ptr(), _dtype_code(dtype), _stream(dev)),
           "mxq_kv_read")
    return k, v


def paged_attention(q, cache, table, lens, scale=None, window=0, sinks=None, out_dtype=None, out=None, workspace=None):
    """Attention of one new token per sequence over the cache: out[batch, q_heads, D].

    q [batch, q_heads, D] bf16 (row stride free); table [batch, width] int32 page
    ids (row stride free); lens [batch] int32 lengths including the new token;
    scale defaults to 1/sqrt(D); window > 0 sees the last `window` positions
    only; sinks [q_heads] fp32 adds exp(sinks) to each head's denominator.  A
    sequence with nothing visible gives zeros.  workspace: a uint8 device
    tensor to use for partial results (allocated if None).  A table no wider
    than the batch needs gives the best split."""
    torch = _torch()
    dev = _index(cache[0])
    pages, heads, page, d, fmt = _cache(cache, dev)
    q_stride = _rows(q, "q", (torch.bfloat16,), None, d)
    batch, q_heads, _ = q.shape
    if q_heads % heads != 0:
        raise ValueError(f"{q_heads} query heads over {heads} cache heads")
    if not isinstance(table, torch.Tensor) or table.dtype is not torch.int32:
        raise TypeError("table must be an int32 tensor")
    shape = table.shape
    if len(shape) != 2 or shape[0] != batch or (shape[1] > 1 and table.stride(1) != 1):
        raise ValueError(f"table must have shape [{batch}, width] with contiguous rows, got {tuple(shape)}")
    width = shape[1]
    table_stride = table.stride(0) if batch > 1 else max(width, table.stride(0))
    if not _same(lens, torch.int32, (batch,), dev):
        _need(lens, "lens", torch.int32, (batch,))
    kq, ks, vq, vs = cache
    out_dtype = out_dtype or (out.dtype if out is not None else torch.bfloat16)
    if out is None and out_dtype is torch.bfloat16:
        out = q.new_empty((batch, q_heads, d))
    else:
        out = _out(out, "out", (batch, q_heads, d), out_dtype, kq.device, real=True)
    if sinks is not None and not _same(sinks, torch.float32, (q_heads,), dev):
        _need(sinks, "sinks", torch.float32, (q_heads,))
    lib = capi()
    need = ctypes.c_int64()
    code = lib.mxq_paged_attention_workspace(batch, q_heads, heads, page, d, width, window, ctypes.byref(need))
    if code != 0:
        _check(code, "mxq_paged_attention_workspace")
    need = need.value
    if workspace is None:
        wp = None
        if need:
            workspace = kq.new_empty(need)
            wp = workspace.data_ptr()
    else:
        _need(workspace, "workspace", torch.uint8, ndim=1)
        need, least = workspace.shape[0], need
        if need < least:
            raise ValueError(f"workspace has {need} bytes, {least} are needed")
        wp = workspace.data_ptr()
    if (dev < 0 or q.get_device() != dev or table.get_device() != dev or lens.get_device() != dev
            or out.get_device() != dev or (sinks is not None and sinks.get_device() != dev)
            or (workspace is not None and workspace.get_device() != dev)):
        on = {"kq": kq, "q": q, "table": table, "lens": lens, "out": out, "sinks": sinks, "workspace": workspace}
        _on_device(**{name: t for name, t in on.items() if t is not None})
    code = lib.mxq_paged_attention(q.data_ptr(), q_stride, kq.data_ptr(), ks.data_ptr(), vq.data_ptr(), vs.data_ptr(),
                                   table.data_ptr(), width, table_stride, lens.data_ptr(),
                                   None if sinks is None else sinks.data_ptr(), batch, q_heads, pages, heads, page, d,
                                   fmt, 1.0 / math.sqrt(d) if scale is None else scale, window, wp, need,
                                   out.data_ptr(), _dtype_code(out_dtype), _stream(dev))
    if code != 0:
        _check(code, "mxq_paged_attention")
    return out


def tree_mask(parents, device="cuda"):
    """The masks of tree_attention, int64 [batch, drafts, words], of trees of
    drafted tokens: parents is a list of lists (one list: a batch of one), where
    parents[b][i] is the index of the drafted token that i follows, below i, or -1
    where it follows the context.  A token sees its ancestors and itself.  Trees
    shorter than the longest are padded with tokens that see no drafted token and
    that none sees."""
    torch = _torch()
    trees = parents.tolist() if isinstance(parents, torch.Tensor) else list(parents)
    if not trees or not hasattr(trees[0], "__len__"):
        trees = [trees]
    drafts = max(len(t) for t in trees)
    if drafts < 1:
        raise ValueError("a tree needs a drafted token")
    words = (drafts + 63) // 64
    masks = torch.zeros(len(trees), drafts, words, dtype=torch.int64)
    for b, tree in enumerate(trees):
        seen = []
        for i, p in enumerate(tree):
            if not -1 <= p < i:
                raise ValueError(f"parents[{b}][{i}] is {p}: a drafted token follows one before it, or -1")
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
            for w in range(words):
                v = seen[i] >> (64 * w) & 0xFFFFFFFFFFFFFFFF
                masks[b, i, w] = v - (1 << 64) if v >> 63 else v
    return masks.to(device)


def tree_attention(q, cache, table, context, mask, scale=None, window=0, first=0, sinks=None, out_dtype=None, out=None,
                   workspace=None):
    """Attention of several drafted tokens per sequence over the cache, which
    holds them already: out[batch * drafts, q_heads, D].

    q [batch * drafts, q_heads, D] bf16 (row stride free), row b * drafts + i the
    i-th drafted token of sequence b, at cache position context[b] + i; context
    [batch] int32, tokens before the drafted ones; mask [batch, drafts, words]
    int64, bit j of token i's words (64 a word): it sees drafted token j
    (tree_mask makes them of a tree); table [batch, width] int32 page ids (row
    stride free).  window > 0 hides positions that far back or further, but not
    the `first` first positions of the sequence; a drafted token's position is
    context + the drafted tokens before it that it sees.  scale, sinks and
    workspace as in paged_attention; out must not overlap q.  A token that sees
    nothing gives zeros."""
    torch = _torch()
    dev = _index(cache[0])
    pages, heads, page, d, fmt = _cache(cache, dev)
    q_stride = _rows(q, "q", (torch.bfloat16,), None, d)
    rows, q_heads, _ = q.shape
    if q_heads % heads != 0:
        raise ValueError(f"{q_heads} query heads over {heads} cache heads")
    if not isinstance(mask, torch.Tensor) or mask.dim() != 3 or not _same(mask, torch.int64, mask.shape, dev):
        _need(mask, "mask", torch.int64, ndim=3)
    batch, drafts, words = mask.shape
    if words != (drafts + 63) // 64:
        raise ValueError(f"mask must have {(drafts + 63) // 64} words for {drafts} drafted tokens, got {words}")
    if rows != batch * drafts:
        raise ValueError(f"q has {rows} rows for {batch} sequences of {drafts} drafted tokens")
    if not isinstance(table, torch.Tensor) or table.dtype is not torch.int32:
        raise TypeError("table must be an int32 tensor")
    shape = table.shape
    if len(shape) != 2 or shape[0] != batch or (shape[1] > 1 and table.stride(1) != 1):
        raise ValueError(f"table must have shape [{batch}, width] with contiguous rows, got {tuple(shape)}")
    width = shape[1]
    table_stride = table.stride(0) if batch > 1 else max(width, table.stride(0))
    if not _same(context, torch.int32, (batch,), dev):
        _need(context, "context", torch.int32, (batch,))
    kq, ks, vq, vs = cache
    out_dtype = out_dtype or (out.dtype if out is not None else torch.bfloat16)
    if out is None and out_dtype is torch.bfloat16:
        out = q.new_empty((rows, q_heads, d))
    else:
        out = _out(out, "out", (rows, q_heads, d), out_dtype, kq.device, real=True)
    if sinks is not None and not _same(sinks, torch.float32, (q_heads,), dev):
        _need(sinks, "sinks", torch.float32, (q_heads,))
    lib = capi()
    need = ctypes.c_int64()
    code = lib.mxq_tree_attention_workspace(batch, drafts, q_heads, heads, page, d, width, window, first,
                                            ctypes.byref(need))
    if code != 0:
        _check(code, "mxq_tree_attention_workspace")
    need = need.value
    if workspace is None:
        wp = None
        if need:
            workspace = kq.new_empty(need)
            wp = workspace.data_ptr()
    else:
        _need(workspace, "workspace", torch.uint8, ndim=1)
        need, least = workspace.shape[0], need
        if need < least:
            raise ValueError(f"workspace has {need} bytes, {least} are needed")
        wp = workspace.data_ptr()
    if (dev < 0 or q.get_device() != dev or table.get_device() != dev or context.get_device() != dev
            or mask.get_device() != dev or out.get_device() != dev or (sinks is not None and sinks.get_device() != dev)
            or (workspace is not None and workspace.get_device() != dev)):
        on = {"kq": kq, "q": q, "table": table, "context": context, "mask": mask, "out": out, "sinks": sinks,
              "workspace": workspace}
        _on_device(**{name: t for name, t in on.items() if t is not None})
    code = lib.mxq_tree_attention(q.data_ptr(), q_stride, kq.data_ptr(), ks.data_ptr(), vq.data_ptr(), vs.data_ptr(),
                                  table.data_ptr(), width, table_stride, context.data_ptr(), mask.data_ptr(),
                                  None if sinks is None else sinks.data_ptr(), batch, drafts, q_heads, pages, heads,
                                  page, d, fmt, 1.0 / math.sqrt(d) if scale is None else scale, window, first, wp, need,
                                  out.data_ptr(), _dtype_code(out_dtype), _stream(dev))
    if code != 0:
        _check(code, "mxq_tree_attention")
    return out


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, tokens=None, shares=None, workspace=None):
    """Draw a token of each row: (tokens int32 [rows], shares fp32 [rows]).

    logits [rows, vocab] bf16 or fp32 (row stride free); u [rows] fp32 random
    numbers in [0, 1).  Weights are exp((logit - largest) / temperature), ordered
    by logit, equal ones by index; what may be drawn is the shortest of three
    prefixes of that order: top_k tokens, of them the fewest whose weights reach
    top_p of theirs, and those of weight min_p and more (of the largest).  The
    token is the first by index where the running sum of these weights passes u
    times their sum; its share is its weight over that sum.  temperature 0: the
    largest.  top_k 0, top_p 1 and min_p 0 leave all.  Each setting is a number or
    a tensor [rows] (top_k int32, the others fp32).  A row with a NaN or +inf, or
    nothing but -inf, gives token -1 and share NaN.  tokens and shares, if given,
    must not overlap what is read."""
    torch = _torch()
    if not isinstance(logits, torch.Tensor):
        raise TypeError(f"logits must be a torch.Tensor, got {type(logits).__name__}")
    code = _dtype_code(logits.dtype)
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError(f"logits must have shape [rows, vocab] with contiguous rows, got {tuple(logits.shape)}")
    dev = logits.get_device()
    rows, vocab = logits.shape
    stride = logits.stride(0) if rows > 1 else vocab
    if not _same(u, torch.float32, (rows,), dev):
        _need(u, "u", torch.float32, (rows,))
    on = {"logits": logits, "u": u}
    given = []
    for name, v, dt in (("temperature", temperature, torch.float32), ("top_k", top_k, torch.int32),
                        ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32)):
        if isinstance(v, torch.Tensor):
            if not _same(v, dt, (rows,), dev):
                _need(v, name, dt, (rows,))
            on[name] = v
            given += [v.data_ptr(), 0]
        else:
            given += [None, v]
    if tokens is None:
        tokens = logits.new_empty(rows, dtype=torch.int32)
    elif not _same(tokens, torch.int32, (rows,), dev):
        _need(tokens, "tokens", torch.int32, (rows,))
    if shares is None:
        shares = logits.new_empty(rows, dtype=torch.float32)
    elif not _same(shares, torch.float32, (rows,), dev):
        _need(shares, "shares", torch.float32, (rows,))
    on["tokens"], on["shares"] = tokens, shares
    lib = capi()
    need = ctypes.c_int64()
    status = lib.mxq_sample_workspace(rows, vocab, ctypes.byref(need))
    if status != 0:
        _check(status, "mxq_sample_workspace")
    need, wp = need.value, None
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, ndim=1)
        on["workspace"] = workspace
        need, least = workspace.shape[0], need
        if need < least:
            raise ValueError(f"workspace has {need} bytes, {least} are needed")
        wp = workspace.data_ptr()
    elif need:
        workspace = logits.new_empty(need, dtype=torch.uint8)
        wp = workspace.data_ptr()
    if dev < 0 or any(t.get_device() != dev for t in on.values()):
        _on_device(**on)
    status = lib.mxq_sample(logits.data_ptr(), code, stride, rows, vocab, u.data_ptr(), *given, wp, need,
                            tokens.data_ptr(), shares.data_ptr(), _stream(dev))
    if status != 0:
        _check(status, "mxq_sample")
    return tokens, shares


from . import nvq  # noqa: E402  (the NVFP4 names: nvq.quantize / nvq.dequantize / nvq.gemm)
