"""Thin Python binding of librq (include/rq.h): argument marshalling only.

Every step of every call runs in librq's sm_100a kernels; torch is used for
device memory, streams and output allocation.  There is no fallback: if
librq.so is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "librq.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "rq.h")

GROUP = 64
MAX_DECODE_M = 32

STATUS = {0: "RQ_OK", 1: "RQ_ERR_NULL", 2: "RQ_ERR_BITS", 3: "RQ_ERR_SHAPE", 4: "RQ_ERR_ALIGN",
          5: "RQ_ERR_NONFINITE", 6: "RQ_ERR_RANGE", 7: "RQ_ERR_TIMEOUT", 8: "RQ_ERR_CUDA"}
OK, ERR_NULL, ERR_BITS, ERR_SHAPE, ERR_ALIGN, ERR_NONFINITE, ERR_RANGE, ERR_TIMEOUT, ERR_CUDA = range(9)
DECODE_KERNELS = {"auto": 0, "rowtile": 1, "cluster": 2, "rowblock": 3, "tensor": 4}

_lib = None


class RQError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = f"{what}: {STATUS.get(status, status)}"
        if status == ERR_CUDA and _lib is not None:
            msg += f" ({_lib.rq_last_cuda_error().decode()})"
        super().__init__(msg)


def lib():
    """Load librq.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"librq.so not built at {LIB_PATH}: run "
                           "`python -m weight_only_quantized_g64_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    i64, vp, i32, u64 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64
    L.rq_codes_bytes.argtypes = [i64, i64, i32]
    L.rq_codes_bytes.restype = ctypes.c_size_t
    L.rq_scales_bytes.argtypes = [i64, i64]
    L.rq_scales_bytes.restype = ctypes.c_size_t
    L.rq_quantize_g64.argtypes = [vp, i64, i64, i32, vp, vp, vp, vp]
    L.rq_quantize_g64.restype = i32
    L.rq_quantize_g64_ex2.argtypes = [vp, i64, i64, i32, vp, vp, i32, vp, vp, vp, vp, vp]
    L.rq_quantize_g64_ex2.restype = i32
    L.rq_gemv_wq.argtypes = [vp, i64, i64, vp, vp, i64, i32, vp, vp]
    L.rq_gemv_wq.restype = i32
    L.rq_gemm_wq.argtypes = [vp, i64, i64, vp, vp, i64, i32, vp, vp]
    L.rq_gemm_wq.restype = i32
    L.rq_gemv_wq_noalloc.argtypes = [vp, i64, i64, vp, vp, i64, i32, vp, vp]
    L.rq_gemv_wq_noalloc.restype = i32
    L.rq_rkv_fused.argtypes = [vp, i64, i64, i64, i32] + [vp] * 9 + [vp]
    L.rq_rkv_fused.restype = i32
    L.rq_gptq_hessian.argtypes = [vp, i64, i64, vp, vp]
    L.rq_gptq_hessian.restype = i32
    L.rq_gptq_factor.argtypes = [vp, i64, ctypes.c_double, vp, vp, vp, vp]
    L.rq_gptq_factor.restype = i32
    L.rq_gptq_g64.argtypes = [vp, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp]
    L.rq_gptq_g64.restype = i32
    L.rq_gemv_wq_ex.argtypes = [vp, i64, i64, vp, vp, i64, i32, vp, i32, i32, vp]
    L.rq_gemv_wq_ex.restype = i32
    L.rq_rkv_fused3.argtypes = [vp, vp, vp, i64, i64, i64, i32] + [vp] * 9 + [i32, vp]
    L.rq_rkv_fused3.restype = i32
    L.rq_quantize_p8_g16.argtypes = [vp, i64, i64, vp, vp, i32, vp, vp, vp, vp, vp]
    L.rq_quantize_p8_g16.restype = i32
    L.rq_quantize_p4a_g32.argtypes = [vp, i64, i64, vp, vp, i32, vp, vp, vp, vp, vp, vp]
    L.rq_quantize_p4a_g32.restype = i32
    L.rq_gemv_p8_g16.argtypes = [vp, i64, i64, vp, vp, i64, vp, vp]
    L.rq_gemv_p8_g16.restype = i32
    L.rq_gemv_p4a_g32.argtypes = [vp, i64, i64, vp, vp, vp, i64, vp, vp]
    L.rq_gemv_p4a_g32.restype = i32
    L.rq_lora_work_bytes.argtypes = [i64, i64]
    L.rq_lora_work_bytes.restype = ctypes.c_size_t
    L.rq_lora_add.argtypes = [vp, i64, i64, vp, vp, i64, i64, vp, vp, vp, vp, vp, i64, i32, i32, vp, vp, vp]
    L.rq_lora_add.restype = i32
    f32 = ctypes.c_float
    L.rq_norm_residual.argtypes = [vp, i64, i64, i64, i32, i32, i64, vp, vp, f32, vp, i64, vp, i64, i32, vp, vp, i32,
                                   vp, vp, f32, vp, vp, vp]
    L.rq_norm_residual.restype = i32
    L.rq_tmix_ckpt_bytes.argtypes = [i64, i64, i64]
    L.rq_tmix_ckpt_bytes.restype = ctypes.c_size_t
    L.rq_tmix_scan.argtypes = [vp] * 6 + [i64, i64, i64, i32, vp, i64, vp, vp, vp, i64, vp, vp, vp, vp]
    L.rq_tmix_scan.restype = i32
    L.rq_tmix_scan_bwd.argtypes = [vp] * 6 + [i64, i64, i64, i32, vp, i64] + [vp] * 13
    L.rq_tmix_scan_bwd.restype = i32
    L.rq_tmix_step.argtypes = [vp] * 6 + [i64, i64, i64, i32, vp, vp, vp, i64, vp, vp, vp]
    L.rq_tmix_step.restype = i32
    L.rq_set_pdl.argtypes = [i32]
    L.rq_set_pdl.restype = i32
    L.rq_set_decode_kernel.argtypes = [i32]
    L.rq_set_decode_kernel.restype = i32
    L.rq_decode_kernel_for.argtypes = [i64, i64, i64, i32, i32, ctypes.POINTER(ctypes.c_int)]
    L.rq_decode_kernel_for.restype = i32
    L.rq_set_wait_limit_ns.argtypes = [u64]
    L.rq_set_wait_limit_ns.restype = i32
    L.rq_read_device_status.argtypes = [ctypes.POINTER(ctypes.c_int), i32]
    L.rq_read_device_status.restype = i32
    L.rq_selftest_bounded_wait.argtypes = [u64, vp]
    L.rq_selftest_bounded_wait.restype = i32
    L.rq_status_string.argtypes = [i32]
    L.rq_status_string.restype = ctypes.c_char_p
    L.rq_last_cuda_error.argtypes = []
    L.rq_last_cuda_error.restype = ctypes.c_char_p
    L.rq_version.argtypes = []
    L.rq_version.restype = ctypes.c_char_p
    _lib = L
    return L


def header_functions() -> list[str]:
    """Names of every function include/rq.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[a-z_]+\s*\*?\s*(rq_[a-z0-9_]+)\s*\(",
                                 text, flags=re.M)))


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _p(t):
    return None if t is None else t.data_ptr()


def _check(st: int, what: str):
    if st != OK:
        raise RQError(st, what)


def codes_bytes(N: int, K: int, bits: int) -> int:
    return int(lib().rq_codes_bytes(N, K, bits))


def scales_bytes(N: int, K: int) -> int:
    return int(lib().rq_scales_bytes(N, K))


def empty_weights(N: int, K: int, bits: int, device="cuda"):
    """Allocate (codes uint8 [N, K*bits/8], scales int16 [N, K/64]) for N x K."""
    codes = torch.empty((N, K * bits // 8), dtype=torch.uint8, device=device)
    scales = torch.empty((N, K // GROUP), dtype=torch.int16, device=device)
    return codes, scales


def quantize_g64(W: torch.Tensor, bits: int, codes=None, scales=None, dev_status=None,
                 stream=None):
    """RTN group-64 quantization of fp32 W[N, K] on the GPU -> (codes, scales)."""
    N, K = W.shape
    if codes is None:
        codes, scales = empty_weights(N, K, bits, W.device)
    _check(lib().rq_quantize_g64(_p(W), N, K, bits, _p(codes), _p(scales), _p(dev_status),
                                 _stream(stream)), "rq_quantize_g64")
    return codes, scales


def quantize_g64_ex2(W: torch.Tensor, e2: torch.Tensor, bits: int, factors: torch.Tensor,
                     codes=None, scales=None, chosen=None, dev_status=None, stream=None):
    """Group-64 quantization of fp32 W[N, K] with each group's scale chosen by
    an E[x^2]-weighted search over `factors` (fp32 device, 1..16 values);
    e2: fp32 [K] device.  Returns (codes, scales, chosen int32 [N, K/64])."""
    N, K = W.shape
    if codes is None:
        codes, scales = empty_weights(N, K, bits, W.device)
    if chosen is None:
        chosen = torch.empty((N, K // GROUP), dtype=torch.int32, device=W.device)
    _check(lib().rq_quantize_g64_ex2(_p(W), N, K, bits, _p(e2), _p(factors), int(factors.numel()),
                                     _p(codes), _p(scales), _p(chosen), _p(dev_status),
                                     _stream(stream)), "rq_quantize_g64_ex2")
    return codes, scales, chosen


def quantize_p8_g16(W: torch.Tensor, e2=None, factors=None, dev_status=None, stream=None):
    """Preset int8 symmetric groups of 16 -> (codes int8-as-uint8 [N, K],
    scales int16 [N, K/16], chosen int32 [N, K/16])."""
    N, K = W.shape
    codes = torch.empty((N, K), dtype=torch.uint8, device=W.device)
    scales = torch.empty((N, K // 16), dtype=torch.int16, device=W.device)
    chosen = torch.empty((N, K // 16), dtype=torch.int32, device=W.device)
    nf = 0 if factors is None else int(factors.numel())
    _check(lib().rq_quantize_p8_g16(_p(W), N, K, _p(e2), _p(factors), nf, _p(codes), _p(scales),
                                    _p(chosen), _p(dev_status), _stream(stream)), "rq_quantize_p8_g16")
    return codes, scales, chosen


def quantize_p4a_g32(W: torch.Tensor, e2=None, factors=None, dev_status=None, stream=None):
    """Preset int4 asymmetric groups of 32 in super-blocks -> (codes uint8
    [N, K/2], sub uint8 [N, K/32, 2], sup int16 [N, K/256, 2], chosen int32 [N, K/32])."""
    N, K = W.shape
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device)
    sub = torch.empty((N, K // 32, 2), dtype=torch.uint8, device=W.device)
    sup = torch.empty((N, K // 256, 2), dtype=torch.int16, device=W.device)
    chosen = torch.empty((N, K // 32), dtype=torch.int32, device=W.device)
    nf = 0 if factors is None else int(factors.numel())
    _check(lib().rq_quantize_p4a_g32(_p(W), N, K, _p(e2), _p(factors), nf, _p(codes), _p(sub), _p(sup),
                                     _p(chosen), _p(dev_status), _stream(stream)), "rq_quantize_p4a_g32")
    return codes, sub, sup, chosen


def gptq_hessian(X: torch.Tensor, H=None, stream=None):
    """H = (2/T) X^T X (fp64 [K, K]) of calibration inputs X fp16 [T, K]."""
    T, K = X.shape
    if H is None:
        H = torch.empty((K, K), dtype=torch.float64, device=X.device)
    _check(lib().rq_gptq_hessian(_p(X), T, K, _p(H), _stream(stream)), "rq_gptq_hessian")
    return H


def gptq_factor(H: torch.Tensor, damp: float = 0.01, stream=None):
    """(U fp32 [K, K], dead uint8 [K]) from H (consumed)."""
    K = H.shape[0]
    U = torch.empty((K, K), dtype=torch.float32, device=H.device)
    dead = torch.empty((K,), dtype=torch.uint8, device=H.device)
    work = torch.empty((K * K + K,), dtype=torch.float64, device=H.device)
    _check(lib().rq_gptq_factor(_p(H), K, float(damp), _p(U), _p(dead), _p(work), _stream(stream)),
           "rq_gptq_factor")
    return U, dead


def gptq_g64(W: torch.Tensor, bits: int, U: torch.Tensor, dead=None, codes=None, scales=None,
             dev_status=None, stream=None):
    """GPTQ column loop on the group-64 grid; W fp32 [N, K] is overwritten with
    the compensated weights.  Returns (codes, scales)."""
    N, K = W.shape
    if codes is None:
        codes, scales = empty_weights(N, K, bits, W.device)
    work = torch.empty((N, 128), dtype=torch.float32, device=W.device)
    _check(lib().rq_gptq_g64(_p(W), N, K, bits, _p(U), _p(dead), _p(codes), _p(scales), _p(work),
                             _p(dev_status), _stream(stream)), "rq_gptq_g64")
    return codes, scales


def gemv_wq(x: torch.Tensor, codes, scales, N: int, bits: int, y=None, stream=None):
    """Decode product y[M, N] = x[M, K] @ w_hat^T, 1 <= M <= 32."""
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _check(lib().rq_gemv_wq(_p(x), M, K, _p(codes), _p(scales), N, bits, _p(y), _stream(stream)),
           "rq_gemv_wq")
    return y


def gemv_p8_g16(x: torch.Tensor, codes, scales, N: int, y=None, stream=None):
    """Decode product of the int8 preset (codes [N, K], scales fp16 [N, K/16])."""
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _check(lib().rq_gemv_p8_g16(_p(x), M, K, _p(codes), _p(scales), N, _p(y), _stream(stream)),
           "rq_gemv_p8_g16")
    return y


def gemv_p4a_g32(x: torch.Tensor, codes, sub, sup, N: int, y=None, stream=None):
    """Decode product of the int4 asymmetric preset (codes [N, K/2], sub
    [N, K/32, 2], sup fp16 [N, K/256, 2])."""
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _check(lib().rq_gemv_p4a_g32(_p(x), M, K, _p(codes), _p(sub), _p(sup), N, _p(y),
                                 _stream(stream)), "rq_gemv_p4a_g32")
    return y


def gemv_wq_noalloc(x: torch.Tensor, codes, scales, N: int, bits: int, y=None, stream=None):
    """Decode product with the library's fixed scratch array: the library
    allocates no device memory (y is allocated here only when not given)."""
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _check(lib().rq_gemv_wq_noalloc(_p(x), M, K, _p(codes), _p(scales), N, bits, _p(y),
                                    _stream(stream)), "rq_gemv_wq_noalloc")
    return y


OUT_F32, OUT_F16 = 0, 1
EPI_NONE, EPI_RELU_SQ = 0, 1


def gemv_wq_ex(x: torch.Tensor, codes, scales, N: int, bits: int, out_dtype=torch.float32,
               epilogue: int = EPI_NONE, y=None, stream=None):
    """Decode product with the output stored as fp32 or fp16 and an optional
    fused epilogue (EPI_RELU_SQ: max(y, 0)^2)."""
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    od = OUT_F16 if y.dtype == torch.float16 else OUT_F32
    _check(lib().rq_gemv_wq_ex(_p(x), M, K, _p(codes), _p(scales), N, bits, _p(y), od, epilogue,
                               _stream(stream)), "rq_gemv_wq_ex")
    return y


def rkv_fused3(xr: torch.Tensor, xk: torch.Tensor, xv: torch.Tensor, wr, wk, wv, N: int, bits: int,
               out_dtype=torch.float32, ys=None, stream=None):
    """R/K/V projections, each with its own input, in one launch."""
    M, K = xr.shape
    if ys is None:
        ys = tuple(torch.empty((M, N), dtype=out_dtype, device=xr.device) for _ in range(3))
    od = OUT_F16 if ys[0].dtype == torch.float16 else OUT_F32
    _check(lib().rq_rkv_fused3(_p(xr), _p(xk), _p(xv), M, K, N, bits, _p(wr[0]), _p(wr[1]),
                               _p(wk[0]), _p(wk[1]), _p(wv[0]), _p(wv[1]), _p(ys[0]), _p(ys[1]),
                               _p(ys[2]), od, _stream(stream)), "rq_rkv_fused3")
    return ys


def gemm_wq(x: torch.Tensor, codes, scales, N: int, bits: int, y=None, stream=None):
    """Prefill product y[M, N] = x[M, K] @ w_hat^T on the tcgen05 tensor cores."""
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _check(lib().rq_gemm_wq(_p(x), M, K, _p(codes), _p(scales), N, bits, _p(y), _stream(stream)),
           "rq_gemm_wq")
    return y


def rkv_fused(x: torch.Tensor, wr, wk, wv, N: int, bits: int, ys=None, stream=None):
    """Three projections of one shared x in one launch; w* = (codes, scales)."""
    M, K = x.shape
    if ys is None:
        ys = tuple(torch.empty((M, N), dtype=torch.float32, device=x.device) for _ in range(3))
    _check(lib().rq_rkv_fused(_p(x), M, K, N, bits, _p(wr[0]), _p(wr[1]), _p(wk[0]), _p(wk[1]),
                              _p(wv[0]), _p(wv[1]), _p(ys[0]), _p(ys[1]), _p(ys[2]),
                              _stream(stream)), "rq_rkv_fused")
    return ys


HEAD = 64


# torch's own short forms of the public calls, where it has them (a torch without CUDA can still import this module)
_this_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", lambda at: torch.cuda.current_stream(at).cuda_stream)
_REAL = {torch.float32: OUT_F32, torch.float16: OUT_F16}


def _placed(fn):
    """The call runs, and allocates, on the device of its first parameter's
    tensor and on the given stream (default: that device's current one)."""
    name = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        first = args[0] if args else kw.get(name)
        at = first.get_device() if isinstance(first, torch.Tensor) else -1
        if at < 0 or (stream is None and at == _this_device()):
            return fn(*args, **kw)
        _need(stream is None or stream.device_index == at, f"{fn.__name__}: the stream is not of {first.device}")
        with torch.cuda.device(at), torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _need(ok: bool, what: str, status: int = ERR_SHAPE):
    if not ok:
        raise RQError(status, what)


def _tensor(call: str, name: str, t, dtype, shape, at: int):
    """t is a contiguous tensor of this type and shape on device number `at` (-1: the host)."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise RQError(ERR_SHAPE, f"{call}: {name} must be a contiguous {dtype} {tuple(shape)}, "
                                 f"not {t.dtype} {tuple(t.shape)} with strides {t.stride()}")
    if t.get_device() != at:
        raise RQError(ERR_SHAPE, f"{call}: {name} is on {t.device}, not with the first tensor")


def _like(t, dtype=None):
    """An empty contiguous tensor of t's shape and device (of t's type if none is given)."""
    if t.is_contiguous():
        return torch.empty_like(t) if dtype is None or t.dtype is dtype else torch.empty_like(t, dtype=dtype)
    return torch.empty(t.shape, dtype=dtype or t.dtype, device=t.device)


def _on_gpu(call: str, at: int):
    if at < 0:
        raise RQError(ERR_SHAPE, f"{call}: the tensors must be on a CUDA device, not on the host")


@_placed
def lora_add(x, A, B, ids, y, out=None, ranks=None, scale=None, epilogue: int = EPI_NONE, dev_status=None):
    """y [M, N] (fp32 or fp16) plus the low-rank adapters of its tokens: x fp16
    [M, K], A fp16 [L, R, K], B fp16 [L, N, R], ids int32 [M] (negative: none),
    ranks int32 [L], scale fp32 [L].  out may be y."""
    c = "rq_lora_add"
    if x.dim() != 2 or A.dim() != 3 or B.dim() != 3:
        raise RQError(ERR_SHAPE, f"{c}: x [M, K], A [L, R, K] and B [L, N, R] are needed")
    (M, K), (L, R), N = x.shape, A.shape[:2], B.shape[1]
    at, dtype = x.get_device(), y.dtype
    if dtype not in _REAL:
        raise RQError(ERR_RANGE, f"{c}: y must be float32 or float16, not {dtype}")
    _tensor(c, "x", x, torch.float16, (M, K), at)
    _tensor(c, "A", A, torch.float16, (L, R, K), at)
    _tensor(c, "B", B, torch.float16, (L, N, R), at)
    _tensor(c, "ids", ids, torch.int32, (M,), at)
    _tensor(c, "y", y, dtype, (M, N), at)
    if ranks is not None:
        _tensor(c, "ranks", ranks, torch.int32, (L,), at)
    if scale is not None:
        _tensor(c, "scale", scale, torch.float32, (L,), at)
    if dev_status is not None:
        _tensor(c, "dev_status", dev_status, torch.int32, (1,), at)
    if out is not None:
        _tensor(c, "out", out, dtype, (M, N), at)
    if at < 0:
        _on_gpu(c, at)
    if out is None:
        out = torch.empty_like(y)
    work = None if M <= MAX_DECODE_M else torch.empty(lib().rq_lora_work_bytes(M, R), dtype=torch.uint8, device=x.device)
    st = lib().rq_lora_add(x.data_ptr(), M, K, A.data_ptr(), B.data_ptr(), L, R, ids.data_ptr(), _p(ranks), _p(scale),
                           y.data_ptr(), out.data_ptr(), N, _REAL[dtype], epilogue, _p(work), _p(dev_status),
                           _stream_of(at))
    if st != OK:
        raise RQError(st, c)
    return out


NORMS = {"none": 0, "layer": 1, "rms": 2}
GATES = {"identity": 0, "sigmoid": 1, "silu": 2}


@_placed
def norm_residual(y, post: str = "none", post_group: int = 0, post_weight=None, post_bias=None, eps_post: float = 1e-5,
                  add=None, gate=None, gate_act: str = "identity", h=None, alpha=None, pre: str = "none",
                  pre_weight=None, pre_bias=None, eps_pre: float = 1e-5, h_out=None, x=None):
    """One pass between two projections: u = (Norm_post(y) + add) * act(gate),
    h' = h + alpha u, x = Norm_pre(h') in fp16.  y, add, gate [M, D] fp32 or fp16
    (rows may be columns of a wider matrix), h [M, D]; weights, biases and alpha
    fp32 [D].  Returns (h', x); h' is None without h and h_out.  h_out may be h."""
    c = "rq_norm_residual"
    at, dtype, shape = y.get_device(), y.dtype, y.shape
    if len(shape) != 2:
        raise RQError(ERR_SHAPE, f"{c}: y must be [M, D], not {tuple(shape)}")
    if dtype not in _REAL:
        raise RQError(ERR_RANGE, f"{c}: y must be float32 or float16, not {dtype}")
    if post not in NORMS or pre not in NORMS or gate_act not in GATES:
        raise RQError(ERR_RANGE, f"{c}: {post}, {pre} or {gate_act} is not known")
    M, D = shape

    def rows(name, t):
        st = t.stride()
        if t.dtype is not dtype or t.shape != shape or st[1] != 1 or t.get_device() != at:
            raise RQError(ERR_SHAPE, f"{c}: {name} must be {dtype} {(M, D)} on {y.device} with rows of stride 1, "
                                     f"not {t.dtype} {tuple(t.shape)} {st} on {t.device}")
        return st[0] if M > 1 else D

    ld_y = rows("y", y)
    ld_add = rows("add", add) if add is not None else D
    ld_gate = rows("gate", gate) if gate is not None else D
    if h is not None:
        _tensor(c, "h", h, dtype, shape, at)
    if h_out is not None:
        _tensor(c, "h_out", h_out, dtype, shape, at)
    if x is not None:
        _tensor(c, "x", x, torch.float16, shape, at)
    for name, t in (("post_weight", post_weight), ("post_bias", post_bias), ("alpha", alpha),
                    ("pre_weight", pre_weight), ("pre_bias", pre_bias)):
        if t is not None:
            _tensor(c, name, t, torch.float32, (D,), at)
    if at < 0:
        _on_gpu(c, at)
    if h_out is None and h is not None:
        h_out = torch.empty_like(h)
    if x is None:
        x = _like(y, torch.float16)
    st = lib().rq_norm_residual(y.data_ptr(), ld_y, M, D, _REAL[dtype], NORMS[post], post_group, _p(post_weight),
                                _p(post_bias), eps_post, _p(add), ld_add, _p(gate), ld_gate, GATES[gate_act], _p(h),
                                _p(alpha), NORMS[pre], _p(pre_weight), _p(pre_bias), eps_pre, _p(h_out), x.data_ptr(),
                                _stream_of(at))
    if st != OK:
        raise RQError(st, c)
    return h_out, x


def _heads(call: str, names: str, tensors):
    """Checks the [T, H, 64] inputs of one call -> (T, H, row stride, device number)."""
    x = tensors[0]
    shape, stride, at, dtype = x.shape, x.stride(), x.get_device(), x.dtype
    if len(shape) != 3 or shape[2] != HEAD:
        raise RQError(ERR_SHAPE, f"{call}: {names[0]} must be [T, H, {HEAD}], not {tuple(shape)}")
    if dtype not in _REAL:
        raise RQError(ERR_RANGE, f"{call}: {names[0]} must be float32 or float16, not {dtype}")
    T, H = shape[0], shape[1]
    ld = stride[0] if T > 1 else H * HEAD
    rows = (ld, HEAD, 1)
    for n, t in zip(names, tensors):
        if t is not x and (t.shape != shape or t.dtype is not dtype or t.get_device() != at):
            raise RQError(ERR_SHAPE, f"{call}: {n} must be {dtype} {tuple(shape)} on {x.device} like {names[0]}, "
                                     f"not {t.dtype} {tuple(t.shape)} on {t.device}")
        st = t.stride()
        if st != rows and t.numel() and (
                st[2] != 1 or (H > 1 and st[1] != HEAD) or (T > 1 and st[0] != ld)):
            raise RQError(ERR_SHAPE, f"{call}: {n} must have strides ({ld}, {HEAD}, 1), not {st}")
    return T, H, ld, at


def _states(call: str, at: int, S: int, H: int, state, state_out, slots, dev_status):
    """Checks states and slots -> the number of states."""
    n = S
    if slots is not None:
        _tensor(call, "slots", slots, torch.int32, (S,), at)
        _need(state is not None or state_out is not None, f"{call}: slots without a state")
        n = (state if state is not None else state_out).shape[0]
    for name, t in (("state", state), ("state_out", state_out)):
        if t is not None:
            _tensor(call, name, t, torch.float32, (n, H, HEAD, HEAD), at)
    if dev_status is not None:
        _tensor(call, "dev_status", dev_status, torch.int32, (1,), at)
    return n


def tmix_ckpt(x: torch.Tensor, S: int) -> torch.Tensor:
    """Memory for the states that tmix_scan keeps for tmix_scan_bwd: x [T, H, 64]
    one of the call's inputs, S its number of sequences."""
    n = int(lib().rq_tmix_ckpt_bytes(x.shape[0], S, x.shape[1]))
    _need(n > 0, "rq_tmix_ckpt_bytes")
    return torch.empty(n // 4, dtype=torch.float32, device=x.device)


@_placed
def tmix_scan(r, d, k, v, a, b, seq_start, state=None, state_out=None, slots=None, y=None, ckpt=None,
              dev_status=None):
    """The time-mix recurrence over sequences: r, d, k, v, a, b fp32 or fp16
    [T, H, 64] (rows may be columns of a wider matrix); seq_start int32 [S + 1]
    device.  state fp32 [S, H, 64, 64] (None: zeros), or a pool of states with
    slots int32 [S].  Returns (y, state_out); state_out may be state itself, is
    allocated when not given, and for a pool must be given."""
    c = "rq_tmix_scan"
    T, H, ld, at = _heads(c, "rdkvab", (r, d, k, v, a, b))
    S = seq_start.numel() - 1
    _tensor(c, "seq_start", seq_start, torch.int32, (max(S, 1) + 1,), at)
    n = _states(c, at, S, H, state, state_out, slots, dev_status)
    if ckpt is not None:
        _tensor(c, "ckpt", ckpt, torch.float32, (lib().rq_tmix_ckpt_bytes(T, S, H) // 4,), at)
    if y is not None:
        _tensor(c, "y", y, r.dtype, (T, H, HEAD), at)
    _on_gpu(c, at)
    if y is None:
        y = _like(r)
    if state_out is None and slots is None:
        state_out = torch.empty_like(state) if state is not None else \
            torch.empty((S, H, HEAD, HEAD), dtype=torch.float32, device=r.device)
    st = lib().rq_tmix_scan(r.data_ptr(), d.data_ptr(), k.data_ptr(), v.data_ptr(), a.data_ptr(), b.data_ptr(), T, H, ld,
                            _REAL[r.dtype], seq_start.data_ptr(), S, _p(state), _p(state_out), _p(slots), n,
                            y.data_ptr(), _p(ckpt), _p(dev_status), _stream_of(at))
    if st != OK:
        raise RQError(st, c)
    return y, state_out


@_placed
def tmix_scan_bwd(r, d, k, v, a, b, seq_start, ckpt, dy, dstate_out=None, grads=None, dstate=None,
                  dev_status=None):
    """Gradients of tmix_scan (called with this ckpt and without slots) from dy
    [T, H, 64] and dstate_out [S, H, 64, 64] (None: zeros).  Returns ((dr, dd,
    dk, dv, da, db), dstate)."""
    c = "rq_tmix_scan_bwd"
    T, H, ld, at = _heads(c, "rdkvab", (r, d, k, v, a, b))
    S = seq_start.numel() - 1
    _tensor(c, "seq_start", seq_start, torch.int32, (max(S, 1) + 1,), at)
    _tensor(c, "ckpt", ckpt, torch.float32, (lib().rq_tmix_ckpt_bytes(T, S, H) // 4,), at)
    _tensor(c, "dy", dy, r.dtype, (T, H, HEAD), at)
    _states(c, at, S, H, dstate_out, dstate, None, dev_status)
    for i, g in enumerate(grads or ()):
        _tensor(c, f"grads[{i}]", g, r.dtype, (T, H, HEAD), at)
    _on_gpu(c, at)
    if grads is None:
        grads = tuple(torch.empty_like(dy) for _ in range(6))
    if dstate is None:
        dstate = torch.empty_like(dstate_out) if dstate_out is not None else \
            torch.empty((S, H, HEAD, HEAD), dtype=torch.float32, device=r.device)
    work = torch.empty_like(ckpt)
    _check(lib().rq_tmix_scan_bwd(_p(r), _p(d), _p(k), _p(v), _p(a), _p(b), T, H, ld, _REAL[r.dtype],
                                  _p(seq_start), S, _p(ckpt), _p(dy), _p(dstate_out), _p(dstate),
                                  *(_p(g) for g in grads), _p(work), _p(dev_status), _stream_of(at)), c)
    return tuple(grads), dstate


@_placed
def tmix_step(r, d, k, v, a, b, state=None, state_out=None, slots=None, y=None, dev_status=None):
    """One token of the time-mix recurrence for each of B sequences: r .. b fp32
    or fp16 [B, H, 64]; state as in tmix_scan.  Returns (y, state_out)."""
    c = "rq_tmix_step"
    B, H, ld, at = _heads(c, "rdkvab", (r, d, k, v, a, b))
    n = _states(c, at, B, H, state, state_out, slots, dev_status)
    if y is not None:
        _tensor(c, "y", y, r.dtype, (B, H, HEAD), at)
    _on_gpu(c, at)
    if y is None:
        y = _like(r)
    if state_out is None and slots is None:
        state_out = torch.empty_like(state) if state is not None else \
            torch.empty((B, H, HEAD, HEAD), dtype=torch.float32, device=r.device)
    st = lib().rq_tmix_step(r.data_ptr(), d.data_ptr(), k.data_ptr(), v.data_ptr(), a.data_ptr(), b.data_ptr(), B, H, ld,
                            _REAL[r.dtype], _p(state), _p(state_out), _p(slots), n, y.data_ptr(), _p(dev_status),
                            _stream_of(at))
    if st != OK:
        raise RQError(st, c)
    return y, state_out


def set_pdl(enable: bool):
    _check(lib().rq_set_pdl(1 if enable else 0), "rq_set_pdl")


def set_decode_kernel(kind: str):
    """Decode kernel for later products: "auto", "rowtile", "cluster" or "rowblock"."""
    _check(lib().rq_set_decode_kernel(DECODE_KERNELS[kind]), "rq_set_decode_kernel")


def decode_kernel_for(M: int, K: int, N: int, bits: int, nmat: int = 1) -> str:
    """The decode kernel ("rowtile", "cluster", "rowblock" or "tensor") a product of this shape runs on."""
    out = ctypes.c_int(-1)
    _check(lib().rq_decode_kernel_for(M, K, N, bits, nmat, ctypes.byref(out)), "rq_decode_kernel_for")
    return {v: k for k, v in DECODE_KERNELS.items()}[out.value]


class decode_kernel:
    """Context manager: run the enclosed decode products on one kernel."""

    def __init__(self, kind: str):
        self.kind = kind

    def __enter__(self):
        set_decode_kernel(self.kind)
        return self

    def __exit__(self, *exc):
        set_decode_kernel("auto")
        return False


def set_wait_limit_ns(ns: int):
    _check(lib().rq_set_wait_limit_ns(ns), "rq_set_wait_limit_ns")


def read_device_status(reset: bool = False) -> int:
    out = ctypes.c_int(-1)
    _check(lib().rq_read_device_status(ctypes.byref(out), 1 if reset else 0),
           "rq_read_device_status")
    return out.value


def selftest_bounded_wait(limit_ns: int, stream=None):
    _check(lib().rq_selftest_bounded_wait(limit_ns, _stream(stream)), "rq_selftest_bounded_wait")
