"""ctypes binding of librad.so (include/rad.h).

Argument marshalling only: every step of the path runs in the library's HIP
kernels.  PyTorch supplies device memory (tensors) and the stream each call is
enqueued on (the current stream of the tensors' device).  Nothing here falls
back to another implementation: if the library is not built, or a tensor is
not on a GPU, the call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librad.so")

# enum rad_status
RAD_OK = 0
RAD_E_NULL = -1
RAD_E_SHAPE = -2
RAD_E_ALIGN = -3
RAD_E_FMT = -4
RAD_E_RANGE = -5
RAD_E_ALIAS = -6
RAD_E_HIP = -7
# enum rad_format
RAD_FMT_U8G256_BF16ROW = 0
RAD_FMT_BF16G128 = 1
RAD_FMT_TBL4_BF16G128 = 2
GROUP_WIDTH = {RAD_FMT_U8G256_BF16ROW: 256, RAD_FMT_BF16G128: 128, RAD_FMT_TBL4_BF16G128: 128}
RAD_QUANT_MAX_K = 65536
RAD_GEMV_MAX_M = 128
RAD_QUANT_WEIGHT_MAX_K = 32768
RAD_LINEAR_MAX_K = 16777216
RAD_PROBE_BLOCK_BYTES = 98304
RAD_PROBE_MAX_BLOCKS = 65536
RAD_PROBE_MAX_KSTEPS = 1073741824

EXPORTS = ("rad_fwht128", "rad_quant_act_i8", "rad_w8a8_gemv", "rad_w8a8_gemm", "rad_w8a8_linear",
           "rad_quant_weight_i8", "rad_kv_quant_i8", "rad_kv_dequant_i8", "rad_w8a8_rescore",
           "rad_add_rmsnorm_quant_i8", "rad_kv4_append", "rad_kv4_read", "rad_attn_kv4_workspace",
           "rad_attn_kv4", "rad_probe_mfma_i8", "rad_strerror")
KV_HEAD_DIMS = (64, 128, 256)
KV4_PAGE_SIZES = (32, 64, 128, 256)
# enum rad_dtype
RAD_DT_F32 = 0
RAD_DT_BF16 = 1
RAD_DT_F16 = 2


class RadError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (call, strerror(status), status))


class WeightDesc(ctypes.Structure):
    """struct rad_w8a8_weight."""
    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("gscale", ctypes.c_void_p),
        ("rscale", ctypes.c_void_p),
        ("N", ctypes.c_int64),
        ("K", ctypes.c_int64),
        ("fmt", ctypes.c_int32),
    ]


class KV4CacheDesc(ctypes.Structure):
    """struct rad_kv4_cache."""
    _fields_ = [
        ("k_codes", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p),
        ("v_codes", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("pages", ctypes.c_int64),
        ("heads", ctypes.c_int64),
        ("page_size", ctypes.c_int64),
        ("D", ctypes.c_int64),
    ]


class KVBatchDesc(ctypes.Structure):
    """struct rad_kv_batch."""
    _fields_ = [
        ("block_table", ctypes.c_void_p),
        ("seq_len", ctypes.c_void_p),
        ("q_start", ctypes.c_void_p),
        ("B", ctypes.c_int64),
        ("max_pages", ctypes.c_int64),
        ("rows", ctypes.c_int64),
        ("max_q", ctypes.c_int64),
    ]


class RopeDesc(ctypes.Structure):
    """struct rad_rope."""
    _fields_ = [
        ("table", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("dim", ctypes.c_int32),
        ("style", ctypes.c_int32),
    ]


_lib = None


def lib() -> ctypes.CDLL:
    """Open librad.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("librad.so is not built; run `python -m rotated_w8a8_int8_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.rad_fwht128.argtypes = [vp, vp, i64, i64, vp]
        L.rad_quant_act_i8.argtypes = [vp, vp, vp, i64, i64, ci, vp]
        L.rad_w8a8_gemv.argtypes = [vp, vp, ctypes.POINTER(WeightDesc), vp, i64, vp, vp]
        L.rad_w8a8_gemm.argtypes = [vp, vp, ctypes.POINTER(WeightDesc), vp, i64, vp, vp]
        L.rad_w8a8_linear.argtypes = [vp, vp, vp, ctypes.POINTER(WeightDesc), vp, i64, vp]
        L.rad_quant_weight_i8.argtypes = [vp, vp, vp, vp, i64, i64, ctypes.c_int32, vp]
        L.rad_kv_quant_i8.argtypes = [vp, vp, vp, i64, i64, vp]
        L.rad_kv_dequant_i8.argtypes = [vp, vp, vp, i64, i64, vp]
        L.rad_w8a8_rescore.argtypes = [vp, vp, ctypes.POINTER(WeightDesc), vp, i64, vp, i64, vp]
        L.rad_probe_mfma_i8.argtypes = [vp, vp, i64, i64, ci, vp]
        i32, f32, cache, batch = ctypes.c_int32, ctypes.c_float, ctypes.POINTER(KV4CacheDesc), ctypes.POINTER(KVBatchDesc)
        L.rad_add_rmsnorm_quant_i8.argtypes = [vp, vp, vp, vp, f32, vp, vp, i64, i64, i32, ci, vp]
        L.rad_kv4_append.argtypes = [cache, batch, vp, i64, vp, i64, vp, i64, i64, vp, ctypes.POINTER(RopeDesc), ci,
                                     i32, vp]
        L.rad_kv4_read.argtypes = [cache, batch, vp, vp, vp]
        L.rad_attn_kv4_workspace.argtypes = [cache, batch, i64, i32, ctypes.POINTER(i64)]
        L.rad_attn_kv4.argtypes = [cache, batch, vp, i64, f32, ci, i64, vp, vp, i64, i32, vp]
        for f in (L.rad_fwht128, L.rad_quant_act_i8, L.rad_w8a8_gemv, L.rad_w8a8_gemm,
                  L.rad_w8a8_linear, L.rad_quant_weight_i8, L.rad_kv_quant_i8, L.rad_kv_dequant_i8,
                  L.rad_w8a8_rescore, L.rad_probe_mfma_i8, L.rad_add_rmsnorm_quant_i8, L.rad_kv4_append,
                  L.rad_kv4_read, L.rad_attn_kv4_workspace, L.rad_attn_kv4):
            f.restype = ci
        L.rad_strerror.argtypes = [ci]
        L.rad_strerror.restype = ctypes.c_char_p
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().rad_strerror(status).decode()


def _check(status: int, call: str) -> None:
    if status != RAD_OK:
        raise RadError(status, call)


# ---------------------------------------------------------------- tensors --

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dev(t, dtype, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a GPU tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _bits16_dev(t, name):
    """A contiguous GPU tensor of 16-bit bit patterns (bf16 or f16 values)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a GPU tensor" % name)
    if t.dtype not in (torch.int16, torch.uint16, torch.bfloat16, torch.float16):
        raise TypeError("%s must hold 16-bit values, got %s" % (name, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _shape(t, shape, name):
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))


def _same_device(ref, *named):
    for t, name in named:
        if t is not None and t.device != ref.device:
            raise ValueError("%s is on %s, expected %s" % (name, t.device, ref.device))


def _stream(t):
    return _torch()._C._cuda_getCurrentRawStream(t.get_device())


@dataclass
class W8A8Weight:
    """Device tensors of one quantised weight in the rotated domain.

    codes  int8 [N][K] (RAD_FMT_TBL4_BF16G128: packed 4-bit indices uint8 [N][K/2])
    gscale uint8 [N][K/256] (RAD_FMT_U8G256_BF16ROW) or int16/uint16 bf16 bits [N][K/128]
    rscale int16/uint16 bf16 bits [N] for RAD_FMT_U8G256_BF16ROW, else None
    """
    codes: object
    gscale: object
    rscale: object
    fmt: int

    @property
    def N(self) -> int:
        return int(self.codes.shape[0])

    @property
    def K(self) -> int:
        return int(self.codes.shape[1]) * (2 if self.fmt == RAD_FMT_TBL4_BF16G128 else 1)

    def desc(self) -> WeightDesc:
        """The C descriptor, after checking every tensor's device, dtype,
        contiguity and shape against the format (so no short or strided buffer
        reaches a kernel)."""
        torch = _torch()
        if self.fmt not in GROUP_WIDTH:
            raise ValueError("unknown weight format %r" % (self.fmt,))
        _dev(self.codes, torch.uint8 if self.fmt == RAD_FMT_TBL4_BF16G128 else torch.int8, "codes")
        if self.codes.dim() != 2:
            raise ValueError("codes must be 2-D, got shape %s" % (tuple(self.codes.shape),))
        G = self.K // GROUP_WIDTH[self.fmt]
        if self.fmt == RAD_FMT_U8G256_BF16ROW:
            _dev(self.gscale, torch.uint8, "gscale")
            if self.rscale is None:
                raise ValueError("the u8 format needs row scales (rscale)")
            _bits16_dev(self.rscale, "rscale")
            _shape(self.rscale, (self.N,), "rscale")
        else:
            _bits16_dev(self.gscale, "gscale")
            if self.rscale is not None:
                raise ValueError("this format takes no row scales (rscale must be None)")
        _shape(self.gscale, (self.N, G), "gscale")
        _same_device(self.codes, (self.gscale, "gscale"), (self.rscale, "rscale"))
        return WeightDesc(self.codes.data_ptr(), self.gscale.data_ptr(),
                          None if self.rscale is None else self.rscale.data_ptr(),
                          self.N, self.K, self.fmt)


def fwht128(x, out=None):
    """Rotate each contiguous 128-block of the last dim of f32 ``x`` (``out`` may be ``x``)."""
    torch = _torch()
    _dev(x, torch.float32, "x")
    K = x.shape[-1]
    if out is None:
        out = torch.empty_like(x)
    _dev(out, torch.float32, "out")
    _shape(out, x.shape, "out")
    _same_device(x, (out, "out"))
    rows = x.numel() // K if K else 0
    _check(lib().rad_fwht128(x.data_ptr(), out.data_ptr(), rows, K, _stream(x)), "rad_fwht128")
    return out


def quant_act_i8(x, rotate: bool = True, q=None, scale=None):
    """Per-token int8 codes and f32 scales of f32 ``x`` [M][K]."""
    torch = _torch()
    _dev(x, torch.float32, "x")
    M, K = x.shape
    if q is None:
        q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if scale is None:
        scale = torch.empty((M,), dtype=torch.float32, device=x.device)
    _dev(q, torch.int8, "q")
    _dev(scale, torch.float32, "scale")
    _shape(q, (M, K), "q")
    _shape(scale, (M,), "scale")
    _same_device(x, (q, "q"), (scale, "scale"))
    _check(lib().rad_quant_act_i8(x.data_ptr(), q.data_ptr(), scale.data_ptr(), M, K,
                                  1 if rotate else 0, _stream(x)), "rad_quant_act_i8")
    return q, scale


def _linear_call(fn, name, q, scale, w: W8A8Weight, y, partials):
    torch = _torch()
    _dev(q, torch.int8, "q")
    _dev(scale, torch.float32, "scale")
    d = w.desc()
    if q.dim() != 2 or q.shape[1] != w.K:
        raise ValueError("q has shape %s, weight has K=%d" % (tuple(q.shape), w.K))
    M = int(q.shape[0])
    _shape(scale, (M,), "scale")
    if y is None:
        y = torch.empty((M, w.N), dtype=torch.float32, device=q.device)
    _dev(y, torch.float32, "y")
    _shape(y, (M, w.N), "y")
    pp = None
    G = w.K // GROUP_WIDTH[w.fmt]
    if partials is True:
        partials = torch.empty((M, w.N, G), dtype=torch.int32, device=q.device)
    if partials is not None and partials is not False:
        _dev(partials, torch.int32, "partials")
        _shape(partials, (M, w.N, G), "partials")
        pp = partials.data_ptr()
    else:
        partials = None
    _same_device(q, (scale, "scale"), (w.codes, "codes"), (y, "y"), (partials, "partials"))
    _check(fn(q.data_ptr(), scale.data_ptr(), ctypes.byref(d), y.data_ptr(), M, pp, _stream(q)), name)
    return y, partials


def w8a8_gemv(q, scale, w: W8A8Weight, y=None, partials=None):
    """y [M][N] (and optionally the int32 group partials) for 1 <= M <= 128."""
    return _linear_call(lib().rad_w8a8_gemv, "rad_w8a8_gemv", q, scale, w, y, partials)


def w8a8_gemm(q, scale, w: W8A8Weight, y=None, partials=None):
    """y [M][N] (and optionally the int32 group partials) for any M."""
    return _linear_call(lib().rad_w8a8_gemm, "rad_w8a8_gemm", q, scale, w, y, partials)


def linear(x, w: W8A8Weight, q=None, scale=None, y=None):
    """The whole layer on f32 ``x`` [M][K]: returns (y, q, scale)."""
    torch = _torch()
    _dev(x, torch.float32, "x")
    M, K = x.shape
    if K != w.K:
        raise ValueError("x has K=%d, weight has K=%d" % (K, w.K))
    if q is None:
        q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if scale is None:
        scale = torch.empty((M,), dtype=torch.float32, device=x.device)
    if y is None:
        y = torch.empty((M, w.N), dtype=torch.float32, device=x.device)
    _dev(q, torch.int8, "q")
    _dev(scale, torch.float32, "scale")
    _dev(y, torch.float32, "y")
    d = w.desc()
    _shape(q, (M, K), "q")
    _shape(scale, (M,), "scale")
    _shape(y, (M, w.N), "y")
    _same_device(x, (q, "q"), (scale, "scale"), (y, "y"), (w.codes, "codes"))
    _check(lib().rad_w8a8_linear(x.data_ptr(), q.data_ptr(), scale.data_ptr(), ctypes.byref(d),
                                 y.data_ptr(), M, _stream(x)), "rad_w8a8_linear")
    return y, q, scale


def quant_weight_i8(W, fmt: int, codes=None, gscale=None, rscale=None) -> W8A8Weight:
    """Rotate and quantise f32 weights ``W`` [N][K] into format ``fmt``."""
    torch = _torch()
    _dev(W, torch.float32, "W")
    N, K = W.shape
    G = K // GROUP_WIDTH[fmt]
    tbl = fmt == RAD_FMT_TBL4_BF16G128
    if codes is None:
        codes = torch.empty((N, K // 2 if tbl else K), dtype=torch.uint8 if tbl else torch.int8,
                            device=W.device)
    if gscale is None:
        gdt = torch.uint8 if fmt == RAD_FMT_U8G256_BF16ROW else torch.int16
        gscale = torch.empty((N, G), dtype=gdt, device=W.device)
    if rscale is None and fmt == RAD_FMT_U8G256_BF16ROW:
        rscale = torch.empty((N,), dtype=torch.int16, device=W.device)
    out = W8A8Weight(codes, gscale, rscale, fmt)
    out.desc()                      # device, dtype, contiguity and shape of every output
    _shape(codes, (N, K // 2 if tbl else K), "codes")
    _same_device(W, (codes, "codes"))
    _check(lib().rad_quant_weight_i8(W.data_ptr(), codes.data_ptr(), gscale.data_ptr(),
                                     None if rscale is None else rscale.data_ptr(), N, K, fmt,
                                     _stream(W)), "rad_quant_weight_i8")
    return out


def kv_quant_i8(x, codes=None, scale=None):
    """int8 KV-cache encode of bf16 rows ``x`` [rows][D]: returns (codes, f16 scales)."""
    torch = _torch()
    _bits16_dev(x, "x")
    rows, D = x.shape
    if codes is None:
        codes = torch.empty((rows, D), dtype=torch.int8, device=x.device)
    if scale is None:
        scale = torch.empty((rows,), dtype=torch.float16, device=x.device)
    _dev(codes, torch.int8, "codes")
    _bits16_dev(scale, "scale")
    _shape(codes, (rows, D), "codes")
    _shape(scale, (rows,), "scale")
    _same_device(x, (codes, "codes"), (scale, "scale"))
    _check(lib().rad_kv_quant_i8(x.data_ptr(), codes.data_ptr(), scale.data_ptr(), rows, D, _stream(x)),
           "rad_kv_quant_i8")
    return codes, scale


def kv_dequant_i8(codes, scale, y=None):
    """Read an int8 KV cache back to bf16 [rows][D]."""
    torch = _torch()
    _dev(codes, torch.int8, "codes")
    _bits16_dev(scale, "scale")
    rows, D = codes.shape
    _shape(scale, (rows,), "scale")
    if y is None:
        y = torch.empty((rows, D), dtype=torch.bfloat16, device=codes.device)
    _bits16_dev(y, "y")
    _shape(y, (rows, D), "y")
    _same_device(codes, (scale, "scale"), (y, "y"))
    _check(lib().rad_kv_dequant_i8(codes.data_ptr(), scale.data_ptr(), y.data_ptr(), rows, D,
                                   _stream(codes)), "rad_kv_dequant_i8")
    return y


def w8a8_rescore(q, scale, w: W8A8Weight, ids, y=None):
    """The layer's outputs at candidate rows ``ids`` (int32 [M][C]) only: y [M][C]."""
    torch = _torch()
    _dev(q, torch.int8, "q")
    _dev(scale, torch.float32, "scale")
    _dev(ids, torch.int32, "ids")
    d = w.desc()
    M, C = ids.shape
    if q.shape[0] != M or q.shape[1] != w.K:
        raise ValueError("q is %s, expected [%d, %d]" % (tuple(q.shape), M, w.K))
    _shape(scale, (M,), "scale")
    if y is None:
        y = torch.empty((M, C), dtype=torch.float32, device=q.device)
    _dev(y, torch.float32, "y")
    _shape(y, (M, C), "y")
    _same_device(q, (scale, "scale"), (ids, "ids"), (y, "y"), (w.codes, "codes"))
    _check(lib().rad_w8a8_rescore(q.data_ptr(), scale.data_ptr(), ctypes.byref(d), ids.data_ptr(), C,
                                  y.data_ptr(), M, _stream(q)), "rad_w8a8_rescore")
    return y


def probe_mfma_i8(src, blocks: int, ksteps: int, lds_fed: bool, out=None):
    """Measurement aid (not a step of the layer): ``ksteps`` k-steps of four
    int8 32x32x32 matrix ops per wave, 8 waves per block, on the operand bytes
    ``src`` (int8, ``blocks * RAD_PROBE_BLOCK_BYTES``); returns the int32
    [blocks * 512] per-lane accumulator sums.  Performs
    ``blocks * 8 * ksteps * 4 * 65536`` int8 operations."""
    torch = _torch()
    _dev(src, torch.int8, "src")
    if src.numel() != blocks * RAD_PROBE_BLOCK_BYTES:
        raise ValueError("src has %d bytes, expected %d" % (src.numel(), blocks * RAD_PROBE_BLOCK_BYTES))
    if out is None:
        out = torch.empty((blocks * 512,), dtype=torch.int32, device=src.device)
    _dev(out, torch.int32, "out")
    _shape(out, (blocks * 512,), "out")
    _same_device(src, (out, "out"))
    _check(lib().rad_probe_mfma_i8(src.data_ptr(), out.data_ptr(), blocks, ksteps, 1 if lds_fed else 0,
                                   _stream(src)), "rad_probe_mfma_i8")
    return out


# ------------------------------------------------- between a layer's linears --

_dtype_codes = {}


def _dtypes():
    if not _dtype_codes:
        torch = _torch()
        _dtype_codes.update({torch.float32: RAD_DT_F32, torch.bfloat16: RAD_DT_BF16, torch.float16: RAD_DT_F16})
    return _dtype_codes


def _values(t, name):
    """A GPU tensor of f32, bf16 or f16 values: its enum rad_dtype."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a GPU tensor" % name)
    dt = _dtypes().get(t.dtype)
    if dt is None:
        raise TypeError("%s must hold f32, bf16 or f16 values, got %s" % (name, t.dtype))
    return dt


def _ptr(t, dtype, shape, ref, name):
    """The address of a contiguous tensor of this type and shape on ref's GPU; raises what is wrong with another."""
    if (isinstance(t, _torch().Tensor) and t.dtype == dtype and t.shape == shape and t.is_contiguous()
            and t.is_cuda and t.get_device() == ref.get_device()):
        return t.data_ptr()
    _dev(t, dtype, name)
    _shape(t, shape, name)
    _same_device(ref, (t, name))
    raise AssertionError(name)


def _enqueue(name, index, fn, *args):
    """Call `fn` on the current stream of GPU `index`, with that GPU current."""
    torch = _torch()
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch.cuda.current_device() == index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status != RAD_OK:
        raise RadError(status, name)


def add_rmsnorm_quant_i8(x, gamma, residual=None, eps: float = 1e-6, rotate: bool = True, q=None, scale=None,
                         residual_out=None):
    """Residual addition, RMS norm, rotation and int8 codes in one call, in front of a linear.

    ``x`` [M][K] (f32, bf16 or f16), ``gamma`` f32 [K].  With ``residual`` [M][K] of the same type the sum
    goes to ``residual_out`` (default: in place, into ``residual``).  Returns (q, scale, the sum or None)."""
    torch = _torch()
    dt, dtype = _values(x, "x"), x.dtype
    if x.dim() != 2:
        raise ValueError("x must be 2-D, got shape %s" % (tuple(x.shape),))
    M, K = x.shape
    xp = _ptr(x, dtype, (M, K), x, "x")
    gp = _ptr(gamma, torch.float32, (K,), x, "gamma")
    if q is None:
        q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if scale is None:
        scale = torch.empty((M,), dtype=torch.float32, device=x.device)
    qp = _ptr(q, torch.int8, (M, K), x, "q")
    sp = _ptr(scale, torch.float32, (M,), x, "scale")
    rp = op = None
    if residual is not None:
        rp = _ptr(residual, dtype, (M, K), x, "residual")
        if residual_out is None:
            residual_out = residual
        op = _ptr(residual_out, dtype, (M, K), x, "residual_out")
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    _enqueue("rad_add_rmsnorm_quant_i8", x.get_device(), lib().rad_add_rmsnorm_quant_i8, xp, rp, op, gp, eps, qp, sp,
             M, K, dt, 1 if rotate else 0)
    return q, scale, residual_out


class KV4Cache:
    """Device tensors of a paged attention cache in 4 bits (layouts in include/rad.h), checked once:

    k_codes uint8 [pages][heads][page_size][D/2], v_codes uint8 [pages][heads][page_size/8][D][4],
    k_scale and v_scale f16 [pages][heads][page_size].
    """

    def __init__(self, k_codes, k_scale, v_codes, v_scale):
        torch = _torch()
        _dev(k_codes, torch.uint8, "k_codes")
        _dev(v_codes, torch.uint8, "v_codes")
        _dev(k_scale, torch.float16, "k_scale")
        _dev(v_scale, torch.float16, "v_scale")
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be 4-D, got shape %s" % (tuple(k_codes.shape),))
        pages, heads, page, half = k_codes.shape
        if page not in KV4_PAGE_SIZES or 2 * half not in KV_HEAD_DIMS:
            raise ValueError("page size %d must be one of %s and head size %d one of %s"
                             % (page, KV4_PAGE_SIZES, 2 * half, KV_HEAD_DIMS))
        _shape(v_codes, (pages, heads, page // 8, 2 * half, 4), "v_codes")
        _shape(k_scale, (pages, heads, page), "k_scale")
        _shape(v_scale, (pages, heads, page), "v_scale")
        _same_device(k_codes, (k_scale, "k_scale"), (v_codes, "v_codes"), (v_scale, "v_scale"))
        self.k_codes, self.k_scale, self.v_codes, self.v_scale = k_codes, k_scale, v_codes, v_scale
        self.pages, self.heads, self.page_size, self.D = pages, heads, page, 2 * half
        self.device_index = k_codes.get_device()
        self._desc = KV4CacheDesc(k_codes.data_ptr(), k_scale.data_ptr(), v_codes.data_ptr(), v_scale.data_ptr(),
                                  pages, heads, page, 2 * half)

    @classmethod
    def empty(cls, pages: int, heads: int, page_size: int, D: int, device="cuda") -> "KV4Cache":
        """A cache over fresh memory (it needs no clearing)."""
        torch = _torch()

        def make(shape, dtype):
            return torch.empty(shape, dtype=dtype, device=device)
        return cls(make((pages, heads, page_size, D // 2), torch.uint8), make((pages, heads, page_size), torch.float16),
                   make((pages, heads, page_size // 8, D, 4), torch.uint8),
                   make((pages, heads, page_size), torch.float16))


class KVBatch:
    """Which tokens a call is about: ``block_table`` int32 [B][max_pages], ``seq_len`` int32 [B] (the call's own
    tokens counted), ``q_start`` int32 [B + 1] or None (one row per sequence), all on the GPU and read there.
    ``rows``: rows of the call's arrays, padding included (default B); ``max_q``: no sequence has more rows
    (default ``rows``)."""

    def __init__(self, block_table, seq_len, q_start=None, rows=None, max_q=None):
        torch = _torch()
        _dev(block_table, torch.int32, "block_table")
        _dev(seq_len, torch.int32, "seq_len")
        if block_table.dim() != 2:
            raise ValueError("block_table must be 2-D, got shape %s" % (tuple(block_table.shape),))
        B, max_pages = block_table.shape
        _shape(seq_len, (B,), "seq_len")
        if q_start is not None:
            _dev(q_start, torch.int32, "q_start")
            _shape(q_start, (B + 1,), "q_start")
            if rows is None:
                raise ValueError("a ragged batch (q_start) needs rows")
        rows = B if rows is None else int(rows)
        _same_device(block_table, (seq_len, "seq_len"), (q_start, "q_start"))
        self.block_table, self.seq_len, self.q_start, self.rows = block_table, seq_len, q_start, rows
        self.max_q = (rows if max_q is None else int(max_q)) if q_start is not None else 1
        self._workspace = {}                    # sizes of a call -> bytes of its workspace
        self._desc = KVBatchDesc(block_table.data_ptr(), seq_len.data_ptr(),
                                 None if q_start is None else q_start.data_ptr(), B, max_pages, rows, self.max_q)


def _head_rows(t, dtype, rows, heads, D, ref, name):
    """[rows][heads][D] values whose token rows may lie apart: address and distance in values."""
    if not isinstance(t, _torch().Tensor) or t.dtype != dtype:
        _values(t, name)
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != (rows, heads, D):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), (rows, heads, D)))
    apart, head, one = t.stride()
    if one != 1 or (head != D and heads > 1):
        raise ValueError("%s must be contiguous in its last two dims" % name)
    if not t.is_cuda or t.get_device() != ref.device_index:
        raise ValueError("%s is on %s, the cache on GPU %d" % (name, t.device, ref.device_index))
    return t.data_ptr(), apart if rows > 1 else heads * D


def _one_device(cache, batch):
    if batch.block_table.get_device() != cache.device_index:
        raise ValueError("the batch is on %s, the cache on GPU %d" % (batch.block_table.device, cache.device_index))


def kv4_append(cache: KV4Cache, batch: KVBatch, k, v, q=None, rope=None, rope_style: int = 0, rotate: bool = True,
               q_out=None):
    """Append ``k`` and ``v`` [rows][heads][D] to the cache at their positions, turned by ``rope`` (f32
    [positions][dim]: dim/2 cosines, then dim/2 sines) and rotated per 128; returns the queries ``q``
    [rows][q_heads][D] turned alike (q.k kept), or None."""
    torch = _torch()
    rows, H, D = batch.rows, cache.heads, cache.D
    _one_device(cache, batch)
    dt, dtype = _values(k, "k"), k.dtype
    kp, ldk = _head_rows(k, dtype, rows, H, D, cache, "k")
    vp, ldv = _head_rows(v, dtype, rows, H, D, cache, "v")
    q_heads, ldq, qp, op = 0, 0, None, None
    if q is not None:
        q_heads = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else -1
        qp, ldq = _head_rows(q, dtype, rows, q_heads, D, cache, "q")
        if q_out is None:
            q_out = torch.empty((rows, q_heads, D), dtype=dtype, device=q.device)
        op = _ptr(q_out, dtype, (rows, q_heads, D), cache.k_codes, "q_out")
    elif q_out is not None:
        raise ValueError("q_out needs q")
    table = None
    if rope is not None:
        if not isinstance(rope, torch.Tensor) or rope.dim() != 2:
            raise ValueError("rope must be a 2-D tensor")
        table = RopeDesc(_ptr(rope, torch.float32, rope.shape, cache.k_codes, "rope"), rope.shape[0], rope.shape[1],
                         rope_style)
    _enqueue("rad_kv4_append", cache.device_index, lib().rad_kv4_append, cache._desc, batch._desc, kp, ldk, vp, ldv,
             qp, ldq, q_heads, op, table, 1 if rotate else 0, dt)
    return q_out


def kv4_read(cache: KV4Cache, batch: KVBatch, k=None, v=None):
    """The cached keys and values of the batch's rows as bf16 [rows][heads][D]."""
    torch = _torch()
    shape = (batch.rows, cache.heads, cache.D)
    _one_device(cache, batch)
    if k is None:
        k = torch.empty(shape, dtype=torch.bfloat16, device=cache.k_codes.device)
    if v is None:
        v = torch.empty(shape, dtype=torch.bfloat16, device=cache.k_codes.device)
    kp = _ptr(k, torch.bfloat16, shape, cache.k_codes, "k")
    vp = _ptr(v, torch.bfloat16, shape, cache.k_codes, "v")
    _enqueue("rad_kv4_read", cache.device_index, lib().rad_kv4_read, cache._desc, batch._desc, kp, vp)
    return k, v


def attn_kv4_workspace(cache: KV4Cache, batch: KVBatch, q_heads: int, dtype) -> int:
    """Bytes of workspace that attn_kv4 needs for these sizes."""
    key = (cache.heads, cache.page_size, cache.D, q_heads, dtype)
    if key not in batch._workspace:
        n = ctypes.c_int64(0)
        _check(lib().rad_attn_kv4_workspace(cache._desc, batch._desc, q_heads, _dtypes()[dtype], ctypes.byref(n)),
               "rad_attn_kv4_workspace")
        batch._workspace[key] = n.value
    return batch._workspace[key]


def attn_kv4(cache: KV4Cache, batch: KVBatch, q, sm_scale: float, causal: bool = True, window: int = 0, o=None,
             workspace=None):
    """Attention of ``q`` [rows][q_heads][D] over the paged 4-bit cache; rows that see nothing give zeros."""
    torch = _torch()
    dt = _values(q, "q")
    shape, dtype = q.shape, q.dtype
    if len(shape) != 3 or shape[0] != batch.rows or shape[2] != cache.D:
        raise ValueError("q has shape %s, expected (%d, heads, %d)" % (tuple(shape), batch.rows, cache.D))
    _one_device(cache, batch)
    qp = _ptr(q, dtype, shape, cache.k_codes, "q")
    if o is None:
        o = torch.empty_like(q)
    op = _ptr(o, dtype, shape, cache.k_codes, "o")
    n = attn_kv4_workspace(cache, batch, shape[1], dtype)
    wp, size = None, 0
    if workspace is not None:
        wp, size = _ptr(workspace, torch.uint8, workspace.shape, cache.k_codes, "workspace"), workspace.numel()
    elif n:
        workspace = torch.empty((n,), dtype=torch.uint8, device=q.device)
        wp, size = workspace.data_ptr(), n
    _enqueue("rad_attn_kv4", cache.device_index, lib().rad_attn_kv4, cache._desc, batch._desc, qp, shape[1], sm_scale,
             1 if causal else 0, window, op, wp, size, dt)
    return o
