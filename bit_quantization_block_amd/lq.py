"""Thin ctypes binding of liblq (include/lq.h): argument marshalling only.

Every computation runs in the HIP library. torch is used for device memory
and streams: tensors are passed as device pointers, the current torch stream
as the hipStream_t. There is no fallback: if liblq.so is missing or fails to
load, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblq.so")

LQ_OK = 0
STATUS = {0: "LQ_OK", -1: "LQ_ERR_NULL", -2: "LQ_ERR_BAD_DESC", -3: "LQ_ERR_SHAPE", -4: "LQ_ERR_ALIGN",
          -5: "LQ_ERR_WORKSPACE", -6: "LQ_ERR_HIP", -7: "LQ_ERR_UNSUPPORTED"}
FORMAT = {"int8": 0, "int4": 1, "e4m3": 2, "e5m2": 3, "e2m1": 4, "e2m3": 5, "e3m2": 6}
GRAN = {"tensor": 0, "channel": 1, "block": 2, "tile": 3}
SCALE_FMT = {"f32": 0, "f16": 1, "ue8m0": 2, "e4m3": 3}
ROUND = {"rne": 0, "rna": 1}
DTYPE = {"f32": 0, "bf16": 1, "f16": 2}

EXPORTS = ("lq_quantize", "lq_dequantize", "lq_fake_quant_qsnr", "lq_hadamard_quant", "lq_workspace_bytes",
           "lq_codes_bytes", "lq_scales_bytes", "lq_zeros_bytes", "lq_workspace_init", "lq_sweep_tally",
           "lq_call_kernels", "lq_set_grid_limit", "lq_status_string", "lq_fake_quant_qsnr_static",
           "lq_mx4_codes_bytes", "lq_mx4_scales_bytes", "lq_ckpt8_codes_bytes", "lq_ckpt8_scales_bytes",
           "lq_linear_workspace_bytes", "lq_mx4_quantize", "lq_mx4_product", "lq_mx4_linear", "lq_mx4_dgrad",
           "lq_ckpt8_wgrad", "lq_linear_kernels", "lq_swiglu_ckpt8", "lq_swiglu_ckpt8_backward",
           "lq_rmsnorm", "lq_rmsnorm_workspace_bytes", "lq_rmsnorm_backward", "lq_int4_packed_bytes",
           "lq_int4_pack", "lq_int4_workspace_bytes", "lq_int4_linear", "lq_experts_workspace_bytes", "lq_mx4_experts",
           "lq_mx4_experts_dgrad", "lq_ckpt8_experts_wgrad")
LINEAR_CALL = {"quantize": 0, "product": 1, "linear": 2, "dgrad": 3, "wgrad": 4}
# output bits of lq_call_kernels
OUT = {"codes": 1, "scales": 2, "zeros": 4, "y": 8, "res": 16}


class LQError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} returned {status} ({STATUS.get(status, '?')}): {status_string(status)}")


class Desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("format", "gran", "block", "scale_fmt", "symmetric", "rounding",
                                               "in_dtype", "out_dtype", "hadamard", "scale_source", "two_level",
                                               "tile_rows")] + [("signs", ctypes.c_void_p)]


class Result(ctypes.Structure):
    _fields_ = [("err2", ctypes.c_double), ("sig2", ctypes.c_double), ("qsnr_db", ctypes.c_double),
                ("nonfinite", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class LinearDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("in_dtype", "out_dtype", "ckpt_format", "reserved")] + \
               [(n, ctypes.c_int64) for n in ("m", "n", "k", "ld_in", "ld_out")]


class SwigluDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("ckpt_format", ctypes.c_int32)] + \
               [(n, ctypes.c_int64) for n in ("rows", "cols", "ld", "ld_h")]


class NormDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "weight_dtype", "ckpt_format")] + [("eps", ctypes.c_float)] + \
               [(n, ctypes.c_int64) for n in ("rows", "cols", "ld_x", "ld_residual", "ld_h", "ld_y")]


class Int4Desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("in_dtype", "x_format", "out_dtype", "group", "zero_points", "reserved")] + \
               [(n, ctypes.c_int64) for n in ("m", "n", "k", "ld_in", "ld_out")]


class ExpertsDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("in_dtype", "out_dtype", "ckpt_format", "experts")] + \
               [(n, ctypes.c_int64) for n in ("m", "n", "k", "ld_in", "ld_out")]


_lib = None


def load(path: str | None = None):
    """Load liblq.so (raises if it is missing: there is no other implementation)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"liblq not built: {p} is missing (run __graft_entry__.build())")
    L = ctypes.CDLL(p)
    vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    dp = ctypes.POINTER(Desc)
    L.lq_quantize.argtypes = [dp, vp, i64, i64, vp, vp, vp, vp, sz, vp]
    L.lq_dequantize.argtypes = [dp, vp, vp, vp, i64, i64, vp, vp]
    L.lq_fake_quant_qsnr.argtypes = [dp, vp, i64, i64, vp, vp, vp, vp, vp, vp, sz, vp]
    L.lq_hadamard_quant.argtypes = [dp, vp, i64, i64, vp, vp, vp, vp, ctypes.c_int, vp, vp, sz, vp]
    L.lq_fake_quant_qsnr_static.argtypes = [dp, vp, i64, i64, vp, vp, vp, vp, vp, vp]
    L.lq_fake_quant_qsnr_static.restype = ctypes.c_int
    for f in ("lq_quantize", "lq_dequantize", "lq_fake_quant_qsnr", "lq_hadamard_quant", "lq_workspace_init",
              "lq_sweep_tally", "lq_set_grid_limit"):
        getattr(L, f).restype = ctypes.c_int
    L.lq_set_grid_limit.argtypes = [ctypes.c_int]
    for f in ("lq_workspace_bytes", "lq_codes_bytes", "lq_scales_bytes", "lq_zeros_bytes"):
        getattr(L, f).argtypes = [dp, i64, i64]
        getattr(L, f).restype = sz
    L.lq_workspace_init.argtypes = [vp, sz, vp]
    L.lq_sweep_tally.argtypes = [ctypes.POINTER(ctypes.c_double), i64, ctypes.c_double, ctypes.c_double,
                                 ctypes.POINTER(ctypes.c_int32)]
    L.lq_call_kernels.argtypes = [dp, i64, i64, ctypes.c_uint32, ctypes.c_int, ctypes.c_char_p, sz]
    L.lq_call_kernels.restype = ctypes.c_int
    for f in ("lq_mx4_codes_bytes", "lq_mx4_scales_bytes", "lq_ckpt8_codes_bytes", "lq_ckpt8_scales_bytes"):
        getattr(L, f).argtypes = [i64, i64]
        getattr(L, f).restype = sz
    lp, sp = ctypes.POINTER(LinearDesc), ctypes.POINTER(SwigluDesc)
    L.lq_linear_workspace_bytes.argtypes = [lp]
    L.lq_linear_workspace_bytes.restype = sz
    L.lq_mx4_quantize.argtypes = [lp, vp, vp, vp, vp, vp, vp]
    L.lq_mx4_product.argtypes = [lp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.lq_mx4_linear.argtypes = [lp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.lq_mx4_dgrad.argtypes = [lp, vp, vp, vp, vp, vp, sz, vp]
    L.lq_ckpt8_wgrad.argtypes = [lp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.lq_swiglu_ckpt8.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.lq_swiglu_ckpt8_backward.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp]
    np_ = ctypes.POINTER(NormDesc)
    L.lq_rmsnorm.argtypes = [np_, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.lq_rmsnorm.restype = ctypes.c_int
    L.lq_rmsnorm_workspace_bytes.argtypes = [np_]
    L.lq_rmsnorm_workspace_bytes.restype = sz
    L.lq_rmsnorm_backward.argtypes = [np_, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.lq_rmsnorm_backward.restype = ctypes.c_int
    ip = ctypes.POINTER(Int4Desc)
    for f in ("lq_int4_packed_bytes", "lq_int4_workspace_bytes"):
        getattr(L, f).argtypes = [ip]
        getattr(L, f).restype = sz
    L.lq_int4_pack.argtypes = [ip, vp, vp, vp, vp, vp]
    L.lq_int4_linear.argtypes = [ip, vp, vp, vp, vp, vp, sz, vp]
    L.lq_int4_pack.restype = L.lq_int4_linear.restype = ctypes.c_int
    ep = ctypes.POINTER(ExpertsDesc)
    L.lq_experts_workspace_bytes.argtypes = [ep]
    L.lq_experts_workspace_bytes.restype = sz
    L.lq_mx4_experts.argtypes = [ep, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.lq_mx4_experts_dgrad.argtypes = [ep, vp, vp, vp, vp, vp, vp, sz, vp]
    L.lq_ckpt8_experts_wgrad.argtypes = [ep, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    for f in ("lq_mx4_experts", "lq_mx4_experts_dgrad", "lq_ckpt8_experts_wgrad"):
        getattr(L, f).restype = ctypes.c_int
    L.lq_linear_kernels.argtypes = [lp, ctypes.c_int, ctypes.c_int, ctypes.c_char_p, sz]
    for f in ("lq_mx4_quantize", "lq_mx4_product", "lq_mx4_linear", "lq_mx4_dgrad", "lq_ckpt8_wgrad",
              "lq_linear_kernels", "lq_swiglu_ckpt8", "lq_swiglu_ckpt8_backward"):
        getattr(L, f).restype = ctypes.c_int
    L.lq_status_string.argtypes = [ctypes.c_int]
    L.lq_status_string.restype = ctypes.c_char_p
    if path is None:
        _lib = L
    return L


def status_string(status: int) -> str:
    return load().lq_status_string(status).decode()


def desc(variant: dict, in_dtype: str, given: bool = False, signs_ptr: int | None = None) -> Desc:
    """Descriptor from a variant dict (fmt, gran, block, scale, sym, round, out, hadamard, two_level,
    tile_rows); signs_ptr: device address of the rotation's sign bits, or None."""
    return Desc(FORMAT[variant["fmt"]], GRAN[variant["gran"]], int(variant.get("block", 0) or 0),
                SCALE_FMT[variant["scale"]], 1 if variant.get("sym", True) else 0,
                ROUND[variant.get("round", "rne")], DTYPE[in_dtype], DTYPE[variant.get("out", "bf16")],
                int(variant.get("hadamard", 0)), 1 if given else 0, 1 if variant.get("two_level", False) else 0,
                int(variant.get("tile_rows", 0) or 0), signs_ptr)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream
    import torch

    return torch.cuda.current_stream().cuda_stream


_raw_stream = None


def _stream_of(device: int, stream):
    """The stream given, or torch's current one on this device, without the objects around it."""
    global _raw_stream
    if stream is not None:
        return stream
    if _raw_stream is None:
        import torch

        _raw_stream = torch._C._cuda_getCurrentRawStream
    return _raw_stream(device)


class _Elsewhere:
    """The library's functions, called with a device current that may not be: a launch goes to the current device
    whatever the memory's is. (With one GPU there is no other, and calls go straight to the library.)"""

    def __init__(self, lib, device):
        self._lib, self._device = lib, device

    def __getattr__(self, name):
        import torch

        fn = getattr(self._lib, name)

        def call(*args):
            if torch.cuda.current_device() == self._device:
                return fn(*args)
            with torch.cuda.device(self._device):
                return fn(*args)

        setattr(self, name, call)
        return call


def _library(lib, device):
    """The library for memory on this device."""
    import torch

    lib = lib or load()
    return _Elsewhere(lib, device) if torch.cuda.device_count() > 1 else lib


def _check(fn, rc):
    if rc != LQ_OK:
        raise LQError(fn, rc)


# ------------------------------------------------------------------ the ABI
def lq_quantize(d: Desc, x, rows, cols, codes, scales, zeros, ws, ws_bytes, stream=None, lib=None):
    L = lib or load()
    _check("lq_quantize", L.lq_quantize(ctypes.byref(d), _ptr(x), rows, cols, _ptr(codes), _ptr(scales),
                                        _ptr(zeros), _ptr(ws), ws_bytes, _stream(stream)))


def lq_dequantize(d: Desc, codes, scales, zeros, rows, cols, y, stream=None, lib=None):
    L = lib or load()
    _check("lq_dequantize", L.lq_dequantize(ctypes.byref(d), _ptr(codes), _ptr(scales), _ptr(zeros), rows, cols,
                                            _ptr(y), _stream(stream)))


def lq_fake_quant_qsnr(d: Desc, x, rows, cols, codes, scales, zeros, y, res, ws, ws_bytes, stream=None, lib=None):
    L = lib or load()
    _check("lq_fake_quant_qsnr", L.lq_fake_quant_qsnr(ctypes.byref(d), _ptr(x), rows, cols, _ptr(codes),
                                                      _ptr(scales), _ptr(zeros), _ptr(y), _ptr(res), _ptr(ws),
                                                      ws_bytes, _stream(stream)))


def lq_fake_quant_qsnr_static(d: Desc, x, rows, cols, codes, scales, zeros, y, res, stream=None, lib=None):
    L = lib or load()
    _check("lq_fake_quant_qsnr_static", L.lq_fake_quant_qsnr_static(ctypes.byref(d), _ptr(x), rows, cols,
                                                                    _ptr(codes), _ptr(scales), _ptr(zeros),
                                                                    _ptr(y), _ptr(res), _stream(stream)))


def lq_hadamard_quant(d: Desc, x, rows, cols, codes, scales, zeros, y, unrotate_y, res, ws, ws_bytes, stream=None,
                      lib=None):
    L = lib or load()
    _check("lq_hadamard_quant", L.lq_hadamard_quant(ctypes.byref(d), _ptr(x), rows, cols, _ptr(codes),
                                                    _ptr(scales), _ptr(zeros), _ptr(y), int(unrotate_y), _ptr(res),
                                                    _ptr(ws), ws_bytes, _stream(stream)))


def lq_workspace_bytes(d: Desc, rows, cols, lib=None) -> int:
    return (lib or load()).lq_workspace_bytes(ctypes.byref(d), rows, cols)


def lq_codes_bytes(d: Desc, rows, cols, lib=None) -> int:
    return (lib or load()).lq_codes_bytes(ctypes.byref(d), rows, cols)


def lq_scales_bytes(d: Desc, rows, cols, lib=None) -> int:
    return (lib or load()).lq_scales_bytes(ctypes.byref(d), rows, cols)


def lq_zeros_bytes(d: Desc, rows, cols, lib=None) -> int:
    return (lib or load()).lq_zeros_bytes(ctypes.byref(d), rows, cols)


def lq_workspace_init(ws, ws_bytes, stream=None, lib=None):
    L = lib or load()
    _check("lq_workspace_init", L.lq_workspace_init(_ptr(ws), ws_bytes, _stream(stream)))


def lq_set_grid_limit(max_workgroups: int, lib=None):
    L = lib or load()
    _check("lq_set_grid_limit", L.lq_set_grid_limit(int(max_workgroups)))


def lq_sweep_tally(qsnr: np.ndarray, tie_db: float, margin_db: float, lib=None) -> np.ndarray:
    """qsnr: [n_tensors, 5 formats, 5 granularities] -> counts [5 granularities, 3 pairs,
    4] = (INT wins, FP wins, ties, undecided)."""
    L = lib or load()
    q = np.ascontiguousarray(qsnr, dtype=np.float64).reshape(-1, 25)
    counts = np.zeros(60, np.int32)
    _check("lq_sweep_tally", L.lq_sweep_tally(q.ctypes.data_as(ctypes.POINTER(ctypes.c_double)), q.shape[0],
                                              float(tie_db), float(margin_db),
                                              counts.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))))
    return counts.reshape(5, 3, 4)


def lq_call_kernels(d: Desc, rows, cols, outputs: int, unrotate_y: int = 0, lib=None) -> list:
    """[(kernel name, workgroups, threads per workgroup)] one call would launch, in order."""
    L = lib or load()
    n = L.lq_call_kernels(ctypes.byref(d), rows, cols, outputs, int(unrotate_y), None, 0)
    if n < 0:
        raise LQError("lq_call_kernels", n)
    buf = ctypes.create_string_buffer(512 * (n + 1))
    _check_count = L.lq_call_kernels(ctypes.byref(d), rows, cols, outputs, int(unrotate_y), buf, len(buf))
    assert _check_count == n
    out = []
    for line in buf.value.decode().splitlines():
        name, nwg, nt = line.rsplit("\t", 2)
        out.append((name, int(nwg), int(nt)))
    return out


def call_kernels(variant: dict, in_dtype: str, rows: int, cols: int,
                 want=("codes", "scales", "zeros", "y", "res"), lib=None) -> list:
    """Kernel names a fake-quant call of this variant with these outputs launches."""
    d = desc(variant, in_dtype, signs_ptr=64 if variant.get("signs") is not None else None)
    bits = sum(OUT[k] for k in want)
    un = bool(variant.get("unrotate", False)) if int(variant.get("hadamard", 0)) else 0
    return [k[0] for k in lq_call_kernels(d, rows, cols, bits, un, lib=lib)]


# ------------------------------------------------------------------ buffers
class Runner:
    """Device buffers for one (variant, shape, input dtype) and calls into the
    ABI. Buffers are torch tensors; sizes come from the library."""

    def __init__(self, variant: dict, rows: int, cols: int, in_dtype: str, device="cuda", given=False,
                 want=("codes", "scales", "zeros", "y", "res"), lib=None):
        import torch

        self.torch = torch
        self.lib = lib or load()
        self.v = variant
        self.rows, self.cols = rows, cols
        # the rotation's random signs (uint32 words, one bit per column) live on the device
        sg = variant.get("signs")
        self.signs = None if sg is None else torch.from_numpy(
            np.ascontiguousarray(sg, np.uint32).view(np.int32).copy()).to(device)
        self.d = desc(variant, in_dtype, given, None if self.signs is None else self.signs.data_ptr())
        self.given = given
        u8 = dict(dtype=torch.uint8, device=device)
        nb = lambda f: f(self.d, rows, cols, lib=self.lib)
        self.codes = torch.zeros(max(16, nb(lq_codes_bytes)), **u8) if "codes" in want else None
        self.scales = torch.zeros(max(16, nb(lq_scales_bytes)), **u8) if ("scales" in want or given) else None
        zb = nb(lq_zeros_bytes)
        self.zeros = torch.zeros(max(16, zb), **u8) if (zb and ("zeros" in want or given)) else None
        ob = {"f32": 4, "bf16": 2, "f16": 2}[variant.get("out", "bf16")]
        self.y = torch.zeros(max(16, rows * cols * ob), **u8) if "y" in want else None
        self.res = torch.zeros(64, **u8) if "res" in want else None
        self.ws_bytes = nb(lq_workspace_bytes)
        self.ws = torch.zeros(self.ws_bytes, **u8)
        lq_workspace_init(self.ws, self.ws_bytes, lib=self.lib)

    def fake_quant(self, x, unrotate=None, stream=None):
        if int(self.v.get("hadamard", 0)):
            un = self.v.get("unrotate", False) if unrotate is None else unrotate
            lq_hadamard_quant(self.d, x, self.rows, self.cols, self.codes, self.scales, self.zeros, self.y, un,
                              self.res, self.ws, self.ws_bytes, stream, lib=self.lib)
        else:
            lq_fake_quant_qsnr(self.d, x, self.rows, self.cols, self.codes, self.scales, self.zeros, self.y,
                               self.res, self.ws, self.ws_bytes, stream, lib=self.lib)

    def quantize(self, x, stream=None):
        lq_quantize(self.d, x, self.rows, self.cols, self.codes, self.scales, self.zeros, self.ws, self.ws_bytes,
                    stream, lib=self.lib)

    def dequantize(self, y=None, stream=None):
        lq_dequantize(self.d, self.codes, self.scales, self.zeros, self.rows, self.cols,
                      self.y if y is None else y, stream, lib=self.lib)

    def result(self) -> dict:
        """Read the device result struct (synchronises the current stream).
        `failed`: the library could not complete the sum (a partial record
        never arrived); the values are then NaN."""
        self.torch.cuda.current_stream().synchronize()
        raw = self.res[:ctypes.sizeof(Result)].cpu().numpy().tobytes()
        r = Result.from_buffer_copy(raw)
        return {"err2": r.err2, "sig2": r.sig2, "qsnr": r.qsnr_db, "nonfinite": r.nonfinite,
                "failed": r.reserved != 0}

    def host(self) -> dict:
        """Copy the outputs to host numpy arrays (bytes trimmed to their sizes)."""
        self.torch.cuda.current_stream().synchronize()
        n = lambda f: f(self.d, self.rows, self.cols, lib=self.lib)
        out = {}
        if self.codes is not None:
            out["codes"] = self.codes[:n(lq_codes_bytes)].cpu().numpy()
        if self.scales is not None:
            out["scales"] = self.scales[:n(lq_scales_bytes)].cpu().numpy()
        if self.zeros is not None:
            out["zeros"] = self.zeros[:n(lq_zeros_bytes)].cpu().numpy()
        if self.y is not None:
            ob = {"f32": 4, "bf16": 2, "f16": 2}[self.v.get("out", "bf16")]
            raw = self.y[:self.rows * self.cols * ob].cpu().numpy()
            out["y"] = raw.view(np.uint32 if ob == 4 else np.uint16).reshape(self.rows, self.cols)
        return out


# ------------------------------------------------------------------ the low-bit linear layer
_TORCH_DTYPE = {"f32": "float32", "bf16": "bfloat16", "f16": "float16"}


def _torch_dtype(name):
    import torch

    return getattr(torch, _TORCH_DTYPE[name])


def _dtype_name(t) -> str:
    for name, full in _TORCH_DTYPE.items():
        if str(t.dtype) == "torch." + full:
            return name
    raise TypeError(f"no lq dtype for {t.dtype}")


def _matrix(t, rows, cols, dtype, what):
    """A 2-D device tensor of this shape and dtype whose rows are contiguous; its row stride."""
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {(rows, cols)}")
    if t.dtype != dtype:
        raise TypeError(f"{what} is {t.dtype}, expected {dtype}")
    if not t.is_cuda:
        raise ValueError(f"{what} is not on the GPU")
    st = t.stride()
    if cols > 1 and st[1] != 1:
        raise ValueError(f"{what}'s rows must be contiguous (strides {st})")
    if rows > 1 and st[0] < cols:
        raise ValueError(f"{what}'s rows overlap (strides {st})")
    return st[0] if rows > 1 else max(st[0], cols)


def _share(a, b) -> bool:
    """Whether two matrices with contiguous rows have a byte in common. (Two column ranges of one matrix interleave and
    share none.)"""
    if a.numel() == 0 or b.numel() == 0:
        return False
    (pa, ma, wa, sa), (pb, mb, wb, sb) = ((t.data_ptr(), t.shape[0], t.shape[1] * t.element_size(),
                                           t.stride(0) * t.element_size()) for t in (a, b))
    if ma == 1:
        sa = sb                              # a single row has any stride
    elif mb == 1:
        sb = sa
    if sa == sb:
        # row i of a and row i + t of b meet where -wb < pb - pa + t sa < wa
        if ma == 1 and mb == 1:
            return pa < pb + wb and pb < pa + wa
        d = pb - pa
        return max(-((wb + d - 1) // sa), 1 - ma) <= min((wa - d - 1) // sa, mb - 1)
    # a row of a meets one of b that starts before the row's end and is the last such, or none
    first = pa + sa * np.arange(ma, dtype=np.int64)
    at = np.searchsorted(pb + sb * np.arange(mb, dtype=np.int64), first + wa) - 1
    return bool(((at >= 0) & (pb + sb * at + wb > first)).any())


def _reach(rows, ld, cols, size):
    """Bytes from a matrix' first element to its last's end."""
    return ((rows - 1) * ld + cols) * size if rows and cols else 0


def _refuse_grad(**tensors):
    """No result is part of autograd's graph: a tensor that waits for a gradient would never get one, without a word."""
    import torch

    if torch.is_grad_enabled():
        for what, t in tensors.items():
            if t.requires_grad:
                raise ValueError(f"{what} requires a gradient, which autograd does not get from this call: detach it "
                                 "(or call under no_grad) and use the layer's own backward calls")


def _empty_for(stream, *size, dtype, device):
    """Memory for a call on this stream (None: the current one), from the stream's own pool: what the current stream's
    pool hands out may still be in use by work that is queued there, which another stream does not wait for."""
    import torch

    if stream is None or stream == torch.cuda.current_stream(device).cuda_stream:
        return torch.empty(size, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)):
        return torch.empty(size, dtype=dtype, device=device)


def linear_kernels(call: str, m: int, n: int, k: int, in_dtype: str = "bf16", out_dtype: str = "bf16", fmt: str = "int8",
                   also: bool = False, ld_in: int | None = None, lib=None) -> list:
    """[(kernel, workgroups, threads per workgroup)] that a call of the linear layer would launch, in order. `call`: of
    LINEAR_CALL; `also`: with a checkpoint, or a dw_in; `ld_in`: its input's row stride, if rows are apart."""
    lib = lib or load()
    ins, outs = {"dgrad": (n, k), "wgrad": (n, k)}.get(call, (k, n))
    d = LinearDesc(DTYPE[in_dtype], DTYPE[out_dtype], FORMAT[fmt], 0, m, n, k, ins if ld_in is None else ld_in, outs)
    buf = ctypes.create_string_buffer(4096)
    count = lib.lq_linear_kernels(ctypes.byref(d), LINEAR_CALL[call], int(also), buf, len(buf))
    if count < 0:
        raise LQError("lq_linear_kernels", count)
    lines = [line.rsplit("\t", 2) for line in buf.value.decode().splitlines()]
    assert len(lines) == count
    return [(name, int(groups), int(threads)) for name, groups, threads in lines]


class Ckpt8:
    """An activation [rows, cols] kept in 8 bits for the backward pass: INT8
    or E4M3 codes (`fmt`), a power-of-two scale per 32 columns. A forward call
    writes it, or save()."""

    def __init__(self, rows: int, cols: int, fmt: str = "int8", device="cuda", lib=None):
        import torch

        if torch.device(device).type != "cuda":
            raise ValueError(f"a checkpoint on {device}: its kernels need it on a GPU")
        sizes = lib or load()
        self.rows, self.cols, self.fmt = rows, cols, fmt
        u8 = dict(dtype=torch.uint8, device=device)
        self.codes = torch.empty(max(16, sizes.lq_ckpt8_codes_bytes(rows, cols)), **u8)
        self.scales = torch.empty(max(16, sizes.lq_ckpt8_scales_bytes(rows, cols)), **u8)
        self._index = self.codes.device.index
        self.lib = _library(lib, self._index)
        self._d = self._values = None

    def save(self, x, stream=None):
        _refuse_grad(x=x)
        ld = _matrix(x, self.rows, self.cols, x.dtype, "x")
        if x.device != self.codes.device:
            raise ValueError(f"x is on {x.device}, the checkpoint on {self.codes.device}")
        d = LinearDesc(DTYPE[_dtype_name(x)], 0, FORMAT[self.fmt], 0, self.rows, 0, self.cols, ld, 0)
        _check("lq_mx4_quantize", self.lib.lq_mx4_quantize(ctypes.byref(d), _ptr(x), None, None, _ptr(self.codes),
                                                           _ptr(self.scales), _stream_of(self._index, stream)))

    def values(self, out=None, stream=None):
        """What the codes stand for, [rows, cols] in bfloat16 (exact but for E4M3 values of scales below 2^-124). The
        result is a view of the object's own buffer, which its next call overwrites, unless the caller passes its own."""
        import torch

        pitch = -(-self.cols // 32) * 32
        if self._d is None:
            self._d = Desc(FORMAT[self.fmt], GRAN["block"], 32, SCALE_FMT["ue8m0"], 1, 0, DTYPE["bf16"], DTYPE["bf16"])
        if out is not None:
            if _matrix(out, self.rows, self.cols, torch.bfloat16, "out") != self.cols or pitch != self.cols:
                raise ValueError("out has rows of a multiple of 32 elements, one after the other")
            if out.device != self.codes.device:
                raise ValueError(f"out is on {out.device}, the checkpoint on {self.codes.device}")
        elif self._values is None:
            self._values = _empty_for(stream, self.rows, pitch, dtype=torch.bfloat16, device=self.codes.device)
        y = self._values if out is None else out
        shown = y if pitch == self.cols else y[:, :self.cols]
        if self.rows == 0 or self.cols == 0:
            return shown
        rc = self.lib.lq_dequantize(ctypes.byref(self._d), self.codes.data_ptr(), self.scales.data_ptr(), None, self.rows,
                                    pitch, y.data_ptr(), _stream_of(self._index, stream))
        if rc != LQ_OK:
            raise LQError("lq_dequantize", rc)
        return shown


def _layout(*tensors):
    """What a call's checks depend on: shapes, strides, types and devices. (Written out where a call has no optional
    tensors: that is 0.4 us less of a small call's 5.)"""
    key = ()
    for t in tensors:
        key += (None,) if t is None else (t.shape, t.stride(), t.dtype, t.get_device())
    return key


_CALL = {"y": "lq_mx4_linear", "dx": "lq_mx4_dgrad", "dw": "lq_ckpt8_wgrad"}


class Mx4Linear:
    """A linear layer y = x W^T with W held in 4 bits (MXFP4), and its
    gradients, as calls of their own: autograd sees none of them, and inputs
    that require a gradient are refused (w may: load() reads its values).
    `w` [n, k] is quantised once; `rows` is the most rows of x or dy a call may
    have, for which the results' buffers are allocated once (a call's result is
    a view of the layer's buffer, which the layer's next call of that kind
    overwrites, unless the caller passes its own as `out`; a call on that very
    result gets a second buffer, and the two take turns).
    `dtype`: of x; `out`: of y and dx; dy is bfloat16 and dw float32. Calls of
    one layer share its buffers and workspace: on two streams at a time, use two
    layers; a stream other than the one on which the layer was made, or last
    called, waits for that one first. `stream` is a stream's handle; tensors
    given to a call on it are kept by the caller until it is done. Tensors have
    contiguous rows of any stride and start at a multiple of 16 bytes."""

    def __init__(self, w, rows: int, dtype: str = "bf16", out: str = "bf16", lib=None):
        import torch

        self.torch = torch
        self._index = w.device.index
        self.lib = _library(lib, self._index)
        self.n, self.k = w.shape
        self.rows, self.dtype, self.out = rows, dtype, out
        self.device = w.device
        u8 = dict(dtype=torch.uint8, device=w.device)
        self.codes = torch.empty(max(16, self.lib.lq_mx4_codes_bytes(self.n, self.k)), **u8)
        self.scales = torch.empty(max(16, self.lib.lq_mx4_scales_bytes(self.n, self.k)), **u8)
        self.load(w)
        self._wc, self._ws = ctypes.c_void_p(self.codes.data_ptr()), ctypes.c_void_p(self.scales.data_ptr())
        self._plans = {}
        self._buffers = {}
        self._workspaces = []

    def load(self, w, stream=None):
        """Quantises w into the layer: its weights from the next call on, as after an optimizer's step."""
        ld = _matrix(w, self.n, self.k, w.dtype, "w")
        if w.device != self.device:
            raise ValueError(f"w is on {w.device}, the layer on {self.device}")
        d = LinearDesc(DTYPE[_dtype_name(w)], 0, 0, 0, self.n, 0, self.k, ld, 0)
        _check("lq_mx4_quantize", self.lib.lq_mx4_quantize(ctypes.byref(d), _ptr(w), _ptr(self.codes),
                                                           _ptr(self.scales), None, None,
                                                           _stream_of(self._index, stream)))

    def _workspace(self, need, stream):
        """One of at least this size. Smaller ones stay alive: a captured graph may hold their addresses."""
        if not self._workspaces or self._workspaces[-1].numel() < need:
            self._workspaces.append(_empty_for(stream, need, dtype=self.torch.uint8, device=self.device))
        return self._workspaces[-1]

    def _plan(self, key, kind, a, what, cols_in, cols_out, in_dtype, out_dtype, fmt, out, stream):
        """A call's function, checked descriptor and workspace for this layout, the result's buffer and its address
        (none and 0 if it is the caller's), and between which addresses from there on an input's meets the result."""
        m = a.shape[0]
        if m > self.rows:
            raise ValueError(f"{m} rows in a layer planned for {self.rows}")
        ld_in = _matrix(a, m, cols_in, _torch_dtype(in_dtype), what)
        for t in (a, out):
            if t is not None and t.device != self.device:
                raise ValueError(f"a tensor is on {t.device}, the layer on {self.device}")
        rows_out = self.n if kind == "dw" else m
        if out is not None:
            buffer, ld_out = None, _matrix(out, rows_out, cols_out, _torch_dtype(out_dtype), "out")
        else:
            b = self._buffers.get(kind)
            if b is None:
                most = self.n if kind == "dw" else self.rows
                b = self._buffers[kind] = _empty_for(stream, most, cols_out, dtype=_torch_dtype(out_dtype),
                                                     device=self.device)
            buffer, ld_out = b[:rows_out], cols_out
        d = LinearDesc(DTYPE[in_dtype], DTYPE[out_dtype], FORMAT[fmt], 0, m, self.n, self.k, ld_in, ld_out)
        ref = ctypes.byref(d)
        need = self.lib.lq_linear_workspace_bytes(ref)
        if need == 0:   # the descriptor is refused: by this call too, with the status
            _check("lq_mx4_quantize", self.lib.lq_mx4_quantize(ref, None, None, None, None, None, None))
        ws = self._workspace(need, stream)
        if len(self._plans) >= 256:
            self._plans.clear()
        at = 0 if buffer is None else buffer.data_ptr()
        plan = self._plans[key] = (getattr(self.lib, _CALL[kind]), ref, ctypes.c_void_p(ws.data_ptr()), ws.numel(), buffer, at,
                                   at - _reach(m, ld_in, cols_in, _torch_dtype(in_dtype).itemsize),
                                   at + _reach(rows_out, ld_out, cols_out, _torch_dtype(out_dtype).itemsize))
        return plan

    def _apart(self, kind, what, a, result, out, stream):
        """Where a call on `a` may write, whose bytes meet those of `result`: nothing that the call still reads may be
        overwritten. The layer's second buffer, if the result is its own."""
        if not _share(a, result):
            return result
        if out is not None:
            raise ValueError(f"{what} and out share memory")
        b = self._buffers.get(kind + " 2")
        if b is None:
            like = self._buffers[kind]
            b = self._buffers[kind + " 2"] = _empty_for(stream, *like.shape, dtype=like.dtype, device=self.device)
        return b[:result.shape[0]]

    def forward(self, x, ckpt: Ckpt8 | None = None, out=None, stream=None):
        """y = Q4(x) W^T; `ckpt` also receives x in 8 bits."""
        if x.requires_grad:
            _refuse_grad(x=x)
        fmt = "int8" if ckpt is None else ckpt.fmt
        key = ("y", fmt, x.shape, x.stride(), x.dtype, x.get_device())
        if out is not None:
            key += _layout(out)
        plan = self._plans.get(key) or self._plan(key, "y", x, "x", self.k, self.n, self.dtype, self.out, fmt, out, stream)
        cc = cs = None
        if ckpt is not None:
            self._check_ckpt(ckpt, x.shape[0])
            cc, cs = ckpt.codes.data_ptr(), ckpt.scales.data_ptr()
        call, ref, ws, ws_bytes, y, yp, low, high = plan
        if out is not None:
            y, yp = out, out.data_ptr()
            low, high = low + yp, high + yp
        xp = x.data_ptr()
        if low < xp < high:
            y = self._apart("y", "x", x, y, out, stream)
            yp = y.data_ptr()
        rc = call(ref, xp, self._wc, self._ws, yp, cc, cs, ws, ws_bytes, _stream_of(self._index, stream))
        if rc != LQ_OK:
            raise LQError("lq_mx4_linear", rc)
        return y

    def dgrad(self, dy, out=None, stream=None):
        """dx = dy W."""
        if dy.requires_grad:
            _refuse_grad(dy=dy)
        key = ("dx", dy.shape, dy.stride(), dy.dtype, dy.get_device())
        if out is not None:
            key += _layout(out)
        plan = self._plans.get(key) or self._plan(key, "dx", dy, "dy", self.n, self.k, "bf16", self.out, "int8", out, stream)
        call, ref, ws, ws_bytes, dx, xp, low, high = plan
        if out is not None:
            dx, xp = out, out.data_ptr()
            low, high = low + xp, high + xp
        yp = dy.data_ptr()
        if low < yp < high:
            dx = self._apart("dx", "dy", dy, dx, out, stream)
            xp = dx.data_ptr()
        rc = call(ref, yp, self._wc, self._ws, xp, ws, ws_bytes, _stream_of(self._index, stream))
        if rc != LQ_OK:
            raise LQError("lq_mx4_dgrad", rc)
        return dx

    def wgrad(self, dy, ckpt: Ckpt8, dw_in=None, out=None, stream=None):
        """dw = dw_in + dy^T x8, x8 the checkpoint that forward wrote; `out` may be dw_in, but not a part of it."""
        if dy.requires_grad:
            _refuse_grad(dy=dy)
        key = ("dw", ckpt.fmt) + _layout(dy, dw_in, out)
        plan = self._plans.get(key)
        if plan is None:
            if dw_in is not None:
                ld = _matrix(dw_in, self.n, self.k, self.torch.float32, "dw_in")
                if dw_in.device != self.device:
                    raise ValueError(f"dw_in is on {dw_in.device}, the layer on {self.device}")
                if ld != (self.k if out is None else _matrix(out, self.n, self.k, self.torch.float32, "out")):
                    raise ValueError("dw_in and the result differ in their row strides")
            plan = self._plan(key, "dw", dy, "dy", self.n, self.k, "bf16", "f32", ckpt.fmt, out, stream)
        self._check_ckpt(ckpt, dy.shape[0])
        call, ref, ws, ws_bytes, dw, wp, low, high = plan
        if out is not None:
            dw, wp = out, out.data_ptr()
            low, high = low + wp, high + wp
        yp, ap = dy.data_ptr(), None
        if low < yp < high and _share(dy, dw):
            raise ValueError("dy and the result share memory")
        if dw_in is not None:
            ap = dw_in.data_ptr()
            if ap != wp and abs(ap - wp) < high - wp and _share(dw_in, dw):
                raise ValueError("dw_in and the result share memory, but are not the same")
        rc = call(ref, yp, ckpt.codes.data_ptr(), ckpt.scales.data_ptr(), ap, wp, ws, ws_bytes,
                  _stream_of(self._index, stream))
        if rc != LQ_OK:
            raise LQError("lq_ckpt8_wgrad", rc)
        return dw

    def _check_ckpt(self, ckpt, m):
        if ckpt.rows != m or ckpt.cols != self.k:
            raise ValueError(f"the checkpoint is {ckpt.rows} x {ckpt.cols}, the call's x {m} x {self.k}")
        if ckpt.codes.device != self.device:
            raise ValueError(f"the checkpoint is on {ckpt.codes.device}, the layer on {self.device}")


class SwigluCkpt8:
    """h = silu(gate) up over [rows, cols], keeping gate and up in 8 bits, and
    its backward pass from those. Results are the object's own buffers unless
    the caller passes its own, and may be a call's inputs (h one of gate and up,
    dgate or dup dh: the same rows), but no other part of them."""

    def __init__(self, rows: int, cols: int, dtype: str = "bf16", fmt: str = "int8", device="cuda", lib=None):
        import torch

        self.torch = torch
        self.rows, self.cols, self.dtype, self.fmt = rows, cols, dtype, fmt
        self._t = _torch_dtype(dtype)
        self.gate = Ckpt8(rows, cols, fmt, device, lib)
        self.up = Ckpt8(rows, cols, fmt, device, lib)
        self._kept = tuple(ctypes.c_void_p(t.data_ptr()) for c in (self.gate, self.up) for t in (c.codes, c.scales))
        self.device = self.gate.codes.device
        self._index = self.device.index
        self.lib = _library(lib, self._index)
        self._plans = {}
        self._buffers = {}

    def _at_home(self, *tensors):
        for t in tensors:
            if t.device != self.device:
                raise ValueError(f"a tensor is on {t.device}, the checkpoints on {self.device}")

    def _result(self, kind, out, stream):
        """The result's tensor if it is the object's own, and its row stride."""
        if out is not None:
            return None, _matrix(out, self.rows, self.cols, self._t, "out")
        b = self._buffers.get(kind)
        if b is None:
            b = self._buffers[kind] = _empty_for(stream, self.rows, self.cols, dtype=self._t, device=self.device)
        return b, self.cols

    def _remember(self, key, name, ld, ld_h, ld_in, ld_out, *own):
        """A call's function and descriptor for this layout, how far below and above a result's address an input's meets
        it, and the results that are the object's own, with their addresses."""
        if len(self._plans) >= 256:
            self._plans.clear()
        d = SwigluDesc(DTYPE[self.dtype], FORMAT[self.fmt], self.rows, self.cols, ld, ld_h)
        low, high = (_reach(self.rows, ld, self.cols, self._t.itemsize) for ld in (ld_in, ld_out))
        plan = self._plans[key] = (getattr(self.lib, name), ctypes.byref(d), -low, high, *own,
                                   *(0 if t is None else t.data_ptr() for t in own))
        return plan

    def _refuse(self, a, result, what):
        """An element is read and written by the same lane: in place is as good as apart, but nothing between."""
        if _share(a, result) and not (a.data_ptr() == result.data_ptr() and (self.rows == 1 or a.stride(0) == result.stride(0))):
            raise ValueError(f"{what} share memory, but are not the same")

    def forward(self, gate, up, out=None, stream=None):
        if gate.requires_grad or up.requires_grad:
            _refuse_grad(gate=gate, up=up)
        key = (gate.shape, gate.stride(), gate.dtype, gate.get_device(), up.shape, up.stride(), up.dtype, up.get_device())
        if out is not None:
            key += _layout(out)
        plan = self._plans.get(key)
        if plan is None:
            ld = _matrix(gate, self.rows, self.cols, self._t, "gate")
            if _matrix(up, self.rows, self.cols, self._t, "up") != ld:
                raise ValueError("gate and up differ in their row strides")
            self._at_home(gate, up, *(() if out is None else (out,)))
            own, ldh = self._result("h", out, stream)
            plan = self._remember(key, "lq_swiglu_ckpt8", ld, ldh, ld, ldh, own)
        call, ref, low, high, h, hp = plan
        if out is not None:
            h, hp = out, out.data_ptr()
        gp, up_ = gate.data_ptr(), up.data_ptr()
        if low < gp - hp < high:
            self._refuse(gate, h, "gate and h")
        if low < up_ - hp < high:
            self._refuse(up, h, "up and h")
        gc, gs, uc, us = self._kept
        rc = call(ref, gp, up_, hp, gc, gs, uc, us, _stream_of(self._index, stream))
        if rc != LQ_OK:
            raise LQError("lq_swiglu_ckpt8", rc)
        return h

    def backward(self, dh, out=None, stream=None):
        """(dgate, dup); `out`: a pair of tensors for them."""
        if dh.requires_grad:
            _refuse_grad(dh=dh)
        key = ("dh", dh.shape, dh.stride(), dh.dtype, dh.get_device())
        if out is not None:
            key += _layout(out[0], out[1])
        plan = self._plans.get(key)
        if plan is None:
            ldh = _matrix(dh, self.rows, self.cols, self._t, "dh")
            own0, ld = self._result("dgate", out[0] if out else None, stream)
            own1, ld1 = self._result("dup", out[1] if out else None, stream)
            if ld != ld1:
                raise ValueError("dgate and dup differ in their row strides")
            self._at_home(dh, *(out or ()))
            plan = self._remember(key, "lq_swiglu_ckpt8_backward", ld, ldh, ldh, ld, own0, own1)
        call, ref, low, high, dg, du, gp, up = plan
        if out is not None:
            dg, du = out
            gp, up = dg.data_ptr(), du.data_ptr()
            if abs(gp - up) < high and _share(dg, du):
                raise ValueError("dgate and dup share memory")
        hp = dh.data_ptr()
        if low < hp - gp < high:
            self._refuse(dh, dg, "dh and dgate")
        if low < hp - up < high:
            self._refuse(dh, du, "dh and dup")
        gc, gs, uc, us = self._kept
        rc = call(ref, hp, gc, gs, uc, us, gp, up, _stream_of(self._index, stream))
        if rc != LQ_OK:
            raise LQError("lq_swiglu_ckpt8_backward", rc)
        return dg, du


class RmsNormCkpt8:
    """y = h / sqrt(mean(h^2) + eps) * weight over the rows of [rows, cols], h = x + residual, keeping y in 8 bits
    (`kept`, a Ckpt8: for the layer behind it, whose weight gradient takes it) and each row's factor, and its backward
    pass from h. `weight` [cols] is of the matrices' dtype or float32. Results are the object's own buffers, which its
    next call of that kind overwrites, unless the caller passes its own; h and y may be x or the residual, dx may be dy,
    dh or h (the same rows), but no other part of them. Calls of one object share its buffers: on two streams at a time,
    use two objects. As the linear layer's, its calls are no part of autograd's graph."""

    _dw = None   # dw, if it is the object's own

    def __init__(self, rows: int, cols: int, dtype: str = "bf16", fmt: str = "int8", eps: float = 1e-6, device="cuda",
                 lib=None):
        import torch

        self.torch = torch
        self.rows, self.cols, self.dtype, self.fmt, self.eps = rows, cols, dtype, fmt, eps
        self._t = _torch_dtype(dtype)
        self.kept = Ckpt8(rows, cols, fmt, device, lib)
        self.device = self.kept.codes.device
        self._index = self.device.index
        self.lib = _library(lib, self._index)
        self.rs = torch.empty(max(4, rows), dtype=torch.float32, device=self.device)
        self._kept = (self.kept.codes.data_ptr(), self.kept.scales.data_ptr(), self.rs.data_ptr())
        self._plans = {}
        self._buffers = {}
        self._ws = None

    def _weight(self, w, what="weight", dtypes=None):
        if w.dim() != 1 or w.shape[0] != self.cols or (self.cols > 1 and w.stride(0) != 1):
            raise ValueError(f"{what} has shape {tuple(w.shape)} and strides {w.stride()}, expected {(self.cols,)}, contiguous")
        if w.dtype not in (dtypes or (self._t, self.torch.float32)):
            raise TypeError(f"{what} is {w.dtype}")
        if not w.is_cuda:
            raise ValueError(f"{what} is not on the GPU")

    def _at_home(self, *tensors):
        for t in tensors:
            if t is not None and t.device != self.device:
                raise ValueError(f"a tensor is on {t.device}, the norm on {self.device}")

    def _stride(self, t, what):
        return self.cols if t is None else _matrix(t, self.rows, self.cols, self._t, what)

    def _own(self, kind, stream, shape=None, dtype=None):
        b = self._buffers.get(kind)
        if b is None:
            b = self._buffers[kind] = _empty_for(stream, *(shape or (self.rows, self.cols)), dtype=dtype or self._t,
                                                 device=self.device)
        return b

    def _remember(self, key, w, *strides):
        if len(self._plans) >= 256:
            self._plans.clear()
        d = NormDesc(DTYPE[self.dtype], DTYPE[_dtype_name(w)], FORMAT[self.fmt], self.eps, self.rows, self.cols, *strides)
        size = self._t.itemsize
        plan = self._plans[key] = (ctypes.byref(d), tuple(_reach(self.rows, ld, self.cols, size) for ld in strides))
        return plan

    @staticmethod
    def _refuse(a, b, what, same=True):
        """An element is read and written by the same lane: in place is as good as apart, but nothing between. (Asked
        only where the two's bytes from the first to the last overlap.)"""
        if _share(a, b) and not (same and a.data_ptr() == b.data_ptr() and (a.shape[0] == 1 or a.stride(0) == b.stride(0))):
            raise ValueError(f"{what} share memory" + (", but are not the same" if same else ""))

    def forward(self, x, weight, residual=None, y=True, out=None, h_out=None, stream=None):
        """(y, h): h is x itself without a residual (which is gone if y takes its place, and with it the backward call's h);
        y is None if it is not asked for (`y` false), `kept` alone then holds it. `out`: a tensor for y, `h_out`: for h. A
        row whose h holds an infinity or a NaN is NaN throughout."""
        if x.requires_grad or weight.requires_grad or (residual is not None and residual.requires_grad):
            _refuse_grad(x=x, weight=weight, **({} if residual is None else {"residual": residual}))
        key = ("y", x.shape, x.stride(), x.dtype, x.get_device(), weight.shape, weight.stride(), weight.dtype,
               weight.get_device())
        if residual is not None:
            key += (residual.shape, residual.stride(), residual.dtype, residual.get_device())
        if out is not None or h_out is not None:
            key += _layout(out, h_out)
        plan = self._plans.get(key)
        if plan is None:
            if h_out is not None and residual is None:
                raise ValueError("h_out without a residual: h is x itself")
            self._weight(weight)
            self._at_home(x, weight, residual, out, h_out)
            plan = self._remember(key, weight, self._stride(x, "x"), self._stride(residual, "residual"),
                                  self._stride(h_out, "h_out"), self._stride(out, "out"))
        ref, (rx, rr, rh, ry) = plan
        h = x if residual is None else h_out if h_out is not None else self._own("h", stream)
        if not y and out is not None:
            raise ValueError("out is for y, which is not asked for")
        y = (out if out is not None else self._own("y", stream)) if y else None
        px, pr, ph, py = x.data_ptr(), None, None, None
        if y is not None:
            py = y.data_ptr()
            if px < py + ry and py < px + rx:
                self._refuse(x, y, "x and y")
        if residual is not None:
            pr, ph = residual.data_ptr(), h.data_ptr()
            if px < ph + rh and ph < px + rx:
                self._refuse(x, h, "x and h")
            if pr < ph + rh and ph < pr + rr:
                self._refuse(residual, h, "the residual and h")
            if y is not None:
                if pr < py + ry and py < pr + rr:
                    self._refuse(residual, y, "the residual and y")
                if ph < py + ry and py < ph + rh:
                    self._refuse(h, y, "h and y", same=False)
        rc = self.lib.lq_rmsnorm(ref, px, pr, weight.data_ptr(), ph, py, *self._kept,
                                 _stream_of(self._index, stream))
        if rc != LQ_OK:
            raise LQError("lq_rmsnorm", rc)
        return y, h

    def backward(self, dy, h, weight, dh=None, dw_in=None, out=None, dw_out=None, stream=None):
        """(dx, dw) of the last forward call, whose h is given back: dx = dh + dy's share, for x and the residual
        alike; dw = dw_in + the rows' sum, in float32. `out`: a tensor for dx, `dw_out`: for dw (it may be dw_in)."""
        if dy.requires_grad or h.requires_grad or weight.requires_grad or (dh is not None and dh.requires_grad):
            _refuse_grad(dy=dy, h=h, weight=weight, **({} if dh is None else {"dh": dh}))
        key = ("dx", dy.shape, dy.stride(), dy.dtype, dy.get_device(), h.shape, h.stride(), h.dtype, h.get_device(),
               weight.shape, weight.stride(), weight.dtype, weight.get_device())
        if dh is not None:
            key += (dh.shape, dh.stride(), dh.dtype, dh.get_device())
        if dw_in is not None or out is not None or dw_out is not None:
            key += _layout(dw_in, out, dw_out)
        plan = self._plans.get(key)
        if plan is None:
            self._weight(weight)
            for t, what in ((dw_in, "dw_in"), (dw_out, "dw_out")):
                if t is not None:
                    self._weight(t, what, (self.torch.float32,))
            self._at_home(dy, h, weight, dh, dw_in, out, dw_out)
            plan = self._remember(key, weight, self._stride(dy, "dy"), self._stride(dh, "dh"), self._stride(h, "h"),
                                  self._stride(out, "out"))
        ref, (ry, rd, rh, rx) = plan
        dx = out if out is not None else self._own("dx", stream)
        dw = dw_out
        if dw is None:
            dw = self._dw
            if dw is None:
                dw = self._dw = self._own("dw", stream, (max(4, self.cols),), self.torch.float32)[:self.cols]
        pdy, pd, ph, px = dy.data_ptr(), None, h.data_ptr(), dx.data_ptr()
        if pdy < px + rx and px < pdy + ry:
            self._refuse(dy, dx, "dy and dx")
        if ph < px + rx and px < ph + rh:
            self._refuse(h, dx, "h and dx")
        if dh is not None:
            pd = dh.data_ptr()
            if pd < px + rx and px < pd + rd:
                self._refuse(dh, dx, "dh and dx")
        if dw_in is not None:
            far = abs(dw_in.data_ptr() - dw.data_ptr())
            if 0 < far < 4 * self.cols:
                raise ValueError("dw_in and dw share memory, but are not the same")
        if self._ws is None:
            self._ws = _empty_for(stream, max(16, self.lib.lq_rmsnorm_workspace_bytes(ref)), dtype=self.torch.uint8,
                                  device=self.device)
        rc = self.lib.lq_rmsnorm_backward(ref, pdy, pd, ph, weight.data_ptr(), self._kept[2], px, _ptr(dw_in),
                                          dw.data_ptr(), self._ws.data_ptr(), self._ws.numel(),
                                          _stream_of(self._index, stream))
        if rc != LQ_OK:
            raise LQError("lq_rmsnorm_backward", rc)
        return dx, dw


class Int4Linear:
    """y = x W^T with W held as 4-bit integers with an fp16 scale, and a zero point unless `symmetric`, for each `group`
    (32, 64 or 128) of columns: for serving, a few rows of x at a time. `w` [n, k] is quantised (lq_quantize's INT4 rules)
    and laid out once; from_codes() takes stored weights. x is a matrix of `dtype`, or a Ckpt8 of either format (as the
    norm's `kept`), taken at the values it holds. `rows` is the most rows a call may have, for which the result's buffer is
    allocated once (a call's result is a view of it, which the next call overwrites, unless the caller passes its own as
    `out`; a call on that very result gets a second buffer). Calls of one layer share its buffers and workspace: on two
    streams at a time, use two layers; a stream other than the one on which the layer was made, or last called, waits for
    that one first. `stream` is a stream's handle. No part of autograd's graph: inputs that require a gradient are
    refused."""

    def __init__(self, w, rows: int, group: int = 64, symmetric: bool = True, dtype: str = "bf16", out: str = "bf16",
                 lib=None):
        self._start(w.shape[0], w.shape[1], group, not symmetric, rows, dtype, out, w.device, lib)
        self.load(w)

    @classmethod
    def from_codes(cls, codes, scales, zeros=None, rows: int = 1, dtype: str = "bf16", out: str = "bf16", lib=None):
        """A layer of stored weights: codes [n, k / 2] uint8 (two's complement nibbles, the even column's low), scales and
        zeros [n, groups] float16, contiguous."""
        n, k, groups = codes.shape[0], codes.shape[1] * 2, scales.shape[1]
        if groups == 0 or k % groups:
            raise ValueError(f"{k} columns in {groups} groups")
        made = cls.__new__(cls)
        made._start(n, k, k // groups, zeros is not None, rows, dtype, out, codes.device, lib)
        made.load_codes(codes, scales, zeros)
        return made

    def _start(self, n, k, group, zero_points, rows, dtype, out, device, lib):
        import torch

        self.torch = torch
        self._index = device.index
        self.lib = _library(lib, self._index)
        self.n, self.k, self.group, self.zero_points = n, k, group, zero_points
        self.rows, self.dtype, self.out, self.device = rows, dtype, out, device
        d = Int4Desc(DTYPE[dtype], -1, DTYPE[out], group, int(zero_points), 0, 0, n, k, 0, 0)
        size = self.lib.lq_int4_packed_bytes(ctypes.byref(d))
        if size == 0 and n > 0 and k > 0:   # the descriptor is refused: by this call too, with the status
            _check("lq_int4_pack", self.lib.lq_int4_pack(ctypes.byref(d), None, None, None, None, None))
        self.packed = torch.empty(max(16, size), dtype=torch.uint8, device=device)
        self._pw = ctypes.c_void_p(self.packed.data_ptr())
        self._plans = {}
        self._buffers = {}
        self._workspaces = []

    _workspace = Mx4Linear._workspace

    def load(self, w, stream=None):
        """Quantises w into the layer: its weights from the next call on."""
        torch = self.torch
        if _matrix(w, self.n, self.k, w.dtype, "w") != self.k:
            raise ValueError("w's rows must lie one after the other")
        groups = self.k // self.group
        codes = _empty_for(stream, self.n, self.k // 2, dtype=torch.uint8, device=self.device)
        scales, zeros = (_empty_for(stream, self.n, groups, dtype=torch.float16, device=self.device) for _ in range(2))
        if w.device != self.device:
            raise ValueError(f"w is on {w.device}, the layer on {self.device}")
        d = Desc(FORMAT["int4"], GRAN["block"], self.group, SCALE_FMT["f16"], int(not self.zero_points), 0,
                 DTYPE[_dtype_name(w)], DTYPE["bf16"])
        if self.n and self.k:
            _check("lq_quantize", self.lib.lq_quantize(ctypes.byref(d), _ptr(w), self.n, self.k, _ptr(codes), _ptr(scales),
                                                       _ptr(zeros) if self.zero_points else None, None, 0,
                                                       _stream_of(self._index, stream)))
        self.load_codes(codes, scales, zeros if self.zero_points else None, stream)

    def load_codes(self, codes, scales, zeros=None, stream=None):
        """Lays stored weights out in the layer, as from_codes() does."""
        groups = self.k // self.group
        if (zeros is not None) != self.zero_points:
            raise ValueError("zero points and a layer without" if zeros is not None else "no zero points for the layer's")
        for t, shape, dtype, what in ((codes, (self.n, self.k // 2), self.torch.uint8, "codes"),
                                      (scales, (self.n, groups), self.torch.float16, "scales"),
                                      (zeros, (self.n, groups), self.torch.float16, "zeros")):
            if t is None:
                continue
            if _matrix(t, *shape, dtype, what) != shape[1]:
                raise ValueError(f"{what} must be contiguous")
            if t.device != self.device:
                raise ValueError(f"{what} are on {t.device}, the layer on {self.device}")
        d = Int4Desc(0, -1, 0, self.group, int(self.zero_points), 0, 0, self.n, self.k, 0, 0)
        _check("lq_int4_pack", self.lib.lq_int4_pack(ctypes.byref(d), _ptr(codes), _ptr(scales), _ptr(zeros),
                                                     _ptr(self.packed), _stream_of(self._index, stream)))

    def _plan(self, key, x, kept, out, stream):
        m = x.rows if kept else x.shape[0]
        if m > self.rows:
            raise ValueError(f"{m} rows in a layer planned for {self.rows}")
        if kept:
            if x.cols != self.k:
                raise ValueError(f"the checkpoint has {x.cols} columns, the layer {self.k}")
            where, ld_in, reach = x.codes.device, self.k, 0
        else:
            where, ld_in = x.device, _matrix(x, m, self.k, _torch_dtype(self.dtype), "x")
            reach = _reach(m, ld_in, self.k, x.element_size())
        for device in (where, self.device if out is None else out.device):
            if device != self.device:
                raise ValueError(f"a tensor is on {device}, the layer on {self.device}")
        if out is None:
            b = self._buffers.get("y")
            if b is None:
                b = self._buffers["y"] = _empty_for(stream, self.rows, self.n, dtype=_torch_dtype(self.out),
                                                    device=self.device)
            buffer, ld_out = b[:m], self.n
        else:
            buffer, ld_out = None, _matrix(out, m, self.n, _torch_dtype(self.out), "out")
        d = Int4Desc(DTYPE[self.dtype], FORMAT[x.fmt] if kept else -1, DTYPE[self.out], self.group, int(self.zero_points), 0,
                     m, self.n, self.k, ld_in, ld_out)
        ref = ctypes.byref(d)
        ws = self._workspace(max(16, self.lib.lq_int4_workspace_bytes(ref)), stream)
        if len(self._plans) >= 256:
            self._plans.clear()
        at = 0 if buffer is None else buffer.data_ptr()
        plan = self._plans[key] = (ref, ctypes.c_void_p(ws.data_ptr()), ws.numel(), buffer, at, at - reach,
                                   at + _reach(m, ld_out, self.n, _torch_dtype(self.out).itemsize))
        return plan

    _apart = Mx4Linear._apart

    def forward(self, x, out=None, stream=None):
        """y = x W^T; x a matrix [m, k], or a Ckpt8 of it."""
        kept = isinstance(x, Ckpt8)
        if kept:
            key = (x.rows, x.cols, x.fmt, x._index)
        else:
            if x.requires_grad:
                _refuse_grad(x=x)
            key = (x.shape, x.stride(), x.dtype, x.get_device())
        if out is not None:
            key += _layout(out)
        plan = self._plans.get(key) or self._plan(key, x, kept, out, stream)
        ref, ws, ws_bytes, y, yp, low, high = plan
        if out is not None:
            y, yp = out, out.data_ptr()
            low, high = low + yp, high + yp
        if kept:
            xp, sp = x.codes.data_ptr(), x.scales.data_ptr()
        else:
            xp, sp = x.data_ptr(), None
            if low < xp < high:
                y = self._apart("y", "x", x, y, out, stream)
                yp = y.data_ptr()
        rc = self.lib.lq_int4_linear(ref, xp, sp, self._pw, yp, ws, ws_bytes, _stream_of(self._index, stream))
        if rc != LQ_OK:
            raise LQError("lq_int4_linear", rc)
        return y


class Mx4Experts:
    """A low-bit linear layer of many experts, and its gradients, as Mx4Linear's calls of their own: each row of x goes
    through the weights of one expert. `w` [experts, n, k] is quantised once. Rows lie expert by expert: `offsets`
    [experts + 1], int32 on the GPU, is where each one's rows begin and, at its end, where the last one's end (as a
    router's counts add up to; nothing waits for their values). Rows behind the last expert's are not written. `rows` is
    the most rows a call may have. Buffers, dtypes, streams, alignment and autograd: as Mx4Linear's."""

    def __init__(self, w, rows: int, dtype: str = "bf16", out: str = "bf16", lib=None):
        import torch

        if w.dim() != 3:
            raise ValueError(f"w has shape {tuple(w.shape)}, expected [experts, n, k]")
        self.torch = torch
        self._index = w.device.index
        self.lib = _library(lib, self._index)
        self.experts, self.n, self.k = w.shape
        self.rows, self.dtype, self.out = rows, dtype, out
        self.device = w.device
        u8 = dict(dtype=torch.uint8, device=w.device)
        self.codes = torch.empty(max(16, self.lib.lq_mx4_codes_bytes(self.experts * self.n, self.k)), **u8)
        self.scales = torch.empty(max(16, self.lib.lq_mx4_scales_bytes(self.experts * self.n, self.k)), **u8)
        self.load(w)
        self._wc, self._ws = ctypes.c_void_p(self.codes.data_ptr()), ctypes.c_void_p(self.scales.data_ptr())
        self._plans = {}
        self._buffers = {}
        self._workspaces = []

    _workspace = Mx4Linear._workspace
    _apart = Mx4Linear._apart
    _check_ckpt = Mx4Linear._check_ckpt

    def load(self, w, stream=None):
        """Quantises w into the layer: its weights from the next call on, as after an optimizer's step."""
        if w.dim() != 3 or tuple(w.shape) != (self.experts, self.n, self.k):
            raise ValueError(f"w has shape {tuple(w.shape)}, expected {(self.experts, self.n, self.k)}")
        if self.experts > 1 and self.n > 1 and w.stride(0) != self.n * w.stride(1):
            raise ValueError(f"w's experts must lie one after the other (strides {w.stride()})")
        flat = w.flatten(0, 1) if self.n > 1 or w.stride(0) == w.stride(1) else w[:, 0]
        ld = _matrix(flat, self.experts * self.n, self.k, w.dtype, "w")
        if w.device != self.device:
            raise ValueError(f"w is on {w.device}, the layer on {self.device}")
        d = LinearDesc(DTYPE[_dtype_name(w)], 0, 0, 0, self.experts * self.n, 0, self.k, ld, 0)
        _check("lq_mx4_quantize", self.lib.lq_mx4_quantize(ctypes.byref(d), _ptr(flat), _ptr(self.codes),
                                                           _ptr(self.scales), None, None,
                                                           _stream_of(self._index, stream)))

    def _cube(self, t, what):
        """A float32 device tensor [experts, n, k], its experts one after the other; the stride of its rows."""
        if tuple(t.shape) != (self.experts, self.n, self.k):
            raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {(self.experts, self.n, self.k)}")
        if not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous")
        if t.dtype != self.torch.float32:
            raise TypeError(f"{what} is {t.dtype}, expected torch.float32")
        if not t.is_cuda or t.device != self.device:
            raise ValueError(f"{what} is on {t.device}, the layer on {self.device}")

    def _plan(self, key, kind, a, what, offsets, cols_in, cols_out, in_dtype, out_dtype, fmt, out, stream):
        m = a.shape[0]
        if m > self.rows:
            raise ValueError(f"{m} rows in a layer planned for {self.rows}")
        if offsets.dtype != self.torch.int32 or tuple(offsets.shape) != (self.experts + 1,) or not offsets.is_contiguous():
            raise ValueError(f"offsets are {offsets.dtype} {tuple(offsets.shape)}, expected int32 {(self.experts + 1,)}, contiguous")
        ld_in = _matrix(a, m, cols_in, _torch_dtype(in_dtype), what)
        for t in (a, offsets, out):
            if t is not None and t.device != self.device:
                raise ValueError(f"a tensor is on {t.device}, the layer on {self.device}")
        if kind == "dw":
            shape, buffer, ld_out = (self.experts, self.n, self.k), None, self.k
            if out is not None:
                self._cube(out, "out")
        else:
            shape, buffer, ld_out = (self.rows, cols_out), None, cols_out
            if out is not None:
                ld_out = _matrix(out, m, cols_out, _torch_dtype(out_dtype), "out")
        if out is None:
            buffer = self._buffers.get(kind)
            if buffer is None:
                buffer = self._buffers[kind] = _empty_for(stream, *shape, dtype=_torch_dtype(out_dtype), device=self.device)
            if kind != "dw":
                buffer = buffer[:m]
        d = ExpertsDesc(DTYPE[in_dtype], DTYPE[out_dtype], FORMAT[fmt], self.experts, m, self.n, self.k, ld_in, ld_out)
        ref = ctypes.byref(d)
        need = self.lib.lq_experts_workspace_bytes(ref)
        if need == 0:   # the descriptor is refused: by this call too, with the status
            _check("lq_mx4_experts", self.lib.lq_mx4_experts(ref, None, None, None, None, None, None, None, None, 0, None))
        ws = self._workspace(need, stream)
        if len(self._plans) >= 256:
            self._plans.clear()
        at = 0 if buffer is None else buffer.data_ptr()
        rows_out = self.experts * self.n if kind == "dw" else m
        plan = self._plans[key] = (ref, ctypes.c_void_p(ws.data_ptr()), ws.numel(), buffer, at,
                                   at - _reach(m, ld_in, cols_in, _torch_dtype(in_dtype).itemsize),
                                   at + _reach(rows_out, ld_out, cols_out, _torch_dtype(out_dtype).itemsize))
        return plan

    def forward(self, x, offsets, ckpt: Ckpt8 | None = None, out=None, stream=None):
        """y_i = Q4(x_i) W_e^T for expert e's rows i; `ckpt` also receives x in 8 bits."""
        if x.requires_grad:
            _refuse_grad(x=x)
        fmt = "int8" if ckpt is None else ckpt.fmt
        key = ("y", fmt) + _layout(x, offsets, out)
        plan = self._plans.get(key) or self._plan(key, "y", x, "x", offsets, self.k, self.n, self.dtype, self.out, fmt, out,
                                                  stream)
        cc = cs = None
        if ckpt is not None:
            self._check_ckpt(ckpt, x.shape[0])
            cc, cs = ckpt.codes.data_ptr(), ckpt.scales.data_ptr()
        ref, ws, ws_bytes, y, yp, low, high = plan
        if out is not None:
            y, yp = out, out.data_ptr()
            low, high = low + yp, high + yp
        xp = x.data_ptr()
        if low < xp < high:
            y = self._apart("y", "x", x, y, out, stream)
            yp = y.data_ptr()
        rc = self.lib.lq_mx4_experts(ref, xp, offsets.data_ptr(), self._wc, self._ws, yp, cc, cs, ws, ws_bytes,
                                     _stream_of(self._index, stream))
        if rc != LQ_OK:
            raise LQError("lq_mx4_experts", rc)
        return y

    def dgrad(self, dy, offsets, out=None, stream=None):
        """dx_i = dy_i W_e."""
        if dy.requires_grad:
            _refuse_grad(dy=dy)
        key = ("dx",) + _layout(dy, offsets, out)
        plan = self._plans.get(key) or self._plan(key, "dx", dy, "dy", offsets, self.n, self.k, "bf16", self.out, "int8", out,
                                                  stream)
        ref, ws, ws_bytes, dx, xp, low, high = plan
        if out is not None:
            dx, xp = out, out.data_ptr()
            low, high = low + xp, high + xp
        yp = dy.data_ptr()
        if low < yp < high:
            dx = self._apart("dx", "dy", dy, dx, out, stream)
            xp = dx.data_ptr()
        rc = self.lib.lq_mx4_experts_dgrad(ref, yp, offsets.data_ptr(), self._wc, self._ws, xp, ws, ws_bytes,
                                           _stream_of(self._index, stream))
        if rc != LQ_OK:
            raise LQError("lq_mx4_experts_dgrad", rc)
        return dx

    def wgrad(self, dy, ckpt: Ckpt8, offsets, dw_in=None, out=None, stream=None):
        """dw_e = dw_in_e + the sum over e's rows of dy_i^T x8_i, x8 the checkpoint that forward wrote; dw_in and `out` are
        float32 [experts, n, k], contiguous, and may be the same."""
        if dy.requires_grad:
            _refuse_grad(dy=dy)
        key = ("dw", ckpt.fmt) + _layout(dy, offsets, dw_in, out)
        plan = self._plans.get(key)
        if plan is None:
            if dw_in is not None:
                self._cube(dw_in, "dw_in")
            plan = self._plan(key, "dw", dy, "dy", offsets, self.n, self.k, "bf16", "f32", ckpt.fmt, out, stream)
        self._check_ckpt(ckpt, dy.shape[0])
        ref, ws, ws_bytes, dw, wp, low, high = plan
        if out is not None:
            dw, wp = out, out.data_ptr()
            low, high = low + wp, high + wp
        yp, ap = dy.data_ptr(), None
        if low < yp < high and _share(dy, dw.view(-1, self.k)):
            raise ValueError("dy and the result share memory")
        if dw_in is not None:
            ap = dw_in.data_ptr()
            if ap != wp and abs(ap - wp) < high - wp:
                raise ValueError("dw_in and the result share memory, but are not the same")
        rc = self.lib.lq_ckpt8_experts_wgrad(ref, yp, offsets.data_ptr(), ckpt.codes.data_ptr(), ckpt.scales.data_ptr(), ap,
                                             wp, ws, ws_bytes, _stream_of(self._index, stream))
        if rc != LQ_OK:
            raise LQError("lq_ckpt8_experts_wgrad", rc)
        return dw


# ------------------------------------------------------------------ ceilings
CEILING_PATH = os.path.join(_HERE, "liblq_ceiling.so")
CEILING_EXPORTS = ("lqc_copy", "lqc_pattern", "lqc_read", "lqc_write")
_ceiling = None


def load_ceiling(path: str | None = None):
    """Load liblq_ceiling.so (include/lq_ceiling.h): the copy, pattern, read-only and write-only kernels."""
    global _ceiling
    if _ceiling is not None and path is None:
        return _ceiling
    p = path or CEILING_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"liblq_ceiling not built: {p} is missing (run __graft_entry__.build())")
    L = ctypes.CDLL(p)
    vp, i64, ci, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    L.lqc_copy.argtypes = [vp, sz, vp, sz, i64, ci, ci, vp]
    L.lqc_copy.restype = ci
    L.lqc_pattern.argtypes = [vp, sz, i64, vp, sz, ci, vp, sz, ci, vp, sz, ci, ci, vp]
    L.lqc_pattern.restype = ci
    L.lqc_read.argtypes = [vp, sz, i64, vp, sz, ci, ci, vp]
    L.lqc_read.restype = ci
    L.lqc_write.argtypes = [vp, sz, i64, ci, ci, vp]
    L.lqc_write.restype = ci
    if path is None:
        _ceiling = L
    return L


def _nbytes(t) -> int:
    """Byte size of a contiguous torch tensor from its data pointer on (the
    buffer the library may touch)."""
    if not t.is_contiguous():
        raise ValueError("the ceiling kernels take contiguous buffers")
    return t.numel() * t.element_size()


def lqc_copy(src, dst, n: int, threads: int, workgroups: int, stream=None, lib=None):
    L = lib or load_ceiling()
    rc = L.lqc_copy(_ptr(src), _nbytes(src), _ptr(dst), _nbytes(dst), n, threads, workgroups, _stream(stream))
    if rc != 0:
        raise RuntimeError(f"lqc_copy returned {rc}")


def lqc_read(src, nbytes: int, sink, threads: int, workgroups: int, stream=None, lib=None):
    L = lib or load_ceiling()
    rc = L.lqc_read(_ptr(src), _nbytes(src), nbytes, _ptr(sink), _nbytes(sink), threads, workgroups, _stream(stream))
    if rc != 0:
        raise RuntimeError(f"lqc_read returned {rc}")


def lqc_write(dst, nbytes: int, threads: int, workgroups: int, stream=None, lib=None):
    L = lib or load_ceiling()
    rc = L.lqc_write(_ptr(dst), _nbytes(dst), nbytes, threads, workgroups, _stream(stream))
    if rc != 0:
        raise RuntimeError(f"lqc_write returned {rc}")


def lqc_pattern(x, n: int, codes, code_bits: int, scales, block: int, y, threads: int, workgroups: int,
                stream=None, lib=None):
    L = lib or load_ceiling()
    rc = L.lqc_pattern(_ptr(x), _nbytes(x), n, _ptr(codes), _nbytes(codes), code_bits, _ptr(scales), _nbytes(scales),
                       block, _ptr(y), _nbytes(y), threads, workgroups, _stream(stream))
    if rc != 0:
        raise RuntimeError(f"lqc_pattern returned {rc}")
