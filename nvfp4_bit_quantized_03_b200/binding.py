"""ctypes binding of libnvfp4.so (include/nvfp4.h).

Argument marshalling only: PyTorch owns the device memory and the streams; every step of the
quantizers and GEMMs runs in the library's CUDA kernels.  There is no fallback: if the
library is missing or a call fails, an exception is raised.

Inside a ``with bounds_checked():`` block the same calls go to libnvfp4_checked.so, the debug
build whose kernels check every global access against its buffer (NVFP4_DEVSTAT_BOUNDS).
"""
import contextlib
import ctypes
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnvfp4.so")
CHECKED_LIB_PATH = os.path.join(_PKG, "libnvfp4_checked.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "nvfp4.h")

# status codes and flags (include/nvfp4.h)
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_DEVICE, ERR_CUDA, ERR_NONFINITE, ERR_TIMEOUT, ERR_ARG = range(9)
DEVSTAT_NONFINITE, DEVSTAT_TIMEOUT, DEVSTAT_BOUNDS, DEVSTAT_INDEX = 1, 2, 4, 8
ROWWISE, COLWISE, BLOCK2D, SR, AMAX_GIVEN, MX, GATHER = 1, 2, 4, 8, 16, 32, 64
OUT_F32, OUT_BF16 = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1


class NVFP4Error(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {lib().nvfp4_status_string(status).decode()} (status {status})")


class Operand(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("amax", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class PlanStruct(ctypes.Structure):
    _fields_ = [("offsets", ctypes.c_void_p), ("pair_row", ctypes.c_void_p),
                ("row_token", ctypes.c_void_p), ("tokens", ctypes.c_int64), ("k", ctypes.c_int64),
                ("experts", ctypes.c_int64), ("rows", ctypes.c_int64)]


_libs = {}               # path -> configured CDLL
_active = LIB_PATH       # the library calls go to
_poison = False


def set_output_poisoning(enabled: bool):
    """Debug aid for tests: when enabled, every output buffer this module allocates is first
    filled with a pattern no kernel writes (codes and scales 0xFF bytes, FP32 / bf16 results and
    amax NaN, indices -2^31; workspaces 0xFF bytes), so that a kernel that leaves part of its output unwritten,
    or reads scratch it did not write, cannot pass a check by finding an earlier, identical
    result in recycled memory."""
    global _poison
    _poison = bool(enabled)


def _poisoned(t):
    if _poison:
        if t.dtype == torch.uint8:
            t.fill_(0xFF)
        elif t.dtype == torch.int32:
            t.fill_(-2 ** 31)
        else:
            t.fill_(float("nan"))
    return t


def lib():
    """The library calls go to: libnvfp4.so, or libnvfp4_checked.so inside bounds_checked()
    (raises if it has not been built)."""
    L = _libs.get(_active)
    if L is None:
        L = _libs[_active] = _open(_active)
    return L


@contextlib.contextmanager
def bounds_checked():
    """Route every call of this module made inside the block to libnvfp4_checked.so (the
    -DNVFP4_BOUNDS_CHECK build: an out-of-extent global access is skipped and sets
    NVFP4_DEVSTAT_BOUNDS in the call's status word).  Calls made without a status word report to
    one of this module, and the block ends with an NVFP4Error if they refused an access.  Yields
    that library.  The switch is process-wide, not per thread: other threads' calls inside the
    block go there too."""
    global _active
    prev = _active
    _active = CHECKED_LIB_PATH
    try:
        L = lib()
        _report_word()
        if prev != CHECKED_LIB_PATH:
            _take_reports()  # of a block that another error ended
        yield L
        if _take_reports() & DEVSTAT_BOUNDS:
            raise NVFP4Error(ERR_ARG, "bounds_checked: a call without a status word refused an "
                                      "access outside its buffer")
    finally:
        _active = prev


_reports = {}  # device -> the status word of checked calls without one, kept for captured graphs


def _report_word():
    """Address of this device's word (None where it cannot be made: no GPU, or while capturing)."""
    if not torch.cuda.is_available():
        return None
    device = torch.cuda.current_device()
    if device not in _reports:
        if torch.cuda.is_current_stream_capturing():
            return None
        _reports[device] = torch.zeros(1, dtype=torch.int32, device=device)
        torch.cuda.synchronize(device)
    return _reports[device].data_ptr()


def _take_reports():
    """The bits of all words, which are cleared.  (None while capturing: nothing runs then, and the
    device cannot be waited for.)"""
    if _reports and torch.cuda.is_current_stream_capturing():
        return 0
    bits = 0
    for device, word in _reports.items():
        torch.cuda.synchronize(device)
        bits |= int(word)
        word.zero_()
        torch.cuda.synchronize(device)
    return bits


def _status(dev_status):
    """Address of a call's status word."""
    if dev_status is None:
        return _report_word() if _active == CHECKED_LIB_PATH else None
    return dev_status.data_ptr()


def _open(path):
    if not os.path.exists(path):
        raise ImportError(f"{os.path.basename(path)} not found at {path}; build it with "
                          "`python -m nvfp4_bit_quantized_03_b200.build` (nvcc, sm_100a)")
    L = ctypes.CDLL(path)
    i64, u64, u16, vp, i32 = (ctypes.c_int64, ctypes.c_uint64, ctypes.c_uint16,
                              ctypes.c_void_p, ctypes.c_int)
    op = ctypes.POINTER(Operand)
    sz = ctypes.c_size_t
    L.nvfp4_version.argtypes, L.nvfp4_version.restype = [], i32
    L.nvfp4_status_string.argtypes, L.nvfp4_status_string.restype = [i32], ctypes.c_char_p
    L.nvfp4_codes_bytes.argtypes, L.nvfp4_codes_bytes.restype = [i64, i64], sz
    L.nvfp4_scales_bytes.argtypes, L.nvfp4_scales_bytes.restype = [i64, i64], sz
    L.nvfp4_workspace_bytes.argtypes = [i64, i64, ctypes.c_uint]
    L.nvfp4_workspace_bytes.restype = sz
    L.nvfp4_linear_workspace_bytes.argtypes = [i64, i64, i64]
    L.nvfp4_linear_workspace_bytes.restype = sz
    L.nvfp4_sign_mask_from_seed.argtypes, L.nvfp4_sign_mask_from_seed.restype = [u64], u16
    L.nvfp4_scales_unswizzle.argtypes = [vp, i64, i64, vp]
    L.nvfp4_scales_unswizzle.restype = i32
    L.nvfp4_quantize.argtypes = [vp, i64, i64, i64, ctypes.c_uint, u64, u64, op, op, vp, vp, vp]
    L.nvfp4_quantize.restype = i32
    L.nvfp4_rht_quantize.argtypes = [vp, i64, i64, i64, u16, ctypes.c_uint, u64, u64, op, vp,
                                     vp, vp]
    L.nvfp4_rht_quantize.restype = i32
    L.nvfp4_quantize_row_rht.argtypes = [vp, i64, i64, i64, u16, ctypes.c_uint, u64, u64, op,
                                         op, vp, vp, vp]
    L.nvfp4_quantize_row_rht.restype = i32
    L.nvfp4_gemm.argtypes = [op, op, vp, i32, i64, vp, vp]
    L.nvfp4_gemm.restype = i32
    L.nvfp4_gemm_mx.argtypes = [op, op, vp, i32, i64, vp, vp]
    L.nvfp4_gemm_mx.restype = i32
    L.nvfp4_gemm_amax.argtypes = [op, op, vp, i64, u16, vp, vp, vp]
    L.nvfp4_gemm_amax.restype = i32
    L.nvfp4_selftest_wait_timeout.argtypes = [vp, vp]
    L.nvfp4_selftest_wait_timeout.restype = i32
    L.nvfp4_bounds_checked.argtypes, L.nvfp4_bounds_checked.restype = [], i32
    L.nvfp4_selftest_bounds.argtypes, L.nvfp4_selftest_bounds.restype = [vp, vp], i32
    L.nvfp4_linear_fprop.argtypes = [vp, vp, i64, i64, i64, vp, i32, vp, vp, vp]
    L.nvfp4_linear_fprop.restype = i32
    L.nvfp4_linear_dgrad.argtypes = [vp, vp, i64, i64, i64, u64, u64, vp, i32, vp, vp, vp]
    L.nvfp4_linear_dgrad.restype = i32
    L.nvfp4_linear_wgrad.argtypes = [vp, vp, i64, i64, i64, u16, u64, u64, vp, i32, vp, vp, vp]
    L.nvfp4_linear_wgrad.restype = i32
    L.nvfp4_linear_dgrad_quantized.argtypes = [vp, vp, i64, i64, i64, u64, u64, vp, u16, u64,
                                               u64, op, op, vp, vp, vp]
    L.nvfp4_linear_dgrad_quantized.restype = i32
    pl, u32, f32 = ctypes.POINTER(PlanStruct), ctypes.c_uint, ctypes.c_float
    L.nvfp4_expert_rows.argtypes, L.nvfp4_expert_rows.restype = [i64, i64, i64], i64
    L.nvfp4_expert_plan_workspace_bytes.argtypes = [i64, i64, i64]
    L.nvfp4_expert_plan_workspace_bytes.restype = sz
    L.nvfp4_experts_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, i64]
    L.nvfp4_experts_workspace_bytes.restype = sz
    for name, argtypes in {
            "route": [vp, i32, i64, i64, i64, vp, i32, i32, i32, i32, i32, f32, vp, vp, vp, vp],
            "route_backward": [vp, i32, i64, i64, i64, vp, vp, i32, i32, i32, f32, vp, i64, vp, vp],
            "plan_experts": [vp, pl, vp, vp, vp],
            "quantize_grouped": [vp, i64, i64, pl, u16, u32, u64, u64, op, op, vp, vp, vp],
            "gemm_grouped": [op, op, pl, vp, i32, i64, vp, vp],
            "gemm_grouped_k": [op, op, pl, vp, i32, i64, vp, vp],
            "experts_fprop": [vp, i64, i32, op, pl, i64, i64, vp, i32, i64, vp, vp, vp],
            "experts_dgrad": [vp, i64, op, pl, i64, i64, u64, u64, vp, i32, i64, vp, vp, vp],
            "experts_wgrad": [vp, i64, vp, i64, i32, pl, i64, i64, u16, u64, u64, vp, i32, i64, vp,
                              vp, vp],
            "combine": [vp, i64, i64, pl, vp, vp, i32, i64, vp, vp],
            "combine_backward": [vp, i32, i64, vp, i64, i64, pl, vp, vp, i64, vp, vp, vp]}.items():
        f = getattr(L, "nvfp4_" + name)
        f.argtypes, f.restype = argtypes, i32
    return L


def declared_functions():
    """Names of the functions include/nvfp4.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(nvfp4_[a-z0-9_]+)\s*\(", text)))


def _check(status, what):
    if status != OK:
        raise NVFP4Error(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# ---- sizes and host helpers -------------------------------------------------------------

def codes_bytes(rows, cols):
    return lib().nvfp4_codes_bytes(rows, cols)


def scales_bytes(rows, cols):
    return lib().nvfp4_scales_bytes(rows, cols)


def workspace_bytes(rows, cols, flags=0):
    return lib().nvfp4_workspace_bytes(rows, cols, flags)


def linear_workspace_bytes(T, I, O):
    return lib().nvfp4_linear_workspace_bytes(T, I, O)


def sign_mask_from_seed(seed):
    return lib().nvfp4_sign_mask_from_seed(seed)


def scales_unswizzle(swizzled, rows, cols):
    """Host (numpy uint8) MMA-layout scales -> row-major [rows x cols/16]."""
    import numpy as np
    src = np.ascontiguousarray(swizzled, dtype=np.uint8)
    out = np.zeros((rows, cols // 16), dtype=np.uint8)
    _check(lib().nvfp4_scales_unswizzle(src.ctypes.data_as(ctypes.c_void_p), rows, cols,
                                        out.ctypes.data_as(ctypes.c_void_p)), "scales_unswizzle")
    return out


# ---- device buffers ---------------------------------------------------------------------

class QuantizedTensor:
    """A quantized operand whose buffers torch allocated: codes [rows x cols/2] uint8,
    scales (MMA layout) uint8, amax float32[1]."""

    def __init__(self, rows, cols, device="cuda"):
        self.rows, self.cols = rows, cols
        self.codes = _poisoned(torch.empty((rows, cols // 2), dtype=torch.uint8, device=device))
        self.scales = _poisoned(torch.empty((scales_bytes(rows, cols),), dtype=torch.uint8,
                                            device=device))
        self.amax = _poisoned(torch.zeros((1,), dtype=torch.float32, device=device))

    @classmethod
    def from_buffers(cls, codes, scales, amax):
        """An operand of buffers that hold one already (codes [rows x cols/2])."""
        if (codes.dtype != torch.uint8 or codes.dim() != 2 or not codes.is_contiguous()
                or scales.dtype != torch.uint8 or not scales.is_contiguous()
                or amax.dtype != torch.float32 or amax.numel() != 1):
            raise ValueError("an operand has contiguous uint8 codes [rows x cols/2], uint8 scales and "
                             "one float32 amax")
        q = cls.__new__(cls)
        q.rows, q.cols = codes.shape[0], 2 * codes.shape[1]
        if scales.device != codes.device or amax.device != codes.device:
            raise ValueError("an operand's codes, scales and amax are on one device")
        if scales.numel() < scales_bytes(q.rows, q.cols):
            raise ValueError(f"scales: {scales.numel()} bytes are too few for {q.rows} x {q.cols}")
        q.codes, q.scales, q.amax = codes, scales, amax
        return q

    def operand(self):
        return Operand(self.codes.data_ptr(), self.scales.data_ptr(), self.amax.data_ptr(),
                       self.rows, self.cols)


def _dtype_code(dtype):
    if dtype == torch.float32:
        return OUT_F32
    if dtype == torch.bfloat16:
        return OUT_BF16
    raise TypeError(f"unsupported output dtype {dtype}")


def _workspace(nbytes, device):
    if nbytes == 0:
        return None
    return _poisoned(torch.empty((nbytes,), dtype=torch.uint8, device=device))


def quantize(x, flags, seed=0, offset=0, out_row=None, out_col=None, workspace=None,
             dev_status=None, stream=None):
    """nvfp4_quantize on a 2D bf16 CUDA tensor (row stride x.stride(0))."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if flags & ROWWISE and out_row is None:
        out_row = QuantizedTensor(rows, cols, x.device)
    if flags & COLWISE and out_col is None:
        out_col = QuantizedTensor(cols, rows, x.device)
    if workspace is None:
        workspace = _workspace(workspace_bytes(rows, cols, flags), x.device)
    op_r = out_row.operand() if out_row is not None else None
    op_c = out_col.operand() if out_col is not None else None
    st = lib().nvfp4_quantize(_ptr(x), rows, cols, x.stride(0), flags, seed, offset,
                              ctypes.byref(op_r) if op_r is not None else None,
                              ctypes.byref(op_c) if op_c is not None else None,
                              _ptr(workspace), _status(dev_status), _stream(stream))
    _check(st, "nvfp4_quantize")
    return out_row, out_col


def rht_quantize(x, sign_mask, flags=0, seed=0, offset=0, out_col=None, workspace=None,
                 dev_status=None, stream=None):
    """nvfp4_rht_quantize: x^T random-Hadamard-transformed and quantized along x's rows."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if out_col is None:
        out_col = QuantizedTensor(cols, rows, x.device)
    if workspace is None:
        workspace = _workspace(workspace_bytes(rows, cols, flags), x.device)
    op_c = out_col.operand()
    st = lib().nvfp4_rht_quantize(_ptr(x), rows, cols, x.stride(0), sign_mask, flags, seed,
                                  offset, ctypes.byref(op_c), _ptr(workspace), _status(dev_status),
                                  _stream(stream))
    _check(st, "nvfp4_rht_quantize")
    return out_col


def quantize_row_rht(x, sign_mask, flags=0, seed=0, offset=0, out_row=None, out_col=None,
                     workspace=None, dev_status=None, stream=None):
    """nvfp4_quantize_row_rht: x row-wise (stream `offset`) and x^T RHT'd column-wise (stream
    `offset + 1`) from one amax pass and one quantize pass."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if out_row is None:
        out_row = QuantizedTensor(rows, cols, x.device)
    if out_col is None:
        out_col = QuantizedTensor(cols, rows, x.device)
    if workspace is None:
        workspace = _workspace(workspace_bytes(rows, cols, flags), x.device)
    op_r, op_c = out_row.operand(), out_col.operand()
    st = lib().nvfp4_quantize_row_rht(_ptr(x), rows, cols, x.stride(0), sign_mask, flags, seed,
                                      offset, ctypes.byref(op_r), ctypes.byref(op_c),
                                      _ptr(workspace), _status(dev_status), _stream(stream))
    _check(st, "nvfp4_quantize_row_rht")
    return out_row, out_col


def _check_out(out, rows, cols, what):
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{what}: output must be float32 or bfloat16, got {out.dtype}")
    if tuple(out.shape) != (rows, cols) or out.stride(1) != 1 or not out.is_cuda:
        raise ValueError(f"{what}: output must be a CUDA [{rows} x {cols}] tensor with unit "
                         f"column stride, got {tuple(out.shape)} strides {out.stride()}")


def gemm(A, B, out=None, out_dtype=torch.float32, dev_status=None, stream=None, mx=False):
    """nvfp4_gemm (nvfp4_gemm_mx with `mx`): D = A . B^T (A, B QuantizedTensor).  The output
    type is out.dtype when `out` is given, else `out_dtype`."""
    name = "nvfp4_gemm_mx" if mx else "nvfp4_gemm"
    if out is None:
        out = _poisoned(torch.empty((A.rows, B.rows), dtype=out_dtype, device=A.codes.device))
    _check_out(out, A.rows, B.rows, name)
    d_dtype = _dtype_code(out.dtype)
    oa, ob = A.operand(), B.operand()
    st = getattr(lib(), name)(ctypes.byref(oa), ctypes.byref(ob), _ptr(out), d_dtype,
                              out.stride(0), _status(dev_status), _stream(stream))
    _check(st, name)
    return out


def gemm_amax(A, B, sign_mask, out=None, amax_out=None, dev_status=None, stream=None):
    """nvfp4_gemm_amax: bf16 D = A . B^T plus amax_out = [max |D|, max |RHT(D)|] (FP32)."""
    if out is None:
        out = _poisoned(torch.empty((A.rows, B.rows), dtype=torch.bfloat16,
                                    device=A.codes.device))
    _check_out(out, A.rows, B.rows, "nvfp4_gemm_amax")
    assert out.dtype == torch.bfloat16
    if amax_out is None:
        amax_out = _poisoned(torch.empty(2, dtype=torch.float32, device=A.codes.device))
    oa, ob = A.operand(), B.operand()
    st = lib().nvfp4_gemm_amax(ctypes.byref(oa), ctypes.byref(ob), _ptr(out), out.stride(0),
                               sign_mask, _ptr(amax_out), _status(dev_status), _stream(stream))
    _check(st, "nvfp4_gemm_amax")
    return out, amax_out


def selftest_wait_timeout(dev_status, stream=None):
    """nvfp4_selftest_wait_timeout: a bounded wait that nothing satisfies; after it the device
    status word has NVFP4_DEVSTAT_TIMEOUT set."""
    _check(lib().nvfp4_selftest_wait_timeout(_status(dev_status), _stream(stream)),
           "nvfp4_selftest_wait_timeout")


def is_bounds_checked():
    """nvfp4_bounds_checked of the library calls currently go to."""
    return bool(lib().nvfp4_bounds_checked())


def selftest_bounds(dev_status, stream=None):
    """nvfp4_selftest_bounds (checked build only): one refused store past a buffer's declared
    end; after it the device status word has NVFP4_DEVSTAT_BOUNDS set."""
    _check(lib().nvfp4_selftest_bounds(_status(dev_status), _stream(stream)),
           "nvfp4_selftest_bounds")


def linear_fprop(X, W, out=None, out_dtype=torch.float32, workspace=None, dev_status=None,
                 stream=None):
    T, I = X.shape
    O = W.shape[0]
    if out is None:
        out = _poisoned(torch.empty((T, O), dtype=out_dtype, device=X.device))
    _check_out(out, T, O, "nvfp4_linear_fprop")
    if workspace is None:
        workspace = _workspace(linear_workspace_bytes(T, I, O), X.device)
    st = lib().nvfp4_linear_fprop(_ptr(X), _ptr(W), T, I, O, _ptr(out), _dtype_code(out.dtype),
                                  _ptr(workspace), _status(dev_status), _stream(stream))
    _check(st, "nvfp4_linear_fprop")
    return out


def linear_dgrad(dY, W, seed, offset, out=None, out_dtype=torch.float32, workspace=None,
                 dev_status=None, stream=None):
    T, O = dY.shape
    I = W.shape[1]
    if out is None:
        out = _poisoned(torch.empty((T, I), dtype=out_dtype, device=dY.device))
    _check_out(out, T, I, "nvfp4_linear_dgrad")
    if workspace is None:
        workspace = _workspace(linear_workspace_bytes(T, I, O), dY.device)
    st = lib().nvfp4_linear_dgrad(_ptr(dY), _ptr(W), T, I, O, seed, offset, _ptr(out),
                                  _dtype_code(out.dtype), _ptr(workspace), _status(dev_status),
                                  _stream(stream))
    _check(st, "nvfp4_linear_dgrad")
    return out


def linear_dgrad_quantized(dY, W, seed, offset, sign_mask, next_seed, next_offset, out=None,
                           out_row=None, out_col=None, workspace=None, dev_status=None,
                           stream=None):
    """nvfp4_linear_dgrad_quantized: bf16 dX = dY . W plus dX's row-wise SR and RHT'd
    column-wise SR operands for the previous layer (returns dX, dX_row, dX_col)."""
    T, O = dY.shape
    I = W.shape[1]
    if out is None:
        out = _poisoned(torch.empty((T, I), dtype=torch.bfloat16, device=dY.device))
    _check_out(out, T, I, "nvfp4_linear_dgrad_quantized")
    if out.dtype != torch.bfloat16:
        raise TypeError("nvfp4_linear_dgrad_quantized: dX must be bfloat16")
    if out_row is None:
        out_row = QuantizedTensor(T, I, dY.device)
    if out_col is None:
        out_col = QuantizedTensor(I, T, dY.device)
    if workspace is None:
        workspace = _workspace(linear_workspace_bytes(T, I, O), dY.device)
    op_r, op_c = out_row.operand(), out_col.operand()
    st = lib().nvfp4_linear_dgrad_quantized(_ptr(dY), _ptr(W), T, I, O, seed, offset, _ptr(out),
                                            sign_mask, next_seed, next_offset,
                                            ctypes.byref(op_r), ctypes.byref(op_c),
                                            _ptr(workspace), _status(dev_status), _stream(stream))
    _check(st, "nvfp4_linear_dgrad_quantized")
    return out, out_row, out_col


def linear_wgrad(dY, X, sign_mask, seed, offset, out=None, out_dtype=torch.float32,
                 workspace=None, dev_status=None, stream=None):
    T, O = dY.shape
    I = X.shape[1]
    if out is None:
        out = _poisoned(torch.empty((O, I), dtype=out_dtype, device=dY.device))
    _check_out(out, O, I, "nvfp4_linear_wgrad")
    if workspace is None:
        workspace = _workspace(linear_workspace_bytes(T, I, O), dY.device)
    st = lib().nvfp4_linear_wgrad(_ptr(dY), _ptr(X), T, I, O, sign_mask, seed, offset, _ptr(out),
                                  _dtype_code(out.dtype), _ptr(workspace), _status(dev_status),
                                  _stream(stream))
    _check(st, "nvfp4_linear_wgrad")
    return out


# ---- mixture-of-experts layers -----------------------------------------------------------

def expert_rows(tokens, k, experts):
    """Rows of an expert-ordered matrix that hold every routing (0: sizes outside the limits)."""
    return lib().nvfp4_expert_rows(tokens, k, experts)


def experts_workspace_bytes(plan, I, O):
    return lib().nvfp4_experts_workspace_bytes(plan.tokens, plan.k, plan.experts, plan.rows, I, O)


def _queue(what, stream, *tensors):
    """The handle of the stream a call goes to (None: the current one).  The calls run on the current
    device, with its kernels: tensors elsewhere are refused."""
    here = -1
    for t in tensors:
        if t is None:
            continue
        d = t.get_device()
        if d >= 0 and here < 0:
            here = torch.cuda.current_device()
        if d < 0 or d != here:
            raise ValueError(f"{what}: every tensor must be on the current CUDA device, got {t.device}")
    return torch._C._cuda_getCurrentRawStream(here) if stream is None else stream.cuda_stream


def _status_word(t):
    if t is None:
        return None if _active is LIB_PATH else _status(None)
    if t.dtype != torch.int32 or t.numel() < 1:
        raise TypeError(f"dev_status must hold an int32, got {t.numel()} of {t.dtype}")
    return t.data_ptr()


def _address(t):
    return None if t is None else t.data_ptr()


def _matrix(what, t, dtypes, rows, cols):
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows) or (
            cols is not None and t.shape[1] != cols) or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be [{'rows' if rows is None else rows} x "
                         f"{'cols' if cols is None else cols}] with unit column stride, got "
                         f"{tuple(t.shape)} strides {t.stride()}")


def _dense(what, t, dtype, shape):
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous {tuple(shape)}, got {tuple(t.shape)}")


def _row_stride(t):
    # a one-row view may carry any stride, aligned or not; it is never used
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _workspace_size(workspace, need):
    if workspace is not None and not workspace.is_contiguous():  # an expanded one has less behind it
        raise ValueError("the workspace must be contiguous")
    have = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if have < need:
        raise ValueError(f"the workspace has {have} bytes, the call needs {need}")


_F32_BF16 = (torch.float32, torch.bfloat16)
_BF16 = (torch.bfloat16,)


def _new(shape, dtype, device):
    """torch.empty without its dispatch over layouts (a third of its time on the host)."""
    if len(shape) == 1:
        return torch.empty_strided(shape, (1,), dtype=dtype, device=device)
    return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=device)


_no_stream = contextlib.nullcontext()


def _allocating(stream):
    """Buffers made for a call belong to the stream that uses them."""
    return _no_stream if stream is None else torch.cuda.stream(stream)


class ExpertPlan:
    """The expert-ordered rows of a routing: offsets [experts + 1], pair_row [tokens, k] and
    row_token [rows], int32 (nvfp4_expert_plan).  The tensors' contents may change, not the tensors:
    the calls use the addresses taken here."""

    _FIXED = frozenset(("offsets", "pair_row", "row_token", "tokens", "k", "experts", "rows",
                        "_struct", "ref"))

    def __setattr__(self, name, value):
        if name in self._FIXED and "ref" in self.__dict__:
            raise AttributeError(f"ExpertPlan.{name} cannot be replaced; make a plan of the new tensors")
        super().__setattr__(name, value)

    def __init__(self, offsets, pair_row, row_token):
        if not (offsets.dtype is pair_row.dtype is row_token.dtype is torch.int32
                and offsets.dim() == row_token.dim() == 1 and pair_row.dim() == 2
                and offsets.is_contiguous() and pair_row.is_contiguous()
                and row_token.is_contiguous()):
            raise ValueError("plan: offsets [experts + 1], pair_row [tokens, k] and row_token [rows] "
                             "must be contiguous int32 tensors")
        if not offsets.device == pair_row.device == row_token.device:
            raise ValueError("plan: its tensors are on one device")
        tokens, k = pair_row.shape
        experts, rows = offsets.numel() - 1, row_token.numel()
        struct = PlanStruct(offsets.data_ptr(), pair_row.data_ptr(), row_token.data_ptr(), tokens, k,
                            experts, rows)
        # at once, not through __setattr__ (half of a plan's time on the host)
        self.__dict__.update(offsets=offsets, pair_row=pair_row, row_token=row_token, tokens=tokens, k=k,
                             experts=experts, rows=rows, _struct=struct,
                             ref=ctypes.byref(struct))  # what the C calls take

    @classmethod
    def empty(cls, tokens, k, experts, rows=None, device="cuda"):
        if rows is None:
            rows = expert_rows(tokens, k, experts)
        if rows == 0:
            raise NVFP4Error(ERR_SHAPE, f"expert plan of {tokens} tokens, {k} of {experts} experts")

        return cls(*(_poisoned(_new(shape, torch.int32, device))
                     for shape in ((experts + 1,), (tokens, k), (rows,))))


def route(logits, k, bias=None, sigmoid=False, groups=1, top_groups=1, renorm=True, scale=1.0,
          experts=None, weights=None, dev_status=None, stream=None):
    """nvfp4_route: the k experts of every token (int32 [T, k]) and their weights (float32)."""
    _matrix("logits", logits, _F32_BF16, None, None)
    T, E = logits.shape
    if bias is not None:
        _dense("bias", bias, torch.float32, (E,))
    with _allocating(stream):
        if experts is None:
            experts = _poisoned(_new((T, max(k, 0)), torch.int32, logits.device))
        if weights is None:
            weights = _poisoned(_new((T, max(k, 0)), torch.float32, logits.device))
    _dense("experts", experts, torch.int32, (T, k))
    _dense("weights", weights, torch.float32, (T, k))
    queue = _queue("nvfp4_route", stream, logits, bias, experts, weights, dev_status)
    _check(lib().nvfp4_route(_address(logits), _dtype_code(logits.dtype), T, E, _row_stride(logits),
                             _address(bias), int(bool(sigmoid)), groups, top_groups, k, int(bool(renorm)),
                             scale, _address(experts), _address(weights), _status_word(dev_status),
                             queue), "nvfp4_route")
    return experts, weights


def route_backward(logits, experts, dweights, sigmoid=False, renorm=True, scale=1.0, dlogits=None,
                   dev_status=None, stream=None):
    """nvfp4_route_backward: gradient of route's weights with respect to the logits."""
    _matrix("logits", logits, _F32_BF16, None, None)
    T, E = logits.shape
    k = experts.shape[-1]
    _dense("experts", experts, torch.int32, (T, k))
    _dense("dweights", dweights, torch.float32, (T, k))
    if dlogits is None:
        with _allocating(stream):
            dlogits = _poisoned(_new((T, E), logits.dtype, logits.device))
    _matrix("dlogits", dlogits, (logits.dtype,), T, E)
    queue = _queue("nvfp4_route_backward", stream, logits, experts, dweights, dlogits, dev_status)
    _check(lib().nvfp4_route_backward(_address(logits), _dtype_code(logits.dtype), T, E,
                                      _row_stride(logits), _address(experts), _address(dweights),
                                      int(bool(sigmoid)), k, int(bool(renorm)), scale,
                                      _address(dlogits), _row_stride(dlogits), _status_word(dev_status),
                                      queue), "nvfp4_route_backward")
    return dlogits


def expert_plan(experts, n_experts, plan=None, workspace=None, dev_status=None, stream=None):
    """nvfp4_plan_experts: the ExpertPlan of a routing experts [T, k] (int32)."""
    T, k = experts.shape
    _dense("experts", experts, torch.int32, (T, k))
    with _allocating(stream):
        if plan is None:
            plan = ExpertPlan.empty(T, k, n_experts, device=experts.device)
        if workspace is None:
            workspace = _workspace(lib().nvfp4_expert_plan_workspace_bytes(T, k, n_experts),
                                   experts.device)
    _workspace_size(workspace, lib().nvfp4_expert_plan_workspace_bytes(T, k, n_experts))
    if (plan.tokens, plan.k, plan.experts) != (T, k, n_experts):
        raise ValueError(f"plan is for {plan.tokens} tokens, {plan.k} of {plan.experts} experts")
    queue = _queue("nvfp4_plan_experts", stream, experts, plan.offsets, workspace, dev_status)
    _check(lib().nvfp4_plan_experts(_address(experts), plan.ref, _address(workspace),
                                    _status_word(dev_status), queue), "nvfp4_plan_experts")
    return plan


def _source_rows(plan, gather):
    return plan.tokens if gather else plan.rows


def quantize_grouped(x, plan, flags, sign_mask=0, seed=0, offset=0, out_row=None, out_col=None,
                     workspace=None, dev_status=None, stream=None):
    """nvfp4_quantize_grouped: an expert-ordered matrix row-wise (out_row) and / or RHT'd
    column-wise (out_col); with GATHER x has a row per token."""
    _matrix("x", x, _BF16, _source_rows(plan, flags & GATHER), None)
    cols = x.shape[1]
    with _allocating(stream):
        if flags & ROWWISE and out_row is None:
            out_row = QuantizedTensor(plan.rows, cols, x.device)
        if flags & COLWISE and out_col is None:
            out_col = QuantizedTensor(cols, plan.rows, x.device)
        if workspace is None:
            workspace = _workspace(workspace_bytes(plan.rows, cols, flags), x.device)
    _workspace_size(workspace, workspace_bytes(plan.rows, cols, flags))
    queue = _queue("nvfp4_quantize_grouped", stream, x, plan.offsets, workspace, dev_status,
                   out_row and out_row.codes, out_col and out_col.codes)
    op_r = out_row.operand() if out_row is not None else None
    op_c = out_col.operand() if out_col is not None else None
    _check(lib().nvfp4_quantize_grouped(
        _address(x), cols, _row_stride(x), plan.ref, sign_mask, flags, seed, offset,
        ctypes.byref(op_r) if op_r is not None else None,
        ctypes.byref(op_c) if op_c is not None else None, _address(workspace), _status_word(dev_status),
        queue), "nvfp4_quantize_grouped")
    return out_row, out_col


def _grouped_out(what, out, rows, cols, out_dtype, device, stream):
    if out is None:
        with _allocating(stream):
            out = _poisoned(_new((rows, cols), out_dtype, device))
    _matrix(what, out, _F32_BF16, rows, cols)
    return out


def gemm_grouped(A, W, plan, out=None, out_dtype=torch.bfloat16, dev_status=None, stream=None):
    """nvfp4_gemm_grouped: every expert's rows of A times its matrix of W, stacked by rows
    ((E * N) x K) or side by side (N x (E * K))."""
    E = plan.experts
    N = W.rows // E if W.cols == A.cols and W.rows % E == 0 else W.rows
    out = _grouped_out("out", out, plan.rows, N, out_dtype, A.codes.device, stream)
    queue = _queue("nvfp4_gemm_grouped", stream, A.codes, W.codes, plan.offsets, out, dev_status)
    oa, ob = A.operand(), W.operand()
    _check(lib().nvfp4_gemm_grouped(ctypes.byref(oa), ctypes.byref(ob), plan.ref,
                                    _address(out), _dtype_code(out.dtype), _row_stride(out),
                                    _status_word(dev_status), queue), "nvfp4_gemm_grouped")
    return out


def gemm_grouped_k(A, B, plan, out=None, out_dtype=torch.float32, dev_status=None, stream=None):
    """nvfp4_gemm_grouped_k: D_e = A . B^T over expert e's rows, [(E * A.rows) x B.rows]."""
    out = _grouped_out("out", out, plan.experts * A.rows, B.rows, out_dtype, A.codes.device, stream)
    queue = _queue("nvfp4_gemm_grouped_k", stream, A.codes, B.codes, plan.offsets, out, dev_status)
    oa, ob = A.operand(), B.operand()
    _check(lib().nvfp4_gemm_grouped_k(ctypes.byref(oa), ctypes.byref(ob),
                                      plan.ref, _address(out), _dtype_code(out.dtype),
                                      _row_stride(out), _status_word(dev_status), queue),
           "nvfp4_gemm_grouped_k")
    return out


def _experts_workspace(workspace, plan, I, O, device, stream):
    need = experts_workspace_bytes(plan, I, O)
    if workspace is None:
        with _allocating(stream):
            return _workspace(need, device)
    _workspace_size(workspace, need)
    return workspace


def experts_fprop(X, W, plan, gather=True, out=None, out_dtype=torch.bfloat16, workspace=None,
                  dev_status=None, stream=None):
    """nvfp4_experts_fprop: Y [rows x O] of X (a row per token, or with gather=False in expert
    order) and the stacked, row-wise quantized weights W [(E * O) x I]."""
    _matrix("X", X, _BF16, _source_rows(plan, gather), W.cols)
    I, O = W.cols, W.rows // plan.experts
    out = _grouped_out("out", out, plan.rows, O, out_dtype, X.device, stream)
    workspace = _experts_workspace(workspace, plan, I, O, X.device, stream)
    queue = _queue("nvfp4_experts_fprop", stream, X, W.codes, plan.offsets, out, workspace, dev_status)
    op = W.operand()
    _check(lib().nvfp4_experts_fprop(_address(X), _row_stride(X), int(bool(gather)), ctypes.byref(op),
                                     plan.ref, I, O, _address(out),
                                     _dtype_code(out.dtype), _row_stride(out), _address(workspace),
                                     _status_word(dev_status), queue), "nvfp4_experts_fprop")
    return out


def experts_dgrad(dY, Wt, plan, seed, offset, out=None, out_dtype=torch.bfloat16, workspace=None,
                  dev_status=None, stream=None):
    """nvfp4_experts_dgrad: dX [rows x I] of dY [rows x O] and the column-wise quantized weights
    Wt [I x (E * O)]."""
    I, O = Wt.rows, Wt.cols // plan.experts
    _matrix("dY", dY, _BF16, plan.rows, O)
    out = _grouped_out("out", out, plan.rows, I, out_dtype, dY.device, stream)
    workspace = _experts_workspace(workspace, plan, I, O, dY.device, stream)
    queue = _queue("nvfp4_experts_dgrad", stream, dY, Wt.codes, plan.offsets, out, workspace, dev_status)
    op = Wt.operand()
    _check(lib().nvfp4_experts_dgrad(_address(dY), _row_stride(dY), ctypes.byref(op),
                                     plan.ref, I, O, seed, offset, _address(out),
                                     _dtype_code(out.dtype), _row_stride(out), _address(workspace),
                                     _status_word(dev_status), queue), "nvfp4_experts_dgrad")
    return out


def experts_wgrad(dY, X, plan, sign_mask, seed, offset, gather=True, out=None,
                  out_dtype=torch.float32, workspace=None, dev_status=None, stream=None):
    """nvfp4_experts_wgrad: dW [(E * O) x I] of dY [rows x O] and X (a row per token, or with
    gather=False in expert order)."""
    _matrix("X", X, _BF16, _source_rows(plan, gather), None)
    _matrix("dY", dY, _BF16, plan.rows, None)
    I, O = X.shape[1], dY.shape[1]
    out = _grouped_out("out", out, plan.experts * O, I, out_dtype, dY.device, stream)
    workspace = _experts_workspace(workspace, plan, I, O, dY.device, stream)
    queue = _queue("nvfp4_experts_wgrad", stream, dY, X, plan.offsets, out, workspace, dev_status)
    _check(lib().nvfp4_experts_wgrad(_address(dY), _row_stride(dY), _address(X), _row_stride(X),
                                     int(bool(gather)), plan.ref, I, O, sign_mask,
                                     seed, offset, _address(out), _dtype_code(out.dtype),
                                     _row_stride(out), _address(workspace), _status_word(dev_status),
                                     queue), "nvfp4_experts_wgrad")
    return out


def combine(Y, plan, weights=None, out=None, out_dtype=torch.bfloat16, dev_status=None, stream=None):
    """nvfp4_combine: out[t] = sum_j weights[t, j] Y[row of pair (t, j)] (weights None: all 1)."""
    _matrix("Y", Y, _BF16, plan.rows, None)
    if weights is not None:
        _dense("weights", weights, torch.float32, (plan.tokens, plan.k))
    out = _grouped_out("out", out, plan.tokens, Y.shape[1], out_dtype, Y.device, stream)
    queue = _queue("nvfp4_combine", stream, Y, plan.pair_row, weights, out, dev_status)
    _check(lib().nvfp4_combine(_address(Y), Y.shape[1], _row_stride(Y), plan.ref,
                               _address(weights), _address(out), _dtype_code(out.dtype), _row_stride(out),
                               _status_word(dev_status), queue), "nvfp4_combine")
    return out


def combine_backward(dout, Y, plan, weights, dy=None, dweights=None, dev_status=None, stream=None):
    """nvfp4_combine_backward: (dY [rows x cols] bf16, dweights [T, k] float32)."""
    _matrix("dout", dout, _F32_BF16, plan.tokens, None)
    cols = dout.shape[1]
    _matrix("Y", Y, _BF16, plan.rows, cols)
    _dense("weights", weights, torch.float32, (plan.tokens, plan.k))
    with _allocating(stream):
        if dy is None:
            dy = _poisoned(_new((plan.rows, cols), torch.bfloat16, Y.device))
        if dweights is None:
            dweights = _poisoned(_new((plan.tokens, plan.k), torch.float32, Y.device))
    _matrix("dy", dy, _BF16, plan.rows, cols)
    _dense("dweights", dweights, torch.float32, (plan.tokens, plan.k))
    queue = _queue("nvfp4_combine_backward", stream, dout, Y, plan.pair_row, weights, dy, dweights, dev_status)
    _check(lib().nvfp4_combine_backward(_address(dout), _dtype_code(dout.dtype), _row_stride(dout),
                                        _address(Y), cols, _row_stride(Y), plan.ref,
                                        _address(weights), _address(dy), _row_stride(dy), _address(dweights),
                                        _status_word(dev_status), queue), "nvfp4_combine_backward")
    return dy, dweights
