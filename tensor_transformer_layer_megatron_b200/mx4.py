"""Microscaled 4-bit operands and operators: the binding of mgt_mx4_* and mgt_gemm_mx4* in
include/mgt_layer.h. Argument checks and marshalling only; the work is in the CUDA kernels."""
from __future__ import annotations

import ctypes

import torch

from . import _check, load_library


class _Mx4Operand(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
            ("ld", ctypes.c_int64), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
            ("factor", ctypes.c_void_p)]


MX4_FORMATS = {"mxfp4": 0, "nvfp4": 1}
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


# Rows and columns of an operand, as the library has it. Sizes travel as int32, and ctypes cuts what
# does not fit without a word, so larger ones are refused here.
_MOST = 1 << 30


def _up128(n):
    return (n + 127) // 128 * 128


class Mx4:
    """A microscaled 4-bit operand of `rows` by `cols` (see mgt_mx4 in include/mgt_layer.h):
    device buffers for its codes [rows, ld / 2] and scale tiles, both uint8, and for "nvfp4" its
    factor {amax, f}, two fp32 on the device. Buffers are allocated (f = 1), or given: codes
    with rows of ld / 2 contiguous bytes, `scales` with room for whole tiles of 128 rows.

    Calls go by the addresses taken here, so the attributes are read-only, but for `factor`: another
    tensor assigned to it is the one that calls use from then on (graphs captured before, and parts
    made before, keep the one they had)."""

    _FIXED = ("fmt", "rows", "cols", "ld", "codes", "scales", "device", "index")

    def __init__(self, fmt, rows, cols, device="cuda", codes=None, scales=None, factor=None):
        if fmt not in MX4_FORMATS:
            raise ValueError("format must be one of %s" % sorted(MX4_FORMATS))
        rows, cols = int(rows), int(cols)
        if rows < 1 or cols < 1:
            raise ValueError("an operand has at least one row and one column")
        if rows > _MOST or cols > _MOST:
            raise ValueError("an operand has at most 2**30 rows and columns")
        block = 32 if fmt == "mxfp4" else 16
        if codes is None:
            codes = torch.empty(rows, _up128(cols) // 2, dtype=torch.uint8, device=device)
        if codes.dim() != 2 or codes.dtype != torch.uint8 or codes.shape[0] < rows or \
            codes.stride(1) != 1 or (codes.shape[0] > 1 and
                                     codes.stride(0) != codes.shape[1]):
            raise TypeError("codes must be contiguous uint8 [rows, ld / 2]")
        ld = 2 * codes.shape[1]
        if ld % 128 or ld < _up128(cols):
            raise ValueError("ld must be a multiple of 128 that holds all columns")
        need = _up128(rows) * ld // block
        if scales is None:
            scales = torch.empty(need, dtype=torch.uint8, device=codes.device)
        if scales.dtype != torch.uint8 or not scales.is_contiguous():
            raise TypeError("scales must be contiguous uint8")
        if scales.numel() < need:
            raise ValueError("scales need %d bytes" % need)
        if scales.device != codes.device:
            raise ValueError("codes, scales and factor must be on one device")
        if fmt == "nvfp4" and factor is None:
            factor = torch.ones(2, dtype=torch.float32, device=codes.device)
        self.__dict__.update(fmt=fmt, rows=rows, cols=cols, ld=ld, codes=codes,
                             scales=scales, device=codes.device, index=codes.get_device())
        self.__dict__["factor"] = self._factor(factor)
        self._bind(0, 0)

    def _factor(self, t):
        """t, checked as this operand's factor (None: an operand without one)."""
        if t is None and self.fmt != "nvfp4":
            return t
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.numel() < 2 or \
            not t.is_contiguous():
            raise TypeError("factor must be two contiguous float32")
        if t.device != self.device:
            raise ValueError("codes, scales and factor must be on one device")
        return t

    def __setattr__(self, name, value):
        if name in self._FIXED:
            raise AttributeError("%s of an operand is fixed: make another one" % name)
        if name == "factor":
            self.__dict__["factor"] = self._factor(value)
            self._bind(self._row, self._col)
        else:
            object.__setattr__(self, name, value)

    def _bind(self, row, col):
        block = 32 if self.fmt == "mxfp4" else 16
        c = _Mx4Operand(
            MX4_FORMATS[self.fmt], self.rows, self.cols, self.ld,
            self.codes.data_ptr() + (row * self.ld + col) // 2,
            self.scales.data_ptr() + 512 * (row // 128 * (self.ld // (4 * block)) +
                                        col // (4 * block)),
            None if self.factor is None else self.factor.data_ptr())
        self.__dict__.update(_row=row, _col=col, _c=c, _addr=ctypes.addressof(c))

    def part(self, row, rows, col, cols):
        """The operand of rows row .. row + rows - 1 and columns col .. col + cols - 1 of this
        one, in the same buffers; row and col are multiples of 128. Where its columns end inside a
        group of 128, a product reads the whole group, whose rest has to hold zeros, as it does
        at the operand's end and in a part that was quantised into."""
        if row % 128 or col % 128 or row < 0 or col < 0 or rows < 1 or cols < 1 or \
            row + rows > self.rows or _up128(col + cols) > _up128(self.cols):
            raise ValueError("a part starts at multiples of 128 and lies inside the operand")
        p = object.__new__(Mx4)
        p.__dict__.update(self.__dict__, rows=int(rows), cols=int(cols))
        p._bind(self._row + row, self._col + col)
        return p

    def rows_view(self, row, rows):
        """The operand of rows row .. row + rows - 1 (row a multiple of 128), all columns."""
        return self.part(row, rows, 0, self.cols)


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_current_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_functions = {}


def _matrix(t, name):
    """(dtype code, row stride, rows, columns) of a 2-D fp32 or bf16 tensor with contiguous rows."""
    dtype = t.dtype
    if dtype is _BF16:
        code = 1
    elif dtype is _F32:
        code = 0
    else:
        raise TypeError("%s must be float32 or bfloat16" % name)
    shape = t.shape
    if len(shape) != 2:
        raise TypeError("%s must be 2-D with contiguous rows" % name)
    rows, cols = shape
    if (rows | cols) >> 31:
        raise ValueError("%s must have fewer than 2**31 rows and columns" % name)
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise TypeError("%s must be 2-D with contiguous rows" % name)
    return code, (ld if rows > 1 else max(ld, cols)), rows, cols


def _index(*things):
    """The CUDA device index that all tensors and operands (or None) share."""
    index = None
    for t in things:
        if t is not None:
            i = t.index if type(t) is Mx4 else t.get_device()
            if index is None:
                index = i
            elif i != index:
                raise ValueError("all tensors must be on one device")
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    return index


def _call(name, index, stream, *args):
    """Launch on device `index`, on its current stream unless one is given."""
    if stream is None:
        handle = _current_stream(index)
    elif stream.device.index != index:
        raise ValueError("the stream belongs to another device than the tensors")
    else:
        handle = stream.cuda_stream
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(load_library(), name)
    if _current_device() == index:
        code = f(*args, handle)
    else:
        with torch.cuda.device(index):
            code = f(*args, handle)
    if code:
        _check(code, name)


def _check_status(status):
    if status.dtype is not _I32:
        raise TypeError("status must be an int32 device word")


def _addr(q):
    return None if q is None else q._addr


def mx4_tensor_factor(x, factor, stream=None):
    """factor = {amax, f} of a 2-D tensor for "nvfp4" (see mgt_mx4_tensor_factor)."""
    code, ld, rows, cols = _matrix(x, "x")
    if factor.dtype != torch.float32 or factor.numel() < 2 or not factor.is_contiguous():
        raise TypeError("factor must be two contiguous float32")
    _call("mgt_mx4_tensor_factor", _index(x, factor), stream, code, rows, cols,
          x.data_ptr(), ld, factor.data_ptr())


def mx4_quantize(x, q=None, qt=None, stream=None):
    """Quantise x [rows, cols] (fp32 or bf16) into q and / or, transposed, into qt (see
    mgt_mx4_quantize)."""
    code, ld, rows, cols = _matrix(x, "x")
    if (q is not None and (q.rows != rows or q.cols != cols)) or \
            (qt is not None and (qt.cols != rows or qt.rows != cols)):
        raise ValueError("q takes x's shape and qt the transposed one")
    _call("mgt_mx4_quantize", _index(x, q, qt), stream, code, x.data_ptr(), ld, _addr(q),
          _addr(qt))


def mx4_dequantize(q, y, stream=None):
    """y [rows, cols] (fp32 or bf16) = what q stands for (see mgt_mx4_dequantize)."""
    code, ld, rows, cols = _matrix(y, "y")
    if rows != q.rows or cols != q.cols:
        raise ValueError("y takes q's shape")
    _call("mgt_mx4_dequantize", _index(y, q), stream, _addr(q), code, y.data_ptr(), ld)


def gemm_mx4(A, B, C, status, stream=None):
    """C [A.rows, B.rows] (fp32 or bf16) = A B^T of two 4-bit operands (see mgt_gemm_mx4);
    status an int32 device tensor that receives timeout codes."""
    code, ld, rows, cols = _matrix(C, "C")
    _check_status(status)
    if rows != A.rows or cols != B.rows or A.cols != B.cols:
        raise ValueError("C must be [A.rows, B.rows], and A and B have the same columns")
    _call("mgt_gemm_mx4", _index(C, A, B, status), stream, A._addr, B._addr, C.data_ptr(), code, ld,
          status.data_ptr())


def gemm_mx4_gated(X, W, a, status, act="silu", u=None, stream=None):
    """a = Q(act(gate) * up) with [gate | up] = X W^T, one kernel (see mgt_gemm_mx4_gated): W has
    a.cols gate rows from row 0 and up rows from row a.cols rounded up to 128. u (bf16
    [X.rows, 2 a.cols], optional) keeps [gate | up] for the backward."""
    _check_status(status)
    ldu = 0
    if u is not None:
        if u.dtype != torch.bfloat16:
            raise TypeError("u must be bfloat16")
        ldu = _matrix(u, "u")[1]
        if tuple(u.shape) != (X.rows, 2 * a.cols):
            raise ValueError("u must be [X.rows, 2 * a.cols]")
    if act not in ACTIVATIONS:
        raise ValueError("act must be one of %s" % sorted(ACTIVATIONS))
    _call("mgt_gemm_mx4_gated", _index(a, X, W, u, status), stream, X._addr, W._addr,
          ACTIVATIONS[act], a._addr, None if u is None else u.data_ptr(), ldu,
          status.data_ptr())


def mx4_gated_bwd(da, u, du=None, dut=None, at=None, act="silu", stream=None):
    """Gradients of the gated product from da (bf16 [rows, ffn]) and u = [gate | up] (bf16
    [rows, 2 ffn]), quantised along the rows (du), along the columns (dut), and the product itself
    transposed (at); see mgt_mx4_gated_bwd for their layouts."""
    if da.dtype != torch.bfloat16 or u.dtype != torch.bfloat16:
        raise TypeError("da and u must be bfloat16")
    ldda, ldu = _matrix(da, "da")[1], _matrix(u, "u")[1]
    if tuple(u.shape) != (da.shape[0], 2 * da.shape[1]):
        raise ValueError("u must be [rows, 2 * ffn]")
    if act not in ACTIVATIONS:
        raise ValueError("act must be one of %s" % sorted(ACTIVATIONS))
    _call("mgt_mx4_gated_bwd", _index(da, u, du, dut, at), stream, ACTIVATIONS[act],
          da.shape[0], da.shape[1], da.data_ptr(), ldda, u.data_ptr(), ldu,
          _addr(du), _addr(dut), _addr(at))
