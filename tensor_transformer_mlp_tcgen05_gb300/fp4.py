"""Microscaled four-bit floating point: quantisation, the product of quantised
matrices and a linear layer on packed weights, as wrappers over the C ABI in
include/tp_fp4.h (which defines the formats).  csrc/pycall.cpp checks shapes, types
and devices; all arithmetic happens in libtpmlp's kernels.

A plain matrix is a bf16 or fp32 CUDA tensor [rows, cols] with consecutive row
elements and any row stride.  It is quantised along its rows, in blocks of 16
elements ("nvfp4") or 32 ("mxfp4"), or along its columns with ``transpose``.

With ``stream`` the work, and the outputs' memory, belong to that stream;
otherwise to the current one of the tensors' device.  The caller keeps the inputs
alive until that stream has read them.
"""
from __future__ import annotations

import torch

from . import binding as B_

_FORMATS = {"nvfp4": B_.TPFP4_NV, "mxfp4": B_.TPFP4_MX}
_DTYPES = {torch.bfloat16: B_.TPMLP_BF16, torch.float32: B_.TPMLP_FP32}


def _format(name: str) -> int:
    if name not in _FORMATS:
        raise ValueError(f"format must be one of {sorted(_FORMATS)}")
    return _FORMATS[name]


def _dtype(t) -> int:
    if t not in _DTYPES:
        raise ValueError("dtype must be torch.bfloat16 or torch.float32")
    return _DTYPES[t]


def _scale(scale) -> float:
    """None (from the matrix) is 0 at the C ABI; a 0 from the caller is not."""
    if scale is None:
        return 0.0
    if not scale > 0:
        raise ValueError("scale must be a power of two, or None")
    return float(scale)


class Fp4Tensor:
    """A packed matrix [rows, cols]: ``buffer`` (uint8, see tp_fp4_bytes) holds
    its codes, scales and header."""

    __slots__ = ("buffer", "rows", "cols", "format", "_code")

    def __init__(self, buffer: torch.Tensor, rows: int, cols: int, format: str):
        self.buffer, self.rows, self.cols = buffer, rows, cols
        self.format, self._code = format, _format(format)

    @property
    def shape(self):
        return (self.rows, self.cols)

    def dequantize(self, dtype=torch.bfloat16, out=None, stream=None):
        """The values, [rows, cols] (exact in bf16 too, but for values out of
        its range)."""
        return B_.tensor_calls().fp4_dequantize(
            self.buffer, self.rows, self.cols, self._code, _dtype(dtype), out,
            stream)

    def codes(self) -> torch.Tensor:
        """[rows, 128 ceil(cols / 256)] bytes of two codes, gathered out of their
        tiles and units."""
        rt, kt = (self.rows + 127) // 128, (self.cols + 255) // 256
        at = B_.tp_fp4_offset(self.rows, self.cols, self._code, B_.TPFP4_CODES)
        t = self.buffer[at:at + rt * kt * 16384].view(rt, kt, 16, 8, 8, 16)
        r = torch.arange(8, device=t.device)
        # [row tile, k tile, row / 8, row % 8, unit, byte]
        t = t[:, :, :, r[:, None], r[None, :] ^ r[:, None]]
        t = t.permute(0, 2, 3, 1, 4, 5)
        return t.reshape(rt * 128, kt * 128)[:self.rows]

    def scales(self) -> torch.Tensor:
        """The scale bytes [rows, blocks], gathered out of their tiles."""
        block = 16 if self.format == "nvfp4" else 32
        per = 256 // block
        rt, kt = (self.rows + 127) // 128, (self.cols + 255) // 256
        at = B_.tp_fp4_offset(self.rows, self.cols, self._code, B_.TPFP4_SCALES)
        t = self.buffer[at:at + rt * kt * 128 * per].view(rt, kt, per // 4, 32, 4, 4)
        # [row tile, k tile, block / 4, row % 32, row / 32, block % 4]
        t = t.permute(0, 4, 3, 1, 2, 5).reshape(rt * 128, kt * per)
        return t[:self.rows, :(self.cols + block - 1) // block]

    def tensor_scale(self) -> torch.Tensor:
        """g, a view of one fp32 value (a matrix of no rows has none)."""
        if self.rows == 0:
            raise ValueError("a packed matrix of no rows has no scale")
        return self.buffer[16:20].view(torch.float32)

    def check(self, stream=None) -> int:
        """Synchronise and return the status of the products that read this
        matrix as ``a`` (TPMLP_OK or an error)."""
        if self.rows == 0:   # (nothing was written)
            return B_.TPMLP_OK
        with torch.cuda.device(self.buffer.device):
            return B_.tp_fp4_check(self.buffer, stream)


def quantize(x, format: str = "nvfp4", scale: "float | Fp4Tensor | None" = None,
             transpose: bool = False, out: Fp4Tensor | None = None,
             stream=None) -> Fp4Tensor:
    """x [rows, cols] quantised along its rows, or with ``transpose`` along its
    columns as a packed [cols, rows].  ``scale``: nvfp4's power of two for the
    whole matrix (blocks with a largest |x| up to 6 * 2^-10 of it become zeros), a
    packed matrix whose own is taken (on the device), or by default
    the one x needs (x is then read twice); mxfp4 has none (None or 1).  ``out``: a
    packed matrix of that shape and format, which is overwritten."""
    code = _format(format)
    like = buffer = None
    if isinstance(scale, Fp4Tensor):
        if scale.format != format:
            raise ValueError(f"scale is in {scale.format}, not in {format}")
        if scale.rows == 0:   # (nothing was written)
            raise ValueError("scale is a packed matrix of no rows, which has none")
        scale, like = None, scale.buffer
    if out is not None:
        shape = (x.shape[1], x.shape[0]) if transpose else tuple(x.shape)
        if out.shape != shape or out.format != format:
            raise ValueError(f"out: expected a packed {shape} in {format}, got "
                             f"{out.shape} in {out.format}")
        buffer = out.buffer
    buffer = B_.tensor_calls().fp4_quantize(x, transpose, code, _scale(scale),
                                            like, buffer, stream)
    if out is not None:
        return out
    rows, cols = x.shape
    return (Fp4Tensor(buffer, cols, rows, format) if transpose
            else Fp4Tensor(buffer, rows, cols, format))


def quantize_both(x, format: str = "nvfp4", scale: float | None = None,
                  stream=None) -> "tuple[Fp4Tensor, Fp4Tensor]":
    """x [rows >= 1, cols] quantised along its rows, [rows, cols], and along its
    columns, [cols, rows], in one pass: quantize(x) and quantize(x, transpose=True),
    which share their g."""
    r, t = B_.tensor_calls().fp4_quantize_both(x, _format(format), _scale(scale),
                                               stream)
    rows, cols = x.shape
    return Fp4Tensor(r, rows, cols, format), Fp4Tensor(t, cols, rows, format)


def matmul(a: Fp4Tensor, b: Fp4Tensor, bias=None, dtype=torch.bfloat16, out=None,
           stream=None) -> torch.Tensor:
    """a [T, K] times the transpose of b [N, K], plus bias [N] (fp32): [T, N],
    summed in fp32 and rounded to ``dtype`` once."""
    if a.cols != b.cols or a.format != b.format:
        raise ValueError(f"a is {a.shape} in {a.format}, b {b.shape} in "
                         f"{b.format}: expected the same columns and format")
    return B_.tensor_calls().fp4_matmul(a.buffer, a.rows, b.buffer, b.rows, a.cols,
                                        a._code, bias, _dtype(dtype), out, stream)


class Fp4Linear:
    """y = x W + bias on four-bit operands: W [K, N] (bf16 or fp32) is packed
    once (both ways: the copy along N is the gradients'), x is quantised in every
    call.

    The gradients are products of quantised matrices too, each quantised along the
    sum it takes part in: dx = dy W^T along N, dW = x^T dy along the tokens (the
    quantisation itself is passed through as the identity)."""

    def __init__(self, W, bias=None, format: str = "nvfp4"):
        self.format, self._code = format, _format(format)
        self.inputs, self.outputs = W.shape
        self.bias = bias
        # [K, N], for dx, and [N, K]
        self.weight_rows, self.weight = quantize_both(W, format)
        self._status = torch.zeros(4, dtype=torch.int32, device=W.device)
        self._calls = B_.tensor_calls()

    def check(self, stream=None) -> int:
        """Synchronise and return the first error of the calls so far, then forget
        it (TPMLP_OK or an error)."""
        with torch.cuda.device(self._status.device):
            return B_.tp_fp4_check(self._status, stream)

    def forward(self, x, x_scale: float | None = 1.0, dtype=torch.bfloat16,
                out=None, stream=None) -> torch.Tensor:
        """x [T, K] -> [T, N].  ``x_scale``: nvfp4's power of two g for x, or None
        to take it from x (which is then read twice, and up to 8 rows are quantised in
        a launch of their own).  With the default of 1 a block of 16 whose largest |x|
        is at most 0.0059 becomes zeros, and below 0.094 its scale is coarse:
        activations that small want a smaller g, or None."""
        return self._calls.fp4_linear(
            x, self.weight.buffer, self.outputs, self.inputs, self._code,
            _scale(x_scale), self.bias, _dtype(dtype), out, self._status, stream)

    def backward(self, dy, x, x_scale: float | None = 1.0,
                 dy_scale: float | None = None, dtype=torch.bfloat16,
                 bias_grad: bool = True, stream=None) -> dict:
        """From dy [T, N] and forward's x (``x_scale`` as there; ``dy_scale`` is taken
        from dy by default): a dict with dx [T, K] (``dtype``), dw
        [K, N] (fp32) and, for a layer with a bias, db [N] (fp32), each new."""
        calls, code = self._calls, self._code
        if dy.dim() != 2 or x.dim() != 2 or dy.shape[0] != x.shape[0] or \
                dy.shape[1] != self.outputs or x.shape[1] != self.inputs:
            raise ValueError(f"expected dy [T, {self.outputs}] and x [T, "
                             f"{self.inputs}], got {tuple(dy.shape)} and "
                             f"{tuple(x.shape)}")
        bias_grad = bias_grad and self.bias is not None
        dx, dw, db = calls.fp4_backward(dy, x, self.weight_rows.buffer, code,
                                        _scale(dy_scale), _scale(x_scale),
                                        _dtype(dtype), bias_grad, self._status,
                                        stream)
        return {"dx": dx, "dw": dw, "db": db}
