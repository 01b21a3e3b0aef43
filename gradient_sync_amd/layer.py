"""What stands in front of a weight that is gathered in 4 bits: the norm with the
residual's addition and its gradients, activations and gradients in 8 bits, their
product with 4-bit and 8-bit operands, and the product of a few rows kept as they are.

One layer, forward and backward:

    n = dp_rms_norm(x, gamma, residual=r, dtype=torch.bfloat16, quantize=True, save=True)
    z = dp_gemm_mxfp8(n.q, w)                              # w: Mxfp4
    dz8, dz8t = dp_mxfp8_quantize(dz, transposed="also")
    dy = dp_gemm_mxfp8(dz8, wt)                            # wt: w's transpose, Mxfp4
    dw = dp_gemm_mxfp8(dz8t, dp_mxfp8_quantize(n.y, transposed="only"))
    dx, dgamma = dp_rms_norm_backward(dy, n.hidden, gamma, n.rstd, dresidual=dr)

The forward product takes the norm's output in 8 bits from fp32, and dw from n.y, which was rounded to its type
before (bfloat16 here; dtype=torch.float32 leaves that rounding out).
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _DTYPES, _check, lib
from .training import _FLOATS, Mxfp4, _at, _empty, _matrix, _output


def _here(*ts):
    """Every tensor is on the current GPU, whose streams the calls use."""
    here = torch.cuda.current_device()
    for t in ts:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"expected a tensor, got a {type(t).__name__}")
        if t.get_device() != here:
            raise ValueError(f"expected tensors on the current GPU {here}, got one on {t.device}")


class Mxfp8:
    """A quantised [rows, cols] matrix: `codes` (rows x 128 ceil(cols / 128)
    bytes) and `scales` (ceil(rows / 16) x ceil(cols / 512) x 256 bytes)."""

    __slots__ = ("rows", "cols", "_buf", "_codes", "_scales")

    def __init__(self, rows: int, cols: int, codes: torch.Tensor | None = None,
                 scales: torch.Tensor | None = None, device="cuda"):
        self.rows, self.cols, self._buf = rows, cols, None
        shapes = self._shapes()
        if codes is None:
            codes = torch.empty(shapes[0], dtype=torch.uint8, device=device)
        if scales is None:
            scales = torch.empty(shapes[1], dtype=torch.uint8, device=device)
        for t in (codes, scales):
            if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous():
                raise ValueError("Mxfp8: codes and scales must be contiguous uint8 GPU tensors")
        if codes.device != scales.device:
            raise ValueError("Mxfp8: codes and scales must be on one GPU")
        self._codes, self._scales = codes.view(shapes[0]), scales.view(shapes[1])

    @classmethod
    def _for(cls, rows: int, cols: int, x: torch.Tensor, stream):
        """Uninitialised, on x's GPU, for use on `stream`: codes and scales of one allocation, as
        tensors only when they are asked for (an allocation costs 2 us, a view 1)."""
        q = cls.__new__(cls)
        q.rows, q.cols = rows, cols
        q._buf = _empty(x, (q._code_bytes() + -(-rows // 16) * -(-cols // 512) * 256,), torch.uint8, stream)
        q._codes = q._scales = None
        return q

    def _code_bytes(self) -> int:
        return self.rows * (-(-self.cols // 128) * 128)

    def _shapes(self):
        return ((self.rows, -(-self.cols // 128) * 128), (-(-self.rows // 16), -(-self.cols // 512), 256))

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            self._codes = self._buf[:self._code_bytes()].view(self._shapes()[0])
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            self._scales = self._buf[self._code_bytes():].view(self._shapes()[1])
        return self._scales

    def _any(self) -> torch.Tensor:
        """A tensor that lies where the matrix does."""
        return self._codes if self._buf is None else self._buf

    def _ptrs(self):
        """Addresses of codes and scales."""
        if self._buf is None:
            return self._codes.data_ptr(), self._scales.data_ptr()
        at = self._buf.data_ptr()
        return at, at + self._code_bytes()


def _quantized(q, rows, cols, like, stream, what):
    """`q` checked, or a new one."""
    if q is None:
        return Mxfp8._for(rows, cols, like, stream)
    if not isinstance(q, Mxfp8):
        raise TypeError(f"{what}: expected an Mxfp8")
    if (q.rows, q.cols) != (rows, cols):
        raise ValueError(f"{what}: expected an Mxfp8 of shape {(rows, cols)}")
    return q


def dp_mxfp8_quantize(x, transposed: str = "no", out: Mxfp8 | None = None,
                      out_t: Mxfp8 | None = None, stream=None):
    """x [rows, cols] in blocks of 32 along its rows ("no"), its transpose in
    blocks along its columns ("only"), or the pair of both from one read ("also")."""
    if transposed not in ("no", "also", "only"):
        raise ValueError("transposed must be 'no', 'also' or 'only'")
    rows, cols, ld = _matrix(x, "x")
    ptrs = [None] * 4
    if transposed == "only":
        out = None
    else:
        out = _quantized(out, rows, cols, x, stream, "out")
        ptrs[:2] = out._ptrs()
    if transposed == "no":
        out_t = None
    else:
        out_t = _quantized(out_t, cols, rows, x, stream, "out_t")
        ptrs[2:] = out_t._ptrs()
    _here(x, *(q._any() for q in (out, out_t) if q is not None))
    _check(lib().dp_mxfp8_quantize(x.data_ptr(), rows, cols, ld, _DTYPES[x.dtype], *ptrs,
                                   _at(stream)), "dp_mxfp8_quantize")
    return (out, out_t) if transposed == "also" else out if out is not None else out_t


def dp_mxfp8_dequantize(q: Mxfp8, out=None, dtype=torch.bfloat16, stream=None):
    """The values `q` stands for: exact, but for what lies below bfloat16's smallest subnormal, and 2^128 (held for
    finite values from 1.9375 * 2^127 on), which becomes an infinity."""
    if not isinstance(q, Mxfp8):
        raise TypeError("dp_mxfp8_dequantize: expected an Mxfp8")
    out = _output(out, (q.rows, q.cols), dtype, q._any(), stream, "out")
    _here(q._any(), out)
    _check(lib().dp_mxfp8_dequantize(*q._ptrs(), q.rows, q.cols, out.data_ptr(), q.cols, _DTYPES[out.dtype], _at(stream)),
           "dp_mxfp8_dequantize")
    return out


def dp_gemm_mxfp8(a: Mxfp8, b, out=None, dtype=torch.bfloat16, accumulate: bool = False,
                  stream=None):
    """a [m, k] in 8 bits times b [n, k] (Mxfp4 or Mxfp8) transposed; accumulate adds to a float32 `out`.

    Sums are kept in fp32, but within each 8 consecutive k the products are first cut to multiples of 2^-13 of the
    largest one's power of two: on normal values a float32 output is off by 5e-6 of its size with b in 4 bits and by
    1.5e-5 in 8, where fp32 products and sums leave 3e-8 and 8e-8."""
    if not isinstance(a, Mxfp8) or not isinstance(b, (Mxfp4, Mxfp8)):
        raise TypeError("dp_gemm_mxfp8: a must be an Mxfp8, b an Mxfp4 or an Mxfp8")
    if a.cols != b.cols:
        raise ValueError("dp_gemm_mxfp8: a and b must be quantised along the same length")
    if accumulate and out is None:
        raise ValueError("dp_gemm_mxfp8: accumulate needs out")
    out = _output(out, (a.rows, b.rows), dtype, a._any(), stream, "out")
    eight = isinstance(b, Mxfp8)
    _here(a._any(), *((b._any(),) if eight else (b.codes, b.scales)), out)
    at = b._ptrs() if eight else (b.codes.data_ptr(), b.scales.data_ptr())
    _check(lib().dp_gemm_mxfp8(*a._ptrs(), *at, 8 if eight else 4, out.data_ptr(), a.rows, b.rows, a.cols, _DTYPES[out.dtype],
                               1 if accumulate else 0, _at(stream)), "dp_gemm_mxfp8")
    return out


def dp_mxfp4_matvec(x, w: Mxfp4, out=None, dtype=torch.bfloat16, stream=None):
    """x [m, k], m <= 64 and not rounded, times w [n, k] transposed, fp32 sums."""
    m, k, ldx = _matrix(x, "x")
    if not isinstance(w, Mxfp4):
        raise TypeError("dp_mxfp4_matvec: w must be an Mxfp4")
    if k != w.cols:
        raise ValueError("dp_mxfp4_matvec: x and w differ in length")
    out = _output(out, (m, w.rows), dtype, x, stream, "out")
    _here(x, w.codes, w.scales, out)
    _check(lib().dp_mxfp4_matvec(x.data_ptr(), ldx, _DTYPES[x.dtype], w.codes.data_ptr(),
                                 w.scales.data_ptr(), out.data_ptr(), m, w.rows, k,
                                 _DTYPES[out.dtype], _at(stream)), "dp_mxfp4_matvec")
    return out


class RmsNorm(NamedTuple):
    """What dp_rms_norm computes: `y` and `q` (the output, plain and in 8 bits),
    `hidden` (x + residual) and `rstd`, each None where it was not asked for."""
    y: torch.Tensor | None
    q: Mxfp8 | None
    hidden: torch.Tensor
    rstd: torch.Tensor | None


def _like(t, x, rows, cols, what):
    """The row stride of a matrix of x's shape and type."""
    if not isinstance(t, torch.Tensor) or t.dtype != x.dtype:
        raise TypeError(f"{what}: expected a tensor of x's type")
    r, c, ld = _matrix(t, what)
    if (r, c) != (rows, cols):
        raise ValueError(f"{what}: expected x's shape")
    return ld


def _vector(t, n, dtypes, what):
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise TypeError(f"{what}: expected one of {dtypes}")
    if not t.is_cuda or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous GPU tensor of {n} elements")


def dp_rms_norm(x, weight, residual=None, eps: float = 1e-6, dtype=None, quantize: bool = False,
                save: bool = False, out=None, out_q: Mxfp8 | None = None, hidden=None, rstd=None,
                stream=None) -> RmsNorm:
    """The norm of each row of x + residual, times weight.

    dtype    : of the plain output (None: x's, or no plain output with quantize)
    quantize : the output in 8 bits, for dp_gemm_mxfp8
    save     : rstd too, for dp_rms_norm_backward
    out, out_q, hidden, rstd : where they go; hidden may be x or residual itself
    """
    rows, cols, ldx = _matrix(x, "x")
    _vector(weight, cols, _FLOATS, "weight")
    _here(x, weight, residual, hidden, out, rstd)
    ldr = ldh = 0
    if residual is not None:
        ldr = _like(residual, x, rows, cols, "residual")
        if hidden is None:
            hidden, ldh = _empty(x, (rows, cols), x.dtype, stream), cols
        else:
            ldh = _like(hidden, x, rows, cols, "hidden")
    elif hidden is not None:
        raise ValueError("hidden: without a residual it is x")
    y = q = None
    if out is not None or dtype is not None or not (quantize or out_q is not None):
        y = _output(out, (rows, cols), x.dtype if dtype is None else dtype, x, stream, "out")
    if quantize or out_q is not None:
        q = _quantized(out_q, rows, cols, x, stream, "out_q")
        if out_q is not None:
            _here(q._any())
    if rstd is not None:
        _vector(rstd, rows, (torch.float32,), "rstd")
    elif save:
        rstd = _empty(x, (rows,), torch.float32, stream)
    ptr = lambda t: None if t is None else t.data_ptr()
    _check(lib().dp_rms_norm(x.data_ptr(), ldx, ptr(residual), ldr, _DTYPES[x.dtype], rows, cols,
                             weight.data_ptr(), _DTYPES[weight.dtype], eps, ptr(hidden), ldh,
                             ptr(y), 0 if y is None else _DTYPES[y.dtype],
                             *((None, None) if q is None else q._ptrs()), ptr(rstd), _at(stream)),
           "dp_rms_norm")
    return RmsNorm(y, q, x if hidden is None else hidden, rstd)


def dp_rms_norm_backward(dy, hidden, weight, rstd, dresidual=None, out=None, dweight=None,
                         weight_grad: bool = True, accumulate: bool = False, stream=None):
    """(dx, dweight) of dp_rms_norm's output gradient dy; dx is the gradient of x and
    of residual alike, with dresidual (what reaches hidden from elsewhere) added.

    out, dweight : where they go; out may be dy, hidden or dresidual itself
    weight_grad  : False leaves dweight out
    accumulate   : adds to the given dweight
    """
    rows, cols, ldh = _matrix(hidden, "hidden")
    r, c, lddy = _matrix(dy, "dy")
    if (r, c) != (rows, cols):
        raise ValueError("dy: expected hidden's shape")
    _vector(weight, cols, _FLOATS, "weight")
    _vector(rstd, rows, (torch.float32,), "rstd")
    lddr = 0 if dresidual is None else _like(dresidual, hidden, rows, cols, "dresidual")
    _here(hidden, dy, weight, rstd, dresidual, out, dweight)
    if out is None:
        out, lddx = _empty(hidden, (rows, cols), hidden.dtype, stream), cols
    else:
        lddx = _like(out, hidden, rows, cols, "out")
    if not weight_grad:
        if dweight is not None or accumulate:
            raise ValueError("dweight: not computed without weight_grad")
    elif dweight is not None:
        _vector(dweight, cols, (torch.float32,), "dweight")
    elif accumulate:
        raise ValueError("accumulate needs dweight")
    else:
        dweight = _empty(hidden, (cols,), torch.float32, stream)
    need = lib().dp_rms_norm_backward_ws_bytes(rows, cols, 1 if weight_grad else 0)
    ws = _empty(hidden, (need,), torch.uint8, stream) if need else None
    _check(lib().dp_rms_norm_backward(dy.data_ptr(), lddy, _DTYPES[dy.dtype], hidden.data_ptr(), ldh,
                                      None if dresidual is None else dresidual.data_ptr(), lddr,
                                      _DTYPES[hidden.dtype], rows, cols, weight.data_ptr(),
                                      _DTYPES[weight.dtype], rstd.data_ptr(), out.data_ptr(), lddx,
                                      dweight.data_ptr() if weight_grad else None,
                                      1 if accumulate else 0, ws.data_ptr() if need else None,
                                      _at(stream)), "dp_rms_norm_backward")
    return out, dweight
