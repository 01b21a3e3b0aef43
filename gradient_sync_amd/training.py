"""The optimizer step of a sharded update, and 4-bit block-scaled weights.

Between the ReduceScatter that leaves each rank its gradient shards and the
AllGather of the updated parameters stand the gradient's norm (GradNorm), the
update of the shards (AdamW, moments in fp32 or in 8 bits) and, where the weights
are gathered in 4 bits, their quantisation and product (dp_mxfp4_*). GradNorm and
AdamW marshal their pointer arrays once at construction; a step checks them and
enqueues its launches. AdamW's check for overlaps sorts the tensors' addresses (on
the host: 5 us for 64 tensors, 24 for 300, 0.25 ms for 1,000), so very long lists of
small tensors are better kept as views of a few buffers. The tensors must stay
where they are while the object is used.
"""
from __future__ import annotations

import contextlib
import ctypes
import struct

import torch

from . import _DTYPES, _check, _stream, lib, ptr_array

STATE_BLOCK = 128               # DP_STATE_BLOCK in include/dpsync.h
GRAD_NORM_WS_BYTES = 4160      # DP_GRAD_NORM_WS_BYTES
DP_ADAMW_STOCHASTIC = 1
_FLOATS = (torch.float32, torch.bfloat16)
_CODES = (torch.uint8, torch.float8_e4m3fn)


def _list(ts, what, dtypes, like=None):
    """A list of contiguous GPU tensors of one of `dtypes`, as long as `like` in each entry."""
    ts = list(ts)
    for i, t in enumerate(ts):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what}: expected torch tensors")
        if t.dtype not in dtypes or t.dtype != ts[0].dtype:
            raise TypeError(f"{what}: expected one of {dtypes} throughout, got {t.dtype}")
        if t.device.type != "cuda":
            raise ValueError(f"{what}: tensors must be on the GPU")
        if not t.is_contiguous():
            raise ValueError(f"{what}: tensors must be contiguous")
        if like is not None and (len(ts) != len(like) or t.numel() != like[i].numel()):
            raise ValueError(f"{what}: need one tensor per gradient, of its size")
    if like is not None and len(ts) != len(like):
        raise ValueError(f"{what}: need one tensor per gradient")
    return ts


def _counts(ts):
    return (ctypes.c_int64 * max(1, len(ts)))(*[t.numel() for t in ts])


def _pointers(ts):
    return ptr_array([t.data_ptr() for t in ts])


def _on(stream):
    """Allocations belong to the stream that uses them."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream)
                             else torch.cuda.ExternalStream(int(stream)))


# the current stream's handle without the object around it (2.8 us a call, a
# third of a small product's time)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _at(stream):
    """The handle of `stream`, or of the current stream."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return _stream(stream).value or 0


def _empty(like, shape, dtype, stream):
    """Uninitialised, on like's GPU, for use on `stream`."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with _on(stream):
        return like.new_empty(shape, dtype=dtype)


class StepCtrl:
    """dp_step_ctrl_t on the GPU: `norm` and `scale` (fp32), `step` and
    `skipped` (int32), 0-dimensional views of it."""

    def __init__(self, scale: float = 1.0, step: int = 0, device="cuda"):
        bits = struct.unpack("i", struct.pack("f", scale))[0]
        self.buf = torch.tensor([0, bits, step, 0], dtype=torch.int32).to(device)
        self.norm = self.buf[0].view(torch.float32)
        self.scale = self.buf[1].view(torch.float32)
        self.step = self.buf[2]
        self.skipped = self.buf[3]


class GradNorm:
    """Global 2-norm of a list of gradients and the factor that clips it
    (dp_grad_norm). `run` advances ctrl.step, or ctrl.skipped where the norm is
    not finite, and returns ctrl. It may run on any stream, one run at a time;
    one that runs on a stream that torch does not own is kept until the run has ended."""

    def __init__(self, grads, ctrl: StepCtrl | None = None):
        self._build(grads, ctrl)
        # a run on another stream than this one finds its workspace zeroed (a
        # stream that captures cannot wait; what it captures is in order)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self.workspace.device).synchronize()

    def _build(self, grads, ctrl):
        self.grads = _list(grads, "grads", _FLOATS)
        device = self.grads[0].device if self.grads else "cuda"
        self.ctrl = StepCtrl(device=device) if ctrl is None else ctrl
        self.workspace = torch.zeros(GRAD_NORM_WS_BYTES, dtype=torch.uint8, device=device)
        # streams that the memory of workspace and ctrl is known to be used on
        self._streams = {torch.cuda.current_stream(self.workspace.device).cuda_stream}
        self._args = (len(self.grads), _counts(self.grads), _pointers(self.grads),
                      _DTYPES[self.grads[0].dtype] if self.grads else 0)

    def run(self, max_norm: float = 0.0, stream=None) -> StepCtrl:
        at = _at(stream)
        if at not in self._streams:
            self._streams.add(at)
            self._use_on(stream)
        _check(lib().dp_grad_norm(*self._args, float(max_norm), self.ctrl.buf.data_ptr(),
                                  self.workspace.data_ptr(), at), "dp_grad_norm")
        return self.ctrl

    def _use_on(self, stream):
        """The object may be dropped while a run is on its way: its memory is kept for that stream. Not for one
        that torch does not own (its id is the handle), which may be gone before the object is."""
        s = torch.cuda.current_stream() if stream is None else stream
        if isinstance(s, torch.cuda.Stream) and (s.cuda_stream == 0 or s.stream_id != s.cuda_stream):
            self.workspace.record_stream(s)
            self.ctrl.buf.record_stream(s)


class AdamWOpts(ctypes.Structure):
    """dp_adamw_opts_t"""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("step", ctypes.c_int64), ("seed", ctypes.c_uint64), ("flags", ctypes.c_int),
                ("reserved", ctypes.c_int)]


class AdamW:
    """AdamW over many tensors at once (dp_adamw; with `scales`, dp_adamw8).

    params, grads  : fp32 or bf16 tensors; params are updated in place
    m, v           : fp32, or with scales 8-bit codes (uint8 or float8_e4m3fn)
    scales         : per tensor ceil(n / 128) x 2 fp32, see dp_adamw8
    copies         : bf16 copies of fp32 params, written by every step
    seed           : rounds 8-bit states at random (None: to nearest)
    """

    def __init__(self, params, grads, m, v, copies=None, scales=None, lr: float = 1e-3,
                 betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
                 seed: int | None = None):
        g = _list(grads, "grads", _FLOATS)
        p = _list(params, "params", _FLOATS, g)
        state = (torch.float32,) if scales is None else _CODES
        m, v = _list(m, "m", state, g), _list(v, "v", state, g)
        if scales is not None:
            scales = _list(scales, "scales", (torch.float32,))
            if len(scales) != len(g) or any(s.numel() != 2 * -(-t.numel() // STATE_BLOCK)
                                            for s, t in zip(scales, g)):
                raise ValueError("scales: need ceil(n / 128) x 2 values per tensor")
        elif seed is not None:
            raise ValueError("seed: only 8-bit states are rounded at random")
        if copies is not None:
            copies = _list(copies, "copies", (torch.bfloat16,), g)
            if p and p[0].dtype != torch.float32:
                raise TypeError("copies: only of float32 params")
        self.tensors = (p, g, m, v, copies, scales)          # keep them alive
        self.opts = AdamWOpts(lr, betas[0], betas[1], eps, weight_decay, 0,
                              (0 if seed is None else seed) & ((1 << 64) - 1),
                              DP_ADAMW_STOCHASTIC if seed is not None else 0, 0)
        dt = lambda ts: _DTYPES[ts[0].dtype] if ts else 0
        self._args = [len(g), _counts(g), _pointers(p), dt(p), _pointers(g), dt(g), _pointers(m),
                      _pointers(v)]
        if scales is not None:
            self._args.append(_pointers(scales))
        self._args.append(None if copies is None else _pointers(copies))
        self._name = "dp_adamw" if scales is None else "dp_adamw8"

    @staticmethod
    def new_state(params, bits: int = 32):
        """(m, v, scales) of zeros for `params`; scales is None with 32 bits."""
        if bits == 32:
            zeros = lambda: [torch.zeros(p.numel(), device=p.device) for p in params]
            return zeros(), zeros(), None
        if bits != 8:
            raise ValueError("bits must be 32 or 8")
        zeros = lambda: [torch.zeros(p.numel(), dtype=torch.uint8, device=p.device) for p in params]
        return zeros(), zeros(), [torch.zeros(-(-p.numel() // STATE_BLOCK), 2, device=p.device)
                                  for p in params]

    def step(self, step: int = 0, ctrl: StepCtrl | None = None, lr: float | None = None,
             stream=None):
        """One update. step: its number (from 1); 0 takes it from ctrl, which
        also gives the clip factor. lr: for this step and those after it."""
        self.opts.step = step
        if lr is not None:
            self.opts.lr = lr
        _check(getattr(lib(), self._name)(*self._args, ctypes.byref(self.opts),
                                          None if ctrl is None else ctrl.buf.data_ptr(),
                                          _at(stream)), self._name)


def dp_grad_norm(grads, ctrl: StepCtrl | None = None, max_norm: float = 0.0, stream=None) -> StepCtrl:
    """GradNorm(grads, ctrl).run(max_norm), for a list that is used once."""
    norm = GradNorm.__new__(GradNorm)
    with _on(stream):                # the stream of its only run: nothing to wait for
        norm._build(grads, ctrl)
    return norm.run(max_norm, stream)


def dp_adamw(params, grads, m, v, step: int = 0, ctrl: StepCtrl | None = None, stream=None, **kw):
    """AdamW(params, grads, m, v, **kw).step(step, ctrl), for lists that are used once."""
    AdamW(params, grads, m, v, **kw).step(step, ctrl, stream=stream)


class Mxfp4:
    """A quantised [rows, cols] matrix: `codes` (rows x 64 ceil(cols / 128)
    bytes) and `scales` (ceil(rows / 16) x ceil(cols / 512) x 256 bytes)."""

    def __init__(self, rows: int, cols: int, codes: torch.Tensor | None = None,
                 scales: torch.Tensor | None = None, device="cuda"):
        self.rows, self.cols = rows, cols
        shapes = ((rows, -(-cols // 128) * 64), (-(-rows // 16), -(-cols // 512), 256))
        if codes is None:
            codes = torch.empty(shapes[0], dtype=torch.uint8, device=device)
        if scales is None:
            scales = torch.empty(shapes[1], dtype=torch.uint8, device=device)
        for t in (codes, scales):
            if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous():
                raise ValueError("Mxfp4: codes and scales must be contiguous uint8 GPU tensors")
        self.codes, self.scales = codes.view(shapes[0]), scales.view(shapes[1])

    @classmethod
    def _for(cls, rows: int, cols: int, x: torch.Tensor, stream):
        """Uninitialised, on x's GPU, for use on `stream`."""
        q = cls.__new__(cls)
        q.rows, q.cols = rows, cols
        q.codes = _empty(x, (rows, -(-cols // 128) * 64), torch.uint8, stream)
        q.scales = _empty(x, (-(-rows // 16), -(-cols // 512), 256), torch.uint8, stream)
        return q


def _matrix(t, what):
    """(rows, columns, row stride) of a GPU matrix whose rows are contiguous."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _FLOATS:
        raise TypeError(f"{what}: expected a float32 or bfloat16 tensor")
    if not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{what}: expected a GPU matrix with contiguous rows")
    (rows, cols), (ld, step) = t.shape, t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{what}: expected a GPU matrix with contiguous rows")
    # the row stride of a single row is free
    return rows, cols, ld if rows > 1 else max(cols, 1)


def _output(t, shape, dtype, like, stream, what):
    if t is None:
        if dtype not in _FLOATS:
            raise TypeError(f"{what}: dtype must be float32 or bfloat16")
        return _empty(like, shape, dtype, stream)
    if t.dtype not in _FLOATS or not t.is_cuda or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous float32 or bfloat16 GPU tensor of shape {shape}")
    return t


def dp_mxfp4_quantize(x, transposed: str = "no", out: Mxfp4 | None = None,
                      out_t: Mxfp4 | None = None, stream=None):
    """x [rows, cols] in blocks of 32 along its rows ("no"), its transpose in
    blocks along its columns ("only"), or the pair of both from one read ("also")."""
    if transposed not in ("no", "also", "only"):
        raise ValueError("transposed must be 'no', 'also' or 'only'")
    rows, cols, ld = _matrix(x, "x")
    ptrs = [None] * 4
    if transposed == "only":
        out = None
    else:
        if out is None:
            out = Mxfp4._for(rows, cols, x, stream)
        elif (out.rows, out.cols) != (rows, cols):
            raise ValueError("dp_mxfp4_quantize: out has another shape than x")
        ptrs[:2] = out.codes.data_ptr(), out.scales.data_ptr()
    if transposed == "no":
        out_t = None
    else:
        if out_t is None:
            out_t = Mxfp4._for(cols, rows, x, stream)
        elif (out_t.rows, out_t.cols) != (cols, rows):
            raise ValueError("dp_mxfp4_quantize: out_t has another shape than x's transpose")
        ptrs[2:] = out_t.codes.data_ptr(), out_t.scales.data_ptr()
    _check(lib().dp_mxfp4_quantize(x.data_ptr(), rows, cols, ld, _DTYPES[x.dtype], *ptrs,
                                   _at(stream)), "dp_mxfp4_quantize")
    return (out, out_t) if transposed == "also" else out if out is not None else out_t


def dp_mxfp4_dequantize(q: Mxfp4, out=None, dtype=torch.bfloat16, stream=None):
    """The values `q` stands for (exact)."""
    out = _output(out, (q.rows, q.cols), dtype, q.codes, stream, "out")
    _check(lib().dp_mxfp4_dequantize(q.codes.data_ptr(), q.scales.data_ptr(), q.rows, q.cols,
                                     out.data_ptr(), q.cols, _DTYPES[out.dtype], _at(stream)),
           "dp_mxfp4_dequantize")
    return out


def dp_gemm_mxfp4(a: Mxfp4, b: Mxfp4, out=None, dtype=torch.bfloat16, accumulate: bool = False,
                  stream=None):
    """a [m, k] times b [n, k] transposed, fp32 sums; accumulate adds to a
    float32 `out`."""
    if a.cols != b.cols:
        raise ValueError("dp_gemm_mxfp4: a and b must be quantised along the same length")
    if accumulate and out is None:
        raise ValueError("dp_gemm_mxfp4: accumulate needs out")
    out = _output(out, (a.rows, b.rows), dtype, a.codes, stream, "out")
    _check(lib().dp_gemm_mxfp4(a.codes.data_ptr(), a.scales.data_ptr(), b.codes.data_ptr(),
                               b.scales.data_ptr(), out.data_ptr(), a.rows, b.rows, a.cols,
                               _DTYPES[out.dtype], 1 if accumulate else 0, _at(stream)),
           "dp_gemm_mxfp4")
    return out


def dp_mxfp4_linear(x, w: Mxfp4, out=None, dtype=torch.bfloat16, stream=None):
    """x [m, k], quantised on the way, times w [n, k] transposed."""
    m, k, ldx = _matrix(x, "x")
    if k != w.cols:
        raise ValueError("dp_mxfp4_linear: x and w differ in length")
    out = _output(out, (m, w.rows), dtype, x, stream, "out")
    need = lib().dp_mxfp4_linear_ws_bytes(m, w.rows, k)
    ws = _empty(x, (need,), torch.uint8, stream) if need else None
    _check(lib().dp_mxfp4_linear(x.data_ptr(), ldx, _DTYPES[x.dtype], w.codes.data_ptr(),
                                 w.scales.data_ptr(), out.data_ptr(), m, w.rows, k,
                                 _DTYPES[out.dtype], ws.data_ptr() if need else None,
                                 _at(stream)), "dp_mxfp4_linear")
    return out
