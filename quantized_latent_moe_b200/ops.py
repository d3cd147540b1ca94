"""Binding of the calls in include/elq_ops.h: the 8-bit-integer expert path (rows
to codes, products of codes, products grouped by expert) and the norms around a
block.

Argument marshalling only, as in ``elq``, but through a compiled module (``_ops.so``,
csrc_ops/ops_binding.cpp), because the host's time bounds the small calls.  Every
function checks what the C entry cannot see (devices, dtypes, shapes, strides),
allocates its outputs, and makes one C call, raising ``elq.ElqError`` where that
refuses.  Nothing is copied or cast on the way: a tensor whose rows are not
contiguous, whose first row is not on a 16-byte boundary (h[1:] of odd width, say), or
whose rows are not whole multiples of 16 bytes apart where the call needs it, is
refused.  There is no fallback; a missing library raises.

The calls infer only: outputs have no autograd graph, whatever their inputs require.
An ``out`` counts as written in place (its version goes up), so that a backward pass
that had saved it says so instead of using it.

``stream`` is a ``torch.cuda.Stream`` (the current one by default); outputs are
allocated on it, and inputs recorded on it, so that their memory is not given out
again while it is read (that they are ready is the caller's to see to).  Calls run on the device of their tensors, whatever the current
device is.  ``lib()`` gives the C entries themselves, for callers that hold addresses.
"""
from __future__ import annotations

import ctypes

import torch

from . import elq
from .elq import I32, I64, V, ElqError

F16, I8 = 1, 24         # type ids beside elq's
F = ctypes.c_float


class ResidualC(ctypes.Structure):
    _fields_ = [("T", I64), ("cols", I32), ("h_type", I32), ("y_type", I32), ("n_type", I32),
                ("h", V), ("y", V), ("post_weight", V), ("gate", V), ("next_weight", V),
                ("h_out", V), ("n", V), ("scale", V),
                ("ldh", I64), ("ldy", I64), ("ld_out", I64), ("ldn", I64),
                ("gate_rows", I64), ("gate_ld", I64), ("gate_cols", I32), ("res_scale", F), ("eps", F)]


SIGNATURES = {
    "elq_quantize_i8": (I32, [V, I32, I64, I32, I64, V, I32, I64, V, I64, V, V]),
    "elq_swiglu_i8": (I32, [V, I32, I64, I32, I64, V, I64, V, V]),
    "elq_combine_i8": (I32, [V, I32, I64, I32, I64, V, V, I64, I32, V, I64, V, V]),
    "elq_i8_matmul": (I32, [V, I64, V, I64, V, I64, V, V, I32, I32, V, I32, I64, V]),
    "elq_grouped_matmul": (I32, [V, I32, I64, V, I64, V, I64, I64, V, I32, I32, I32, V, V, I32, I64, V]),
    "elq_rms_norm": (I32, [V, I32, I64, I32, I64, V, F, V, I32, I64, V, V]),
    "elq_residual_norm": (I32, [ctypes.POINTER(ResidualC), V]),
    "elq_ops_status": (I32, [V]),
    "elq_test_i8_matmul_timeout": (I32, [V, I64, V, I64, V, I64, V, I32, I32, V, I64, I32, ctypes.c_uint64, V]),
}

_L = None


def lib() -> ctypes.CDLL:
    global _L
    if _L is None:
        L = elq.lib()
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _L = L
    return _L


class I8Rows:
    """Rows as 8-bit codes ``q`` (int8 [..., rows, cols], rows a multiple of 16
    bytes apart) with one fp32 ``scale`` [..., rows] each: row r stands for
    q[r] * scale[r].  Activations have one row a token, weights one a channel,
    expert weights [E, N, K] one a channel of each expert.

    Rows that a call here made lie in one buffer, the codes, then the scales; q
    and scale are views of it, made when asked for."""

    __slots__ = ("_q", "_scale", "_buf", "_cols")

    def __init__(self, q: torch.Tensor, scale: torch.Tensor):
        self._q, self._scale, self._buf = q, scale, None

    def _layout(self):
        """Rows, and bytes between them, in the buffer."""
        ld = (self._cols + 15) // 16 * 16
        return self._buf.numel() // (ld + 4), ld

    @property
    def q(self) -> torch.Tensor:
        if self._q is None:
            rows, ld = self._layout()
            self._q = self._buf.as_strided((rows, self._cols), (ld, 1))
        return self._q

    @property
    def scale(self) -> torch.Tensor:
        if self._scale is None:
            rows, ld = self._layout()
            self._scale = self._buf[rows * ld:].view(torch.float32)
        return self._scale

    @property
    def shape(self):
        return self.q.shape

    def dequantize(self, dtype=torch.float32) -> torch.Tensor:
        return (self.q.to(torch.float32) * self.scale.unsqueeze(-1)).to(dtype)


_N = None


def _native():
    """The compiled binding, loaded at the first call."""
    global _N
    if _N is None:
        lib()                   # raises if the library is not built
        try:
            from . import _ops
        except ImportError as e:
            raise RuntimeError("_ops.so is not built or does not load (%s); run `python -m quantized_latent_moe_b200.build`"
                               % e) from e
        _ops.bind(I8Rows, ElqError, torch.OutOfMemoryError)
        _N = _ops
    return _N


def _on(stream, x, call, *args, **kw):
    """The call on `stream`, of x's device."""
    t = x if isinstance(x, torch.Tensor) else x._buf if x._buf is not None else x._q
    if stream.device != t.device:
        raise ElqError(-1, "stream: of another device")
    with torch.cuda.stream(stream):
        out = call(x, *args, **kw)
    for a in (x, *args, *kw.values()):
        for t in (a._q, a._scale, a._buf) if isinstance(a, I8Rows) else (a,):
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
    return out


# ---- rows to codes --------------------------------------------------------------

def quantize_i8(x: torch.Tensor, index: torch.Tensor | None = None, index_div: int = 1, stream=None) -> I8Rows:
    """Codes of the rows of x [rows, K] (fp32, bf16, fp16), or of the gathered
    rows index[i] // index_div (int32 [n]; elq.route_bucket's pair order with
    index_div = k).  A contiguous expert stack [E, N, K] is quantised row by row."""
    if stream is not None:
        return _on(stream, x, quantize_i8, index, index_div)
    if index is None and isinstance(x, torch.Tensor) and x.dim() == 3 and x.is_contiguous():
        E, N, K = x.shape
        r = (_N or _native()).quantize_i8(x.view(E * N, K), None, 1)
        ld = r._layout()[1]
        return I8Rows(r._buf.as_strided((E, N, K), (N * ld, ld, 1)), r.scale.view(E, N))
    return (_N or _native()).quantize_i8(x, index, index_div)


def swiglu_i8(gu: torch.Tensor, stream=None) -> I8Rows:
    """Codes of silu(gate) * up for gu [rows, 2 I] = [gate | up]."""
    if stream is not None:
        return _on(stream, gu, swiglu_i8)
    return (_N or _native()).swiglu_i8(gu)


def combine_i8(o: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor, stream=None) -> I8Rows:
    """Codes of sum_j weights[t, j] * o[pos[t, j]]: o [rows, L], weights fp32
    [T, k], pos int32 of T * k row numbers (elq.route_bucket's pos)."""
    if stream is not None:
        return _on(stream, o, combine_i8, pos, weights)
    return (_N or _native()).combine_i8(o, pos, weights)


# ---- products -------------------------------------------------------------------

def i8_matmul(x: I8Rows, w: I8Rows, bias: torch.Tensor | None = None, out_dtype=torch.float32,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [T, N] = x [T, K] times w [N, K] transposed, from their codes, plus bias
    (fp32 [N])."""
    if stream is not None:
        return _on(stream, x, i8_matmul, w, bias, out_dtype, out)
    return (_N or _native()).i8_matmul(x, w, bias, out_dtype, out)


def grouped_matmul(x, w, offsets: torch.Tensor, out_dtype=None, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """y [M, N]: rows offsets[e] .. offsets[e+1]-1 of x [M, K] times expert e's
    matrix w[e] [N, K] transposed.  x and w both I8Rows, or both bf16 or fp16;
    offsets int32 [E+1].  out_dtype: for codes any of fp32 (default), bf16, fp16;
    for 16-bit x fp32 or its own (default).  Rows outside every group stay as out
    has them (undefined without out)."""
    if stream is not None:
        return _on(stream, x, grouped_matmul, w, offsets, out_dtype, out)
    if isinstance(w, I8Rows) and w._q is None:
        w.q, w.scale            # views of rows made here (one expert as a 2-D matrix is refused below)
    return (_N or _native()).grouped_matmul(x, w, offsets, out_dtype, out)


# ---- norms ----------------------------------------------------------------------

def rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6, out_dtype=None,
             out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x / sqrt(mean(x^2) + eps) * weight, row by row, in x's dtype or out_dtype;
    out may be x."""
    if stream is not None:
        return _on(stream, x, rms_norm, weight, eps, out_dtype, out)
    return (_N or _native()).rms_norm(x, weight, eps, out_dtype, out, False)


def rms_norm_i8(x: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6, stream=None) -> I8Rows:
    """rms_norm handed straight to the row quantiser (the fp32 norm, unrounded)."""
    if stream is not None:
        return _on(stream, x, rms_norm_i8, weight, eps)
    return (_N or _native()).rms_norm(x, weight, eps, None, None, True)


def residual_norm(h: torch.Tensor, y: torch.Tensor, post_weight: torch.Tensor | None = None, *,
                  gate: torch.Tensor | None = None, gate_rows: int | None = None, res_scale: float = 1.0,
                  next_weight: torch.Tensor | None = None, next_dtype=None, eps: float = 1e-6,
                  out: torch.Tensor | None = None, stream=None):
    """(h', n): h' = res_scale * h + gate * (rms(y) * post_weight) in h's dtype,
    and n = rms(h') * next_weight of the unrounded h' in next_dtype (None: n is
    None; torch.int8: I8Rows).

    gate: fp32 [C] (a value a channel), [G, C], or [G, 1] (a value a row); row t
    takes gate row t // gate_rows, by default T for G = 1 and 1 for G = T.  out: h'
    (h itself for in-place)."""
    if stream is not None:
        return _on(stream, h, residual_norm, y, post_weight, gate=gate, gate_rows=gate_rows, res_scale=res_scale,
                   next_weight=next_weight, next_dtype=next_dtype, eps=eps, out=out)
    return (_N or _native()).residual_norm(h, y, post_weight, gate, gate_rows, res_scale, next_weight, next_dtype, eps, out)


def status(device=None, stream=None) -> int:
    """Blocking: whether a product's bounded device wait ran out since the last
    call (0, or the timeout status), on the device of ``stream``, or on ``device``
    (by default the current one, its current stream)."""
    if stream is not None:
        if device is not None and torch.cuda.device(device).idx != stream.device.index:
            raise ElqError(-1, "status: stream of another device")
        device = stream.device
    with torch.cuda.device(device):
        s = torch.cuda.current_stream() if stream is None else stream
        return int(lib().elq_ops_status(s.cuda_stream))
