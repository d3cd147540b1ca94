"""ctypes binding of the calls in include/elq_ops.h: the 8-bit-integer expert
path (rows to codes, products of codes, products grouped by expert) and the
norms around a block.

As in ``elq``: argument marshalling only.  Every function checks what the C
entry cannot see (devices, dtypes, shapes, inner strides), allocates its outputs,
and hands device pointers and a stream to one C call, raising ``elq.ElqError``
where that refuses.  Nothing is copied or cast on the way: a tensor whose rows
are not contiguous, or whose rows are not whole multiples of 16 bytes apart
where the call needs it, is refused.

``stream`` is a ``torch.cuda.Stream`` (the current one by default); outputs are
allocated on it.  Calls run on the device of their tensors, whatever the current
device is.
"""
from __future__ import annotations

import ctypes

import torch

from . import elq
from .elq import BF16, F32, I32, I64, V, ElqError

F16, I8 = 1, 24
TYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16, torch.int8: I8}
FLOATS = {t: TYPES[t] for t in (torch.float32, torch.bfloat16, torch.float16)}
HALVES = {t: TYPES[t] for t in (torch.bfloat16, torch.float16)}
CODES, GATES = {torch.int8: I8}, {torch.float32: F32}
F = ctypes.c_float
INVALID, UNSUPPORTED = -1, -2


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

    __slots__ = ("_q", "_scale", "_buf", "_rows", "_cols", "_ld")

    def __init__(self, q: torch.Tensor, scale: torch.Tensor):
        self._q, self._scale, self._buf = q, scale, None

    @classmethod
    def _new(cls, like, rows, cols):
        """Uninitialised rows on like's device: (rows, codes' address, elements between rows, scales' address)."""
        r = cls.__new__(cls)
        ld = (cols + 15) & ~15
        r._q = r._scale = None
        r._buf, r._rows, r._cols, r._ld = like.new_empty(rows * (ld + 4), dtype=torch.int8), rows, cols, ld
        p = r._buf.data_ptr()
        return r, p, ld, p + rows * ld

    @property
    def q(self) -> torch.Tensor:
        if self._q is None:
            self._q = self._buf.as_strided((self._rows, self._cols), (self._ld, 1))
        return self._q

    @property
    def scale(self) -> torch.Tensor:
        if self._scale is None:
            self._scale = self._buf[self._rows * self._ld:].view(torch.float32)
        return self._scale

    @property
    def shape(self):
        return self.q.shape

    def dequantize(self, dtype=torch.float32) -> torch.Tensor:
        return (self.q.to(torch.float32) * self.scale.unsqueeze(-1)).to(dtype)


# ---- argument checks ------------------------------------------------------------

def _refuse(what, status=INVALID):
    raise ElqError(status, what)


def _matrix(t, what, types, dev=None):
    """Checks t (2-D, a dtype of types, contiguous rows, on device number dev); returns its address, type, rows,
    columns and the elements between rows."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        _refuse(what + ": a 2-D tensor")
    ty = types.get(t.dtype)
    if ty is None:
        _refuse(what + ": dtype %s" % t.dtype, UNSUPPORTED)
    at = t.get_device()
    if at < 0 or (dev is not None and at != dev):
        _refuse(what + ": device")
    rows, cols = t.shape
    ld, one = t.stride()
    if cols < 1 or (one != 1 and cols != 1):
        _refuse(what + ": contiguous rows")
    return t.data_ptr(), ty, rows, cols, ld if rows > 1 else (cols + 15) & ~15


def _vector(t, n, what, dev, dtype=torch.float32):
    """The address of a contiguous vector of n values, or None for None."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.get_device() == dev and t.numel() == n
            and t.is_contiguous()):
        _refuse("%s: %d contiguous %s values on the call's device" % (what, n, dtype))
    return t.data_ptr()


def _codes(m, what, dev=None):
    """Codes' address, elements between rows, scales' address, rows, columns and device number of 2-D I8Rows."""
    if not isinstance(m, I8Rows):
        _refuse(what + ": I8Rows")
    if m._buf is not None:
        at = m._buf.get_device()
        if dev is not None and at != dev:
            _refuse(what + ": device")
        p = m._buf.data_ptr()
        return p, m._ld, p + m._rows * m._ld, m._rows, m._cols, at
    p, _, rows, cols, ld = _matrix(m._q, what, CODES, dev)
    at = m._q.get_device()
    return p, ld, _vector(m._scale, rows, what + ".scale", at), rows, cols, at


def _experts(t, what, types, dev):
    """Address, elements between rows and experts, and shape of a stack [E, N, K] with contiguous rows."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        _refuse(what + ": a 3-D tensor")
    if t.dtype not in types:
        _refuse(what + ": dtype %s" % t.dtype, UNSUPPORTED)
    if t.get_device() != dev:
        _refuse(what + ": device")
    E, N, K = t.shape
    st, ld, one = t.stride()
    if K < 1 or (one != 1 and K != 1):
        _refuse(what + ": contiguous rows")
    return t.data_ptr(), ld if N > 1 else (K + 15) & ~15, st, E, N, K


# The current device's number, and the current stream of a device as an address: the getters under
# torch.cuda.current_device() and torch.cuda.current_stream(), without the objects around them (4 us a call).
_current = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _elsewhere(dev, stream, call, *args, **kw):
    """The call again with its device and its stream (if one was given) current."""
    if stream is None:
        with torch.cuda.device(dev):
            return call(*args, **kw)
    if stream.device.index != dev:
        _refuse("stream: of another device")
    with torch.cuda.stream(stream):
        return call(*args, **kw)


def _ck(status, what):
    if status != 0:
        raise ElqError(status, what)


def _out(out, like, rows, cols, dtype, dev, what):
    """The caller's out [rows, cols], or a new one beside `like`: tensor, address, elements between its rows."""
    if out is None:
        out = like.new_empty((rows, cols), dtype=dtype)
        return out, out.data_ptr(), cols
    p, ty, r, c, ld = _matrix(out, what, FLOATS, dev)
    if out.dtype != dtype or r != rows or c != cols:
        _refuse(what + ": shape or dtype")
    return out, p, ld


# ---- rows to codes --------------------------------------------------------------

def quantize_i8(x: torch.Tensor, index: torch.Tensor | None = None, index_div: int = 1, stream=None) -> I8Rows:
    """Codes of the rows of x [rows, K] (fp32, bf16, fp16), or of the gathered
    rows index[i] // index_div (int32 [n]; elq.route_bucket's pair order with
    index_div = k).  An expert stack [E, N, K] is quantised row by row."""
    if isinstance(x, torch.Tensor) and x.dim() == 3:
        if index is not None or not x.is_contiguous():
            _refuse("quantize_i8: a contiguous [E, N, K]")
        E, N, K = x.shape
        r = quantize_i8(x.view(-1, K), stream=stream)
        return I8Rows(r._buf.as_strided(x.shape, (N * r._ld, r._ld, 1)), r.scale.view(E, N))
    p, ty, n, cols, ld = _matrix(x, "quantize_i8: x", FLOATS)
    dev, rows, ip = x.get_device(), n, None
    if index is not None:
        rows = index.numel()
        ip = _vector(index, rows, "quantize_i8: index", dev, torch.int32)
    if stream is not None or dev != _current():
        return _elsewhere(dev, stream, quantize_i8, x, index, index_div)
    r, q, ldq, scale = I8Rows._new(x, rows, cols)
    _ck(lib().elq_quantize_i8(p, ty, n, cols, ld, ip, index_div, rows, q, ldq, scale, _raw_stream(dev)),
        "elq_quantize_i8")
    return r


def swiglu_i8(gu: torch.Tensor, stream=None) -> I8Rows:
    """Codes of silu(gate) * up for gu [rows, 2 I] = [gate | up]."""
    p, ty, rows, cols, ld = _matrix(gu, "swiglu_i8: gu", FLOATS)
    if cols % 2:
        _refuse("swiglu_i8: an even number of columns")
    dev = gu.get_device()
    if stream is not None or dev != _current():
        return _elsewhere(dev, stream, swiglu_i8, gu)
    r, q, ldq, scale = I8Rows._new(gu, rows, cols // 2)
    _ck(lib().elq_swiglu_i8(p, ty, rows, cols // 2, ld, q, ldq, scale, _raw_stream(dev)), "elq_swiglu_i8")
    return r


def combine_i8(o: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor, stream=None) -> I8Rows:
    """Codes of sum_j weights[t, j] * o[pos[t, j]]: o [rows, L], weights fp32
    [T, k], pos int32 of T * k row numbers (elq.route_bucket's pos)."""
    p, ty, n, cols, ld = _matrix(o, "combine_i8: o", FLOATS)
    dev = o.get_device()
    if weights.dim() != 2:
        _refuse("combine_i8: weights [T, k]")
    T, k = weights.shape
    wp = _vector(weights, T * k, "combine_i8: weights", dev)
    pp = _vector(pos, T * k, "combine_i8: pos", dev, torch.int32)
    if stream is not None or dev != _current():
        return _elsewhere(dev, stream, combine_i8, o, pos, weights)
    r, q, ldq, scale = I8Rows._new(o, T, cols)
    _ck(lib().elq_combine_i8(p, ty, n, cols, ld, pp, wp, T, k, q, ldq, scale, _raw_stream(dev)), "elq_combine_i8")
    return r


# ---- products -------------------------------------------------------------------

def i8_matmul(x: I8Rows, w: I8Rows, bias: torch.Tensor | None = None, out_dtype=torch.float32,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [T, N] = x [T, K] times w [N, K] transposed, from their codes, plus bias
    (fp32 [N])."""
    xp, ldx, sx, T, K, dev = _codes(x, "i8_matmul: x")
    wp, ldw, sw, N, Kw, _ = _codes(w, "i8_matmul: w", dev)
    if K != Kw:
        _refuse("i8_matmul: K of x and w")
    yt = FLOATS.get(out_dtype)
    if yt is None:
        _refuse("i8_matmul: out_dtype", UNSUPPORTED)
    bp = _vector(bias, N, "i8_matmul: bias", dev)
    if stream is not None or dev != _current():
        return _elsewhere(dev, stream, i8_matmul, x, w, bias, out_dtype, out)
    y, yp, ldy = _out(out, w._q if w._buf is None else w._buf, T, N, out_dtype, dev, "i8_matmul: out")
    _ck(lib().elq_i8_matmul(xp, ldx, sx, T, wp, ldw, sw, bp, N, K, yp, yt, ldy, _raw_stream(dev)), "elq_i8_matmul")
    return y


def grouped_matmul(x, w, offsets: torch.Tensor, out_dtype=None, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """y [M, N]: rows offsets[e] .. offsets[e+1]-1 of x [M, K] times expert e's
    matrix w[e] [N, K] transposed.  x and w both I8Rows, or both bf16 or fp16;
    offsets int32 [E+1].  out_dtype: for codes any of fp32 (default), bf16, fp16;
    for 16-bit x fp32 or its own (default).  Rows outside every group stay as out
    has them (undefined without out)."""
    codes = isinstance(x, I8Rows)
    if codes:
        xp, ldx, sx, M, K, dev = _codes(x, "grouped_matmul: x")
        if not isinstance(w, I8Rows):
            _refuse("grouped_matmul: w: I8Rows")
        xt, wt = I8, w.q
        wp, ldw, st, E, N, Kw = _experts(wt, "grouped_matmul: w", CODES, dev)
        sw = _vector(w.scale, E * N, "grouped_matmul: w.scale", dev)
    else:
        xp, xt, M, K, ldx = _matrix(x, "grouped_matmul: x", HALVES)
        dev, wt = x.get_device(), w
        wp, ldw, st, E, N, Kw = _experts(wt, "grouped_matmul: w", (x.dtype,), dev)
        sx = sw = None
    if K != Kw:
        _refuse("grouped_matmul: K of x and w")
    if offsets is None:
        _refuse("grouped_matmul: offsets")
    op = _vector(offsets, E + 1, "grouped_matmul: offsets", dev, torch.int32)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.float32 if codes else x.dtype
    yt = FLOATS.get(out_dtype)
    if yt is None:
        _refuse("grouped_matmul: out_dtype", UNSUPPORTED)
    if stream is not None or dev != _current():
        return _elsewhere(dev, stream, grouped_matmul, x, w, offsets, out_dtype, out)
    y, yp, ldy = _out(out, wt, M, N, out_dtype, dev, "grouped_matmul: out")
    _ck(lib().elq_grouped_matmul(xp, xt, ldx, sx, M, wp, ldw, st, sw, E, N, K, op, yp, yt, ldy, _raw_stream(dev)),
        "elq_grouped_matmul")
    return y


# ---- norms ----------------------------------------------------------------------

def rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6, out_dtype=None,
             out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x / sqrt(mean(x^2) + eps) * weight, row by row, in x's dtype or out_dtype;
    out may be x."""
    p, ty, T, C, ld = _matrix(x, "rms_norm: x", FLOATS)
    dev = x.get_device()
    wp = _vector(weight, C, "rms_norm: weight", dev)
    if out_dtype is None:
        out_dtype = x.dtype if out is None else out.dtype
    nt = FLOATS.get(out_dtype)
    if nt is None:
        _refuse("rms_norm: out_dtype", UNSUPPORTED)
    if stream is not None or dev != _current():
        return _elsewhere(dev, stream, rms_norm, x, weight, eps, out_dtype, out)
    n, np, ldn = _out(out, x, T, C, out_dtype, dev, "rms_norm: out")
    _ck(lib().elq_rms_norm(p, ty, T, C, ld, wp, eps, np, nt, ldn, None, _raw_stream(dev)), "elq_rms_norm")
    return n


def rms_norm_i8(x: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6, stream=None) -> I8Rows:
    """rms_norm handed straight to the row quantiser (the fp32 norm, unrounded)."""
    p, ty, T, C, ld = _matrix(x, "rms_norm_i8: x", FLOATS)
    dev = x.get_device()
    wp = _vector(weight, C, "rms_norm_i8: weight", dev)
    if stream is not None or dev != _current():
        return _elsewhere(dev, stream, rms_norm_i8, x, weight, eps)
    r, q, ldq, scale = I8Rows._new(x, T, C)
    _ck(lib().elq_rms_norm(p, ty, T, C, ld, wp, eps, q, I8, ldq, scale, _raw_stream(dev)), "elq_rms_norm")
    return r


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
    hp, ht, T, C, ldh = _matrix(h, "residual_norm: h", FLOATS)
    dev = h.get_device()
    yp, yt, Ty, Cy, ldy = _matrix(y, "residual_norm: y", FLOATS, dev)
    if T != Ty or C != Cy:
        _refuse("residual_norm: shapes of h and y")
    pw = _vector(post_weight, C, "residual_norm: post_weight", dev)
    gp, g_rows, gc, ldg = None, 1, 1, 1
    if gate is not None:
        if gate.dim() == 1:
            G, gc, ldg, gp = 1, gate.numel(), gate.numel(), _vector(gate, gate.numel(), "residual_norm: gate", dev)
        else:
            gp, _, G, gc, ldg = _matrix(gate, "residual_norm: gate", GATES, dev)
        if gc != C and gc != 1:
            _refuse("residual_norm: gate columns")
        g_rows = gate_rows
        if g_rows is None:
            if G != 1 and G != T:
                _refuse("residual_norm: gate rows")
            g_rows = max(T, 1) if G == 1 else 1
        if g_rows < 1 or G * g_rows < T:
            _refuse("residual_norm: gate rows")
    if stream is not None or dev != _current():
        return _elsewhere(dev, stream, residual_norm, h, y, post_weight, gate=gate, gate_rows=gate_rows,
                          res_scale=res_scale, next_weight=next_weight, next_dtype=next_dtype, eps=eps, out=out)
    h_out, op, ldo = _out(out, h, T, C, h.dtype, dev, "residual_norm: out")
    n = nw = np = scale = None
    nt = ldn = 0
    if next_dtype is not None:
        nw = _vector(next_weight, C, "residual_norm: next_weight", dev)
        nt = TYPES.get(next_dtype)
        if nt is None:
            _refuse("residual_norm: next_dtype", UNSUPPORTED)
        if nt == I8:
            n, np, ldn, scale = I8Rows._new(h, T, C)
        else:
            n, np, ldn = _out(None, h, T, C, next_dtype, dev, "")
    r = ResidualC(T, C, ht, yt, nt, hp, yp, pw, gp, nw, op, np, scale, ldh, ldy, ldo, ldn, g_rows, ldg, gc, res_scale, eps)
    _ck(lib().elq_residual_norm(ctypes.byref(r), _raw_stream(dev)), "elq_residual_norm")
    return h_out, n


def status(device=None, stream=None) -> int:
    """Blocking: whether a product's bounded device wait ran out since the last
    call (0, or the timeout status)."""
    dev = torch.cuda.current_device() if device is None else torch.cuda.device(device).idx
    if stream is not None or dev != _current():
        return _elsewhere(dev, stream, status, dev)
    return int(lib().elq_ops_status(_raw_stream(dev)))
