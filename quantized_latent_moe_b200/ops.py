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
FLOATS = (torch.float32, torch.bfloat16, torch.float16)
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
    expert weights [E, N, K] one a channel of each expert."""

    __slots__ = ("q", "scale")

    def __init__(self, q: torch.Tensor, scale: torch.Tensor):
        self.q, self.scale = q, scale

    @property
    def shape(self):
        return self.q.shape

    def dequantize(self, dtype=torch.float32) -> torch.Tensor:
        return (self.q.to(torch.float32) * self.scale.unsqueeze(-1)).to(dtype)


# ---- argument checks ------------------------------------------------------------

def _refuse(ok, what, status=INVALID):
    if not ok:
        raise ElqError(status, what)


def _matrix(t, what, dtypes, device=None, dims=2):
    """Checks t (dims-D, one of dtypes, contiguous rows, on device) and returns the elements between rows."""
    _refuse(isinstance(t, torch.Tensor) and t.dim() == dims, what + ": a %d-D tensor" % dims)
    _refuse(t.dtype in dtypes, what + ": dtype %s" % t.dtype, UNSUPPORTED)
    _refuse(t.is_cuda and (device is None or t.device == device), what + ": device")
    cols = t.shape[-1]
    _refuse(cols >= 1 and (cols == 1 or t.stride(-1) == 1), what + ": contiguous rows")
    return t.stride(-2) if t.shape[-2] > 1 else (cols + 15) // 16 * 16


def _vector(t, n, what, device, dtype=torch.float32):
    """A contiguous vector of n (or None)."""
    if t is not None:
        _refuse(isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == device and t.numel() == n
                and t.is_contiguous(), what + ": contiguous %s of %d values on the call's device" % (dtype, n))
        return t.data_ptr()
    return None


def _i8(m, what, device, dims=2):
    _refuse(isinstance(m, I8Rows), what + ": I8Rows")
    ld = _matrix(m.q, what, (torch.int8,), device, dims)
    return ld, _vector(m.scale, m.q.numel() // m.q.shape[-1], what + ".scale", m.q.device)


class _On:
    """The device and stream of a call: ``with _On(device, stream) as raw``."""

    __slots__ = ("guard", "raw")

    def __init__(self, device, stream):
        self.guard = None
        if stream is not None:
            _refuse(stream.device == device, "stream: of another device")
            self.guard = torch.cuda.stream(stream)
            self.raw = stream.cuda_stream
        else:
            if device.index != torch.cuda.current_device():
                self.guard = torch.cuda.device(device)
            self.raw = torch.cuda.current_stream(device).cuda_stream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.raw

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _ck(status, what):
    if status != 0:
        raise ElqError(status, what)


def _new_rows(rows, cols, device):
    """Codes with rows padded to whole 16 bytes, and scales."""
    ld = (cols + 15) // 16 * 16
    q = torch.empty((rows, ld), dtype=torch.int8, device=device)
    return (q if ld == cols else q[:, :cols]), ld, torch.empty(rows, dtype=torch.float32, device=device)


def _out(out, rows, cols, dtype, device, what):
    """The caller's out [rows, cols], or a new one; and the elements between its rows."""
    if out is None:
        return torch.empty((rows, cols), dtype=dtype, device=device), cols
    ld = _matrix(out, what, (dtype,), device)
    _refuse(out.shape[0] == rows and out.shape[1] == cols, what + ": shape")
    return out, ld


# ---- rows to codes --------------------------------------------------------------

def quantize_i8(x: torch.Tensor, index: torch.Tensor | None = None, index_div: int = 1, stream=None) -> I8Rows:
    """Codes of the rows of x [rows, K] (fp32, bf16, fp16), or of the gathered
    rows index[i] // index_div (int32 [n]; elq.route_bucket's pair order with
    index_div = k).  An expert stack [E, N, K] is quantised row by row."""
    if x.dim() == 3:
        _refuse(index is None and x.is_contiguous(), "quantize_i8: a contiguous [E, N, K]")
        r = quantize_i8(x.view(-1, x.shape[-1]), stream=stream)
        ld = (x.shape[-1] + 15) // 16 * 16
        return I8Rows(r.q.as_strided(x.shape, (x.shape[1] * ld, ld, 1)), r.scale.view(x.shape[:2]))
    ld = _matrix(x, "quantize_i8: x", FLOATS)
    dev = x.device
    rows = x.shape[0]
    ip = None
    if index is not None:
        rows = index.numel()
        ip = _vector(index, rows, "quantize_i8: index", dev, torch.int32)
    with _On(dev, stream) as s:
        q, ldq, scale = _new_rows(rows, x.shape[1], dev)
        _ck(lib().elq_quantize_i8(x.data_ptr(), TYPES[x.dtype], x.shape[0], x.shape[1], ld, ip, index_div, rows,
                                  q.data_ptr(), ldq, scale.data_ptr(), s), "elq_quantize_i8")
    return I8Rows(q, scale)


def swiglu_i8(gu: torch.Tensor, stream=None) -> I8Rows:
    """Codes of silu(gate) * up for gu [rows, 2 I] = [gate | up]."""
    ld = _matrix(gu, "swiglu_i8: gu", FLOATS)
    _refuse(gu.shape[1] % 2 == 0, "swiglu_i8: an even number of columns")
    rows, I = gu.shape[0], gu.shape[1] // 2
    with _On(gu.device, stream) as s:
        q, ldq, scale = _new_rows(rows, I, gu.device)
        _ck(lib().elq_swiglu_i8(gu.data_ptr(), TYPES[gu.dtype], rows, I, ld, q.data_ptr(), ldq, scale.data_ptr(), s),
            "elq_swiglu_i8")
    return I8Rows(q, scale)


def combine_i8(o: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor, stream=None) -> I8Rows:
    """Codes of sum_j weights[t, j] * o[pos[t, j]]: o [rows, L], weights fp32
    [T, k], pos int32 of T * k row numbers (elq.route_bucket's pos)."""
    ld = _matrix(o, "combine_i8: o", FLOATS)
    dev = o.device
    _refuse(weights.dim() == 2, "combine_i8: weights [T, k]")
    T, k = weights.shape
    wp = _vector(weights, T * k, "combine_i8: weights", dev)
    pp = _vector(pos, T * k, "combine_i8: pos", dev, torch.int32)
    with _On(dev, stream) as s:
        q, ldq, scale = _new_rows(T, o.shape[1], dev)
        _ck(lib().elq_combine_i8(o.data_ptr(), TYPES[o.dtype], o.shape[0], o.shape[1], ld, pp, wp, T, k,
                                 q.data_ptr(), ldq, scale.data_ptr(), s), "elq_combine_i8")
    return I8Rows(q, scale)


# ---- products -------------------------------------------------------------------

def i8_matmul(x: I8Rows, w: I8Rows, bias: torch.Tensor | None = None, out_dtype=torch.float32,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [T, N] = x [T, K] times w [N, K] transposed, from their codes, plus bias
    (fp32 [N])."""
    ldx, sx = _i8(x, "i8_matmul: x", None)
    dev = x.q.device
    ldw, sw = _i8(w, "i8_matmul: w", dev)
    T, K = x.q.shape
    N = w.q.shape[0]
    _refuse(w.q.shape[1] == K, "i8_matmul: K of x and w")
    _refuse(out_dtype in FLOATS, "i8_matmul: out_dtype", UNSUPPORTED)
    bp = _vector(bias, N, "i8_matmul: bias", dev)
    with _On(dev, stream) as s:
        y, ldy = _out(out, T, N, out_dtype, dev, "i8_matmul: out")
        _ck(lib().elq_i8_matmul(x.q.data_ptr(), ldx, sx, T, w.q.data_ptr(), ldw, sw, bp, N, K, y.data_ptr(),
                                TYPES[out_dtype], ldy, s), "elq_i8_matmul")
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
        ldx, sx = _i8(x, "grouped_matmul: x", None)
        ldw, sw = _i8(w, "grouped_matmul: w", x.q.device, 3)
        xt, wt = x.q, w.q
    else:
        ldx, sx = _matrix(x, "grouped_matmul: x", (torch.bfloat16, torch.float16)), None
        ldw, sw = _matrix(w, "grouped_matmul: w", (x.dtype,), x.device, 3), None
        xt, wt = x, w
    dev = xt.device
    M, K = xt.shape
    E, N = wt.shape[0], wt.shape[1]
    _refuse(wt.shape[2] == K, "grouped_matmul: K of x and w")
    op = _vector(offsets, E + 1, "grouped_matmul: offsets", dev, torch.int32)
    _refuse(op is not None, "grouped_matmul: offsets")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.float32 if codes else x.dtype
    _refuse(out_dtype in FLOATS, "grouped_matmul: out_dtype", UNSUPPORTED)
    with _On(dev, stream) as s:
        y, ldy = _out(out, M, N, out_dtype, dev, "grouped_matmul: out")
        _ck(lib().elq_grouped_matmul(xt.data_ptr(), TYPES[xt.dtype], ldx, sx, M, wt.data_ptr(), ldw, wt.stride(0), sw,
                                     E, N, K, op, y.data_ptr(), TYPES[out_dtype], ldy, s), "elq_grouped_matmul")
    return y


# ---- norms ----------------------------------------------------------------------

def rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6, out_dtype=None,
             out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x / sqrt(mean(x^2) + eps) * weight, row by row, in x's dtype or out_dtype;
    out may be x."""
    ld = _matrix(x, "rms_norm: x", FLOATS)
    dev = x.device
    T, C = x.shape
    wp = _vector(weight, C, "rms_norm: weight", dev)
    if out_dtype is None:
        out_dtype = x.dtype if out is None else out.dtype
    _refuse(out_dtype in FLOATS, "rms_norm: out_dtype", UNSUPPORTED)
    with _On(dev, stream) as s:
        n, ldn = _out(out, T, C, out_dtype, dev, "rms_norm: out")
        _ck(lib().elq_rms_norm(x.data_ptr(), TYPES[x.dtype], T, C, ld, wp, eps, n.data_ptr(), TYPES[out_dtype], ldn,
                               None, s), "elq_rms_norm")
    return n


def rms_norm_i8(x: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6, stream=None) -> I8Rows:
    """rms_norm handed straight to the row quantiser (the fp32 norm, unrounded)."""
    ld = _matrix(x, "rms_norm_i8: x", FLOATS)
    dev = x.device
    T, C = x.shape
    wp = _vector(weight, C, "rms_norm_i8: weight", dev)
    with _On(dev, stream) as s:
        q, ldq, scale = _new_rows(T, C, dev)
        _ck(lib().elq_rms_norm(x.data_ptr(), TYPES[x.dtype], T, C, ld, wp, eps, q.data_ptr(), I8, ldq,
                               scale.data_ptr(), s), "elq_rms_norm")
    return I8Rows(q, scale)


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
    ldh = _matrix(h, "residual_norm: h", FLOATS)
    dev = h.device
    ldy = _matrix(y, "residual_norm: y", FLOATS, dev)
    T, C = h.shape
    _refuse(y.shape == h.shape, "residual_norm: shapes of h and y")
    r = ResidualC()
    r.T, r.cols, r.h_type, r.y_type = T, C, TYPES[h.dtype], TYPES[y.dtype]
    r.h, r.y, r.ldh, r.ldy = h.data_ptr(), y.data_ptr(), ldh, ldy
    r.post_weight = _vector(post_weight, C, "residual_norm: post_weight", dev)
    if gate is not None:
        g = gate.unsqueeze(0) if gate.dim() == 1 else gate
        r.gate_ld = _matrix(g, "residual_norm: gate", (torch.float32,), dev)
        G = g.shape[0]
        _refuse(g.shape[1] in (1, C), "residual_norm: gate columns")
        if gate_rows is None:
            _refuse(G == 1 or G == T, "residual_norm: gate rows")
            gate_rows = max(T, 1) if G == 1 else 1
        _refuse(gate_rows >= 1 and G * gate_rows >= T, "residual_norm: gate rows")
        r.gate, r.gate_rows, r.gate_cols = g.data_ptr(), gate_rows, g.shape[1]
    r.res_scale, r.eps = res_scale, eps
    with _On(dev, stream) as s:
        h_out, r.ld_out = _out(out, T, C, h.dtype, dev, "residual_norm: out")
        r.h_out = h_out.data_ptr()
        n = None
        if next_dtype is not None:
            r.next_weight = _vector(next_weight, C, "residual_norm: next_weight", dev)
            if next_dtype == torch.int8:
                q, r.ldn, scale = _new_rows(T, C, dev)
                n = I8Rows(q, scale)
                r.n, r.scale = q.data_ptr(), scale.data_ptr()
            else:
                _refuse(next_dtype in FLOATS, "residual_norm: next_dtype", UNSUPPORTED)
                n, r.ldn = _out(None, T, C, next_dtype, dev, "")
                r.n = n.data_ptr()
            r.n_type = TYPES[next_dtype]
        _ck(lib().elq_residual_norm(ctypes.byref(r), s), "elq_residual_norm")
    return h_out, n


def status(device=None, stream=None) -> int:
    """Blocking: whether a product's bounded device wait ran out since the last
    call (0, or the timeout status)."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with _On(device, stream) as s:
        return int(lib().elq_ops_status(s))
