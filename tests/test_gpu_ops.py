"""The calls of include/elq_ops.h against their formulas in 64 bits.

Tolerances count roundings: u32 = 2^-24 for an fp32 operation, and half a step
of the output type (bf16 2^-8, fp16 2^-11, fp32 2^-24 relative; fp16 also
2^-25 absolute, half its smallest step) for the one rounding of an output.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
GUARD = 77.0


@pytest.fixture(scope="module")
def O():
    from quantized_latent_moe_b200 import build, ops
    build.build()
    ops.lib()
    assert torch.cuda.is_available()
    return ops


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32, ld=None):
    """Normal values; with ld, a view of rows ld apart whose gaps hold NaN."""
    x = torch.randn(*shape, generator=g, device="cuda").to(dtype)
    if ld is None:
        return x
    full = torch.full((*shape[:-1], ld), float("nan"), dtype=dtype, device="cuda")
    full[..., :shape[-1]] = x
    return full[..., :shape[-1]]


def codes(g, *shape, ld=None):
    """Codes over the whole int8 range (gaps between rows hold -128), scales over five binades."""
    k = shape[-1]
    ld = (k + 15) // 16 * 16 if ld is None else ld
    full = torch.full((*shape[:-1], ld), -128, dtype=torch.int8, device="cuda")
    full[..., :k] = torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int8)
    scale = torch.exp2(torch.rand(shape[:-1], generator=g, device="cuda") * 5 - 8)
    return full[..., :k], scale


def check(got, ref, bound, dtype):
    """|got - ref| <= bound (of the fp32 value) + one rounding to dtype."""
    got = got.double()
    tol = bound + half_step(dtype) * (ref.abs() + bound) * (1 + 2.0 ** -10) + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -149)
    over = ((got - ref).abs() > tol) | got.isnan()
    assert not bool(over.any()), "%d of %d over, worst %.3g against %.3g" % (
        int(over.sum()), over.numel(), float((got - ref).abs().max()), float(tol[(got - ref).abs() == (got - ref).abs().max()].max()))


# ---- rows to codes ------------------------------------------------------------

def codes64(v):
    """Scale (fp32) and codes of rows from their definition, in 64 bits."""
    v = v.double()
    s = (v.abs().amax(-1).float().double() / 127).float()
    r = v / torch.where(s > 0, s, torch.ones_like(s)).double().unsqueeze(-1)
    q = torch.sign(r) * torch.floor(r.abs() + 0.5)
    return q.clamp(-127, 127), s


@pytest.mark.parametrize("x", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,K,ld", [(1, 1, None), (1, 4096, None), (3, 7, None), (5, 8, 11), (1, 1003, None), (77, 1003, 1009),
                                    (700, 64, None), (700, 520, None), (2048, 1792, 1800), (9, 16384, None),
                                    (3, 16385, None), (400, 16392, 16400), (3, 40000, 40001)])
def test_quantize_exact(O, x, T, K, ld):
    v = randn(rng(T * 7 + K), T, K, dtype=DT[x], ld=ld)
    r = O.quantize_i8(v)
    q, s = codes64(v)
    assert torch.equal(r.scale, s) and torch.equal(r.q.double(), q)


def test_quantize_ties_extremes_and_magnitudes(O):
    # halves of the scale exactly: amax = 127 * 2^e gives s = 2^e, and (n + 1/2) s are ties, away from zero
    n = torch.arange(-127, 127, device="cuda", dtype=torch.float32) + 0.5
    for e in (-140, -126, -120, -101, -100, -99, -60, 0, 60, 120):
        if e < -126:
            continue
        row = torch.cat([n, torch.tensor([127.0, -127.0, 0.0, -0.0], device="cuda")]) * 2.0 ** e
        r = O.quantize_i8(row.unsqueeze(0))
        q, s = codes64(row.unsqueeze(0))
        assert torch.equal(r.scale, s) and torch.equal(r.q.double(), q), e
    # magnitudes from subnormal to the largest
    g = rng(5)
    for mag in (1e-44, 1e-41, 3e-39, 1e-37, 1e-30, 1e30, 3e38):
        v = (torch.rand(4, 300, generator=g, device="cuda") * 2 - 1) * mag
        r = O.quantize_i8(v)
        q, s = codes64(v)
        q = torch.where((s == 0).unsqueeze(-1), torch.zeros_like(q), q)
        assert torch.equal(r.scale, s) and torch.equal(r.q.double(), q), mag


def test_quantize_zero_and_nonfinite_rows(O):
    for K in (5, 300, 17000):
        v = torch.randn(6, K, generator=rng(K), device="cuda")
        v[1] = 0
        v[2, K // 2] = float("inf")
        v[3, 0] = float("nan")
        v[4, K - 1] = -float("inf")
        r = O.quantize_i8(v)
        q, s = codes64(v[[0, 5]])
        assert torch.equal(r.q[[0, 5]].double(), q) and torch.equal(r.scale[[0, 5]], s)
        assert float(r.scale[1]) == 0 and not bool(r.q[1:5].any()) and bool(r.scale[2:5].isnan().all())


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("K", [7, 64, 1792, 17000])
def test_quantize_gather(O, x, K):
    v = randn(rng(K), 11, K, dtype=DT[x])
    idx = torch.tensor([0, 87, 5, 5, 86, -1, 88, 2 ** 31 - 1, -2 ** 31, 16, 44], dtype=torch.int32, device="cuda")
    r = O.quantize_i8(v, index=idx, index_div=8)
    q, s = codes64(v)
    for i, p in enumerate(idx.tolist()):
        row = p // 8
        if 0 <= p and row < 11:
            assert torch.equal(r.q[i].double(), q[row]) and r.scale[i] == s[row]
        else:
            assert not bool(r.q[i].any()) and float(r.scale[i]) == 0
    assert O.quantize_i8(v, index=idx[:0], index_div=3).q.shape == (0, K)


def test_quantize_padding_and_experts(O):
    # the bytes between rows stay as they are, and an expert stack is its rows
    import ctypes
    v = torch.randn(5, 37, generator=rng(3), device="cuda")
    q = torch.full((5, 64), 99, dtype=torch.int8, device="cuda")
    s = torch.empty(5, device="cuda")
    st = O.lib().elq_quantize_i8(v.data_ptr(), 0, 5, 37, 37, None, 1, 5, q.data_ptr(), 64, s.data_ptr(),
                                 ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert st == 0 and bool((q[:, 37:] == 99).all()) and torch.equal(q[:, :37].double(), codes64(v)[0])
    w = torch.randn(3, 5, 37, generator=rng(4), device="cuda")
    r = O.quantize_i8(w)
    q, s = codes64(w)
    assert torch.equal(r.q.double(), q) and torch.equal(r.scale, s)


def check_codes(r, v, err):
    """The codes of computed rows: v in 64 bits, each fp32 value within err of it.  The scale is an fp32
    division of the largest magnitude, and a code's value at most half a scale from the fp32 value."""
    s = r.scale.double().unsqueeze(-1)
    amax = v.abs().amax(-1, keepdim=True)
    worst = err.amax(-1, keepdim=True)
    assert bool(((s * 127 - amax).abs() <= worst + 2 * U32 * amax).all())
    assert int(r.q.int().abs().max()) <= 127
    off = (r.q.double() * s - v).abs()
    # the largest value's code is 127: 127 s is within two roundings of it
    assert bool((off <= 0.5 * s * (1 + 2.0 ** -20) + err + 4 * U32 * amax).all())


@pytest.mark.parametrize("x", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,I,pad", [(1, 1, 0), (1, 1024, 0), (6, 7, 3), (300, 333, 0), (1000, 1024, 16), (64, 4100, 4),
                                     (2, 17000, 0)])
def test_swiglu(O, x, T, I, pad):
    gu = (randn(rng(I + T), T, 2 * I, dtype=DT[x]) * 4).to(DT[x])
    if pad:
        full = torch.full((T, 2 * I + pad), float("nan"), dtype=DT[x], device="cuda")
        full[:, :2 * I] = gu
        gu = full[:, :2 * I]
    gu[0, 0] = -100.0
    g, u = gu[:, :I].double(), gu[:, I:].double()
    v = g / (1 + torch.exp(-g)) * u
    # exp 2^-21, the sum 2^-24, quotient and product 2^-24 each; below exp's range g / (1 + e^-g) is under
    # 88 * 2^-126 * |u| and may be flushed
    err = (2.0 ** -21 + 4 * U32) * v.abs() + 2.0 ** -118 * u.abs()
    check_codes(O.swiglu_i8(gu), v, err)


@pytest.mark.parametrize("I", [1, 8])
def test_swiglu_value(O, I):
    """The value itself, over all of g's range: a row of one value (or eight alike, which go the aligned way)
    has the scale |h| / 127, so that |h| shows to within that division's rounding."""
    g = rng(3)
    gate = torch.cat([torch.linspace(-88.7, 88.7, 1 << 19, device="cuda"), torch.randn(1 << 19, generator=g, device="cuda")])
    up = torch.exp2(torch.rand(gate.numel(), generator=g, device="cuda") * 8 - 4)
    r = O.swiglu_i8(torch.cat([gate[:, None].expand(-1, I), up[:, None].expand(-1, I)], 1).contiguous())
    ref = gate.double() / (1 + torch.exp(-gate.double())) * up.double()
    # exp within an ulp (two units of 2^-24) and by its share of the sum; the sum, the quotient, the product; then the
    # scale's division, whose half step is 2^-150 where it is subnormal.  Zero is allowed below exp's range.
    share = torch.sigmoid(-gate.double())
    tol = (2 * share + 3 + 1) * U32 * (1 + 2.0 ** -16) * ref.abs() + 127 * 2.0 ** -150
    tol = tol + torch.where(gate < -87, 2.0 ** -119, 0.0) * up.double()
    off = (r.scale.double() * 127 - ref.abs()).abs()
    assert bool((off <= tol).all()), "%d of %d over" % (int((off > tol).sum()), off.numel())
    # the steps themselves: torch's exp is CUDA's too, and a quotient good to 2^-45 before its rounding is rounded
    # as the exact one but for 2^-20 of them
    steps = (gate / (1 + torch.exp(-gate)) * up).abs()[gate > -87]
    assert int((r.scale[gate > -87] != (steps.double() / 127).float()).sum()) <= gate.numel() // 1000


def test_swiglu_nonfinite(O):
    gu = torch.randn(4, 128, generator=rng(1), device="cuda")
    gu[1, 3], gu[2, 70], gu[3, 0] = float("nan"), float("inf"), float("-inf")
    r = O.swiglu_i8(gu)
    assert bool(r.scale[0].isfinite()) and bool(r.scale[1:3].isnan().all())
    assert not bool(r.q[1:3].any())


@pytest.mark.parametrize("o", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,k,L", [(1, 8, 1792), (6, 1, 33), (32, 8, 1792), (700, 2, 256), (3, 64, 1000), (2, 3, 17001)])
def test_combine(O, o, T, k, L):
    g = rng(T * k + L)
    rows = randn(g, T * k, L, dtype=DT[o])
    pos = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)
    w = torch.rand(T, k, generator=g, device="cuda")
    pos[0] = -1 if T > 1 else pos[0]
    if T > 1:
        pos[1] = T * k
    ok = (pos >= 0) & (pos < T * k)
    parts = rows.double()[pos.clamp(0, T * k - 1).long()] * (ok * w.reshape(-1).double()).unsqueeze(-1)
    parts = parts.reshape(T, k, L)
    check_codes(O.combine_i8(rows, pos, w), parts.sum(1), (k + 1) * U32 * parts.abs().sum(1))


# ---- norms --------------------------------------------------------------------

# relative error of an fp32 norm's factor 1 / sqrt(mean + eps): the sum of squares of at most 64 values a
# thread (one rounding each), 5 shuffles and 16 partial sums, halved by the root; the reciprocal of the length
# and the fused multiply-add with eps, halved; rsqrtf's 2 ulp, which are 4 of these units.  Then the two
# products of a value.
RSTD = ((64 + 5 + 16 + 2) / 2 + 4) * U32
NORM = RSTD + 2 * U32


def rms64(x, w, eps):
    x = x.double()
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return n if w is None else n * w.double()


@pytest.mark.parametrize("x,n", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f16")])
@pytest.mark.parametrize("T,C,ld,weight", [(1, 1, None, True), (1, 4096, None, True), (5, 13, 17, True), (777, 1283, 1289, True),
                                           (2048, 256, None, False), (500, 4096, 4104, True), (2, 16384, None, True),
                                           (2, 20000, None, True), (301, 12, None, True)])
def test_rms_norm(O, x, n, T, C, ld, weight):
    g = rng(C + T)
    v = randn(g, T, C, dtype=DT[x], ld=ld)
    w = randn(g, C) if weight else None
    ref = rms64(v, w, 1e-5)
    check(O.rms_norm(v, w, eps=1e-5, out_dtype=DT[n]), ref, NORM * ref.abs(), DT[n])
    check_codes(O.rms_norm_i8(v, w, eps=1e-5), ref, NORM * ref.abs())


def test_rms_norm_in_place_zero_and_out(O):
    for C in (100, 4096, 17000):
        v = randn(rng(C), 40, C)
        v[3] = 0
        ref = O.rms_norm(v)
        assert not bool(ref[3].any())
        wide = torch.full((40, C + 5), GUARD, device="cuda")
        out = O.rms_norm(v, out=wide[:, :C])
        check(out, rms64(v, None, 1e-6), NORM * rms64(v, None, 1e-6).abs(), torch.float32)
        assert bool((wide[:, C:] == GUARD).all())
        O.rms_norm(v, out=v)
        assert torch.equal(v, ref)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("T,C,ld", [(1, 4096, None), (700, 4096, None), (5, 1283, 1289), (2, 12000, None), (2, 20000, None), (400, 64, None)])
def test_norms_of_large_values(O, x, T, C, ld):
    """Rows whose sum of squares passes fp32, up to 1e36, beside ordinary ones, and rows with an infinity or a NaN."""
    g = rng(C)
    v = randn(g, T, C, ld=ld)
    v *= torch.tensor([5e17, 1.0, 1e25, 1e35, 1e-3], device="cuda").repeat(T)[:T, None]
    v = torch.nn.functional.pad(v, (0, 7))[:, :C].to(DT[x])
    w = randn(g, C)
    ref = rms64(v, w, 1e-5)
    check(O.rms_norm(v, w, eps=1e-5, out_dtype=torch.float32), ref, NORM * ref.abs(), torch.float32)
    check_codes(O.rms_norm_i8(v, w, eps=1e-5), ref, NORM * ref.abs())
    ones = torch.ones(T, C, device="cuda")
    h, n = O.residual_norm(ones, v, w, next_dtype=torch.float32)
    ref = rms64(v, w, 1e-6)
    check(h, ref + 1, NORM * ref.abs() + 2 * U32 * (ref.abs() + 1), torch.float32)
    # h' large: y is zero, the gate irrelevant, n the norm of h alone
    h, n = O.residual_norm(v.float(), torch.zeros(T, C, device="cuda"), next_weight=w, next_dtype=torch.float32)
    check(n, ref, NORM * ref.abs(), torch.float32)
    v[0, C // 2] = float("inf")
    assert not bool(O.rms_norm(v)[0].isfinite().all()) and bool(O.rms_norm_i8(v).scale[0].isnan())


@pytest.mark.parametrize("h,y,n", [("f32", "f32", "bf16"), ("bf16", "bf16", "bf16"), ("f16", "f32", "i8"), ("f32", "bf16", "i8"),
                                   ("bf16", "f16", "f32"), ("f16", "f16", None)])
@pytest.mark.parametrize("T,C,pad,gate", [(1, 4096, 0, "channel"), (1, 1, 0, "token"), (6, 9, 2, "none"), (777, 1283, 6, "token"),
                                          (600, 4096, 8, "full"), (33, 520, 0, "blocks"), (2, 17001, 0, "channel"),
                                          (3, 16384, 0, "full")])
def test_residual_norm(O, h, y, n, T, C, pad, gate):
    g = rng(T + C)
    H = randn(g, T, C, dtype=DT[h], ld=C + pad)
    Y = (randn(g, T, C, dtype=DT[y], ld=C + pad) * 3)[:, :C]
    post, pre = randn(g, C), randn(g, C)
    G, rows, gr = {"none": (None, None, None), "channel": (randn(g, C), None, T), "token": (randn(g, T, 1), None, 1),
                   "full": (randn(g, T, C, ld=C + pad), None, 1), "blocks": (randn(g, 5, C), 7, 7)}[gate]
    nd = torch.int8 if n == "i8" else None if n is None else DT[n]
    out = torch.full((T, C + pad + 3), GUARD, dtype=DT[h], device="cuda")
    hn, nn = O.residual_norm(H, Y, post, gate=G, gate_rows=rows, res_scale=0.75, next_weight=pre, next_dtype=nd, eps=1e-5,
                             out=out[:, :C])
    v = rms64(Y, post, 1e-5)
    if G is not None:
        full = (G.reshape(1, -1) if G.dim() == 1 else G).double()
        v = v * full[torch.arange(T, device="cuda") // gr]
    res = 0.75 * H.double()
    ref = res + v
    err = NORM * v.abs() + 2 * U32 * (res.abs() + v.abs())
    check(hn, ref, err, DT[h])
    assert hn.data_ptr() == out.data_ptr() and bool((out[:, C:] == GUARD).all())
    if n is None:
        assert nn is None
        return
    # the next norm of the unrounded h': its values' errors, and theirs on the norm's factor
    ref2 = rms64(ref, pre, 1e-5)
    f = (err.square().sum(-1, keepdim=True) / ref.square().sum(-1, keepdim=True)).sqrt()
    rstd = 1 / torch.sqrt(ref.square().mean(-1, keepdim=True) + 1e-5)
    err2 = (err * rstd * pre.double().abs() + (f + NORM) * ref2.abs()) * (1 + 2.0 ** -10)
    if n == "i8":
        check_codes(nn, ref2, err2)
    else:
        check(nn, ref2, err2, DT[n])


def test_residual_norm_in_place(O):
    for C in (64, 1000, 4096, 17000):
        g = rng(C)
        H, Y, G = randn(g, 50, C), randn(g, 50, C), randn(g, C)
        a, n = O.residual_norm(H, Y, gate=G, next_dtype=torch.float32)
        b, m = O.residual_norm(H, Y, gate=G, next_dtype=torch.float32, out=H)
        assert b.data_ptr() == H.data_ptr() and torch.equal(a, b) and torch.equal(n, m)


@pytest.mark.parametrize("T", [2, 310])
def test_wide_aligned_rows(O, T):
    """Aligned rows longer than the ring in shared memory takes: 14336 values, and fp32 rows of 10248 with a gate a row."""
    g, C = rng(T), 14336
    v = randn(g, T, C, dtype=torch.bfloat16)
    r, (q, s) = O.quantize_i8(v), codes64(v)
    assert torch.equal(r.scale, s) and torch.equal(r.q.double(), q)
    w = randn(g, C)
    ref = rms64(v, w, 1e-6)
    check(O.rms_norm(v, w), ref, NORM * ref.abs(), torch.bfloat16)
    gu = randn(g, T, 2 * C, dtype=torch.bfloat16)
    a, b = gu[:, :C].double(), gu[:, C:].double()
    ref = a * torch.sigmoid(a) * b
    check_codes(O.swiglu_i8(gu), ref, 5 * U32 * (1 + 2.0 ** -16) * ref.abs() + 2.0 ** -119 * b.abs())
    for H, Y, G in ((randn(g, T, C, dtype=torch.bfloat16), v, randn(g, C)), (randn(g, T, 10248), randn(g, T, 10248), randn(g, T, 10248))):
        post, pre = randn(g, H.shape[1]), randn(g, H.shape[1])
        want = O.residual_norm(H, Y, post, gate=G, next_weight=pre, next_dtype=torch.float32)
        n = rms64(Y, post, 1e-6) * G.double()
        ref = H.double() + n
        err = NORM * n.abs() + 2 * U32 * (H.double().abs() + n.abs())
        check(want[0], ref, err, H.dtype)
        f = (err.square().sum(-1, keepdim=True) / ref.square().sum(-1, keepdim=True)).sqrt()
        rstd = 1 / torch.sqrt(ref.square().mean(-1, keepdim=True) + 1e-6)
        ref2 = rms64(ref, pre, 1e-6)
        check(want[1], ref2, (err * rstd * pre.double().abs() + (f + NORM) * ref2.abs()) * (1 + 2.0 ** -10), torch.float32)
        got = O.residual_norm(H, Y, post, gate=G, next_weight=pre, next_dtype=torch.float32, out=H)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_vectors_off_sixteen_bytes(O):
    """Weights, gates, bias and scales that start on a 4-byte boundary only."""
    g = rng(31)
    C, T = 520, 400
    off = lambda n: torch.randn(n + 1, generator=g, device="cuda")[1:]
    H, Y, post, pre, gate = randn(g, T, C), randn(g, T, C, dtype=torch.bfloat16), off(C), off(C), off(C)
    a = O.residual_norm(H, Y, post, gate=gate, next_weight=pre, next_dtype=torch.bfloat16)
    v = rms64(Y, post, 1e-6) * gate.double()
    check(a[0], H.double() + v, NORM * v.abs() + 2 * U32 * (H.double().abs() + v.abs()), torch.float32)
    ref = rms64(H, post, 1e-6)
    check(O.rms_norm(H, post), ref, NORM * ref.abs(), torch.float32)
    for rows in (3, 200):
        (x, sx), (w, sw) = codes(g, rows, 64), codes(g, 50, 64)
        sx2, sw2, bias = torch.empty(rows + 1, device="cuda")[1:].copy_(sx), torch.empty(51, device="cuda")[1:].copy_(sw), off(50)
        y = O.i8_matmul(O.I8Rows(x, sx2), O.I8Rows(w, sw2), bias=bias)
        ref = product64(x, sx, w, sw)
        check(y, ref + bias.double(), 3.01 * U32 * ref.abs() + U32 * (ref + bias.double()).abs(), torch.float32)


def test_no_rows(O):
    z = torch.empty(0, 64, device="cuda")
    w = O.quantize_i8(torch.randn(32, 64, device="cuda"))
    ws = O.I8Rows(w.q.view(2, 16, 64), w.scale.view(2, 16))
    assert O.quantize_i8(z).q.shape == (0, 64) and O.swiglu_i8(z).q.shape == (0, 32)
    assert O.combine_i8(torch.ones(3, 64, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"),
                        torch.empty(0, 2, device="cuda")).q.shape == (0, 64)
    assert O.rms_norm(z).shape == (0, 64) and O.rms_norm_i8(z).scale.shape == (0,)
    for gate in (None, torch.ones(64, device="cuda"), torch.ones(0, 64, device="cuda"), torch.ones(0, 1, device="cuda")):
        h, n = O.residual_norm(z, z.clone(), gate=gate, next_dtype=torch.int8)
        assert h.shape == (0, 64) and n.q.shape == (0, 64)
    assert O.i8_matmul(O.quantize_i8(z), w).shape == (0, 32)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert O.grouped_matmul(O.quantize_i8(z), ws, off).shape == (0, 16)
    assert O.grouped_matmul(z.half(), torch.ones(2, 16, 64, device="cuda").half(), off).shape == (0, 16)
    torch.cuda.synchronize()


def test_single_expert_and_single_columns(O):
    g = rng(41)
    for M in (1, 7, 50):
        (x, sx), (w, sw) = codes(g, M, 33), codes(g, 1, 70, 33)
        y = O.grouped_matmul(O.I8Rows(x, sx), O.I8Rows(w, sw), offsets_of([M]))
        ref = product64(x, sx, w[0], sw[0])
        check(y, ref, 3.01 * U32 * ref.abs(), torch.float32)
        assert torch.equal(y, O.i8_matmul(O.I8Rows(x, sx), O.I8Rows(w[0], sw[0])))
        (x, sx), (w, sw) = codes(g, M, 1), codes(g, 4, 1, 1)
        y = O.grouped_matmul(O.I8Rows(x, sx), O.I8Rows(w, sw), offsets_of([0, M // 2, 0, M - M // 2]))
        ref = torch.cat([product64(x[:M // 2], sx[:M // 2], w[1], sw[1]), product64(x[M // 2:], sx[M // 2:], w[3], sw[3])])
        check(y, ref, 3.01 * U32 * ref.abs(), torch.float32)


# ---- products -----------------------------------------------------------------

def product64(q, s, w, sw):
    return (q.double() @ w.double().transpose(-1, -2)) * s.double().unsqueeze(-1) * sw.double()


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (1, 1792, 4096), (2, 129, 15), (3, 517, 1003), (5, 2, 16), (7, 64, 31), (8, 1000, 4096),
                                   (9, 128, 128), (16, 129, 127), (31, 1, 33), (33, 517, 129), (64, 384, 1003), (77, 517, 1003),
                                   (100, 100, 100), (255, 130, 64), (257, 300, 256), (300, 4096, 1792), (1025, 257, 513),
                                   (2048, 1792, 4096), (40, 70, 65536)])
def test_i8_matmul(O, out, T, N, K):
    g = rng(T + N + K)
    (x, sx), (w, sw) = codes(g, T, K), codes(g, N, K, ld=(K + 15) // 16 * 16 + 16)
    if out == "f16":
        sx = sx * 2.0 ** -14    # stay below 65504
    bias = randn(g, N) if (T + N) % 2 else None
    buf = torch.full((T, N + 3), GUARD, dtype=DT[out], device="cuda")
    y = O.i8_matmul(O.I8Rows(x, sx), O.I8Rows(w, sw), bias=bias, out_dtype=DT[out], out=buf[:, :N])
    ref = product64(x, sx, w, sw)
    err = 3.01 * U32 * ref.abs()                     # the sum's conversion, two products
    if bias is not None:
        ref = ref + bias.double()
        err = err + U32 * ref.abs()
    check(y, ref, err, DT[out])
    assert bool((buf[:, N:] == GUARD).all())
    assert torch.equal(y, O.i8_matmul(O.I8Rows(x, sx), O.I8Rows(w, sw), bias=bias, out_dtype=DT[out]))
    assert O.status() == 0


def test_i8_matmul_exact_sums(O):
    """Unit scales: sums below 2^24 come out exactly, the extreme codes among them."""
    for T in (1, 8, 64, 300):
        x = torch.full((T, 1000), -128, dtype=torch.int8, device="cuda")
        x = torch.nn.functional.pad(x, (0, 8))[:, :1000]
        w = torch.nn.functional.pad(torch.full((130, 1000), -128, dtype=torch.int8, device="cuda"), (0, 8), value=1)[:, :1000]
        w[::2] = 127
        y = O.i8_matmul(O.I8Rows(x, torch.ones(T, device="cuda")), O.I8Rows(w, torch.ones(130, device="cuda")))
        assert torch.equal(y.double(), x.double() @ w.double().T)


@pytest.mark.parametrize("T,N,K", [(1, 300, 512), (4, 130, 1003), (20, 517, 2048), (300, 300, 256), (2100, 2050, 256)])
def test_i8_matmul_scales_in_order(O, T, N, K):
    """((sum * sx) * sw) + bias, each step one fp32 rounding: the same bits from every form of the product."""
    g = rng(T * N)
    (x, sx), (w, sw), bias = codes(g, T, K), codes(g, N, K), randn(g, N)
    s = (x.double() @ w.double().T).float()
    want = s * sx.unsqueeze(1) * sw + bias
    assert torch.equal(O.i8_matmul(O.I8Rows(x, sx), O.I8Rows(w, sw), bias=bias), want)
    y = O.grouped_matmul(O.I8Rows(x, sx), O.I8Rows(w.unsqueeze(0), sw.unsqueeze(0)), offsets_of([T]))
    assert torch.equal(y, s * sx.unsqueeze(1) * sw)


def test_i8_matmul_nan_rows_and_empty(O):
    for T in (6, 60):
        (x, sx), (w, sw) = codes(rng(T), T, 256), codes(rng(9), 200, 256)
        clean = O.i8_matmul(O.I8Rows(x, sx), O.I8Rows(w, sw))
        x2, s2 = x.clone(), sx.clone()
        x2[3], s2[3] = 0, float("nan")
        y = O.i8_matmul(O.I8Rows(x2, s2), O.I8Rows(w, sw))
        keep = [i for i in range(T) if i != 3]
        assert bool(y[3].isnan().all()) and torch.equal(y[keep], clean[keep])
    assert O.i8_matmul(O.I8Rows(x[:0], sx[:0]), O.I8Rows(w, sw)).shape == (0, 200)


def offsets_of(counts, lead=0):
    return torch.tensor(np.concatenate([[lead], lead + np.cumsum(counts)]), dtype=torch.int32, device="cuda")


GROUPS = [
    ("one", [5], 0, 0), ("one big", [700], 0, 0), ("decode", [0, 1, 0, 0, 1, 1, 0, 1], 0, 0), ("two of one", [0, 2, 0, 6], 0, 0),
    ("small", [3, 0, 9, 1, 0, 20], 0, 0), ("lead and tail", [4, 0, 30, 2], 3, 5), ("tail at decode", [2, 0, 1], 1, 3),
    ("ragged", [0, 1, 17, 255, 256, 257, 0, 33, 513, 31], 0, 0), ("none", [0, 0, 0], 2, 10), ("none at decode", [0, 0], 0, 4),
    ("many", [i % 5 for i in range(1024)], 0, 7),
]


def grouped64(x, w, off):
    y = torch.full((x.shape[0], w.shape[1]), float("nan"), dtype=torch.float64, device="cuda")
    o = off.tolist()
    for e in range(w.shape[0]):
        if o[e + 1] > o[e]:
            y[o[e]:o[e + 1]] = x[o[e]:o[e + 1]].double() @ w[e].double().T
    return y


@pytest.mark.parametrize("kind,out", [("i8", "f32"), ("i8", "bf16"), ("i8", "f16"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("N,K", [(130, 72), (256, 512), (37, 1003)])
@pytest.mark.parametrize("name,counts,lead,tail", GROUPS, ids=[g[0] for g in GROUPS])
def test_grouped(O, kind, out, N, K, name, counts, lead, tail):
    if name == "many" and K == 1003:
        N, K = 20, 33
    M, E = lead + sum(counts) + tail, len(counts)
    off = offsets_of(counts, lead)
    g = rng(M + N)
    buf = torch.full((M, N + 1), GUARD, dtype=DT[out], device="cuda")
    rows = (torch.arange(M, device="cuda") >= lead) & (torch.arange(M, device="cuda") < lead + sum(counts))
    if kind == "i8":
        (x, sx), (w, sw) = codes(g, M, K), codes(g, E, N, K)
        sx = sx * 2.0 ** -12
        y = O.grouped_matmul(O.I8Rows(x, sx), O.I8Rows(w, sw), off, out_dtype=DT[out], out=buf[:, :N])
        ref = grouped64(x.double() * sx.double().unsqueeze(-1), w.double() * sw.double().unsqueeze(-1), off)
        err = 3.01 * U32 * ref.abs() + 2.0 ** -45 * ref.abs()       # the reference's own 64-bit sum is not exact here
        err = err + 2.0 ** -40 * grouped64(x.double().abs() * sx.double().unsqueeze(-1),
                                           w.double().abs() * sw.double().unsqueeze(-1), off)
    else:
        pad = -K % 8 + 8
        x, w = randn(g, M, K, dtype=DT[kind], ld=K + pad), randn(g, E, N, K, dtype=DT[kind], ld=K + pad)
        x[~rows] = float("nan")                                       # never seen by the groups
        y = O.grouped_matmul(x, w, off, out_dtype=DT[out], out=buf[:, :N])
        ref = grouped64(x, w, off)
        # K fp32 additions, each at most one step (2^-23) of the sum of magnitudes, whatever their order
        err = K * 2.0 ** -23 * grouped64(x.double().abs(), w.double().abs(), off)
    check(y[rows], ref[rows], err[rows], DT[out])
    assert bool((buf[~rows] == GUARD).all()) and bool((buf[:, N:] == GUARD).all())
    assert O.status() == 0


def pair_tiles(M, N, E=1):
    """The host's rule: products whose tiles of 256 channels fill the SMs more than once go to pairs of CTAs."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return -(-N // 256) * max(min(E, M), -(-M // 256)) > sms // 2


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,N,K", [(2100, 2050, 1003), (4001, 1300, 272), (700, 7000, 130), (2600, 4096, 1792)])
def test_pairs_dense(O, out, T, N, K):
    """Pairs of CTAs: several tiles a pair (accumulators handed back and forth), tiles of up to 256 rows, a bias."""
    assert pair_tiles(T, N)
    g = rng(T + K)
    (x, sx), (w, sw), bias = codes(g, T, K), codes(g, N, K), randn(g, N)
    sx = sx * 2.0 ** -14
    buf = torch.full((T, N + 3), GUARD, dtype=DT[out], device="cuda")
    O.i8_matmul(O.I8Rows(x, sx), O.I8Rows(w, sw), bias=bias, out_dtype=DT[out], out=buf[:, :N])
    ref = product64(x, sx, w, sw)
    check(buf[:, :N], ref + bias.double(), 3.01 * U32 * ref.abs() + U32 * (ref + bias.double()).abs(), DT[out])
    assert bool((buf[:, N:] == GUARD).all()) and O.status() == 0


@pytest.mark.parametrize("kind,out", [("i8", "f32"), ("i8", "bf16"), ("i8", "f16"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("N,K", [(1000, 1003), (2048, 256)])
def test_pairs_grouped(O, kind, out, N, K):
    """Pairs of CTAs on ragged groups: none, one and several row tiles a group, tiles of 32 to 256 rows."""
    counts = [0, 700, 1, 33, 64, 0, 65, 129, 257, 512, 513, 31, 255, 256, 97, 0, 300, 2, 40, 161]
    lead, tail, E = 5, 9, len(counts)
    M = lead + sum(counts) + tail
    assert pair_tiles(M, N, E)
    off, g = offsets_of(counts, lead), rng(N + K)
    rows = slice(lead, M - tail)
    buf = torch.full((M, N + 1), GUARD, dtype=DT[out], device="cuda")
    if kind == "i8":
        (x, sx), (w, sw) = codes(g, M, K), codes(g, E, N, K)
        sx = sx * 2.0 ** -14
        O.grouped_matmul(O.I8Rows(x, sx), O.I8Rows(w, sw), off, out_dtype=DT[out], out=buf[:, :N])
        ref = grouped64(x, w, off) * sx.double().unsqueeze(-1)      # whole numbers below 2^53, then two products
        ref = ref * torch.cat([sw[0].expand(lead, N)] + [sw[e].expand(c, N) for e, c in enumerate(counts)] +
                              [sw[0].expand(tail, N)]).double()
        err = 3.01 * U32 * ref.abs()
    else:
        pad = -K % 8
        x, w = randn(g, M, K, dtype=DT[kind], ld=K + pad), randn(g, E, N, K, dtype=DT[kind], ld=K + pad)
        O.grouped_matmul(x, w, off, out_dtype=DT[out], out=buf[:, :N])
        ref = grouped64(x, w, off)
        err = K * 2.0 ** -23 * grouped64(x.double().abs(), w.double().abs(), off)       # as in test_grouped
    check(buf[rows, :N], ref[rows], err[rows], DT[out])
    assert bool((buf[:lead] == GUARD).all()) and bool((buf[M - tail:] == GUARD).all()) and bool((buf[:, N:] == GUARD).all())
    assert O.status() == 0


@pytest.mark.parametrize("M", [6, 300])
def test_grouped_bad_offsets(O, M):
    """Offsets out of range are clamped, and raised to the largest before them."""
    g = rng(M)
    (x, sx), (w, sw) = codes(g, M, 64), codes(g, 6, 50, 64)
    for bad in ([-5, 2, 2 ** 31 - 1, 3, -2 ** 31, 5, 2 ** 30], [0, 1, 0, 1, 0, M - 1, 2], [4, 2, 3, -1, 5, 4, 4],
                [2 ** 31 - 1, 0, 0, 0, 0, 0, M]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        c = np.maximum.accumulate(np.clip(np.array(bad), 0, M))
        buf = torch.full((M, 50), GUARD, device="cuda")
        O.grouped_matmul(O.I8Rows(x, sx), O.I8Rows(w, sw), off, out=buf)
        for e in range(6):
            r = slice(int(c[e]), int(c[e + 1]))
            ref = product64(x[r], sx[r], w[e], sw[e])
            check(buf[r], ref, 3.01 * U32 * ref.abs(), torch.float32)
        assert bool((buf[:int(c[0])] == GUARD).all()) and bool((buf[int(c[6]):] == GUARD).all())


def test_grouped_infinities_stay_in_their_rows(O):
    g = rng(2)
    for M in (8, 90):
        x, w = randn(g, M, 96, dtype=torch.bfloat16), randn(g, 3, 70, 96, dtype=torch.bfloat16)
        off = offsets_of([2, M - 5, 3])
        clean = O.grouped_matmul(x, w, off)
        x2 = x.clone()
        x2[1, 5], x2[M - 1, 95] = float("inf"), float("nan")
        y = O.grouped_matmul(x2, w, off)
        keep = [i for i in range(M) if i not in (1, M - 1)]
        assert torch.equal(y[keep], clean[keep])
        assert not bool(y[1].isfinite().any()) and bool(y[M - 1].isnan().all())


def test_grouped_far_experts(O):
    """Expert matrices whose offsets pass 32 bits of elements."""
    E, N, K = 9, 16384, 32768
    w = torch.empty(E, N, K, dtype=torch.int8, device="cuda")
    w.random_(-127, 128, generator=rng(1))
    sw = torch.full((E, N), 2.0 ** -10, device="cuda")
    for counts in ([0, 0, 0, 0, 0, 0, 0, 0, 3], [0, 0, 0, 0, 0, 0, 0, 0, 20]):
        (x, sx) = codes(rng(2), sum(counts), K)
        y = O.grouped_matmul(O.I8Rows(x, sx), O.I8Rows(w, sw), offsets_of(counts))
        ref = product64(x, sx, w[8, -300:], sw[8, -300:])
        check(y[:, -300:], ref, 3.01 * U32 * ref.abs(), torch.float32)


# ---- in use -------------------------------------------------------------------

def expert_block(O, E, s):
    """Pre-norm to codes, D, router, bucketing, the experts, U, post-norm with gate and residual."""
    xq = O.rms_norm_i8(s["h"], s["pre"])
    z = O.i8_matmul(xq, s["D"])
    idx, wts, _ = E.router_topk(z, s["router"], None, s["k"])
    _, off, perm, pos = E.route_bucket(idx, s["E"])
    zq = O.quantize_i8(z, index=perm, index_div=s["k"])
    gu = O.grouped_matmul(zq, s["gate_up"], off, out_dtype=torch.bfloat16)
    o = O.grouped_matmul(O.swiglu_i8(gu), s["down"], off, out_dtype=torch.bfloat16)
    y = O.i8_matmul(O.combine_i8(o, pos, wts), s["U"], out_dtype=torch.bfloat16)
    h, n = O.residual_norm(s["h"], y, s["post"], gate=s["gate"], next_weight=s["pre"], next_dtype=torch.int8)
    return h, n.dequantize(), (xq, z, idx, wts, off, perm, pos, zq, gu, o, y)


def block_state(O, T, H=512, L=256, I=256, E=8, k=2, seed=0):
    g = rng(seed)
    w = lambda *s: O.quantize_i8(randn(g, *s) * s[-1] ** -0.5)
    return dict(h=randn(g, T, H), pre=1 + 0.1 * randn(g, H), post=1 + 0.1 * randn(g, H), gate=randn(g, H), k=k, E=E,
                router=randn(g, E, L) * L ** -0.5, D=w(L, H), U=w(H, L), gate_up=w(E, 2 * I, L), down=w(E, L, I))


@pytest.mark.parametrize("T", [1, 4, 16, 129])
def test_whole_block(O, T):
    """The calls in a row, as a serving step makes them: each step's output against the formula on the
    step's own inputs, so that a wrong pairing of rows, experts or scales shows at once."""
    from quantized_latent_moe_b200 import elq
    s = block_state(O, T)
    h, n, (xq, z, idx, wts, off, perm, pos, zq, gu, o, y) = expert_block(O, elq, s)
    deq = lambda r: r.q.double() * r.scale.double().unsqueeze(-1)
    k = s["k"]
    zref = deq(xq) @ deq(s["D"]).T
    assert bool(((z.double() - zref).abs() <= 4 * U32 * zref.abs() + 1e-12).all())
    tok = perm.long() // k
    exp = idx.reshape(-1)[perm.long()].long()
    assert torch.equal(zq.q.double(), codes64(z)[0][tok])
    gref = torch.einsum("mk,mnk->mn", deq(zq), deq(s["gate_up"])[exp])
    check(gu, gref, 4 * U32 * gref.abs() + 1e-12, torch.bfloat16)
    hq = O.swiglu_i8(gu)
    oref = torch.einsum("mk,mnk->mn", deq(hq), deq(s["down"])[exp])
    check(o, oref, 4 * U32 * oref.abs() + 1e-12, torch.bfloat16)
    yq = O.combine_i8(o, pos, wts)
    assert bool(((deq(yq) - (o.double()[pos.long()].view(T, k, -1) * wts.double().unsqueeze(-1)).sum(1)).abs()
                 <= 0.51 * yq.scale.double().unsqueeze(-1)).all())
    yref = deq(yq) @ deq(s["U"]).T
    check(y, yref, 4 * U32 * yref.abs() + 1e-12, torch.bfloat16)
    href = s["h"].double() + s["gate"].double() * rms64(y, s["post"], 1e-6)
    assert bool(((h.double() - href).abs() <= (NORM + 4 * U32) * (href.abs() + s["h"].double().abs() * 2)).all())
    assert n.shape == h.shape and O.status() == 0


@pytest.mark.parametrize("T", [1, 24])
def test_captured_and_replayed(O, T):
    """Graphs of whole blocks, two of them replayed on two streams at once, give what eager calls give."""
    from quantized_latent_moe_b200 import elq
    states = [block_state(O, T, seed=i) for i in (1, 2)]
    want = [expert_block(O, elq, s)[:2] for s in states]
    torch.cuda.synchronize()
    streams, graphs, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [], []
    for s, st in zip(states, streams):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            outs.append(expert_block(O, elq, s)[:2])
        graphs.append(gr)
    for s in states:        # new inputs in the same buffers
        s["h"].mul_(-0.5)
    want = [expert_block(O, elq, s)[:2] for s in states]
    torch.cuda.synchronize()
    for _ in range(3):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, outs):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_chains_of_calls(O):
    """Bursts of calls with nothing between them (gathered rows to codes, then the product that reads
    them; buffers come back from the allocator at once) give every time what the first call gave.  Rows
    of odd width and ragged experts on pairs of CTAs stopped such a chain when its kernels overlapped."""
    cases = []
    for T, k, E, N, K in ((647, 2, 128, 675, 1217), (33, 1, 8, 1073, 357), (300, 8, 32, 512, 256)):
        g = rng(T)
        idx = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.reshape(-1)
        perm = torch.argsort(idx, stable=True).to(torch.int32)
        off = torch.searchsorted(idx.sort().values, torch.arange(E + 1, device="cuda")).to(torch.int32)
        x, (w, sw) = randn(g, T, K, dtype=torch.bfloat16), codes(g, E, N, K)
        cases.append(lambda x=x, w=w, sw=sw, off=off, perm=perm, k=k: O.grouped_matmul(
            O.quantize_i8(x, index=perm, index_div=k), O.I8Rows(w, sw * 2.0 ** -12), off, out_dtype=torch.float16))
    for T, N, K in ((77, 517, 1003), (300, 700, 130), (2048, 1792, 512)):
        g = rng(T)
        x, (w, sw) = randn(g, T, K), codes(g, N, K)
        cases.append(lambda x=x, w=w, sw=sw: O.i8_matmul(O.quantize_i8(x), O.I8Rows(w, sw)))
    for call in cases:
        want = call()
        torch.cuda.synchronize()
        for burst in (8, 8, 8, 300):
            for _ in range(burst):
                y = call()
            torch.cuda.synchronize()
            assert torch.equal(y, want)
    assert O.status() == 0


def test_two_streams_at_once(O):
    """Products on two streams at once: pairs of CTAs against clusters that split K, and both against row
    kernels, each giving what it gives alone."""
    g = rng(77)
    x, w = O.quantize_i8(randn(g, 2048, 1024)), O.quantize_i8(randn(g, 2048, 1024))
    xs, ws = randn(g, 40, 2048), O.quantize_i8(randn(g, 1000, 2048))
    big = lambda: O.i8_matmul(x, w, out_dtype=torch.bfloat16)
    small = lambda: O.i8_matmul(O.quantize_i8(xs), ws)
    want = big(), small()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        got = [[], []]
        for i in range(10):
            for j, call in enumerate((big, small)):
                with torch.cuda.stream(streams[j]):
                    got[j].append(call())
        torch.cuda.synchronize()
        for j in range(2):
            assert all(torch.equal(y, want[j]) for y in got[j])
    assert O.status() == 0


def test_pairs_on_two_streams(O):
    """Products on pairs of CTAs on one stream, on the other products of clusters that split K, row kernels, and
    pairs again: each gives what it gives alone."""
    g = rng(78)
    assert pair_tiles(2500, 2304) and not pair_tiles(40, 1000)
    x, w = O.quantize_i8(randn(g, 2500, 512)), O.quantize_i8(randn(g, 2304, 512))
    xs, ws = randn(g, 40, 2048), O.quantize_i8(randn(g, 1000, 2048))
    big = lambda: O.i8_matmul(x, w, out_dtype=torch.bfloat16)
    calls = [[big], [lambda: O.i8_matmul(O.quantize_i8(xs), ws), big]]
    want = [[c() for c in cs] for cs in calls]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        got = [[], []]
        for i in range(10):
            for j in range(2):
                with torch.cuda.stream(streams[j]):
                    got[j].append([c() for c in calls[j]])
        torch.cuda.synchronize()
        for j in range(2):
            assert all(torch.equal(a, b) for ys in got[j] for a, b in zip(ys, want[j]))
    assert O.status() == 0


def pointers(O, x, w, y):
    return (x.q.data_ptr(), x.q.stride(0), x.scale.data_ptr(), x.q.shape[0], w.q.data_ptr(), w.q.stride(0), w.scale.data_ptr(),
            w.q.shape[0], x.q.shape[1], y.data_ptr(), y.stride(0))


@pytest.mark.parametrize("T,N,K,stall", [(16, 300, 2048, 1), (2048, 1792, 1024, 1), (2500, 2304, 1024, 1), (2500, 2304, 64, 1),
                                         (8192, 4096, 1024, 2)])
def test_wait_that_runs_out(O, T, N, K, stall):
    """A product whose device wait cannot end (split over K, single CTAs, pairs): it comes back within its limits, the
    error word says so once, and the next product is right."""
    import ctypes
    g = rng(T + N)
    x, w = O.quantize_i8(randn(g, T, K)), O.quantize_i8(randn(g, N, K))
    want, y = O.i8_matmul(x, w), torch.empty(T, N, device="cuda")
    assert O.status() == 0
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert O.lib().elq_test_i8_matmul_timeout(*pointers(O, x, w, y), stall, 20_000_000, stream) == 0
    assert O.status() == -6 and O.status() == 0
    assert torch.equal(O.i8_matmul(x, w), want) and O.status() == 0


def test_status_waits_for_its_own_stream_only(O):
    """While the default stream is busy, another stream's status comes back; what the default stream's product sets
    after that is still reported."""
    import ctypes
    side, (x, w) = torch.cuda.Stream(), (O.quantize_i8(torch.randn(16, 512, device="cuda")), O.quantize_i8(torch.randn(300, 512, device="cuda")))
    y, done = O.i8_matmul(x, w), torch.cuda.Event()
    assert O.status(stream=side) == 0       # the first use of a kernel loads it, which may wait for the device
    torch.cuda._sleep(1_000_000_000)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert O.lib().elq_test_i8_matmul_timeout(*pointers(O, x, w, y), 1, 5_000_000, stream) == 0
    done.record()
    seen = O.status(stream=side)
    assert seen == 0 and not done.query()
    reports = 0
    while not done.query():
        reports += O.status(stream=side) == -6
    reports += O.status() == -6
    assert reports == 1 and O.status() == 0


def test_stream_argument(O):
    st = torch.cuda.Stream()
    g = rng(8)
    x, w = randn(g, 300, 512), randn(g, 256, 512)
    wq = O.quantize_i8(w)
    want = O.i8_matmul(O.quantize_i8(x), wq)
    st.wait_stream(torch.cuda.current_stream())
    got = O.i8_matmul(O.quantize_i8(x, stream=st), wq, stream=st)
    st.synchronize()
    assert torch.equal(got, want)


def test_stream_argument_keeps_inputs(O):
    """Inputs dropped right after a call on another stream keep their memory until that stream has read them."""
    side, g, n = torch.cuda.Stream(), rng(9), 1 << 22
    w = O.quantize_i8(randn(g, 64, 1024))
    calls = [lambda t: O.quantize_i8(t, stream=side), lambda t: O.rms_norm(t, stream=side),
             lambda t: O.residual_norm(t, t, next_dtype=torch.int8, stream=side)]
    make = lambda: torch.ones(n // 1024, 1024, device="cuda")
    for call in calls:
        call(make())                                    # kernels loaded, streams known to the allocator
    O.i8_matmul(O.quantize_i8(make()), w, stream=side)
    torch.cuda.synchronize()
    for call in calls:
        t = make()
        at = t.data_ptr()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)
        call(t)
        del t
        assert make().data_ptr() != at
        torch.cuda.synchronize()
    xq = O.quantize_i8(make())
    at = xq.q.data_ptr()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    O.i8_matmul(xq, w, stream=side)
    del xq
    assert O.quantize_i8(make()).q.data_ptr() != at
    torch.cuda.synchronize()


def test_stream_argument_in_a_capture(O):
    """Calls that name the stream being captured, their intermediates dropped as they go, replay as eager calls."""
    st, g = torch.cuda.Stream(), rng(10)
    x, w = randn(g, 40, 512), O.quantize_i8(randn(g, 256, 512))
    call = lambda: O.i8_matmul(O.rms_norm_i8(x, stream=st), w, stream=st)
    call()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=st):
        y = call()
        z = O.i8_matmul(O.quantize_i8(y, stream=st), O.I8Rows(w.q[:, :256], w.scale), stream=st)
    x.mul_(-2)
    torch.cuda.synchronize()
    for _ in range(3):
        gr.replay()
    torch.cuda.synchronize()
    want = call()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(z, O.i8_matmul(O.quantize_i8(want), O.I8Rows(w.q[:, :256], w.scale)))


def test_out_counts_as_written_in_place(O):
    """A backward pass that saved what a call then writes raises, and does not use the new values."""
    h, y = torch.randn(4, 64, device="cuda"), torch.randn(4, 64, device="cuda")
    w = torch.ones(4, 64, device="cuda", requires_grad=True)
    (xq, m), off = (O.quantize_i8(h), O.quantize_i8(torch.randn(64, 64, device="cuda"))), offsets_of([4])
    for write in (lambda: O.rms_norm(h, out=h), lambda: O.residual_norm(h, y, out=h), lambda: O.i8_matmul(xq, m, out=h),
                  lambda: O.grouped_matmul(xq, O.I8Rows(m.q.unsqueeze(0), m.scale.unsqueeze(0)), off, out=h)):
        loss = (w * h).sum()
        before = h._version
        write()
        assert h._version > before
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    with torch.inference_mode():
        t = torch.randn(4, 64, device="cuda")
        O.rms_norm(t, out=t)
    O.rms_norm(t, out=t)


def test_binding_refusals(O):
    from quantized_latent_moe_b200.elq import ElqError
    g = rng(1)
    x = randn(g, 8, 64)
    xq, w = O.quantize_i8(x), O.quantize_i8(randn(g, 32, 64))
    off = offsets_of([8])
    bad = [lambda: O.quantize_i8(x.t()), lambda: O.quantize_i8(x, index=torch.zeros(3, device="cuda")),
           lambda: O.quantize_i8(x[:, 1:]),                                   # not 16-byte aligned
           lambda: O.quantize_i8(x[:1].expand(8, 64)), lambda: O.swiglu_i8(x[:, :63]),
           lambda: O.i8_matmul(xq, O.quantize_i8(randn(g, 32, 48))), lambda: O.i8_matmul(xq, w, bias=x[0]),
           lambda: O.i8_matmul(xq, w, out=torch.empty(8, 31, device="cuda")), lambda: O.i8_matmul(xq, w, out_dtype=torch.int8),
           lambda: O.grouped_matmul(xq, O.I8Rows(w.q.view(1, 32, 64), w.scale), off.long()),
           lambda: O.grouped_matmul(xq, O.I8Rows(w.q.view(2, 16, 64), w.scale), off),
           lambda: O.grouped_matmul(x, x.view(1, 8, 64), off),
           lambda: O.grouped_matmul(x.half(), x.bfloat16().view(1, 8, 64), off),
           lambda: O.grouped_matmul(x.half(), x.half().view(1, 8, 64), off, out_dtype=torch.bfloat16),
           lambda: O.grouped_matmul(x.half()[:, :60].contiguous(), x.half()[:, :60].contiguous().view(1, 8, 60), off),
           lambda: O.rms_norm(x, weight=x[0, :32]), lambda: O.rms_norm(x, eps=0.0), lambda: O.rms_norm(x, out_dtype=torch.int8),
           lambda: O.residual_norm(x, x[:4]), lambda: O.residual_norm(x, x.clone(), gate=x[:3]),
           lambda: O.residual_norm(x, x.clone(), gate=x[:3], gate_rows=2), lambda: O.residual_norm(x, x.clone(), gate=x[:, :5]),
           lambda: O.residual_norm(x, x.clone(), out=x.clone()[:, :32]),
           lambda: O.combine_i8(x, torch.zeros(3, dtype=torch.int32, device="cuda"), torch.ones(2, 2, device="cuda"))]
    for i, call in enumerate(bad):
        with pytest.raises(ElqError):
            call()
            raise AssertionError("call %d was not refused" % i)
