"""The 8-bit-integer expert path and the norms around it, operator by operator.

Each case is one pass a serving program makes over this library's layer shapes
(hidden 4096, latent 1792, 128 experts top-8, expert width 1024, and the small
512 / 256 / 8 top-2 / 256 layer), from one token to thousands:

  norm     h' = res_scale * h + gate * rms(y) * w_post, and the next block's
           input rms(h') * w_pre, in one pass (residual_norm)
  codes    the norm before a block handed on as 8-bit codes, and the product
           of those codes with a weight matrix (rms_norm_i8, i8_matmul)
  linear   rows quantised with one scale a token, times a matrix of 8-bit
           codes with one scale a channel (quantize_i8, i8_matmul)
  experts  rows sorted by expert times their expert's matrix, ragged groups
           (grouped_matmul), in bf16, fp16, or 8-bit codes of gathered tokens
  mlp      the experts whole: gather and quantise, gate/up, SwiGLU and
           quantise, down, weighted combine and quantise, U projection

With `own` false run() computes them from elementary torch operations in
32 bits (quotients next to a rounding border in 64).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ---- cases --------------------------------------------------------------------

def listed():
    return [
        # one decoded token's residual update between two blocks: launch latency
        {"name": "norm decode", "op": "norm", "T": 1, "C": 4096, "h": "f32", "y": "f32", "n": "bf16",
         "gate": "channel", "pad": 0},
        # a prefill's residual stream held in bf16
        {"name": "norm prefill", "op": "norm", "T": 2048, "C": 4096, "h": "bf16", "y": "bf16", "n": "bf16",
         "gate": "channel", "pad": 0},
        # odd width, rows that are slices of wider ones, one gate value a token
        {"name": "norm odd", "op": "norm", "T": 777, "C": 1283, "h": "f16", "y": "f16", "n": "f16", "gate": "token",
         "pad": 6},
        # a verify step of six tokens: norm before the block, D projection of its codes
        {"name": "codes verify", "op": "codes", "T": 6, "K": 4096, "N": 1792, "x": "f32", "out": "bf16"},
        # one decoded token's D projection (fp32 latent for the router)
        {"name": "linear decode", "op": "linear", "T": 1, "K": 4096, "N": 1792, "x": "bf16", "out": "f32",
         "bias": False},
        # odd sizes: a batch that fills no tile, a bias
        {"name": "linear odd", "op": "linear", "T": 77, "K": 1003, "N": 517, "x": "f16", "out": "f16", "bias": True},
        # the U projection of a prefill
        {"name": "linear prefill", "op": "linear", "T": 2048, "K": 1792, "N": 4096, "x": "f32", "out": "bf16",
         "bias": False},
        # a long prompt through a square projection: the largest product
        {"name": "linear large", "op": "linear", "T": 8192, "K": 4096, "N": 4096, "x": "bf16", "out": "bf16",
         "bias": False},
        # one token's eight experts, gate and up
        {"name": "experts decode", "op": "experts", "T": 1, "k": 8, "E": 128, "K": 1792, "N": 2048, "x": "i8",
         "out": "bf16", "skew": 0.0},
        # a prefill's experts, gate and up, skewed routing
        {"name": "experts prefill", "op": "experts", "T": 2048, "k": 8, "E": 128, "K": 1792, "N": 2048, "x": "i8",
         "out": "bf16", "skew": 0.33},
        # the same prefill's down product in bf16
        {"name": "experts bf16", "op": "experts", "T": 2048, "k": 8, "E": 128, "K": 1024, "N": 1792, "x": "bf16",
         "out": "bf16", "skew": 0.33},
        # 32 sequences' next tokens through all of the experts and U
        {"name": "mlp batch", "op": "mlp", "T": 32, "k": 8, "E": 128, "L": 1792, "I": 1024, "H": 4096, "skew": 0.33},
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, even over the logarithm; half of them odd."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, n if rng.random() < 0.5 else n | 1))


def draw(rng):
    op = rng.choice(["norm", "codes", "linear", "experts", "experts", "mlp"])
    if op == "norm":
        t = rng.choice(["f32", "bf16", "f16"])
        return {"op": op, "T": _size(rng, 1, 2048), "C": _size(rng, 256, 4096), "h": rng.choice([t, "f32"]), "y": t,
                "n": rng.choice(["f32", "bf16", "f16"]), "gate": rng.choice(["channel", "token", "full", "none"]),
                "pad": rng.choice([0, 8, 3])}
    if op == "codes":
        return {"op": op, "T": _size(rng, 1, 2048), "K": _size(rng, 256, 4096), "N": _size(rng, 256, 4096),
                "x": rng.choice(list(DTYPES)), "out": rng.choice(["bf16", "f16"])}
    if op == "linear":
        return {"op": op, "T": _size(rng, 1, 4096), "K": _size(rng, 256, 4096), "N": _size(rng, 256, 4096),
                "x": rng.choice(list(DTYPES)), "out": rng.choice(list(DTYPES)), "bias": rng.random() < 0.5}
    if op == "experts":
        E = rng.choice([8, 32, 128])
        x = rng.choice(["i8", "bf16", "f16"])
        out = rng.choice(["f32", "bf16"] if x == "bf16" else ["f32", "f16"] if x == "f16" else list(DTYPES))
        return {"op": op, "T": _size(rng, 1, 1024), "k": rng.choice([1, 2, 8]), "E": E, "K": _size(rng, 256, 1792),
                "N": _size(rng, 256, 2048), "x": x, "out": out, "skew": rng.choice([0.0, 0.33, 1.0])}
    E, k = rng.choice([(8, 2), (32, 4), (128, 8)])
    return {"op": op, "T": _size(rng, 1, 128), "k": k, "E": E, "L": _size(rng, 256, 1792), "I": _size(rng, 256, 1024),
            "H": _size(rng, 512, 4096), "skew": rng.choice([0.0, 0.33, 1.0])}


# ---- inputs -------------------------------------------------------------------

class _Draws:
    """Normal draws on the GPU from one seed."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, std=1.0, dtype=torch.float32, pad=0):
        full = torch.randn(*shape[:-1], shape[-1] + pad, generator=self.g, device="cuda").mul_(std).to(dtype)
        return full[..., :shape[-1]] if pad else full


def _activations(d, T, C, dtype, pad=0):
    """A residual stream's rows: normal values, a few channels ten times as wide."""
    wide = torch.ones(C, device="cuda")
    wide[torch.randint(0, C, (max(1, C // 256),), generator=d.g, device="cuda")] = 10.0
    return (d.normal(T, C + pad) * torch.nn.functional.pad(wide, (0, pad), value=1.0)).to(dtype)[:, :C]


def _code_matrix(d, n, k, E=None):
    """Weights N(0, 0.02) as 8-bit codes with one scale a row, rows padded to whole 16 bytes."""
    shape = (n, k) if E is None else (E, n, k)
    w = d.normal(*shape, std=0.02)
    s = w.abs().amax(-1) / 127
    q = torch.zeros(*shape[:-1], (k + 15) // 16 * 16, dtype=torch.int8, device="cuda")
    q[..., :k] = torch.round(w / s[..., None]).to(torch.int8)
    return q[..., :k], s


def _routing(T, k, E, skew, seed):
    """Top-k of noisy skewed logits, bucketed by expert (a router's output): offsets, pairs in order of expert, each
    pair's place, softmax weights, and the largest group."""
    g = torch.Generator()
    g.manual_seed(seed)
    rank = torch.argsort(torch.randn(E, generator=g)) + 1
    logits = torch.randn(T, E, generator=g) - skew * torch.log(rank.float())
    top, idx = torch.topk(logits, k, dim=1)
    flat = idx.reshape(-1)
    perm = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64)
    offsets[1:] = torch.cumsum(counts, 0)
    pos = torch.empty_like(perm)
    pos[perm] = torch.arange(T * k)
    cu = lambda t: t.to(torch.int32).cuda()  # noqa: E731
    return {"offsets": cu(offsets), "perm": cu(perm), "pos": cu(pos), "weights": torch.softmax(top, 1).cuda(),
            "cap": int(counts.max())}


def prepare(case, seed):
    c, d = dict(case), _Draws(seed)
    s = {"case": c}
    if c["op"] == "norm":
        T, C, pad = c["T"], c["C"], c["pad"]
        s["h"] = _activations(d, T, C, DTYPES[c["h"]], pad)
        s["y"] = d.normal(T, C, std=0.5, pad=pad).to(DTYPES[c["y"]])
        s["post"] = 1 + d.normal(C, std=0.1)
        s["pre"] = 1 + d.normal(C, std=0.1)
        s["gate"] = {"none": lambda: None, "channel": lambda: d.normal(1, C, std=0.5),
                     "token": lambda: torch.sigmoid(d.normal(T, 1)), "full": lambda: d.normal(T, C, std=0.5)}[c["gate"]]()
        s["res_scale"] = 0.875
    elif c["op"] == "codes":
        s["x"] = _activations(d, c["T"], c["K"], DTYPES[c["x"]])
        s["pre"] = 1 + d.normal(c["K"], std=0.1)
        s["w"] = _code_matrix(d, c["N"], c["K"])
    elif c["op"] == "linear":
        s["x"] = _activations(d, c["T"], c["K"], DTYPES[c["x"]])
        s["w"] = _code_matrix(d, c["N"], c["K"])
        s["bias"] = d.normal(c["N"]) if c["bias"] else None
    elif c["op"] == "experts":
        s |= _routing(c["T"], c["k"], c["E"], c["skew"], seed)
        if c["x"] == "i8":
            s["x"] = _activations(d, c["T"], c["K"], torch.bfloat16)
            s["w"] = _code_matrix(d, c["N"], c["K"], c["E"])
        else:
            # rows already in order of expert, both padded to whole 16 bytes
            pad, t = -c["K"] % 8, DTYPES[c["x"]]
            s["x"] = d.normal(c["T"] * c["k"], c["K"], dtype=t, pad=pad)
            s["w"] = d.normal(c["E"], c["N"], c["K"], std=0.02, dtype=t, pad=pad)
    else:
        s |= _routing(c["T"], c["k"], c["E"], c["skew"], seed)
        s["z"] = _activations(d, c["T"], c["L"], torch.float32)
        s["gate_up"] = _code_matrix(d, 2 * c["I"], c["L"], c["E"])
        s["down"] = _code_matrix(d, c["L"], c["I"], c["E"])
        s["U"] = _code_matrix(d, c["H"], c["L"])
    return s


# ---- one pass -----------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    if own:
        from quantized_latent_moe_b200 import ops
        c = s["case"]
        if c["op"] == "norm":
            h, n = ops.residual_norm(s["h"], s["y"], s["post"], gate=s["gate"], res_scale=s["res_scale"],
                                     next_weight=s["pre"], eps=EPS, next_dtype=DTYPES[c["n"]])
            return {"h": h, "n": n}
        if c["op"] == "codes":
            return ops.i8_matmul(ops.rms_norm_i8(s["x"], s["pre"], eps=EPS), ops.I8Rows(*s["w"]),
                                 out_dtype=DTYPES[c["out"]])
        if c["op"] == "linear":
            return ops.i8_matmul(ops.quantize_i8(s["x"]), ops.I8Rows(*s["w"]), bias=s["bias"],
                                 out_dtype=DTYPES[c["out"]])
        if c["op"] == "experts":
            if c["x"] == "i8":
                x = ops.quantize_i8(s["x"], index=s["perm"], index_div=c["k"])
                return ops.grouped_matmul(x, ops.I8Rows(*s["w"]), s["offsets"], out_dtype=DTYPES[c["out"]])
            return ops.grouped_matmul(s["x"], s["w"], s["offsets"], out_dtype=DTYPES[c["out"]])
        x = ops.quantize_i8(s["z"], index=s["perm"], index_div=c["k"])
        gu = ops.grouped_matmul(x, ops.I8Rows(*s["gate_up"]), s["offsets"], out_dtype=torch.bfloat16)
        o = ops.grouped_matmul(ops.swiglu_i8(gu), ops.I8Rows(*s["down"]), s["offsets"], out_dtype=torch.bfloat16)
        return ops.i8_matmul(ops.combine_i8(o, s["pos"], s["weights"]), ops.I8Rows(*s["U"]), out_dtype=torch.bfloat16)


def _quantize(x):
    """Codes as fp32 whole numbers, and the scales: s = amax / 127, q = x / s to the nearest, halves away from zero."""
    s = (x.abs().amax(-1).double() / 127).float()
    r = x.double() / torch.where(s > 0, s, 1.0).double()[..., None]
    return (torch.sign(r) * torch.floor(r.abs() + 0.5)).float(), s


def _rms(x):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _i8_matmul(x, w):
    (qx, sx), (qw, sw) = x, w
    return (qx @ qw.float().T) * sx[:, None] * sw


def _grouped(x, w, s):
    """x's rows, in order of expert, times their expert's matrix w [E, N, K], the groups padded to the largest."""
    M, E = x.shape[0], w.shape[0]
    first, rows = s["offsets"][:-1].long(), torch.arange(M, device=x.device)
    expert = torch.searchsorted(s["offsets"][1:].long(), rows, right=True).clamp(max=E - 1)
    if M <= E // 2:     # few rows: each with a copy of its own expert's matrix
        return (w[expert].float() @ x.float()[..., None])[..., 0], expert
    slots = first[:, None] + torch.arange(s["cap"], device=x.device)
    y = torch.bmm(x.float()[slots.clamp(max=M - 1)], w.float().transpose(1, 2))
    return y[expert, rows - first[expert]], expert


def _grouped_i8(x, w, s):
    y, expert = _grouped(x[0], w[0], s)
    return y * x[1][:, None] * w[1][expert]


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        v = _rms(s["y"].float()) * s["post"]
        h = s["res_scale"] * s["h"].float() + (v if s["gate"] is None else s["gate"] * v)
        return {"h": h.to(s["h"].dtype), "n": (_rms(h) * s["pre"]).to(DTYPES[c["n"]])}
    if c["op"] == "codes":
        return _i8_matmul(_quantize(_rms(s["x"].float()) * s["pre"]), s["w"]).to(DTYPES[c["out"]])
    if c["op"] == "linear":
        y = _i8_matmul(_quantize(s["x"].float()), s["w"])
        return (y if s["bias"] is None else y + s["bias"]).to(DTYPES[c["out"]])
    if c["op"] == "experts":
        if c["x"] == "i8":
            x = _quantize(s["x"].float()[s["perm"].long() // c["k"]])
            return _grouped_i8(x, s["w"], s).to(DTYPES[c["out"]])
        return _grouped(s["x"], s["w"], s)[0].to(DTYPES[c["out"]])
    gu = _grouped_i8(_quantize(s["z"][s["perm"].long() // c["k"]]), s["gate_up"], s).to(torch.bfloat16).float()
    g, u = gu[:, :c["I"]], gu[:, c["I"]:]
    o = _grouped_i8(_quantize(g / (1 + torch.exp(-g)) * u), s["down"], s).to(torch.bfloat16).float()
    y = (o[s["pos"].long()].view(c["T"], c["k"], -1) * s["weights"][..., None]).sum(1)
    return _i8_matmul(_quantize(y), s["U"]).to(torch.bfloat16)


# ---- what a pass cannot do without ---------------------------------------------

def work(case):
    c = case
    b = {"f32": 4, "bf16": 2, "f16": 2, "i8": 1}
    if c["op"] == "norm":
        T, C = c["T"], c["C"]
        gate = {"none": 0, "channel": C, "token": T, "full": T * C}[c["gate"]] * 4
        return {"bytes": T * C * (2 * b[c["h"]] + b[c["y"]] + b[c["n"]]) + 8 * C + gate, "flops": 10 * T * C}
    if c["op"] in ("codes", "linear"):
        T, K, N = c["T"], c["K"], c["N"]
        return {"bytes": T * K * b[c["x"]] + N * K + 4 * N + T * N * b[c["out"]] + (4 * K if c["op"] == "codes" else 0),
                "flops": 2 * T * K * N}
    # the experts that T tokens reach: all of them, or as many as there are pairs
    hit = min(c["E"], c["T"] * c["k"])
    M = c["T"] * c["k"]
    if c["op"] == "experts":
        K, N = c["K"], c["N"]
        x = c["T"] * K * 2 if c["x"] == "i8" else M * K * 2
        return {"bytes": x + hit * N * (K * b[c["x"]] + (4 if c["x"] == "i8" else 0)) + M * N * b[c["out"]],
                "flops": 2 * M * K * N}
    L, I, H = c["L"], c["I"], c["H"]
    return {"bytes": c["T"] * L * 4 + hit * (3 * I * L + 4 * (2 * I + L)) + H * L + 4 * H + c["T"] * H * 2,
            "flops": 6 * M * I * L + 2 * c["T"] * H * L}


# ---- the definition in 64 bits ---------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]

    def codes(v):
        """What the codes of 64-bit rows stand for; the scale is the fp32 number that is stored."""
        scale = (v.abs().max(dim=1).values.float().double() / 127).float().double().unsqueeze(1)
        scale = torch.where(scale == 0, torch.ones_like(scale), scale)
        whole = torch.trunc(v / scale)
        up = ((v / scale - whole).abs() >= 0.5).double() * torch.sign(v)
        return (whole + up) * scale

    def norm(v, w):
        return v / torch.sqrt((v ** 2).sum(1, keepdim=True) / v.shape[1] + EPS) * w.double()

    def stands(w):
        return w[0].double() * w[1].double().unsqueeze(-1)

    def by_expert(rows, w):
        off = s["offsets"].tolist()
        n = (w[0] if isinstance(w, tuple) else w).shape[1]
        out = rows.new_zeros(rows.shape[0], n)
        for e in range(c["E"]):
            a, z = off[e], off[e + 1]
            if z > a:
                we = stands((w[0][e], w[1][e])) if isinstance(w, tuple) else w[e].double()
                out[a:z] = torch.einsum("mk,nk->mn", rows[a:z], we)
        return out

    if c["op"] == "norm":
        g = 1.0 if s["gate"] is None else s["gate"].double()
        h = s["h"].double() * s["res_scale"] + g * norm(s["y"].double(), s["post"])
        return {"h": h, "n": norm(h, s["pre"])}
    if c["op"] == "codes":
        return torch.einsum("mk,nk->mn", codes(norm(s["x"].double(), s["pre"])), stands(s["w"]))
    if c["op"] == "linear":
        y = torch.einsum("mk,nk->mn", codes(s["x"].double()), stands(s["w"]))
        return y if s["bias"] is None else y + s["bias"].double()
    if c["op"] == "experts":
        if c["x"] == "i8":
            return by_expert(codes(s["x"].double())[s["perm"].long() // c["k"]], s["w"])
        return by_expert(s["x"].double(), s["w"])
    # the expert rows are stored as bf16 between the products: their values are part of what is computed next
    pairs = codes(s["z"].double())[s["perm"].long() // c["k"]]
    gu = by_expert(pairs, s["gate_up"]).bfloat16().double()
    g, u = gu[:, :c["I"]], gu[:, c["I"]:]
    o = by_expert(codes(u * g * torch.sigmoid(g)), s["down"]).bfloat16().double()
    picked = o[s["pos"].long()].reshape(c["T"], c["k"], c["L"])
    return torch.einsum("mk,nk->mn", codes(torch.einsum("tkl,tk->tl", picked, s["weights"].double())), stands(s["U"]))
