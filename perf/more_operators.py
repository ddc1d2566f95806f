"""Microscaled 4-bit floating point and the layers it is stored for, in plain torch form, and the calls of the library
that compute the same: quantising rows and reading them back, the product of 4-bit activations with 4-bit weights, and
a whole mixture-of-experts layer for a few tokens.

A case is a dict of plain values; ``op`` says which operator it is:

* ``quant``: rows into the 4-bit form (``q4_mx_quant``, plain, behind an RMSNorm or behind a SwiGLU) and back into
  values (``q4_mx_dequant``);
* ``gemm``: rows quantised and multiplied with a 4-bit weight matrix, plus a residual (``q4_mx_gemm``);
* ``moe``: router, top-k, the chosen experts' SwiGLU MLPs and their weighted sum (``q4_moe``).

``fmt``: ``mx``, blocks of 32 values of E2M1 (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign) that share a power of two, the
smallest that keeps the block's largest value within 6; ``nv``, blocks of 16 that share an E4M3 factor, and one fp32
factor of the whole matrix.  Codes are stored two a byte (the even one in the low nibble).

Quantised values are returned in bf16, which holds every one of them (``mx``) or more than their precision (``nv``):
a value next to the border of two codes may take the other one where a norm's last bit differs.  For the same reason
the forms with a norm, a SwiGLU or a layer's inner quantisation give their results in 16 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = {"mx": 32, "nv": 16}
EPS = 1e-6


def listed():
    return [
        # a decode step's activations before its projections, the widest batch of the matrix-vector calls: latency
        {"name": "quant 16 x 4096 norm", "op": "quant", "fmt": "mx", "dtype": "bf16", "rows": 16, "k": 4096,
         "form": "norm"},
        # the rows of a few packed prompts before the projections
        {"name": "quant 8191 x 4096 norm nv", "op": "quant", "fmt": "nv", "dtype": "bf16", "rows": 8191, "k": 4096,
         "form": "norm"},
        # an fp32 weight matrix quantised when a model is loaded
        {"name": "quant 14336 x 4096 f32", "op": "quant", "fmt": "mx", "dtype": "f32", "rows": 14336, "k": 4096,
         "form": "plain"},
        # an MLP's activations before its down projection: gate and up are halves of one buffer
        {"name": "quant 1000 x 14336 glu", "op": "quant", "fmt": "mx", "dtype": "f16", "rows": 1000, "k": 14336,
         "form": "glu"},
        # one token's up projection
        {"name": "gemm 1 f32", "op": "gemm", "fmt": "mx", "dtype": "f32", "rows": 1, "n": 14336, "k": 4096,
         "form": "plain", "residual": False},
        # a decode batch's down projection onto the residual stream
        {"name": "gemm 16 nv", "op": "gemm", "fmt": "nv", "dtype": "bf16", "rows": 16, "n": 4096, "k": 14336,
         "form": "plain", "residual": True},
        # a short prompt, sizes that no tile divides
        {"name": "gemm 100 ragged f16", "op": "gemm", "fmt": "mx", "dtype": "f16", "rows": 100, "n": 5000, "k": 2080,
         "form": "norm", "residual": False},
        # a long prompt's up projection
        {"name": "gemm 4096 nv", "op": "gemm", "fmt": "nv", "dtype": "bf16", "rows": 4096, "n": 14336, "k": 4096,
         "form": "norm", "residual": False},
        # several prompts' down projection onto the residual stream
        {"name": "gemm 8191 mx", "op": "gemm", "fmt": "mx", "dtype": "bf16", "rows": 8191, "n": 4096, "k": 14336,
         "form": "plain", "residual": True},
        # one token through a layer of many small experts
        {"name": "moe 1 of 128 experts", "op": "moe", "fmt": "mx", "dtype": "bf16", "rows": 1, "experts": 128,
         "top_k": 8, "hidden": 2048, "inter": 768, "renormalize": True},
        # a decode batch through it: most experts have a token
        {"name": "moe 16 of 128 experts", "op": "moe", "fmt": "mx", "dtype": "bf16", "rows": 16, "experts": 128,
         "top_k": 8, "hidden": 2048, "inter": 768, "renormalize": True},
        # a few sequences through a layer of a few large experts
        {"name": "moe 4 of 8 experts", "op": "moe", "fmt": "mx", "dtype": "f16", "rows": 4, "experts": 8,
         "top_k": 2, "hidden": 4096, "inter": 14336, "renormalize": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A multiple of 32."""
    return 32 * _log_int(rng, lo // 32, hi // 32)


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "gemm", "moe", "moe"])
    fmt, dtype = rng.choice(["mx", "nv"]), rng.choice(["f32", "f16", "bf16"])
    if op == "quant":
        k = _width(rng, 32, 16384)
        return {"op": op, "fmt": fmt, "dtype": dtype, "rows": _log_int(rng, 1, min(16384, 50_000_000 // k)), "k": k,
                "form": rng.choice(["plain", "norm", "glu"])}
    if op == "gemm":
        n, k = _log_int(rng, 8, 14336), _width(rng, 32, 14336)
        return {"op": op, "fmt": fmt, "dtype": dtype, "rows": _log_int(rng, 1, 8191), "n": n, "k": k,
                "form": "plain" if dtype == "f32" else rng.choice(["plain", "norm", "glu"]),
                "residual": rng.choice([True, False])}
    hidden, inter = _width(rng, 128, 4096), _width(rng, 64, 8192)
    experts = _log_int(rng, 2, min(160, 400_000_000 // (hidden * inter)))
    top_k = rng.randint(1, min(8, experts))
    most = min(16, max(1, 1_000_000_000 // (top_k * hidden * inter)))  # the plain form has a copy for every choice
    return {"op": op, "fmt": "mx", "dtype": rng.choice(["f16", "bf16"]), "rows": rng.randint(1, most),
            "experts": experts, "top_k": top_k, "hidden": hidden, "inter": inter,
            "renormalize": rng.choice([True, False])}


# ------------------------------------------------------------------ the 4-bit forms, plainly

def _grid(device):
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)
    return torch.cat([v, -v])


def _quantise(x, fmt, scale):
    """x [..., k] fp32 -> codes uint8 [..., k / 2], scales uint8 [..., k / block]."""
    b = x.unflatten(-1, (-1, BLOCK[fmt]))
    a = b.abs().amax(-1, keepdim=True)
    if fmt == "mx":
        m, e = torch.frexp(a)  # a = m 2^e: within 6 2^s = 0.75 2^(s + 3)
        s = torch.where(a == 0, -127, (e - 3 + (m > 0.75)).clamp_min(-127))
        byte = (s + 127).to(torch.uint8)
        half = torch.div(s, 2, rounding_mode="floor")  # 2^-s in two steps, each a normal number
        v = torch.ldexp(torch.ldexp(b, -half), half - s)
    else:
        f8 = (a / (6.0 * torch.tensor(scale, device=x.device))).clamp_max(448.0).to(torch.float8_e4m3fn)
        byte = f8.view(torch.uint8)
        s = f8.float() * scale
        v = torch.where(s > 0, b * (1.0 / s), torch.zeros_like(b))
    w = v.abs()  # the number of borders below: ties go to the even code
    code = ((w > 0.25).to(torch.uint8) + (w >= 0.75) + (w > 1.25) + (w >= 1.75) + (w > 2.5) + (w >= 3.5) + (w > 5.0))
    code = (code + 8 * (v < 0)).flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte.squeeze(-1)


def _values(codes, scales, fmt, scale):
    """The fp32 values that codes and scales stand for."""
    grid = _grid(codes.device)
    v = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], -1).flatten(-2)
    if fmt == "mx":
        s = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127)
    else:
        s = scales.view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (-1, BLOCK[fmt])) * s[..., None]).flatten(-2) * scale


def _norm(x, gamma):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma


def _glu(g, u):
    return g / (1.0 + torch.exp(-g)) * u


# ------------------------------------------------------------------ inputs

def _weights(randn, lead, n, k, fmt, scale):
    """Codes and scales of normal weights, some rows and columns larger than others as trained ones have them."""
    codes = torch.empty(*lead, n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(*lead, n, k // BLOCK[fmt], dtype=torch.uint8, device="cuda")
    flat_c, flat_s = codes.view(-1, n, k // 2), scales.view(-1, n, k // BLOCK[fmt])
    part = max(1, (1 << 26) // (n * k))
    for i in range(0, flat_c.shape[0], part):
        m = min(part, flat_c.shape[0] - i)
        w = randn(m, n, k) * (torch.exp(0.3 * randn(m, n, 1)) / math.sqrt(k))
        flat_c[i:i + m], flat_s[i:i + m] = _quantise(w, fmt, scale)
    return codes, scales


def _weight_scale(fmt, k):
    """The matrix's factor: its largest values (about 16 of the common deviation) at the top of E4M3."""
    return 1.0 if fmt == "mx" else 16.0 / math.sqrt(k) / (6.0 * 448.0)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    randn = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    op, fmt, rows, dt = case["op"], case["fmt"], case["rows"], DTYPES[case["dtype"]]
    k = case["hidden"] if op == "moe" else case["k"]
    # activations: a few channels much larger than the rest
    spread = torch.exp(0.5 * randn(k))
    # the activations' factor of the whole matrix, as a calibration finds it: its largest value, 61.37, at E4M3's top
    s = {"case": case, "scale": 1.0 if fmt == "mx" else 61.37 / (6.0 * 448.0)}
    form = "norm" if op == "moe" else case["form"]
    if form == "glu":
        s["both"] = torch.cat([randn(rows, k) * spread, randn(rows, k)], 1).to(dt)  # one projection's halves
        s["x"], s["up"] = s["both"][:, :k], s["both"][:, k:]
    else:
        s["x"] = (randn(rows, k) * spread * 2.0).to(dt)
    if form == "norm":
        s["gamma"] = 1.0 + 0.1 * randn(k)
    if op == "gemm":
        s["w_scale"] = _weight_scale(fmt, k)
        w = _weights(randn, (), case["n"], k, fmt, s["w_scale"])
        s["r"] = randn(rows, case["n"]).to(dt) if case["residual"] else None
    if op == "moe":
        E, inter = case["experts"], case["inter"]
        s["router"] = randn(E, k) / math.sqrt(k) * 1.5
        w = [_weights(randn, (E,), inter, k, fmt, 1.0), _weights(randn, (E,), inter, k, fmt, 1.0),
             _weights(randn, (E,), k, inter, fmt, 1.0)]
        s["r"] = randn(rows, k).to(dt)
    if own:
        import bit_weight_quantized_q4_gb300 as q4
        s["fmt"] = q4.Q4_MX_MXFP4 if fmt == "mx" else q4.Q4_MX_NVFP4
        if op == "gemm":
            s["W"] = q4.MXMatrix.from_codes(*w, s["fmt"], s["w_scale"])
            s["ws"] = q4.q4_mx_gemm_workspace(s["W"], rows)
        elif op == "moe":
            s["layer"] = q4.MoELayer(s["router"], *(q4.MXMatrix.from_codes(*m, s["fmt"]) for m in w),
                                     top_k=case["top_k"], renormalize=case["renormalize"])
            s["ws"] = q4.q4_moe_workspace(s["layer"], rows)
    elif op != "quant":
        s["w"] = w
    return s


# ------------------------------------------------------------------ the operators, plainly

def _plain_rows(s, form):
    x = s["x"].float()
    return _norm(x, s["gamma"]) if form == "norm" else _glu(x, s["up"].float()) if form == "glu" else x


def _plain_moe(s):
    case = s["case"]
    rows, k, T = case["rows"], case["top_k"], s["x"].dtype
    xh = _plain_rows(s, "norm")
    logits = torch.matmul(xh, s["router"].T)
    top, idx = (t[:, :k] for t in torch.sort(logits, dim=-1, descending=True, stable=True))
    m = logits.amax(-1, keepdim=True)
    over = top if case["renormalize"] else logits
    weight = (top - m).exp() / (over - m).exp().sum(-1, keepdim=True)
    X = _values(*_quantise(xh, "mx", 1.0), "mx", 1.0)
    pair = idx.flatten()  # (token, choice) pairs
    gate, up, down = ((c[pair], sc[pair]) for c, sc in s["w"])
    X = X.repeat_interleave(k, 0)[..., None]
    h = _glu(torch.matmul(_values(*gate, "mx", 1.0), X), torch.matmul(_values(*up, "mx", 1.0), X))[..., 0]
    h = _values(*_quantise(h, "mx", 1.0), "mx", 1.0)[..., None]
    y = torch.matmul(_values(*down, "mx", 1.0), h).view(rows, k, -1)
    y = s["r"].float() + (weight[..., None] * y).sum(1)
    return {"out": y.to(T), "index": idx.to(torch.int32).contiguous(), "weight": weight}


def run(state):
    s, case = state, state["case"]
    op, fmt = case["op"], case["fmt"]
    if own:
        import bit_weight_quantized_q4_gb300 as q4
        if op == "quant":
            m = q4.q4_mx_quant(s["x"], s["fmt"], gamma=s.get("gamma"), eps=EPS, up=s.get("up"), scale=s["scale"])
            return q4.q4_mx_dequant(m, dtype=torch.bfloat16)
        if op == "gemm":
            return q4.q4_mx_gemm(s["W"], s["x"], r=s["r"], gamma=s.get("gamma"), eps=EPS, up=s.get("up"),
                                 scale=s["scale"], workspace=s["ws"])
        out, index, weight = q4.q4_moe(s["x"], s["layer"], gamma=s["gamma"], eps=EPS, r=s["r"], workspace=s["ws"])
        return {"out": out, "index": index, "weight": weight}
    if op == "moe":
        return _plain_moe(s)
    X = _values(*_quantise(_plain_rows(s, case["form"]), fmt, s["scale"]), fmt, s["scale"])
    if op == "quant":
        return X.to(torch.bfloat16)
    y = torch.matmul(X, _values(*s["w"], fmt, s["w_scale"]).T)
    return (y if s["r"] is None else y + s["r"].float()).to(s["x"].dtype)


def work(case):
    B, per = BYTES[case["dtype"]], 0.5 + 1.0 / BLOCK[case["fmt"]]  # bytes of a 4-bit value and its share of a scale
    rows = case["rows"]
    if case["op"] == "moe":
        E, hid, inter = case["experts"], case["hidden"], case["inter"]
        # the experts that uniform choices are expected to reach
        active = E * (1.0 - (1.0 - case["top_k"] / E) ** rows)
        return {"bytes": int(active * 3 * hid * inter * per + 4 * E * hid + 4 * hid + 3 * rows * hid * B
                             + 8 * rows * case["top_k"]),
                "flops": 2 * rows * hid * (3 * case["top_k"] * inter + E)}
    k = case["k"]
    read = rows * k * B * (2 if case["form"] == "glu" else 1) + (4 * k if case["form"] == "norm" else 0)
    if case["op"] == "quant":  # quantised, and read back as bf16
        return {"bytes": int(read + 2 * rows * k * per + 2 * rows * k), "flops": 8 * rows * k}
    n = case["n"]
    return {"bytes": int(read + n * k * per + rows * n * B * (2 if case["residual"] else 1)), "flops": 2 * rows * n * k}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_quantised(x, fmt, scale):
    """The values that x (64 bits) is stored as, from the definition of the formats."""
    b = x.reshape(*x.shape[:-1], -1, BLOCK[fmt])
    least = b.abs().max(-1, keepdim=True).values / 6.0
    if fmt == "mx":
        m, e = torch.frexp(least)
        s = torch.ldexp(torch.ones_like(least), torch.where(m == 0.5, e - 1, e).clamp_min(-127))
        s = torch.where(least == 0, torch.full_like(s, 2.0 ** -127), s)
    else:  # to the nearest of 8 steps an octave, 2^-9 at least
        q = (least / scale).clamp_max(448.0)
        step = torch.ldexp(torch.ones_like(q), torch.frexp(q)[1] - 4).clamp_min(2.0 ** -9)
        s = torch.round(q / step) * step * scale
    v = torch.where(s > 0, b / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(b))
    size = v.abs()
    step = 0.5 * (1.0 + (size >= 2.0).double() + 2.0 * (size >= 4.0).double())
    return (torch.sign(v) * (torch.round(size / step) * step).clamp_max(6.0) * s).reshape(x.shape)


def _exact_stored(codes, scales, fmt, scale):
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int32)
    mant, ex = code & 1, (code >> 1) & 3
    size = torch.where(ex == 0, 0.5 * mant, torch.ldexp(1.0 + 0.5 * mant.double(), ex - 1))
    sc = scales.to(torch.int32)
    if fmt == "mx":
        sc = torch.ldexp(torch.ones_like(sc, dtype=torch.float64), sc - 127)
    else:
        sub = torch.ldexp((sc & 7).double(), torch.full_like(sc, -9))
        sc = torch.where(sc < 8, sub, torch.ldexp(1.0 + (sc & 7).double() / 8.0, (sc >> 3) - 7))
    size = size * (1.0 - 2.0 * (code >> 3).double())
    return (size.unflatten(-1, (-1, BLOCK[fmt])) * sc[..., None]).flatten(-2) * scale


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, fmt = case["op"], case["fmt"]
    x = s["x"].double()
    if op == "moe" or case["form"] == "norm":
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * s["gamma"].double()
    elif case["form"] == "glu":
        x = x * torch.sigmoid(x) * s["up"].double()
    X = _exact_quantised(x, fmt, s["scale"])
    if op == "quant":
        return X
    if op == "gemm":
        y = X @ _exact_stored(*s["w"], fmt, s["w_scale"]).T
        return y if s["r"] is None else y + s["r"].double()
    logits = x @ s["router"].double().T
    idx = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :case["top_k"]]
    if case["renormalize"]:
        weight = torch.softmax(logits.gather(1, idx), -1)
    else:
        weight = torch.softmax(logits, -1).gather(1, idx)
    out = s["r"].double()
    for e in idx.unique().tolist():
        t, j = torch.nonzero(idx == e, as_tuple=True)
        gate, up, down = (_exact_stored(c[e], sc[e], fmt, 1.0) for c, sc in s["w"])
        g, u = X[t] @ gate.T, X[t] @ up.T
        h = _exact_quantised(g * torch.sigmoid(g) * u, fmt, 1.0)
        out[t] += weight[t, j, None] * (h @ down.T)
    return {"out": out, "index": None, "weight": weight}
