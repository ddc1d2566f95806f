"""The microscaled 4-bit formats by their definitions, in 64 bits (torch, any device)."""
import torch

BLOCK = (32, 16)  # columns that share a scale: MXFP4, NVFP4
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def exp2i(e):
    """2^e in 64 bits of whole e from -1022 to 1023, exactly (torch.ldexp goes by a rounded power)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def e2m1(v):
    """The nearest grid value (ties to the even code, at most 6 in magnitude), and half the grid's step there."""
    size = v.abs()
    step = torch.where(size < 2, 0.5, torch.where(size < 4, 1.0, 2.0)).double()
    q = (torch.round(size / step) * step).clamp_max(6.0)
    return torch.where(torch.signbit(v), -q, q), step / 2


def e4m3(v):
    """The nearest E4M3 value of v >= 0 (ties to even, 448 at most)."""
    v = v.clamp_max(448.0)
    step = exp2i(torch.frexp(v)[1] - 4).clamp_min(2.0 ** -9)
    return torch.round(v / step) * step


def mx_scale(a):
    """MXFP4: the smallest power of two s >= 2^-127 with a <= 6 s, of 64-bit a >= 0."""
    m, e = torch.frexp(a / 6.0)
    s = exp2i(torch.where(m == 0.5, e - 1, e).clamp(-127, 1000))
    return torch.where(a == 0, torch.full_like(s, 2.0 ** -127), s)


def quantise(x, fmt, scale=1.0):
    """The values (64 bits) that x [.., k] is stored as.  NVFP4's scale and factor are the fp32 ones that the format
    names: a / (6 scale), and 1 / (s scale) times the value."""
    b = x.double().unflatten(-1, (-1, BLOCK[fmt]))
    a = b.abs().amax(-1, keepdim=True)
    if fmt == 0:
        s = mx_scale(a)
        q = e2m1(b / s)[0] * s
    else:
        f32 = lambda t: t.float()  # noqa: E731
        g = f32(torch.tensor(scale, dtype=torch.float64, device=x.device))
        e = e4m3((f32(a) / (f32(torch.tensor(6.0, device=x.device)) * g)).double())
        sg = f32(e) * g
        v = torch.where(e > 0, f32(b) * (torch.ones_like(sg) / sg), torch.zeros_like(f32(b)))
        q = e2m1(v.double())[0] * e * g.double()
    q = torch.where(torch.isfinite(a), q, torch.full_like(q, float("nan")))
    return q.flatten(-2)


def stored(codes, scales, fmt, scale=1.0):
    """The values (64 bits) of plain rows of codes and scale bytes."""
    grid = torch.tensor(GRID + tuple(-x for x in GRID), dtype=torch.float64, device=codes.device)
    v = grid[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]
    e = scales.long()
    if fmt == 0:
        s = torch.where(e == 255, float("nan"), exp2i(e - 127))
    else:
        mant, ex = (e & 7).double(), e >> 3
        s = torch.where(ex == 0, mant * 2.0 ** -9, (1.0 + mant / 8.0) * exp2i(ex - 7))
        s = torch.where(e == 127, float("nan"), s)
    return (v.unflatten(-1, (-1, BLOCK[fmt])) * s[..., None]).flatten(-2) * scale


def random_codes(gen, shape, k, fmt, lo=-3, hi=3):
    """Codes of all kinds and scales 2^lo .. 2^hi (NVFP4: any E4M3 between them)."""
    dev = gen.device
    codes = torch.randint(0, 256, (*shape, k // 2), generator=gen, device=dev, dtype=torch.uint8)
    if fmt == 0:
        scales = torch.randint(127 + lo, 128 + hi, (*shape, k // 32), generator=gen, device=dev).to(torch.uint8)
    else:
        scales = torch.randint((7 + lo) * 8, (8 + hi) * 8, (*shape, k // 16), generator=gen, device=dev).to(torch.uint8)
    return codes, scales
