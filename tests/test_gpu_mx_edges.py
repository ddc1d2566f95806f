"""Microscaled 4-bit matrices on the GPU at their edges: zeros, subnormal numbers, infinities and NaN behind a norm and a
SwiGLU and in rows that the product quantises; NVFP4's reciprocals; and results that are rounded once."""
import pytest

import mx_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def q4():
    import bit_weight_quantized_q4_gb300 as m
    m.build()
    m.lib()
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


# ------------------------------------------------------------------ behind a norm

# rows and columns of every form of the kernel: one to eight warps a row, one or two of its sixteens in registers, the
# rest read again; few rows and many
SHAPES = [(4, 96), (9, 288), (5, 1056), (7, 4096), (4, 4128), (3, 8224), (2, 20000), (2100, 512), (1100, 1024), (600, 2048),
          (300, 4096)]


@pytest.mark.parametrize("rows,k", SHAPES)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("fmt,scale", [(0, 1.0), (1, 0.01)])
def test_zeros_behind_a_norm_stay_zeros(q4, fmt, scale, dtype, rows, k):
    # rows of a root mean square of 0.05 (their factor is 20), with blocks of zeros, blocks whose gammas are zeros, and a
    # row of zeros (eps alone: a factor of 1000)
    g = gen(rows + k)
    x = (0.05 * randn(g, rows, k)).to(dtype)
    x[:, :32] = 0.0
    x[0, k - 32:] = 0.0
    x[1] = 0.0
    gamma = 1 + 0.1 * torch.rand(k, generator=g, device="cuda")
    gamma[32:48] = 0.0  # an NVFP4 block, half an MXFP4 one
    if k > 128:
        gamma[96:128] = 0.0
    zero = torch.zeros(rows, k, dtype=torch.bool, device="cuda")
    zero[:, :48], zero[0, k - 32:], zero[1] = True, True, True
    if k > 128:
        zero[:, 96:128] = True
    m = q4.q4_mx_quant(x, fmt, gamma=gamma, eps=1e-6, scale=scale)
    c, s = m.codes()
    code = torch.stack([c & 15, c >> 4], -1).flatten(-2)
    assert bool((code[zero] % 8 == 0).all())  # (the sign is the value's)
    block = zero.unflatten(-1, (-1, m.block)).all(-1)
    assert bool((s[block] == 0).all()) and bool((s[~block] > 0).all())
    back = q4.q4_mx_dequant(m)
    assert bool((back[zero] == 0).all()) and bool((back[~zero] != 0).any())
    W = q4.q4_mx_quant(randn(g, 130, k), fmt, scale=1.0 if fmt == 0 else 1e-3)
    y = q4.q4_mx_gemm(W, x, gamma=gamma, eps=1e-6, scale=scale, dtype=F32)
    assert bool((y[1] == 0).all()) and bool((y[0] != 0).any())
    q4.q4_device_check()


@pytest.mark.parametrize("k", [128, 512, 4096, 16384])
@pytest.mark.parametrize("fmt,scale,c,tiny", [
    (0, 1.0, 2.0 ** -10, 2.0 ** -138),  # a factor of 2^11, values of the grid times 2^-127: the least scale, subnormal
    (0, 1.0, 2.0 ** -20, 2.0 ** -147),  # 2^21, times 2^-126
    (1, 2.0 ** -60, 2.0 ** -59, 2.0 ** -129)])  # 2^60, times 2^-69: NVFP4's least scale, 2^-9, and the least factor
def test_tiny_blocks_behind_a_norm_keep_their_codes(q4, fmt, scale, c, tiny, k):
    # a quarter of the columns +-c, the others next to nothing: the root mean square is c / 2, to the last bit
    g = gen(k)
    grid = torch.tensor(mx_ref.GRID + tuple(-v for v in mx_ref.GRID), device="cuda", dtype=torch.float64)
    codes = grid[torch.randint(0, 16, (3, k), generator=g, device="cuda")].clamp(-4, 4)
    codes[:, ::16] = 4.0  # every block's largest: away from where its scale would change
    x = codes * tiny
    x[:, :k // 4] = c
    x[:, 1:k // 4:2] = -c
    want = codes * tiny * (2.0 / c)
    x = x.float()
    m = q4.q4_mx_quant(x, fmt, gamma=torch.ones(k, device="cuda"), eps=0.0, scale=scale)
    got = mx_ref.stored(*m.codes(), fmt, scale)[:, k // 4:]
    # (the factor is a few units in the last place off at most: no code is that near to a border)
    assert torch.equal(got, mx_ref.quantise(want, fmt, scale)[:, k // 4:])
    assert torch.equal(got, want[:, k // 4:])
    q4.q4_device_check()


@pytest.mark.parametrize("k", [96, 1056, 4096, 8224, 20000])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("fmt,scale", [(0, 1.0), (1, 0.01)])
def test_infinities_and_nan_behind_a_norm(q4, fmt, scale, dtype, k):
    # by the formula: an infinite sum makes every finite value of its row zero and the infinite ones NaN; a NaN its whole
    # row; a gamma that is no number its column's block
    g = gen(k)
    x = randn(g, 5, k).to(dtype)
    x[1, 40], x[2, 70] = float("inf"), float("nan")
    x[3, k - 1] = float("-inf")
    gamma = 1 + 0.1 * randn(g, k)
    clean = q4.q4_mx_quant(x, fmt, gamma=gamma, eps=1e-6, scale=scale)
    for bad in (None, float("nan"), float("inf")):
        gm = gamma.clone()
        if bad is not None:
            gm[50] = bad
        m = q4.q4_mx_quant(x, fmt, gamma=gm, eps=1e-6, scale=scale)
        B = m.block
        back = q4.q4_mx_dequant(m).unflatten(-1, (-1, B))
        nan = torch.zeros(5, k // B, dtype=torch.bool, device="cuda")
        nan[1, 40 // B], nan[2], nan[3, -1] = True, True, True
        if bad is not None:
            nan[:, 50 // B] = True
        assert torch.equal(torch.isnan(back).all(-1), nan) and torch.equal(torch.isnan(back).any(-1), nan)
        for row in (1, 3):
            assert bool((back[row][~nan[row]] == 0).all())
        c, s = m.codes()
        assert bool((c.unflatten(-1, (-1, B // 2))[nan] == 0).all())
        for row in (0, 4):
            want = q4.q4_mx_dequant(clean).unflatten(-1, (-1, B))[row]
            assert torch.equal(back[row][~nan[row]], want[~nan[row]])
    q4.q4_device_check()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("fmt,scale", [(0, 1.0), (1, 0.01)])
@pytest.mark.parametrize("rows,k", [(1, 64), (5, 544), (2200, 4096)])
def test_zeros_infinities_and_nan_behind_a_swiglu(q4, fmt, scale, dtype, rows, k):
    g = gen(rows + k)
    x, up = randn(g, rows, k).to(dtype), randn(g, rows, k).to(dtype)
    r = rows - 1
    x[r, :16], up[r, 16:32] = 0.0, 0.0
    clean = q4.q4_mx_quant(x, fmt, up=up, scale=scale)
    back = q4.q4_mx_dequant(clean)
    assert bool((back[r, :32] == 0).all()) and bool((back[r, 32:] != 0).any())
    for where, v, other in (("x", float("inf"), 0.0), ("x", float("-inf"), 1.0), ("x", float("nan"), 1.0), ("up", float("inf"), 0.0),
                            ("up", float("-inf"), 2.0), ("up", float("nan"), -1.0)):
        xs, us = x.clone(), up.clone()
        xs[r, 40], us[r, 40] = (v, other) if where == "x" else (other, v)
        m = q4.q4_mx_quant(xs, fmt, up=us, scale=scale)
        B = m.block
        got, want = q4.q4_mx_dequant(m), q4.q4_mx_dequant(clean)
        hit = torch.zeros(rows, k, dtype=torch.bool, device="cuda")
        hit[r, 40 // B * B:40 // B * B + B] = True
        assert bool(torch.isnan(got[hit]).all()) and torch.equal(got[~hit], want[~hit])
    # a gate far below zero closes: exp(-x) is infinite, the quotient zero
    x[r, 32:] = -200.0
    assert bool((q4.q4_mx_dequant(q4.q4_mx_quant(x, fmt, up=up, scale=scale))[r, 32:] == 0).all())
    q4.q4_device_check()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("nb,n,k", [(1, 300, 544), (4, 130, 4096), (8, 20000, 288), (40, 300, 544), (300, 300, 544)])
def test_the_product_of_rows_with_zeros_infinities_and_nan(q4, nb, n, k, dtype, fmt):
    # rows that the product quantises itself, and those that the quantiser does: as quantising first
    g = gen(nb + n)
    sc = 1.0 if fmt == 0 else 0.01
    W = q4.q4_mx_quant(randn(g, n, k) * 0.1, fmt, scale=1.0 if fmt == 0 else 1e-3)
    x, up = randn(g, nb, k).to(dtype), randn(g, nb, k).to(dtype)
    x[0, :64] = 0.0
    kinds = [float("inf"), float("nan"), float("-inf"), 0.0]
    for t in range(nb):
        if t % 2:
            x[t, 100 + t % 100] = kinds[t // 2 % 4]
    x[nb - 1] = 0.0
    for kw in ({}, {"up": up}, {"gamma": 1 + 0.1 * randn(g, k), "eps": 1e-6}):
        y = q4.q4_mx_gemm(W, x, scale=sc, **kw)
        want = q4.q4_mx_gemm(W, q4.q4_mx_quant(x, fmt, scale=sc, **kw), dtype=dtype)
        assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(torch.nan_to_num(y), torch.nan_to_num(want))
        odd = torch.tensor([t for t in range(nb - 1) if t % 2 and kinds[t // 2 % 4] != 0.0], dtype=torch.long, device="cuda")
        assert bool(torch.isnan(y[odd]).all())
        assert bool((y[nb - 1] == 0).all())
    q4.q4_device_check()


# ------------------------------------------------------------------ NVFP4's factors

def test_reciprocals_are_the_nearest_ones(q4):
    # x (1 / (s g)) next to a border: a factor g whose products with every scale have all kinds of significands, those of
    # ones alone among them, where Newton's step ends at a tie
    ones = [2.0 - 2.0 ** -23, (2.0 - 2.0 ** -23) * 2.0 ** -7, (2.0 - 2.0 ** -22), 1.0 + 2.0 ** -23]
    g = gen(3)
    some = (1.0 + torch.randint(0, 1 << 23, (60,), generator=g, device="cuda").double() / (1 << 23)).tolist()
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for scale in ones + some:
        gf = torch.tensor(scale, device="cuda", dtype=F32)
        e = torch.arange(1, 127, device="cuda").to(torch.uint8).view(torch.float8_e4m3fn).float()
        sg = e * gf
        # the largest value gives the scale; the others are the fp32 numbers around every border
        b = borders[None] * sg[:, None]
        near = (b.view(torch.int32)[:, :, None] + torch.tensor([-2, -1, 0, 1, 2], device="cuda", dtype=torch.int32)).view(F32)
        near = near.flatten(1)  # 35 for each scale
        x = torch.zeros(126, 48, device="cuda")
        x[:, 1:16], x[:, 17:32], x[:, 33:38] = near[:, :15], near[:, 15:30], near[:, 30:]
        x[:, ::16] = 6.0 * sg[:, None]
        x = torch.nn.functional.pad(x, (0, 16))
        m = q4.q4_mx_quant(x, 1, scale=scale)
        c, s = m.codes()
        assert torch.equal(s[:, :3].long(), torch.arange(1, 127, device="cuda")[:, None].expand(126, 3))
        assert torch.equal(mx_ref.stored(c, s, 1, float(gf)), mx_ref.quantise(x, 1, scale))
    q4.q4_device_check()


# ------------------------------------------------------------------ results

@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("nb,n", [(1, 515), (1, 20000), (7, 515), (40, 515), (64, 20000), (300, 515), (300, 516), (1000, 130)])
def test_results_are_rounded_once(q4, nb, n, dtype, fmt):
    # scales of one, sums of quarters below 2^15 and residuals of eighths: fp32 numbers, so that the output's rounding is
    # the only one
    g = gen(nb + n)
    k = 2080
    one = 127 if fmt == 0 else 56
    wc, xc = (torch.randint(0, 256, (rows, k // 2), generator=g, device="cuda", dtype=torch.uint8) for rows in (n, nb))
    ws, xs = (torch.full((rows, k // mx_ref.BLOCK[fmt]), one, device="cuda", dtype=torch.uint8) for rows in (n, nb))
    W, X = q4.MXMatrix.from_codes(wc, ws, fmt), q4.MXMatrix.from_codes(xc, xs, fmt)
    total = mx_ref.stored(xc, xs, fmt) @ mx_ref.stored(wc, ws, fmt).T
    assert float(total.abs().max()) < 2 ** 15
    assert torch.equal(q4.q4_mx_gemm(W, X, dtype=dtype), total.float().to(dtype))
    r = (torch.randint(-64, 65, (nb, n), generator=g, device="cuda").double() / 8)
    want = (total + r).float().to(dtype)
    r = r.to(dtype)
    assert torch.equal(q4.q4_mx_gemm(W, X, r=r, dtype=dtype), want)
    assert torch.equal(q4.q4_mx_gemm(W, X, r=r, out=r), want)
    q4.q4_device_check()


def test_a_layers_results_are_rounded_once(q4):
    g = gen(2)
    mats = [q4.q4_mx_quant(randn(g, 8, a, b) * b ** -0.5) for a, b in ((160, 256), (160, 256), (256, 160))]
    layer = q4.MoELayer(randn(g, 8, 256) / 16, *mats, top_k=2)
    for rows in (1, 5, 16):
        for dtype in (F16, BF16):
            x, r = randn(g, rows, 256).to(dtype), randn(g, rows, 256).to(dtype)
            for res in (None, r):
                fine = q4.q4_moe(x, layer, r=None if res is None else res.float(), dtype=F32)
                coarse = q4.q4_moe(x, layer, r=res)
                assert torch.equal(coarse[0], fine[0].to(dtype)) and torch.equal(coarse[1], fine[1])
    q4.q4_device_check()
