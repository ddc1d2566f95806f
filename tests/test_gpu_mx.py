"""Microscaled 4-bit matrices on the GPU: quantising, reading back, and the product, against the formats' definitions
in 64 bits (mx_ref.py)."""
import numpy as np
import pytest

import mx_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}  # half a step, relative


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


def same(got, want):
    """The same numbers, NaN where NaN is."""
    got, want = got.double(), want.double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])


# ------------------------------------------------------------------ quantising

@pytest.mark.parametrize("rows,k", [(1, 32), (3, 64), (127, 288), (129, 256), (5, 4096), (300, 1056), (2, 65536)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("fmt,scale", [(0, 1.0), (1, 0.0123), (1, 2.0 ** -40)])
def test_quantised_values_are_the_definitions(q4, fmt, scale, dtype, rows, k):
    g = gen(rows * 7 + k + fmt)
    # sizes from 2^-20 to 2^20 in one row, zeros, whole blocks of zeros, ties
    x = randn(g, rows, k) * torch.exp2(torch.randint(-20, 21, (rows, k // 32), generator=g, device="cuda").float()
                                       ).repeat_interleave(32, 1)
    x[torch.rand(rows, k, generator=g, device="cuda") < 0.1] = 0.0
    x[:, :32] = 0.0
    if k > 64:
        x[:, 32:64] = torch.tensor(mx_ref.GRID, device="cuda").repeat(4) * 0.5 + 0.125  # next to and on borders
    x = x.to(dtype)
    x[~torch.isfinite(x)] = 1.0
    m = q4.q4_mx_quant(x, fmt, scale=scale)
    want = mx_ref.quantise(x, fmt, scale)
    c, s = m.codes()
    same(mx_ref.stored(c, s, fmt, float(np.float32(scale))), want)
    # read back: rounded once to the type
    for t in (F32, F16, BF16):
        back = q4.q4_mx_dequant(m, t)
        fine = want.abs() < torch.finfo(t).max
        err = (back.double() - want).abs()[fine]
        # (NVFP4 in fp32: two products, each rounded)
        tiny = torch.finfo(t).tiny * EPS[t] * 2
        assert bool((err <= (EPS[t] + (2.0 ** -23 if fmt else 0.0)) * want.abs()[fine] + tiny).all())
    q4.q4_device_check()


@pytest.mark.parametrize("fmt", [0, 1])
def test_extreme_values(q4, fmt):
    big = torch.finfo(F32).max
    rows = [
        [0.0] * 32,
        [big] + [big / 2] * 31,                            # the largest scale
        [2.0 ** -149] + [0.0] * 31,                        # a subnormal
        [2.0 ** -126, -2.0 ** -127] + [2.0 ** -149] * 30,
        [6.0] * 32, [6.0000005] + [3.0] * 31,              # at a power of two's end, and behind it
        [-0.0] * 32,
        [float("nan")] + [1.0] * 31, [1.0] * 31 + [float("inf")], [float("-inf")] + [0.0] * 31,
        [-5.0, 5.0, 2.5, -2.5, 3.5, 1.75, 1.25, 0.75, 0.25, -0.25, 6.0, 0.0] + [0.0] * 20,  # ties
    ]
    x = torch.tensor(rows, device="cuda")
    m = q4.q4_mx_quant(x, fmt)
    c, s = m.codes()
    same(mx_ref.stored(c, s, fmt), mx_ref.quantise(x, fmt))
    if fmt == 0:
        assert s[:, 0].tolist() == [0, 253, 0, 0, 127, 128, 0, 255, 255, 255, 127]
    back = q4.q4_mx_dequant(m)
    assert torch.isnan(back[7:10]).sum(1).tolist() == ([16] * 3 if fmt else [32] * 3)  # the block's, no others


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("fmt,scale", [(0, 1.0), (1, 0.013)])
@pytest.mark.parametrize("form", ["norm", "glu"])
@pytest.mark.parametrize("rows,k", [(1, 32), (2, 512), (9, 544), (3, 1056), (5, 2080), (4, 4096), (130, 4128), (3, 8224), (2, 20000)])
def test_quantised_behind_a_norm_or_a_swiglu(q4, rows, k, form, fmt, scale, dtype):
    g = gen(k + rows)
    x = (randn(g, rows, k) * 2).to(dtype)
    a, v = x.double(), None
    if form == "norm":
        gamma = 1 + 0.2 * randn(g, k)
        m = q4.q4_mx_quant(x, fmt, gamma=gamma, eps=1e-5, scale=scale)
        v = a / torch.sqrt(a.square().mean(-1, keepdim=True) + 1e-5) * gamma.double()
        # fp32: a chain of k / 256 + 16 sums of squares, then a handful of roundings
        delta = (k / 256 + 48) * 2.0 ** -24 * torch.ones_like(v)
    else:
        up = randn(g, rows, k).to(dtype)
        m = q4.q4_mx_quant(x, fmt, up=up, scale=scale)
        v = a * torch.sigmoid(a) * up.double()
        # the fast exponential is within 2 + 1.173 |x| units in the last place, the fast quotient within 2
        delta = (2 + 1.173 * a.abs() + 4) * 2.0 ** -23
    c, s = m.codes()
    got = mx_ref.stored(c, s, fmt, float(np.float32(scale)))
    # the scale is that of a largest value within delta
    B = mx_ref.BLOCK[fmt]
    blocks = lambda t: t.unflatten(-1, (-1, B))  # noqa: E731
    vb, db = blocks(v), blocks(delta)
    hi, lo = (vb.abs() * (1 + db)).amax(-1), (vb.abs() * (1 - db)).amax(-1)
    if fmt == 0:
        sv = mx_ref.exp2i(s.long() - 127)
        assert bool(((sv >= mx_ref.mx_scale(lo)) & (sv <= mx_ref.mx_scale(hi))).all())
        unit = sv
    else:
        ex = s.long() >> 3
        mant = (s.long() & 7).double()
        sv = torch.where(ex == 0, mant * 2.0 ** -9, (1.0 + mant / 8.0) * mx_ref.exp2i(ex - 7))
        near = 2.0 ** -22  # 6 scale, the quotient
        assert bool(((sv >= mx_ref.e4m3(lo / (6 * scale) * (1 - near))) & (sv <= mx_ref.e4m3(hi / (6 * scale) * (1 + near)))).all())
        unit = sv * scale
    # a value is within half a step of the grid of what it stands for, plus delta; beyond 6 it is 6
    u = unit[..., None].clamp_min(1e-300)
    want = (vb / u).clamp(-6.25, 6.25)
    err = (blocks(got) / u - want.clamp(-6, 6)).abs()
    half = torch.where(want.abs() < 2, 0.25, torch.where(want.abs() < 4, 0.5, 1.0)).double()
    slack = (db + 2.0 ** -22) * want.abs()
    half = torch.where((want.abs() + slack >= 2) & (want.abs() < 2), 0.5, half)
    half = torch.where((want.abs() + slack >= 4) & (want.abs() < 4), 1.0, half)
    assert bool((err <= half + slack).all() if fmt == 0 else (err <= half + slack)[unit > 0].all())
    q4.q4_device_check()


def test_strided_rows_batches_and_the_halves_of_one_buffer(q4):
    g = gen(3)
    both = randn(g, 37, 2 * 288).to(BF16)
    gate, up = both[:, :288], both[:, 288:]
    a = q4.q4_mx_quant(gate, 0, up=up).codes()
    b = q4.q4_mx_quant(gate.contiguous(), 0, up=up.contiguous()).codes()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    wide = randn(g, 9, 1024)
    a = q4.q4_mx_quant(wide[:, 256:544], 1, scale=0.1).codes()
    b = q4.q4_mx_quant(wide[:, 256:544].contiguous(), 1, scale=0.1).codes()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # a batch: each matrix is padded by itself
    x = randn(g, 3, 130, 96)
    m = q4.q4_mx_quant(x, 0, gamma=torch.ones(96, device="cuda"), eps=1e-6)
    assert (m.batch, m.rows, m.k) == (3, 130, 96)
    for i in range(3):
        one = q4.q4_mx_quant(x[i], 0, gamma=torch.ones(96, device="cuda"), eps=1e-6)
        assert torch.equal(m.codes()[0][i], one.codes()[0]) and torch.equal(m.codes()[1][i], one.codes()[1])
        assert torch.equal(q4.q4_mx_dequant(m)[i], q4.q4_mx_dequant(one))


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("shape,k", [((1,), 32), ((130,), 288), ((3, 129), 544), ((2, 256), 256)])
def test_codes_round_trip(q4, fmt, shape, k):
    g = gen(11)
    c, s = mx_ref.random_codes(g, shape, k, fmt)
    m = q4.MXMatrix.from_codes(c, s, fmt, 1.0 if fmt == 0 else 0.5)
    c2, s2 = m.codes()
    assert torch.equal(c, c2) and torch.equal(s, s2)
    assert torch.equal(q4.q4_mx_dequant(m).double(), mx_ref.stored(c, s, fmt, 1.0 if fmt == 0 else 0.5))


# ------------------------------------------------------------------ the product

def product(q4, g, fmt, nb, n, k, residual=None, dtype=F32):
    wc, ws = mx_ref.random_codes(g, (n,), k, fmt)
    xc, xs = mx_ref.random_codes(g, (nb,), k, fmt)
    gw, gx = (1.0, 1.0) if fmt == 0 else (0.5, 0.37)
    W, X = q4.MXMatrix.from_codes(wc, ws, fmt, gw), q4.MXMatrix.from_codes(xc, xs, fmt, gx)
    w, x = mx_ref.stored(wc, ws, fmt, gw), mx_ref.stored(xc, xs, fmt, float(np.float32(gx)))
    r = None if residual is None else randn(g, nb, n).to(dtype)
    ref, S = x @ w.T, x.abs() @ w.abs().T
    if r is not None:
        ref = ref + r.double()
    return W, X, r, ref, S


def bound(ref, S, k, dtype):
    # each of the k / 64 steps rounds the sum once (truncation: a whole unit), and within a step 64
    # products meet at the largest one's precision; the factors of the matrices, the residual and the output
    # round once each
    return (k / 64 + 64 + 4) * 2.0 ** -23 * S + 2 * EPS[dtype] * ref.abs() + 1e-30


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("nb,n,k", [
    (1, 1, 32), (1, 129, 288), (16, 128, 256), (17, 300, 1056), (1, 4096, 4096), (5, 2048, 8224),  # few rows, k shared
    (33, 1000, 2080), (64, 640, 544), (65, 640, 544), (100, 5000, 96), (128, 127, 8192), (129, 384, 512),
    (192, 385, 768), (193, 257, 1024), (256, 256, 256), (511, 1300, 320), (1000, 130, 2048), (700, 4100, 288)])
def test_product(q4, fmt, nb, n, k):
    for dtype, residual in ((F32, None), (F32, 1), (BF16, 1), (F16, None)):
        W, X, r, ref, S = product(q4, gen(nb + n + k + fmt), fmt, nb, n, k, residual, dtype)
        y = q4.q4_mx_gemm(W, X, r=r, dtype=dtype)
        lim = torch.finfo(dtype).max
        fine = ref.abs() < lim * 0.99
        assert y.shape == (nb, n) and y.dtype == dtype
        assert bool(((y.double() - ref).abs() <= bound(ref, S, k, dtype))[fine].all())
        if r is not None:  # in place on the residual
            out = r.clone()
            assert q4.q4_mx_gemm(W, X, r=out, out=out) is out and torch.equal(out, y)
    q4.q4_device_check()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("nb,n,k", [
    (70, 1500, 96), (129, 333, 288), (150, 2000, 288), (193, 1000, 64), (980, 3900, 256), (1540, 2300, 288),
    (400, 5000, 512), (2500, 1100, 160), (300, 301, 544), (2000, 1025, 288), (17, 10000, 288), (65, 20000, 32)])
def test_product_of_whole_and_cut_tiles(q4, fmt, nb, n, k):
    # columns that end inside a tile's part or before it, rounds that end anywhere, odd rows of results
    for dtype, residual in ((F32, 1), (BF16, 1), (F16, None)):
        W, X, r, ref, S = product(q4, gen(nb + n + k + fmt), fmt, nb, n, k, residual, dtype)
        out = torch.full((nb + 2, n), 7.0, dtype=dtype, device="cuda")
        y = out[1:-1]
        if (n * y.element_size()) % 16 == 0:
            q4.q4_mx_gemm(W, X, r=r, out=y)
        else:
            y = q4.q4_mx_gemm(W, X, r=r, dtype=dtype)
        fine = ref.abs() < torch.finfo(dtype).max * 0.99
        assert bool(((y.double() - ref).abs() <= bound(ref, S, k, dtype))[fine].all())
        assert bool((out[0] == 7).all() and (out[-1] == 7).all())
    q4.q4_device_check()


@pytest.mark.parametrize("nb", [1, 40, 300])
def test_product_of_whole_numbers_is_exact(q4, nb):
    # scales of one: sums of products of halves below 2^24 are fp32 numbers
    g = gen(nb)
    wc, ws = mx_ref.random_codes(g, (515,), 4128, 0, 0, 0)
    xc, xs = mx_ref.random_codes(g, (nb,), 4128, 0, 0, 0)
    y = q4.q4_mx_gemm(q4.MXMatrix.from_codes(wc, ws, 0), q4.MXMatrix.from_codes(xc, xs, 0))
    assert torch.equal(y.double(), mx_ref.stored(xc, xs, 0) @ mx_ref.stored(wc, ws, 0).T)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("nb,n,k", [(1, 333, 544), (3, 1200, 1056), (8, 20000, 544), (2, 130, 8224), (1, 640, 16384), (5, 64, 32),
                                    (7, 40000, 288), (9, 333, 544), (200, 333, 544)])
def test_product_quantises_its_rows_as_the_quantiser_does(q4, nb, n, k, dtype, fmt):
    g = gen(5 + nb)
    W = q4.q4_mx_quant(randn(g, n, k) * 0.1, fmt, scale=1.0 if fmt == 0 else 1e-3)
    sc = 1.0 if fmt == 0 else 0.01
    x, up, gamma = randn(g, nb, k).to(dtype), randn(g, nb, k).to(dtype), 1 + 0.1 * randn(g, k)
    for kw in ({}, {"gamma": gamma, "eps": 1e-6}, {"up": up}):
        X = q4.q4_mx_quant(x, fmt, scale=sc, **kw)
        want = q4.q4_mx_gemm(W, X, dtype=dtype)
        assert torch.equal(q4.q4_mx_gemm(W, x, scale=sc, **kw), want)
        ws = q4.q4_mx_gemm_workspace(W, nb)
        ws.fill_(255)  # any contents
        out = torch.empty_like(want)
        assert torch.equal(q4.q4_mx_gemm(W, x, scale=sc, out=out, workspace=ws, **kw), want)
    # rows of a wider buffer, another output type
    wide = torch.zeros(nb, 2 * k, dtype=dtype, device="cuda")
    wide[:, k:] = x
    assert torch.equal(q4.q4_mx_gemm(W, wide[:, k:], scale=sc), q4.q4_mx_gemm(W, q4.q4_mx_quant(x, fmt, scale=sc), dtype=dtype))
    other = F16 if dtype == F32 else F32
    assert torch.equal(q4.q4_mx_gemm(W, x, scale=sc, dtype=other), q4.q4_mx_gemm(W, q4.q4_mx_quant(x, fmt, scale=sc), dtype=other))
    q4.q4_device_check()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("nb,n", [(2, 130), (70, 200), (300, 300)])
def test_a_nan_stays_in_its_row(q4, fmt, nb, n):
    g = gen(6)
    x, w = randn(g, nb, 288), randn(g, n, 288)
    x[1, 40], w[7, 200] = float("inf"), float("nan")
    W, X = q4.q4_mx_quant(w, fmt, scale=1.0 if fmt == 0 else 0.01), q4.q4_mx_quant(x, fmt, scale=1.0 if fmt == 0 else 0.01)
    y = q4.q4_mx_gemm(W, X)
    nan = torch.zeros(nb, n, dtype=torch.bool, device="cuda")
    nan[1], nan[:, 7] = True, True
    assert torch.equal(torch.isnan(y), nan) and bool(torch.isfinite(y[~nan]).all())


@pytest.mark.parametrize("nb,n,k", [(1, 4096, 2048), (16, 300, 4096), (64, 512, 512), (300, 1000, 288), (2000, 300, 512)])
def test_what_lies_behind_the_last_row_reaches_nothing(q4, nb, n, k):
    # records of 128 rows whose rows behind the last hold NaN scales; and the same bits every time
    g = gen(8)
    wc, ws = mx_ref.random_codes(g, (n,), k, 0)
    xc, xs = mx_ref.random_codes(g, (nb,), k, 0)
    outs = []
    for fill in (0, 255):
        mats = []
        for c, s in ((wc, ws), (xc, xs)):
            m = q4.MXMatrix(0, c.shape[0], k)
            m.tensor.fill_(fill)
            full = q4.MXMatrix.from_codes(c, s, 0)
            q4._check(q4._launch(m.device, q4.lib().q4_mx_pack, c.data_ptr(), s.data_ptr(), m.cref()), "pack")
            assert torch.equal(m.codes()[0], full.codes()[0])
            mats.append(m)
        out = torch.full((nb + 2, n), 7.0, device="cuda")
        q4.q4_mx_gemm(mats[0], mats[1], out=out[1:-1])
        assert bool((out[0] == 7).all() and (out[-1] == 7).all())
        outs.append(out)
    assert torch.equal(outs[0], outs[1])


def test_streams_and_captured_calls(q4):
    g = gen(9)
    W = [q4.q4_mx_quant(randn(g, 700, 1024) * 0.1) for _ in range(2)]
    xs = [randn(g, nb, 1024) for nb in (4, 300)]
    want = [q4.q4_mx_gemm(W[i], xs[i]).clone() for i in range(2)]
    torch.cuda.synchronize()
    # a weight quantised and used at once, on two streams
    raw = [randn(g, 700, 1024) * 0.1 for _ in range(2)]
    wq = [q4.q4_mx_gemm(q4.q4_mx_quant(raw[i]), xs[i]).clone() for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(20):
        got = []
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append((q4.q4_mx_gemm(W[i], xs[i]), q4.q4_mx_gemm(q4.q4_mx_quant(raw[i]), xs[i])))
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(got[i][0], want[i]) and torch.equal(got[i][1], wq[i])
    # captured, replayed on other values, beside each other
    graphs, outs = [], []
    for i in range(2):
        xin, out, ws = xs[i].clone(), torch.empty_like(want[i]), q4.q4_mx_gemm_workspace(W[i], xs[i].shape[0])
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            q4.q4_mx_gemm(W[i], xin, out=out, workspace=ws)
        graphs.append((gr, xin))
        outs.append(out)
    for f in (1.0, -2.0):
        for gr, xin in graphs:
            xin.copy_(xs[0] * f if xin.shape[0] == 4 else xs[1] * f)
        torch.cuda.synchronize()
        for (gr, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for i in range(2):  # a power of two: the same codes, other scales
            assert torch.equal(outs[i], want[i] * f)
    q4.q4_device_check()


def test_refusals(q4):
    x = torch.randn(4, 288, device="cuda")
    W = q4.q4_mx_quant(torch.randn(40, 288, device="cuda"))
    ok = q4.q4_mx_gemm(W, x)
    for bad in (lambda: q4.q4_mx_quant(x.double()), lambda: q4.q4_mx_quant(x[0]), lambda: q4.q4_mx_quant(x[:0]),
                lambda: q4.q4_mx_quant(x[:, :40]), lambda: q4.q4_mx_quant(x.T), lambda: q4.q4_mx_quant(x, 2),
                lambda: q4.q4_mx_quant(x, gamma=torch.ones(32, device="cuda")),
                lambda: q4.q4_mx_quant(x, gamma=torch.ones(288, device="cuda"), up=x),
                lambda: q4.q4_mx_quant(x, up=x[:2]), lambda: q4.q4_mx_quant(x, up=torch.randn(4, 576, device="cuda")[:, ::2]),
                lambda: q4.q4_mx_quant(x, out=W), lambda: q4.q4_mx_quant(x, scale=2.0), lambda: q4.q4_mx_quant(x, 1, scale=0.0),
                lambda: q4.q4_mx_quant(torch.randn(8 * 288 + 1, device="cuda")[1:].view(8, 288)),
                lambda: q4.q4_mx_gemm(W, torch.randn(4, 256, device="cuda")), lambda: q4.q4_mx_gemm(W, x[None]),
                lambda: q4.q4_mx_gemm(W, x, dtype=torch.float64), lambda: q4.q4_mx_gemm(W, x, r=torch.randn(4, 41, device="cuda")),
                lambda: q4.q4_mx_gemm(W, x, r=torch.randn(4, 40, device="cuda").half()),
                lambda: q4.q4_mx_gemm(W, x, out=torch.empty(40, 4, device="cuda").T),
                lambda: q4.q4_mx_gemm(W, x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                lambda: q4.q4_mx_gemm(W, q4.q4_mx_quant(x, 1)), lambda: q4.q4_mx_gemm(W, q4.q4_mx_quant(x), up=x),
                lambda: q4.q4_mx_gemm(q4.q4_mx_quant(torch.randn(2, 40, 288, device="cuda")), x),
                lambda: q4.q4_mx_dequant(W, torch.float64), lambda: q4.q4_mx_dequant(W, out=torch.empty(40, 256, device="cuda")),
                lambda: q4.MXMatrix.from_codes(torch.zeros(4, 16, dtype=torch.uint8, device="cuda"),
                                               torch.zeros(4, 2, dtype=torch.uint8, device="cuda"), 0),
                lambda: q4.MXMatrix(0, 4, 64, tensor=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((TypeError, ValueError, q4.Q4Error)):
            bad()
    # outputs that overlap an input
    buf = torch.randn(4, 288, device="cuda")
    with pytest.raises(ValueError):
        q4.q4_mx_gemm(W, buf, out=buf.view(-1)[:160].view(4, 40))
    r = torch.randn(5, 40, device="cuda")
    with pytest.raises(ValueError):
        q4.q4_mx_gemm(W, x, r=r[:4], out=r[1:])
    assert torch.equal(q4.q4_mx_gemm(W, x), ok)
    q4.q4_device_check()


@pytest.mark.parametrize("nb,n,k,inside", [(1, 512, 4096, False), (40, 300, 1024, False), (300, 300, 4096, False), (2, 640, 8192, True)])
def test_a_wait_that_gives_up_is_reported_and_the_next_call_is_unchanged(q4, nb, n, k, inside):
    g = gen(10)
    W, X = q4.q4_mx_quant(randn(g, n, k)), randn(g, nb, k)
    X = X if inside else q4.q4_mx_quant(X)
    y0 = q4.q4_mx_gemm(W, X)
    q4.q4_device_check()
    q4.q4_debug_wait_limits(copy_wait_cycles=200000, copy_extra_bytes=16)
    try:
        q4.q4_mx_gemm(W, X)
        with pytest.raises(q4.Q4Error) as e:
            q4.q4_device_check()
        assert e.value.status == 6
    finally:
        q4.q4_debug_wait_limits()
    assert torch.equal(q4.q4_mx_gemm(W, X), y0)
    q4.q4_device_check()


def test_offsets_beyond_32_bits(q4):
    # 2.4e9 values of x and of y, 4.8 GB of records: the last rows against those of a small matrix of the same bytes
    k = 65536
    x = torch.empty(37000, k, dtype=BF16, device="cuda").random_(-8, 9)
    for fmt in (0, 1):
        m = q4.q4_mx_quant(x, fmt)
        first = 37000 // 128 * 128
        part = q4.q4_mx_quant(x[first:], fmt)
        used = part.nbytes
        assert torch.equal(q4.q4_mx_dequant(part, BF16), q4.q4_mx_dequant(m, BF16)[first:])
        gamma = torch.ones(k, device="cuda")
        behind = q4.q4_mx_quant(x, fmt, gamma=gamma, eps=1e-6)
        assert torch.equal(q4.q4_mx_dequant(behind, BF16)[first:],
                           q4.q4_mx_dequant(q4.q4_mx_quant(x[first:], fmt, gamma=gamma, eps=1e-6), BF16))
        assert used < m.nbytes
    del x, m, part, behind
    W = q4.MXMatrix(0, 140000, k)
    W.tensor.random_(0, 118)
    last = 140000 // 128
    w = q4.MXMatrix(0, 140000 - 128 * last, k, tensor=W.tensor[last * 256 * 17408:])
    for nb in (1, 50, 90):
        X = q4.MXMatrix(0, nb, k)
        X.tensor.random_(0, 118)
        # (the small matrix's k may be shared by more CTAs: against 64 bits)
        w64, x64 = mx_ref.stored(*w.codes(), 0), mx_ref.stored(*X.codes(), 0)
        ref, S = x64 @ w64.T, x64.abs() @ w64.abs().T
        for y in (q4.q4_mx_gemm(W, X)[:, 128 * last:], q4.q4_mx_gemm(w, X)):
            assert bool(((y.double() - ref).abs() <= bound(ref, S, k, F32)).all())
    del W, w
    W, X = q4.MXMatrix(0, 8192, 64), q4.MXMatrix(0, 300000, 64)
    W.tensor.random_(0, 118), X.tensor.random_(0, 118)
    first = 300000 // 128
    tail = q4.MXMatrix(0, 300000 - 128 * first, 64, tensor=X.tensor[first * 17408:])
    r = torch.zeros(300000, 8192, dtype=F16, device="cuda")
    y = q4.q4_mx_gemm(W, X, r=r, dtype=F16)
    assert torch.equal(y[128 * first:], q4.q4_mx_gemm(W, tail, dtype=F16))
    q4.q4_device_check()


@pytest.mark.parametrize("nb", [1, 8, 9, 70])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_float_rows_onto_the_residual_in_place(q4, nb, dtype):
    g = gen(12)
    W, x, r = q4.q4_mx_quant(randn(g, 512, 288)), randn(g, nb, 288).to(dtype), randn(g, nb, 512).to(dtype)
    want = q4.q4_mx_gemm(W, x, r=r)
    out = r.clone()
    assert q4.q4_mx_gemm(W, x, r=out, out=out) is out and torch.equal(out, want)
    # the result of one product as the rows of the next, without anything in between
    V = q4.q4_mx_quant(randn(g, 288, 512))
    for _ in range(5):
        assert torch.equal(q4.q4_mx_gemm(V, q4.q4_mx_gemm(W, x, r=r)), q4.q4_mx_gemm(V, want))
    q4.q4_device_check()
