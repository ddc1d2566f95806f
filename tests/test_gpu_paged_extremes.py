"""GPU tests of the paged cache's attention at values of very different sizes: what one
sequence, or a later token, holds must not reach another row's bits; and at infinities
that are attended, which give what the formula gives."""
import numpy as np
import pytest

from paged_ref import Pool, attend, check
from parity import case_seed
from test_gpu_paged import DTYPES, I, T, f64, q4  # noqa: F401  (q4: the fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _prefill(q4, k, v, table, q, cu, starts, **kw):  # noqa: F811
    """k, v: float32 [pages][Hkv][page][D] arrays; also checks the error word."""
    out = q4.q4_attn_prefill(T(q), q4.KVPages(T(k), T(v), I(table)), I(cu), I(starts), **kw)
    q4.q4_device_check()
    return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("big_k,big_v", [(2.0 ** 30, 2.0 ** 30), (1.0, 2.0 ** 45), (2.0 ** 60, 1.0), (2.0 ** -60, 2.0 ** -60)])
def test_sequences_do_not_share_precision(q4, D, big_k, big_v):  # noqa: F811
    # fp32: two sequences in one call, one with far larger (or smaller) values: the
    # other's output is that of the sequence alone, bit for bit
    rng = np.random.default_rng(case_seed("share", D, big_v))
    H, Hkv, page, n = 8, 2, 32, [300, 300]
    npg = 10
    k, v = (rng.standard_normal((2 * npg, Hkv, page, D)).astype(np.float32) for _ in range(2))
    k[:npg] *= big_k
    v[:npg] *= big_v
    q = rng.standard_normal((400, H, D)).astype(np.float32)
    q[:200] /= big_k
    table = np.arange(2 * npg).reshape(2, npg).tolist()
    both = _prefill(q4, k, v, table, q, [0, 200, 400], [100, 100])
    alone = _prefill(q4, k, v, table[1:], q[200:], [0, 200], [100])
    assert torch.equal(both[200:], alone)
    # and it is the formula's
    ks, vs, got = (x.astype(np.float64) for x in (k, v, f64(both)))
    for b in range(2):
        K, V = (x[npg * b:npg * (b + 1)].transpose(0, 2, 1, 3).reshape(-1, Hkv, D) for x in (ks, vs))
        for i in (0, 1, 27, 28, 29, 130, 199):
            for h in (0, 3, 7):
                p = 100 + i
                ref, bound = attend(q[200 * b + i, h].astype(np.float64), K[:p + 1, h // 4], V[:p + 1, h // 4], D ** -0.5)
                check(got[200 * b + i, h], ref, bound + 1e-38, "b=%d i=%d h=%d" % (b, i, h))


@pytest.mark.parametrize("D", [64, 128])
def test_shared_pages_attended_to_different_lengths(q4, D):  # noqa: F811
    # fp32: two sequences over the same pages, one reaching far larger values behind
    # the other's end (in the same page): the shorter one's bits are its own
    rng = np.random.default_rng(case_seed("lengths", D))
    k, v = (rng.standard_normal((4, 1, 64, D)).astype(np.float32) for _ in range(2))
    for x in (k, v):
        x[2, 0, 10:] *= 2.0 ** 40
    q = rng.standard_normal((90, 4, D)).astype(np.float32)
    table = [[0, 1, 2, 3], [0, 1, 2, 3]]
    both = _prefill(q4, k, v, table, q, [0, 40, 90], [98, 150])
    alone = _prefill(q4, k, v, table[:1], q[:40], [0, 40], [98])
    assert torch.equal(both[:40], alone)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("factor", [2.0 ** 20, 2.0 ** 45, 2.0 ** -45])
def test_rows_do_not_follow_later_tokens(q4, D, factor):  # noqa: F811
    # fp32, one prompt: later positions (of the same key tiles, and of later ones)
    # become far larger; no earlier row changes a bit
    rng = np.random.default_rng(case_seed("later", D, factor))
    rows, first = 330, 150
    k, v = (rng.standard_normal((1, 2, 384, D)).astype(np.float32) for _ in range(2))
    q = rng.standard_normal((rows, 4, D)).astype(np.float32)
    outs = []
    for f in (1.0, factor):
        k2, v2 = k.copy(), v.copy()
        k2[:, :, first:] *= f
        v2[:, :, first:] *= f
        outs.append(_prefill(q4, k2, v2, [[0]], q, [0, rows], [0]))
    assert torch.equal(outs[0][:first], outs[1][:first])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ln_w,big", [(-30.0, 2.0 ** 40), (-60.0, 2.0 ** 80), (-60.0, 2.0 ** 90), (-20.0, 2.0 ** 60),
                                      (0.0, 2.0 ** -60)])
def test_large_values_of_small_weight(q4, D, ln_w, big):  # noqa: F811
    # fp32: some positions' values are `big` times the others' at e^ln_w times their
    # weight, in the same key tile and in another.  The values enter with 22 bits or to
    # 2^-27 of their row's largest, R_j, which is scaled into [2^2, 2^14).  The weights
    # times the rows' scales enter with 22 bits or to 2^-25 when the largest of them is
    # 2^13: off by 2^-38 of it, by a value below 2^14, over a row's scale of R_j / 2^2 at
    # most: 2^-26 of max_j w_j R_j a position
    rng = np.random.default_rng(case_seed("small weight", D, ln_w, big))
    n, at = 300, np.array([5, 70, 131, 250])
    k = np.zeros((1, 1, n, D), np.float32)
    k[0, 0, at, 0] = 1.0
    v = rng.standard_normal((1, 1, n, D)).astype(np.float32)
    v[0, 0, at] *= big
    q = np.zeros((1, 1, D), np.float32)
    q[0, 0, 0] = -1.0  # the scale is not negative
    got = f64(_prefill(q4, k, v, [[0]], q, [0, 1], [n - 1], scale=abs(ln_w)))[0, 0]
    K, V = k[0, 0].astype(np.float64), v[0, 0].astype(np.float64)
    ref, bound = attend(q[0, 0].astype(np.float64), K, V, -ln_w)
    s = -ln_w * (K @ q[0, 0])
    w = np.exp(s - s.max())
    w /= w.sum()
    rowmax = np.abs(V).max(1)
    bound = bound + 3 * 2.0 ** -22 * (w @ np.abs(V)) + 2.0 ** -27 * (w @ rowmax) + n * 2.0 ** -26 * (w * rowmax).max()
    check(got, ref, bound, "small weights")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("eq,ek,ev", [(100, -96, 0), (-108, 108, 96), (0, 0, -84), (-80, -84, 0), (100, -100, 0),
                                      (-100, 100, 100), (0, 0, -90), (7, -5, 11)])
def test_powers_of_two_change_nothing(q4, D, eq, ek, ev):  # noqa: F811
    # fp32: q, k and v times powers of two.  Of q any, of k and v the scales' steps of
    # 2^12: the same bits, scaled; others: the formula's.  (Scores that leave fp32's
    # range at the bottom: the mean of the attended values.)
    rng = np.random.default_rng(case_seed("powers", D))
    rows, f = 140, [np.float32(2.0 ** e) for e in (eq, ek, ev)]
    k, v = (rng.standard_normal((1, 1, rows, D)).astype(np.float32) for _ in range(2))
    q = rng.standard_normal((rows, 2, D)).astype(np.float32)
    gone = eq + ek < -140
    got = _prefill(q4, k * f[1], v * f[2], [[0]], q * f[0], [0, rows], [0], scale=D ** -0.5 / (1.0 if gone else 2.0 ** (eq + ek)))
    if ek % 12 == 0 and ev % 12 == 0:
        want = _prefill(q4, k, v, [[0]], q, [0, rows], [0], scale=0.0 if gone else D ** -0.5)
        assert torch.equal(want * float(f[2]), got)
    K, V, got = k[0, 0].astype(np.float64), v[0, 0].astype(np.float64), f64(got) / float(f[2])
    for i in range(0, rows, 3):
        for h in range(2):
            ref, bound = attend(q[i, h].astype(np.float64), K[:i + 1], V[:i + 1], 0.0 if gone else D ** -0.5)
            check(got[i, h], ref, bound, "i=%d h=%d" % (i, h))


@pytest.mark.parametrize("D", [64, 128])
def test_values_of_zero_and_a_page_of_zeros(q4, D):  # noqa: F811
    rng = np.random.default_rng(case_seed("zeros", D))
    rows = 200
    k, v = (rng.standard_normal((1, 1, rows, D)).astype(np.float32) for _ in range(2))
    v[0, 0, :150:2] = 0.0
    k[0, 0, 40:60] = 0.0
    q = rng.standard_normal((rows, 2, D)).astype(np.float32)
    q[7] = 0.0
    got = f64(_prefill(q4, k, v, [[0]], q, [0, rows], [0]))
    K, V = k[0, 0].astype(np.float64), v[0, 0].astype(np.float64)
    for i in range(0, rows, 3):
        for h in range(2):
            ref, bound = attend(q[i, h].astype(np.float64), K[:i + 1], V[:i + 1], D ** -0.5)
            check(got[i, h], ref, bound + 1e-30, "zeros %d" % i)
    assert not f64(_prefill(q4, k, v * 0, [[0]], q, [0, rows], [0])).any()


# ------------------------------------------------------------------ infinities

def _formula(q, K, V, scale):
    """The definition in 64 bits with IEEE rules: weights of +inf scores are NaN, of
    -inf scores 0 (all of them -inf: NaN), an attended infinity is one."""
    with np.errstate(all="ignore"):
        s = scale * (K @ q)
        w = np.exp(s - s.max())
        w /= w.sum()
        return w @ V


def _same(got, ref, tol, what):
    """NaN and infinities where the formula has them, the rest within tol (below: scores
    off by 2 (D + 16) 2^-24 A, A = scale sum |q k| < 8 for q of 0.5, so 2^-12 of the
    values' scale, 1 here, covers it with the sums and the exponential)."""
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]) and np.isfinite(got[~inf & ~np.isnan(ref)]).all(), what
    fin = np.isfinite(ref)
    assert (np.abs(got[fin] - ref[fin]) <= tol * (1 + np.abs(ref[fin]))).all(), what


INF = float("inf")
# (which of k and v, position from the end, dim, value)
INFS = {"v": [("v", 3, 5, INF)], "v both": [("v", 3, 5, INF), ("v", 40, 6, -INF)],
        "v cancels": [("v", 3, 5, INF), ("v", 2, 5, -INF)], "v nan": [("v", 7, 9, float("nan"))],
        "k": [("k", 11, 2, INF)], "new": [("v", 0, 1, -INF)], "k new": [("k", 0, 1, INF)],
        "far": [("v", 299, 63, INF), ("k", 290, 0, -INF)]}


def _with_infs(rng, n, Hkv, D, t, infs):
    """k, v [n][Hkv][D] in the cache's type, the infinities in kv head 1."""
    k, v = (torch.from_numpy(rng.standard_normal((n, Hkv, D)).astype(np.float32)).to(t) for _ in range(2))
    for which, back, dim, x in infs:
        (k if which == "k" else v)[n - 1 - back, 1, dim] = x
    return k, v


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("case", list(INFS))
def test_prefill_attended_infinities(q4, dtype, D, case):  # noqa: F811
    t, H, Hkv, n, rows = DTYPES[dtype], 6, 2, 300, 40
    rng = np.random.default_rng(case_seed("inf prompt", dtype, D))
    k, v = _with_infs(rng, n, Hkv, D, t, INFS[case])
    q = torch.from_numpy((0.5 * rng.standard_normal((rows, H, D))).astype(np.float32)).to(t)
    pages = q4.KVPages(*(x.transpose(0, 1)[None].contiguous().cuda() for x in (k, v)), I([[0]]))
    got = f64(q4.q4_attn_prefill(q.cuda(), pages, I([0, rows]), I([n - rows])))
    q4.q4_device_check()
    K, V, Q = k.double().numpy(), v.double().numpy(), q.double().numpy()
    for i in range(rows):
        p = n - rows + i
        for h in range(H):
            ref = _formula(Q[i, h], K[:p + 1, h // 3], V[:p + 1, h // 3], D ** -0.5)
            # three roundings of the 16-bit types (q is given): weights, output, and a margin of one
            _same(got[i, h], ref, 2.0 ** -12 + 3 * float(torch.finfo(t).eps) / 2, "%s i=%d h=%d" % (case, i, h))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_scores_all_minus_infinity(q4, dtype, D):  # noqa: F811
    # every attended key is -inf against a positive q: 0 / 0, as the formula has it (the
    # other head's q is negative: +inf, NaN too); the other sequence is untouched
    t = DTYPES[dtype]
    k = torch.full((2, 1, 160, D), 0.25, dtype=t, device="cuda")
    k[0, 0, :, 3] = -INF
    pages = q4.KVPages(k, torch.ones_like(k), I([[0], [1]]))
    q = torch.ones(40, 2, D, device="cuda", dtype=t)
    q[:, 1] = -1.0
    got = q4.q4_attn_prefill(q, pages, I([0, 20, 40]), I([100, 100])).float()
    q4.q4_device_check()
    # the others' values are ones: weights that add up to one, rounded once
    assert torch.isnan(got[:20]).all()
    assert float((got[20:] - 1).abs().max()) <= float(torch.finfo(t).eps) + 2.0 ** -17


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_scale_zero_takes_the_same_path(q4, dtype, D):  # noqa: F811
    # masked scores must not become -inf * 0: rows of NaN weights are taken one by one,
    # a hundred times as long and more.  The values are multiples of 1/8, so their sums
    # are exact, and the mean is off by its division and the output's rounding
    t, rows = DTYPES[dtype], 1024
    v = torch.from_numpy(np.random.default_rng(5).integers(-8, 9, (1, 2, rows, D)).astype(np.float32) / 8)
    k = torch.from_numpy(np.random.default_rng(6).standard_normal((1, 2, rows, D)).astype(np.float32))
    q = torch.from_numpy(np.random.default_rng(7).standard_normal((rows, 8, D)).astype(np.float32)).to(t).cuda()
    pages = q4.KVPages(k.to(t).cuda(), v.to(t).cuda(), I([[0]]))
    args, ws = (q, pages, I([0, rows]), I([0])), q4.q4_attn_prefill_workspace(pages, rows, 8)
    out = torch.empty_like(q)
    took = []
    for scale in (None, 0.0):
        q4.q4_attn_prefill(*args, scale=scale, out=out, workspace=ws)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(3):
            q4.q4_attn_prefill(*args, scale=scale, out=out, workspace=ws)
        b.record()
        torch.cuda.synchronize()
        took.append(a.elapsed_time(b))
    assert took[1] < 10 * took[0], took
    mean = v[0].double().cumsum(1) / torch.arange(1, rows + 1).double()[:, None]
    got = out.double().cpu().view(rows, 2, 4, D).permute(1, 2, 0, 3)
    err = (got - mean[:, None]).abs()
    assert bool((err <= (2.0 ** -18 + float(torch.finfo(t).eps) / 2 * mean.abs()[:, None])).all()), float(err.max())


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_of_nan_ends_soon(q4, dtype, D):  # noqa: F811
    # a prompt whose q is NaN is NaN, and whose rows all are: each is taken by the
    # definition, which must not walk on once its weights are NaN (75 ms against 0.04)
    t, rows = DTYPES[dtype], 1024
    k, v = (torch.randn(1, 2, rows, D, device="cuda").to(t) for _ in range(2))
    q = torch.randn(rows, 8, D, device="cuda").to(t)
    pages = q4.KVPages(k, v, I([[0]]))
    ws = q4.q4_attn_prefill_workspace(pages, rows, 8)
    took = []
    for bad in (False, True):
        if bad:
            q[:, :, 3] = float("nan")
        out = q4.q4_attn_prefill(q, pages, I([0, rows]), I([0]), workspace=ws)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        cu, st = I([0, rows]), I([0])
        a.record()
        for _ in range(3):
            q4.q4_attn_prefill(q, pages, cu, st, out=out, workspace=ws)
        b.record()
        torch.cuda.synchronize()
        took.append(a.elapsed_time(b))
        assert bool(torch.isnan(out).all()) == bad and bool(torch.isfinite(out).all()) != bad
    assert took[1] < 200 * took[0], took


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H,D,n", [(8, 64, 300), (24, 128, 300), (8, 64, 9000), (2, 128, 300)])
@pytest.mark.parametrize("case", list(INFS))
def test_paged_attended_infinities(q4, dtype, H, D, n, case):  # noqa: F811
    # whole in one CTA's share or joined from many; q, k, v of order one: no weight is
    # zero, so an infinity is attended wherever its position is
    t, Hkv = DTYPES[dtype], 2
    rng = np.random.default_rng(case_seed("inf", dtype, H, D, n))
    k, v = _with_infs(rng, n, Hkv, D, t, INFS[case])
    q = (0.5 * rng.standard_normal((2, H, D))).astype(np.float32)
    # sequence 1 is finite: a part of the same positions
    page, npg = 128, -(-n // 128)
    pool = torch.full((2, 2 * npg, Hkv, page, D), float("nan"), dtype=t)
    for i, x in enumerate((k, v)):
        flat = pool[i].transpose(1, 2).reshape(2 * npg * page, Hkv, D)
        flat[:n - 1] = x[:n - 1]
        flat[npg * page:npg * page + 200] = torch.nan_to_num(x[:200].float(), 0.5, 0.5, 0.5).to(t)
        pool[i] = flat.reshape(2 * npg, page, Hkv, D).transpose(1, 2)
    pages = q4.KVPages(pool[0].cuda(), pool[1].cuda(), I(np.arange(2 * npg).reshape(2, npg).tolist()))
    new = [torch.stack([x[n - 1].float(), torch.ones(Hkv, D)]).cuda() for x in (k, v)]
    got = q4.q4_attn_paged(T(q), *new, pages, I([n - 1, 200]))
    assert torch.equal(got.view(torch.int32), q4.q4_attn_paged(T(q), *new, pages, I([n - 1, 200])).view(torch.int32))
    q4.q4_device_check()
    got = f64(got)
    K, V = k.double().numpy(), v.double().numpy()
    assert np.isfinite(got[1]).all()
    for h in range(H):
        hk = h // (H // Hkv)
        ref = _formula(q[0, h].astype(np.float64), K[:, hk], V[:, hk], D ** -0.5)
        _same(got[0, h], ref, 2.0 ** -12, "%s h=%d" % (case, h))


@pytest.mark.parametrize("D", [64, 128])
def test_paged_values_that_overflow_the_cache(q4, D):  # noqa: F811
    # f16: a new value beyond 65504 is stored as infinity, and attended as one
    n = 30
    pages = q4.KVPages(torch.zeros(1, 1, 32, D, device="cuda", dtype=torch.float16),
                       torch.ones(1, 1, 32, D, device="cuda", dtype=torch.float16), I([[0]]))
    f = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    v = f(1, 1, D)
    v[0, 0, 7], v[0, 0, 8] = 1e5, -1e5
    got = f64(q4.q4_attn_paged(f(1, 4, D) + 1, f(1, 1, D), v, pages, I([n - 1])))[0]
    ref = np.full(D, (n - 1) / n)
    ref[7], ref[8] = INF, -INF
    for h in range(4):
        _same(got[h], ref, 2.0 ** -20, "overflow")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [150, 9000])
def test_paged_scores_all_minus_infinity(q4, dtype, D, n):  # noqa: F811
    t = DTYPES[dtype]
    k = torch.full((2, 1, n + 10, D), 0.25, dtype=t, device="cuda")
    k[0, 0, :, 3] = -INF
    pages = q4.KVPages(k, torch.ones_like(k), I([[0], [1]]))
    q = torch.ones(2, 2, D, device="cuda")
    q[:, 1] = -1.0
    kn = torch.stack([k[0, :, 0].float(), k[1, :, 0].float()])
    got = q4.q4_attn_paged(q, kn, torch.ones_like(kn), pages, I([n - 1, n - 1]))
    q4.q4_device_check()
    assert torch.isnan(got[0]).all() and float((got[1] - 1).abs().max()) <= (n / 4 + 64) * 2.0 ** -24 + 2.0 ** -20


def test_paged_pages_that_are_all_gone(q4):  # noqa: F811
    # no attended position has a page: zeros, and recorded
    pages = q4.KVPages(torch.ones(2, 1, 16, 64, device="cuda"), torch.ones(2, 1, 16, 64, device="cuda"), I([[7, -1], [0, 1]]))
    x = torch.ones(2, 3, 64, device="cuda")
    new = torch.ones(2, 1, 64, device="cuda")
    got = q4.q4_attn_paged(x, new, new, pages, I([20, 20]))
    with pytest.raises(q4.Q4Error):
        q4.q4_device_check()
    assert not got[0].any() and float((got[1] - 1).abs().max()) <= 2.0 ** -18


# ------------------------------------------------------------------ fp32 prompts of mixed sizes

@pytest.mark.parametrize("H,Hkv,D", [(32, 8, 64), (4, 4, 128), (6, 2, 64), (7, 1, 128), (16, 1, 128)])
@pytest.mark.parametrize("rows,starts,window,page", [([1], [0], 0, 16), ([33, 0, 1, 130], [0, 4, 77, 0], 0, 48),
                                                     ([257, 64], [100, 0], 70, 64), ([5], [400], 0, 128), ([300], [0], 1, 256),
                                                     ([150], [51], 0, 201), ([700, 90, 600], [0, 500, 33], 300, 16)])
def test_prefill_values_of_mixed_sizes(q4, H, Hkv, D, rows, starts, window, page):  # noqa: F811
    # fp32: every position's k and v have a size of their own, in some sequences' parts
    # the usual one, so that each way of taking the factors meets the others in one call
    rng = np.random.default_rng(case_seed("mixed", H, D, rows, window))
    lens = [s + r for s, r in zip(starts, rows)]
    pool = Pool(rng, [max(1, x) for x in lens], Hkv, page, D, torch.float32)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        kv = rng.standard_normal((2, n, Hkv, D)).astype(np.float32)
        wild = (np.arange(n) // 100 % 2 == 0) if b % 2 == 0 else np.zeros(n, bool)
        kv[0, wild] *= np.exp2(rng.integers(-30, 3, (int(wild.sum()), Hkv, 1))).astype(np.float32)
        kv[1, wild] *= np.exp2(rng.integers(-40, 40, (int(wild.sum()), Hkv, 1))).astype(np.float32)
        kv[:, rng.integers(0, n, 2)] = 0.0
        pool.put(b, np.arange(n), *kv)
    dev, used = pool.device(q4), sum(rows)
    q = rng.standard_normal((used + 2, H, D)).astype(np.float32)
    cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
    outs = []
    for _ in range(2):
        out = torch.full((used + 2, H, D), 9.0, device="cuda")
        outs.append(q4.q4_attn_prefill(T(q), dev, I(cu), I(starts), window=window, out=out))
    q4.q4_device_check()
    assert torch.equal(outs[0], outs[1]) and bool((outs[0][used:] == 9.0).all())
    got = f64(outs[0])
    sc = D ** -0.5
    for b, r in enumerate(rows):
        K, V = (pool.get(x, b, np.arange(lens[b])) for x in (pool.k, pool.v))
        for i in range(r) if r <= 40 else sorted({0, 1, r - 1, r - 2, *rng.integers(0, r, 24).tolist()}):
            p = starts[b] + i
            lo = max(0, p + 1 - window) if window else 0
            for h in range(H) if H <= 8 else sorted({0, H - 1, *rng.integers(0, H, 4).tolist()}):
                q1, K1, V1 = q[cu[b] + i, h].astype(np.float64), K[lo:p + 1, h // (H // Hkv)], V[lo:p + 1, h // (H // Hkv)]
                ref, bound = attend(q1, K1, V1, sc)
                s = sc * (K1 @ q1)
                w = np.exp(s - s.max())
                w /= w.sum()
                # the parts: of v and of the weights as in test_large_values_of_small_weight; of
                # k 22 bits or 2^-27 of its row's largest, so a score by 2^-27 |q| max |k|, twice
                rv, rk = np.abs(V1).max(1), np.abs(K1).max(1)
                bound = bound + (3 * 2.0 ** -22 + 2 * 2.0 ** -27 * sc * np.abs(q1).sum() * rk.max()) * (w @ np.abs(V1))
                bound = bound + 2.0 ** -27 * (w @ rv) + len(w) * 2.0 ** -26 * (w * rv).max()
                check(got[cu[b] + i, h], ref, bound + 1e-30, "mixed b=%d i=%d h=%d" % (b, i, h))


@pytest.mark.parametrize("D", [64, 128])
def test_waits_give_up_with_factors_of_their_own(q4, D):  # noqa: F811
    # a copy that never completes while the positions' factors are looked at: the call
    # ends and records it, and the next one has its usual bits
    rng = np.random.default_rng(case_seed("give up", D))
    k, v = (rng.standard_normal((1, 2, 400, D)).astype(np.float32) for _ in range(2))
    v[:, :, ::3] *= 2.0 ** 30
    q = rng.standard_normal((400, 8, D)).astype(np.float32)
    want = _prefill(q4, k, v, [[0]], q, [0, 400], [0])
    q4.q4_debug_wait_limits(copy_wait_cycles=200000, copy_extra_bytes=16)
    try:
        with pytest.raises(q4.Q4Error) as e:
            _prefill(q4, k, v, [[0]], q, [0, 400], [0])
        assert e.value.status == 6
    finally:
        q4.q4_debug_wait_limits()
    assert torch.equal(want, _prefill(q4, k, v, [[0]], q, [0, 400], [0]))


@pytest.mark.parametrize("D", [64, 128])
def test_captured_prompt_follows_the_sizes_of_its_values(q4, D):  # noqa: F811
    # fp32: one captured call, its values usual, mixed and usual again (the workspace
    # keeps what the call before left), beside another prompt on a second stream
    rng = np.random.default_rng(case_seed("captured sizes", D))
    rows, page, npg = 500, 64, 8
    kv = [T(rng.standard_normal((2, npg, 2, page, D)).astype(np.float32)) for _ in range(2)]
    mixed = [x.clone() for x in kv]
    for x in mixed:
        x[1] *= torch.exp2(torch.from_numpy(rng.integers(-30, 30, (npg, 2, page, 1))).cuda().float())
    q = [T(rng.standard_normal((rows, 8, D)).astype(np.float32)) for _ in range(2)]
    table, cu, st = I([list(range(npg))]), I([0, rows]), I([7])
    buf = [x.clone() for x in kv]
    pages = [q4.KVPages(x[0], x[1], table) for x in buf]
    ws = [q4.q4_attn_prefill_workspace(p, rows, 8) for p in pages]
    out = [torch.empty_like(x) for x in q]
    alone = {}
    for name, vals in (("usual", kv), ("mixed", mixed)):
        alone[name] = []
        for i in range(2):
            p = q4.KVPages(vals[i][0].clone(), vals[i][1].clone(), table)
            alone[name].append(q4.q4_attn_prefill(q[i], p, cu, st))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q4.q4_attn_prefill(q[0], pages[0], cu, st, out=out[0], workspace=ws[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.q4_attn_prefill(q[0], pages[0], cu, st, out=out[0], workspace=ws[0])
    for a, b in (("usual", "mixed"), ("mixed", "usual"), ("mixed", "mixed"), ("usual", "usual")):
        for i, name in ((0, a), (1, b)):
            buf[i].copy_(kv[i] if name == "usual" else mixed[i])
            out[i].zero_()
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            for _ in range(3):
                q4.q4_attn_prefill(q[1], pages[1], cu, st, out=out[1], workspace=ws[1])
        torch.cuda.synchronize()
        assert torch.equal(out[0], alone[a][0]) and torch.equal(out[1], alone[b][1])
    q4.q4_device_check()
