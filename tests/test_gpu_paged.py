"""GPU tests of the paged KV cache: q4_kv_append, q4_attn_prefill and
q4_attn_paged against plain 64-bit forms (paged_ref), one by one and as a
request uses them.  Unwritten cache positions hold NaN, so any read of them
shows."""
import numpy as np
import pytest

from paged_ref import U32, Pool, attend, check, half_step, rope64, rotate
from parity import case_seed

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def q4():
    import bit_weight_quantized_q4_gb300 as m
    m.build()
    m.lib()
    return m


def T(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def I(a):  # noqa: E743
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().cpu().double().numpy()


def _rounded(x, dtype):
    return torch.from_numpy(np.asarray(x, np.float32)).to(dtype).double().numpy()


# ------------------------------------------------------------------ append

def _append_case(q4, dtype, H, Hkv, D, page, rows, starts, rope, tail, seed, with_q=True):
    rng = np.random.default_rng(seed)
    lens = [s + r for s, r in zip(starts, rows)]
    pool = Pool(rng, lens, Hkv, page, D, dtype)
    dev = pool.device(q4)
    n = sum(rows) + tail
    q, k, v = (rng.standard_normal((n, h, D)).astype(np.float32) for h in (H, Hkv, Hkv))
    cu = np.concatenate([[0], np.cumsum(rows)])
    c, s = rope64(max(lens) + 1, D)
    q_out = torch.full((n, H, D), 7.0, dtype=dtype, device="cuda")
    got = q4.q4_kv_append(T(k), T(v), dev, I(cu.tolist()), I(starts), q=T(q) if with_q else None,
                          rope=(T(c), T(s)) if rope else None, q_out=q_out if with_q else None)
    kd, vd = dev.k.cpu(), dev.v.cpu()
    kept_k, kept_v = pool.k.clone(), pool.v.clone()
    eps = half_step(dtype)
    for b, r in enumerate(rows):
        if r == 0:
            continue
        pos = np.arange(starts[b], starts[b] + r)
        sl = slice(cu[b], cu[b + 1])
        pg, slot = pool.where(b, pos)
        kept_k[pg, :, slot] = kd[pg, :, slot]
        kept_v[pg, :, slot] = vd[pg, :, slot]
        assert np.array_equal(pool.get(vd, b, pos), _rounded(v[sl], dtype)), "v"
        for name, x, y in (("k", k[sl], pool.get(kd, b, pos)), ("q", q[sl], f64(q_out[sl]))):
            if name == "q" and not with_q:
                continue
            if not rope:
                assert np.array_equal(y, _rounded(x, dtype)), name
                continue
            ref, off = rotate(x.astype(np.float64), c[pos][:, None].astype(np.float64), s[pos][:, None].astype(np.float64))
            check(y, ref, eps * np.abs(ref) + (1 + eps) * off + 2.0 ** -25, "append " + name)
    # nothing else moved: other slots, other pages, rows behind the last sequence
    assert torch.equal(kept_k.view(torch.uint8), kd.view(torch.uint8)) and torch.equal(kept_v.view(torch.uint8), vd.view(torch.uint8))
    if with_q:
        assert torch.all(q_out[n - tail:] == 7.0) if tail else True
        assert got is q_out
    q4.q4_device_check()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H,Hkv,D,page", [(32, 8, 64, 16), (6, 2, 128, 48), (1, 1, 64, 64), (16, 1, 128, 128)])
@pytest.mark.parametrize("rows,starts,rope,tail", [([1], [0], True, 0), ([3, 0, 20, 1], [5, 9, 0, 200], True, 2),
                                                   ([17, 33], [15, 47], False, 0)])
def test_append(q4, dtype, H, Hkv, D, page, rows, starts, rope, tail):
    _append_case(q4, DTYPES[dtype], H, Hkv, D, page, rows, starts, rope, tail, case_seed("append", dtype, H, D, rows))


def test_append_many_sequences_and_no_q(q4):
    # more sequences than threads, most of them with one row, some with none
    rng = np.random.default_rng(3)
    rows = [int(x) for x in rng.integers(0, 3, 700)]
    rows[-1] = 1
    _append_case(q4, torch.float16, 2, 1, 64, 16, rows, [int(x) for x in rng.integers(0, 30, 700)], True, 5, 4)
    _append_case(q4, torch.bfloat16, 2, 1, 64, 16, [4], [0], True, 0, 5, with_q=False)


def test_append_contiguous_cache_as_one_page(q4):
    _append_case(q4, torch.float32, 4, 2, 64, 100, [37], [60], True, 0, 6)


def test_append_nothing(q4):
    pool = Pool(np.random.default_rng(0), [4], 1, 16, 64, torch.float16)
    dev = pool.device(q4)
    e = torch.empty((0, 1, 64), device="cuda")
    assert q4.q4_kv_append(e, e, dev, I([0, 0])) is None
    assert torch.isnan(dev.k).all()


# ------------------------------------------------------------------ single token

def _decode_case(q4, dtype, H, Hkv, D, page, positions, window, rope, seed, scale=None, qmul=1.0, table_width=None):
    rng = np.random.default_rng(seed)
    lens = [max(p, -1) + 1 for p in positions]
    pool = Pool(rng, [max(1, n) for n in lens], Hkv, page, D, dtype, width=table_width)
    for b, p in enumerate(positions):
        if p > 0:
            pool.put(b, np.arange(p), *(rng.standard_normal((2, p, Hkv, D))))
    dev = pool.device(q4)
    n = len(positions)
    q = (qmul * rng.standard_normal((n, H, D))).astype(np.float32)
    kn, vn = (rng.standard_normal((n, Hkv, D)).astype(np.float32) for _ in range(2))
    c, s = rope64(max(lens) + 1, D)
    out = torch.full((n, H, D), 9.0, device="cuda")
    args = (T(q), T(kn), T(vn), dev, I(positions))
    kw = dict(window=window, scale=scale, rope=(T(c), T(s)) if rope else None)
    ws = q4.q4_attn_paged_workspace(dev, H)
    q4.q4_attn_paged(*args, out=out, workspace=ws, **kw)
    again = q4.q4_attn_paged(*args, workspace=ws, **kw)  # the same workspace, the same bits
    assert torch.equal(out, again)
    q4.q4_device_check()
    kd, vd = dev.k.cpu(), dev.v.cpu()
    got = f64(out)
    eps = half_step(dtype)
    G = H // Hkv
    sc = 1 / np.sqrt(D) if scale is None else scale
    for b, p in enumerate(positions):
        if p < 0:
            assert not got[b].any()
            continue
        if rope:
            c1, s1 = c[p].astype(np.float64), s[p].astype(np.float64)
            kr, off = rotate(kn[b].astype(np.float64), c1, s1)
            qr, qoff = rotate(q[b].astype(np.float64), c1, s1)
        else:
            kr, off, qr, qoff = kn[b].astype(np.float64), 0.0, q[b].astype(np.float64), np.zeros_like(q[b])
        check(pool.get(kd, b, [p])[0], kr, eps * np.abs(kr) + (1 + eps) * off + 2.0 ** -25, "appended k")
        assert np.array_equal(pool.get(vd, b, [p])[0], _rounded(vn[b], dtype))
        seen = np.arange(max(0, p + 1 - window) if window else 0, p + 1)
        K, V = pool.get(kd, b, seen), pool.get(vd, b, seen)
        for h in range(H):
            ref, bound = attend(qr[h], K[:, h // G], V[:, h // G], sc)
            # the rotation's own rounding of q, through the scores
            extra = 2 * sc * (np.abs(K[:, h // G]) @ qoff[h]).max() * np.abs(V[:, h // G]).max()
            check(got[b, h], ref, bound + extra + 1e-30, "paged b=%d h=%d" % (b, h))
    return out


GEOM = [(32, 8, 64), (8, 8, 128), (6, 2, 64), (7, 1, 128), (16, 1, 64), (22, 2, 128), (8, 1, 128)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H,Hkv,D", GEOM)
@pytest.mark.parametrize("positions,window,page", [([0], 0, 16), ([299, -1, 15, 16, 0, 127, 128], 0, 48),
                                                   ([700, 63], 100, 64), ([513], 1, 128)])
def test_paged(q4, dtype, H, Hkv, D, positions, window, page):
    _decode_case(q4, DTYPES[dtype], H, Hkv, D, page, positions, window, True,
                 case_seed("paged", dtype, H, D, positions, window))


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_paged_long_context_split_and_joined(q4, dtype):
    # a long sequence among short and idle ones: its splits span many CTAs
    _decode_case(q4, DTYPES[dtype], 8, 2, 64, 64, [20000, 3, -1, 500], 0, True, 21)
    _decode_case(q4, DTYPES[dtype], 4, 1, 128, 256, [9001], 7000, False, 22)


def test_paged_contiguous_cache_as_one_page(q4):
    # a page that is no multiple of 16: a contiguous cache
    _decode_case(q4, torch.float32, 8, 2, 64, 1003, [1002], 0, True, 23)
    _decode_case(q4, torch.float16, 8, 2, 64, 77, [76], 0, True, 24)


def test_paged_many_sequences(q4):
    rng = np.random.default_rng(25)
    _decode_case(q4, torch.bfloat16, 2, 1, 64, 16, [int(x) for x in rng.integers(-1, 40, 1024)], 0, True, 26)


def test_paged_all_idle(q4):
    out = _decode_case(q4, torch.float16, 4, 2, 64, 16, [-1, -5, -1], 0, True, 27)
    assert not out.any()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("qmul", [1e-4, 30.0])
def test_paged_scales(q4, dtype, qmul):
    # nearly uniform weights, and weights that fall on a few positions
    _decode_case(q4, DTYPES[dtype], 8, 2, 128, 32, [333], 0, False, 28, qmul=qmul)


def test_paged_matches_decode_attention(q4):
    # one sequence on a contiguous fp32 cache: q4_attn_decode's own operation
    rng = np.random.default_rng(29)
    H, Hkv, D, ms, pos = 32, 8, 64, 512, 400
    kc, vc = (T(rng.standard_normal((Hkv, ms, D)).astype(np.float32)) for _ in range(2))
    q, kn, vn = (T(rng.standard_normal((h, D)).astype(np.float32)) for h in (H, Hkv, Hkv))
    c, s = q4.rope_table(ms, D)
    rope = (T(c), T(s))
    k2, v2 = kc.clone(), vc.clone()
    a = q4.q4_attn_decode(q, kn, vn, kc, vc, pos, 0, None, rope=rope)
    pages = q4.KVPages(k2[None], v2[None], I([[0]]))
    b = q4.q4_attn_paged(q[None], kn[None], vn[None], pages, I([pos]), rope=rope)[0]
    assert torch.equal(vc, v2) and torch.allclose(kc, k2, rtol=0, atol=1e-6)
    # both within the fp32 attention bound (2^-16 of values of order one)
    assert torch.allclose(a, b, rtol=0, atol=2.0 ** -16)


# ------------------------------------------------------------------ prompts

def _prefill_case(q4, dtype, H, Hkv, D, page, rows, starts, window, seed, tail=0, poison=None, qmul=1.0, scale=None):
    rng = np.random.default_rng(seed)
    lens = [s + r for s, r in zip(starts, rows)]
    pool = Pool(rng, [max(1, x) for x in lens], Hkv, page, D, dtype)
    for b, n in enumerate(lens):
        if n:
            kv = rng.standard_normal((2, n, Hkv, D))
            if poison is not None and b == 0:  # the last positions: seen by the last rows only
                kv[:, n - poison:] = np.nan
                kv[0, n - 1] = np.inf
            pool.put(b, np.arange(n), *kv)
    dev = pool.device(q4)
    n = sum(rows) + tail
    q = torch.from_numpy((qmul * rng.standard_normal((n, H, D))).astype(np.float32)).to(dtype)
    cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
    out = torch.full((n, H, D), 9.0, dtype=dtype, device="cuda")
    ws = q4.q4_attn_prefill_workspace(dev, n, H)
    qd = q.cuda()
    q4.q4_attn_prefill(qd, dev, I(cu), I(starts), window=window, scale=scale, out=out, workspace=ws)
    assert torch.equal(out.view(torch.uint8), q4.q4_attn_prefill(qd, dev, I(cu), I(starts), window=window, scale=scale)
                       .view(torch.uint8)) or tail
    q4.q4_device_check()
    got = f64(out)
    assert (got[cu[-1]:] == 9.0).all()
    G = H // Hkv
    eps = half_step(dtype)
    wtype = None if dtype == torch.float32 else dtype
    sc = 1 / np.sqrt(D) if scale is None else scale
    q64 = q.double().numpy()
    for b, r in enumerate(rows):
        K, V = pool.get(pool.k, b, np.arange(lens[b])), pool.get(pool.v, b, np.arange(lens[b]))
        picks = range(r) if r <= 40 else sorted({0, 1, r - 1, r - 2, *rng.integers(0, r, 24).tolist()})
        for i in picks:
            p = starts[b] + i
            lo = max(0, p + 1 - window) if window else 0
            for h in (range(H) if H <= 8 else sorted({0, H - 1, *rng.integers(0, H, 4).tolist()})):
                x = got[cu[b] + i, h]
                if poison is not None and b == 0 and p >= lens[0] - poison:
                    assert np.isnan(x).all()
                    continue
                ref, bound = attend(q64[cu[b] + i, h], K[lo:p + 1, h // G], V[lo:p + 1, h // G], sc, wtype)
                check(x, ref, bound * (1 + eps) + eps * np.abs(ref) + 2.0 ** -25, "prefill b=%d i=%d h=%d" % (b, i, h))
    return out


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H,Hkv,D", [(32, 8, 64), (4, 4, 128), (6, 2, 64), (7, 1, 128), (16, 1, 128), (2, 1, 64)])
@pytest.mark.parametrize("rows,starts,window,page", [([1], [0], 0, 16), ([33, 0, 1, 130], [0, 4, 77, 0], 0, 48),
                                                     ([257, 64], [100, 0], 70, 64), ([5], [400], 0, 128),
                                                     ([300], [0], 1, 256)])
def test_prefill(q4, dtype, H, Hkv, D, rows, starts, window, page):
    _prefill_case(q4, DTYPES[dtype], H, Hkv, D, page, rows, starts, window,
                  case_seed("prefill", dtype, H, D, rows, window), tail=3)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_prefill_long_prompt(q4, dtype):
    _prefill_case(q4, DTYPES[dtype], 8, 2, 64, 64, [1500, 700], [0, 333], 0, 41)
    _prefill_case(q4, DTYPES[dtype], 2, 1, 128, 16, [1111], [2000], 1500, 42)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_prefill_masked_values_do_not_reach_out(q4, dtype):
    # NaN and infinities in the prompt's last positions: earlier rows do not see them
    _prefill_case(q4, DTYPES[dtype], 4, 2, 64, 32, [200, 50], [10, 0], 0, 43, poison=7)
    _prefill_case(q4, DTYPES[dtype], 4, 2, 128, 32, [140], [0], 60, 44, poison=20)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("qmul", [1e-4, 25.0])
def test_prefill_scales(q4, dtype, qmul):
    _prefill_case(q4, DTYPES[dtype], 4, 2, 64, 64, [290], [0], 0, 45, qmul=qmul)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_stale_values_below_the_window_change_nothing(q4, dtype, D):
    # finite but huge values at positions before every row's window, some of them
    # in the window's own key tile: not a bit of the result may follow them
    rng = np.random.default_rng(case_seed("stale", dtype, D))
    t = DTYPES[dtype]
    start, rows, window, page = 200, 50, 40, 32
    lo, n = start + 1 - window, start + rows
    outs = []
    q = torch.from_numpy(rng.standard_normal((rows, 4, D)).astype(np.float32)).to(t).cuda()
    kv = torch.from_numpy(rng.standard_normal((2, 8, 2, page, D)).astype(np.float32)).to(t)
    table = I([list(range(8))])
    for big in (None, 3e4):
        k, v = kv[0].cuda(), kv[1].cuda()
        if big is not None:
            for x in (k, v):
                flat = x.transpose(1, 2).reshape(8 * page, 2, D).clone()
                flat[:lo] = -big if t == torch.float16 else -big * 1e25
                x.copy_(flat.reshape(8, page, 2, D).transpose(1, 2))
        pages = q4.KVPages(k, v, table)
        outs.append(q4.q4_attn_prefill(q, pages, I([0, rows]), I([start]), window=window))
    q4.q4_device_check()
    assert n <= 8 * page and torch.isfinite(outs[0]).all()
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_prefill_many_small_weights(q4, dtype):
    # one position of weight 1 whose value is zero, 4095 of weight w = 0.7 * 2^-22:
    # f16 and fp32 weights are held to 2^-31 of the largest, bf16 ones to half a
    # step; the output is rounded once; (n / 4 + 64) 2^-24 for the sums, 1e-5 for
    # the scores' fp32 (ln w = -15.6 times 2^-24, twice) and the exponential
    t, D, n, w = DTYPES[dtype], 64, 4096, 0.7 * 2.0 ** -22
    k, v = torch.zeros(1, 1, n, D), torch.ones(1, 1, n, D)
    k[0, 0, 0, 0] = 16.0
    v[0, 0, 0] = 0.0
    q = torch.zeros(1, 1, D)
    q[0, 0, 0] = 1.0
    pages = q4.KVPages(k.to(t).cuda(), v.to(t).cuda(), I([[0]]))
    out = f64(q4.q4_attn_prefill(q.to(t).cuda(), pages, I([0, 1]), I([n - 1]), scale=float(-np.log(w) / 16)))
    ref = w * (n - 1) / (1 + w * (n - 1))
    tol = 1e-5 + (n / 4 + 64) * U32 + (2 * half_step(t) if t == torch.bfloat16 else 2.0 ** -31 / w + half_step(t))
    assert (np.abs(out - ref) <= tol * ref).all(), (out.min(), out.max(), ref)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_prefill_scale_zero_is_the_mean(q4, dtype):
    # every weight is equal, whatever the scores
    _prefill_case(q4, DTYPES[dtype], 4, 2, 64, 32, [150], [20], 0, 51, scale=0.0)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_more_work_than_runs_at_once(q4, dtype, D):
    # several hundred tiles of all sizes, so that a CTA goes from one to the next
    # (other sequences, other row tiles, partly filled key tiles), some of their rows
    # not finite; the second call inside must give the same bits
    _prefill_case(q4, DTYPES[dtype], 32, 8, D, 48, [310, 1, 700, 0, 64, 33, 129, 500, 2, 257, 96, 31],
                  [0, 900, 0, 5, 64, 31, 17, 300, 1000, 3, 200, 1], 0, case_seed("work", dtype, D), poison=40)
    _prefill_case(q4, DTYPES[dtype], 16, 16, D, 16, [400, 90, 222], [0, 400, 7], 100, case_seed("work1", dtype, D))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("step", [3.0, 60.0, 2000.0])
def test_prefill_scores_that_grow_along_the_sequence(q4, dtype, D, step):
    # the maximum grows by `step` (in units of the exponent) every 64 positions, so
    # each key tile outweighs all before it; and by three steps in a descending one.
    # Exact scores (powers of two and small integers), so the plain form's softmax
    # decides the same: one tile counts, its 64 equal weights are 1/64 each
    t, n = DTYPES[dtype], 520
    for sign in (1.0, -1.0):
        k = torch.zeros(1, 1, n, D)
        k[0, 0, :, 0] = (torch.arange(n) // 64).float() * sign
        v = torch.from_numpy(np.random.default_rng(7).standard_normal((1, 1, n, D)).astype(np.float32))
        q = torch.zeros(n, 1, D)
        q[:, 0, 0] = 1.0
        k, v, q = k.to(t), v.to(t), q.to(t)
        pages = q4.KVPages(k.cuda(), v.cuda(), I([[0]]))
        out = f64(q4.q4_attn_prefill(q.cuda(), pages, I([0, n]), I([0]), scale=step))[:, 0]
        q4.q4_device_check()
        K, V = k[0, 0].double().numpy(), v[0, 0].double().numpy()
        for p in (0, 1, 63, 64, 65, 127, 128, 129, 200, 256, 300, 383, 384, 447, 448, 500, 519):
            ref, bound = attend(q[p, 0].double().numpy(), K[:p + 1], V[:p + 1], step, None if t == torch.float32 else t)
            eps = half_step(t)
            check(out[p], ref, bound * (1 + eps) + eps * np.abs(ref) + 2.0 ** -25, "growing %g at %d" % (sign * step, p))


def test_prefill_contiguous_cache_as_one_page(q4):
    _prefill_case(q4, torch.float32, 8, 2, 64, 333, [300], [33], 0, 46)
    _prefill_case(q4, torch.float16, 8, 2, 64, 201, [200], [1], 0, 47)


def test_prefill_many_sequences(q4):
    rng = np.random.default_rng(48)
    rows = [int(x) for x in rng.integers(0, 4, 1024)]
    _prefill_case(q4, torch.float16, 2, 1, 64, 16, rows, [int(x) for x in rng.integers(0, 20, 1024)], 0, 49)


def test_prefill_nothing(q4):
    pool = Pool(np.random.default_rng(0), [4], 1, 16, 64, torch.float16)
    out = q4.q4_attn_prefill(torch.empty((0, 2, 64), dtype=torch.float16, device="cuda"), pool.device(q4), I([0, 0]))
    assert out.shape == (0, 2, 64)


# ------------------------------------------------------------------ pages and positions out of range

@pytest.mark.parametrize("dtype", list(DTYPES))
def test_bad_pages_and_positions_are_recorded(q4, dtype):
    dt = DTYPES[dtype]
    rng = np.random.default_rng(51)
    Hkv, H, D, page = 2, 4, 64, 16
    pool = Pool(rng, [40, 40], Hkv, page, D, dt, spare=0)
    for b in range(2):
        pool.put(b, np.arange(40), *rng.standard_normal((2, 40, Hkv, D)))
    good = pool.device(q4)
    table = pool.table.copy()
    table[1, 1], table[1, 2] = pool.k.shape[0], -7   # out of range on both sides
    bad = q4.KVPages(good.k.clone(), good.v.clone(), T(table))
    q, kn, vn = (T(rng.standard_normal((2, h, D)).astype(np.float32)) for h in (H, Hkv, Hkv))
    want = q4.q4_attn_paged(q, kn, vn, good, I([39, 39]))
    q4.q4_device_check()
    got = q4.q4_attn_paged(q, kn, vn, bad, I([39, 39]))
    with pytest.raises(q4.Q4Error):
        q4.q4_device_check()
    q4.q4_device_check()  # cleared
    assert torch.equal(want[0], got[0]) and torch.isfinite(got[1]).all()
    # a position the table does not have: like an idle row, and recorded
    got = q4.q4_attn_paged(q, kn, vn, good, I([39, 48]))
    assert not got[1].any()
    with pytest.raises(q4.Q4Error):
        q4.q4_device_check()
    k, v = (T(rng.standard_normal((3, Hkv, D)).astype(np.float32)) for _ in range(2))
    before = good.k.clone()
    q4.q4_kv_append(k, v, good, I([0, 3, 3]), I([47, 0]))  # one row fits, two do not
    with pytest.raises(q4.Q4Error):
        q4.q4_device_check()
    changed = (before.view(torch.uint8) != good.k.view(torch.uint8)).flatten(1).any(1)  # bits: NaN differs from itself
    assert changed.sum() == 1
    qr = T(rng.standard_normal((60, H, D)).astype(np.float32)).to(dt)
    a = q4.q4_attn_prefill(qr, good, I([0, 30, 60]), I([0, 0]))
    q4.q4_device_check()
    b = q4.q4_attn_prefill(qr, bad, I([0, 30, 60]), I([0, 0]))
    with pytest.raises(q4.Q4Error):
        q4.q4_device_check()
    assert torch.equal(a[:30], b[:30]) and torch.equal(a[30:46], b[30:46])
    # out of range row offsets: nothing is read or written out of bounds
    for cu, st in (([0, 50, 90], [0, 0]), ([5, 2, 60], [0, 0]), ([0, 30, 60], [-3, 0]), ([0, 30, 60], [30, 2 ** 31 - 40])):
        q4.q4_attn_prefill(qr, good, I(cu), I(st))
        q4.q4_kv_append(T(np.zeros((60, Hkv, D), np.float32)), T(np.zeros((60, Hkv, D), np.float32)), good, I(cu), I(st))
    try:
        q4.q4_device_check()
    except q4.Q4Error:
        pass


# ------------------------------------------------------------------ graphs, streams, a request

def test_captured_calls_follow_their_positions(q4):
    rng = np.random.default_rng(61)
    H, Hkv, D, page = 8, 2, 64, 32
    pool = Pool(rng, [300, 200], Hkv, page, D, torch.bfloat16)
    for b, n in enumerate((300, 200)):
        pool.put(b, np.arange(n), *rng.standard_normal((2, n, Hkv, D)))
    dev, ref = pool.device(q4), pool.device(q4)
    q, kn, vn = (T(rng.standard_normal((2, h, D)).astype(np.float32)) for h in (H, Hkv, Hkv))
    pos = I([5, 7])
    out, ws = torch.empty((2, H, D), device="cuda"), q4.q4_attn_paged_workspace(dev, H)
    qp = T(rng.standard_normal((90, H, D)).astype(np.float32)).to(torch.bfloat16)
    cu, st = I([0, 50, 90]), I([0, 0])
    pws = q4.q4_attn_prefill_workspace(dev, 90, H)
    pout = torch.empty_like(qp)

    def step():
        q4.q4_attn_paged(q, kn, vn, dev, pos, out=out, workspace=ws)
        q4.q4_attn_prefill(qp, dev, cu, st, out=pout, workspace=pws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for p, c, s in (([250, 30], [0, 70, 90], [100, 20]), ([0, -1], [0, 1, 60], [0, 3]), ([299, 199], [0, 90, 90], [5, 0])):
        pos.copy_(I(p))
        cu.copy_(I(c))
        st.copy_(I(s))
        pout.zero_()
        g.replay()
        ref.k.copy_(dev.k)
        ref.v.copy_(dev.v)
        want = q4.q4_attn_paged(q, kn, vn, ref, I(p))
        assert torch.equal(out, want)
        wantp = torch.zeros_like(qp)
        q4.q4_attn_prefill(qp, ref, I(c), I(s), out=wantp)
        assert torch.equal(pout, wantp)
    q4.q4_device_check()


def test_one_workspace_for_calls_of_several_shapes(q4):
    # the counters of a wide batch lie where a narrow one has none
    ws = None
    for H, Hkv, D, positions in ((16, 1, 128, [5000]), (8, 2, 64, [700] * 40), (16, 1, 128, [4000, 100]), (4, 4, 64, [900])):
        rng = np.random.default_rng(len(positions) + D)
        pool = Pool(rng, [p + 1 for p in positions], Hkv, 64, D, torch.bfloat16)
        for b, p in enumerate(positions):
            pool.put(b, np.arange(p), *rng.standard_normal((2, p, Hkv, D)))
        dev = pool.device(q4)
        if ws is None:
            ws = q4.q4_attn_paged_workspace(dev, H)
        q, kn, vn = (T(rng.standard_normal((len(positions), h, D)).astype(np.float32)) for h in (H, Hkv, Hkv))
        want = q4.q4_attn_paged(q, kn, vn, dev, I(positions))
        assert torch.equal(q4.q4_attn_paged(q, kn, vn, dev, I(positions), workspace=ws), want)
        assert int(ws[:1 << 18].view(torch.int32).abs().max()) == 0


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_copy_waits_give_up_and_the_next_call_is_unchanged(q4, dtype):
    rng = np.random.default_rng(65)
    H, Hkv, D = 8, 2, 64
    pool = Pool(rng, [300, 200], Hkv, 32, D, DTYPES[dtype])
    for b, n in enumerate((300, 200)):
        pool.put(b, np.arange(n), *rng.standard_normal((2, n, Hkv, D)))
    dev = pool.device(q4)
    q, kn, vn = (T(rng.standard_normal((2, h, D)).astype(np.float32)) for h in (H, Hkv, Hkv))
    qp = T(rng.standard_normal((90, H, D)).astype(np.float32)).to(DTYPES[dtype])
    ws = q4.q4_attn_paged_workspace(dev, H)

    def calls():
        return (q4.q4_attn_paged(q, kn, vn, dev, I([250, 100]), workspace=ws),
                q4.q4_attn_prefill(qp, dev, I([0, 50, 90]), I([100, 30])))

    want = calls()
    q4.q4_device_check()
    for which in range(2):
        q4.q4_debug_wait_limits(copy_wait_cycles=200000, copy_extra_bytes=16)
        try:
            calls()[which]
            with pytest.raises(q4.Q4Error) as e:
                q4.q4_device_check()
            assert e.value.status == 6
        finally:
            q4.q4_debug_wait_limits()
        for a, b in zip(want, calls()):
            assert torch.equal(a, b)
        q4.q4_device_check()


def test_two_streams_with_a_workspace_each(q4):
    rng = np.random.default_rng(62)
    H, Hkv, D = 8, 2, 128
    outs, wants, keep = [], [], []
    for i in range(2):
        pool = Pool(rng, [3000], Hkv, 64, D, torch.float16)
        pool.put(0, np.arange(3000), *rng.standard_normal((2, 3000, Hkv, D)))
        dev = pool.device(q4)
        q, kn, vn = (T(rng.standard_normal((1, h, D)).astype(np.float32)) for h in (H, Hkv, Hkv))
        wants.append(q4.q4_attn_paged(q, kn, vn, dev, I([2999])))
        keep.append((dev, q, kn, vn, I([2999]), q4.q4_attn_paged_workspace(dev, H), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for dev, q, kn, vn, pos, ws, st in keep:
            with torch.cuda.stream(st):
                outs.append(q4.q4_attn_paged(q, kn, vn, dev, pos, workspace=ws))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, wants[i % 2])


def test_prompts_on_two_streams_and_replayed(q4):
    # two prompts, each more work than runs at once, on two streams at the same time
    # and replayed from a graph while the other runs: the bits of each alone
    cases = []
    for seed, t, D, rows in ((1, torch.float16, 64, [1500, 700]), (2, torch.bfloat16, 128, [900, 1100])):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n, H, Hkv, page = sum(rows), 32, 8, 64
        width = -(-max(rows) // page)
        k, v = (torch.randn(2 * width, Hkv, page, D, device="cuda", generator=g).to(t) for _ in range(2))
        pages = q4.KVPages(k, v, I(np.arange(2 * width).reshape(2, width).tolist()))
        q = torch.randn(n, H, D, device="cuda", generator=g).to(t)
        cases.append((q, pages, I([0, rows[0], n])))
    alone = [q4.q4_attn_prefill(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.empty_like(x) for x in alone]
    torch.cuda.synchronize()
    for _ in range(6):
        for c, s, o in zip(cases, streams, outs):
            with torch.cuda.stream(s):
                o.zero_()
                q4.q4_attn_prefill(*c, out=o)
    torch.cuda.synchronize()
    for x, o in zip(alone, outs):
        assert torch.equal(x, o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            q4.q4_attn_prefill(*cases[0], out=outs[0])
    outs[0].zero_()
    outs[1].zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(streams[0]):
            graph.replay()
        with torch.cuda.stream(streams[1]):
            q4.q4_attn_prefill(*cases[1], out=outs[1])
    torch.cuda.synchronize()
    for x, o in zip(alone, outs):
        assert torch.equal(x, o)
    q4.q4_device_check()


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_request_prompt_then_tokens(q4, dtype):
    """Two requests through quantised projections: the prompts at once (q4_gemm,
    q4_kv_append, q4_attn_prefill), then one token each (q4_gemv, q4_attn_paged,
    q4_argmax's logits, q4_logprobs); the prompt's attention equals that of the
    same rows taken one token at a time."""
    import q4_workloads as wl
    from parity import dev_weight
    dt = DTYPES[dtype]
    rng = np.random.default_rng(63)
    H, Hkv, D, hidden, vocab, page = 8, 2, 64, 256, 500, 16
    Wq, Wk, Wv = (dev_weight(wl.draw_q4_0(rng, n * D, hidden)) for n in (H, Hkv, Hkv))
    Wl = dev_weight(wl.draw_q4_0(rng, vocab, H * D))
    rows = [23, 40]
    n = sum(rows)
    x = T(wl.draw_x(rng, n, hidden))
    cu, start = I([0, 23, 63]), I([0, 0])
    c, s = q4.rope_table(128, D)
    rope = (T(c), T(s))
    pools = [Pool(np.random.default_rng(64), [80, 80], Hkv, page, D, dt).device(q4) for _ in range(2)]
    # the prompt's projections row by row (the single-token path has them as 1..16 row products)
    proj = [torch.cat([q4.q4_gemv(W, x[i:i + 1]) for i in range(n)]).view(n, -1, D) for W in (Wq, Wk, Wv)]
    big = [q4.q4_gemm(W, x).view(n, -1, D) for W in (Wq, Wk, Wv)]
    for a, b in zip(proj, big):
        assert torch.allclose(a, b, rtol=0, atol=2e-2 * float(a.abs().max()))
    q, k, v = proj
    qr = q4.q4_kv_append(k, v, pools[0], cu, start, q=q, rope=rope)
    out = q4.q4_attn_prefill(qr, pools[0], cu, start)
    each = torch.empty((n, H, D), device="cuda")
    for i in range(max(rows)):
        pos = [i if i < r else -1 for r in rows]
        at = [min(i, r - 1) + o for r, o in zip(rows, (0, 23))]
        y = q4.q4_attn_paged(q[at], k[at], v[at], pools[1], I(pos), rope=rope)
        for b in range(2):
            if pos[b] >= 0:
                each[at[b]] = y[b]
    for a, b in ((pools[0].k, pools[1].k), (pools[0].v, pools[1].v)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # 16-bit: q, the weights and the output each rounded to the type; fp32: sums
    # of a few hundred terms.  Values are averages of v, so bounded by |v|max.
    eps = half_step(dt)
    A = float((q.norm(dim=-1).max() * k.norm(dim=-1).max()) / 8)
    tol = float(v.abs().max()) * ((2 * A * eps + 2 * eps if dt != torch.float32 else 0) + 2 * (D + 16) * U32 * A + 2 ** -17)
    assert float((out.float() - each).abs().max()) <= tol
    # the next token of both requests
    xt = T(wl.draw_x(rng, 2, hidden))
    qt, kt, vt = (q4.q4_gemv(W, xt).view(2, -1, D) for W in (Wq, Wk, Wv))
    att = q4.q4_attn_paged(qt, kt, vt, pools[0], I(rows), rope=rope)
    idx, val, logits = q4.q4_argmax(Wl, att.view(2, H * D), want_val=True, want_logits=True)
    lp, ent, tv, ti = q4.q4_logprobs(logits, idx, top=5)
    assert torch.equal(ti[:, 0], idx) and torch.equal(lp, tv[:, 0])
    ref = torch.log_softmax(logits.double(), -1)
    assert torch.allclose(lp.double(), ref.gather(1, idx.long()[:, None])[:, 0], rtol=0, atol=1e-5)
    assert torch.allclose(ent.double(), -(ref.exp() * ref).sum(-1), rtol=0, atol=1e-5)
    q4.q4_device_check()


def test_device_refusals(q4):
    pool = Pool(np.random.default_rng(0), [40], 2, 16, 64, torch.float16)
    dev = pool.device(q4)
    f = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    h = lambda *s: torch.zeros(s, device="cuda", dtype=torch.float16)  # noqa: E731
    with pytest.raises(TypeError):   # the cache's type is wanted
        q4.q4_attn_prefill(f(3, 4, 64), dev, I([0, 3]))
    with pytest.raises(ValueError):  # out must be apart from q
        x = h(3, 4, 64)
        q4.q4_attn_prefill(x, dev, I([0, 3]), out=x)
    with pytest.raises(ValueError):  # strided rows
        q4.q4_attn_prefill(h(3, 8, 64)[:, ::2], dev, I([0, 3]))
    with pytest.raises(ValueError):  # one offset per sequence and one more
        q4.q4_attn_prefill(h(3, 4, 64), dev, I([0, 1, 3]))
    with pytest.raises(q4.Q4Error) as e:  # heads in whole groups
        q4.q4_attn_prefill(h(3, 3, 64), dev, I([0, 3]))
    assert e.value.status == 2
    with pytest.raises(q4.Q4Error) as e:  # 17 query heads a kv head
        q4.q4_attn_paged(f(1, 34, 64), f(1, 2, 64), f(1, 2, 64), dev, I([3]), workspace=torch.zeros(1 << 25, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
    with pytest.raises(q4.Q4Error) as e:
        q4.q4_attn_paged(f(1, 4, 64), f(1, 2, 64), f(1, 2, 64), dev, I([3]), window=-1)
    assert e.value.status == 2
    with pytest.raises(ValueError):
        q4.q4_attn_paged(f(2, 4, 64), f(2, 2, 64), f(2, 2, 64), dev, I([3, 4]))
    with pytest.raises(ValueError):
        q4.q4_attn_paged(f(1, 4, 64), f(1, 2, 64), f(1, 2, 64), dev, I([3]),
                         workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        q4.q4_kv_append(f(3, 2, 64), f(3, 2, 64), dev, I([0, 3]), q_out=h(3, 4, 64))
    with pytest.raises(TypeError):
        q4.KVPages(torch.zeros((1, 1, 16, 64), dtype=torch.int8, device="cuda"), f(1, 1, 16, 64), I([[0]]))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("step", [6.0, 40.0])
def test_prefill_sums_rescaled_in_every_key_tile(q4, D, step):
    # fp32: each key tile's product is added to the sum beside it, and the maximum
    # grows by `step` (log units; e^6 > 2^8) a key tile of 128, so that sum is rescaled
    # right after it was stored, in every row tile of several sequences.  At step 6 the
    # key tile before has a weight of 128 e^-6 = 0.3 in a key tile's first row and
    # 0.0025 in its last, a hundred and five times the bound: a lost one shows
    rng = np.random.default_rng(case_seed("rescaled", D, step))
    H, Hkv, page, rows, starts = 4, 2, 64, [700, 300, 515], [0, 400, 5]
    lens = [s + r for s, r in zip(starts, rows)]
    pool = Pool(rng, lens, Hkv, page, D, torch.float32)
    for b, n in enumerate(lens):
        kv = rng.standard_normal((2, n, Hkv, D)).astype(np.float32)
        kv[0] = 0.0
        kv[0, :, :, 0] = (np.arange(n) // 128)[:, None]
        pool.put(b, np.arange(n), *kv)
    dev = pool.device(q4)
    q = np.zeros((sum(rows), H, D), np.float32)
    q[:, :, 0] = 1.0
    cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
    outs = [q4.q4_attn_prefill(T(q), dev, I(cu), I(starts), scale=step) for _ in range(4)]
    q4.q4_device_check()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    got = f64(outs[0])
    for b, r in enumerate(rows):
        K, V = (pool.get(x, b, np.arange(lens[b])) for x in (pool.k, pool.v))
        for i in sorted({0, r - 1, *(x for e in range(128, 900, 128) for x in (e - 1 - starts[b], e - starts[b], e + 1 - starts[b])
                                     if 0 <= x < r), *rng.integers(0, r, 20).tolist()}):
            p = starts[b] + i
            for h in range(H):
                ref, bound = attend(q[cu[b] + i, h].astype(np.float64), K[:p + 1, h // 2], V[:p + 1, h // 2], step)
                check(got[cu[b] + i, h], ref, bound + 2.0 ** -25, "rescaled b=%d p=%d h=%d" % (b, p, h))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H,Hkv,D", [(32, 8, 64), (4, 4, 128), (6, 2, 64), (7, 1, 128), (16, 1, 128), (2, 1, 64)])
@pytest.mark.parametrize("rows,starts,window,page", [([1], [0], 0, 16), ([33, 0, 1, 130], [0, 4, 77, 0], 0, 48),
                                                     ([257, 64], [100, 0], 70, 64), ([5], [400], 0, 128),
                                                     ([300], [0], 1, 256), ([900, 1200], [0, 300], 0, 64)])
def test_prefill_repeats_its_bits(q4, dtype, H, Hkv, D, rows, starts, window, page):
    # the rows that a call writes are the same bits every time, with rows behind the
    # last sequence (left alone) too, and on workspaces with other contents
    t, rng = DTYPES[dtype], np.random.default_rng(case_seed("repeat", dtype, H, D, rows))
    lens = [s + r for s, r in zip(starts, rows)]
    pool = Pool(rng, [max(1, x) for x in lens], Hkv, page, D, t)
    for b, n in enumerate(lens):
        if n:
            pool.put(b, np.arange(n), *rng.standard_normal((2, n, Hkv, D)))
    dev = pool.device(q4)
    used = sum(rows)
    q = torch.from_numpy(rng.standard_normal((used + 3, H, D)).astype(np.float32)).to(t).cuda()
    cu, st = I(np.concatenate([[0], np.cumsum(rows)]).tolist()), I(starts)
    ws = q4.q4_attn_prefill_workspace(dev, used + 3, H)
    outs = []
    for fill in (0, 255, 63, 127):
        if ws is not None:
            ws.fill_(fill)
        out = torch.full_like(q, 9.0)
        q4.q4_attn_prefill(q, dev, cu, st, window=window, out=out, workspace=ws)
        assert bool((out[used:] == 9.0).all()) and bool(torch.isfinite(out).all())
        outs.append(out[:used].contiguous().view(torch.uint8))
    for o in outs[1:]:
        assert torch.equal(outs[0], o)
    q4.q4_device_check()
