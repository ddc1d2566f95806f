"""GPU tests of q4_logprobs (log probabilities of tokens, entropy, top
alternatives) against a plain 64-bit form: row lengths around the vector and
split sizes, ties, forbidden tokens, NaN and infinities, determinism.

Bounds: an exponential is off by at most 2^-21 relatively plus 2^-24 of its
argument (its product with log2 e; at most 88 where it is not zero), so a sum of
them, in fp32 over at most n / 512 + 64 sequential additions, by rel = 2^-21 +
88 2^-23 + (n / 512 + 64) 2^-24, which is the absolute error of lse beside its
own rounding; the entropy weighs the terms p (x - m) the same way."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def q4():
    import bit_weight_quantized_q4_gb300 as m
    m.build()
    m.lib()
    return m


def _rel(n):
    return 2.0 ** -21 + 88 * 2.0 ** -23 + (n / 512 + 64) * U32


def _check(q4, x, tokens, top):
    """x float32 [rows, n] (host); compares everything with the 64-bit form."""
    rows, n = x.shape
    xd = torch.from_numpy(x).cuda()
    got = q4.q4_logprobs(xd, torch.from_numpy(tokens.astype(np.int32)).cuda(), top=top)
    again = q4.q4_logprobs(xd, torch.from_numpy(tokens.astype(np.int32)).cuda(), top=top)
    for a, b in zip(got, again):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))
    lp, ent, tv, ti = (t.cpu().numpy() for t in got)
    x64 = x.astype(np.float64)
    m = x64.max(1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        d = np.where(np.isneginf(m), -np.inf, x64 - m)
        s = np.exp(d).sum(1, keepdims=True)
        empty = np.isneginf(m[:, 0])
        lse = np.where(empty[:, None], 0.0, m + np.log(s))
        p = np.exp(d) / s
        t = np.where(p > 0, p * d, 0.0)
        want_ent = np.where(empty, 0.0, (np.log(s) - t.sum(1, keepdims=True))[:, 0])
        ent_bound = _rel(n) * (2 + 2 * np.abs(t).sum(1)) + 4 * U32 * np.abs(np.log(s[:, 0]))
        ref = x64 - lse
    bound = _rel(n) + 4 * U32 * (np.abs(lse) + np.abs(np.where(np.isfinite(x64), x64, 0)))
    r = np.arange(rows)
    tok = np.clip(tokens, 0, n - 1)
    want = np.where(tokens < 0, 0.0, ref[r, tok])
    fin = np.isfinite(want)
    assert np.array_equal(fin, np.isfinite(lp)) and np.array_equal(want[~fin], lp[~fin])
    assert (np.abs(lp - want)[fin] <= bound[r, tok][fin]).all()
    assert (np.abs(ent - want_ent) <= np.where(empty, 0.0, ent_bound)).all()
    k = min(top, n)
    order = np.argsort(-x64, axis=1, kind="stable")[:, :k]
    assert np.array_equal(order, ti)
    want = np.take_along_axis(ref, order, 1)
    fin = np.isfinite(want)
    assert np.array_equal(fin, np.isfinite(tv)) and np.array_equal(want[~fin], tv[~fin])
    assert (np.abs(tv - want)[fin] <= np.take_along_axis(bound, order, 1)[fin]).all()
    q4.q4_device_check()


@pytest.mark.parametrize("n", [1, 2, 3, 5, 31, 33, 511, 513, 1000, 2049, 4097, 8191, 65536, 100003])
@pytest.mark.parametrize("rows", [1, 3, 40])
def test_logprobs(q4, n, rows):
    rng = np.random.default_rng(n + rows)
    x = (4 * rng.standard_normal((rows, n))).astype(np.float32)
    for top in (0, 1, 20, 32):
        _check(q4, x, rng.integers(0, n, rows), top)


@pytest.mark.parametrize("rows,n", [(1, 1200003), (2, 140001), (170, 139264)])
def test_rows_longer_than_the_batches_held_apart(q4, rows, n):
    # the largest values 8192 apart and so a thread's own, beside ordinary ones
    rng = np.random.default_rng(n)
    x = (2 * rng.standard_normal((rows, n))).astype(np.float32)
    for r in range(min(rows, 3)):
        at = np.arange(17 + 4 * r, n, 8192)
        x[r, at] = 20 + rng.standard_normal(len(at)).astype(np.float32)
    _check(q4, x, rng.integers(0, n, rows), 32)


def test_more_rows_than_the_device_holds(q4):
    rng = np.random.default_rng(1)
    x = (3 * rng.standard_normal((700, 5001))).astype(np.float32)
    _check(q4, x, rng.integers(-1, 5001, 700), 7)


@pytest.mark.parametrize("rows,n", [(1, 65536), (5, 3001), (400, 2500)])
def test_ties_and_forbidden_tokens(q4, rows, n):
    rng = np.random.default_rng(2)
    tok = rng.integers(0, n, rows)
    _check(q4, np.full((rows, n), 1.5, np.float32), tok, 32)                       # everything equal
    _check(q4, rng.integers(-2, 3, (rows, n)).astype(np.float32), tok, 32)         # long ties
    z = np.where(rng.random((rows, n)) < 0.5, 0.0, -0.0).astype(np.float32)        # the zeros are equal
    _check(q4, z, tok, 20)
    x = np.full((rows, n), -np.inf, np.float32)                                    # a few allowed tokens
    for r in range(rows):
        x[r, rng.integers(0, n, 3)] = rng.standard_normal(3)
    _check(q4, x, tok, 20)
    x[0] = -np.inf                                                                 # none allowed
    _check(q4, x, tok, 20)
    y = (3 * rng.standard_normal((rows, n))).astype(np.float32)
    y[rng.random((rows, n)) < 0.9] = -np.inf
    y[:, 7] = 0.0
    _check(q4, y, tok, 32)


def test_large_and_small_logits(q4):
    rng = np.random.default_rng(3)
    for scale, shift in ((1e-6, 0.0), (30.0, 1000.0), (1.0, -1e6), (1e4, 0.0)):
        x = (scale * rng.standard_normal((4, 4096)) + shift).astype(np.float32)
        _check(q4, x, rng.integers(0, 4096, 4), 10)
    x = np.full((2, 9000), -np.finfo(np.float32).max, np.float32)  # the type's lowest value as a mask
    x[:, 4000] = 2.0
    _check(q4, x, np.array([4000, 0]), 5)


def test_nan_and_infinity_make_their_row_nan(q4):
    rng = np.random.default_rng(4)
    x = rng.standard_normal((4, 3000)).astype(np.float32)
    x[1, 77] = np.nan
    x[2, 5] = np.inf
    x[3] = np.nan
    lp, ent, tv, ti = q4.q4_logprobs(torch.from_numpy(x).cuda(), torch.zeros(4, dtype=torch.int32, device="cuda"), top=4)
    assert torch.isfinite(lp[0]) and torch.isnan(lp[1:]).all()
    assert torch.isfinite(ent[0]) and torch.isnan(ent[1:]).all()
    assert torch.isnan(tv[1:]).all()
    x1 = np.where(np.isnan(x[1]), -np.inf, x[1])
    assert np.array_equal(ti[1].cpu().numpy(), np.argsort(-x1, kind="stable")[:4])  # NaN ranks lowest
    assert int(ti[2, 0]) == 5 and ti[3].tolist() == [0, 1, 2, 3]
    q4.q4_device_check()


def test_token_out_of_range_is_recorded(q4):
    x = torch.zeros((2, 100), device="cuda")
    lp, _, _, _ = q4.q4_logprobs(x, torch.tensor([100, 5], dtype=torch.int32, device="cuda"))
    assert torch.isnan(lp[0]) and abs(float(lp[1]) + np.log(100)) < 1e-5
    with pytest.raises(q4.Q4Error):
        q4.q4_device_check()
    q4.q4_device_check()


def test_optional_outputs_and_refusals(q4):
    x = torch.randn((3, 50), device="cuda")
    lp, ent, tv, ti = q4.q4_logprobs(x[:, :20].contiguous(), entropy=False, top=32)
    assert lp is None and ent is None and tv.shape == (3, 20)
    assert q4.q4_logprobs(torch.empty((0, 5), device="cuda"))[1].shape == (0,)
    with pytest.raises(q4.Q4Error) as e:
        q4.q4_logprobs(x, top=33)
    assert e.value.status == 2
    with pytest.raises(ValueError):
        q4.q4_logprobs(x, torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        q4.q4_logprobs(x.half())


def test_captured(q4):
    x = torch.randn((2, 70000), device="cuda")
    tok = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    q4.q4_logprobs(x, tok, top=5)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = q4.q4_logprobs(x, tok, top=5)
    x.copy_(torch.randn((2, 70000), device="cuda") * 2)
    tok.copy_(torch.tensor([7, 69999], dtype=torch.int32))
    g.replay()
    for a, b in zip(got, q4.q4_logprobs(x, tok, top=5)):
        assert torch.equal(a, b)
