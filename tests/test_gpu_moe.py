"""The mixture-of-experts layer on the GPU against its formula in 64 bits.

The inner roundings to 4 bits make a layer's result jump where a value lies next to a border.  So the inputs are such
that what is rounded first is exact: rows of +-1 (their root mean square is 1) with gammas of the grid times powers of
two, whole-number router weights (exact logits) and products of grid values (exact gates and ups).  What remains are the
h whose fp32 value may fall on the other side of a border: the bound has their step times the weight it meets."""
import pytest

import mx_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}


@pytest.fixture(scope="module")
def q4():
    import bit_weight_quantized_q4_gb300 as m
    m.build()
    m.lib()
    return m


def draw(q4, seed, rows, E, top_k, hidden, inter, renormalize=True, dtype=BF16, norm=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    raw = [mx_ref.random_codes(g, (E, n), k, 0, -5, -4) for n, k in ((inter, hidden), (inter, hidden), (hidden, inter))]
    router = torch.randint(-4, 5, (E, hidden), generator=g, device="cuda").float() / 64
    layer = q4.MoELayer(router, *(q4.MXMatrix.from_codes(c, s, 0) for c, s in raw), top_k=top_k, renormalize=renormalize)
    sign = torch.randint(0, 2, (rows, hidden), generator=g, device="cuda").float() * 2 - 1
    # gammas on the grid of blocks whose largest value is 6 (so that the block's scale is a power of two times 1)
    gamma = torch.tensor([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 6.0], device="cuda").repeat(hidden // 8) / 8
    x = sign if norm else sign * gamma
    return {"layer": layer, "raw": raw, "router": router, "x": x.to(dtype), "gamma": gamma if norm else None, "g": g,
            "xh": (sign * gamma).double(), "top_k": top_k, "renormalize": renormalize}


def reference(s, idle=()):
    """(out, bound without the output's rounding, experts, weights) in 64 bits."""
    x, k = s["xh"], s["top_k"]
    assert torch.equal(mx_ref.quantise(x, 0), x)
    logits = x @ s["router"].double().T
    idx = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :k]
    w = torch.softmax(logits.gather(1, idx), -1) if s["renormalize"] else torch.softmax(logits, -1).gather(1, idx)
    out, bound = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(x.shape[0]):
        if t in idle:
            idx[t], w[t] = -1, 0
            continue
        for j in range(k):
            e = int(idx[t, j])
            G, U, D = (mx_ref.stored(c[e], sc[e], 0) for c, sc in s["raw"])
            a, u = G @ x[t], U @ x[t]
            h = a * torch.sigmoid(a) * u
            # fp32: the fast exponential (2 + 1.173 |a| units in the last place), the quotient (2), two products
            delta = (2 + 1.173 * a.abs() + 4) * 2.0 ** -23
            hb, db = h.unflatten(-1, (-1, 32)), delta.unflatten(-1, (-1, 32))
            lo, hi = (mx_ref.mx_scale((hb.abs() * f).amax(-1, keepdim=True)) for f in (1 - db, 1 + db))
            sc = mx_ref.mx_scale(hb.abs().amax(-1, keepdim=True))
            q, half = mx_ref.e2m1(hb / sc)
            below, above = (mx_ref.e2m1(hb * f / sc)[0] for f in (1 - db, 1 + db))
            # values that may take another code, or all of a block whose scale may be another one
            off = torch.where(lo == hi, (above - below).abs() * sc, 2 * half * hi).flatten()
            q = (q * sc).flatten()
            out[t] += w[t, j] * (D @ q)
            # the sum over k (64 a step), the weight (exp, a sum and a quotient: a few 2^-22), the sum over experts
            S = D.abs() @ q.abs()
            bound[t] += w[t, j] * (D.abs() @ off + (D.shape[1] / 64 + 64 + 32) * 2.0 ** -23 * S)
    return out, bound, idx, w


def check(got, want, r, dtype):
    (out, idx, w), (ref, bound, ridx, rw) = got, want
    assert torch.equal(idx.long(), ridx)
    assert bool(((w.double() - rw).abs() <= 2.0 ** -19 * rw).all())  # exp of differences up to 16: 16 2^-24, and a few roundings
    ref = ref if r is None else ref + r.double()
    err = (out.double() - ref).abs()
    # the output's rounding: half a step, which below the smallest normal number stays the step there (f16: 2^-25)
    most = bound + 2 * EPS[dtype] * ref.abs().clamp_min(torch.finfo(dtype).tiny)
    assert bool((err <= most).all()), float((err / most).max())


@pytest.mark.parametrize("rows,E,top_k,hidden,inter", [
    (1, 1, 1, 32, 32), (1, 4, 1, 128, 64), (2, 3, 3, 96, 96), (16, 4, 2, 256, 320), (5, 7, 4, 544, 160), (3, 40, 16, 160, 64),
    (16, 16, 16, 128, 128), (7, 300, 3, 64, 32), (4, 1024, 2, 32, 32), (1, 128, 8, 2048, 768), (16, 128, 8, 512, 256),
    (9, 8, 2, 1024, 2080), (1, 2, 1, 4096, 32), (2, 2, 2, 32, 4096)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_layer(q4, rows, E, top_k, hidden, inter, renormalize):
    for dtype, norm in ((F32, True), (BF16, True), (F16, False)):
        s = draw(q4, rows * 31 + E, rows, E, top_k, hidden, inter, renormalize, dtype, norm)
        want = reference(s)
        got = q4.q4_moe(s["x"], s["layer"], gamma=s["gamma"])
        assert got[0].dtype == dtype and got[1].dtype == torch.int32 and got[2].dtype == F32
        check(got, want, None, dtype)
        r = torch.randn(rows, hidden, generator=s["g"], device="cuda").to(dtype)
        check(q4.q4_moe(s["x"], s["layer"], gamma=s["gamma"], r=r), want, r, dtype)
    q4.q4_device_check()


@pytest.mark.parametrize("rows,E,top_k,hidden,inter", [(2, 2, 1, 65536, 64), (1, 3, 2, 32, 65536), (16, 16, 16, 32, 32), (16, 1024, 16, 64, 32)])
def test_layer_at_its_limits(q4, rows, E, top_k, hidden, inter):
    s = draw(q4, rows + E, rows, E, top_k, hidden, inter)
    r = torch.randn(rows, hidden, generator=s["g"], device="cuda").to(BF16)
    check(q4.q4_moe(s["x"], s["layer"], gamma=s["gamma"], r=r), reference(s), r, BF16)
    q4.q4_device_check()


def test_other_output_types_and_places(q4):
    s = draw(q4, 1, 5, 8, 2, 256, 96)
    want = reference(s)
    r = torch.randn(5, 256, device="cuda")
    a = q4.q4_moe(s["x"], s["layer"], gamma=s["gamma"], r=r, dtype=F32)
    check(a, want, r, F32)
    out = r.clone()  # onto the residual, in a workspace of any contents
    ws = q4.q4_moe_workspace(s["layer"], 5)
    ws.fill_(255)
    b = q4.q4_moe(s["x"], s["layer"], gamma=s["gamma"], r=out, out=out, workspace=ws)
    assert b[0] is out and torch.equal(out, a[0])
    x = s["x"].clone()  # onto x
    c = q4.q4_moe(x, s["layer"], gamma=s["gamma"], out=x)
    assert c[0] is x and torch.equal(x, q4.q4_moe(s["x"], s["layer"], gamma=s["gamma"])[0])
    # rows of a wider buffer; a workspace that another layer used; the same bits every time
    wide = torch.zeros(5, 512, dtype=BF16, device="cuda")
    wide[:, 128:384] = s["x"]
    big = draw(q4, 2, 16, 32, 4, 512, 128)
    ws = q4.q4_moe_workspace(big["layer"], 16)
    for _ in range(3):
        q4.q4_moe(big["x"], big["layer"], gamma=big["gamma"], workspace=ws)
        d = q4.q4_moe(wide[:, 128:384], s["layer"], gamma=s["gamma"], r=r, dtype=F32, workspace=ws)
        assert torch.equal(d[0], a[0])


@pytest.mark.parametrize("idle", [(0,), (1, 3), (0, 1, 2, 3, 4)])
def test_idle_rows_take_no_experts(q4, idle):
    s = draw(q4, 3, 5, 8, 2, 128, 64)
    pos = torch.tensor([-1 if t in idle else 10 + t for t in range(5)], dtype=torch.int32, device="cuda")
    x = s["x"].clone()
    x[list(idle)] = float("nan")  # whatever they hold
    r = torch.randn(5, 128, generator=s["g"], device="cuda").to(BF16)
    check(q4.q4_moe(x, s["layer"], gamma=s["gamma"], positions=pos, r=r), reference(s, idle), r, BF16)
    out = q4.q4_moe(x, s["layer"], gamma=s["gamma"], positions=pos)[0]
    assert bool((out[list(idle)] == 0).all())
    q4.q4_device_check()


def test_ties_and_logits_that_are_no_numbers(q4):
    s = draw(q4, 4, 3, 40, 4, 64, 32, norm=False)
    # all logits equal: the lowest indices, even weights
    zero = q4.MoELayer(torch.zeros(40, 64, device="cuda"), *(q4.MXMatrix.from_codes(c, sc, 0) for c, sc in s["raw"]), top_k=4)
    out, idx, w = q4.q4_moe(s["x"], zero)
    assert idx.tolist() == [[0, 1, 2, 3]] * 3 and bool((w == 0.25).all())
    # NaN logits rank behind every number, and -inf is one
    router = torch.zeros(40, 64, device="cuda")
    router[:36] = float("nan")
    router[36, 0], router[37, 0] = float("inf"), float("-inf")
    odd = q4.MoELayer(router, *(q4.MXMatrix.from_codes(c, sc, 0) for c, sc in s["raw"]), top_k=6)
    x = torch.zeros(1, 64, device="cuda")
    x[0, 0] = -1.0
    out, idx, w = q4.q4_moe(x, odd)
    assert idx.tolist() == [[37, 38, 39, 36, 0, 1]] and bool(torch.isnan(w).all()) and bool(torch.isnan(out).all())
    # one token's NaN is its own
    x = s["x"].clone()
    x[1, 5] = float("nan")
    good, bad = q4.q4_moe(s["x"], s["layer"]), q4.q4_moe(x, s["layer"])
    assert bool(torch.isnan(bad[0][1]).all()) and bool(torch.isnan(bad[2][1]).all())
    for t in (0, 2):
        assert torch.equal(bad[1][t], good[1][t]) and bool(torch.isfinite(bad[0][t]).all())
    q4.q4_device_check()


def test_captured_and_on_two_streams(q4):
    sets = [draw(q4, 10 + i, rows, 16, 3, 256, 128) for i, rows in enumerate((2, 11))]
    run = lambda s, **kw: q4.q4_moe(s["x"], s["layer"], gamma=s["gamma"], r=s["x"], **kw)  # noqa: E731
    want = [tuple(t.clone() for t in run(s)) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        got = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(run(s))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    graphs = []
    for s in sets:
        st = {**s, "x": s["x"].clone()}
        ws, out = q4.q4_moe_workspace(s["layer"], s["x"].shape[0]), torch.empty_like(s["x"])
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            res = run(st, workspace=ws, out=out)
        graphs.append((gr, st["x"], res))
    flip = [s["x"].flip(0) for s in sets]
    for turn in range(4):
        for (gr, x, _), s, f in zip(graphs, sets, flip):
            x.copy_(f if turn % 2 else s["x"])
        torch.cuda.synchronize()
        for (gr, _, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for (_, _, res), b in zip(graphs, want):
            # (the experts with a token are the same ones: so are the sums, row by row)
            assert all(torch.equal(p.flip(0) if turn % 2 else p, q) for p, q in zip(res, b))
    q4.q4_device_check()


def test_refusals(q4):
    s = draw(q4, 20, 4, 8, 2, 128, 64)
    L, x, r = s["layer"], s["x"], s["x"].clone()
    mats = [q4.MXMatrix.from_codes(c, sc, 0) for c, sc in s["raw"]]
    ok = q4.q4_moe(x, L)[0]
    for bad in (lambda: q4.q4_moe(x, None), lambda: q4.q4_moe(x[0], L), lambda: q4.q4_moe(x[:, :64], L), lambda: q4.q4_moe(x[:0], L),
                lambda: q4.q4_moe(x.repeat(5, 1), L), lambda: q4.q4_moe(x[None], L), lambda: q4.q4_moe(x.double(), L),
                lambda: q4.q4_moe(x, L, gamma=torch.ones(64, device="cuda")), lambda: q4.q4_moe(x, L, dtype=torch.int32),
                lambda: q4.q4_moe(x, L, r=r.float()), lambda: q4.q4_moe(x, L, r=r[:2]), lambda: q4.q4_moe(x, L, out=r[:2]),
                lambda: q4.q4_moe(x, L, positions=torch.zeros(3, dtype=torch.int32, device="cuda")),
                lambda: q4.q4_moe(x, L, positions=torch.zeros(4, dtype=torch.int64, device="cuda")),
                lambda: q4.q4_moe(x, L, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")),
                lambda: q4.MoELayer(s["router"], *mats, top_k=0), lambda: q4.MoELayer(s["router"], *mats, top_k=9),
                lambda: q4.MoELayer(s["router"][:, :64], *mats, top_k=2), lambda: q4.MoELayer(s["router"].half(), *mats, top_k=2),
                lambda: q4.MoELayer(s["router"], mats[2], mats[1], mats[0], top_k=2),
                lambda: q4.MoELayer(s["router"], mats[0], mats[1], q4.q4_mx_quant(torch.randn(8, 128, 64, device="cuda"), 1), top_k=2)):
        with pytest.raises((TypeError, ValueError, q4.Q4Error)):
            bad()
    buf = torch.zeros(6, 128, dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        q4.q4_moe(x, L, r=buf[:4], out=buf[1:5])
    with pytest.raises(ValueError):
        q4.q4_moe(buf[:4], L, out=buf[1:5])
    assert torch.equal(q4.q4_moe(x, L)[0], ok)
    q4.q4_device_check()


def test_a_layer_behind_attention_scores_and_logits(q4):
    """A decode step's end as it is used: a residual stream through a 4-bit projection, the experts and a 4-bit head."""
    s = draw(q4, 30, 4, 8, 2, 256, 128)
    g = s["g"]
    Wo, head = (q4.q4_mx_quant(torch.randn(n, 256, generator=g, device="cuda") / 16) for n in (256, 500))
    a = torch.randn(4, 256, generator=g, device="cuda")
    hid = torch.randn(4, 256, generator=g, device="cuda")
    pos = torch.tensor([5, -1, 9, 0], dtype=torch.int32, device="cuda")

    def step(hid):
        q4.q4_mx_gemm(Wo, a, r=hid, out=hid)
        q4.q4_moe(hid, s["layer"], gamma=s["gamma"], eps=1e-6, r=hid, out=hid, positions=pos)
        logits = q4.q4_mx_gemm(head, hid, gamma=s["gamma"], eps=1e-6)
        return q4.q4_logprobs(logits, torch.tensor([1, -1, 3, 4], dtype=torch.int32, device="cuda"), top=2)

    h1, h2 = hid.clone(), hid.clone()
    one = step(h1)
    # the same through the parts
    q4.q4_mx_gemm(Wo, q4.q4_mx_quant(a), r=h2, out=h2, dtype=F32)
    before = h2.clone()
    out, idx, w = q4.q4_moe(h2, s["layer"], gamma=s["gamma"], eps=1e-6, r=h2, positions=pos)
    assert torch.equal(out[1], before[1]) and idx[1].tolist() == [-1, -1]
    logits = q4.q4_mx_gemm(head, q4.q4_mx_quant(out, gamma=s["gamma"], eps=1e-6), dtype=F32)
    assert torch.equal(h1, out)
    lp = torch.log_softmax(logits.double(), -1)
    assert bool(((one[0].double() - torch.stack([lp[0, 1], lp[0, 0] * 0, lp[2, 3], lp[3, 4]])).abs() <= 1e-5).all())
    q4.q4_device_check()


@pytest.mark.parametrize("kw", [{"copy_wait_cycles": 200000, "copy_extra_bytes": 16}, {"barrier_polls": 256, "barrier_extra": 1, "copy_wait_cycles": 2000000}])
def test_a_wait_that_gives_up_is_reported_and_the_next_call_is_unchanged(q4, kw):
    s = draw(q4, 40, 3, 8, 2, 512, 256)
    y0 = q4.q4_moe(s["x"], s["layer"], gamma=s["gamma"])[0]
    q4.q4_device_check()
    q4.q4_debug_wait_limits(**kw)
    try:
        q4.q4_moe(s["x"], s["layer"], gamma=s["gamma"])
        with pytest.raises(q4.Q4Error) as e:
            q4.q4_device_check()
        assert e.value.status == 6
    finally:
        q4.q4_debug_wait_limits()
    assert torch.equal(q4.q4_moe(s["x"], s["layer"], gamma=s["gamma"])[0], y0)
    q4.q4_device_check()


def test_weights_beyond_32_bits(q4):
    # 72 experts of 4096 x 14336: 4.5 GB of gate and up; tokens that choose the last eight, against a layer of those alone
    E, hidden, inter = 72, 4096, 14336
    g = torch.Generator(device="cuda").manual_seed(7)
    mats = []
    for n, k in ((inter, hidden), (inter, hidden), (hidden, inter)):
        m = q4.MXMatrix(0, n, k, batch=E)
        m.tensor.random_(100, 118, generator=g)
        mats.append(m)
    assert 2 * mats[0].nbytes > 1 << 32
    router = torch.zeros(E, hidden, device="cuda")
    router[64:] = torch.randint(1, 5, (8, hidden), generator=g, device="cuda").float() / 64
    x = torch.randint(1, 4, (3, hidden), generator=g, device="cuda").to(BF16)
    few = [q4.MXMatrix(0, m.rows, m.k, batch=8, tensor=m.tensor[m.nbytes // E * 64:]) for m in mats]
    out, idx, w = q4.q4_moe(x, q4.MoELayer(router, *mats, top_k=2))
    want, widx, ww = q4.q4_moe(x, q4.MoELayer(router[64:].contiguous(), *few, top_k=2))
    assert torch.equal(idx, widx + 64) and torch.equal(w, ww) and torch.equal(out, want) and bool(out.abs().max() > 0)
    q4.q4_device_check()
