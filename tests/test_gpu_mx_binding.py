"""What the Python calls of the microscaled matrices and of the mixture-of-experts layer take and refuse."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def q4():
    import bit_weight_quantized_q4_gb300 as m
    m.build()
    m.lib()
    return m


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def test_a_given_matrix_keeps_its_format_and_factor(q4):
    x = randn(1, 5, 96)
    nv, mx = q4.MXMatrix(q4.Q4_MX_NVFP4, 5, 96, scale=0.5), q4.MXMatrix(q4.Q4_MX_MXFP4, 5, 96)
    # without a word on them they are the matrix's; the same words are fine
    want = q4.q4_mx_quant(x, q4.Q4_MX_NVFP4, scale=0.5).codes()
    for kw in ({}, {"fmt": q4.Q4_MX_NVFP4}, {"scale": 0.5}, {"fmt": q4.Q4_MX_NVFP4, "scale": 0.5}):
        assert q4.q4_mx_quant(x, out=nv, **kw) is nv
        assert all(torch.equal(a, b) for a, b in zip(nv.codes(), want))
    assert q4.q4_mx_quant(x, out=mx) is mx and torch.equal(mx.codes()[0], q4.q4_mx_quant(x).codes()[0])
    # other ones are refused, not passed over
    before = [t.clone() for t in nv.codes()]
    for m, kw in ((mx, {"fmt": q4.Q4_MX_NVFP4}), (mx, {"fmt": q4.Q4_MX_NVFP4, "scale": 0.5}), (nv, {"fmt": q4.Q4_MX_MXFP4}),
                  (nv, {"scale": 0.25}), (nv, {"fmt": q4.Q4_MX_NVFP4, "scale": 1.0}), (mx, {"scale": 2.0})):
        with pytest.raises(ValueError):
            q4.q4_mx_quant(2 * x, out=m, **kw)
    assert all(torch.equal(a, b) for a, b in zip(nv.codes(), before))
    q4.q4_device_check()


def test_a_quantised_matrix_lies_apart_from_its_rows(q4):
    # (17408 bytes a matrix of up to 128 rows x 256 columns)
    buf = torch.zeros(65536, dtype=torch.uint8, device="cuda")
    x = buf[16384:16384 + 4 * 256 * 4].view(torch.float32).view(4, 256)
    x.copy_(randn(2, 4, 256))
    up, gamma = randn(3, 4, 256), torch.ones(256, device="cuda")
    at = lambda first: q4.MXMatrix(0, 4, 256, tensor=buf[first:first + 17408])  # noqa: E731
    for first in (0, 1024, 16384, 20464):
        with pytest.raises(ValueError):
            q4.q4_mx_quant(x, out=at(first))
        with pytest.raises(ValueError):
            q4.q4_mx_quant(up, up=x, out=at(first))
        with pytest.raises(ValueError):
            # (the first row ends at 17408, the last one begins at 19456)
            q4.q4_mx_quant(up, gamma=x[3] if first >= 16384 else x[0], out=at(first))
    # next to them is fine
    want = q4.q4_mx_quant(x).codes()
    m = q4.q4_mx_quant(x, out=at(20480))
    assert all(torch.equal(a, b) for a, b in zip(m.codes(), want))
    m = q4.q4_mx_quant(x, gamma=gamma, eps=1e-6, out=q4.MXMatrix(0, 4, 256))
    with pytest.raises(ValueError):  # nor are values written over the matrix that they are read from
        q4.q4_mx_dequant(m, out=m.tensor[:4096].view(torch.float32).view(4, 256))
    q4.q4_device_check()


def test_a_batch_of_one_matrix_is_a_batch(q4):
    x = randn(4, 1, 40, 96)
    m = q4.q4_mx_quant(x)
    assert m.batch == 1 and q4.q4_mx_dequant(m).shape == x.shape
    c, s = m.codes()
    assert c.shape == (1, 40, 48) and s.shape == (1, 40, 3)
    again = q4.MXMatrix.from_codes(c, s, 0)
    assert all(torch.equal(a, b) for a, b in zip(again.codes(), (c, s)))
    assert torch.equal(q4.q4_mx_dequant(again, out=torch.empty_like(x)), q4.q4_mx_dequant(m))
    one = q4.q4_mx_quant(x[0])
    assert q4.q4_mx_dequant(one).shape == x[0].shape and one.codes()[0].shape == (40, 48)
    assert torch.equal(q4.q4_mx_dequant(one), q4.q4_mx_dequant(m)[0])
    # a matrix made for either takes both
    assert q4.q4_mx_quant(x, out=one) is one and q4.q4_mx_quant(x[0], out=m) is m
    two = q4.MXMatrix(0, 40, 96, batch=2)
    assert q4.q4_mx_dequant(q4.q4_mx_quant(x.expand(2, 40, 96).contiguous(), out=two)).shape == (2, 40, 96)
    assert q4.q4_mx_dequant(q4.MXMatrix(0, 40, 96)).shape == (40, 96)
    # a single matrix in a product, and a layer of one expert
    w = q4.q4_mx_quant(randn(5, 1, 64, 96))
    assert torch.equal(q4.q4_mx_gemm(w, x[0]), q4.q4_mx_gemm(q4.q4_mx_quant(q4.q4_mx_dequant(w)[0]), x[0]))
    up, down = (q4.q4_mx_quant(randn(i, 1, a, b)) for i, a, b in ((6, 64, 96), (7, 96, 64)))
    assert q4.q4_moe(x[0, :2], q4.MoELayer(torch.ones(1, 96, device="cuda"), w, up, down, top_k=1))[0].shape == (2, 96)
    q4.q4_device_check()


def test_factors_that_a_format_does_not_take_are_named(q4):
    x = randn(8, 4, 96)
    W = q4.q4_mx_quant(x)
    V = q4.q4_mx_quant(x, 1)
    c, s = W.codes()
    cn, sn = V.codes()
    for bad in (lambda: q4.MXMatrix(0, 4, 96, scale=2.0), lambda: q4.q4_mx_quant(x, scale=2.0), lambda: q4.MXMatrix.from_codes(c, s, 0, 0.5),
                lambda: q4.q4_mx_gemm(W, x, scale=2.0), lambda: q4.q4_mx_quant(x, 1, scale=0.0), lambda: q4.q4_mx_quant(x, 1, scale=-1.0),
                lambda: q4.q4_mx_quant(x, 1, scale=float("nan")), lambda: q4.q4_mx_gemm(V, x, scale=2.0 ** 61),
                lambda: q4.MXMatrix.from_codes(cn, sn, 1, float("inf"))):
        with pytest.raises(ValueError, match="scale"):
            bad()
    for ok in (2.0 ** -60, 1.0, 2.0 ** 60):
        q4.q4_mx_quant(x, 1, scale=ok)
        q4.q4_mx_gemm(V, x, scale=ok)
    q4.q4_device_check()


def test_workspaces_of_token_counts_that_a_layer_refuses(q4):
    mats = [q4.q4_mx_quant(randn(i, 4, a, b)) for i, (a, b) in enumerate(((64, 96), (64, 96), (96, 64)))]
    layer = q4.MoELayer(torch.ones(4, 96, device="cuda"), *mats, top_k=2)
    for rows in (0, -1, 17, 1000):
        with pytest.raises(ValueError):
            q4.q4_moe_workspace(layer, rows)
        with pytest.raises(ValueError):
            layer.workspace_bytes(rows)
    assert q4.q4_moe_workspace(layer, 16).numel() == layer.workspace_bytes(16) > layer.workspace_bytes(1) > 0
