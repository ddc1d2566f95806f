"""The host side of the microscaled 4-bit calls and of the mixture-of-experts layer: sizes, and arguments that are
refused before anything is launched (no GPU needed)."""
import ctypes

import pytest

import bit_weight_quantized_q4_gb300 as q4

OK, NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE, CUDA = range(7)
A = 1 << 20  # an address that is aligned and never followed


@pytest.fixture(scope="module")
def L():
    q4.build()
    return q4.lib()


def mx(rows=128, k=256, fmt=0, batch=1, dev=A, scale=1.0, short=0):
    one = int(q4.lib().q4_mx_bytes(fmt, rows, k)) if fmt in (0, 1) else 0
    return q4._CMx(fmt, rows, k, batch, dev, one * batch - short, scale)


def src(x=A, up=None, gamma=None, ld=256, dtype=0, rows=128, k=256, eps=1e-6):
    return q4._CMxSrc(x, up, gamma, ld, dtype, rows, k, eps)


def test_sizes(L):
    # records of 128 rows x 256 columns: 16384 bytes of codes and 1024 (MXFP4) or 2048 of scales
    assert L.q4_mx_bytes(0, 1, 32) == 17408 and L.q4_mx_bytes(1, 1, 32) == 18432
    assert L.q4_mx_bytes(0, 129, 288) == 4 * 17408 and L.q4_mx_bytes(1, 256, 512) == 4 * 18432
    assert L.q4_mx_bytes(0, 1 << 24, 65536) == (1 << 17) * 256 * 17408
    for bad in ((2, 1, 32), (-1, 1, 32), (0, 0, 32), (0, 1, 31), (0, 1, 0), (0, 1, 48), (0, (1 << 24) + 1, 32), (0, 1, 65568)):
        assert L.q4_mx_bytes(*bad) == 0
    for fmt, rows, k in ((0, 1, 32), (1, 129, 288), (0, 14336, 4096)):
        assert q4._mx_bytes(fmt, rows, k) == L.q4_mx_bytes(fmt, rows, k)
    with pytest.raises(ValueError):
        q4._mx_bytes(0, 1, 33)


@pytest.mark.parametrize("s,m,status", [
    (None, mx, NULL), (src, None, NULL),
    (lambda: src(x=None), mx, NULL), (src, lambda: mx(dev=None), NULL),
    (lambda: src(x=A + 8), mx, ALIGN), (lambda: src(gamma=A + 4), mx, ALIGN), (lambda: src(up=A + 8), mx, ALIGN),
    (src, lambda: mx(dev=A + 8), ALIGN), (lambda: src(ld=257), mx, ALIGN), (lambda: src(dtype=1, ld=260), mx, ALIGN),
    (lambda: src(ld=255), mx, SHAPE), (lambda: src(k=255, ld=256), mx, SHAPE), (lambda: src(rows=0), mx, SHAPE),
    (lambda: src(rows=64), mx, SHAPE), (lambda: src(k=512, ld=512), mx, SHAPE), (src, lambda: mx(short=1), SHAPE),
    (src, lambda: mx(batch=2), SHAPE), (src, lambda: mx(batch=0), SHAPE),
    (lambda: src(dtype=3), mx, UNSUPPORTED), (lambda: src(up=A, gamma=A), mx, UNSUPPORTED),
    (src, lambda: mx(fmt=2), UNSUPPORTED),
    (src, lambda: mx(scale=2.0), SHAPE), (src, lambda: mx(scale=float("nan")), SHAPE),
    (src, lambda: mx(fmt=1, scale=0.0), SHAPE), (src, lambda: mx(fmt=1, scale=float("inf")), SHAPE),
    (src, lambda: mx(fmt=1, scale=-1.0), SHAPE), (src, lambda: mx(fmt=1, scale=2.0 ** 61), SHAPE),
])
def test_quant_refuses(L, s, m, status):
    sp = None if s is None else ctypes.byref(s())
    mp = None if m is None else ctypes.byref(m())
    assert L.q4_mx_quant(sp, mp, None) == status


def test_copies_refuse(L):
    m = mx()
    r = ctypes.byref
    assert L.q4_mx_dequant(None, 0, A, None) == NULL and L.q4_mx_dequant(r(m), 0, None, None) == NULL
    assert L.q4_mx_dequant(r(m), 3, A, None) == UNSUPPORTED and L.q4_mx_dequant(r(m), 0, A + 4, None) == ALIGN
    for f in (lambda c, s: L.q4_mx_pack(c, s, r(m), None), lambda c, s: L.q4_mx_unpack(r(m), c, s, None)):
        assert f(None, A) == NULL and f(A, None) == NULL and f(A + 1, A) == ALIGN and f(A, A + 2) == ALIGN
    assert L.q4_mx_pack(A, A, r(mx(fmt=5)), None) == UNSUPPORTED


@pytest.mark.parametrize("w,x,r,dtype,y,status", [
    (None, mx, None, 0, A, NULL), (mx, None, None, 0, A, NULL), (mx, mx, None, 0, None, NULL),
    (mx, mx, None, 3, A, UNSUPPORTED), (mx, lambda: mx(fmt=1), None, 0, A, UNSUPPORTED),
    (lambda: mx(batch=2), mx, None, 0, A, UNSUPPORTED), (mx, lambda: mx(batch=2), None, 0, A, UNSUPPORTED),
    (mx, lambda: mx(k=512), None, 0, A, SHAPE), (mx, lambda: mx(rows=(1 << 20) + 1), None, 0, A, SHAPE),
    (mx, mx, None, 0, A + 8, ALIGN), (mx, mx, A + 2, 1, A, ALIGN),
])
def test_gemm_refuses(L, w, x, r, dtype, y, status):
    wp = None if w is None else ctypes.byref(w())
    xp = None if x is None else ctypes.byref(x())
    assert L.q4_mx_gemm(wp, xp, r, dtype, y, None) == status
    s = src(rows=x().rows if x else 128, k=x().k if x else 256, ld=x().k if x else 256)
    assert L.q4_mx_linear(wp, ctypes.byref(s), xp, r, dtype, y, None) == status


def test_linear_refuses_what_quant_does(L):
    w, x = mx(), mx(rows=5)
    f = lambda s: L.q4_mx_linear(ctypes.byref(w), ctypes.byref(s), ctypes.byref(x), None, 0, A, None)  # noqa: E731
    assert f(src(rows=4)) == SHAPE and f(src(rows=5, ld=128)) == SHAPE and f(src(rows=5, x=None)) == NULL
    assert f(src(rows=5, up=A, gamma=A)) == UNSUPPORTED
    assert L.q4_mx_linear(ctypes.byref(w), None, ctypes.byref(x), None, 0, A, None) == NULL


def layer(E=4, hidden=128, inter=64, top_k=2, router=A, gate_up=None, down=None):
    return q4._CMoELayer(gate_up or mx(2 * inter, hidden, batch=E), down or mx(hidden, inter, batch=E), router, E, hidden,
                         inter, top_k, 1)


def test_moe_refuses(L):
    r = ctypes.byref

    def call(lay=None, s=None, positions=None, res=None, dtype=0, y=A, idx=A, weight=A, ws=A, n=1 << 40):
        lay = layer() if lay is None else lay
        s = src(rows=2, k=128, ld=128) if s is None else s
        return L.q4_moe(r(lay), r(s), positions, res, dtype, y, idx, weight, ws, n, None)

    assert L.q4_moe(None, r(src(rows=2, k=128, ld=128)), None, None, 0, A, A, A, A, 1 << 40, None) == NULL
    assert call(layer(router=None)) == NULL and call(layer(router=A + 4)) == ALIGN
    assert call(layer(top_k=0)) == SHAPE and call(layer(top_k=5)) == SHAPE and call(layer(E=32, top_k=17)) == SHAPE
    assert call(layer(E=1025)) == SHAPE and call(layer(hidden=144, gate_up=mx(128, 160, batch=4), down=mx(160, 64, batch=4))) == SHAPE
    assert call(layer(gate_up=mx(128, 128, fmt=1, batch=4))) == UNSUPPORTED
    assert call(layer(gate_up=mx(64, 128, batch=4))) == SHAPE and call(layer(down=mx(128, 128, batch=4))) == SHAPE
    assert call(layer(down=mx(128, 64, batch=3))) == SHAPE
    assert call(s=src(rows=17, k=128, ld=128)) == UNSUPPORTED and call(s=src(rows=2, k=128, ld=128, up=A)) == UNSUPPORTED
    assert call(s=src(rows=2, k=160, ld=160)) == SHAPE and call(dtype=7) == UNSUPPORTED
    assert call(y=None) == NULL and call(idx=None) == NULL and call(weight=None) == NULL
    assert call(res=A + 8) == ALIGN and call(positions=A + 2) == ALIGN and call(y=A + 4) == ALIGN
    need = L.q4_moe_workspace_bytes(r(layer()), 2)
    assert need > 0 and call(ws=None) == WORKSPACE and call(n=need - 1) == WORKSPACE and call(ws=A + 8) == ALIGN
    assert L.q4_moe_workspace_bytes(r(layer()), 0) == 0 and L.q4_moe_workspace_bytes(r(layer()), 17) == 0
    assert L.q4_moe_workspace_bytes(None, 1) == 0
    # more tokens and experts need no less
    sizes = [L.q4_moe_workspace_bytes(r(layer(E=e, top_k=k)), n) for e, k, n in ((4, 2, 1), (4, 2, 16), (64, 8, 16))]
    assert sizes == sorted(sizes)


def test_moe_pack_refuses(L):
    r = ctypes.byref
    g, u, o = mx(64, 128, batch=2), mx(64, 128, batch=2), mx(128, 128, batch=2)
    f = lambda *m: L.q4_moe_pack(*(None if x is None else r(x) for x in m), None)  # noqa: E731
    assert f(None, u, o) == NULL and f(g, None, o) == NULL and f(g, u, None) == NULL
    assert f(mx(64, 128, fmt=1, batch=2), u, o) == UNSUPPORTED
    assert f(mx(48, 128, batch=2), mx(48, 128, batch=2), mx(96, 128, batch=2)) == SHAPE
    assert f(g, mx(64, 160, batch=2), o) == SHAPE and f(g, u, mx(64, 128, batch=2)) == SHAPE and f(g, u, mx(128, 128)) == SHAPE


def test_python_refuses_host_tensors(L):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64)
    with pytest.raises(TypeError):
        q4.q4_mx_quant(x)
    with pytest.raises(TypeError):
        q4.MXMatrix.from_codes(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8), 0)
    with pytest.raises(TypeError):
        q4.q4_mx_dequant(x)
    with pytest.raises(TypeError):
        q4.q4_mx_gemm(x, x)
    with pytest.raises(TypeError):
        q4.q4_moe(x, None)
