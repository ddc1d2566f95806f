"""Host-side tests of the paged cache and sampling calls (no GPU): workspace
sizes, and invalid arguments refused before anything is launched."""
import ctypes

import pytest

import bit_weight_quantized_q4_gb300 as q4


@pytest.fixture(scope="module", autouse=True)
def built():
    q4.build()


def pages(k=0x1000, v=0x2000, table=0x3000, dtype=1, num_pages=10, page=16, hkv=2, D=64, nseq=3, width=4):
    return q4._CKvPages(k, v, table, dtype, num_pages, page, hkv, D, nseq, width)


BAD_PAGES = [(dict(k=None), 1), (dict(v=0), 1), (dict(table=None), 1), (dict(k=0x1008), 3), (dict(table=0x3002), 3),
             (dict(dtype=3), 4), (dict(dtype=-1), 4), (dict(D=96), 4), (dict(num_pages=0), 2), (dict(page=0), 2),
             (dict(page=24), 2), (dict(page=(1 << 24) + 16), 2), (dict(hkv=0), 2), (dict(nseq=0), 2),
             (dict(nseq=1025), 2), (dict(width=0), 2), (dict(page=1 << 24, width=65), 2),
             (dict(nseq=1024, page=1 << 24, width=8), 2)]


def _calls(c):
    """Each call over the pages `c` with otherwise valid arguments."""
    L = q4.lib()
    r = None if c is None else ctypes.byref(c)
    A = 0x4000
    return {
        "append": lambda **o: L.q4_kv_append(r, o.get("q", A), o.get("k", A), o.get("v", A), o.get("rows", 5),
                                             o.get("cu", A), o.get("start", A), o.get("H", 4), o.get("cos", A),
                                             o.get("sin", A), o.get("rope_rows", 64), o.get("out", A), None),
        "prefill": lambda **o: L.q4_attn_prefill(r, o.get("q", A), o.get("rows", 5), o.get("cu", A),
                                                 o.get("start", A), o.get("H", 4), o.get("window", 0),
                                                 o.get("scale", 0.125), o.get("out", A), o.get("ws", A), o.get("wsb", 1 << 40), None),
        "paged": lambda **o: L.q4_attn_paged(r, o.get("q", A), o.get("k", A), o.get("v", A), o.get("positions", A),
                                             o.get("H", 4), o.get("window", 0), o.get("scale", 0.125), o.get("cos", A),
                                             o.get("sin", A), o.get("rope_rows", 64), o.get("out", A),
                                             o.get("ws", A), o.get("wsb", 1 << 40), None),
    }


@pytest.mark.parametrize("call", ["append", "prefill", "paged"])
@pytest.mark.parametrize("case,expect", BAD_PAGES)
def test_bad_pages(call, case, expect):
    assert _calls(pages(**case))[call]() == expect


@pytest.mark.parametrize("call", ["append", "prefill", "paged"])
def test_no_pages(call):
    assert _calls(None)[call]() == 1


@pytest.mark.parametrize("call,case,expect", [
    ("append", dict(rows=-1), 2), ("append", dict(rows=(1 << 24) + 1), 2), ("append", dict(k=None), 1),
    ("append", dict(v=0x4008), 3), ("append", dict(q=0x4004), 3), ("append", dict(out=None), 1),
    ("append", dict(cu=None), 1), ("append", dict(cu=0x4001), 3), ("append", dict(start=0x4002), 3),
    ("append", dict(H=5), 2), ("append", dict(H=0), 2), ("append", dict(H=34), 4), ("append", dict(sin=None), 1),
    ("append", dict(cos=0x4004), 3), ("append", dict(rope_rows=0), 2),
    ("prefill", dict(rows=-1), 2), ("prefill", dict(q=None), 1), ("prefill", dict(out=0x4004), 3),
    ("prefill", dict(cu=None), 1), ("prefill", dict(start=0x4002), 3), ("prefill", dict(H=3), 2),
    ("prefill", dict(H=34), 4), ("prefill", dict(window=-1), 2), ("prefill", dict(scale=-0.1), 2),
    ("prefill", dict(scale=float("nan")), 2), ("paged", dict(scale=float("inf")), 2), ("paged", dict(scale=-1.0), 2),
    ("paged", dict(q=None), 1), ("paged", dict(k=0x4004), 3), ("paged", dict(v=None), 1),
    ("paged", dict(positions=None), 1), ("paged", dict(positions=0x4002), 3), ("paged", dict(H=1), 2),
    ("paged", dict(H=64), 4), ("paged", dict(window=-3), 2), ("paged", dict(out=None), 1),
    ("paged", dict(ws=None), 5), ("paged", dict(wsb=100), 5), ("paged", dict(ws=0x4008), 3),
    ("paged", dict(cos=None), 1), ("paged", dict(rope_rows=-2), 2)])
def test_bad_arguments(call, case, expect):
    assert _calls(pages())[call](**case) == expect


@pytest.mark.parametrize("call", ["append", "prefill"])
def test_no_rows_launch_nothing(call):
    assert _calls(pages())[call](rows=0) == 0
    assert _calls(pages())[call](rows=0, H=5) == 2  # the other arguments are still looked at


def test_workspace_bytes():
    L = q4.lib()
    c = pages()
    assert L.q4_attn_paged_workspace_bytes(ctypes.byref(c), 4) >= 3 * 2 * 4
    # sized by the heads, not by the cache's length
    big = pages(width=1000)
    assert L.q4_attn_paged_workspace_bytes(ctypes.byref(big), 4) == L.q4_attn_paged_workspace_bytes(ctypes.byref(c), 4)
    # and its counters do not move with the geometry: calls of several shapes share one
    assert L.q4_attn_paged_workspace_bytes(ctypes.byref(pages(nseq=9, hkv=1)), 2) == L.q4_attn_paged_workspace_bytes(ctypes.byref(c), 4)
    assert L.q4_attn_paged_workspace_bytes(ctypes.byref(pages(nseq=1024, hkv=128)), 128) == 0  # too many pairs
    assert _calls(pages(nseq=1024, hkv=128))["paged"](H=128) == 2
    # the fp32 prompt attention: the parts of the cache and of q
    f = pages(dtype=0, num_pages=10, page=16, hkv=2, D=64)
    kv = 10 * 16 * 2 * 64
    assert L.q4_attn_prefill_workspace_bytes(ctypes.byref(f), 5, 4) >= 2 * 2 * 2 * kv + 5 * 4 * (4 + 2 * 2 * 64)
    assert L.q4_attn_prefill_workspace_bytes(ctypes.byref(f), 0, 4) == 0
    assert L.q4_attn_prefill_workspace_bytes(ctypes.byref(c), 5, 4) == 0
    assert _calls(f)["prefill"](ws=None) == 5 and _calls(f)["prefill"](wsb=100) == 5 and _calls(f)["prefill"](ws=0x4008) == 3
    for bad in (pages(D=32), pages(nseq=0)):
        assert L.q4_attn_paged_workspace_bytes(ctypes.byref(bad), 4) == 0
        assert L.q4_attn_prefill_workspace_bytes(ctypes.byref(bad), 10, 4) == 0
    assert L.q4_attn_paged_workspace_bytes(ctypes.byref(c), 5) == 0
    assert L.q4_attn_paged_workspace_bytes(None, 4) == 0


@pytest.mark.parametrize("case,expect", [
    (dict(rows=-1), 2), (dict(n=0), 2), (dict(n=(1 << 24) + 1), 2), (dict(top=-1), 2), (dict(top=33), 2),
    (dict(n=10, top=11), 2), (dict(logits=None), 1), (dict(logits=0x4004), 3), (dict(tokens=0x4002), 3),
    (dict(logprob=None), 1), (dict(tokens=None), 1), (dict(logprob=0x4004), 3), (dict(entropy=0x4008), 3),
    (dict(val=None), 1), (dict(idx=0x4004), 3)])
def test_logprobs_arguments(case, expect):
    o = dict(logits=0x4000, rows=2, n=100, tokens=0x4000, top=5, logprob=0x4000, entropy=0x4000, val=0x4000, idx=0x4000)
    o.update(case)
    assert q4.lib().q4_logprobs(o["logits"], o["rows"], o["n"], o["tokens"], o["top"], o["logprob"], o["entropy"],
                                o["val"], o["idx"], None) == expect


def test_logprobs_no_rows():
    assert q4.lib().q4_logprobs(None, 0, 100, None, 0, None, None, None, None, None) == 0


def test_pages_must_be_on_the_gpu():
    torch = pytest.importorskip("torch")
    z = torch.zeros((1, 1, 16, 64))
    with pytest.raises(TypeError):
        q4.KVPages(z, z, torch.zeros((1, 1), dtype=torch.int32))
    with pytest.raises(TypeError):
        q4.q4_attn_prefill(z, "pages", z)
