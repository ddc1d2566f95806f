"""Waits of the mixture-of-experts layer that give up at any point: every call ends, and the next one is unchanged."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def q4():
    import bit_weight_quantized_q4_gb300 as m
    m.build()
    m.lib()
    return m


@pytest.mark.parametrize("rows,E,top_k,hidden,inter", [(16, 64, 8, 2048, 768), (1, 2, 1, 65536, 32), (16, 64, 8, 65536, 96)])
def test_every_call_ends_however_short_its_waits_are(q4, rows, E, top_k, hidden, inter):
    # limits from less than a copy's time to more than a call's: the warps of a unit start their waits at different times, so
    # that near a unit's time one of them gives up and another's wait passes
    g = torch.Generator(device="cuda").manual_seed(rows)
    mats = []
    for n, k in ((inter, hidden), (inter, hidden), (hidden, inter)):
        m = q4.MXMatrix(q4.Q4_MX_MXFP4, n, k, batch=E)
        m.tensor.random_(100, 118, generator=g)
        mats.append(m)
    layer = q4.MoELayer(torch.randn(E, hidden, generator=g, device="cuda") / hidden ** 0.5, *mats, top_k=top_k)
    x = torch.randn(rows, hidden, generator=g, device="cuda").bfloat16()
    ws = q4.q4_moe_workspace(layer, rows)
    want = [t.clone() for t in q4.q4_moe(x, layer, r=x, workspace=ws)]
    assert bool(torch.isfinite(want[0]).all())
    q4.q4_device_check()
    gave_up = 0
    limits = [int(100 * 1.03 ** i) for i in range(300)]  # cycles: 100 .. 689000
    try:
        for limit in limits:
            q4.q4_debug_wait_limits(copy_wait_cycles=limit)
            got = q4.q4_moe(x, layer, r=x, workspace=ws)
            try:
                q4.q4_device_check()
            except q4.Q4Error as e:
                assert e.status == 6
                gave_up += 1
            else:
                assert all(torch.equal(a, b) for a, b in zip(got, want))
    finally:
        q4.q4_debug_wait_limits()
    assert 0 < gave_up < len(limits)
    assert all(torch.equal(a, b) for a, b in zip(q4.q4_moe(x, layer, r=x, workspace=ws), want))
    q4.q4_device_check()
