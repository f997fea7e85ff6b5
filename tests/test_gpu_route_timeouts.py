"""The router of at most eight tokens, whose waits are bounded: a limit far below a copy's round trip
makes one run out, without a fault.  The rows are then marked, and the next call is right."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SHAPES = [  # T, H, E: the ring holds a token's chunks, or waits for free slots
    (1, 512, 64), (2, 1024, 128), (3, 8192, 256), (8, 16384, 256), (5, 16384, 100)]


@pytest.fixture(scope="module")
def moe(cuda_ok):
    import moe_expert_layer_fp32_gb300 as m
    return m


def inputs(T, H, E):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn((H, E), generator=g, device="cuda") * 0.05
    return x, w, torch.randn(E, generator=g, device="cuda") * 0.1


def limited(moe, limit, call):
    try:
        moe.moe_set_wait_limit(limit)
        r = call()
        torch.cuda.synchronize()
        return r
    finally:
        moe.moe_set_wait_limit(0)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("T,H,E", SHAPES)
def test_route_timeout_marks_every_row(moe, T, H, E, kind):
    """Index -1 and weight 0 for the call's rows, or the right rows where no wait ran out: never
    rows chosen from logits that were not computed."""
    k = 8
    x, wr, b = inputs(T, H, E)
    d, o = moe.dims(T, H, E, k, 128), moe.router_opts(kind)

    def run():
        idx = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
        w = torch.full((T, k), 77.0, device="cuda")
        moe.moe_route_ex(x, wr, b, o, d, idx, w)
        return idx, w

    want = run()
    marked = 0
    for limit in (16, 16, 16, 300, 1000, 2000, 3000, 5000):
        idx, w = limited(moe, limit, run)
        if (idx == -1).any():
            marked += 1
            assert (idx == -1).all() and (w == 0).all()
        else:
            assert torch.equal(idx, want[0]) and torch.equal(w, want[1])
        again = run()
        assert all(torch.equal(p, q) for p, q in zip(again, want))
    assert marked >= 3


@pytest.mark.parametrize("T,H,E", SHAPES)
def test_router_logits_timeout_is_nan(moe, T, H, E):
    """The projection alone: every logit of the call NaN, or right; nothing else is written."""
    x, wr, b = inputs(T, H, E)
    d = moe.dims(T, H, E, 8, 128)

    def run():
        both = torch.full((T + 1, E), 77.0, device="cuda")
        moe.moe_router_logits(x, wr, b, d, both[:T])
        return both

    want = run()
    assert torch.isfinite(want).all()
    marked = 0
    for limit in (16, 16, 16, 300, 1000, 2000, 3000, 5000):
        got = limited(moe, limit, run)
        assert (got[T] == 77.0).all()
        if torch.isnan(got).any():
            marked += 1
            assert torch.isnan(got[:T]).all()
        else:
            assert torch.equal(got, want)
        assert torch.equal(run(), want)
    assert marked >= 3


@pytest.mark.parametrize("T,E", [(1, 64), (8, 256)])
def test_mx4_layer_timeout_is_reported(moe, T, E):
    H, k, I = 512, 4, 128
    x, wr, b = inputs(T, H, E)
    d = moe.dims(T, H, E, k, I)
    g = torch.Generator(device="cuda").manual_seed(E)

    def normal(*shape):
        return (torch.randn(shape, generator=g, device="cuda") * 0.05).to(torch.bfloat16)

    gu, dn = moe.mx4_prepack(normal(E, H, I), normal(E, H, I)), moe.mx4_prepack(normal(E, I, H))
    ws = moe.mx4_new_layer_workspace(d)

    def run():
        return moe.mx4_layer_forward(x, wr, b, gu, dn, d, ws, want_routing=True)

    want = run()
    assert moe.moe_read_device_status(ws) == 0
    for _ in range(3):
        out, idx, w, counts = limited(moe, 16, run)
        assert moe.STATUS[moe.moe_read_device_status(ws)] == "MOE_ERR_TIMEOUT"
        assert (w == 0).all() and ((idx >= 0) & (idx < E)).all()  # NaN logits mask every expert
        assert all(torch.equal(p, q) for p, q in zip(run(), want))
        assert moe.moe_read_device_status(ws) == 0
