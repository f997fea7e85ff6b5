"""Kernels whose CTA pairs share MMAs: the odd CTA stays until every commit that arrives in its shared memory has
arrived, at its ordinary end and after any role's wait ran out.  A late arrival would meet the shared memory of
whichever kernel came next, so each call is followed at once by the others, many times, and has to keep its bits."""
import pytest
import torch

from test_gpu_train import gen, normal, offsets_of

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def moe(cuda_ok):
    import moe_expert_layer_fp32_gb300 as m
    return m


def calls(moe):
    """The pair forms: the layer's GEMMs, the 4-bit product, the training products; and their status words."""
    g, counts = gen(21), [700, 900, 0, 1100]
    off, E, R, H, I = offsets_of(counts), len(counts), sum(counts), 1024, 1024
    x = normal(g, R, H, dtype=BF)
    d = moe.dims(R, H, E, 1, I)
    packed = moe.prepack(*(normal(g, E, a, b, dtype=BF, std=0.05) for a, b in ((H, I), (H, I), (I, H))), d)
    ws, y = moe.new_workspace(d), torch.empty((R, H), device="cuda")
    w, dy = normal(g, E, H, 2 * I, dtype=BF), normal(g, R, 2 * I, dtype=BF)
    mx, mws = moe.mx4_prepack(w), moe.mx4_new_workspace(R, H, 2 * I, E)
    gws = moe.grouped_new_workspace(E, H, 2 * I)
    m = normal(g, 9, 640, 1000, dtype=BF)
    ows = moe.orthogonalize_new_workspace(9, 640, 1000)

    def ffn():
        moe.moe_expert_ffn(x, off, packed, d, y, ws)
        return y.clone()

    return [(ffn, ws), (lambda: moe.mx4_expert_product(x, off, mx, 2 * I, mws), mws),
            (lambda: moe.grouped_product(x, off, w, gws), gws), (lambda: moe.grouped_weight_grad(x, dy, off, gws), gws),
            (lambda: moe.orthogonalize(m, ows, steps=2), ows)]


def test_one_behind_the_other(moe):
    fs = calls(moe)
    want = [f() for f, _ in fs]
    for _ in range(30):
        assert all(torch.equal(f(), w) for (f, _), w in zip(fs, want))
    assert all(moe.moe_read_device_status(ws) == 0 for _, ws in fs)


@pytest.mark.parametrize("which", range(5))
def test_after_a_wait_that_ran_out(moe, which):
    fs = calls(moe)
    want = [f() for f, _ in fs]
    f, ws = fs[which]
    seen = []
    for i in range(40):
        limit = 16 + 150 * i  # (whoever waits longest gives up: at first the MMAs' thread, then those behind it)
        try:
            moe.moe_set_wait_limit(limit)
            f()
        finally:
            moe.moe_set_wait_limit(0)
        got = [h() for h, _ in fs]  # (launched before the status is read)
        seen.append(moe.moe_read_device_status(ws))
        assert all(torch.equal(a, b) for a, b in zip(got, want)), limit
    assert 6 in seen and set(seen) <= {0, 6}, seen
    assert all(moe.moe_read_device_status(w) == 0 for _, w in fs)
