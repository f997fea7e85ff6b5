"""Failure detection in every form of the grouped expert GEMMs, without a fault: under a limit far
below a copy's round trip some bounded wait runs out, in whichever role (and CTA of a pair) it is.
The call reports MOE_ERR_TIMEOUT, its copies and MMAs have ended when it ends, and the next
call in the same context is right."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe(cuda_ok):
    import moe_expert_layer_fp32_gb300 as m
    return m


@pytest.mark.parametrize("counts,H,I,form", [
    ([100, 0, 300, 112], 128, 128, 0),    # single CTAs: two k-blocks, the ring holds every unit
    ([100, 0, 300, 112], 1152, 640, 0),   # single CTAs that wait for free slots
    ([700, 900], 1024, 1024, 0),          # pairs
    ([1, 0, 3, 12], 256, 128, 1),         # swapped: four k-blocks
    ([40, 0, 3, 12, 1, 2, 3, 3], 1024, 512, 1),  # swapped: waits for free slots, several token tiles
    ([1, 1, 0, 1, 1], 2048, 1024, 1),     # swapped, the few-token form
])
def test_timeout_in_every_form(moe, counts, H, I, form):
    E, R = len(counts), sum(counts)
    g = torch.Generator(device="cuda").manual_seed(H + R)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)

    d = moe.dims(R, H, E, 1, I)  # k = 1: R rows
    assert moe.moe_expert_ffn_form(d) == form
    packed = moe.prepack(normal(E, H, I, std=0.05), normal(E, H, I, std=0.05), normal(E, I, H, std=0.05), d)
    off = torch.tensor([0] + counts).cumsum(0).int().cuda()
    x, ws = normal(R, H), moe.new_workspace(d)

    def run():
        y = torch.zeros((R, H), device="cuda")
        moe.moe_expert_ffn(x, off, packed, d, y, ws)
        return y

    want = run()
    assert moe.moe_read_device_status(ws) == 0
    seen = []
    for limit in (16, 16, 16, 200, 1000, 3000):
        try:
            moe.moe_set_wait_limit(limit)
            run()
            seen.append(moe.moe_read_device_status(ws))
        finally:
            moe.moe_set_wait_limit(0)
        assert torch.equal(run(), want)
        assert moe.moe_read_device_status(ws) == 0
    assert 6 in seen[:3] and set(seen) <= {0, 6}, seen
