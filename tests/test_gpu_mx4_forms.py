"""The two forms of the grouped 4-bit product, pairs of CTAs and single CTAs, against one another:
every output element is the same sequence of MMAs, so the bits are equal."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe(cuda_ok):
    import moe_expert_layer_fp32_gb300 as m
    return m


def operands(moe, E, K, N, R, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda").to(torch.uint8)
    scales = torch.randint(118, 124, (E, N, K // 32), generator=g, device="cuda").to(torch.uint8)
    x = torch.randn((R, K), generator=g, device="cuda").to(torch.bfloat16)
    return moe.mx4_pack(codes, scales), x


@pytest.mark.parametrize("K,N", [(256, 256), (1664, 384), (4096, 512)])
def test_pairs_are_single_ctas(moe, K, N):
    """Tiles of every height (16 to 224 rows: every set of boxes that the odd CTA loads), odd and
    even numbers of weight tiles, one k-block and more than the ring holds; three inputs on one
    workspace, so that bytes of an earlier stage or call would show."""
    counts = [16 * i - i % 3 for i in range(1, 15)]
    E, R = len(counts), sum(counts)
    assert R >= 64 * E  # pairs; the few rows below are single CTAs
    off = torch.tensor([0] + counts).cumsum(0).int()
    ws, ws1 = moe.mx4_new_workspace(R, K, N, E), moe.mx4_new_workspace(R, K, N, E)
    for seed in range(3):
        packed, x = operands(moe, E, K, N, R, 10 * seed + K)
        y = moe.mx4_expert_product(x, off.cuda(), packed, N, ws, torch.float32)
        assert moe.moe_read_device_status(ws) == 0
        for e in range(E):
            r = slice(int(off[e]), int(off[e + 1]))
            o1 = torch.tensor([0] * (e + 1) + [counts[e]] * (E - e), dtype=torch.int32, device="cuda")
            y1 = moe.mx4_expert_product(x[r].contiguous(), o1, packed, N, ws1, torch.float32)
            assert torch.equal(y1, y[r]), (seed, e)
        assert moe.moe_read_device_status(ws1) == 0


@pytest.mark.parametrize("counts,K,N", [
    ([7, 0, 400, 9], 256, 128),        # single CTAs: one k-block a unit, the ring holds every unit
    ([7, 0, 20, 9], 1536, 128),        # six k-blocks: no wait for a free slot
    ([7, 0, 400, 9], 4096, 128),       # sixteen k-blocks: waits for free slots
    ([300, 0, 225, 129], 256, 256),    # pairs: the ring holds every unit
    ([300, 16, 225, 129], 1536, 384),  # pairs, an odd number of weight tiles
    ([300, 0, 225, 129], 4096, 512),   # pairs, waits for free slots
    ([90000], 256, 256),               # pairs with several units each
])
def test_timeout_in_every_form(moe, counts, K, N):
    """Under a limit far below a copy's round trip some wait runs out, in whichever role and CTA:
    the call reports it, its copies have landed when it ends, and the next call is right."""
    E, R = len(counts), sum(counts)
    packed, x = operands(moe, E, K, N, R, K + N)
    off = torch.tensor([0] + counts).cumsum(0).int().cuda()
    ws = moe.mx4_new_workspace(R, K, N, E)
    want = moe.mx4_expert_product(x, off, packed, N, ws)
    assert moe.moe_read_device_status(ws) == 0
    seen = []
    for limit in (16, 16, 16, 200, 1000, 3000):
        try:
            moe.moe_set_wait_limit(limit)
            moe.mx4_expert_product(x, off, packed, N, ws)
            seen.append(moe.moe_read_device_status(ws))
        finally:
            moe.moe_set_wait_limit(0)
        assert torch.equal(moe.mx4_expert_product(x, off, packed, N, ws), want)
        assert moe.moe_read_device_status(ws) == 0
    assert 6 in seen[:3] and set(seen) <= {0, 6}, seen
