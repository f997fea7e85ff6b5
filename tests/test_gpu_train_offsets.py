"""Offsets that are no sequence from 0 to R: every grouped call of the training side flags them and leaves all of its
outputs as they were, also where a good call used the same workspace before and where there are no rows."""
import pytest
import torch

from test_gpu_train import gen, normal, offsets_of

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEVICE_CHECK = 7


@pytest.fixture(scope="module")
def moe(cuda_ok):
    import moe_expert_layer_fp32_gb300 as m
    return m


def ints(*v):
    return torch.tensor(v).int().cuda()


@pytest.mark.parametrize("kept", [True, False])
@pytest.mark.parametrize("R", [40, 2000])
def test_experts_backward_writes_nothing(moe, R, kept):
    g, E, H, I = gen(R), 3, 64, 128
    x, dy = normal(g, R, H, dtype=BF), normal(g, R, H, dtype=BF)
    wgu, wd = normal(g, E, H, 2 * I, dtype=BF), normal(g, E, I, H, dtype=BF)
    w, ws = torch.rand(R, generator=g, device="cuda"), moe.expert_ffn_backward_new_workspace(R, H, I, E)
    good = offsets_of([10, R - 20, 10])
    gu = moe.grouped_product(x, good, wgu, moe.grouped_new_workspace(E, H, 2 * I)) if kept else None
    out = lambda: [torch.full(s, 7.0, device="cuda", dtype=t)  # noqa: E731
                   for s, t in (((R, H), BF), ((E, H, 2 * I), F32), ((E, I, H), F32), ((R,), F32))]

    def run(off):
        dx, dgu, dd, dw = o = out()
        moe.moe_expert_ffn_bwd(x, off, wgu, wd, gu, w, dy, moe.MOE_DTYPE_BF16, R, H, I, E, dx, moe.MOE_DTYPE_BF16,
                               dgu, dd, moe.MOE_DTYPE_F32, False, dw, ws)
        return o, moe.moe_read_device_status(ws)

    want, status = run(good)
    assert status == 0 and all(torch.isfinite(t).all() for t in want)
    for bad in (ints(0, 10, 5, R), ints(0, 10, 20, R + 1), ints(1, 10, 20, R), ints(0, 10, 20, R - 1),
                ints(0, R + 10, 20, R), ints(0, -5, 20, R), ints(-2 ** 31, 0, 0, R)):
        got, status = run(bad)
        assert status == DEVICE_CHECK and all((t == 7).all() for t in got)
        again, status = run(good)
        assert status == 0 and all(torch.equal(a, b) for a, b in zip(again, want))


def test_without_rows(moe):
    E, H, I = 3, 64, 128
    none, w = torch.empty((0, H), dtype=BF, device="cuda"), torch.zeros((E, H, I), dtype=BF, device="cuda")
    ws, bws = moe.grouped_new_workspace(E, H, I), moe.expert_ffn_backward_new_workspace(0, H, I, E)
    wide = torch.empty((0, I), dtype=BF, device="cuda")
    wgu, wd = torch.zeros((E, H, 2 * I), dtype=BF, device="cuda"), torch.zeros((E, I, H), dtype=BF, device="cuda")
    for off in (ints(0, 0, 0, 1), ints(0, 0, 5, 0), ints(1, 1, 1, 1), ints(0, -1, 0, 0)):
        d = torch.full((E, H, I), 7.0, device="cuda")
        assert moe.grouped_product(none, off, w, ws).shape == (0, I)
        assert moe.moe_read_device_status(ws) == DEVICE_CHECK
        for add in (False, True):
            moe.grouped_weight_grad(none, wide, off, ws, out=d, accumulate=add)
            assert moe.moe_read_device_status(ws) == DEVICE_CHECK and (d == 7).all()
        du, dd = torch.full((E, H, 2 * I), 7.0, device="cuda"), torch.full((E, I, H), 7.0, device="cuda")
        moe.expert_ffn_backward(none, off, wgu, wd, none, bws, d_w_gate_up=du, d_w_down=dd)
        assert moe.moe_read_device_status(bws) == DEVICE_CHECK and (du == 7).all() and (dd == 7).all()
    # good ones: zeros between what lies beside them, or nothing where the gradient is added
    off = ints(0, 0, 0, 0)
    for dt in (F32, BF, torch.float16):
        d = torch.full((E, H + 1, 2 * I), 7.0, device="cuda", dtype=dt)
        moe.grouped_weight_grad(none, wide, off, ws, out=d[:, 1:, I:])
        assert not d[:, 1:, I:].any() and (d[:, 0] == 7).all() and (d[:, :, :I] == 7).all()
    d = torch.full((E, H, I), 7.0, device="cuda")
    moe.grouped_weight_grad(none, wide, off, ws, out=d, accumulate=True)
    assert (d == 7).all() and moe.moe_read_device_status(ws) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.grouped_weight_grad(none, wide, off, ws, out=d)
    graph.replay()
    torch.cuda.synchronize()
    assert not d.any()
