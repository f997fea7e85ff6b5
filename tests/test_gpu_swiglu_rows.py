"""SwiGLU and its gradient over rows on both sides of the border between their two kernels: against 64 bits, and the
same bits for the same values in rows of either length."""
import pytest
import torch

import train_ref as ref
from test_gpu_train import gen, normal

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def moe(cuda_ok):
    import moe_expert_layer_fp32_gb300 as m
    return m


@pytest.mark.parametrize("I", [8, 248, 256, 264, 512, 2040, 2048, 2056, 3080, 8192, 8200])
@pytest.mark.parametrize("dt", [BF, HF])
def test_lengths(moe, I, dt):
    """Tolerances as in test_gpu_train.py's test of the same calls."""
    g, R = gen(I), 37
    gu, d = normal(g, R, 2 * I, dtype=dt, std=2.0), normal(g, R, I, dtype=dt, std=0.1)
    w = torch.rand(R, generator=g, device="cuda")
    dgu, h, dw = ref.swiglu_backward(gu, d, w)
    got, fwd = moe.swiglu_backward(gu, d, w), moe.swiglu(gu, w)
    half, least = ref.EPS2[dt], 2.0 ** -25 if dt == HF else 0.0
    gg, u = gu[:, :I].double(), gu[:, I:].double()
    rel = 2.0 ** -23 * (8 + 2 * gg.abs())
    wd = d.double().abs() * w.double().unsqueeze(1)
    size = torch.cat([wd * u.abs() * (1 + gg.abs()), wd * gg.abs()], 1) * torch.cat([rel, rel], 1)
    assert ((got[0].double() - dgu).abs() <= half * dgu.abs() + size + least).all()
    for v in (got[1], fwd):
        assert ((v.double() - h).abs() <= half * h.abs() + rel * h.abs() + least).all()
    mag = (d.double() * ref.swiglu(gu)).abs()
    assert ((got[2].double() - dw).abs() <= (mag * (rel + (I / 32 + 8) * 2.0 ** -24)).sum(1)).all()


def test_same_bits_in_either_kernel(moe):
    """Rows of 1000 values, and the same with zeros behind them up to 4000: a value's results do not change, nor does
    the sum over a row (zeros add nothing, and a lane's order is the same)."""
    g, R, I, L = gen(5), 50, 1000, 4000
    gu, d = normal(g, R, 2 * I, dtype=BF), normal(g, R, I, dtype=BF)
    w = torch.rand(R, generator=g, device="cuda")
    wide, dl = torch.zeros((R, 2 * L), dtype=BF, device="cuda"), torch.zeros((R, L), dtype=BF, device="cuda")
    wide[:, :I], wide[:, L:L + I], dl[:, :I] = gu[:, :I], gu[:, I:], d
    a, b = moe.swiglu_backward(gu, d, w), moe.swiglu_backward(wide, dl, w)
    assert torch.equal(a[0], torch.cat([b[0][:, :I], b[0][:, L:L + I]], 1))
    assert torch.equal(a[1], b[1][:, :I]) and torch.equal(a[2], b[2])
    assert torch.equal(moe.swiglu(gu, w), moe.swiglu(wide, w)[:, :I])
