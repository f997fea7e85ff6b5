"""Orthogonalised updates of matrices of any size: norms below FP32's smallest normal number and above its largest, with
and without eps, values of both ends in one matrix, in the one-kernel form and in the chain of kernels."""
import pytest
import torch

import orth_ref
import train_ref as ref
from test_gpu_train import gen, normal

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def moe(cuda_ok):
    import moe_expert_layer_fp32_gb300 as m
    return m


def check(x, m, eps, extra=0.0):
    """Twice the emulated error of this matrix, and bf16's rounding."""
    want = orth_ref.exact(m, eps=eps)
    tol = 2 * orth_ref.error(orth_ref.rounded(m, eps=eps), want) + ref.EPS2[BF] + extra
    err = orth_ref.error(x, want)
    assert err <= tol, (err, tol)


@pytest.mark.parametrize("rows,cols", [(60, 100), (130, 300), (300, 130), (129, 263)])
@pytest.mark.parametrize("eps", [0.0, 1e-7])
def test_sizes_of_matrices(moe, rows, cols, eps):
    """Relative to eps every size counts: with eps = 0 the result depends on it by roundings only."""
    g = gen(rows + cols)
    sizes = [2.0 ** k for k in (-126, -100, -70, -66, -40, -36, -30, 0, 40, 50, 60, 63, 80, 100, 120)]
    one = normal(g, 1, rows, cols).clamp(-6, 6)
    one = torch.where(one.abs() < 0.01, torch.zeros_like(one), one)
    m = torch.cat([one * s for s in sizes])
    m = torch.cat([m, one * 2.0 ** 125 / 6 * 7.9])  # elements up to FP32's largest, a norm above it
    ws = moe.orthogonalize_new_workspace(len(m), rows, cols)
    x = moe.orthogonalize(m, ws, eps=eps)
    assert torch.isfinite(x).all()
    for e in range(len(m)):
        if eps == 0.0 or m[e].double().norm() > 1e3 * eps:
            check(x[e:e + 1], m[e:e + 1], eps)
    if eps > 0.0:  # far below eps: linear, too small to see
        assert x[0].abs().max() <= 2.0 ** -90
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("rows,cols", [(60, 100), (130, 300)])
def test_subnormal_and_mixed(moe, rows, cols):
    g = gen(rows)
    tiny = (torch.randint(-40, 41, (1, rows, cols), generator=g, device="cuda").double() * 2.0 ** -149).float()
    big = normal(g, 1, rows, cols) * 2.0 ** 100
    both = torch.where(torch.rand((1, rows, cols), generator=g, device="cuda") < 0.5, normal(g, 1, rows, cols) * 2.0 ** -100, big)
    ends = torch.where(torch.rand((1, rows, cols), generator=g, device="cuda") < 0.5, tiny, normal(g, 1, rows, cols) * 2.0 ** -41)
    m = torch.cat([tiny, big, both, ends, torch.zeros_like(big)])
    ws = moe.orthogonalize_new_workspace(len(m), rows, cols)
    for eps in (0.0, 1e-45, 1e-39):
        x = moe.orthogonalize(m, ws, eps=eps)
        assert torch.isfinite(x).all() and not x[4].any()
        for e in range(4):
            check(x[e:e + 1], m[e:e + 1], eps)
    # an infinity among the largest finite values, a NaN among the smallest: theirs alone
    m[0, 1, 1], m[1, 0, 0] = float("nan"), float("inf")
    y = moe.orthogonalize(m, ws, eps=1e-39)
    assert torch.isnan(y[0]).all() and torch.isnan(y[1]).all() and torch.equal(y[2:], x[2:])


@pytest.mark.parametrize("rows,cols", [(60, 100), (130, 300)])
def test_far_below_eps(moe, rows, cols):
    """|M| a millionth of eps: X is a^steps M / eps, to within what the last two iterates' 11 bits leave of it."""
    m = normal(gen(3), 2, rows, cols)
    m = m / m.square().sum((1, 2), keepdim=True).sqrt() * 1e-6
    x = moe.orthogonalize(m, moe.orthogonalize_new_workspace(2, rows, cols), eps=1.0)
    check(x, m, 1.0)


@pytest.mark.parametrize("rows,cols", [(60, 100), (130, 300)])
def test_zero_matrices(moe, rows, cols):
    """Zeros give zeros for every eps, one whose reciprocal is no FP32 number too."""
    m = torch.zeros((2, rows, cols), device="cuda")
    ws = moe.orthogonalize_new_workspace(2, rows, cols)
    for eps in (0.0, 1e-45, 1e-39, 1e-7, 1e30):
        assert not moe.orthogonalize(m, ws, eps=eps).any()
