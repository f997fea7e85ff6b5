"""Orthogonalised updates against their definition in 64 bits, at the error that the kernels' own roundings make
(emulated in 64 bits) and not much more: low rank over many steps, where what a rounding leaves outside of the
matrix's span is lifted again and again, and full rank on both sides of the border between the two forms."""
import pytest
import torch

import orth_ref
import train_ref as ref
from test_gpu_train import gen, normal

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
CONVERGENT, CUBE = (1.875, -1.25, 0.375), (2.0, -1.5, 0.5)


@pytest.fixture(scope="module")
def moe(cuda_ok):
    import moe_expert_layer_fp32_gb300 as m
    return m


def low_rank(g, E, rows, cols, rank):
    return normal(g, E, rows, rank) @ normal(g, E, rank, cols)


@pytest.mark.parametrize("rows,cols,rank", [(300, 500, 8), (500, 300, 8), (300, 500, 64), (520, 260, 3), (128, 256, 8), (256, 100, 8),
                                            (120, 130, 2), (40, 600, 3)])
@pytest.mark.parametrize("co,steps", [(orth_ref.DEFAULT, n) for n in (5, 6, 7, 8, 10)] + [(CONVERGENT, 15), (CUBE, 12)])
def test_low_rank_over_many_steps(moe, rows, cols, rank, co, steps):
    """Twice the emulated error, and what the first step's FP32 sums may leave outside of the span (ref.sums_tol of a X, as
    |B| < a), lifted by each step that follows."""
    E = 6
    m = low_rank(gen(rows + rank), E, rows, cols, rank)
    ws = moe.orthogonalize_new_workspace(E, rows, cols)
    want = orth_ref.exact(m, co, steps)
    tol = 2 * orth_ref.error(orth_ref.rounded(m, co, steps), want) + co[0] ** (steps - 1) * ref.sums_tol(min(rows, cols))
    assert tol <= (0.5 if steps == 10 else 0.05)
    for dt in (HF, BF):
        err = orth_ref.error(moe.orthogonalize(m, ws, coefficients=co, steps=steps, dtype=dt), want)
        assert err <= tol + ref.EPS2[dt], (err, tol)
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("E,rows,cols", [(256, 8, 8), (256, 1, 256), (128, 5, 256), (32, 128, 128), (16, 128, 256), (16, 256, 128),
                                         (256, 5, 257), (32, 257, 40), (16, 129, 200), (16, 200, 129), (128, 1, 1000), (16, 40, 1000),
                                         (4, 300, 520), (2, 1000, 700), (2, 513, 511)])
@pytest.mark.parametrize("dt", [F32, BF])
def test_full_rank(moe, E, rows, cols, dt):
    """A quarter more than the emulated error in mean square, and fp16's own rounding beside it (independent)."""
    m = normal(gen(rows * cols), E, rows, cols, dtype=dt)
    ws = moe.orthogonalize_new_workspace(E, rows, cols)
    for co, steps in ((orth_ref.DEFAULT, 5), (orth_ref.DEFAULT, 2), (orth_ref.DEFAULT, 8), (CONVERGENT, 15)):
        want = orth_ref.exact(m, co, steps)
        emulated = orth_ref.error(orth_ref.rounded(m, co, steps), want)
        err = orth_ref.error(moe.orthogonalize(m, ws, coefficients=co, steps=steps, dtype=HF), want)
        assert err <= ((1.25 * emulated) ** 2 + 2.0 ** -22) ** 0.5, (err, emulated)
    assert moe.moe_read_device_status(ws) == 0


def test_more_steps_than_buffers(moe):
    """Every number of steps up to the limit: finite, and a convergent triple's result stays orthogonal."""
    g = gen(4)
    for rows, cols in ((100, 200), (200, 300)):
        m = normal(g, 3, rows, cols)
        ws = moe.orthogonalize_new_workspace(3, rows, cols)
        for steps in (1, 2, 3, 4, 5, 6, 7, 12, 31, 64):
            x = moe.orthogonalize(m, ws, coefficients=CONVERGENT, steps=steps, dtype=HF).double()
            assert torch.isfinite(x).all()
            if steps >= 31:  # singular values within what holding X, A and B in 11 bits leaves, and fp16's rounding
                s = torch.linalg.svdvals(x)
                assert (s - 1).abs().max() <= 0.01
