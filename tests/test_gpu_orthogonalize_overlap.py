"""Orthogonalised updates written over their own input: the same tensor, the same bytes as another type, other strides and
a shifted place give what a result elsewhere gives."""
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


def close(x, want, emulated):
    """Twice the emulated error of either form, and the output's rounding."""
    err = orth_ref.error(x, want)
    assert err <= 2 * max(emulated, 2.0 ** -10) + ref.EPS2[x.dtype], (err, emulated)


# (as many matrices as there may be: more than there are SMs, so that some start when others have ended)
@pytest.mark.parametrize("E,rows,cols", [(256, 128, 256), (256, 40, 64), (256, 200, 64), (40, 130, 264), (1, 128, 256)])
def test_result_over_its_input(moe, E, rows, cols):
    g = gen(rows)
    ws = moe.orthogonalize_new_workspace(E, rows, cols)
    m32, n = normal(g, E, rows, cols), E * rows * cols
    want = orth_ref.exact(m32)
    emulated = orth_ref.error(orth_ref.rounded(m32[:4]), want[:4])
    # FP32 momenta, the 16-bit result in the first half of their bytes: result 1 lies in matrix 0
    for dt in (BF, HF):
        m = m32.clone()
        out = m.view(-1).view(dt)[:n].view(E, rows, cols)
        assert moe.orthogonalize(m, ws, dtype=dt, out=out) is out
        close(out, want, emulated)
        m = m32.clone()  # and in the second half
        out = m.view(-1).view(dt)[n:].view(E, rows, cols)
        moe.orthogonalize(m, ws, dtype=dt, out=out)
        close(out, want, emulated)
    m16 = m32.to(BF)
    elsewhere, want = moe.orthogonalize(m16, ws), orth_ref.exact(m16)
    m = m16.clone()
    moe.orthogonalize(m, ws, out=m)
    assert torch.equal(m, elsewhere)
    # dense matrices, results with a gap between them; and the other way round
    buf = torch.zeros(E * (rows + 3) * cols, dtype=BF, device="cuda")
    dense, wide = buf[:n].view(E, rows, cols), buf.view(E, rows + 3, cols)[:, :rows]
    for src, dst in ((dense, wide), (wide, dense)):
        src.copy_(m16)
        moe.orthogonalize(src, ws, out=dst)
        close(dst, want, emulated)
    # one matrix further
    buf = torch.zeros((E + 1, rows, cols), dtype=BF, device="cuda")
    for src, dst in ((buf[:E], buf[1:]), (buf[1:], buf[:E])):
        src.copy_(m16)
        moe.orthogonalize(src, ws, out=dst)
        close(dst, want, emulated)
    assert moe.moe_read_device_status(ws) == 0
