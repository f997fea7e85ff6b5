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


@pytest.mark.parametrize("rows,cols", [(60, 100), (130, 300)])
def test_zero_matrices(moe, rows, cols):
    """Zeros give zeros for every eps, one whose reciprocal is no FP32 number too."""
    m = torch.zeros((2, rows, cols), device="cuda")
    ws = moe.orthogonalize_new_workspace(2, rows, cols)
    for eps in (0.0, 1e-45, 1e-39, 1e-7, 1e30):
        assert not moe.orthogonalize(m, ws, eps=eps).any()
