"""Rows past the limits, through the native path of the tensor calls and through Python: refused before an output of
that size (here up to 140 TB) is allocated."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def moe(cuda_ok):
    import moe_expert_layer_fp32_gb300 as m
    return m


@pytest.mark.parametrize("native", [True, False])
def test_rows_past_the_limits(moe, native, monkeypatch):
    if native and not moe.NATIVE_TENSOR_CALLS:
        pytest.skip("no native tensor calls here")
    if not native:
        class Declines:
            def __getattr__(self, name):
                return lambda *a: None
        monkeypatch.setattr(moe, "_calls", Declines())
    x = torch.empty((2 ** 31 - 511, 8), dtype=BF, device="cuda")  # (never read)
    off, ws = torch.zeros(2, dtype=torch.int32, device="cuda"), moe.grouped_new_workspace(1, 8, 32768)
    wide = torch.zeros((1, 8, 32768), dtype=BF, device="cuda")
    torch.cuda.reset_peak_memory_stats()
    held = torch.cuda.memory_allocated()
    for call in (lambda: moe.grouped_product(x, off, wide, ws), lambda: moe.grouped_product(x[:2 ** 29], off, wide, ws),
                 lambda: moe.grouped_product(x, off, wide[:, :, :8].contiguous(), ws),
                 lambda: moe.grouped_weight_grad(x, x, off, ws)):
        with pytest.raises(moe.MoEError) as e:
            call()
        assert moe.STATUS[e.value.code] == "MOE_ERR_UNSUPPORTED"
    assert torch.cuda.max_memory_allocated() <= held + 1024
