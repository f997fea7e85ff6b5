"""Arguments of the training calls that are no tensors.  CPU only: every refusal comes before anything is launched."""
import pytest
import torch

from test_abi_host import moe  # noqa: F401  (the built library)


@pytest.mark.parametrize("bad", [[1.0, 2.0], 7, "out", object()], ids=["list", "int", "text", "object"])
def test_no_tensors(moe, bad, monkeypatch):  # noqa: F811
    monkeypatch.setattr(moe, "_on_device", lambda *t: [x.get_device() for x in t if x is not None])
    bf, off = lambda *s: torch.zeros(s, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)  # noqa: E731
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    x, w, dy, gu = bf(4, 64), bf(2, 64, 128), bf(4, 128), bf(4, 32)
    wgu, wd = bf(2, 64, 32), bf(2, 16, 64)
    for call in (
            lambda: moe.grouped_product(x, off, w, ws, out=bad),
            lambda: moe.grouped_weight_grad(x, dy, off, ws, out=bad),
            lambda: moe.grouped_weight_grad(x, dy, off, ws, out=bad, accumulate=True),
            lambda: moe.orthogonalize(w, ws, out=bad),
            lambda: moe.orthogonalize(w, bad),
            lambda: moe.swiglu(gu, row_weights=bad),
            lambda: moe.swiglu(bad),
            lambda: moe.swiglu_backward(gu, bad),
            lambda: moe.swiglu_backward(gu, bf(4, 16), row_weights=bad),
            lambda: moe.expert_ffn_backward(x, off, wgu, wd, x, ws, row_weights=bad),
            lambda: moe.expert_ffn_backward(x, off, wgu, wd, x, ws, gate_up=bad),
            lambda: moe.expert_ffn_backward(x, off, wgu, wd, x, ws, d_w_gate_up=bad),
            lambda: moe.expert_ffn_backward(x, off, wgu, wd, x, ws, d_w_down=bad)):
        with pytest.raises(TypeError, match="a tensor, not"):
            call()
