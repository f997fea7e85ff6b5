"""Arguments of the training calls that are no tensors, and sizes past the limits.  CPU only: every refusal comes before
anything is allocated or launched."""
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


def test_sizes_are_refused_before_an_allocation(moe, monkeypatch):  # noqa: F811
    """(Outputs of these sizes would take terabytes, or the input's bytes once more.)"""
    monkeypatch.setattr(moe, "_on_device", lambda *t: None)
    make = torch.empty
    bf = lambda *s: make(s, dtype=torch.bfloat16, device="meta")  # noqa: E731
    off, ws, rows = torch.zeros(2, dtype=torch.int32), torch.zeros(1024, dtype=torch.uint8), 2 ** 31 - 511
    calls = [lambda: moe.grouped_product(bf(rows, 8), off, bf(1, 8, 8), ws),
             lambda: moe.grouped_product(bf(2 ** 29, 8), off, bf(1, 8, 32768), ws),     # rows, but too many tiles
             lambda: moe.grouped_product(bf(2 ** 29, 8), off, bf(1, 32768, 8), ws, transposed=True),
             lambda: moe.grouped_product(bf(4, 12), off, bf(1, 12, 8), ws),
             lambda: moe.grouped_weight_grad(bf(rows, 8), bf(rows, 8), off, ws),
             lambda: moe.grouped_weight_grad(bf(2 ** 29, 32768), bf(2 ** 29, 32768), off, ws),
             lambda: moe.expert_ffn_backward(bf(rows, 8), off, bf(1, 8, 16), bf(1, 8, 8), bf(rows, 8), ws),
             lambda: moe.expert_ffn_backward(bf(2 ** 29, 8), off, bf(1, 8, 32768), bf(1, 16384, 8), bf(2 ** 29, 8), ws),
             lambda: moe.swiglu(bf(3, 2 ** 25 + 16)),
             lambda: moe.swiglu(bf(3, 24)),
             lambda: moe.swiglu_backward(bf(3, 2 ** 25 + 16), bf(3, 2 ** 24 + 8)),
             lambda: moe.orthogonalize(bf(1, 16385, 8), ws),
             lambda: moe.orthogonalize(bf(257, 8, 8), ws)]

    def allocates(*a, **k):
        raise AssertionError("allocated")

    monkeypatch.setattr(torch, "empty", allocates)
    for call in calls:
        with pytest.raises(moe.MoEError) as e:
            call()
        assert moe.STATUS[e.value.code] == "MOE_ERR_UNSUPPORTED"
