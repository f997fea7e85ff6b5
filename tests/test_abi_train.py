"""Argument checks of the calls that train the experts: every refusal comes before anything is launched or
allocated.  CPU only (the addresses below are never read)."""
import pytest
import torch

from test_abi_host import moe  # noqa: F401  (the built library)

P, WS = 4096, (1 << 20, 1 << 40)
F32, BF16, F16 = 0, 1, 2


def refused(moe, code, call):
    with pytest.raises(moe.MoEError) as e:
        call()
    assert moe.STATUS[e.value.code] == "MOE_ERR_" + code


def test_workspaces(moe):  # noqa: F811
    w = moe.moe_grouped_workspace_bytes(8, 128, 256)
    assert w % 256 == 0 and w >= 256 + 8 * 64 * (128 + 256) * 2
    for E, K, N in ((0, 128, 128), (257, 128, 128), (2, 100, 128), (2, 128, 36), (2, 32776, 128), (2, 128, 32776),
                    (2, 0, 128), (2, 128, -8)):
        assert moe.moe_grouped_workspace_bytes(E, K, N) == 0
    assert moe.moe_expert_ffn_bwd_workspace_bytes(100, 128, 256, 8) >= moe.moe_grouped_workspace_bytes(8, 128, 512)
    for R, H, I, E in ((-1, 128, 256, 8), (100, 100, 256, 8), (100, 128, 16392, 8), (100, 128, 256, 300)):
        assert moe.moe_expert_ffn_bwd_workspace_bytes(R, H, I, E) == 0
    assert moe.moe_orthogonalize_workspace_bytes(3, 100, 70) > 2 * 3 * 100 * 72
    for E, r, c in ((0, 8, 8), (257, 8, 8), (1, 0, 8), (1, 8, 0), (1, 16385, 8), (1, 8, 16385)):
        assert moe.moe_orthogonalize_workspace_bytes(E, r, c) == 0


def test_product(moe):  # noqa: F811
    need = moe.moe_grouped_workspace_bytes(8, 64, 128)
    f = lambda **a: moe.moe_grouped_product(  # noqa: E731
        a.get("x", P), a.get("xl", 64), a.get("dt", BF16), a.get("o", P), a.get("w", P), a.get("wl", 128),
        a.get("we", 64 * 128), a.get("t", 0), a.get("R", 100), a.get("K", 64), a.get("N", 128), a.get("E", 8),
        a.get("y", P), a.get("yl", 128), a.get("yt", BF16), a.get("ws", (WS[0], need)), stream=0)
    for dt in (F32, 3, -1):
        refused(moe, "INVALID_ARG", lambda: f(dt=dt))
    refused(moe, "INVALID_ARG", lambda: f(yt=3))
    refused(moe, "INVALID_ARG", lambda: f(R=-1))
    refused(moe, "UNSUPPORTED", lambda: f(R=2 ** 31 - 1, N=32768, wl=32768, we=64 * 32768, yl=32768,
                                          ws=(WS[0], 1 << 40)))
    refused(moe, "UNSUPPORTED", lambda: f(R=2 ** 31 - 511))
    refused(moe, "UNSUPPORTED", lambda: f(K=60))
    refused(moe, "UNSUPPORTED", lambda: f(N=124))
    refused(moe, "UNSUPPORTED", lambda: f(E=257))
    refused(moe, "INVALID_ARG", lambda: f(E=0))
    refused(moe, "INVALID_ARG", lambda: f(xl=56))
    refused(moe, "INVALID_ARG", lambda: f(wl=120))
    refused(moe, "INVALID_ARG", lambda: f(we=64 * 128 - 128))       # matrices that overlap
    refused(moe, "INVALID_ARG", lambda: f(we=64 * 128 + 8))         # no whole number of rows
    refused(moe, "INVALID_ARG", lambda: f(yl=120))
    refused(moe, "UNSUPPORTED", lambda: f(xl=1 << 31))
    refused(moe, "MISALIGNED", lambda: f(xl=68))
    refused(moe, "MISALIGNED", lambda: f(yl=132))
    refused(moe, "MISALIGNED", lambda: f(x=P + 8))
    refused(moe, "MISALIGNED", lambda: f(w=P + 2))
    refused(moe, "MISALIGNED", lambda: f(y=P + 4))
    refused(moe, "MISALIGNED", lambda: f(o=P + 4))
    for k in ("x", "w", "y", "o"):
        refused(moe, "INVALID_ARG", lambda: f(**{k: None}))
    refused(moe, "INVALID_ARG", lambda: f(ws=(None, need)))
    refused(moe, "MISALIGNED", lambda: f(ws=(WS[0] + 16, need)))
    refused(moe, "WORKSPACE", lambda: f(ws=(WS[0], need - 1)))
    # transposed: the matrices are [N, K]
    refused(moe, "INVALID_ARG", lambda: f(t=1, wl=56, we=64 * 128))
    refused(moe, "INVALID_ARG", lambda: f(t=1, wl=64, we=64 * 64))


def test_weight_grad(moe):  # noqa: F811
    need = moe.moe_grouped_workspace_bytes(8, 64, 128)
    f = lambda **a: moe.moe_grouped_weight_grad(  # noqa: E731
        a.get("x", P), a.get("xl", 64), a.get("dy", P), a.get("dl", 128), a.get("dt", BF16), a.get("o", P),
        a.get("R", 100), a.get("K", 64), a.get("N", 128), a.get("E", 8), a.get("w", P), a.get("wl", 128),
        a.get("we", 64 * 128), a.get("wt", F32), a.get("acc", 0), a.get("ws", (WS[0], need)), stream=0)
    refused(moe, "INVALID_ARG", lambda: f(dt=F32))
    refused(moe, "INVALID_ARG", lambda: f(wt=5))
    refused(moe, "INVALID_ARG", lambda: f(wt=BF16, acc=1))          # sums are added to FP32 only
    refused(moe, "INVALID_ARG", lambda: f(R=-1))
    refused(moe, "UNSUPPORTED", lambda: f(N=100))
    refused(moe, "INVALID_ARG", lambda: f(dl=120))
    refused(moe, "MISALIGNED", lambda: f(wl=130, we=64 * 130))
    refused(moe, "INVALID_ARG", lambda: f(we=100))
    for k in ("x", "dy", "w", "o"):
        refused(moe, "INVALID_ARG", lambda: f(**{k: None}))
        refused(moe, "MISALIGNED", lambda: f(**{k: P + 8}))
    refused(moe, "WORKSPACE", lambda: f(ws=(WS[0], need - 1)))


def test_swiglu(moe):  # noqa: F811
    f = lambda **a: moe.moe_swiglu(a.get("g", P), a.get("gl", 128), a.get("w"), a.get("dt", BF16), a.get("R", 5),  # noqa: E731
                                   a.get("I", 64), a.get("h", P), a.get("hl", 64), stream=0)
    b = lambda **a: moe.moe_swiglu_bwd(  # noqa: E731
        a.get("g", P), a.get("gl", 128), a.get("d", P), a.get("dl", 64), a.get("w"), a.get("dt", BF16), a.get("R", 5),
        a.get("I", 64), a.get("dg", P), a.get("dgl", 128), a.get("h", P), a.get("hl", 64), a.get("dw"), stream=0)
    for c in (f, b):
        refused(moe, "INVALID_ARG", lambda: c(dt=F32))
        refused(moe, "INVALID_ARG", lambda: c(R=-1))
        refused(moe, "INVALID_ARG", lambda: c(I=0))
        refused(moe, "UNSUPPORTED", lambda: c(I=60))
        refused(moe, "INVALID_ARG", lambda: c(gl=120))
        refused(moe, "MISALIGNED", lambda: c(gl=132))
        refused(moe, "INVALID_ARG", lambda: c(hl=56))
        refused(moe, "INVALID_ARG", lambda: c(g=None))
        refused(moe, "MISALIGNED", lambda: c(w=P + 4))
    refused(moe, "INVALID_ARG", lambda: f(h=None))
    refused(moe, "INVALID_ARG", lambda: b(d=None))
    refused(moe, "INVALID_ARG", lambda: b(dg=None))
    refused(moe, "MISALIGNED", lambda: b(dw=P + 4))
    refused(moe, "INVALID_ARG", lambda: b(dl=56))


def test_experts_backward(moe):  # noqa: F811
    need = moe.moe_expert_ffn_bwd_workspace_bytes(100, 64, 128, 8)
    f = lambda **a: moe.moe_expert_ffn_bwd(  # noqa: E731
        a.get("x", P), a.get("o", P), a.get("wgu", P), a.get("wd", P), a.get("gu"), a.get("w"), a.get("dy", P),
        a.get("dt", BF16), a.get("R", 100), a.get("H", 64), a.get("I", 128), a.get("E", 8), a.get("dx"),
        a.get("dxt", BF16), a.get("dgu"), a.get("dd"), a.get("dwt", F32), a.get("acc", 0), a.get("dw"),
        a.get("ws", (WS[0], need)), stream=0)
    refused(moe, "INVALID_ARG", lambda: f(dt=F32))
    refused(moe, "INVALID_ARG", lambda: f(dwt=BF16, acc=1))
    refused(moe, "INVALID_ARG", lambda: f(dxt=9))
    refused(moe, "UNSUPPORTED", lambda: f(H=68))
    refused(moe, "UNSUPPORTED", lambda: f(I=16392))
    refused(moe, "INVALID_ARG", lambda: f(R=-1))
    for k in ("x", "o", "wgu", "wd", "dy"):
        refused(moe, "INVALID_ARG", lambda: f(**{k: None}))
    for k in ("gu", "w", "dx", "dgu", "dd", "dw"):
        refused(moe, "MISALIGNED", lambda: f(**{k: P + 8}))
    refused(moe, "WORKSPACE", lambda: f(ws=(WS[0], need - 1)))


def test_orthogonalize(moe):  # noqa: F811
    need = moe.moe_orthogonalize_workspace_bytes(3, 200, 300)
    f = lambda **a: moe.moe_orthogonalize(  # noqa: E731
        a.get("m", P), a.get("dt", F32), a.get("ld", 300), a.get("es", 60000), a.get("E", 3), a.get("r", 200),
        a.get("c", 300), a.get("co", (3.0, -4.0, 2.0)), a.get("steps", 5), a.get("eps", 1e-7), a.get("scale", 1.0),
        a.get("out", P), a.get("ot", BF16), a.get("ol", 300), a.get("oe", 60000), a.get("ws", (WS[0], need)), stream=0)
    refused(moe, "INVALID_ARG", lambda: f(dt=4))
    refused(moe, "INVALID_ARG", lambda: f(ot=F32))
    for steps in (0, -1):
        refused(moe, "INVALID_ARG", lambda: f(steps=steps))
    refused(moe, "UNSUPPORTED", lambda: f(steps=65))
    refused(moe, "UNSUPPORTED", lambda: f(E=257))
    refused(moe, "UNSUPPORTED", lambda: f(r=16385))
    refused(moe, "INVALID_ARG", lambda: f(E=0))
    refused(moe, "INVALID_ARG", lambda: f(co=None))
    refused(moe, "INVALID_ARG", lambda: f(co=(float("nan"), 1.0, 1.0)))
    for eps in (-1.0, float("nan"), float("inf")):
        refused(moe, "INVALID_ARG", lambda: f(eps=eps))
    refused(moe, "INVALID_ARG", lambda: f(scale=float("inf")))
    refused(moe, "INVALID_ARG", lambda: f(ld=299))
    refused(moe, "INVALID_ARG", lambda: f(es=59999))
    refused(moe, "INVALID_ARG", lambda: f(ol=299))
    refused(moe, "INVALID_ARG", lambda: f(oe=100))
    refused(moe, "INVALID_ARG", lambda: f(m=None))
    refused(moe, "MISALIGNED", lambda: f(out=P + 2))
    refused(moe, "WORKSPACE", lambda: f(ws=(WS[0], need - 1)))


def test_tensor_calls(moe):  # noqa: F811
    bf, off = lambda *s: torch.zeros(s, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)  # noqa: E731
    ws = torch.zeros(1024, dtype=torch.uint8)
    x, w, dy = bf(4, 64), bf(2, 64, 128), bf(4, 128)
    for call, kind in (
            (lambda: moe.grouped_product(x, off, w, ws), ValueError),                       # not on a GPU
            (lambda: moe.grouped_product(x.float(), off, w, ws), TypeError),
            (lambda: moe.grouped_product(x, off.long(), w, ws), ValueError),
            (lambda: moe.grouped_product(x, off[:1], w, ws), ValueError),
            (lambda: moe.grouped_product(x, off, w.half(), ws), ValueError),
            (lambda: moe.grouped_product(x, off, bf(3, 64, 128), ws), ValueError),
            (lambda: moe.grouped_product(x, off, bf(2, 72, 128), ws), ValueError),
            (lambda: moe.grouped_product(x, off, w, ws, transposed=True), ValueError),
            (lambda: moe.grouped_product(x, off, w.transpose(1, 2), ws), ValueError),
            (lambda: moe.grouped_product(x[:, ::2], off, w[:, ::2], ws), ValueError),
            (lambda: moe.grouped_product(x, off, w, None), TypeError),
            (lambda: moe.grouped_weight_grad(x, dy.half(), off, ws), TypeError),
            (lambda: moe.grouped_weight_grad(x, dy[:3], off, ws), ValueError),
            (lambda: moe.grouped_weight_grad(x, dy, off, ws, accumulate=True), ValueError),
            (lambda: moe.grouped_weight_grad(x, dy, off, ws), ValueError),
            (lambda: moe.swiglu(bf(4, 33)), ValueError),
            (lambda: moe.swiglu(bf(4, 32).float()), TypeError),
            (lambda: moe.swiglu(bf(4, 32), row_weights=torch.zeros(3)), ValueError),
            (lambda: moe.swiglu_backward(bf(4, 32), bf(4, 32)), ValueError),
            (lambda: moe.swiglu_backward(bf(4, 32), bf(4, 16)), ValueError),
            (lambda: moe.orthogonalize(bf(4, 32), ws), ValueError),
            (lambda: moe.orthogonalize(bf(2, 4, 32).int(), ws), TypeError),
            (lambda: moe.orthogonalize(bf(2, 4, 32).transpose(1, 2), ws), ValueError),
            (lambda: moe.orthogonalize(bf(2, 4, 32), ws, coefficients=(1.0, 2.0)), ValueError),
            (lambda: moe.orthogonalize(bf(2, 4, 32), ws, dtype=torch.float32), TypeError),
            (lambda: moe.orthogonalize(bf(2, 4, 32), ws), ValueError),
            (lambda: moe.expert_ffn_backward(x, off, bf(2, 64, 33), bf(2, 16, 64), x, ws), ValueError),
            (lambda: moe.expert_ffn_backward(x, off, bf(2, 64, 32), bf(2, 64, 16), x, ws), ValueError),
            (lambda: moe.expert_ffn_backward(x, off, bf(2, 64, 32), bf(2, 16, 64), x, ws, accumulate=True), ValueError),
            (lambda: moe.expert_ffn_backward(x, off, bf(2, 64, 32), bf(2, 16, 64), x, ws), ValueError)):
        with pytest.raises(kind):
            call()
