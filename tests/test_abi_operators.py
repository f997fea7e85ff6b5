"""Argument checks of the selection and microscaled 4-bit calls: every refusal comes before
anything is launched.  CPU only (the addresses below are never read)."""
import math

import numpy as np
import pytest
import torch

import mx4_ref
import select_ref
from test_abi_host import moe  # noqa: F401  (the built library)

P, WS = 4096, (1 << 20, 1 << 40)


def refused(moe, code, call):
    with pytest.raises(moe.MoEError) as e:
        call()
    assert moe.STATUS[e.value.code] == "MOE_ERR_" + code


@pytest.mark.parametrize("E,k,opts,code", [
    (8, 0, {}, "INVALID_ARG"), (8, 9, {}, "INVALID_ARG"), (0, 1, {}, "INVALID_ARG"),
    (257, 2, {}, "UNSUPPORTED"), (64, 17, {}, "UNSUPPORTED"),
    (64, 8, dict(kind=2), "INVALID_ARG"), (64, 8, dict(kind=-1), "INVALID_ARG"),
    (64, 8, dict(n_group=0), "INVALID_ARG"), (64, 8, dict(n_group=3), "INVALID_ARG"),
    (64, 8, dict(n_group=64, topk_group=64), "UNSUPPORTED"),
    (64, 8, dict(n_group=8, topk_group=9), "INVALID_ARG"),
    (64, 8, dict(n_group=8, topk_group=0), "INVALID_ARG"),
    (64, 8, dict(n_group=16, topk_group=1), "INVALID_ARG"),   # 4 experts left for 8 slots
    (64, 8, dict(group_top=3), "INVALID_ARG"), (64, 8, dict(group_top=0), "INVALID_ARG")])
def test_selection_rules(moe, E, k, opts, code):  # noqa: F811
    o = moe.select_opts(**opts)
    refused(moe, code, lambda: moe.moe_route_select(P, 0, max(E, 1), None, o, 4, E, k, P, P, stream=0))
    refused(moe, code, lambda: moe.moe_route_select_bwd(P, 0, max(E, 1), None, o, 4, E, k, P, P, None,
                                                        P, max(E, 1), stream=0))


def test_selection_pointers(moe):  # noqa: F811
    o = moe.select_opts()
    fwd = lambda **a: moe.moe_route_select(  # noqa: E731
        a.get("l", P), a.get("dt", 0), a.get("ld", 64), a.get("b"), a.get("o", o), a.get("T", 4), 64, 8,
        a.get("i", P), a.get("w", P), a.get("p"), a.get("ws"), stream=0)
    refused(moe, "INVALID_ARG", lambda: fwd(l=None))
    refused(moe, "INVALID_ARG", lambda: fwd(o=None))
    refused(moe, "INVALID_ARG", lambda: fwd(ld=63))
    refused(moe, "INVALID_ARG", lambda: fwd(dt=3))
    refused(moe, "INVALID_ARG", lambda: fwd(T=-1))
    refused(moe, "UNSUPPORTED", lambda: fwd(T=1 << 28))
    refused(moe, "INVALID_ARG", lambda: fwd(i=None))
    refused(moe, "MISALIGNED", lambda: fwd(w=P + 4))
    refused(moe, "MISALIGNED", lambda: fwd(l=P + 8))
    refused(moe, "MISALIGNED", lambda: fwd(b=P + 8))
    refused(moe, "INVALID_ARG", lambda: fwd(p=P))                       # prob_sum without workspace
    refused(moe, "MISALIGNED", lambda: fwd(p=P, ws=(WS[0] + 16, WS[1])))
    refused(moe, "WORKSPACE", lambda: fwd(p=P, ws=(WS[0], moe.moe_select_workspace_bytes(4, 64) - 1)))
    bwd = lambda **a: moe.moe_route_select_bwd(  # noqa: E731
        P, 0, 64, a.get("b"), a.get("o", o), 4, 64, 8, a.get("i", P), a.get("w", P), None,
        a.get("d", P), a.get("ld", 64), a.get("db"), a.get("ws"), stream=0)
    refused(moe, "INVALID_ARG", lambda: bwd(d=None))
    refused(moe, "INVALID_ARG", lambda: bwd(ld=8))
    refused(moe, "INVALID_ARG", lambda: bwd(w=None))
    refused(moe, "INVALID_ARG", lambda: bwd(db=P))
    refused(moe, "INVALID_ARG", lambda: bwd(db=P, ws=WS, o=moe.select_opts(1)))  # no such gradient
    assert moe.moe_select_workspace_bytes(-1, 8) == 0 and moe.moe_select_workspace_bytes(8, 257) == 0


def test_quantize_arguments(moe):  # noqa: F811
    q = lambda **a: moe.moe_mx4_quantize(  # noqa: E731
        a.get("x", P), a.get("dt", 1), a.get("ld", 64), a.get("R", 3), a.get("K", 64), a.get("c", P),
        a.get("s", P), a.get("v", P), stream=0)
    refused(moe, "INVALID_ARG", lambda: q(dt=7))
    refused(moe, "INVALID_ARG", lambda: q(K=0))
    refused(moe, "INVALID_ARG", lambda: q(R=-1))
    refused(moe, "INVALID_ARG", lambda: q(ld=32))
    refused(moe, "UNSUPPORTED", lambda: q(K=48, ld=48))
    refused(moe, "UNSUPPORTED", lambda: q(R=1 << 40))
    refused(moe, "MISALIGNED", lambda: q(ld=65))
    refused(moe, "INVALID_ARG", lambda: q(x=None))
    refused(moe, "MISALIGNED", lambda: q(c=P + 1))
    refused(moe, "MISALIGNED", lambda: q(v=P + 2))


def test_product_and_pack_arguments(moe):  # noqa: F811
    assert moe.moe_mx4_packed_bytes(2, 256, 128) == 2 * 17408
    for E, K, N in ((0, 128, 128), (257, 128, 128), (2, 64, 128), (2, 128, 200), (2, 16512, 128),
                    (2, 128, 32896)):
        assert moe.moe_mx4_packed_bytes(E, K, N) == 0
    need = moe.moe_mx4_product_workspace_bytes(100, 256, 8)
    assert need % 256 == 0 and need >= 100 * 128 + 256
    assert moe.moe_mx4_product_workspace_bytes(-1, 256, 8) == 0
    pr = lambda **a: moe.moe_mx4_expert_product(  # noqa: E731
        a.get("x", P), a.get("dt", 1), a.get("o", P), a.get("w", P), a.get("R", 100), a.get("K", 256),
        a.get("N", 128), a.get("E", 8), a.get("y", P), a.get("yt", 0), a.get("ws", (WS[0], need)), stream=0)
    refused(moe, "INVALID_ARG", lambda: pr(dt=3))
    refused(moe, "INVALID_ARG", lambda: pr(yt=2))
    refused(moe, "INVALID_ARG", lambda: pr(R=-1))
    refused(moe, "UNSUPPORTED", lambda: pr(K=192))
    refused(moe, "UNSUPPORTED", lambda: pr(N=64))
    refused(moe, "UNSUPPORTED", lambda: pr(E=300))
    refused(moe, "INVALID_ARG", lambda: pr(x=None))
    refused(moe, "INVALID_ARG", lambda: pr(o=None))
    refused(moe, "MISALIGNED", lambda: pr(w=P + 8))
    refused(moe, "MISALIGNED", lambda: pr(y=P + 4))
    refused(moe, "INVALID_ARG", lambda: pr(ws=(None, need)))
    refused(moe, "MISALIGNED", lambda: pr(ws=(WS[0] + 128, need)))
    refused(moe, "WORKSPACE", lambda: pr(ws=(WS[0], need - 1)))
    refused(moe, "UNSUPPORTED", lambda: moe.moe_mx4_pack(P, P, 2, 100, 128, P, stream=0))
    refused(moe, "INVALID_ARG", lambda: moe.moe_mx4_pack(None, P, 2, 128, 128, P, stream=0))
    refused(moe, "INVALID_ARG", lambda: moe.moe_mx4_prepack(P, 2, 128, 128, 128, 128, P, stream=0))
    refused(moe, "INVALID_ARG", lambda: moe.moe_mx4_prepack(P, 2, 128, 128, 64, 512, P, stream=0))
    refused(moe, "INVALID_ARG", lambda: moe.moe_mx4_prepack(P, 2, 128, 128, -128, 512, P, stream=0))


def test_layer_arguments(moe):  # noqa: F811
    d = moe.dims(16, 256, 8, 2, 128)
    need = moe.moe_mx4_layer_workspace_bytes(d)
    assert moe.moe_mx4_layer_workspace_bytes(moe.dims(16, 200, 8, 2, 128)) == 0
    ly = lambda **a: moe.moe_mx4_layer_fwd(  # noqa: E731
        a.get("x", P), P, a.get("b"), a.get("o", moe.select_opts()), a.get("s", 1.0), a.get("g", P), P, d,
        a.get("out", P), None, None, None, a.get("ws", (WS[0], need)), stream=0)
    refused(moe, "INVALID_ARG", lambda: ly(o=None))
    refused(moe, "INVALID_ARG", lambda: ly(s=0.0))
    refused(moe, "INVALID_ARG", lambda: ly(s=math.inf))
    refused(moe, "INVALID_ARG", lambda: ly(g=None))
    refused(moe, "INVALID_ARG", lambda: ly(x=None))
    refused(moe, "MISALIGNED", lambda: ly(out=P + 2))
    refused(moe, "WORKSPACE", lambda: ly(ws=(WS[0], need - 1)))
    refused(moe, "INVALID_ARG", lambda: moe.moe_router_logits(None, P, None, d, P, stream=0))
    refused(moe, "UNSUPPORTED",
            lambda: moe.moe_router_logits(P, P, None, moe.dims(4, 100, 8, 2, 128), P, stream=0))


def test_tensor_calls_refuse_what_they_would_misread(moe):  # noqa: F811
    l = torch.randn(4, 8)
    with pytest.raises(ValueError, match="CUDA device"):
        moe.route_select(l, 2)
    with pytest.raises(TypeError):
        moe.route_select(l.double(), 2)
    with pytest.raises(ValueError, match="adjacent"):
        moe.route_select(torch.randn(8, 4).t(), 2)
    with pytest.raises(ValueError, match="overlap"):
        moe.route_select(l[:1].expand(4, 8), 2)
    with pytest.raises(ValueError, match="bias"):
        moe.route_select(l, 2, bias=torch.zeros(7))
    with pytest.raises(ValueError, match="d_topk_w"):
        moe.route_select_backward(l, torch.zeros((4, 2), dtype=torch.int32), torch.zeros(4, 3))
    with pytest.raises(ValueError, match="topk_idx"):
        moe.route_select_backward(l, torch.zeros((4, 2), dtype=torch.int64), torch.zeros(4, 2))
    with pytest.raises(ValueError, match="CUDA device"):
        moe.mx4_quantize(torch.randn(4, 64))
    with pytest.raises(ValueError, match="2D"):
        moe.mx4_quantize(torch.randn(64))
    with pytest.raises(ValueError, match="dense"):
        moe.mx4_expert_product(torch.randn(4, 256)[:, :128], torch.zeros(3, dtype=torch.int32),
                               torch.zeros(8), 128, None)
    with pytest.raises(ValueError, match="packed"):
        moe.mx4_expert_product(torch.randn(4, 128), torch.zeros(3, dtype=torch.int32),
                               torch.zeros(8), 128, None)
    with pytest.raises(ValueError, match="scales"):
        moe.mx4_pack(torch.zeros((2, 128, 64), dtype=torch.uint8), torch.zeros((2, 128, 3), dtype=torch.uint8))


# ---------------------------------------------------- the references themselves ---
def test_quantize_reference():
    c, s = mx4_ref.quantize(np.array([[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9] + [0.0] * 24]))
    assert mx4_ref.values(c, s)[0, :8].tolist() == [0, 1, 1, 2, 2, 4, 4, 6] and s[0, 0] == 127
    c, s = mx4_ref.quantize(np.full((1, 32), 2.0 ** -140))
    assert s[0, 0] == 0 and (c == 0).all()
    assert (mx4_ref.quantize(np.full((1, 32), np.inf))[1] == 255).all()
    assert (mx4_ref.unpack(mx4_ref.pack(np.arange(16, dtype=np.uint8)[None])) == np.arange(16)).all()


def test_selection_reference():
    l = np.array([[1.0, 3.0, 2.0, 2.0, -np.inf, 0.0, 2.5, 2.5]])
    i, w, p, _ = select_ref.select(l, None, 0, 2)
    assert i.tolist() == [[1, 6]] and abs(w.sum() - 1) < 1e-15 and abs(p.sum() - 1) < 1e-15
    # groups of two: sums 4, 4, 0, 5; the last and, of the equal ones, the first
    i, _, _, _ = select_ref.select(l, None, 0, 3, groups=4, keep=2, top=2)
    assert i.tolist() == [[1, 6, 7]]
    # a mistake in the rule shows: groups by their largest key keep {1, 3} instead of {0, 3}
    l2 = np.array([[3.0, 0.0, 2.0, 2.0]])
    assert select_ref.select(l2, None, 0, 1, 2, 1, 2)[0].tolist() == [[2]]
    assert select_ref.select(l2, None, 0, 1, 2, 1, 1)[0].tolist() == [[0]]
