"""Selection from router logits and its gradient (moe_router_logits, moe_route_select,
moe_route_select_bwd) against plain 64-bit references.

Tolerances, u = 2^-24 (half a step of FP32, relative).  expf is within 2 steps (4u), the
fixed-step sigmoid's exponential within 6u (seven rounded Horner steps, each later one
damped by |r| <= 0.35, and the reduction), so a sigmoid is within 6u + 2u; a sum over the
lane's E/32 values and 5 butterfly steps adds E/32 + 5 u, over the k chosen 5 u; a
division 1 u."""
import numpy as np
import pytest
import torch

import select_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def moe(cuda_ok):
    import moe_expert_layer_fp32_gb300 as m
    return m


def grid_logits(T, E, seed, dtype):
    """Logits on a grid of 1/8 in [-4, 4]: exact in every type, with many exact ties."""
    g = np.random.default_rng(seed)
    return torch.from_numpy(g.integers(-32, 33, (T, E)) / 8.0).to(DT[dtype])


def grid_bias(E, seed):
    return np.random.default_rng(seed + 99).integers(-3, 4, E) / 4.0


CASES = [  # T, E, k, groups, keep, top
    (1, 256, 8, 8, 4, 2), (5, 256, 16, 32, 3, 1), (37, 256, 8, 1, 1, 1), (33, 64, 6, 4, 2, 2),
    (7, 8, 2, 1, 1, 1), (9, 1, 1, 1, 1, 1), (3, 33, 5, 3, 2, 2), (16, 40, 8, 8, 2, 2),
    (2, 100, 16, 4, 4, 1), (130, 128, 8, 16, 5, 2), (11, 96, 1, 32, 1, 2), (8, 32, 16, 32, 16, 2),
]


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k,groups,keep,top", CASES)
def test_select(moe, T, E, k, groups, keep, top, dtype, kind):
    l = grid_logits(T, E, 7 * E + T, dtype)
    for bias in (None, grid_bias(E, E)):
        for renorm in (True, False):
            o = moe.select_opts(kind, groups, keep, top, renorm)
            tb = None if bias is None else torch.from_numpy(bias).float().cuda()
            idx, w, prob = moe.route_select(l.cuda(), k, o, bias=tb, want_prob_sum=True)
            i0, w0, p0, gap = ref.select(l.double().numpy(), bias, kind, k, groups, keep, top, renorm)
            assert gap > 1e-6, "the inputs leave a choice to the last bits"
            np.testing.assert_array_equal(idx.cpu().numpy(), i0)
            np.testing.assert_allclose(w.cpu().numpy(), w0, rtol=(E / 32 + 5 + 5 + 18) * U, atol=0)
            np.testing.assert_allclose(prob.cpu().numpy(), p0, rtol=(T + E / 32 + 5 + 60) * U, atol=0)
            i2, w2 = moe.route_select(l.cuda(), k, o, bias=tb)
            assert torch.equal(i2, idx) and torch.equal(w2, w)


@pytest.mark.parametrize("T,E,k,kind", [(1, 64, 8, 0), (40, 256, 8, 0), (300, 128, 4, 1),
                                        (1100, 64, 8, 0), (20, 10, 3, 1)])
def test_router_logits_and_selection_are_moe_route(moe, T, E, k, kind):
    """The projection's logits selected without groups give moe_route's choice and weights."""
    H = 256
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    wr = (torch.randn((H, E), generator=g) * 0.02).cuda()
    b = (torch.randn(E, generator=g) * 0.1).cuda()
    d = moe.dims(T, H, E, k, 128)
    logits = torch.empty((T, E), device="cuda")
    moe.moe_router_logits(x, wr, None, d, logits)
    exact = x.double().cpu() @ wr.double().cpu()
    scale = x.double().cpu().abs() @ wr.double().cpu().abs()
    assert ((logits.double().cpu() - exact).abs() <= H * U * scale).all()
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    moe.moe_route_ex(x, wr, b, moe.router_opts(kind), d, idx, w)
    i2, w2 = moe.route_select(logits, k, moe.select_opts(kind), bias=b)
    assert torch.equal(i2, idx)
    # both renormalise k exponentials (or sigmoids) of the same keys
    assert ((w - w2).abs() <= (2 * k + 16) * U * w.abs()).all()


@pytest.mark.parametrize("kind", [0, 1])
def test_masked_rows(moe, kind):
    """-inf and NaN mask an expert; a row without any left has weights 0 and gradient 0."""
    E, k = 64, 4
    l = grid_logits(8, E, 3, "f32")
    l[0] = -np.inf
    l[1] = np.nan
    l[2, :61] = -np.inf                       # three left: one masked expert is chosen, weight 0
    l[3, ::2] = -np.inf
    l[4, 5] = np.inf
    l[5] = torch.finfo(torch.float32).min     # the type's lowest value is a number
    l[6, :32] = np.nan                        # a whole group masked
    for groups, keep, top in ((1, 1, 1), (4, 2, 2)):
        for renorm in (True, False):
            o = moe.select_opts(kind, groups, keep, top, renorm)
            idx, w, prob = moe.route_select(l.cuda(), k, o, want_prob_sum=True)
            i0, w0, p0, _ = ref.select(l.double().numpy(), None, kind, k, groups, keep, top, renorm)
            np.testing.assert_array_equal(idx.cpu().numpy(), i0)
            np.testing.assert_allclose(w.cpu().numpy(), w0, rtol=(2 + 5 + 5 + 18) * U, atol=1e-30)
            np.testing.assert_allclose(prob.cpu().numpy(), p0, rtol=(8 + 70) * U, atol=1e-30)
            assert (w[:2] == 0).all()
            d = moe.route_select_backward(l.cuda(), idx, torch.ones_like(w), o,
                                          d_prob_sum=torch.ones(E, device="cuda"))
            rows = [0, 1, 2, 3, 5, 6, 7] if kind == 0 else range(8)
            assert torch.isfinite(d[list(rows)]).all()
            assert (d[:2] == 0).all() and (d[2, :61] == 0).all() and (d[3, ::2] == 0).all()


def test_far_below_the_maximum(moe):
    """Group sums can drop the row's largest logit; the chosen ones, 200 below it, keep their
    weights and their gradient."""
    E, k = 8, 2
    l = torch.full((1, E), -100.0)
    l[0, 0] = 100.0
    l[0, 1] = -1000.0
    l[0, 4:8] = torch.tensor([-99.0, -98.0, -97.5, -99.5])
    o = moe.select_opts(0, 2, 1, 2, True)  # group 0: 100 - 100 = 0; group 1 is below
    l[0, 2] = l[0, 3] = -400.0             # group 0: 100 - 400
    idx, w = moe.route_select(l.cuda(), k, o)
    assert idx.tolist() == [[6, 5]]
    e = np.exp(np.array([0.0, -0.5]))
    np.testing.assert_allclose(w.cpu().numpy()[0], e / e.sum(), rtol=12 * U)
    dw = torch.tensor([[1.0, -1.0]], device="cuda")
    d = moe.route_select_backward(l.cuda(), idx, dw, o).cpu().numpy()[0]
    p = e / e.sum()
    np.testing.assert_allclose(d[[6, 5]], p * (np.array([1, -1]) - (p[0] - p[1])), rtol=40 * U)


def grad_scale(l, bias, kind, idx, renorm, d_w, d_prob):
    """Per element, the sum of the magnitudes that meet in the gradient (float64)."""
    if kind == 0:
        q = torch.softmax(l if bias is None else l + bias, dim=1)
        score = q
    else:
        score = torch.sigmoid(l)
        q = score / score.sum(1, keepdim=True)
    c = score.gather(1, idx)
    a = d_w.abs()
    if renorm:
        S = c.sum(1, keepdim=True)
        a = (a + (a * c / S).sum(1, keepdim=True)) / S
    big = torch.zeros_like(l).scatter_add_(1, idx, a)
    g = torch.zeros_like(l) if d_prob is None else d_prob.abs().expand_as(l)
    if kind == 0:
        D = big + g
        return q * (D + (D * q).sum(1, keepdim=True))
    g = (g + (g * q).sum(1, keepdim=True)) / score.sum(1, keepdim=True)
    return score * (big + g)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k,groups,keep,top", CASES)
def test_gradient(moe, T, E, k, groups, keep, top, dtype, kind):
    l = grid_logits(T, E, 11 * E + T, dtype)
    gen = torch.Generator().manual_seed(T * E)
    d_w = torch.randn((T, k), generator=gen)
    d_p = torch.randn(E, generator=gen)
    for bias in (None, torch.from_numpy(grid_bias(E, 1)).float()):
        for renorm in (True, False):
            for prob in (None, d_p):
                o = moe.select_opts(kind, groups, keep, top, renorm)
                tb = None if bias is None else bias.cuda()
                idx, _ = moe.route_select(l.cuda(), k, o, bias=tb)
                want = kind == 0 and bias is not None
                r = moe.route_select_backward(l.cuda(), idx, d_w.cuda(), o, bias=tb,
                                              d_prob_sum=None if prob is None else prob.cuda(),
                                              want_d_bias=want)
                d = (r[0] if want else r).cpu()
                assert d.dtype == DT[dtype]
                l64 = l.double().requires_grad_(True)
                b64 = None if bias is None else bias.double()
                p64 = None if prob is None else prob.double()
                i = idx.cpu().long()
                L = ref.loss(l64, b64, kind, i, renorm, d_w.double(), p64)
                g = torch.autograd.grad(L, l64)[0]
                # roundings on the way to one element: sums (E/32 + 5 twice, k), the
                # exponential or sigmoid of each factor, products and divisions
                n = 2 * (E / 32 + 5) + 2 * 5 + 40
                M = grad_scale(l64.detach(), b64, kind, i, renorm, d_w.double(), p64)
                tol = n * U * M + torch.finfo(DT[dtype]).eps / 2 * g.abs() + 6e-8 * (dtype == "f16")
                assert ((d.double() - g).abs() <= tol).all()
                if want:
                    tol = (n + T + 60) * U * M.sum(0)
                    assert ((r[1].cpu().double() - g.sum(0)).abs() <= tol).all()
                # a central difference along a random direction of the 64-bit loss
                v = torch.randn((T, E), generator=gen).double()
                h = 1e-5
                with torch.no_grad():
                    f = [ref.loss(l.double() + s * h * v, b64, kind, i, renorm, d_w.double(), p64)
                         for s in (1, -1)]
                if dtype == "f32":
                    assert abs((f[0] - f[1]) / (2 * h) - (d.double() * v).sum()) <= \
                        1e-6 * max(1.0, float((M * v.abs()).sum()))


def test_ids_out_of_range_and_strides(moe):
    E, k, T = 40, 4, 9
    l = torch.randn((T, 56), generator=torch.Generator().manual_seed(1))
    wide = l.cuda()
    for dt in (torch.float32, torch.bfloat16):
        v = wide.to(dt)[:, :E]          # rows 56 apart
        o = moe.select_opts(1, 8, 3, 2)
        a = moe.route_select(v, k, o, want_prob_sum=True)
        b = moe.route_select(v.contiguous(), k, o, want_prob_sum=True)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        dw = torch.randn((T, k), device="cuda")
        assert torch.equal(moe.route_select_backward(v, a[0], dw, o),
                           moe.route_select_backward(v.contiguous(), a[0], dw, o))
    # odd rows: neither vector loads nor aligned stores
    v = wide[:, :33].contiguous()
    idx, w = moe.route_select(v, k)
    i0, w0, _, _ = ref.select(v.double().cpu().numpy(), None, 0, k)
    np.testing.assert_array_equal(idx.cpu().numpy(), i0)
    # an id outside [0, E) contributes nothing
    o = moe.select_opts(0, renorm=False)
    dw = torch.randn((T, k), device="cuda")
    bad, dz = idx.clone(), dw.clone()
    bad[:, 1] = 33
    bad[:, 2] = -5
    dz[:, 1:3] = 0
    assert torch.equal(moe.route_select_backward(v, bad, dw, o),
                       moe.route_select_backward(v, idx, dz, o))


def test_empty_batch_stream_and_graph(moe):
    E, k = 64, 4
    z = torch.empty((0, E), device="cuda")
    idx, w, p = moe.route_select(z, k, want_prob_sum=True)
    assert idx.shape == (0, k) and (p == 0).all()
    d, db = moe.route_select_backward(z, idx, w, want_d_bias=True,
                                      bias=torch.zeros(E, device="cuda"))
    assert d.shape == (0, E) and (db == 0).all()
    l = torch.randn((257, E), device="cuda")
    dw = torch.randn((257, k), device="cuda")
    want = moe.route_select(l, k, want_prob_sum=True)
    dwant = moe.route_select_backward(l, want[0], dw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = moe.route_select(l, k, want_prob_sum=True)
        dgot = moe.route_select_backward(l, got[0], dw)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(dgot, dwant)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = moe.route_select(l, k, want_prob_sum=True)
        dgot = moe.route_select_backward(l, got[0], dw)
    l.copy_(torch.randn((257, E), device="cuda"))
    graph.replay()
    want = moe.route_select(l, k, want_prob_sum=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(dgot, moe.route_select_backward(l, want[0], dw))


def test_both_ways_of_calling(moe):
    """The native fast path (dense rows) and the Python path (rows of a wider tensor) are one call,
    on the current stream and on one that is given."""
    wide = torch.randn((33, 72), device="cuda")
    v = wide[:, :64]
    l = v.contiguous()
    b = torch.randn(64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ways = [(l, None), (v, None), (l, side), (v, side), (l, side.cuda_stream)]
    for kind in (0, 1):
        o = moe.select_opts(kind, 8, 3, 2)
        r = [moe.route_select(x, 4, o, bias=b, want_prob_sum=True, stream=s) for x, s in ways]
        torch.cuda.synchronize()
        for c in r[1:]:
            assert len(c) == 3 and all(torch.equal(p, q) and p.dtype == q.dtype for p, q in zip(r[0], c))
        assert all(len(moe.route_select(x, 4, stream=s)) == 2 for x, s in ways)
        idx, dw, g = r[0][0], torch.randn((33, 4), device="cuda"), torch.randn(64, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        for want in (False, True) if kind == 0 else (False,):
            r = [moe.route_select_backward(x, idx, dw, o, bias=b, d_prob_sum=g, want_d_bias=want, stream=s)
                 for x, s in ways]
            torch.cuda.synchronize()
            r = [x if want else (x,) for x in r]
            assert all(torch.equal(p, q) for c in r[1:] for p, q in zip(r[0], c))
    for bad in (dict(k=65), dict(k=4, opts=moe.select_opts(7))):
        for x, s in ways:
            with pytest.raises(moe.MoEError):
                moe.route_select(x, stream=s, **bad)
    with pytest.raises(ValueError, match="bias"):
        moe.route_select(l, 4, bias=b[:32])
    with pytest.raises(ValueError, match="overlap"):
        moe.route_select(l[:1].expand(3, 64), 4)


def test_large_batch_is_its_rows(moe):
    """Every token's choice, weights and gradient are those it has alone in another batch."""
    T, E, k = 20011, 256, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    l = torch.randn((T, E), generator=g, device="cuda")
    b = torch.randn(E, generator=g, device="cuda") * 0.1
    o = moe.select_opts(1, 8, 4, 2)
    idx, w = moe.route_select(l, k, o, bias=b)
    dw = torch.randn((T, k), generator=g, device="cuda")
    d = moe.route_select_backward(l, idx, dw, o, bias=b)
    for r in (slice(0, 1), slice(12345, 12350), slice(T - 3, T)):
        i2, w2 = moe.route_select(l[r].contiguous(), k, o, bias=b)
        assert torch.equal(i2, idx[r]) and torch.equal(w2, w[r])
        assert torch.equal(moe.route_select_backward(l[r].contiguous(), i2, dw[r].contiguous(), o,
                                                     bias=b), d[r])


def test_past_32_bits(moe):
    """Logits of more than 2^31 elements: the last tokens are those they are alone."""
    T, E, k = 8_400_000, 256, 4
    l = torch.empty((T, E), dtype=torch.bfloat16, device="cuda")
    tile = torch.randn((10_000, E), device="cuda").to(torch.bfloat16)
    for t in range(0, T, 10_000):
        l[t:t + 10_000].copy_(tile)
    l[-9:] = torch.randn((9, E), device="cuda").to(torch.bfloat16)
    idx, w = moe.route_select(l, k)
    i2, w2 = moe.route_select(l[-500:], k)
    assert torch.equal(idx[-500:], i2) and torch.equal(w[-500:], w2)
    dw = torch.randn((T, k), device="cuda")
    d = moe.route_select_backward(l, idx, dw)
    assert torch.equal(d[-500:], moe.route_select_backward(l[-500:], i2, dw[-500:].contiguous()))
