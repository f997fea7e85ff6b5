"""Selection where a trained router or a mask takes it: experts switched off through their bias,
logits far from zero, masks of the type's lowest value.

Tolerances, u = 2^-24 (half a step of FP32, relative), are those of the sums, divisions and
exponentials that meet in a value; they stand beside each test."""
import numpy as np
import pytest
import torch

import select_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def moe(cuda_ok):
    import moe_expert_layer_fp32_gb300 as m
    return m


def grid(shape, seed, top=32):
    """Values on a grid of 1/8: exact, with many exact ties."""
    g = np.random.default_rng(seed)
    return torch.from_numpy(g.integers(-top, top + 1, shape) / 8.0).float()


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("T,E,k,groups,keep,top", [
    (9, 64, 4, 1, 1, 1), (9, 64, 6, 4, 2, 2), (5, 256, 8, 8, 4, 2), (7, 40, 8, 8, 2, 1), (3, 33, 5, 3, 2, 2),
    (4, 8, 6, 1, 1, 1)])
def test_a_bias_of_minus_infinity_or_nan_masks_its_expert(moe, T, E, k, groups, keep, top, kind):
    """It is what a logit of -inf is: key -inf, score 0, no share of prob_sum, no gradient; the
    same bits as with the logits masked.  (8 experts, 6 slots: masked ones have to be chosen.)"""
    l = grid((T, E), E + T).cuda()
    b = (grid((E,), E, 6) / 4).cuda()
    off = torch.zeros(E, dtype=torch.bool)
    off[::3] = True
    bad = b.clone()
    bad[off] = torch.tensor([-np.inf, np.nan], device="cuda").repeat(E)[:int(off.sum())]
    b[off] = 0.0
    masked = l.clone()
    masked[:, off] = -np.inf
    g = torch.Generator(device="cuda").manual_seed(E)
    dw = torch.randn((T, k), generator=g, device="cuda")
    dp = torch.randn(E, generator=g, device="cuda")
    for renorm in (True, False):
        o = moe.select_opts(kind, groups, keep, top, renorm)
        want = moe.route_select(masked, k, o, bias=b, want_prob_sum=True)
        i0, w0, p0, _ = ref.select(masked.double().cpu().numpy(), b.double().cpu().numpy(), kind, k, groups, keep,
                                   top, renorm)
        np.testing.assert_array_equal(want[0].cpu().numpy(), i0)
        for prob in (True, False):
            got = moe.route_select(l, k, o, bias=bad, want_prob_sum=prob)
            assert all(torch.equal(p, q) for p, q in zip(got, want)), (renorm, prob)
        np.testing.assert_allclose(want[1].cpu().numpy(), w0, rtol=(E / 32 + 5 + 5 + 18) * U, atol=0)
        np.testing.assert_allclose(want[2].cpu().numpy(), p0, rtol=(T + E / 32 + 5 + 60) * U, atol=0)
        assert (want[2][off.cuda()] == 0).all()
        for d_prob in (None, dp):
            a = moe.route_select_backward(l, want[0], dw, o, bias=bad, d_prob_sum=d_prob)
            c = moe.route_select_backward(masked, want[0], dw, o, bias=b, d_prob_sum=d_prob)
            assert torch.equal(a, c) and (a[:, off] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,far", [(40, 64, 6, 20.0), (17, 256, 8, 20.0), (9, 40, 4, 12.0), (3, 8, 8, 20.0)])
def test_sigmoid_gradient_of_a_saturated_router(moe, T, E, k, far, dtype):
    """d l carries s (1 - s), relative to itself also where s is 1 to the last bit.

    On the way to one element: sums (E/32 + 5 twice, k), 10 products and divisions, and at most five
    exponentials (its own three times, those of the two sums), each within 2 + |l| / 2 steps of 2u on
    the special-function unit and 6u more for the reciprocal and the sum it stands in."""
    gen = torch.Generator().manual_seed(E)
    l = ((torch.rand((T, E), generator=gen) * 2 - 1) * far).to(dtype)
    l[0, :3] = torch.tensor([10.0, 12.0, 16.0]).to(dtype)
    d_w, d_p = torch.randn((T, k), generator=gen), torch.randn(E, generator=gen)
    n = 2 * (E / 32 + 5) + 2 * 5 + 10 + 5 * (2 * (2 + far / 2) + 6)
    for renorm in (True, False):
        o = moe.select_opts(1, renorm=renorm)
        idx, _ = moe.route_select(l.cuda(), k, o)
        for prob in (None, d_p):
            d = moe.route_select_backward(l.cuda(), idx, d_w.cuda(), o,
                                          d_prob_sum=None if prob is None else prob.cuda()).cpu()
            x = l.double().requires_grad_(True)
            i = idx.cpu().long()
            p64 = None if prob is None else prob.double()
            g = torch.autograd.grad(ref.loss(x, None, 1, i, renorm, d_w.double(), p64), x)[0]
            x = x.detach()
            s, one_minus = torch.sigmoid(x), torch.sigmoid(-x)
            a = d_w.double().abs()
            if renorm:
                c = s.gather(1, i)
                a = (a + (a * c).sum(1, keepdim=True) / c.sum(1, keepdim=True)) / c.sum(1, keepdim=True)
            M = torch.zeros_like(x).scatter_(1, i, a)
            if prob is not None:
                z = s.sum(1, keepdim=True)
                M = M + (p64.abs() + (p64.abs() * s).sum(1, keepdim=True) / z) / z
            # (the reference's own 1 - s loses 2^-53 / (1 - s) of itself: nothing at these tolerances)
            tol = n * U * s * one_minus * M + torch.finfo(dtype).eps / 2 * g.abs()
            err = (d.double() - g).abs()
            assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())


def test_sigmoid_gradient_at_the_ends(moe):
    """Logits of any size give finite gradients; 0 where the exponential is."""
    l = torch.tensor([[-1e30, -200.0, -80.0, 0.0, 80.0, 200.0, 1e30, float("inf")]])
    for renorm in (True, False):
        o = moe.select_opts(1, renorm=renorm)
        idx, w = moe.route_select(l.cuda(), 8, o)
        for prob in (None, torch.linspace(-1, 1, 8).cuda()):
            d = moe.route_select_backward(l.cuda(), idx, torch.linspace(1, 2, 8).cuda()[None], o, d_prob_sum=prob)
            assert torch.isfinite(d).all() and (d[0, [0, 1, 5, 6, 7]] == 0).all()
            # e^-80 of a term of size 1 (and not 0)
            assert 1e-37 < abs(float(d[0, 4])) < 1e-33 and 1e-37 < abs(float(d[0, 2])) < 1e-33


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_groups_of_lowest_values_stand_above_masked_groups(moe, kind, dtype):
    """Keys of the type's lowest value are numbers: their group's sum of two is one too, and a group
    of masked experts does not tie with it."""
    low = torch.finfo(dtype).min
    if kind == 0:
        l, b = torch.full((3, 16), low, dtype=dtype), None
    else:
        l, b = torch.zeros((3, 16), dtype=dtype), torch.full((16,), torch.finfo(torch.float32).min)
    l[0, :4] = -np.inf
    l[1, :8] = np.nan
    l[2, :12] = -np.inf
    o = moe.select_opts(kind, 4, 1, 2)
    idx, w = moe.route_select(l.cuda(), 2, o, bias=None if b is None else b.cuda())
    i0, w0, _, _ = ref.select(l.double().numpy(), None if b is None else b.double().numpy(), kind, 2, 4, 1, 2)
    assert i0.tolist() == [[4, 5], [8, 9], [12, 13]]
    np.testing.assert_array_equal(idx.cpu().numpy(), i0)
    np.testing.assert_allclose(w.cpu().numpy(), w0, rtol=8 * U)
