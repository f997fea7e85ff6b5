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
