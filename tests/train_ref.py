"""The operators that train the experts, plainly in 64 bits, and the error that their kernels may have."""
import torch

EPS2 = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def spans(offsets):
    o = offsets.tolist()
    return list(zip(o[:-1], o[1:]))


def product(x, offsets, w, transposed=False):
    n = w.shape[1] if transposed else w.shape[2]
    y = torch.zeros((x.shape[0], n), dtype=torch.float64, device=x.device)
    for e, (a, b) in enumerate(spans(offsets)):
        m = w[e].double()
        y[a:b] = x[a:b].double() @ (m.T if transposed else m)
    return y


def weight_grad(x, dy, offsets):
    return torch.stack([x[a:b].double().T @ dy[a:b].double() for a, b in spans(offsets)])


def sums_tol(depth):
    """Relative 2-norm error of FP32 sums of `depth` exact products, made sixteen at a time: each step aligns
    its products and drops at most 2^-23 of the running sum, whose norm does not exceed the result's (as for
    products of independent signs); sixteen more for the alignment within a step."""
    return (depth / 16 + 16) * 2.0 ** -23


def close(got, want, depth, size=None):
    """got against 64 bits: the sums' error by norm, and one rounding of the output a value.  size: the sums of
    the products' magnitudes, which bound every value's error too."""
    got64 = got.double()
    assert torch.isfinite(got64).all()
    half, tol = EPS2[got.dtype], sums_tol(depth)
    norm = want.norm()
    assert (got64 - want).norm() <= (half + tol) * norm + 1e-300, \
        ((got64 - want).norm() / norm, half + tol)
    # fp16's subnormals round to a multiple of 2^-24
    least = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    if size is None:
        size = norm / max(1, want.numel()) ** 0.5 * max(1, depth) ** 0.5
    assert ((got64 - want).abs() <= half * want.abs() + depth * 2.0 ** -23 * size + tol * size + least).all()


def swiglu(gate_up, w=None):
    i = gate_up.shape[1] // 2
    g, u = gate_up[:, :i].double(), gate_up[:, i:].double()
    h = g * torch.sigmoid(g) * u
    return h if w is None else w.double().unsqueeze(1) * h


def swiglu_backward(gate_up, d, w=None):
    i = gate_up.shape[1] // 2
    g, u, d = gate_up[:, :i].double(), gate_up[:, i:].double(), d.double()
    s = torch.sigmoid(g)
    ww = 1.0 if w is None else w.double().unsqueeze(1)
    return torch.cat([ww * d * u * s * (1 + g * (1 - s)), ww * d * g * s], 1), ww * g * s * u, (d * g * s * u).sum(1)


def orthogonalize(m, coefficients=(3.4445, -4.7750, 2.0315), steps=5, eps=1e-7):
    """(result, relative error that holding X, A and B in FP16 may leave): a step's rounding (2^-12 of each
    value, of X, of A and of B, so three) is lifted by the steps that follow, at most a times each."""
    a, b, c = coefficients
    x = m.double()
    turned = x.shape[1] > x.shape[2]
    if turned:
        x = x.transpose(1, 2)
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + eps)
    noise = 3 * 2.0 ** -12 * x.square().sum((1, 2)).sqrt()
    for _ in range(steps):
        g = x @ x.transpose(1, 2)
        x = a * x + (b * g + c * g @ g) @ x
        noise = noise * abs(a) + 3 * 2.0 ** -12 * x.square().sum((1, 2)).sqrt()
    tol = noise / x.square().sum((1, 2)).sqrt().clamp(min=1e-300)
    return (x.transpose(1, 2) if turned else x), tol
