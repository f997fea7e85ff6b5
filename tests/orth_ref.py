"""moe_orthogonalize in 64 bits: the definition, and the same with the roundings that the kernels make (X, A and B to
FP16 times 1024, the tensor cores' sums, the result of a step to FP32), whose distance from the definition is the
error to expect."""
import torch

DEFAULT = (3.4445, -4.7750, 2.0315)
HELD = 1024.0


def _fp16(x):
    return x.to(torch.float16).double()


def _fp32(x):
    return x.float().double()


def _held(x):
    return _fp16(x * HELD) / HELD


def _t(x):
    return x.transpose(1, 2)


def sums(x, y):
    """x @ y as the tensor cores sum it: sixteen products at a time, the running sum cut off towards zero.  At 23 bits,
    which loses 0.7 2^-23 of it a step on average (measured, sums of one sign of 4096 products: 1.43e-5, or 0.94)."""
    s = torch.zeros(x.shape[:-1] + y.shape[-1:], dtype=torch.float64, device=x.device)
    for k in range(0, x.shape[-1], 16):
        s += x[..., k:k + 16] @ y[..., k:k + 16, :]
        f, e = torch.frexp(s)
        s = torch.ldexp((f * 2.0 ** 23).trunc(), e - 23)
    return s


def one_kernel(rows, cols):
    return min(rows, cols) <= 128 and max(rows, cols) <= 256


def exact(m, coefficients=DEFAULT, steps=5, eps=1e-7):
    a, b, c = coefficients
    turned = m.shape[1] > m.shape[2]
    x = _t(m.double()) if turned else m.double()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + eps)
    for _ in range(steps):
        g = x @ _t(x)
        x = a * x + (b * g + c * g @ g) @ x
    return _t(x) if turned else x


def rounded(m, coefficients=DEFAULT, steps=5, eps=1e-7):
    a, b, c = coefficients
    turned, small = m.shape[1] > m.shape[2], one_kernel(*m.shape[1:])
    m64 = _t(m.double()) if turned else m.double()
    norm = m64.square().sum((1, 2), keepdim=True).sqrt()
    power = torch.exp2(9 - torch.log2(norm).floor())  # brings the norm to [512, 1024)
    x = _fp32(m64 / (norm + eps)) if small else m64 / (norm + eps)
    for i in range(steps):
        if small or i > 0:
            xh = _held(x)
            low = _fp16((x - xh) * HELD * 2048) / (HELD * 2048)
        else:
            xh = _fp16(m64 * power)
            low = _fp16((m64 * power - xh) * 2048) / 2048
            xh, low = xh / (power * (norm + eps)), low / (power * (norm + eps))
        g = sums(xh, _t(xh))
        ah = _held(g)
        bb = _fp32(b * (g if small else ah) + c * sums(ah, ah))
        bh = _held(bb)
        if small:  # what the rounding of B's diagonal left joins a
            left = torch.diagonal(bb - bh, dim1=1, dim2=2).unsqueeze(2)
            x = _fp32((a + left) * x + sums(bh, xh))
        else:
            kept = i < (steps - 2 if steps > 5 else 3)
            x = _fp32(a * (xh + low if kept else xh) + sums(bh, xh))
    return _t(x) if turned else x


def error(got, want):
    """Relative 2-norm error of a whole stack of equal weight a matrix."""
    e = (got.double() - want).square().sum((1, 2)) / want.square().sum((1, 2))
    return e.mean().sqrt().item()
