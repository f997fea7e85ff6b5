"""Plain references of microscaled 4-bit quantisation (numpy, 64 bits), written from the format."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """codes [R, K] 0..15, scale bytes [R, K/32] of float64 rows (values exactly representable
    in FP32): nearest grid value, ties to the even code, block scale 2^(floor(log2 amax) - 2)."""
    R, K = x.shape
    v = x.reshape(R, K // 32, 32)
    a = np.abs(v)
    bad = ~np.isfinite(a).all(axis=2)
    amax = np.where(bad, 0.0, a.max(axis=2, initial=0.0))
    _, e = np.frexp(amax)                     # amax = m 2^e, m in [0.5, 1)
    byte = np.where(amax > 0, np.clip(e - 1 - 2 + 127, 0, 254), 0)
    s = np.ldexp(1.0, byte - 127)
    q = np.where(bad[..., None], 0.0, a / s[..., None])
    dist = np.abs(q[..., None] - GRID)        # nearest; on a tie the even code of the two
    best = dist.min(axis=-1, keepdims=True)
    cand = dist == best
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])
    code = order[np.argmax(cand[..., order], axis=-1)]
    code = np.where(bad[..., None], 0, code + 8 * np.signbit(v))
    byte = np.where(bad, 255, byte)
    return code.reshape(R, K).astype(np.uint8), byte.astype(np.uint8)


def values(codes, scales):
    """float64 values of codes [..., K] and scale bytes [..., K/32]."""
    v = np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def unpack(b):
    return np.stack([b & 15, b >> 4], axis=-1).reshape(*b.shape[:-1], 2 * b.shape[-1])


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
