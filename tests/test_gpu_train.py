"""The operators that train the experts, against plain 64-bit forms: ragged and empty experts, odd sizes, strides,
types, both forms of the kernels, captured and repeated calls, other streams."""
import pytest
import torch

import train_ref as ref

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def moe(cuda_ok):
    import moe_expert_layer_fp32_gb300 as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def offsets_of(counts):
    return torch.tensor([0] + list(counts)).cumsum(0).int().cuda()


# experts without rows first, between and last; one row; tile borders on either side; many rows (the pair form)
FEW = [0, 1, 16, 17, 0, 127, 128, 129, 3, 0]
MANY = [0, 255, 256, 257, 700, 0, 1, 1024, 33, 0]
SIZES = [(8, 8), (64, 128), (72, 136), (200, 264), (1000, 520), (2048, 256)]


@pytest.mark.parametrize("counts", [FEW, MANY, [1], [0, 0], [300]], ids=["few", "many", "one", "none", "alone"])
@pytest.mark.parametrize("K,N", SIZES)
@pytest.mark.parametrize("turn", [False, True])
def test_product(moe, counts, K, N, turn):
    g, off, E, R = gen(K + N + len(counts)), offsets_of(counts), len(counts), sum(counts)
    ws = moe.grouped_new_workspace(E, K, N)
    for xt, yt in ((BF, BF), (HF, F32), (BF, F32), (HF, HF)):
        x = normal(g, R, K, dtype=xt)
        w = normal(g, *((E, N, K) if turn else (E, K, N)), dtype=xt, std=0.05)
        y = moe.grouped_product(x, off, w, ws, transposed=turn, dtype=yt)
        assert y.dtype == yt and y.shape == (R, N)
        if R:
            size = ref.product(x.abs(), off, w.abs(), turn)
            ref.close(y, ref.product(x, off, w, turn), K, size)
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("counts", [FEW, MANY, [1], [0, 0], [300]], ids=["few", "many", "one", "none", "alone"])
@pytest.mark.parametrize("K,N", SIZES)
def test_weight_grad(moe, counts, K, N):
    g, off, E, R = gen(K + N + len(counts)), offsets_of(counts), len(counts), sum(counts)
    ws = moe.grouped_new_workspace(E, K, N)
    most = max(counts)
    for xt, yt in ((BF, F32), (HF, HF), (BF, BF), (HF, F32)):
        x, dy = normal(g, R, K, dtype=xt), normal(g, R, N, dtype=xt, std=0.01)
        d = moe.grouped_weight_grad(x, dy, off, ws, dtype=yt)
        assert d.dtype == yt and d.shape == (E, K, N)
        for e, (a, b) in enumerate(ref.spans(off)):
            if a == b:
                assert not d[e].any()
        ref.close(d, ref.weight_grad(x, dy, off), most, ref.weight_grad(x.abs(), dy.abs(), off))
    # added to what is there; experts without rows keep their bits, NaN among them
    d = normal(g, E, K, N)
    empty = [e for e, (a, b) in enumerate(ref.spans(off)) if a == b]
    for e in empty:
        d[e, 0, 0] = float("nan")
    was = d.clone()
    r = moe.grouped_weight_grad(x, dy, off, ws, out=d, accumulate=True)
    assert r is d
    full = [e for e in range(E) if e not in empty]
    for e in empty:
        assert torch.equal(d[e].view(torch.int32), was[e].view(torch.int32))
    if full:
        want = ref.weight_grad(x, dy, off)
        size = ref.weight_grad(x.abs(), dy.abs(), off) + was.double().abs()
        ref.close(d[full], (want + was.double())[full], most, size[full])
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("counts", [FEW, MANY], ids=["few", "many"])
def test_other_experts_rows_stay_out(moe, counts):
    """Infinities and NaN in one expert's rows, and behind the last row, reach no other expert."""
    g, K, N, E, R = gen(5), 136, 264, len(counts), sum(counts)
    off = offsets_of(counts)
    ws = moe.grouped_new_workspace(E, K, N)
    x, dy, w = normal(g, R + 64, K, dtype=BF), normal(g, R + 64, N, dtype=BF), normal(g, E, K, N, dtype=BF)
    bad = max(range(E), key=lambda e: counts[e])
    clean = [moe.grouped_product(x[:R], off, w, ws), moe.grouped_weight_grad(x[:R], dy[:R], off, ws)]
    a, b = ref.spans(off)[bad]
    for t in (x, dy):
        t[R:] = float("nan")
        t[a:b] = float("inf")
    y = moe.grouped_product(x[:R], off, w, ws)
    d = moe.grouped_weight_grad(x[:R], dy[:R], off, ws)
    keep = [e for e in range(E) if e != bad]
    assert torch.equal(d[keep], clean[1][keep]) and not torch.isfinite(d[bad]).any()
    for e in keep:
        s, t = ref.spans(off)[e]
        assert torch.equal(y[s:t], clean[0][s:t])


@pytest.mark.parametrize("counts", [FEW, MANY], ids=["few", "many"])
def test_strided_operands_and_outputs(moe, counts):
    """Column slices of wider tensors in and out; what lies beside them keeps its bits."""
    g, K, N, E, R = gen(7), 72, 136, len(counts), sum(counts)
    off = offsets_of(counts)
    ws = moe.grouped_new_workspace(E, K, N)
    x, dy = normal(g, R, 2 * K, dtype=BF)[:, K:], normal(g, R, 3 * N, dtype=BF)[:, N:2 * N]
    w = normal(g, E, K, 2 * N, dtype=BF)[:, :, N:]
    y = torch.full((R, 2 * N + 8), 7.0, device="cuda", dtype=BF)
    moe.grouped_product(x, off, w, ws, out=y[:, N:2 * N])
    assert torch.equal(y[:, N:2 * N], moe.grouped_product(x.contiguous(), off, w.contiguous(), ws))
    assert (y[:, :N] == 7).all() and (y[:, 2 * N:] == 7).all()
    d = torch.full((E, K, 2 * N), 7.0, device="cuda")
    moe.grouped_weight_grad(x, dy, off, ws, out=d[:, :, N:])
    assert torch.equal(d[:, :, N:], moe.grouped_weight_grad(x.contiguous(), dy.contiguous(), off, ws))
    assert (d[:, :, :N] == 7).all()
    wt = normal(g, E, 2 * N, K, dtype=BF)[:, N:]
    assert torch.equal(moe.grouped_product(x, off, wt, ws, transposed=True),
                       moe.grouped_product(x, off, wt.contiguous(), ws, transposed=True))


def test_rows_do_not_depend_on_the_others(moe):
    """The same rows and matrices among few and many rows (both forms of the kernel): the same bits."""
    g, K, N = gen(9), 520, 392
    w, x = normal(g, 3, K, N, dtype=BF), normal(g, 3000, K, dtype=BF)
    ws = moe.grouped_new_workspace(3, K, N)
    whole = moe.grouped_product(x, offsets_of([1000, 900, 1100]), w, ws, dtype=F32)
    part = torch.cat([x[:5], x[1000:1007], x[1900:1950]])
    y = moe.grouped_product(part, offsets_of([5, 7, 50]), w, ws, dtype=F32)
    assert torch.equal(y, torch.cat([whole[:5], whole[1000:1007], whole[1900:1950]]))


def test_256_experts(moe):
    """As many experts as there may be, most of them with a row or two or none, one with many."""
    g, K, N, E = gen(13), 72, 200, 256
    counts = [(7 * e) % 3 for e in range(E)]
    counts[200] = 900
    off, R = offsets_of(counts), sum(counts)
    ws = moe.grouped_new_workspace(E, K, N)
    x, dy, w = normal(g, R, K, dtype=BF), normal(g, R, N, dtype=BF), normal(g, E, K, N, dtype=BF)
    ref.close(moe.grouped_product(x, off, w, ws, dtype=F32), ref.product(x, off, w), K, ref.product(x.abs(), off, w.abs()))
    d = moe.grouped_weight_grad(x, dy, off, ws)
    ref.close(d, ref.weight_grad(x, dy, off), 900, ref.weight_grad(x.abs(), dy.abs(), off))
    assert all(not d[e].any() for e in range(E) if counts[e] == 0)
    assert moe.moe_read_device_status(ws) == 0


def test_bad_offsets_are_flagged(moe):
    g, K, N, R = gen(11), 64, 128, 40
    x, dy, w = normal(g, R, K, dtype=BF), normal(g, R, N, dtype=BF), normal(g, 3, K, N, dtype=BF)
    ws = moe.grouped_new_workspace(3, K, N)
    for off in ([0, 10, 5, 40], [0, 10, 20, 41], [1, 10, 20, 40], [0, 10, 20, 39], [0, 50, 20, 40], [0, -5, 20, 40],
                [0, 2 ** 31 - 1, 2 ** 31 - 1, 40], [-2 ** 31, 0, 0, 40]):
        off = torch.tensor(off).int().cuda()
        y = torch.full((R, N), 7.0, device="cuda", dtype=BF)
        d = torch.full((3, K, N), 7.0, device="cuda")
        moe.grouped_product(x, off, w, ws, out=y)
        assert moe.moe_read_device_status(ws) == 7 and (y == 7).all()
        moe.grouped_weight_grad(x, dy, off, ws, out=d)
        assert moe.moe_read_device_status(ws) == 7 and (d == 7).all()
    moe.grouped_product(x, offsets_of([10, 10, 20]), w, ws, out=y)
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("R,I", [(1, 8), (3, 72), (257, 768), (40, 1024), (5000, 264), (2, 16384)])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("weighted", [True, False])
def test_swiglu(moe, R, I, dt, weighted):
    g = gen(R + I)
    gu, d = normal(g, R, 2 * I, dtype=dt, std=2.0), normal(g, R, I, dtype=dt, std=0.1)
    w = torch.rand(R, generator=g, device="cuda") if weighted else None
    gu[0, 0], gu[-1, 1] = 60.0, -60.0
    dgu, h, dw = ref.swiglu_backward(gu, d, w)
    got = moe.swiglu_backward(gu, d, w)
    fwd = moe.swiglu(gu, w)
    half = ref.EPS2[dt]
    least = 2.0 ** -25 if dt == HF else 0.0
    # sigmoid by the special-function unit: the exponential's argument rounds at 2^-24 |g| log2 e, and it, the sum
    # and the reciprocal have a few units of 2^-23 each
    gg, u = gu[:, :I].double(), gu[:, I:].double()
    rel = 2.0 ** -23 * (8 + 2 * gg.abs())
    wd = d.double().abs() * (w.double().unsqueeze(1) if weighted else 1.0)
    size = torch.cat([wd * u.abs() * (1 + gg.abs()), wd * gg.abs()], 1) * torch.cat([rel, rel], 1)
    # (one minus a sigmoid that is near one has the sigmoid's absolute error)
    assert ((got[0].double() - dgu).abs() <= half * dgu.abs() + size + least).all()
    for v in (got[1], fwd):
        assert ((v.double() - h).abs() <= half * h.abs() + rel * h.abs() + least).all()
    assert torch.equal(got[1], fwd)
    if weighted:
        mag = (d.double() * ref.swiglu(gu)).abs()
        assert ((got[2].double() - dw).abs() <= (mag * (rel + (I / 32 + 8) * 2.0 ** -24)).sum(1)).all()


def test_swiglu_strides(moe):
    g = gen(3)
    gu, d = normal(g, 50, 400, dtype=BF)[:, 8:280], normal(g, 50, 200, dtype=BF)[:, 64:200]
    w = torch.rand(50, generator=g, device="cuda")
    a, b = moe.swiglu_backward(gu, d, w), moe.swiglu_backward(gu.contiguous(), d.contiguous(), w)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert torch.equal(moe.swiglu(gu, w), moe.swiglu(gu.contiguous(), w))


def updates(g, E, rows, cols, dtype, low=None):
    """Matrices whose singular values fall by a factor of a hundred, of different sizes."""
    k = min(rows, cols)
    u = torch.linalg.qr(torch.randn((E, rows, k), generator=g, device="cuda")).Q
    v = torch.linalg.qr(torch.randn((E, cols, k), generator=g, device="cuda")).Q
    s = torch.logspace(0, -2, k, device="cuda")
    if low is not None:
        s[low:] = 0
    m = (u * s) @ v.transpose(1, 2) * torch.logspace(-4, 4, E, device="cuda")[:, None, None]
    return m.to(dtype)


@pytest.mark.parametrize("E,rows,cols", [(1, 1, 1), (2, 1, 9), (2, 9, 1), (3, 8, 8), (2, 33, 65), (2, 65, 33), (3, 128, 128),
                                         (2, 128, 256), (2, 129, 200), (2, 200, 129), (2, 256, 512), (2, 511, 513),
                                         (1, 1000, 700), (40, 40, 24), (2, 1, 1000), (2, 1000, 1), (2, 5, 300),
                                         (1, 3000, 40), (256, 9, 300), (1, 257, 257)])
@pytest.mark.parametrize("dt,out", [(F32, BF), (BF, BF), (HF, HF)])
def test_orthogonalize(moe, E, rows, cols, dt, out):
    m = updates(gen(rows + cols), E, rows, cols, dt)
    ws = moe.orthogonalize_new_workspace(E, rows, cols)
    for steps in (1, 2, 5):
        x = moe.orthogonalize(m, ws, steps=steps, dtype=out)
        want, tol = ref.orthogonalize(m, steps=steps)
        err = (x.double() - want).square().sum((1, 2)).sqrt() / want.square().sum((1, 2)).sqrt()
        assert torch.isfinite(x).all() and (err <= tol + ref.EPS2[out]).all(), (err, tol)
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("E,rows,cols,rank", [(2, 300, 500, 8), (2, 500, 300, 8), (1, 128, 700, 3), (2, 260, 520, 64)])
@pytest.mark.parametrize("dt", [F32, BF])
def test_orthogonalize_of_low_rank(moe, E, rows, cols, rank, dt):
    """A few rows' gradients: what rounding leaves outside their span is not lifted step by step.  The first three
    iterates count with 22 bits in a X, so a rounding of 2^-12 (of X, A and B) is lifted by two steps at most."""
    g = gen(rank)
    u, v = normal(g, E, rows, rank), normal(g, E, rank, cols)
    m = (u @ v).to(dt)  # (BF16: of full rank again, by its rounding, which belongs to the input)
    ws = moe.orthogonalize_new_workspace(E, rows, cols)
    x = moe.orthogonalize(m, ws)
    want, _ = ref.orthogonalize(m)
    norm = want.square().sum((1, 2)).sqrt()
    # roundings of X_3 and X_4 lifted twice and once, in 2-norms of at most 1.2 sqrt(rank) + what bf16 noise adds
    tol = 3 * 2.0 ** -12 * (3.4445 ** 2 + 3.4445 + 1) + 2.0 ** -8
    assert ((x.double() - want).square().sum((1, 2)).sqrt() <= tol * norm).all()
    assert moe.moe_read_device_status(ws) == 0


def test_orthogonalize_bad_and_zero_matrices(moe):
    """Zeros stay zeros, an infinity or a NaN stays in its matrix, and sizes up to FP32's ends are no matter."""
    g = gen(1)
    m = updates(g, 7, 130, 70, F32)
    ws = moe.orthogonalize_new_workspace(7, 130, 70)
    m[0] /= m[0].norm()
    for e in range(1, 7):
        m[e] = m[0]
    clean = moe.orthogonalize(m, ws, eps=0.0)
    m[1] = 0
    m[2, 5, 5] = float("inf")
    m[3, 0, 69] = float("nan")
    m[4] *= 1e36
    m[5] *= 1e-30
    x = moe.orthogonalize(m, ws, eps=0.0)
    assert torch.equal(x[0], clean[0]) and torch.equal(x[6], clean[6])
    assert not x[1].any() and torch.isnan(x[2]).all() and torch.isnan(x[3]).all()
    for e in (4, 5):
        want, tol = ref.orthogonalize(m[e:e + 1], eps=0.0)
        assert (x[e].double() - want[0]).norm() <= (tol[0] + 2.0 ** -8) * want.norm()


def test_orthogonalize_strides_scale_in_place(moe):
    g = gen(2)
    wide = updates(g, 3, 70, 200, BF)
    ws = moe.orthogonalize_new_workspace(3, 70, 133)
    m = wide[:, :, 8:141]
    want = moe.orthogonalize(m.contiguous(), ws, scale=0.25)
    assert torch.equal(moe.orthogonalize(m, ws, scale=0.25), want)
    one = moe.orthogonalize(m, ws)
    assert torch.equal(one.float() * 0.25, want.float())
    beside = wide.clone()
    r = moe.orthogonalize(m, ws, scale=0.25, out=m)
    assert r is m and torch.equal(m, want)
    assert torch.equal(wide[:, :, :8], beside[:, :, :8]) and torch.equal(wide[:, :, 141:], beside[:, :, 141:])
    c = (2.0, -1.5, 0.5)
    x = moe.orthogonalize(wide, moe.orthogonalize_new_workspace(3, 70, 200), coefficients=c, steps=3)
    want, tol = ref.orthogonalize(wide, coefficients=c, steps=3)
    assert ((x.double() - want).square().sum((1, 2)).sqrt() <= (tol + 2.0 ** -8) * want.square().sum((1, 2)).sqrt()).all()
