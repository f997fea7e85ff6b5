"""Microscaled 4-bit quantisation, weight packing, the grouped experts' product and the layer
that runs them (moe_mx4_*) against plain 64-bit references.

The quantisation divides by powers of two and rounds once: bit-exact.  In the product every
term is exact; FP32 accumulation adds 64 terms a step, so with u = 2^-24 and each step's
rounding at most two u of the running sum (a truncating adder), an element is within
(K / 64 + 4) 2 u of the sum of its terms' magnitudes, plus half a step of the output type."""
import numpy as np
import pytest
import torch

import mx4_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def moe(cuda_ok):
    import moe_expert_layer_fp32_gb300 as m
    return m


def rows(R, K, seed, dtype, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((R, K), generator=g) * torch.exp(spread * torch.randn((R, 1), generator=g))
    return x.to(DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("R,K", [(1, 32), (3, 96), (64, 2048), (1000, 160), (17, 4096), (2, 128)])
def test_quantize(moe, R, K, dtype):
    x = rows(R, K, R + K, dtype)
    codes, scales, values = moe.mx4_quantize(x.cuda(), want_values=True)
    c0, s0 = ref.quantize(x.double().numpy())
    np.testing.assert_array_equal(scales.cpu().numpy(), s0)
    np.testing.assert_array_equal(codes.cpu().numpy(), ref.pack(c0))
    np.testing.assert_array_equal(values.double().cpu().numpy(), ref.values(c0, s0))
    c2, s2 = moe.mx4_quantize(x.cuda())
    assert torch.equal(c2, codes) and torch.equal(s2, scales)


def test_quantize_special_blocks(moe):
    """Zeros, signed zeros, ties, the format's ends, subnormals, infinities and NaN."""
    lo, hi = float(np.finfo(np.float32).smallest_subnormal), float(np.finfo(np.float32).max)
    x = np.zeros((12, 32), np.float32)
    x[1] = -0.0
    x[2, :16] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -7.0]
    x[3] = np.float32(hi)
    x[4, 0], x[4, 1] = lo, -lo
    x[5, 0] = 2.0 ** -126
    x[6, 0] = 2.0 ** -125 * 1.75
    x[7, 3] = np.inf
    x[8, 31] = -np.inf
    x[9, 7] = np.nan
    x[10] = np.linspace(-8, 8, 32)
    x[11, 0] = 7.999999
    codes, scales, values = moe.mx4_quantize(torch.from_numpy(x).cuda(), want_values=True)
    c0, s0 = ref.quantize(x.astype(np.float64))
    np.testing.assert_array_equal(scales.cpu().numpy(), s0)
    np.testing.assert_array_equal(codes.cpu().numpy(), ref.pack(c0))
    got = values.double().cpu().numpy()
    np.testing.assert_array_equal(got, ref.values(c0, s0))
    assert np.isnan(got[7:10]).all() and (got[0:2] == 0).all()
    assert got[2, 0] == 0 and got[2, 1] == 1 and got[2, 6] == 4 and got[2, 7] == 6


def test_quantize_strides_outputs_and_empty(moe):
    x = rows(9, 256, 5, "bf16").cuda()
    v = x[:, 64:192]                       # 16-byte aligned rows, 256 apart
    a, b = moe.mx4_quantize(v, want_values=True), moe.mx4_quantize(v.contiguous(), want_values=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    vals = torch.empty((9, 128), dtype=torch.bfloat16, device="cuda")
    moe.moe_mx4_quantize(v, moe.MOE_DTYPE_BF16, 256, 9, 128, None, None, vals)
    assert torch.equal(vals, a[2])
    c, s = moe.mx4_quantize(torch.empty((0, 64), device="cuda"))
    assert c.shape == (0, 32) and s.shape == (0, 2)


def test_quantize_past_32_bits(moe):
    """More than 2^31 elements: the last rows are quantised as they are alone."""
    R, K = 1_100_000, 2048
    x = torch.empty((R, K), dtype=torch.bfloat16, device="cuda")
    tile = torch.randn((1000, K), device="cuda").to(torch.bfloat16)
    for r in range(0, R, 1000):
        x[r:r + 1000].copy_(tile)
    x[-7:] = torch.randn((7, K), device="cuda").to(torch.bfloat16) * 3
    codes, scales, values = moe.mx4_quantize(x, want_values=True)
    c, s, v = moe.mx4_quantize(x[-1000:], want_values=True)
    assert torch.equal(codes[-1000:], c) and torch.equal(scales[-1000:], s)
    assert torch.equal(values[-1000:], v)


def weights(E, K, N, seed):
    """(codes [E, N, K/2], scales [E, N, K/32], values [E, N, K]) with scales over 2^-10 .. 2^4."""
    g = np.random.default_rng(seed)
    codes = g.integers(0, 16, (E, N, K), dtype=np.uint8)
    scales = g.integers(117, 132, (E, N, K // 32), dtype=np.uint8)
    return ref.pack(codes), scales, ref.values(codes, scales)


def product_ref(x, off, w):
    c, s = ref.quantize(x.double().numpy())
    xq = ref.values(c, s)
    y = np.zeros((x.shape[0], w.shape[1]))
    mag = np.zeros_like(y)
    for e in range(w.shape[0]):
        r = slice(off[e], off[e + 1])
        y[r] = xq[r] @ w[e].T
        mag[r] = np.abs(xq[r]) @ np.abs(w[e]).T
    return y, mag


def check_product(moe, counts, K, N, x_dtype, y_dtype, seed=0):
    E, R = len(counts), int(sum(counts))
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    codes, scales, wv = weights(E, K, N, seed)
    x = rows(R, K, seed + 1, x_dtype)
    packed = moe.mx4_pack(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    ws = moe.mx4_new_workspace(R, K, N, E)
    ws[256:].fill_(255)                    # stale scratch: NaN scales in every padding row
    y = moe.mx4_expert_product(x.cuda(), torch.from_numpy(off).cuda(), packed, N, ws, DT[y_dtype])
    assert moe.moe_read_device_status(ws) == 0
    y0, mag = product_ref(x, off, wv)
    tol = (K / 64 + 4) * 2 * U * mag
    if y_dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(y0) + tol)
    got = y.double().cpu().numpy()
    nan = np.isnan(y0)                     # rows with a block beyond the type's range
    np.testing.assert_array_equal(np.isnan(got), nan)
    err, tol = np.abs(got - y0)[~nan], tol[~nan]
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())
    return x, off, packed, ws, y


@pytest.mark.parametrize("x_dtype,y_dtype", [("bf16", "f32"), ("f16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("counts,K,N", [
    ([1], 128, 128), ([0, 3, 0], 256, 256), ([16, 17, 15, 1, 0, 33], 384, 128),
    ([224], 512, 256), ([225, 223], 256, 128), ([128, 129, 127], 640, 128), ([449, 1, 448], 256, 384),
    ([1] * 37, 1024, 256), ([0] * 30 + [700] + [0] * 5, 128, 256), ([5, 90, 2, 61], 2048, 512),
    ([128], 2048, 384), ([97, 0, 31], 640, 128), ([48, 49, 0, 7], 256, 1152), ([129], 2048, 256)])
def test_product(moe, counts, K, N, x_dtype, y_dtype):
    check_product(moe, counts, K, N, x_dtype, y_dtype, seed=len(counts) + K)


@pytest.mark.parametrize("x_dtype,y_dtype", [("bf16", "f32"), ("f16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("counts,K,N", [
    ([1], 2176, 128), ([0, 3, 0], 2304, 256), ([16, 17, 15, 1, 0, 33], 2432, 128), ([300, 0, 225], 2176, 384),
    ([1] * 37, 4096, 256)])
def test_product_long_rows(moe, counts, K, N, x_dtype, y_dtype):
    """K past 2048: the rows' codes go through memory; single CTAs and pairs."""
    check_product(moe, counts, K, N, x_dtype, y_dtype, seed=len(counts) + K)


@pytest.mark.parametrize("x_dtype,y_dtype", [("bf16", "bf16"), ("f16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("counts,K,N", [
    ([9728], 128, 128), ([5000, 0, 1, 4900, 223, 7000], 256, 384), ([100] * 130, 128, 256),
    ([15000, 2, 0, 300], 384, 128)])
def test_product_many_rows(moe, counts, K, N, x_dtype, y_dtype):
    """From 9728 rows on the tiles are quantised and multiplied chunk by chunk."""
    check_product(moe, counts, K, N, x_dtype, y_dtype, seed=len(counts) + K)


def test_product_many_rows_again(moe):
    """Calls that follow one another at once, on one workspace, of many chunks each."""
    E, K, N, R = 64, 512, 256, 40000
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda").to(torch.uint8)
    scales = torch.randint(118, 124, (E, N, K // 32), generator=g, device="cuda").to(torch.uint8)
    packed = moe.mx4_pack(codes, scales)
    ws = moe.mx4_new_workspace(R, K, N, E)
    xs = [torch.randn((R, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]
    cut = [torch.sort(torch.randint(0, R + 1, (E - 1,), generator=g, device="cuda")).values for _ in xs]
    offs = [torch.cat([c.new_zeros(1), c, c.new_full((1,), R)]).int() for c in cut]
    want = []
    for x, o in zip(xs, offs):
        want.append(moe.mx4_expert_product(x, o, packed, N, ws, torch.float32))
        torch.cuda.synchronize()
    for _ in range(3):
        got = [moe.mx4_expert_product(x, o, packed, N, ws, torch.float32) for x, o in zip(xs, offs)]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # a few rows of it by themselves (another form of the product) are the same bits
    o = offs[0].cpu()
    e = int(torch.argmax(o[1:] - o[:-1]))
    r = slice(int(o[e]), int(o[e]) + 150)
    o1 = torch.tensor([0] * (e + 1) + [150] * (E - e), dtype=torch.int32, device="cuda")
    y = moe.mx4_expert_product(xs[0][r].contiguous(), o1, packed, N, ws, torch.float32)
    assert torch.equal(y, want[0][r])


def test_product_many_experts_and_tiles(moe):
    g = np.random.default_rng(4)
    check_product(moe, g.integers(0, 40, 256).tolist(), 256, 128, "bf16", "f32")
    check_product(moe, [3000, 0, 1111], 128, 1024, "bf16", "bf16")


def test_product_row_alone(moe):
    """A row's result is the same bits whatever else is in the batch."""
    x, off, packed, ws, y = check_product(moe, [300, 7, 0, 130], 512, 256, "bf16", "f32")
    E = 4
    for r in (0, 299, 303, 307, 436):
        e = int(np.searchsorted(off, r, side="right")) - 1
        o = torch.tensor([0] * (e + 1) + [1] * (E - e), dtype=torch.int32, device="cuda")
        ws1 = moe.mx4_new_workspace(1, 512, 256, E)
        y1 = moe.mx4_expert_product(x[r:r + 1].cuda(), o, packed, 256, ws1, torch.float32)
        assert torch.equal(y1[0], y[r])


def test_product_past_32_bits(moe):
    """An output of more than 2^31 elements: the last expert's rows are those they are alone."""
    R, K, N, E = 540_000, 128, 4096, 5
    codes, scales, _ = weights(E, K, N, 6)
    packed = moe.mx4_pack(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    x = torch.randn((R, K), device="cuda").to(torch.bfloat16)
    off = torch.tensor([0, 130_000, 400_001, 400_001, R - 500, R], dtype=torch.int32, device="cuda")
    ws = moe.mx4_new_workspace(R, K, N, E)
    y = moe.mx4_expert_product(x, off, packed, N, ws)
    assert moe.moe_read_device_status(ws) == 0
    for e, a, b in ((4, R - 500, R), (3, R - 700, R - 500), (0, 0, 100)):
        o = torch.tensor([0] * (e + 1) + [b - a] * (E - e), dtype=torch.int32, device="cuda")
        assert torch.equal(moe.mx4_expert_product(x[a:b], o, packed, N, ws), y[a:b])


def test_product_nan_stays_in_its_row(moe):
    K, N, E = 256, 128, 2
    codes, scales, wv = weights(E, K, N, 9)
    packed = moe.mx4_pack(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    x = rows(40, K, 3, "bf16")
    bad = x.clone()
    bad[5, 17], bad[21, 200], bad[39, 0] = float("nan"), float("inf"), float("-inf")
    off = torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda")
    ws = moe.mx4_new_workspace(40, K, N, E)
    y = moe.mx4_expert_product(x.cuda(), off, packed, N, ws, torch.float32)
    z = moe.mx4_expert_product(bad.cuda(), off, packed, N, ws, torch.float32)
    keep = [r for r in range(40) if r not in (5, 21, 39)]
    assert torch.equal(z[keep], y[keep]) and torch.isnan(z[[5, 21, 39]]).all()


def test_bad_offsets_are_flagged(moe):
    K, N, E, R = 128, 128, 3, 50
    codes, scales, _ = weights(E, K, N, 2)
    packed = moe.mx4_pack(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    x = rows(R, K, 3, "bf16").cuda()
    ws = moe.mx4_new_workspace(R, K, N, E)
    for off in ([0, 20, 10, 50], [1, 20, 30, 50], [0, 20, 30, 49], [0, 20, 60, 50], [0, -4, 30, 50]):
        y = torch.full((R, N), 7.0, device="cuda")
        moe.moe_mx4_expert_product(x, moe.MOE_DTYPE_BF16,
                                   torch.tensor(off, dtype=torch.int32, device="cuda"), packed, R, K,
                                   N, E, y, moe.MOE_DTYPE_F32, ws)
        assert moe.STATUS[moe.moe_read_device_status(ws)] == "MOE_ERR_DEVICE_CHECK"
        assert (y == 7.0).all()
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("R,K", [(512, 256), (64, 512)])
def test_wait_timeout_is_reported_and_context_survives(moe, R, K):
    """The products' bounded waits run out under a limit far below a copy's round trip: the call
    reports it, and the next one is right.  (N = 128: single CTAs.)"""
    E, N = 4, 128
    codes, scales, _ = weights(E, K, N, 5)
    packed = moe.mx4_pack(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    x = rows(R, K, 1, "bf16").cuda()
    off = torch.tensor([0, 7, 7, R - 9, R], dtype=torch.int32, device="cuda")
    ws = moe.mx4_new_workspace(R, K, N, E)
    want = moe.mx4_expert_product(x, off, packed, N, ws)
    assert moe.moe_read_device_status(ws) == 0
    statuses = []
    try:
        moe.moe_set_wait_limit(16)
        for _ in range(3):
            moe.mx4_expert_product(x, off, packed, N, ws)
            statuses.append(moe.moe_read_device_status(ws))
    finally:
        moe.moe_set_wait_limit(0)
    assert 6 in statuses and set(statuses) <= {0, 6}, statuses
    assert torch.equal(moe.mx4_expert_product(x, off, packed, N, ws), want)
    assert moe.moe_read_device_status(ws) == 0


def test_prepack_is_quantize_and_pack(moe):
    E, K, N = 3, 384, 256
    g = torch.Generator().manual_seed(8)
    w = (torch.randn((E, K, N), generator=g) * 0.02).to(torch.bfloat16).cuda()
    w2 = (torch.randn((E, K, 128), generator=g) * 0.5).to(torch.bfloat16).cuda()
    both = torch.cat([w, w2], dim=2)
    kt = both.transpose(1, 2).contiguous().view(-1, K)
    codes, scales = moe.mx4_quantize(kt)
    want = moe.mx4_pack(codes.view(E, N + 128, K // 2), scales.view(E, N + 128, K // 32))
    assert torch.equal(moe.mx4_prepack(w, w2), want)
    assert torch.equal(moe.mx4_prepack(both), want)


def test_both_ways_of_calling(moe):
    """The native fast path and the Python path (a workspace of another type, rows of a wider
    tensor) are one call, on the current stream and on one that is given."""
    K, N, E, R = 256, 128, 3, 70
    codes, scales, _ = weights(E, K, N, 2)
    packed = moe.mx4_pack(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    off = torch.tensor([0, 30, 30, R], dtype=torch.int32, device="cuda")
    ws = moe.mx4_new_workspace(R, K, N, E)
    side = torch.cuda.Stream()
    for dt in ("bf16", "f16", "f32"):
        wide = rows(R, K + 64, 3, dt, spread=1.0).cuda()
        v = wide[:, :K]
        x = v.contiguous()
        side.wait_stream(torch.cuda.current_stream())
        for out in (torch.bfloat16, torch.float32):
            a = moe.mx4_expert_product(x, off, packed, N, ws, out)
            for w, s in ((ws.view(torch.int32), None), (ws, side), (ws.view(torch.int32), side.cuda_stream)):
                torch.cuda.synchronize()  # one workspace
                b = moe.mx4_expert_product(x, off, packed, N, w, out, stream=s)
                torch.cuda.synchronize()
                assert a.dtype == b.dtype == out and torch.equal(a, b)
        for want in (False, True):
            q = [moe.mx4_quantize(t, want, stream=s) for t, s in ((x, None), (v, None), (x, side), (v, side))]
            torch.cuda.synchronize()
            assert all(len(c) == 2 + want and all(torch.equal(a, b) for a, b in zip(q[0], c)) for c in q)
    for s in (None, side):
        with pytest.raises(moe.MoEError):      # K not a multiple of 32
            moe.mx4_quantize(x[:, :40].contiguous(), stream=s)
        with pytest.raises(moe.MoEError):      # a workspace too small
            moe.mx4_expert_product(x, off, packed, N, ws[:256], stream=s)
    with pytest.raises(ValueError, match="packed"):
        moe.mx4_expert_product(x, off, packed[256:], N, ws)
    with pytest.raises(TypeError, match="y:"):
        moe.mx4_expert_product(x, off, packed, N, ws, torch.float16)


def test_stream_and_graph(moe):
    K, N, E, R = 512, 256, 4, 100
    codes, scales, _ = weights(E, K, N, 2)
    packed = moe.mx4_pack(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    x = rows(R, K, 3, "bf16").cuda()
    off = torch.tensor([0, 10, 10, 70, 100], dtype=torch.int32, device="cuda")
    ws = moe.mx4_new_workspace(R, K, N, E)
    want = moe.mx4_expert_product(x, off, packed, N, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = moe.mx4_expert_product(x, off, packed, N, ws)
        q = moe.mx4_quantize(x)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and torch.equal(q[0], moe.mx4_quantize(x)[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = moe.mx4_expert_product(x, off, packed, N, ws)
    x.copy_(rows(R, K, 4, "bf16"))
    off.copy_(torch.tensor([0, 50, 60, 60, 100], dtype=torch.int32))
    graph.replay()
    assert torch.equal(got, moe.mx4_expert_product(x, off, packed, N, ws))


@pytest.mark.parametrize("T,H,E,k,I,kind,groups,keep,top", [
    (1, 256, 8, 2, 128, 0, 1, 1, 1), (37, 384, 16, 4, 256, 1, 4, 2, 2), (300, 512, 32, 8, 384, 1, 8, 4, 2),
    (1300, 512, 32, 8, 256, 1, 8, 4, 2), (40, 2304, 8, 2, 128, 0, 1, 1, 1)])
def test_layer(moe, T, H, E, k, I, kind, groups, keep, top):
    """The layer is its parts: the logits' selection, the products of the gathered rows, the
    SwiGLU rows quantised, the weighted sum.  Its SiLU uses the special-function unit, a few
    FP32 steps from torch's, so a 4-bit rounding of the hidden rows may fall the other way for
    a few values in 10^5: the layer tolerance (rel-L2 5e-3) holds them."""
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    wr = (torch.randn((H, E), generator=g) * 0.05).cuda()
    b = (torch.randn(E, generator=g) * 0.02).cuda()
    wg, wu = ((torch.randn((E, H, I), generator=g) * 0.05).to(torch.bfloat16).cuda() for _ in "gu")
    wd = (torch.randn((E, I, H), generator=g) * 0.05).to(torch.bfloat16).cuda()
    d = moe.dims(T, H, E, k, I)
    gu, dn = moe.mx4_prepack(wg, wu), moe.mx4_prepack(wd)
    o = moe.select_opts(kind, groups, keep, top)
    ws = moe.mx4_new_layer_workspace(d)
    out, idx, w, counts = moe.mx4_layer_forward(x, wr, b, gu, dn, d, ws, o, route_scale=2.5,
                                                want_routing=True)
    assert moe.moe_read_device_status(ws) == 0
    logits = torch.empty((T, E), device="cuda")
    moe.moe_router_logits(x, wr, None, d, logits)
    i2, w2 = moe.route_select(logits, k, o, bias=b)
    assert torch.equal(idx, i2) and torch.equal(w, w2)
    order = torch.argsort(idx.flatten().long(), stable=True)
    cnt = torch.bincount(idx.flatten().long(), minlength=E)
    assert torch.equal(counts.long(), cnt)
    off = torch.cat([cnt.new_zeros(1), cnt.cumsum(0)]).int()
    R = T * k
    h = moe.mx4_expert_product(x[order // k], off, gu, 2 * I, moe.mx4_new_workspace(R, H, 2 * I, E))
    h = torch.nn.functional.silu(h[:, :I].float()) * h[:, I:].float()
    y = moe.mx4_expert_product(h, off, dn, H, moe.mx4_new_workspace(R, I, H, E), torch.float32)
    back = torch.empty_like(y)
    back[order] = y
    want = (back.view(T, k, H).double() * (2.5 * w.double()).unsqueeze(2)).sum(1)
    rel = (out.double() - want).norm() / want.norm()
    assert rel <= 5e-3, rel
    out2 = moe.mx4_layer_forward(x, wr, b, gu, dn, d, ws, o, route_scale=2.5)
    assert torch.equal(out2, out)
