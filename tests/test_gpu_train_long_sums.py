"""Long contractions: sums of many products keep FP32's accuracy to within what one part of them may lose, however long
they are, with signs at random and with one sign (where nothing cancels and truncation always goes one way)."""
import pytest
import torch

import train_ref as ref
from test_gpu_train import gen, offsets_of

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
PART = 4096  # products that one accumulator sums


@pytest.fixture(scope="module")
def moe(cuda_ok):
    import moe_expert_layer_fp32_gb300 as m
    return m


def values(g, one_sign, *shape, dtype):
    t = torch.randn(shape, generator=g, device="cuda")
    return (t.abs() if one_sign else t).to(dtype)


def tolerance(depth):
    """Of a part: its steps of sixteen products and the alignment within one, each up to 2^-23 of the running sum,
    which is no larger than the part's end, in 2-norm over the values; then an FP32 addition a part."""
    return ref.sums_tol(min(depth, PART)) + -(-depth // PART) * 2.0 ** -24


def close(got, want, depth):
    err = (got.double() - want).norm() / want.norm()
    assert err <= tolerance(depth) + (ref.EPS2[got.dtype] if got.dtype != F32 else 0), (err, tolerance(depth))


def transposed_product(x, dy):
    out = torch.zeros((x.shape[1], dy.shape[1]), dtype=torch.float64, device="cuda")
    for a in range(0, x.shape[0], 65536):
        out += x[a:a + 65536].double().T @ dy[a:a + 65536].double()
    return out


@pytest.mark.parametrize("one_sign", [False, True])
@pytest.mark.parametrize("K,N", [(256, 520), (136, 64)])
@pytest.mark.parametrize("rows", [4096, 4097, 8192, 16384 - 7, 131072 + 33])
def test_weight_grad(moe, rows, K, N, one_sign):
    g, counts = gen(rows + K), [5, rows, 0, 4160, 1]
    off, E, R = offsets_of(counts), len(counts), sum(counts)
    x, dy = values(g, one_sign, R, K, dtype=BF), values(g, one_sign, R, N, dtype=BF)
    ws = moe.grouped_new_workspace(E, K, N)
    want = torch.stack([transposed_product(x[a:b], dy[a:b]) for a, b in ref.spans(off)])
    for dt in (F32, BF, HF):
        if dt == HF and rows > 16384:
            continue  # (sums past fp16's largest)
        d = moe.grouped_weight_grad(x, dy, off, ws, dtype=dt)
        for e in range(E):
            if counts[e]:
                close(d[e], want[e], counts[e])
        assert not d[2].any()
    was = torch.randn((E, K, N), generator=g, device="cuda")
    d = moe.grouped_weight_grad(x, dy, off, ws, out=was.clone(), accumulate=True)
    assert torch.equal(d, was + moe.grouped_weight_grad(x, dy, off, ws))
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("one_sign", [False, True])
@pytest.mark.parametrize("counts", [[3, 0, 130, 17], [600, 900, 0, 257]], ids=["few", "many"])
@pytest.mark.parametrize("K,N,turn", [(4104, 264, False), (8192, 72, True), (32768, 136, False), (32760, 520, True)])
def test_product(moe, counts, K, N, turn, one_sign):
    g = gen(K + N)
    off, E, R = offsets_of(counts), len(counts), sum(counts)
    x, w = values(g, one_sign, R, K, dtype=BF), values(g, one_sign, *((E, N, K) if turn else (E, K, N)), dtype=BF)
    ws = moe.grouped_new_workspace(E, K, N)
    want = ref.product(x, off, w, turn)
    for dt in (F32, BF):
        y = moe.grouped_product(x, off, w, ws, transposed=turn, dtype=dt)
        close(y, want, K)
    # a row's bits do not depend on the form
    part = torch.cat([x[:2], x[off[2].item():off[2].item() + 9]])
    y = moe.grouped_product(x, off, w, ws, transposed=turn, dtype=F32)
    few = moe.grouped_product(part, offsets_of([2, 0, 9, 0] if counts[2] else [2, 0, 0, 9]), w, ws, transposed=turn, dtype=F32)
    assert torch.equal(few, torch.cat([y[:2], y[off[2].item():off[2].item() + 9]]))
    assert moe.moe_read_device_status(ws) == 0


def test_waits_that_run_out(moe):
    g, K, N = gen(3), 520, 392
    off = offsets_of([9000, 0, 13000])
    x, dy = values(g, False, 22000, K, dtype=BF), values(g, False, 22000, N, dtype=BF)
    ws = moe.grouped_new_workspace(3, K, N)
    want = moe.grouped_weight_grad(x, dy, off, ws)
    seen = []
    for i in range(40):
        try:
            moe.moe_set_wait_limit(16 + 500 * i)
            moe.grouped_weight_grad(x, dy, off, ws)
            seen.append(moe.moe_read_device_status(ws))
        finally:
            moe.moe_set_wait_limit(0)
        assert torch.equal(moe.grouped_weight_grad(x, dy, off, ws), want)
        assert moe.moe_read_device_status(ws) == 0
    assert 6 in seen and set(seen) <= {0, 6}, seen
