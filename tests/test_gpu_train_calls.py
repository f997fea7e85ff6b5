"""The calls that train the experts as a program makes them: the experts' forward and backward pass end to end, on
other streams, captured and replayed, two at once, through either path of the tensor calls, with waits that run
out, and past 2^31 elements."""
import pytest
import torch

import train_ref as ref
from test_gpu_train import FEW, MANY, gen, normal, offsets_of, updates

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def moe(cuda_ok):
    import moe_expert_layer_fp32_gb300 as m
    return m


def layer64(x, wgu, wd, idx, w):
    """The layer in 64 bits, under autograd: x [T, H], experts' matrices, routing."""
    T, k = idx.shape
    out = torch.zeros_like(x)
    i = wd.shape[1]
    for e in range(wgu.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if t.numel():
            gu = x[t] @ wgu[e]
            h = torch.nn.functional.silu(gu[:, :i]) * gu[:, i:]
            out = out.index_add(0, t, (h @ wd[e]) * w[t, j].unsqueeze(1))
    return out


@pytest.mark.parametrize("T,H,E,k,I", [(256, 128, 8, 2, 256), (1, 256, 8, 3, 128), (700, 384, 16, 4, 128), (33, 128, 64, 2, 128)])
@pytest.mark.parametrize("kept", [True, False])
def test_layer_forward_and_backward(moe, T, H, E, k, I, kept):
    """Router to updated matrices: the layer's own steps around the grouped calls, against autograd in 64 bits."""
    g = gen(T + H)
    x = normal(g, T, H, dtype=BF)
    wgu, wd = normal(g, E, H, 2 * I, dtype=BF, std=0.05), normal(g, E, I, H, dtype=BF, std=0.05)
    logits = normal(g, T, E)
    d_out = normal(g, T, H, dtype=BF, std=0.01)
    d = moe.dims(T, H, E, k, I)
    ws = moe.new_workspace(d)
    idx, w = moe.route_select(logits, k)
    counts, off = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    moe.moe_load_stats(idx, d, counts, off, ws)
    R = T * k

    def rows_of(t):
        p = torch.empty((R, H), dtype=BF, device="cuda")
        ros, sor = (torch.empty(R, dtype=torch.int32, device="cuda") for _ in range(2))
        moe.moe_permute(t, idx, off, d, p, ros, sor, ws)
        return p, ros, sor

    xp, ros, sor = rows_of(x)
    gws = moe.grouped_new_workspace(E, H, 2 * I)
    gate_up = moe.grouped_product(xp, off, wgu, gws)
    y = moe.grouped_product(moe.swiglu(gate_up), off, wd, moe.grouped_new_workspace(E, I, H), dtype=F32)
    out = torch.empty((T, H), dtype=BF, device="cuda")
    moe.moe_combine(y, w, ros, d, out)
    row_w = w.flatten()[sor.long()].contiguous()
    bws = moe.expert_ffn_backward_new_workspace(R, H, I, E)
    dxp, dgu, dd, drw = moe.expert_ffn_backward(xp, off, wgu, wd, rows_of(d_out)[0], bws, row_weights=row_w,
                                                gate_up=gate_up if kept else None, d_x_dtype=F32)
    dx = torch.empty((T, H), dtype=BF, device="cuda")
    moe.moe_combine(dxp, torch.ones_like(w), ros, d, dx)
    d_logits = moe.route_select_backward(logits, idx, drw[ros.long()].view(T, k).contiguous())
    assert moe.moe_read_device_status(bws) == 0 and moe.moe_read_device_status(gws) == 0
    update = moe.orthogonalize(dgu, moe.orthogonalize_new_workspace(E, H, 2 * I))

    x64, wgu64, wd64 = (t.double().requires_grad_(True) for t in (x, wgu, wd))
    l64 = logits.double().requires_grad_(True)
    p = torch.softmax(l64, 1).gather(1, idx.long())
    o64 = layer64(x64, wgu64, wd64, idx, p / p.sum(1, keepdim=True))
    want = torch.autograd.grad(o64, [x64, wgu64, wd64, l64], d_out.double())
    # Each result passes at most five roundings to bf16 on its way (gate and up, the activation or its gradient,
    # the gradient of the product, the rows, the output); a rounding's relative error is at most 2^-8, and the
    # products that follow add errors of independent values no faster than the values themselves.
    for got, exact in ((out, o64), (dx, want[0]), (dgu, want[1]), (dd, want[2]), (d_logits, want[3])):
        err = (got.double() - exact).norm() / exact.norm()
        assert err <= 5 * 2.0 ** -8, err
    for e in (counts == 0).nonzero().flatten().tolist():
        assert not dgu[e].any() and not dd[e].any() and not update[e].any()
    assert torch.isfinite(update).all()


def test_backward_is_its_steps(moe):
    """The one call's outputs are those of its steps, with and without routing weights, and added to what is there."""
    g, H, I = gen(3), 136, 72
    off, E, R = offsets_of(FEW), len(FEW), sum(FEW)
    x, dy = normal(g, R, H, dtype=HF), normal(g, R, H, dtype=HF, std=0.1)
    wgu, wd = normal(g, E, H, 2 * I, dtype=HF, std=0.1), normal(g, E, I, H, dtype=HF, std=0.1)
    ws, bws = moe.grouped_new_workspace(E, H, 2 * I), moe.expert_ffn_backward_new_workspace(R, H, I, E)
    for w in (None, torch.rand(R, generator=g, device="cuda")):
        gu = moe.grouped_product(x, off, wgu, ws)
        s = moe.swiglu_backward(gu, moe.grouped_product(dy, off, wd, ws, transposed=True), w)
        want = [moe.grouped_product(s[0], off, wgu, ws, transposed=True), moe.grouped_weight_grad(x, s[0], off, ws),
                moe.grouped_weight_grad(s[1], dy, off, ws)] + ([] if w is None else [s[2]])
        for kept in (gu, None):
            got = moe.expert_ffn_backward(x, off, wgu, wd, dy, bws, row_weights=w, gate_up=kept)
            assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
    more = moe.expert_ffn_backward(x, off, wgu, wd, dy, bws, row_weights=w, d_w_gate_up=want[1].clone(),
                                   d_w_down=want[2].clone(), accumulate=True)
    assert torch.equal(more[1], 2 * want[1]) and torch.equal(more[2], 2 * want[2])
    empty = moe.expert_ffn_backward(x[:0], off * 0, wgu, wd, dy[:0], bws)
    assert empty[0].shape == (0, H) and not empty[1].any() and not empty[2].any()


def work(moe, seed):
    """One of each call, as (function of its inputs, inputs)."""
    g = gen(seed)
    out = []
    for counts in (FEW, MANY):
        off, E, R, K, N = offsets_of(counts), len(counts), sum(counts), 264, 392
        x, dy = normal(g, R, K, dtype=BF), normal(g, R, N, dtype=BF)
        w = normal(g, E, K, N, dtype=BF)
        ws = moe.grouped_new_workspace(E, K, N)
        out += [(lambda x=x, off=off, w=w, ws=ws: moe.grouped_product(x, off, w, ws)),
                (lambda x=x, dy=dy, off=off, ws=ws: moe.grouped_weight_grad(x, dy, off, ws))]
    gu, d = normal(g, 300, 400, dtype=BF), normal(g, 300, 200, dtype=BF)
    rw = torch.rand(300, generator=g, device="cuda")
    out += [lambda: moe.swiglu_backward(gu, d, rw)[0], lambda: moe.swiglu(gu)]
    for rows, cols, E in ((100, 200, 3), (300, 520, 2), (640, 500, 8)):
        m = updates(g, E, rows, cols, BF)
        ws = moe.orthogonalize_new_workspace(E, rows, cols)
        out.append(lambda m=m, ws=ws: moe.orthogonalize(m, ws))
    return out


def test_streams_graphs_and_repeats(moe):
    """The same bits on another stream, after a replay over new inputs, and while another call of the same kind runs
    with a workspace of its own."""
    one, two = work(moe, 1), work(moe, 2)
    want = [[f() for f in fs] for fs in (one, two)]
    again = [f() for f in one]
    assert all(torch.equal(a, b) for a, b in zip(again, want[0]))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[], []]
    for f, h in zip(one, two):
        with torch.cuda.stream(a):
            got[0].append(f())
        with torch.cuda.stream(b):
            got[1].append(h())
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(x, y))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = [f() for f in one]
    for _ in range(3):
        for t in kept:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(kept, want[0]))


def test_given_stream(moe):
    """A stream argument: outputs belong to it, on either path."""
    g, s = gen(4), torch.cuda.Stream()
    off, E, R = offsets_of(FEW), len(FEW), sum(FEW)
    x, w, dy = normal(g, R, 64, dtype=BF), normal(g, E, 64, 72, dtype=BF), normal(g, R, 72, dtype=BF)
    ws, ows = moe.grouped_new_workspace(E, 64, 72), moe.orthogonalize_new_workspace(E, 64, 72)
    gu = normal(g, R, 144, dtype=BF)
    calls = [lambda **k: moe.grouped_product(x, off, w, ws, **k), lambda **k: moe.grouped_weight_grad(x, dy, off, ws, **k),
             lambda **k: moe.swiglu(gu, **k), lambda **k: moe.swiglu_backward(gu, dy, **k)[0],
             lambda **k: moe.orthogonalize(w, ows, **k)]
    for f in calls:
        want = f()
        torch.cuda.synchronize()
        for stream in (s, s.cuda_stream):
            got = f(stream=stream)
            s.synchronize()
            assert torch.equal(got, want)


def test_python_path_and_native_path(moe, monkeypatch):
    if not moe.NATIVE_TENSOR_CALLS:
        pytest.skip("no native tensor calls here")
    want = [f() for f in work(moe, 5)]
    fs = work(moe, 5)
    for name in ("grouped_product", "grouped_weight_grad", "swiglu", "swiglu_backward", "orthogonalize"):
        assert getattr(moe._calls, name) is not None
    class Declines:  # noqa: E306
        def __getattr__(self, name):
            return lambda *a: None
    monkeypatch.setattr(moe, "_calls", Declines())
    assert all(torch.equal(f(), w) for f, w in zip(fs, want))


@pytest.mark.parametrize("kind", range(9))
def test_waits_that_run_out(moe, kind):
    """Under a limit far below a copy's round trip some bounded wait runs out, whoever's it is; the call reports it,
    its copies and MMAs have ended when it ends, and the next call in the same context is right."""
    g = gen(6)
    counts = FEW if kind % 2 else [900, 700, 0, 1100, 800]
    off, E, R = offsets_of(counts), len(counts), sum(counts)
    if kind < 6:
        K, N = ((72, 136), (1160, 648), (2048, 2560))[kind // 2]
        x, dy, w = normal(g, R, K, dtype=BF), normal(g, R, N, dtype=BF), normal(g, E, K, N, dtype=BF)
        ws = moe.grouped_new_workspace(E, K, N)
        run = lambda: (moe.grouped_product(x, off, w, ws), moe.grouped_weight_grad(x, dy, off, ws))  # noqa: E731
    else:
        rows, cols, n = ((128, 256, 3), (300, 520, 2), (640, 1000, 9))[kind - 6]
        m = updates(g, n, rows, cols, BF)
        ws = moe.orthogonalize_new_workspace(n, rows, cols)
        run = lambda: (moe.orthogonalize(m, ws),)  # noqa: E731
    want = run()
    assert moe.moe_read_device_status(ws) == 0
    seen = []
    for limit in (16, 16, 16, 200, 1000, 3000):
        try:
            moe.moe_set_wait_limit(limit)
            run()
            seen.append(moe.moe_read_device_status(ws))
        finally:
            moe.moe_set_wait_limit(0)
        assert all(torch.equal(a, b) for a, b in zip(run(), want))
        assert moe.moe_read_device_status(ws) == 0
    assert 6 in seen[:3] and set(seen) <= {0, 6}, seen


def test_past_32_bit_offsets(moe):
    """More than 2^31 elements of rows, of weights' gradients and of a stack of updates: the last ones are right."""
    g = gen(8)
    K, N, E = 2056, 8, 3
    R = (1 << 31) // K + 5000
    off = offsets_of([7, R - 1207, 1200])
    ws = moe.grouped_new_workspace(E, K, N)
    x = torch.empty((R, K), dtype=BF, device="cuda").normal_(generator=g)
    w, dy = normal(g, E, K, N, dtype=BF), normal(g, R, N, dtype=BF)
    y = moe.grouped_product(x, off, w, ws, dtype=F32)
    ref.close(y[-1200:], x[-1200:].double() @ w[2].double(), K)
    d = moe.grouped_weight_grad(x, dy, off, ws)
    ref.close(d[2], x[-1200:].double().T @ dy[-1200:].double(), 1200)
    wide = moe.grouped_product(dy, off, w.transpose(1, 2).contiguous(), ws)     # [R, K] out
    ref.close(wide[-1200:], dy[-1200:].double() @ w[2].double().T, N)
    del x, wide
    E, K, N = 140, 4096, 4096
    off = offsets_of([3] * E)
    x, dy = normal(g, 3 * E, K, dtype=BF), normal(g, 3 * E, N, dtype=BF)
    d = moe.grouped_weight_grad(x, dy, off, moe.grouped_new_workspace(E, K, N))
    ref.close(d[-1], x[-3:].double().T @ dy[-3:].double(), 3)
    ws = moe.orthogonalize_new_workspace(E, K, N)
    u = moe.orthogonalize(d.to(BF), ws, steps=1)
    want, tol = ref.orthogonalize(d[-1:].to(BF), steps=1)
    assert (u[-1].double() - want[0]).norm() <= (tol[0] + 2.0 ** -8) * want.norm()


def test_gradients_are_differences(moe):
    """The gradients against differences of the forward calls, in fp16 with FP32 outputs."""
    g, E, K, N = gen(9), 3, 64, 72
    off = offsets_of([5, 0, 4])
    ws = moe.grouped_new_workspace(E, K, N)
    x, w, c = normal(g, 9, K, dtype=HF), normal(g, E, K, N, dtype=HF, std=0.1), normal(g, 9, N, dtype=HF)
    loss = lambda x, w: (moe.grouped_product(x, off, w, ws, dtype=F32).double() * c.double()).sum()  # noqa: E731
    dx, dw = moe.grouped_product(c, off, w, ws, transposed=True, dtype=F32), moe.grouped_weight_grad(x, c, off, ws)
    for t, d, f in ((x, dx, lambda t: loss(t, w)), (w, dw, lambda t: loss(x, t))):
        step = normal(g, *t.shape).sign().to(HF) * 2.0 ** -4
        up, down = t + step, t - step
        diff = f(up) - f(down)
        # (the rounded inputs' own difference; the function is linear in each)
        want = (d.double() * (up.double() - down.double())).sum()
        size = (d.double().abs() * (up.double() - down.double()).abs()).sum()
        assert (diff - want).abs() <= (ref.sums_tol(K) + 2.0 ** -20) * size * 64, (diff, want, size)
