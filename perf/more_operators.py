"""The operators that train the experts, as cases: what a user's program has in hand, the call, and the
same computed plainly.

  product     the grouped product of rows sorted by expert with the experts' matrices in their logical
              layout: y[r] = x[r] W_e, or (transposed) y[r] = x[r] W_e^T, which is also the gradient of the
              first for its rows
  wgrad       the gradient of that product for the matrices: dW_e = sum over the rows r of expert e of
              x[r]^T dy[r], zero for an expert without rows
  swiglu_bwd  the gradient of w[r] silu(gate) up for gate, up and the routing weight w[r], with the weighted
              activations that the down projection's gradient needs
  orth        a stack of update matrices, one an expert, orthogonalised by Newton-Schulz steps
              X <- a X + (b X X^T + c (X X^T)^2) X from X = M / (|M| + eps)

``own`` selects the side: the plain form (torch operations in 32 bits), or the library's calls.
"""
import math

import torch

own = False

# Sizes are those of the layers the library's benchmark runs (tiny: H=128, E=8, k=2, I=256; fine_grained: H=2048,
# E=64, k=8, I=1024; packed_rl: H=2048, E=128, k=8, I=768), or generic.
_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}
_COEF = (3.4445, -4.7750, 2.0315)  # the quintic that lifts small singular values fastest, five steps
_EPS = 1e-7


def listed():
    return [
        # one token through the gate and up projections of a fine-grained layer: eight rows, eight experts
        dict(name="product_token", op="product", T=1, K=2048, N=2048, E=64, k=8, zipf=0.0, turn=False, x="bf16", y="bf16"),
        # a rollout's decode batch of 64 tokens, about eight rows an expert, unevenly spread; FP32 rows
        dict(name="product_batch", op="product", T=64, K=1024, N=2048, E=64, k=8, zipf=1.0, turn=False, x="bf16", y="f32"),
        # gate and up of a packed row of 16384 tokens with popular and rare experts
        dict(name="product_packed", op="product", T=16384, K=2048, N=1536, E=128, k=8, zipf=1.0, turn=False, x="bf16", y="bf16"),
        # the gradient through a projection whose sizes are no multiples of a tile, fp16, an odd token count
        dict(name="product_grad_odd", op="product", T=4001, K=1440, N=2888, E=40, k=6, zipf=0.5, turn=True, x="f16", y="f16"),
        # gate and up weights' gradient of a 4096-token micro-batch, FP32 for the optimiser
        dict(name="wgrad_micro", op="wgrad", T=4096, K=2048, N=2048, E=64, k=8, zipf=0.0, x="bf16", y="f32"),
        # down weights' gradient of a packed row, popular and rare experts, bf16
        dict(name="wgrad_packed", op="wgrad", T=16384, K=768, N=2048, E=128, k=8, zipf=1.0, x="bf16", y="bf16"),
        # a short sequence: a few rows an expert, some experts without any, odd sizes
        dict(name="wgrad_short", op="wgrad", T=77, K=1000, N=1440, E=64, k=2, zipf=1.0, x="f16", y="f32"),
        # the activations' gradient of a packed row
        dict(name="swiglu_packed", op="swiglu_bwd", R=131072, I=768, dtype="bf16", weighted=True),
        # the same of a short sequence, without routing weights
        dict(name="swiglu_short", op="swiglu_bwd", R=513, I=1024, dtype="bf16", weighted=False),
        # every expert's down projection of a fine-grained layer
        dict(name="orth_experts", op="orth", E=64, rows=1024, cols=2048, x="bf16", y="bf16"),
        # a tiny layer's
        dict(name="orth_tiny", op="orth", E=8, rows=128, cols=256, x="f32", y="bf16"),
        # FP32 momenta of matrices that are taller than wide, odd sizes
        dict(name="orth_odd", op="orth", E=5, rows=1439, cols=1001, x="f32", y="bf16"),
    ]


def _between(rng, lo, hi):
    """A whole number, spread over the logarithm of the range."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["product", "product", "wgrad", "swiglu_bwd", "orth"])
    if op == "swiglu_bwd":
        I = 8 * _between(rng, 1, 512)
        return dict(op=op, R=_between(rng, 1, min(131072, 131072 * 768 // I)), I=I, dtype=rng.choice(["bf16", "f16"]),
                    weighted=rng.random() < 0.7)
    if op == "orth":
        E, rows, cols = _between(rng, 1, 64), _between(rng, 8, 2048), _between(rng, 8, 2048)
        m, n = min(rows, cols), max(rows, cols)
        E = max(1, min(E, 64 * 1024 * 1024 * 2048 // (m * m * n)))
        return dict(op=op, E=E, rows=rows, cols=cols, x=rng.choice(["bf16", "f32"]), y=rng.choice(["bf16", "f16"]))
    E = rng.choice([1, 8, 16, 40, 64, 128])
    k = rng.randint(1, min(8, E))
    K, N = 8 * _between(rng, 1, 256), 8 * _between(rng, 1, 256)
    T = _between(rng, 1, 16384 // k)
    c = dict(op=op, T=T, K=K, N=N, E=E, k=k, zipf=rng.choice([0.0, 0.5, 1.0]), x=rng.choice(["bf16", "f16"]),
             y=rng.choice(["bf16", "f16", "f32"]))
    if op == "product":
        c["turn"] = rng.random() < 0.5
    return c


def _active(c):
    """About how many experts get rows."""
    return c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])


def work(case):
    c = case
    if c["op"] == "swiglu_bwd":
        n = c["R"] * c["I"]
        # gate, up and the gradient in; their gradients and the activations out
        return {"bytes": 6 * n * _BYTES[c["dtype"]] + (8 * c["R"] if c["weighted"] else 0), "flops": 16 * n}
    if c["op"] == "orth":
        m, n = min(c["rows"], c["cols"]), max(c["rows"], c["cols"])
        # a step: half of X X^T and of its square (both symmetric), and the product with X
        return {"bytes": c["E"] * m * n * (_BYTES[c["x"]] + _BYTES[c["y"]]),
                "flops": 5.0 * c["E"] * (m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n)}
    R, K, N = c["T"] * c["k"], c["K"], c["N"]
    if c["op"] == "product":
        b = R * K * _BYTES[c["x"]] + _active(c) * K * N * _BYTES[c["x"]] + R * N * _BYTES[c["y"]]
    else:
        b = R * (K + N) * _BYTES[c["x"]] + c["E"] * K * N * _BYTES[c["y"]]
    return {"bytes": b, "flops": 2.0 * R * K * N}


# ------------------------------------------------------------------ inputs ---
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _hidden(R, K, dtype, g):
    """Rows as a norm leaves them: unit scale, and a few channels that are much larger than the rest."""
    x = torch.randn((R, K), generator=g, device="cuda")
    x *= torch.exp(0.7 * torch.randn(K, generator=g, device="cuda"))
    return x.to(_DT[dtype])


def _back(R, N, dtype, g):
    """What a layer above sends back: small, and of another size from row to row."""
    d = torch.randn((R, N), generator=g, device="cuda")
    d *= 0.01 * torch.exp(0.5 * torch.randn((R, 1), generator=g, device="cuda"))
    return d.to(_DT[dtype])


def _momenta(E, rows, cols, dtype, g):
    """Running means of gradients: a few strong directions over the noise of many batches, of a size that differs
    from expert to expert as their loads do."""
    r = max(1, min(rows, cols) // 16)
    u = torch.randn((E, rows, r), generator=g, device="cuda") * torch.exp(torch.randn((E, 1, r), generator=g, device="cuda"))
    m = torch.bmm(u, torch.randn((E, r, cols), generator=g, device="cuda")) / math.sqrt(r)
    m += 0.5 * torch.randn((E, rows, cols), generator=g, device="cuda")
    return (m * 1e-4 * torch.exp(torch.randn((E, 1, 1), generator=g, device="cuda"))).to(_DT[dtype])


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": dict(c)}
    if own:
        import moe_expert_layer_fp32_gb300 as moe
        s["moe"] = moe
    if c["op"] == "swiglu_bwd":
        R, I = c["R"], c["I"]
        s["gate_up"] = torch.randn((R, 2 * I), generator=g, device="cuda").to(_DT[c["dtype"]])
        s["d"] = _back(R, I, c["dtype"], g)
        s["w"] = (0.02 + 0.4 * torch.rand(R, generator=g, device="cuda")) if c["weighted"] else None
        return s
    if c["op"] == "orth":
        s["m"] = _momenta(c["E"], c["rows"], c["cols"], c["x"], g)
        if own:
            s["workspace"] = moe.orthogonalize_new_workspace(c["E"], c["rows"], c["cols"])
        return s
    T, K, N, E, k = c["T"], c["K"], c["N"], c["E"], c["k"]
    # k distinct experts a token, popularity falling as rank^-zipf: the largest of log p + Gumbel noise
    p = -c["zipf"] * torch.log(1.0 + torch.randperm(E, generator=g, device="cuda").float())
    u = torch.rand((T, E), generator=g, device="cuda").clamp(1e-7, 1 - 1e-7)
    ids = (p - torch.log(-torch.log(u))).topk(k, dim=1).indices
    counts = torch.bincount(ids.flatten(), minlength=E)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["piece"] = min(512, int(counts.max()))  # rows a piece of the plain form
    s["pieces"] = int(((counts + s["piece"] - 1) // s["piece"]).sum())
    s["x"] = _hidden(T * k, K, c["x"], g)
    if c["op"] == "product":
        shape = (E, N, K) if c["turn"] else (E, K, N)
        s["weights"] = (torch.randn(shape, generator=g, device="cuda") * 0.02).to(_DT[c["x"]])
    else:
        s["dy"] = _back(T * k, N, c["x"], g)
    if own:
        s["workspace"] = moe.grouped_new_workspace(E, K, N)
    return s


# ------------------------------------------------------------- plain forms ---
def _pieces(s):
    """Each expert's rows in pieces: (expert [P], row numbers [P, piece], which of those are rows of the expert)."""
    off, n = s["offsets"].long(), s["piece"]
    counts = off[1:] - off[:-1]
    of = (counts + n - 1) // n
    expert = torch.repeat_interleave(of, output_size=s["pieces"])
    at = (torch.arange(s["pieces"], device=off.device) - (of.cumsum(0) - of)[expert]) * n
    row = (off[expert] + at).unsqueeze(1) + torch.arange(n, device=off.device)
    return expert, row, row < off[expert + 1].unsqueeze(1)


def _gathered(rows, row, mine):
    return rows.float()[row.clamp(max=rows.shape[0] - 1)] * mine.unsqueeze(2)


def _product_plain(c, s):
    expert, row, mine = _pieces(s)
    w = s["weights"][expert].float()
    y = torch.bmm(_gathered(s["x"], row, mine), w.transpose(1, 2) if c["turn"] else w)
    out = torch.empty((s["x"].shape[0], c["N"]), dtype=torch.float32, device=y.device)
    out[row[mine]] = y[mine]
    return out.to(_DT[c["y"]])


def _wgrad_plain(c, s):
    expert, row, mine = _pieces(s)
    d = torch.bmm(_gathered(s["x"], row, mine).transpose(1, 2), _gathered(s["dy"], row, mine))
    out = torch.zeros((c["E"], c["K"], c["N"]), dtype=torch.float32, device=d.device)
    return out.index_add_(0, expert, d).to(_DT[c["y"]])


def _swiglu_bwd_plain(c, s):
    gate, up = s["gate_up"].float().chunk(2, dim=1)
    d = s["d"].float()
    w = s["w"].unsqueeze(1) if c["weighted"] else 1.0
    sig = 1.0 / (1.0 + torch.exp(-gate))
    act = gate * sig
    h = act * up
    dh = w * d
    dt = _DT[c["dtype"]]
    out = {"d_gate_up": torch.cat([dh * up * sig * (1.0 + gate * (1.0 - sig)), dh * act], dim=1).to(dt),
           "h": (w * h).to(dt)}
    if c["weighted"]:
        out["d_w"] = (d * h).sum(dim=1)
    return out


def _orth_plain(c, s):
    x = s["m"].float()
    if c["rows"] > c["cols"]:
        x = x.transpose(1, 2)
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + _EPS)
    a, b, cc = _COEF
    x = _orth_step(_orth_step(_orth_step(_orth_step(_orth_step(x, a, b, cc), a, b, cc), a, b, cc), a, b, cc), a, b, cc)
    return (x.transpose(1, 2) if c["rows"] > c["cols"] else x).contiguous().to(_DT[c["y"]])


def _orth_step(x, a, b, c):
    g = torch.bmm(x, x.transpose(1, 2))
    return a * x + torch.bmm(b * g + c * torch.bmm(g, g), x)


# -------------------------------------------------------------------- run ---
def run(state):
    s, c = state, state["case"]
    if c["op"] == "product":
        if own:
            return s["moe"].grouped_product(s["x"], s["offsets"], s["weights"], s["workspace"], transposed=c["turn"],
                                            dtype=_DT[c["y"]])
        return _product_plain(c, s)
    if c["op"] == "wgrad":
        if own:
            return s["moe"].grouped_weight_grad(s["x"], s["dy"], s["offsets"], s["workspace"], dtype=_DT[c["y"]])
        return _wgrad_plain(c, s)
    if c["op"] == "swiglu_bwd":
        if own:
            r = s["moe"].swiglu_backward(s["gate_up"], s["d"], row_weights=s["w"])
            out = {"d_gate_up": r[0], "h": r[1]}
            if c["weighted"]:
                out["d_w"] = r[2]
            return out
        return _swiglu_bwd_plain(c, s)
    if own:
        return s["moe"].orthogonalize(s["m"], s["workspace"], dtype=_DT[c["y"]], coefficients=_COEF, steps=5, eps=_EPS)
    return _orth_plain(c, s)


# ------------------------------------------------------------------ 64 bits ---
def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "swiglu_bwd":
        # the forward pass's definition, differentiated by torch in 64 bits
        gu = s["gate_up"].double().requires_grad_(True)
        w = s["w"].double() if c["weighted"] else torch.ones(c["R"], dtype=torch.float64, device="cuda")
        w.requires_grad_(True)
        with torch.enable_grad():
            h = w.unsqueeze(1) * torch.nn.functional.silu(gu[:, :c["I"]]) * gu[:, c["I"]:]
            d_gu, d_w = torch.autograd.grad(h, [gu, w], s["d"].double())
        out = {"d_gate_up": d_gu, "h": h.detach()}
        if c["weighted"]:
            out["d_w"] = d_w
        return out
    if c["op"] == "orth":
        out = torch.empty((c["E"], c["rows"], c["cols"]), dtype=torch.float64, device="cuda")
        a, b, cc = _COEF
        for e in range(c["E"]):
            m = s["m"][e].double()
            m = m / (torch.linalg.norm(m) + _EPS)
            for _ in range(5):
                if c["rows"] <= c["cols"]:
                    g = m @ m.T
                    m = a * m + b * (g @ m) + cc * (g @ (g @ m))
                else:
                    g = m.T @ m
                    m = a * m + b * (m @ g) + cc * ((m @ g) @ g)
            out[e] = m
        return out
    off, x = s["offsets"].tolist(), s["x"].double()
    if c["op"] == "product":
        y = torch.empty((x.shape[0], c["N"]), dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            w = s["weights"][e].double()
            y[off[e]:off[e + 1]] = x[off[e]:off[e + 1]] @ (w.T if c["turn"] else w)
        return y
    d = torch.zeros((c["E"], c["K"], c["N"]), dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        if off[e + 1] > off[e]:
            d[e] = x[off[e]:off[e + 1]].T @ s["dy"][off[e]:off[e + 1]].double()
    return d
