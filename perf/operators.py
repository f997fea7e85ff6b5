"""The operators of the 4-bit expert path, as cases: what a user's program has in hand, the call, and
the same computed plainly.

  select      from router logits to k experts a token: softmax or sigmoid scores, a bias for balance,
              groups of experts, weights (renormalised or not), and the sum of each expert's
              probability over the tokens (what a load-balance loss is made of)
  select_bwd  its gradient for the logits (and, where the bias joins the logits, for the bias)
  quantize    microscaled 4-bit floating point: blocks of 32 values of a row share one power-of-two
              scale, each value is one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign
  product     the grouped experts' product of rows and weights that are both held so

``own`` selects the side: the plain form (torch operations in 32 bits), or the library's calls.
"""
import math

import torch

own = False

# Sizes are those of the layers the library's benchmark runs (fine_grained: H=2048, E=64, k=8, I=1024;
# packed_rl: H=2048, E=128, k=8, I=768; large: T=32768, E=256, k=8), or generic.
_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one token of a decode step: 256 experts in eight groups, four of them kept
        dict(name="select_token", op="select", T=1, E=256, k=8, kind="sigmoid", groups=8, keep=4, top=2, renorm=True,
             bias=True, prob=False, dtype="f32"),
        # a long prompt or a training micro-batch of the same layer, with the sums a balance loss needs
        dict(name="select_prompt", op="select", T=32768, E=256, k=8, kind="sigmoid", groups=8, keep=4, top=2,
             renorm=True, bias=True, prob=True, dtype="f32"),
        # softmax scores without groups, bf16 logits as a matrix product leaves them, an odd token count
        dict(name="select_softmax_odd", op="select", T=4097, E=64, k=6, kind="softmax", groups=1, keep=1, top=1,
             renorm=False, bias=False, prob=False, dtype="bf16"),
        # the gradient of the long batch, the balance loss's part in it
        dict(name="select_bwd_prompt", op="select_bwd", T=32768, E=256, k=8, kind="sigmoid", groups=8, keep=4, top=2,
             renorm=True, bias=True, prob=True, dtype="f32"),
        # softmax scores over 128 experts with a popularity bias that learns with the logits
        dict(name="select_bwd_softmax", op="select_bwd", T=16384, E=128, k=8, kind="softmax", groups=1, keep=1, top=1,
             renorm=False, bias=True, prob=True, dtype="bf16"),
        # hidden rows of a decode batch
        dict(name="quantize_batch", op="quantize", R=64, K=2048, dtype="bf16"),
        # hidden rows of a prompt
        dict(name="quantize_prompt", op="quantize", R=32768, K=4096, dtype="bf16"),
        # an odd number of fp32 rows whose length is no power of two
        dict(name="quantize_f32_odd", op="quantize", R=4099, K=1440, dtype="f32"),
        # one token through the gate and up projections of a fine-grained layer: eight rows, eight experts
        dict(name="product_token", op="product", T=1, K=2048, N=2048, E=64, k=8, zipf=0.0, x="bf16", y="bf16"),
        # a decode batch of 64 tokens, about eight rows an expert, unevenly spread
        dict(name="product_batch", op="product", T=64, K=2048, N=2048, E=64, k=8, zipf=1.0, x="bf16", y="bf16"),
        # the down projection of a 4096-token prompt, FP32 rows for the weighted sum that follows
        dict(name="product_down", op="product", T=4096, K=1024, N=2048, E=64, k=8, zipf=0.0, x="bf16", y="f32"),
        # gate and up of a packed row of 16384 tokens with popular and rare experts
        dict(name="product_packed", op="product", T=16384, K=2048, N=1536, E=128, k=8, zipf=1.0, x="bf16", y="bf16"),
    ]


def _between(rng, lo, hi):
    """A whole number, spread over the logarithm of the range."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _times(rng, lo, hi, unit):
    n = unit * _between(rng, lo, hi)
    return n if n != 3072 else n + unit


def draw(rng):
    op = rng.choice(["select", "select_bwd", "quantize", "product"])
    if op in ("select", "select_bwd"):
        groups = rng.choice([1, 1, 2, 4, 8])
        per = rng.randint(2, 256 // groups)
        keep = rng.randint(1, groups)
        kind = rng.choice(["sigmoid", "softmax"])
        return dict(op=op, T=_between(rng, 1, 32768), E=groups * per, k=rng.randint(1, min(16, keep * per)), kind=kind,
                    groups=groups, keep=keep, top=rng.choice([1, 2]), renorm=rng.random() < 0.7,
                    bias=rng.random() < 0.7, prob=rng.random() < 0.5, dtype=rng.choice(["f32", "bf16", "f16"]))
    if op == "quantize":
        K = _times(rng, 1, 128, 32)
        return dict(op=op, R=_between(rng, 1, min(32768, 32768 * 4096 // K)), K=K, dtype=rng.choice(["f32", "bf16", "f16"]))
    k, E = rng.randint(1, 8), rng.choice([8, 16, 40, 64, 128])
    K, N = _times(rng, 1, 16, 128), _times(rng, 1, 16, 128)
    return dict(op=op, T=_between(rng, 1, 16384 // k), K=K, N=N, E=E, k=k, zipf=rng.choice([0.0, 0.5, 1.0]),
                x=rng.choice(["bf16", "f16", "f32"]), y=rng.choice(["bf16", "f32"]))


def _active(c):
    """About how many experts get rows."""
    return c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])


def work(case):
    c = case
    if c["op"] == "select":
        b, n = _BYTES[c["dtype"]], c["T"] * c["E"]
        return {"bytes": n * b + 8 * c["T"] * c["k"] + (4 * c["E"] if c["prob"] else 0) + (4 * c["E"] if c["bias"] else 0),
                "flops": 4 * n}
    if c["op"] == "select_bwd":
        b, n = _BYTES[c["dtype"]], c["T"] * c["E"]
        dense = c["prob"] or (c["kind"] == "softmax" and not c["renorm"])  # else only the chosen logits matter
        return {"bytes": n * b + (n * b if dense else c["T"] * c["k"] * b) + 8 * c["T"] * c["k"], "flops": 8 * n}
    if c["op"] == "quantize":
        n = c["R"] * c["K"]
        return {"bytes": n * (_BYTES[c["dtype"]] + 2 + 0.5 + 1 / 32), "flops": 2 * n}
    R = c["T"] * c["k"]
    w = _active(c) * c["K"] * c["N"] * (0.5 + 1 / 32)
    return {"bytes": R * c["K"] * _BYTES[c["x"]] + w + R * c["N"] * _BYTES[c["y"]], "flops": 2.0 * R * c["K"] * c["N"]}


# ------------------------------------------------------------------ inputs ---
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _keys64(l, bias, kind):
    l = l.double()
    b = 0.0 if bias is None else bias.double()
    return (l + b) if kind == "softmax" else torch.sigmoid(l) + b


def _near(c, l, bias):
    """Rows whose choice hangs on a difference in the last bits of 32 (and is not an exact tie): two correct
    exponentials could choose differently there."""
    key = _keys64(l, bias, c["kind"])
    T, E = key.shape
    tight = 2e-6 * key.abs().amax(dim=1, keepdim=True).clamp(min=1.0)
    per = E // c["groups"]
    bad = torch.zeros(T, dtype=torch.bool, device=l.device)
    if c["keep"] < c["groups"]:
        g = key.view(T, c["groups"], per).sort(dim=2, descending=True).values[:, :, :min(c["top"], per)].sum(2)
        s, order = g.sort(dim=1, descending=True, stable=True)
        gap = s[:, c["keep"] - 1:c["keep"]] - s[:, c["keep"]:c["keep"] + 1]
        bad |= ((gap > 0) & (gap < tight)).squeeze(1)
        kept = torch.zeros_like(g, dtype=torch.bool).scatter_(1, order[:, :c["keep"]], True)
        key = key.masked_fill(~kept.repeat_interleave(per, dim=1), -math.inf)
    s = key.sort(dim=1, descending=True).values[:, :min(c["k"] + 1, E)]
    gap = s[:, :-1] - s[:, 1:]  # the order within the chosen counts too
    return bad | ((gap > 0) & (gap < tight)).any(1)


def _logits(c, g):
    T, E = c["T"], c["E"]
    bias = None
    if c["bias"]:
        # a correction learnt by small steps, or the log popularity of the experts
        bias = torch.randn(E, generator=g, device="cuda") * (0.02 if c["kind"] == "sigmoid" else 0.5)
    l = (torch.randn((T, E), generator=g, device="cuda") * 1.3).to(_DT[c["dtype"]])
    for _ in range(20):
        rows = _near(c, l, bias).nonzero().squeeze(1)
        if rows.numel() == 0:
            break
        l[rows] = (torch.randn((rows.numel(), E), generator=g, device="cuda") * 1.3).to(l.dtype)
    return l, bias


def _hidden(R, K, dtype, g):
    """Rows as a norm leaves them: unit scale, and a few channels that are much larger than the rest."""
    x = torch.randn((R, K), generator=g, device="cuda")
    x *= torch.exp(0.7 * torch.randn(K, generator=g, device="cuda"))
    return x.to(_DT[dtype])


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": dict(c)}
    if own:
        import moe_expert_layer_fp32_gb300 as moe
        s["moe"] = moe
    if c["op"] in ("select", "select_bwd"):
        s["logits"], s["bias"] = _logits(c, g)
        if own:
            kind = moe.MOE_ROUTER_SOFTMAX if c["kind"] == "softmax" else moe.MOE_ROUTER_SIGMOID_BIAS_SELECT
            s["opts"] = moe.select_opts(kind, n_group=c["groups"], topk_group=c["keep"], group_top=c["top"],
                                        renorm=c["renorm"])
        if c["op"] == "select_bwd":
            # what the forward pass chose and what the layer above sends back
            s["idx"] = _select_plain(c, s["logits"], s["bias"])[0]
            s["d_w"] = torch.randn((c["T"], c["k"]), generator=g, device="cuda")
            s["d_prob"] = torch.randn(c["E"], generator=g, device="cuda") if c["prob"] else None
        return s
    if c["op"] == "quantize":
        s["x"] = _hidden(c["R"], c["K"], c["dtype"], g)
        return s
    T, K, N, E, k = c["T"], c["K"], c["N"], c["E"], c["k"]
    R = T * k
    # k distinct experts a token, popularity falling as rank^-zipf: the largest of log p + Gumbel noise
    p = -c["zipf"] * torch.log(1.0 + torch.randperm(E, generator=g, device="cuda").float())
    u = torch.rand((T, E), generator=g, device="cuda").clamp(1e-7, 1 - 1e-7)
    ids = (p - torch.log(-torch.log(u))).topk(k, dim=1).indices
    counts = torch.bincount(ids.flatten(), minlength=E)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["most"], s["active"] = int(counts.max()), int((counts > 0).sum())
    s["x"] = _hidden(R, K, c["x"], g)
    s["codes"] = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    s["scales"] = torch.empty((E, N, K // 32), dtype=torch.uint8, device="cuda")
    for e in range(E):  # the checkpoint: rows over K, two values a byte, a scale a block
        code, sc = _quantize_plain(torch.randn((N, K), generator=g, device="cuda") * 0.02)
        s["codes"][e] = code[:, 0::2] | (code[:, 1::2] << 4)
        s["scales"][e] = sc
    if own:
        s["packed"] = moe.mx4_pack(s["codes"], s["scales"])
        s["workspace"] = moe.mx4_new_workspace(R, K, N, E)
        del s["codes"], s["scales"]
    return s


# ------------------------------------------------------------- plain forms ---
def _select_plain(c, logits, bias):
    l = logits.float()
    T, E = l.shape
    per = E // c["groups"]
    if c["kind"] == "softmax":
        key = l if bias is None else l + bias
        p = torch.exp(key - key.amax(dim=1, keepdim=True))
        score = q = p / p.sum(dim=1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
        key = score if bias is None else score + bias
        q = score / score.sum(dim=1, keepdim=True)
    if c["keep"] < c["groups"]:
        top = key.view(T, c["groups"], per).sort(dim=2, descending=True).values[:, :, :min(c["top"], per)].sum(2)
        kept = top.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        mask = torch.zeros((T, c["groups"]), dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        key = key.masked_fill(~mask.repeat_interleave(per, dim=1), -math.inf)
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = score.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return idx.to(torch.int32), w, (q.double().sum(0).float() if c["prob"] else None)


def _select_bwd_plain(c, s):
    l, idx, dw = s["logits"].float(), s["idx"].long(), s["d_w"]
    if c["kind"] == "softmax":
        key = l if s["bias"] is None else l + s["bias"]
        p = torch.exp(key - key.amax(dim=1, keepdim=True))
        score = q = p / p.sum(dim=1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
        total = score.sum(dim=1, keepdim=True)
        q = score / total
    # the gradient for the chosen scores, then for every score
    if c["renorm"]:
        chosen = score.gather(1, idx)
        total_chosen = chosen.sum(dim=1, keepdim=True)
        d_chosen = (dw - (dw * chosen).sum(dim=1, keepdim=True) / total_chosen) / total_chosen
    else:
        d_chosen = dw
    d_score = torch.zeros_like(l).scatter_(1, idx, d_chosen)
    if c["kind"] == "softmax":
        if s["d_prob"] is not None:
            d_score = d_score + s["d_prob"]
        d = q * (d_score - (d_score * q).sum(dim=1, keepdim=True))
    else:
        if s["d_prob"] is not None:
            d_score = d_score + (s["d_prob"] - (s["d_prob"] * q).sum(dim=1, keepdim=True)) / total
        d = d_score * score * (1.0 - score)
    out = {"d_logits": d.to(s["logits"].dtype)}
    if s["bias"] is not None and c["kind"] == "softmax":
        out["d_bias"] = d.double().sum(0).float()
    return out


def _quantize_plain(x):
    """(codes [R, K] 0..15, scale bytes [R, K/32]): the scale is 2^(byte - 127), the block's largest value has
    the exponent of 4 or is the smallest scale's; values round to nearest, ties to the even code, at most 6."""
    R, K = x.shape
    v = x.float().view(R, K // 32, 32)
    byte = ((v.abs().amax(dim=2).view(torch.int32) >> 23) - 2).clamp(min=0)
    a = torch.ldexp(v.abs(), (127 - byte).unsqueeze(2))
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + 8 * torch.signbit(v).to(torch.uint8)
    return code.view(R, K), byte.to(torch.uint8)


def _value(code, byte):
    """The values that codes and scale bytes stand for, in fp32."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    table = torch.cat([table, -table])
    v = table[code.long()].view(*byte.shape, 32)
    return torch.ldexp(v, (byte.to(torch.int32) - 127).unsqueeze(-1)).view(code.shape)


def _product_plain(c, s):
    x, off = s["x"], s["offsets"].long()
    R, A, cap = x.shape[0], s["active"], s["most"]
    xq = _value(*_quantize_plain(x))
    counts = off[1:] - off[:-1]
    experts = (counts == 0).to(torch.int32).sort(stable=True).indices[:A]  # those with rows
    row = off[experts].unsqueeze(1) + torch.arange(cap, device=x.device)    # [A, cap]
    mine = torch.arange(cap, device=x.device) < counts[experts].unsqueeze(1)
    xe = xq[row.clamp(max=R - 1)] * mine.unsqueeze(2)
    codes = s["codes"][experts]
    w = _value(torch.stack([codes & 15, codes >> 4], dim=3).view(A, c["N"], c["K"]), s["scales"][experts])
    y = torch.bmm(xe, w.transpose(1, 2))
    out = torch.empty((R, c["N"]), dtype=torch.float32, device=x.device)
    out[row[mine]] = y[mine]
    return out.to(_DT[c["y"]])


# -------------------------------------------------------------------- run ---
def run(state):
    s, c = state, state["case"]
    if c["op"] == "select":
        if own:
            r = s["moe"].route_select(s["logits"], c["k"], s["opts"], bias=s["bias"], want_prob_sum=c["prob"])
        else:
            r = _select_plain(c, s["logits"], s["bias"])
        out = {"idx": r[0], "w": r[1]}
        if c["prob"]:
            out["prob_sum"] = r[2]
        return out
    if c["op"] == "select_bwd":
        if not own:
            return _select_bwd_plain(c, s)
        want = s["bias"] is not None and c["kind"] == "softmax"
        r = s["moe"].route_select_backward(s["logits"], s["idx"], s["d_w"], s["opts"], bias=s["bias"],
                                           d_prob_sum=s["d_prob"], want_d_bias=want)
        return {"d_logits": r[0], "d_bias": r[1]} if want else {"d_logits": r}
    if c["op"] == "quantize":
        if own:
            return s["moe"].mx4_quantize(s["x"], want_values=True)[2]
        code, byte = _quantize_plain(s["x"])
        return _value(code, byte).to(torch.bfloat16)
    if own:
        return s["moe"].mx4_expert_product(s["x"], s["offsets"], s["packed"], c["N"], s["workspace"], dtype=_DT[c["y"]])
    return _product_plain(c, s)


# ------------------------------------------------------------------ 64 bits ---
def _exact_scores(c, l, bias):
    """(key, score, probability) of every expert in 64 bits."""
    l = l.double()
    if c["kind"] == "softmax":
        key = l if bias is None else l + bias.double()
        p = torch.softmax(key, dim=1)
        return key, p, p
    sc = torch.sigmoid(l)
    return (sc if bias is None else sc + bias.double()), sc, sc / sc.sum(1, keepdim=True)


def _exact_weights(c, score, idx):
    w = torch.gather(score, 1, idx)
    return w / w.sum(1, keepdim=True) if c["renorm"] else w


def _exact_rows(x):
    """Rows rounded to microscaled 4 bits, in 64 bits: a grid of steps 2^(e - 1) above 2^e, 0.5 below 2."""
    v = x.double().reshape(x.shape[0], -1, 32)
    m = v.abs().amax(2, keepdim=True)
    e = torch.where(m > 0, torch.frexp(m).exponent.double() - 1, torch.full_like(m, -1000.0))  # m = f 2^(e+1), f >= 0.5
    scale = torch.exp2((e - 2).clamp(min=-127.0))
    a = v.abs() / scale
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.sign(v) * (torch.round(a / step) * step).clamp(max=6.0) * scale).reshape(x.shape)


def exact(case, seed):
    global own
    keep, own = own, False  # the checkpoint's codes, not the library's layout of them
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    c = case
    if c["op"] == "select":
        key, score, q = _exact_scores(c, s["logits"], s["bias"])
        T, E = key.shape
        per = E // c["groups"]
        if c["keep"] < c["groups"]:
            g = torch.topk(key.view(T, c["groups"], per), min(c["top"], per), dim=2).values.sum(2)
            lose = torch.argsort(g, dim=1, descending=True, stable=True)[:, c["keep"]:]
            gone = (lose.unsqueeze(2) * per + torch.arange(per, device=g.device)).flatten(1)
            key = key.scatter(1, gone, -math.inf)
        idx = torch.argsort(key, dim=1, descending=True, stable=True)[:, :c["k"]]
        out = {"idx": idx.to(torch.int32), "w": _exact_weights(c, score, idx)}
        if c["prob"]:
            out["prob_sum"] = q.sum(0)
        return out
    if c["op"] == "select_bwd":
        # the forward pass's definition, differentiated by torch in 64 bits
        l = s["logits"].double().requires_grad_(True)
        b = s["bias"].double().requires_grad_(True) if s["bias"] is not None else None
        with torch.enable_grad():
            _, score, q = _exact_scores(c, l, b)
            loss = (_exact_weights(c, score, s["idx"].long()) * s["d_w"].double()).sum()
            if s["d_prob"] is not None:
                loss = loss + (q.sum(0) * s["d_prob"].double()).sum()
        if b is not None and c["kind"] == "softmax":
            d, db = torch.autograd.grad(loss, [l, b])
            return {"d_logits": d, "d_bias": db}
        return {"d_logits": torch.autograd.grad(loss, [l])[0]}
    if c["op"] == "quantize":
        return _exact_rows(s["x"])
    xq, off = _exact_rows(s["x"]), s["offsets"].tolist()
    y = torch.empty((xq.shape[0], c["N"]), dtype=torch.float64, device=xq.device)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                        device=xq.device)
    for e in range(c["E"]):
        if off[e + 1] > off[e]:
            code = s["codes"][e].long()
            w = grid[torch.stack([code % 16, code // 16], 2).flatten(1)].view(c["N"], -1, 32)
            w = (w * torch.exp2(s["scales"][e].double() - 127).unsqueeze(2)).flatten(1)
            y[off[e]:off[e + 1]] = xq[off[e]:off[e + 1]] @ w.T
    return y
