"""A layer with microscaled 4-bit experts, and one step of its router's training.

    python examples/mx4_layer.py [--tokens T]

Packs bf16 expert weights to 4 bits, runs the layer's forward pass (router logits, selection in
groups of experts, the two grouped 4-bit products, the weighted sum) for a prompt and for a
single token, and compares it with the bf16 layer.  Then takes the router apart as a training
step does: logits, selection with the probability sums of a load-balance loss, and the gradient
for the logits, from which the router weight's gradient is one matrix product.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_layer_fp32_gb300 as moe  # noqa: E402


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=1024)
    T, H, E, k, I = ap.parse_args().tokens, 1024, 64, 8, 512
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    x = normal(T, H)
    w_router = normal(H, E, std=0.03, dtype=torch.float32)
    balance = normal(E, std=0.01, dtype=torch.float32)  # the selection-only correction bias
    w_gate, w_up = normal(E, H, I, std=0.03), normal(E, H, I, std=0.03)
    w_down = normal(E, I, H, std=0.03)

    # one-time preparation: gate and up share an operand
    gate_up, down = moe.mx4_prepack(w_gate, w_up), moe.mx4_prepack(w_down)
    kinds = moe.MOE_ROUTER_SIGMOID_BIAS_SELECT
    rule = moe.select_opts(kinds, n_group=8, topk_group=4, group_top=2)  # 4 of 8 groups, then 8 experts
    d = moe.dims(T, H, E, k, I)
    workspace = moe.mx4_new_layer_workspace(d)
    out, idx, w, counts = moe.mx4_layer_forward(x, w_router, balance, gate_up, down, d, workspace, rule,
                                                want_routing=True)
    status = moe.moe_read_device_status(workspace)
    assert status == 0, moe.STATUS[status]

    # a token of the batch alone is the same bits
    d1 = moe.dims(1, H, E, k, I)
    one = moe.mx4_layer_forward(x[:1].contiguous(), w_router, balance, gate_up, down, d1,
                                moe.mx4_new_layer_workspace(d1), rule)
    assert torch.equal(one[0], out[0])

    # the bf16 experts on the same routing
    packed = moe.prepack(w_gate, w_up, w_down, d)
    ws = moe.new_workspace(d)
    order = torch.argsort(idx.flatten().long(), stable=True)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0, dtype=torch.int32)])
    y = torch.empty((T * k, H), device="cuda")
    moe.moe_expert_ffn(x[order // k], offsets, packed, d, y, ws)
    rows = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device="cuda")).int()
    ref = torch.empty_like(out)
    moe.moe_combine(y, w, rows, d, ref)
    rel = ((out.float() - ref.float()).norm() / ref.float().norm()).item()
    size = (gate_up.numel() + down.numel()) / (2 * packed.numel())
    print(f"{T} tokens through {E} experts: weights {size:.3f} of the bf16 bytes, output {rel:.3f} "
          f"(relative L2) from the bf16 experts', load {counts.min().item()}..{counts.max().item()} rows")

    # the router's training step: L = sum(w * u) + alpha * E / (k T^2) * sum_e counts_e * prob_sum_e
    logits = torch.empty((T, E), device="cuda")
    moe.moe_router_logits(x, w_router, None, d, logits)
    idx, w, prob = moe.route_select(logits, k, rule, bias=balance, want_prob_sum=True)
    load = torch.bincount(idx.flatten().long(), minlength=E).float()
    u = normal(T, k, dtype=torch.float32)  # dL/dw from the layer above
    alpha = 1e-2 * E / (k * T * T)
    d_logits = moe.route_select_backward(logits, idx, u, rule, bias=balance, d_prob_sum=alpha * load)
    d_w_router = x.float().t() @ d_logits
    loss = (w * u).sum() + alpha * (load * prob).sum()
    print(f"router step: loss {loss.item():.4f}, balance part {(alpha * (load * prob).sum()).item():.4f}, "
          f"|d w_router| {d_w_router.norm().item():.4f}")


if __name__ == "__main__":
    main()
