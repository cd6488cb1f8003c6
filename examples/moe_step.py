"""One training step of a mixture-of-experts feed-forward layer on libufp4:
tokens into expert order, the two grouped FP4 products with the gated
activation between them, and back to token order; then the backward pass.

What the forward pass keeps for the backward one is small: the operands of the
weight gradients in 4 bits (the column-wise halves of the dual quantizations),
gate, up and the experts' outputs in 8 bits, and the plan.

    python examples/moe_step.py                 # 16384 tokens x top-6 of 64 experts, 2048 -> 1408 -> 2048
    python examples/moe_step.py --tokens 512    # a smaller batch

prints the step's time, what it keeps, and the distance of its result from
the same layer in fp32 (the 4-bit operands' quantization error).
"""
import argparse
import os
import sys
from types import SimpleNamespace

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp4_quantized_numerics_gb300 import ufp4 as U  # noqa: E402

GRID, RHT = U.UFP4_E1M2, dict(rht=True, rht_seed=2)


def quantize_weights(w, experts):
    """Both quantizations of the stacked expert weights [experts * out, in]."""
    return U.ufp4_quantize_grouped_dual(w, GRID, [w.shape[0] // experts] * experts, **RHT)


def _products(a, b, c, counts, kind, k, n):
    """The grouped product of every expert into its rows of c: "y", tokens by
    weights (inner dimension k, n outputs); "dx", gradients by transposed
    weights (inner dimension k); "dw", k x n with the tokens inside."""
    rows, ks = U.grouped_offsets(counts, False), U.grouped_offsets(counts, True)
    w_rows, w_ks = U.grouped_offsets([n] * len(counts), False), U.grouped_offsets([k] * len(counts), True)
    at, groups = 0, []
    for e, t in enumerate(counts):
        if kind == "dw":
            g = dict(M=k, N=n, K=(t + 15) // 16 * 16, a_row=0, a_k=ks[e], b_row=0, b_k=ks[e], c=c[e * k:(e + 1) * k])
        elif t == 0:
            continue
        else:
            g = dict(M=t, N=n, K=k, a_row=rows[e], a_k=0, b_row=w_rows[e] if kind == "y" else 0,
                     b_k=w_ks[e] if kind == "dx" else 0, c=c[at:at + t])
        groups.append(dict(g, a_seg=e, b_seg=e))
        at += t
    U.ufp4_gemm_grouped(a, b, groups)
    return c


def forward(x, ids, weights, w13, w2, experts, ffn):
    """x [tokens, hidden] bf16, ids [tokens, topk] experts, weights fp32 of
    the same shape; w13 / w2: quantize_weights of [experts * 2 ffn, hidden]
    (gate rows, then up rows, per expert) and [experts * hidden, ffn].
    Returns the layer's output in bf16 and what the backward pass needs."""
    hidden = x.shape[1]
    plan = U.ufp4_moe_sort(ids, experts)
    xs = U.ufp4_moe_dispatch(x, plan)
    counts = plan.counts.tolist()            # the grouped calls take their segments from the host
    n = sum(counts)
    x_row, x_col = U.ufp4_quantize_grouped_dual(xs[:n], GRID, counts, **RHT)
    gu = torch.empty(n, 2 * ffn, device=x.device)
    _products(x_row, w13[0], gu, counts, "y", hidden, 2 * ffn)
    h, keep_gate, keep_up = U.ufp4_swiglu(gu[:, :ffn], gu[:, ffn:], ckpt=U.UFP4_CKPT_INT8, dtype=torch.bfloat16)
    h_row, h_col = U.ufp4_quantize_grouped_dual(h, GRID, counts, **RHT)
    y = torch.empty(plan.tokens * plan.topk, hidden, device=x.device)   # dropped slots' rows are not read
    _products(h_row, w2[0], y, counts, "y", ffn, hidden)
    out = U.ufp4_moe_combine(y, plan, weights, dtype=torch.bfloat16)
    keep_y = U.ufp4_ckpt_save(y[:n])
    return out, SimpleNamespace(plan=plan, counts=counts, weights=weights, x_col=x_col, h_col=h_col,
                                keep_gate=keep_gate, keep_up=keep_up, keep_y=keep_y, ffn=ffn)


def backward(dout, s, w13, w2, seed=0):
    """Gradients of forward's inputs from dout [tokens, hidden] bf16: dx
    (bf16), the router weights', w13's and w2's (fp32)."""
    plan, counts, ffn = s.plan, s.counts, s.ffn
    n, hidden, experts, dev = sum(counts), dout.shape[1], len(counts), dout.device
    y = torch.empty(plan.tokens * plan.topk, hidden, dtype=torch.bfloat16, device=dev)
    U.ufp4_ckpt_load(s.keep_y, out=y[:n])
    dy, dweights = U.ufp4_moe_combine_bwd(dout, y, plan, s.weights, dtype=torch.bfloat16)
    sr = dict(round=U.UFP4_SR, sr_seed=seed, **RHT)
    dy_row, dy_col = U.ufp4_quantize_grouped_dual(dy[:n], GRID, counts, sr_counter_row=0, sr_counter_col=1, **sr)
    dw2 = _products(dy_col, s.h_col, torch.empty(experts * hidden, ffn, device=dev), counts, "dw", hidden, ffn)
    dh = _products(dy_row, w2[1], torch.empty(n, ffn, device=dev), counts, "dx", hidden, ffn)
    dgu = torch.empty(n, 2 * ffn, dtype=torch.bfloat16, device=dev)
    U.ufp4_swiglu_bwd(dh, s.keep_gate, s.keep_up, dgate=dgu[:, :ffn], dup=dgu[:, ffn:])
    d_row, d_col = U.ufp4_quantize_grouped_dual(dgu, GRID, counts, sr_counter_row=2, sr_counter_col=3, **sr)
    dw13 = _products(d_col, s.x_col, torch.empty(experts * 2 * ffn, hidden, device=dev), counts, "dw", 2 * ffn, hidden)
    dxs = torch.empty(plan.tokens * plan.topk, hidden, device=dev)
    _products(d_row, w13[1], dxs, counts, "dx", 2 * ffn, hidden)
    dx = U.ufp4_moe_combine(dxs, plan, dtype=torch.bfloat16)
    return dx, dweights, dw13, dw2


def plain(x, ids, weights, w13, w2, dout, experts, ffn):
    """The same layer in fp32 torch, expert by expert, with autograd."""
    x, weights, w13, w2 = (t.float().detach().requires_grad_() for t in (x, weights, w13, w2))
    hidden = x.shape[1]
    out = torch.zeros(x.shape, device=x.device)
    for e in range(experts):
        t, j = torch.where(ids == e)
        gu = x[t] @ w13[e * 2 * ffn:(e + 1) * 2 * ffn].T
        h = torch.nn.functional.silu(gu[:, :ffn]) * gu[:, ffn:]
        out = out.index_add(0, t, weights[t, j][:, None] * (h @ w2[e * hidden:(e + 1) * hidden].T))
    out.backward(dout.float())
    return out.detach(), x.grad, weights.grad, w13.grad, w2.grad


def make(tokens, topk, experts, hidden, ffn, seed=0, device="cuda"):
    """A random layer and batch, a router's choices and weights among them."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    new = lambda std, *shape: (torch.randn(shape, generator=g, device=device) * std).to(torch.bfloat16)  # noqa: E731
    top, ids = torch.topk(torch.randn(tokens, experts, generator=g, device=device) +
                          torch.randn(experts, generator=g, device=device), topk, dim=1)
    return dict(x=new(1.0, tokens, hidden), ids=ids, weights=torch.softmax(top, dim=1),
                w13=new(hidden ** -0.5, experts * 2 * ffn, hidden), w2=new(ffn ** -0.5, experts * hidden, ffn),
                dout=new(1e-3, tokens, hidden))


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 16384), ("topk", 6), ("experts", 64), ("hidden", 2048), ("ffn", 1408)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    d = make(a.tokens, a.topk, a.experts, a.hidden, a.ffn)
    w13, w2 = quantize_weights(d["w13"], a.experts), quantize_weights(d["w2"], a.experts)

    def step():
        out, kept = forward(d["x"], d["ids"], d["weights"], w13, w2, a.experts, a.ffn)
        return (out, *backward(d["dout"], kept, w13, w2)), kept

    for _ in range(3):
        got, kept = step()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(10):
        step()
    end.record()
    torch.cuda.synchronize()
    size = lambda t: t.numel() * t.element_size()  # noqa: E731
    bits4 = sum(size(q.codes) + size(q.scales) for q in (kept.x_col, kept.h_col))
    bits8 = sum(size(c.codes) + size(c.scales) for c in (kept.keep_gate, kept.keep_up, kept.keep_y))
    print("step %.3f ms; kept for the backward pass: %.1f MB in 4 bits, %.1f MB in 8 bits" %
          (begin.elapsed_time(end) / 10, bits4 / 1e6, bits8 / 1e6))
    want = plain(**d, experts=a.experts, ffn=a.ffn)
    for name, u, v in zip(("out", "dx", "dweights", "dw13", "dw2"), got, want):
        print("%-9s off by %.3f of its norm from fp32" % (name, ((u.float() - v).norm() / v.norm()).item()))


if __name__ == "__main__":
    main()
