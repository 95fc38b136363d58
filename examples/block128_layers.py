"""8-bit layers with one scale for each block of 128, from training to decoding.

    python examples/block128_layers.py

1. A few steps of gradient descent on one linear layer: quantised activations,
   the forward product, the input gradient and the weight gradient, with the
   master weights in float32.
2. The trained layer decodes single tokens: quantise, product.
3. A mixture-of-experts block for a decode batch: router product, then the whole
   expert layer, with 16-bit and with 8-bit weights, captured in one CUDA graph.

Each part prints how far it is from the same mathematics in float32.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_fp16_tensor_gemm_gb300 as gnt  # noqa: E402


def relative(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def train_linear(tokens=2048, n_in=1024, n_out=1536, steps=3, lr=0.5):
    """Fits Y = X W^T to targets; returns the codes of the trained weights and
    their scales, and the errors of the last step's gradients."""
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    w = torch.randn(n_out, n_in, generator=g, device="cuda") * n_in ** -0.5
    target = torch.randn(n_out, n_in, generator=g, device="cuda") * n_in ** -0.5
    losses, errors = [], {}
    for _ in range(steps):
        x = torch.randn(tokens, n_in, generator=g, device="cuda").to(torch.bfloat16)
        # both orders of the weights' codes, once after each update
        q, s, qt, st = gnt.quantize_block128(w, block_rows=128, transposed=True)
        y, saved = gnt.linear_block128(x, q, s)
        dy = ((y.float() - x.float() @ target.t()) / tokens).to(torch.bfloat16)
        losses.append(float(dy.float().square().sum() * tokens / 2))
        dx, dw = gnt.linear_block128_backward(dy, saved, qt, st)
        errors = {"Y": relative(y, x.float() @ w.t()), "dX": relative(dx, dy.float() @ w),
                  "dW": relative(dw, dy.float().t() @ x.float())}
        w -= lr * dw
    gnt.gemm_nt_check(torch.cuda.current_stream().cuda_stream)
    return (*gnt.quantize_block128(w, block_rows=128), w, losses, errors)


def decode_linear(q, s, w, tokens=1):
    """Single tokens through the trained layer."""
    x = torch.randn(tokens, w.shape[1], device="cuda").to(torch.bfloat16)
    a, sa = gnt.quantize_block128(x)
    y = gnt.gemm_nt_block128_tensors(a, sa, q, s, out_dtype=torch.bfloat16)
    return relative(y, x.float() @ w.t())


def reference_experts(x, logits, w13, w2, topk):
    p, idx = torch.softmax(logits, -1).topk(topk, -1)
    p = p / p.sum(-1, keepdim=True)
    out = torch.zeros(x.shape, device="cuda")
    for t in range(x.shape[0]):
        for pj, e in zip(p[t], idx[t]):
            gate, up = (w13[e].float() @ x[t].float()).chunk(2)
            out[t] += pj * (w2[e].float() @ (torch.nn.functional.silu(gate) * up))
    return out


def experts(tokens=8, experts_=16, topk=4, hidden=1024, inner=512):
    """Router and expert layer on a decode batch, eagerly and from a graph."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)
    x, router = normal(tokens, hidden), normal(experts_, hidden, scale=hidden ** -0.5)
    w13 = normal(experts_, 2 * inner, hidden, scale=hidden ** -0.5)
    w2 = normal(experts_, hidden, inner, scale=inner ** -0.5)
    logits = torch.empty(tokens, experts_, device="cuda")
    gnt.gemm_nt(x, router, out=logits)
    ref = reference_experts(x, logits, w13, w2, topk)
    errors = {"bf16": relative(gnt.moe_few_tokens(x, logits, w13, w2, topk), ref)}

    def codes(w):
        parts = [gnt.quantize_block128(m, block_rows=128) for m in w]
        return torch.stack([q.view(torch.uint8) for q, _ in parts]).view(torch.float8_e4m3fn), \
            torch.stack([s for _, s in parts])
    (q13, s13), (q2, s2) = codes(w13), codes(w2)
    # what a decoding loop keeps: outputs, workspace and the captured step
    out = torch.empty_like(x)
    ws = torch.empty(gnt.gemm_nt_moe_workspace_bytes(tokens, topk, inner), dtype=torch.uint8, device="cuda")

    def step():
        gnt.gemm_nt(x, router, out=logits)
        gnt.moe_few_tokens(x, logits, q13, q2, topk, S13=s13, S2=s2, out=out, workspace=ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    out.zero_()
    graph.replay()
    errors["e4m3, from a graph"] = relative(out, ref)
    gnt.gemm_nt_check(torch.cuda.current_stream().cuda_stream)
    return errors


def main():
    q, s, w, losses, errors = train_linear()
    print("loss per step: " + ", ".join("%.4f" % v for v in losses))
    print("against float32: " + ", ".join("%s %.2g" % kv for kv in errors.items()))
    print("one decoded token: %.2g" % decode_linear(q, s, w))
    print("expert layer: " + ", ".join("%s %.2g" % kv for kv in experts().items()))


if __name__ == "__main__":
    main()
