"""A gated feed-forward block, from a training step to decoding in 4 bits.

    python examples/feed_forward.py

1. A few steps of gradient descent on the block Y = (act(X Wg^T) * (X Wu^T)) W2^T: the
   fused first half, which keeps what the backward pass needs, the second product, and
   the gradients of X, W13 and W2, with the master weights in float32.
2. Both weights quantised to 4 bits, and single tokens decoded with them from one CUDA
   graph.

Each part prints how far it is from the same mathematics in float32.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_fp16_tensor_gemm_gb300 as gnt  # noqa: E402

BF16 = torch.bfloat16
K, MN = gnt.Major.K, gnt.Major.MN


def relative(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def product(a, a_major, b, b_major, m, n, k):
    """An (m, n) bf16 product of two operands as they lie."""
    out = torch.empty(m, n, dtype=BF16, device="cuda")
    gnt.gemm_nt_batched_major(a.data_ptr(), a_major, b.data_ptr(), b_major, out.data_ptr(), gnt.DType.BF16, gnt.DType.BF16,
                              m, n, k, a.stride(0), b.stride(0), n, 0, 0, 0, 1, 0, torch.cuda.current_stream().cuda_stream)
    return out


def forward(x, w13, w2):
    h, gu = gnt.gated_linear(x, w13, keep=True)
    return gnt.gemm_nt(h, w2, out_dtype=BF16), h, gu


def backward(dy, h, gu, x, w13, w2):
    tokens, hidden = x.shape
    inner = h.shape[1]
    dh = product(dy, K, w2, MN, tokens, inner, hidden)
    dw2 = product(dy, MN, h, MN, hidden, inner, tokens)
    dx, dw13 = gnt.gated_linear_backward(dh, gu, x, w13)
    return dx, dw13, dw2


def train(tokens=1024, hidden=512, inner=1376, steps=3, lr=0.02):
    """Returns the trained weights, and the last step's errors against float32."""
    g = torch.Generator(device="cuda")
    g.manual_seed(0)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale
    m13, m2 = normal(2 * inner, hidden, scale=hidden ** -0.5), normal(hidden, inner, scale=inner ** -0.5)
    errors = {}
    for _ in range(steps):
        x, target = normal(tokens, hidden).to(BF16), normal(tokens, hidden)
        w13, w2 = m13.to(BF16), m2.to(BF16)
        y, h, gu = forward(x, w13, w2)
        dy = ((y.float() - target) / tokens).to(BF16)
        dx, dw13, dw2 = backward(dy, h, gu, x, w13, w2)
        # the same in float32
        leaves = [t.float().requires_grad_() for t in (x, w13, w2)]
        gate, up = (leaves[0] @ leaves[1].t()).chunk(2, 1)
        ref = (gate * torch.sigmoid(gate) * up) @ leaves[2].t()
        ref.backward(dy.float())
        errors = {"Y": relative(y, ref.detach()), "dX": relative(dx, leaves[0].grad),
                  "dW13": relative(dw13, leaves[1].grad), "dW2": relative(dw2, leaves[2].grad)}
        m13 -= lr * dw13.float()
        m2 -= lr * dw2.float()
    gnt.gemm_nt_check(torch.cuda.current_stream().cuda_stream)
    return m13, m2, errors


def decode(w13, w2, tokens=1):
    """Tokens through the block in 4 bits, replayed from a graph; the error against float32
    weights."""
    x = torch.randn(tokens, w13.shape[1], device="cuda").to(BF16)
    q13, s13, z13 = gnt.quantize_w4(w13, group=64, zeros=True)
    q2, s2, z2 = gnt.quantize_w4(w2, group=64, zeros=True)
    h = torch.empty(tokens, w2.shape[1], dtype=BF16, device="cuda")
    y = torch.empty(tokens, w2.shape[0], dtype=BF16, device="cuda")

    def step():
        gnt.gated_linear_w4(x, q13, s13, z13, group=64, out=h)
        gnt.linear_w4(h, q2, s2, z2, group=64, out=y)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    y.zero_()
    graph.replay()
    gnt.gemm_nt_check(torch.cuda.current_stream().cuda_stream)
    gate, up = (x.float() @ w13.t()).chunk(2, 1)
    return relative(y, (gate * torch.sigmoid(gate) * up) @ w2.t())


def main():
    w13, w2, errors = train()
    print("training step against float32: " + ", ".join("%s %.2g" % kv for kv in errors.items()))
    print("one token in 4 bits: %.2g" % decode(w13, w2))


if __name__ == "__main__":
    main()
