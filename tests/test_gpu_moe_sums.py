"""Long sums of the expert layer carry no bias.

All terms are positive, so that every rounding towards zero of a running sum shows
as a result that is too small, and the mean relative deviation over N outputs is
compared with what the arithmetic allows.  An item of 64 elements of K is a chain
of m MMAs (4 for x; for h in two parts 8, in tf32 16), each of which cuts off less
than a unit in the last place of its sum, 2^-23 of it, and of its products as much
again: m * 2^-22 for an item, and no more for a sum of items, which are added to
nearest in fp32.  Those additions wander without direction: over 1024 items, 2^-20
covers their mean.  h takes two such sums, Out one.  The last rounding adds up to
u = 2^-10 (fp16) or 2^-7 (bf16) to an output, u / sqrt(12) in the mean square, and
1 / sqrt(N) of that to the mean; six times it is allowed.  Outputs are compared with
the exact values rounded to their type: where many lie around a power of two that
rounding itself has a mean, of 1.9e-5 in the third case.
"""
import pytest

import dense_fp16_tensor_gemm_gb300 as gnt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,T,H,I", [
    (torch.float16, 1, 65536, 64), (torch.float16, 16, 65536, 64), (torch.bfloat16, 16, 65536, 64),  # the first product
    (torch.float16, 8, 4096, 65536), (torch.float16, 16, 4096, 65536),                              # the second
    (torch.float16, 16, 2056, 1000)])
def test_long_positive_sums(dtype, T, H, I):
    g = torch.Generator(device="cuda")
    g.manual_seed(T + H)

    def positive(*shape, scale=1.0):
        return ((torch.rand(*shape, generator=g, device="cuda") + 0.5) * scale).to(dtype)
    x, w13, w2 = positive(T, H), positive(1, 2 * I, H, scale=16 / H), positive(1, H, I, scale=16 / I)
    out = gnt.moe_few_tokens(x, torch.zeros(T, 1, device="cuda"), w13, w2, 1)
    gnt.gemm_nt_check(torch.cuda.current_stream().cuda_stream)
    gate, up = (x.double() @ w13[0].double().t()).chunk(2, -1)
    ref = (gate * torch.sigmoid(gate) * up) @ w2[0].double().t()
    bias = float(((out.double() - ref.to(dtype).double()) / ref).mean())
    chain, ulp = (16, 2.0 ** -10) if dtype == torch.float16 else (8, 2.0 ** -7)
    limit = (2 * 4 + chain) * 2.0 ** -22 + 2.0 ** -20 + 6 * ulp / (12 * out.numel()) ** 0.5
    assert abs(bias) <= limit, "mean deviation %.3g, %.3g allowed" % (bias, limit)
