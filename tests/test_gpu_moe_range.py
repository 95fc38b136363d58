"""h of the expert layer near the end of fp32's range, where the nearest bf16 value is
an infinity but h is not one: Out is W2 h, rounded."""
import pytest

import dense_fp16_tensor_gemm_gb300 as gnt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16_MAX = (2 - 2.0 ** -7) * 2.0 ** 127


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("T,I", [(1, 8), (1, 100), (40, 24)])
@pytest.mark.parametrize("eight_bits", [False, True])
def test_largest_values(T, I, sign, eight_bits):
    """gate = 64, whose silu is 64 in fp32; up = (BF16_MAX + 0.75 * 2^120) / 64 as a sum
    of two terms, so h is nearer to 2^128 than to BF16_MAX and below FLT_MAX; W2 2^-100."""
    H = 256
    parts = [BF16_MAX / 64, 0.75 * 2.0 ** 114]
    h = 64.0 * sum(parts)
    w13, w2 = torch.zeros(1, 2 * I, H), torch.zeros(1, H, I)
    s13 = s2 = None
    if eight_bits:  # 256 - 1 and 0.75 in units of 2^114
        w13[0, :I, 0], w13[0, I:, 0], w13[0, I:, 128], w13[0, I:, 1] = 64.0, 256.0 * sign, 0.75 * sign, -1.0 * sign
        w2[0, :, I - 1] = 1.0
        w13, w2 = w13.cuda().to(torch.float8_e4m3fn), w2.cuda().to(torch.float8_e4m3fn)
        s13 = torch.ones(1, 2 * I, 2)
        s13[0, I:] = 2.0 ** 114
        s13, s2 = s13.cuda(), torch.full((1, H, 1), 2.0 ** -100, device="cuda")
        assert 255 * 2.0 ** 114 == parts[0]
    else:
        w13[0, :I, 0], w13[0, I:, 0], w13[0, I:, 1] = 64.0, parts[0] * sign, parts[1] * sign
        w2[0, :, I - 1] = 2.0 ** -100
        w13, w2 = w13.cuda().to(torch.bfloat16), w2.cuda().to(torch.bfloat16)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = x[:, 1] = 1.0
    x[:, 128] = 1.0 if eight_bits else 0.0
    out = gnt.moe_few_tokens(x, torch.zeros(T, 1, device="cuda"), w13, w2, 1, S13=s13, S2=s2)
    gnt.gemm_nt_check(torch.cuda.current_stream().cuda_stream)
    want = torch.tensor(sign * h * 2.0 ** -100, dtype=torch.float64).to(torch.bfloat16)
    assert bool((out == want.item()).all()), (float(out[0, 0]), float(want))


def test_infinities_and_not_a_number_of_h_stay():
    """A product past FLT_MAX is infinite; zero weights times an infinite x are not a number."""
    H, I, inf = 64, 8, float("inf")
    w13 = torch.zeros(1, 2 * I, H, dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros(1, H, I, dtype=torch.bfloat16, device="cuda")
    w13[0, 0, 0], w13[0, I, 0], w2[0, :, 0] = 64.0, 2.0 ** 126, 1.0
    x = torch.zeros(2, H, dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[1, 0] = 1.0, inf
    out = gnt.moe_few_tokens(x, torch.zeros(2, 1, device="cuda"), w13, w2, 1)
    gnt.gemm_nt_check(torch.cuda.current_stream().cuda_stream)
    assert bool((out[0] == inf).all()) and bool(out[1].isnan().all())
