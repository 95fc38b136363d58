"""The 8-bit layers and the expert layer on nothing: no tokens, no columns, no batch."""
import pytest

import dense_fp16_tensor_gemm_gb300 as gnt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


def codes(*shape):
    return torch.zeros(*shape, dtype=torch.uint8, device="cuda").view(F8)


def scales(*shape):
    return torch.ones(*shape, device="cuda")


def test_linear_step_without_tokens():
    """The weights' gradient is zero, the others are empty."""
    n_in, n_out = 256, 136
    x = torch.empty(0, n_in, dtype=torch.bfloat16, device="cuda")
    y, saved = gnt.linear_block128(x, codes(n_out, n_in), scales(2, 2))
    dx, dw = gnt.linear_block128_backward(y, saved, codes(n_in, n_out), scales(2, 2))
    gnt.gemm_nt_check(torch.cuda.current_stream().cuda_stream)
    assert y.shape == (0, n_out) and dx.shape == (0, n_in)
    assert dw.shape == (n_out, n_in) and bool((dw == 0).all())


@pytest.mark.parametrize("shape", [(0, 300), (300, 0), (0, 0)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantise_nothing(shape, block_rows):
    q, s, qt, st = gnt.quantize_block128(torch.empty(shape, device="cuda"), block_rows=block_rows, transposed=True)
    assert q.shape == shape and qt.shape == shape[::-1]
    rows = [n if block_rows == 1 else -(-n // 128) for n in shape]
    assert s.shape == (rows[0], -(-shape[1] // 128)) and st.shape == (rows[1], -(-shape[0] // 128))


@pytest.mark.parametrize("M,N", [(0, 5), (5, 0)])
def test_products_without_rows(M, N):
    out = gnt.gemm_nt_block128_tensors(codes(M, 256), scales(M, 2), codes(N, 256), scales(N, 2))
    assert out.shape == (M, N)
    out = gnt.gemm_nt_block128_tensors(codes(0, 4, 256), scales(0, 4, 2), codes(0, 3, 256), scales(0, 3, 2))
    assert out.shape == (0, 4, 3)


def test_experts_without_tokens_or_columns():
    for T, H in ((0, 64), (3, 0)):
        out = gnt.moe_few_tokens(*(torch.zeros(*s, dtype=d, device="cuda") for s, d in (
            ((T, H), torch.bfloat16), ((T, 4), torch.float32), ((4, 32, H), torch.bfloat16),
            ((4, H, 16), torch.bfloat16))), 2)
        assert out.shape == (T, H)
    gnt.gemm_nt_check(torch.cuda.current_stream().cuda_stream)
