"""The expert layer's one wait, for a warp's turn to add to a CTA's sums, runs out: the
status says so, and the next call is right."""
import pytest

import dense_fp16_tensor_gemm_gb300 as gnt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_gpu_moe as moe  # noqa: E402


@pytest.mark.parametrize("wt", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("T,E,k,H,I", [(64, 4, 2, 64, 4096), (128, 16, 4, 512, 1024)])
def test_a_turn_that_does_not_come_in_time(wt, T, E, k, H, I):
    """A limit of one cycle: eight warps start together, and all but one wait longer."""
    g = moe.gen(T)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device="cuda")
    w13, w2, s13, s2, d13, d2 = moe.weights(g, E, H, I, wt)
    stream = torch.cuda.current_stream().cuda_stream
    gnt.gemm_nt_check(stream)
    gnt.gemm_nt_debug_set_wait_limit(1)
    try:
        gnt.moe_few_tokens(x, logits, w13, w2, k, S13=s13, S2=s2)
        with pytest.raises(gnt.GemmError) as e:
            gnt.gemm_nt_check(stream)
        assert e.value.status == gnt.Status.DEVICE_TIMEOUT
    finally:
        gnt.gemm_nt_debug_set_wait_limit(0)
    gnt.gemm_nt_check(stream)
    moe.check(moe.run(x, logits, w13, w2, k, s13, s2), *moe.reference(x, logits, d13, d2, k, True))
