"""Bounded waits of the gated product's kernels: a lost stage ends the kernel with
an error that the host reads, and the next call is right."""
import pytest
import torch

import dense_fp16_tensor_gemm_gb300 as gnt
from ffn_util import check, gated_bound, rounded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("path,tokens", [(gnt.Path.TC05_PAIR, 300)])
@pytest.mark.parametrize("fault", [1, 2])
def test_a_lost_stage_is_reported(path, tokens, fault):
    g = torch.Generator(device="cuda")
    g.manual_seed(fault)
    x = torch.randn(tokens, 2048, generator=g, device="cuda").bfloat16()
    w = (torch.randn(512, 2048, generator=g, device="cuda") / 45).bfloat16()
    gnt.gated_linear(x, w, path=path)
    gnt.gemm_nt_check()
    gnt.gemm_nt_debug_set_wait_limit(20_000_000)
    gnt.gemm_nt_debug_set_fault(fault)
    try:
        gnt.gated_linear(x, w, path=path)
    finally:
        gnt.gemm_nt_debug_set_fault(0)
    with pytest.raises(gnt.GemmError) as e:
        gnt.gemm_nt_check()
    gnt.gemm_nt_debug_set_wait_limit(0)
    assert e.value.status == gnt.Status.DEVICE_TIMEOUT
    h, _, err, _ = gated_bound(x, w, "silu")
    check(gnt.gated_linear(x, w, path=path), h, rounded(err, h, x.dtype))
    gnt.gemm_nt_check()
