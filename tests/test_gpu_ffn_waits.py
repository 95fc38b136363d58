"""Bounded waits of the gated product's kernels: a lost stage ends the kernel with
an error that the host reads, and the next call is right."""
import pytest
import torch

import dense_fp16_tensor_gemm_gb300 as gnt
from ffn_util import check, gated_bound, rounded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("path,tokens", [(gnt.Path.TC05_PAIR, 300), (gnt.Path.TC05, 64)])
@pytest.mark.parametrize("fault", [1, 2])
def test_a_lost_stage_is_reported(path, tokens, fault):
    g = torch.Generator(device="cuda")
    g.manual_seed(fault)
    x = torch.randn(tokens, 8192, generator=g, device="cuda").bfloat16()  # K is longer than the ring, split or not
    w = (torch.randn(512, 8192, generator=g, device="cuda") / 90).bfloat16()
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


@pytest.mark.parametrize("tokens,rows", [(64, 256), (300, 20000)])  # a split of K, whole tiles
@pytest.mark.parametrize("fault", [1, 2])
def test_a_lost_stage_of_codes_is_reported(tokens, rows, fault):
    g = torch.Generator(device="cuda")
    g.manual_seed(fault)
    x = torch.randn(tokens, 16384, generator=g, device="cuda").half()  # an eighth of K is longer than the ring
    q, s = gnt.quantize_w4(torch.randn(rows, 16384, generator=g, device="cuda") / 128, scale_dtype=torch.half)
    good = gnt.linear_w4(x, q, s, path=gnt.Path.TC05)
    gnt.gemm_nt_check()
    gnt.gemm_nt_debug_set_wait_limit(20_000_000)
    gnt.gemm_nt_debug_set_fault(fault)
    try:
        gnt.linear_w4(x, q, s, path=gnt.Path.TC05)
    finally:
        gnt.gemm_nt_debug_set_fault(0)
    with pytest.raises(gnt.GemmError) as e:
        gnt.gemm_nt_check()
    gnt.gemm_nt_debug_set_wait_limit(0)
    assert e.value.status == gnt.Status.DEVICE_TIMEOUT
    assert torch.equal(gnt.linear_w4(x, q, s, path=gnt.Path.TC05), good)
    gnt.gemm_nt_check()
