"""What the few-token expert layer refuses, beyond its other argument checks (all on
the host, no GPU)."""
import pytest

import dense_fp16_tensor_gemm_gb300 as gnt
from test_block128_abi import S13, S2, SA, SB, lib, moe, scale  # noqa: F401

D, Status = gnt.DType, gnt.Status


@pytest.mark.parametrize("ws", [SA, SB])
def test_workspace_over_the_scales(lib, ws):  # noqa: F811
    """The workspace is written before S2 is read."""
    assert moe(lib, wt=D.E4M3, s13=S13, s2=S2, ws=ws) == Status.OVERLAP
    # the last byte of the workspace on the first scale, and right behind it
    need = gnt.gemm_nt_moe_workspace_bytes(4, 2, 128)
    assert moe(lib, wt=D.E4M3, s13=S13, s2=S2, ws=ws - need + 16, nbytes=need) == Status.OVERLAP
    assert moe(lib, wt=D.E4M3, s13=S13, s2=S2, ws=ws - need, nbytes=need) != Status.OVERLAP
