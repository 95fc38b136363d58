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


@pytest.mark.parametrize("change,status", [
    (dict(k=17), Status.INVALID_VALUE),
    (dict(H=2 ** 20 + 1, ldx=2 ** 20 + 1, ldo=2 ** 20 + 1, ldw13=2 ** 20 + 1, sw13=0), Status.NOT_SUPPORTED),
    (dict(I=2 ** 20 + 1, ldw2=2 ** 20 + 1, sw2=0, w13=1 << 40, w2=1 << 44), Status.NOT_SUPPORTED),
])
def test_documented_limits(lib, change, status):  # noqa: F811
    assert moe(lib, x=1 << 50, l=1 << 51, out=1 << 52, ws=1 << 53, nbytes=1 << 40, **change) == status


def test_without_inner_columns_no_limit_applies(lib):  # noqa: F811
    """Good arguments fail for want of a device only."""
    never = (Status.OK, Status.INVALID_VALUE, Status.OVERLAP, Status.NOT_SUPPORTED)
    assert moe(lib, I=0, w13=0, w2=0, ws=0, nbytes=0, T=500, E=2000, ldl=2000, k=40, x=1 << 50, out=1 << 52) not in never


def test_workspace_bytes_that_do_not_fit():
    """The number of bytes, or -1: never one that wrapped around."""
    f = gnt.gemm_nt_moe_workspace_bytes
    assert f(128, 32, 2 ** 20) == 128 * 32 * 2 ** 20 * 4
    assert f(2 ** 31, 2 ** 31, 1) == -1 and f(2 ** 30, 2 ** 30, 2 ** 30) == -1
    assert f(1, 1, 2 ** 63 - 1) == -1 and f(2 ** 62, 1, 1) == -1
    assert f(2 ** 27, 2 ** 27, 1) == 2 ** 60 and f(0, 2 ** 62, 2 ** 62) == 0


@pytest.mark.gpu
def test_nothing_is_allocated_for_what_is_refused():
    """A workspace for a billion experts a token is not asked of the allocator."""
    torch = pytest.importorskip("torch")
    x, logits = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 4, device="cuda")
    w13, w2 = (torch.zeros(*s, dtype=torch.bfloat16, device="cuda") for s in ((4, 32, 64), (4, 64, 16)))
    for topk, status in ((10 ** 9, Status.INVALID_VALUE), (2 ** 62, Status.INVALID_VALUE), (0, Status.INVALID_VALUE)):
        with pytest.raises(gnt.GemmError) as e:
            gnt.moe_few_tokens(x, logits, w13, w2, topk)
        assert e.value.status == status
