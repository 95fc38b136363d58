"""The expert layer without inner columns: Out is zero, wherever its rows lie, and
nothing beside it is touched."""
import pytest

import dense_fp16_tensor_gemm_gb300 as gnt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,pitch", [(1, 64), (3, 64), (300, 70), (2, 2 ** 30 + 8), (3, 2 ** 30), (1, 2 ** 31 + 8)])
def test_no_inner_columns(T, pitch):
    H, E = 64, 4
    x = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    logits = torch.full((T, E), float("nan"), device="cuda")
    w13, w2 = (torch.empty(*s, dtype=torch.bfloat16, device="cuda") for s in ((E, 0, H), (E, H, 0)))
    buf = torch.full(((T - 1) * pitch + H + 6,), 5.0, dtype=torch.bfloat16, device="cuda")
    out = buf.as_strided((T, H), (pitch, 1))
    gnt.moe_few_tokens(x, logits, w13, w2, 2, out=out)
    gnt.gemm_nt_check(torch.cuda.current_stream().cuda_stream)
    assert bool((out == 0).all())
    assert int((buf != 5).sum()) == T * H
