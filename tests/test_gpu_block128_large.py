"""The block-scaled product up to the largest number of rows, 2^31 - 1: the tiles at the
end are counted and stored like the others."""
import pytest

import dense_fp16_tensor_gemm_gb300 as gnt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
ONE = 0x38  # 1.0 in E4M3


def codes(rows, K, pitch):
    """Ones, but for the last 200 rows: 2 from column 1 on."""
    t = torch.full((rows * pitch,), ONE, dtype=torch.uint8, device="cuda")
    v = t.view(rows, pitch)[:, :K]
    v[-200:, 1:] = 0x40
    return v.view(F8)


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 130])
@pytest.mark.parametrize("path,K,pitch", [(gnt.Path.MMASYNC, 3, 3), (gnt.Path.SKINNY, 16, 16), (gnt.Path.TC05_PAIR, 16, 16)])
@pytest.mark.parametrize("side", ["A", "B"])
def test_as_many_rows_as_fit(rows, path, K, pitch, side):
    long, short = codes(rows, K, pitch), torch.full((2, pitch), ONE, dtype=torch.uint8, device="cuda").view(F8)[:1, :K]
    s_long, s_short = torch.ones((rows + 127) // 128, 1, device="cuda"), torch.ones(1, 1, device="cuda")
    if side == "A":
        out = gnt.gemm_nt_block128_tensors(long, s_long, short, s_short, path=path, out_dtype=torch.float16)
    else:
        out = gnt.gemm_nt_block128_tensors(short, s_short, long, s_long, path=path, out_dtype=torch.float16)
    gnt.gemm_nt_check(torch.cuda.current_stream().cuda_stream)
    out = out.view(rows)
    assert bool((out[:-200] == K).all()) and bool((out[-200:] == 2 * K - 1).all())
