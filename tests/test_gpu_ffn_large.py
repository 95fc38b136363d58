"""Offsets past 32 bits in the gated and 4-bit operators: rows that lie far apart,
and outputs of more than 2^31 elements (on the GPU)."""
import pytest

import dense_fp16_tensor_gemm_gb300 as gnt
from ffn_util import EPS, check, gated_bound, rounded, sum_error, w4_values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
P = gnt.Path


def far(rows, cols, dtype, g, scale=1.0):
    """A matrix whose rows lie 128 MB apart."""
    pitch = (128 << 20) // torch.empty(0, dtype=dtype).element_size()
    out = torch.empty(rows * pitch, dtype=dtype, device="cuda").view(rows, pitch)[:, :cols]
    if dtype == torch.uint8:
        out.copy_(torch.randint(0, 256, (rows, cols), generator=g, device="cuda", dtype=dtype))
    else:
        out.copy_(torch.randn(rows, cols, generator=g, device="cuda") * scale)
    return out


@pytest.mark.parametrize("path,m", [(P.SKINNY, 3), (P.TC05, 40), (P.TC05_PAIR, 40), (P.MMASYNC, 40)])
def test_rows_far_apart(path, m):
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    x, n, k = far(m, 520, BF16, g), 24, 520
    w = far(2 * n, k, BF16, g, k ** -0.5)
    out = far(m, n, BF16, g)
    h, _, eh, _ = gated_bound(x, w, "silu")
    gnt.gated_linear(x, w, out=out, path=path)
    check(out, h, rounded(eh, h, BF16))
    del w
    if path != P.TC05_PAIR:
        q, s = far(n, (k + 1) // 2, torch.uint8, g), (torch.rand(n, 5, generator=g, device="cuda") / 100).to(BF16)
        z = torch.randint(0, 16, (n, 5), generator=g, device="cuda", dtype=torch.uint8)
        v = w4_values(q, s, z, 128, k)
        ref, mag = x.double() @ v.t(), x.double().abs() @ v.abs().t()
        wide = x.double().abs() @ (v.abs() + 31 * s.double()[:, torch.arange(k, device="cuda") // 128]).t()
        gnt.linear_w4(x, q, s, z, out=out, path=path)
        check(out, ref, rounded(sum_error(wide, k) + EPS[BF16] * (path == P.TC05) * mag, ref, BF16))
    gnt.gemm_nt_check()


@pytest.mark.parametrize("op", ["gated", "w4", "backward"])
def test_more_than_2_to_the_31_outputs(op):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    m, k, n = 70001, 64, 32768  # 2.29e9 elements
    x = torch.randn(m, k, generator=g, device="cuda").to(BF16)
    rows = torch.tensor([0, 1, 255, 256, 32767, 65535, 65537, 69999, 70000], device="cuda")
    if op == "gated":
        w = (torch.randn(2 * n, k, generator=g, device="cuda") / 8).to(BF16)
        out = gnt.gated_linear(x, w)
        h, _, eh, _ = gated_bound(x[rows], w, "silu")
        check(out[rows], h, rounded(eh, h, BF16))
    elif op == "w4":
        q = torch.randint(0, 256, (n, 32), generator=g, device="cuda", dtype=torch.uint8)
        s = (torch.rand(n, 1, generator=g, device="cuda") / 50).to(BF16)
        v = w4_values(q, s, None, 128, k)
        ref, mag = x[rows].double() @ v.t(), x[rows].double().abs() @ v.abs().t()
        out = gnt.linear_w4(x, q, s)
        check(out[rows], ref, rounded(sum_error(mag, k) + EPS[BF16] * mag, ref, BF16))
    else:
        n = 16400  # [g u] and its gradient hold 2.3e9 elements each
        gu = torch.empty(m, 2 * n, dtype=BF16, device="cuda").normal_(generator=g)
        dh = torch.empty(m, n, dtype=BF16, device="cuda").normal_(generator=g)
        d = torch.empty_like(gu)
        gnt.gemm_nt_gated_grad(dh.data_ptr(), n, gu.data_ptr(), 2 * n, d.data_ptr(), 2 * n, 1, 0, m, n,
                               torch.cuda.current_stream().cuda_stream)
        gate, up, t = gu[rows, :n].double(), gu[rows, n:].double(), dh[rows].double()
        p = torch.sigmoid(gate)
        ref = torch.cat((t * up * (p + gate * p * (1 - p)), t * gate * p), 1)
        err = 2.0 ** -19 * torch.cat(((t * up).abs() * (1 + gate.abs()), (t * gate).abs()), 1)
        check(d[rows], ref, rounded(err, ref, BF16))
    gnt.gemm_nt_check()


@pytest.mark.parametrize("op", ["tokens", "outputs"])
def test_as_many_rows_as_an_int_counts(op):
    """2^31 - 1 tokens, and 2^31 - 1 rows of 4-bit weights, with sums of one element."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    many = 2 ** 31 - 1
    rows = torch.tensor([0, 1, 63, 64, 2 ** 30, many - 65, many - 64, many - 63, many - 1], device="cuda")
    if op == "tokens":
        x = torch.empty(many, 1, dtype=BF16, device="cuda").normal_(generator=g)
        w = torch.randn(2, 1, generator=g, device="cuda").to(BF16)
        out = torch.empty(many, 1, dtype=BF16, device="cuda")
        gnt.gated_linear(x, w, out=out, path=P.MMASYNC)
        h, _, eh, _ = gated_bound(x[rows], w, "silu")
        check(out[rows], h, rounded(eh, h, BF16))
    else:
        x = torch.randn(1, 1, generator=g, device="cuda").to(BF16)
        q = torch.empty(many, 1, dtype=torch.uint8, device="cuda").random_(0, 256, generator=g)
        s = torch.empty(many, 1, dtype=BF16, device="cuda").uniform_(0.01, 1, generator=g)
        out = gnt.linear_w4(x, q, s, path=P.MMASYNC)[:, rows]
        v = w4_values(q[rows], s[rows], None, 128, 1)
        ref, mag = x.double() @ v.t(), x.double().abs() @ v.abs().t()
        check(out, ref, rounded(sum_error(mag, 1), ref, BF16))
    gnt.gemm_nt_check()
