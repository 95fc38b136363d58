"""More tiles than the GPU takes at once, and sums longer than the kernels' rings: every CTA goes
on from tile to tile with its rings, accumulators and barriers as the last one left them, an odd
number of stages at a time (on the GPU, against 64 bits).

4-bit weights are compared with what each kernel is to multiply: (code - zero) * scale, or on
tcgen05 that rounded to the tokens' type, so that a bound is the sums' and the output's rounding
and nothing else."""
import pytest
import torch

import dense_fp16_tensor_gemm_gb300 as gnt
from ffn_util import check, gated_bound, rounded, sum_error, w4_values
from test_gpu_ffn import gen, normal, weights4

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
P = gnt.Path


def check_gated(path, m, k, n, dtype, act, extra=0):
    g = gen(m + k + n)
    x = normal(g, m, k, dtype=dtype, pitch=(k + 7) // 8 * 8 + extra)
    w = normal(g, 2 * n, k, scale=k ** -0.5, dtype=dtype, pitch=(k + 7) // 8 * 8 + extra)
    out, gu = gnt.gated_linear(x, w, act, keep=True, path=path)
    assert torch.equal(gnt.gated_linear(x, w, act, path=path), out)
    h, y, eh, ey = gated_bound(x, w, act)
    check(out, h, rounded(eh, h, dtype))
    check(gu, y, rounded(ey, y, dtype), "gu")
    gnt.gemm_nt_check()


def check_w4(path, m, k, n, dtype, group, zeros, act=None, pitch=0, extra=0):
    g = gen(m + k + n)
    x = normal(g, m, k, dtype=dtype, pitch=(k + 7) // 8 * 8 + extra)
    q, s, z = weights4(g, n if act is None else 2 * n, k, group, zeros, dtype, pitch)
    w = w4_values(q, s, z, group, k)
    if path == P.TC05:
        w = w.to(dtype).double()  # (a product of 4 bits and 8 or 11: rounded once)
    if act is None:
        ref = x.double() @ w.t()
        bound = sum_error(x.double().abs() @ w.abs().t(), k)
        out = gnt.linear_w4(x, q, s, z, group=group, path=path)
    else:
        ref, _, bound, _ = gated_bound(x, w, act)
        out = gnt.gated_linear_w4(x, q, s, z, group=group, activation=act, path=path)
    check(out, ref, rounded(bound, ref, dtype))
    gnt.gemm_nt_check()


@pytest.mark.parametrize("m,k,n,dtype,act", [(1, 1000, 8200, BF16, "silu"), (7, 1000, 8200, F16, "gelu"),
                                             (12, 1032, 8200, BF16, "gelu_tanh"), (16, 4096, 4100, F16, "silu")])
def test_gated_stream(m, k, n, dtype, act):
    """Up to 456 CTAs take tiles of 8 outputs."""
    check_gated(P.SKINNY, m, k, n, dtype, act)


@pytest.mark.parametrize("m,k,n,dtype,act", [(40, 1032, 20000, BF16, "silu"), (30, 1032, 20008, F16, "gelu_tanh"),
                                             (64, 2056, 19999, BF16, "gelu"), (3, 72, 20000, F16, "silu")])
def test_gated_single_ctas(m, k, n, dtype, act):
    """152 CTAs, 313 tiles of 64 outputs, two accumulators in turns."""
    check_gated(P.TC05, m, k, n, dtype, act)


@pytest.mark.parametrize("m,k,n,dtype,act", [(1000, 1032, 5000, BF16, "silu"), (2100, 584, 3001, F16, "gelu"),
                                             (65, 8200, 20000, BF16, "gelu_tanh")])
def test_gated_pairs(m, k, n, dtype, act):
    """76 pairs, 157 tiles and more of 256 x 128, six stages for 17, 10 and 129 k-blocks."""
    check_gated(P.TC05_PAIR, m, k, n, dtype, act)


@pytest.mark.parametrize("extra", [0, 1])
def test_any_layout(extra):
    """1216 CTAs, 3008 and 6000 tiles."""
    check_gated(P.MMASYNC, 1000, 200, 6001, BF16, "silu", extra)
    check_w4(P.MMASYNC, 1000, 200, 12000, F16, 32, True, pitch=101 + 10 * extra, extra=extra)
    check_w4(P.MMASYNC, 1000, 333, 6000, BF16, 128, False, "gelu", pitch=167 + 10 * extra, extra=extra)


@pytest.mark.parametrize("dtype,group,zeros", [(BF16, 128, True), (F16, 64, False), (BF16, 32, False)])
@pytest.mark.parametrize("m,k", [(1, 1000), (7, 1030), (12, 700), (5, 8192)])
def test_stream_of_codes(m, k, dtype, group, zeros):
    check_w4(P.SKINNY, m, k, 20000, dtype, group, zeros)
    check_w4(P.SKINNY, m, k, 8200, dtype, group, zeros, "silu")


@pytest.mark.parametrize("dtype,group,zeros", [(BF16, 128, False), (F16, 64, True), (BF16, 32, True), (F16, 128, True)])
@pytest.mark.parametrize("m", [30, 60, 128, 600])
@pytest.mark.parametrize("k", [700, 1030, 2050])
def test_codes_on_single_ctas(k, m, dtype, group, zeros):
    """152 CTAs, more than twice as many tiles; 3, 5 and 9 stages of codes to a tile in rings of
    3, 5 and 6."""
    check_w4(P.TC05, m, k, 40000 if m <= 256 else 13100, dtype, group, zeros)
    check_w4(P.TC05, m, k, 20000 if m <= 256 else 6600, dtype, group, zeros, "gelu_tanh")


@pytest.mark.parametrize("m", [40, 65, 128, 300])
@pytest.mark.parametrize("n", [4096, 12000])
def test_long_rings_of_codes(n, m):
    """79 stages of codes to a tile: whole tiles, and K split over clusters."""
    check_w4(P.TC05, m, 20000, n, BF16, 128, False)
    check_w4(P.TC05, m, 20000, n // 2, F16, 32, True, "silu")


@pytest.mark.parametrize("path", [P.SKINNY, P.TC05, P.MMASYNC])
@pytest.mark.parametrize("at", [0, 5998, 5999])
def test_the_bounds_see_one_element_of_a_long_sum(path, at):
    """What the checks above rest on: 64 bits with one element of 6000 left out are not taken
    for a kernel's sums."""
    g = gen(4)
    m, k, n = 8, 6000, 500
    x = normal(g, m, k, dtype=F16)
    q, s, _ = weights4(g, n, k, 128, False, F16)
    w = w4_values(q, s, None, 128, k)
    if path == P.TC05:
        w = w.to(F16).double()
    out = gnt.linear_w4(x, q, s, path=path)
    ref, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    check(out, ref, rounded(sum_error(mag, k), ref, F16))
    x[:, at] = 0
    less = x.double() @ w.t()
    with pytest.raises(AssertionError):
        check(out, less, rounded(sum_error(mag, k), less, F16))
