"""Infinities and NaN in tokens, weights and scales on every kernel of the gated and 4-bit products:
they reach what they belong to as in IEEE arithmetic, and nothing beside it (on the GPU)."""
import math

import pytest
import torch

import dense_fp16_tensor_gemm_gb300 as gnt
from ffn_util import ACTS, EPS, check, gated_bound, rounded, sum_error, w4_values
from test_gpu_ffn import gen, normal, weights4

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
P = gnt.Path
INF, NAN = math.inf, math.nan
# Columns end inside a tile of the weights and a step of K; on tcgen05 tiles of 32, 64, 128 and
# 256 tokens, with K split over clusters and not.
KERNELS = [(P.SKINNY, 1, 200, 100), (P.SKINNY, 7, 200, 100), (P.SKINNY, 16, 1000, 36), (P.TC05, 20, 200, 100),
           (P.TC05, 50, 2056, 72), (P.TC05, 40, 72, 20000), (P.MMASYNC, 40, 201, 100)]
GATED = KERNELS + [(P.TC05_PAIR, 70, 200, 100), (P.TC05_PAIR, 300, 1032, 520)]
CODES = KERNELS + [(P.TC05, 100, 2056, 72), (P.TC05, 300, 200, 100)]


def same(out, ref, bound, what=""):
    """NaN where the formula has it, its infinities, and the rest within the bound."""
    out = out.double()
    assert torch.equal(out.isnan(), ref.isnan()), what
    far = ref.isinf()
    assert torch.equal(out[far], ref[far]), what
    fine = ref.isfinite()
    check(out[fine], ref[fine], bound[fine], what)


def spoil(x, rows, cols):
    """An infinity of either sign, a NaN, and two infinities that cancel, each in a row of its own
    as far as there are rows."""
    for i, (r, c) in enumerate(zip(rows, cols)):
        x[r, c] = (INF, -INF, NAN, INF)[i]
        if i == 3:
            x[r, c - 1] = -INF


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("path,m,k,n", GATED)
def test_gated_tokens(path, m, k, n, dtype):
    g = gen(m + k)
    x, w = normal(g, m, k, dtype=dtype, pitch=(k + 7) // 8 * 8), normal(g, 2 * n, k, scale=k ** -0.5, dtype=dtype,
                                                                      pitch=(k + 7) // 8 * 8)
    w[3, k - 1] = w[n + 5, k - 1] = 0  # (infinity times zero)
    spoil(x, range(0, m, max(1, m // 4)), [k - 1, 0, k // 2, k - 1])
    finite = x.nan_to_num(0, 0, 0)
    for act in ACTS:
        out, gu = gnt.gated_linear(x, w, act, keep=True, path=path)
        h, y, _, _ = gated_bound(x, w, act)
        # (bounds of the finite ones, which have no such term)
        h0, y0, eh, ey = gated_bound(finite, w, act)
        same(out, h, rounded(eh, h0, dtype), act)
        same(gu, y, rounded(ey, y0, dtype), act + " gu")
    gnt.gemm_nt_check()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("path,m,k,n", GATED)
def test_gated_weights(path, m, k, n, dtype):
    g = gen(m + k)
    x, w = normal(g, m, k, dtype=dtype, pitch=(k + 7) // 8 * 8), normal(g, 2 * n, k, scale=k ** -0.5, dtype=dtype,
                                                                      pitch=(k + 7) // 8 * 8)
    x[0, k - 1] = 0
    spoil(w, [n - 1, 0, 2 * n - 1, n + 2], [k - 1, 0, k // 2, k - 1])
    finite = w.nan_to_num(0, 0, 0)
    out, gu = gnt.gated_linear(x, w, keep=True, path=path)
    h, y, _, _ = gated_bound(x, w, "silu")
    h0, y0, eh, ey = gated_bound(x, finite, "silu")
    same(out, h, rounded(eh, h0, dtype))
    same(gu, y, rounded(ey, y0, dtype), "gu")
    gnt.gemm_nt_check()


@pytest.mark.parametrize("dtype,group,zeros", [(BF16, 128, False), (F16, 32, True), (BF16, 64, True)])
@pytest.mark.parametrize("path,m,k,n", CODES)
def test_tokens_with_codes(path, m, k, n, dtype, group, zeros):
    g = gen(m + k)
    x = normal(g, m, k, dtype=dtype, pitch=(k + 7) // 8 * 8)
    q, s, z = weights4(g, 2 * n, k, group, zeros, dtype)
    spoil(x, range(0, m, max(1, m // 4)), [k - 1, 0, k // 2, k - 1])
    finite = x.nan_to_num(0, 0, 0).double()
    w = w4_values(q, s, z, group, k)
    if path == P.TC05:
        w = w.to(dtype).double()
    y, y0 = x.double() @ w.t(), finite @ w.t()
    same(gnt.linear_w4(x, q, s, z, group=group, path=path), y, rounded(sum_error(finite.abs() @ w.abs().t(), k), y0, dtype))
    h, _, _, _ = gated_bound(x, w, "silu")
    h0, _, eh, _ = gated_bound(finite, w, "silu")
    same(gnt.gated_linear_w4(x, q, s, z, group=group, path=path), h, rounded(eh, h0, dtype))
    gnt.gemm_nt_check()


@pytest.mark.parametrize("dtype,group,zeros", [(BF16, 128, False), (F16, 32, True), (BF16, 64, True)])
@pytest.mark.parametrize("path,m,k,n", CODES)
def test_scales(path, m, k, n, dtype, group, zeros):
    """An infinite or NaN scale makes its row's sums NaN or infinite, those of a token of zeros too,
    and no other row's."""
    g = gen(m + k)
    x = normal(g, m, k, dtype=dtype, pitch=(k + 7) // 8 * 8)
    x[m // 2] = 0
    q, s, z = weights4(g, 2 * n, k, group, zeros, dtype)
    bad = torch.tensor([0, 17, n - 1, n + 1, 2 * n - 1], device="cuda")
    w = w4_values(q, s, z, group, k)
    if path == P.TC05:
        w = w.to(dtype).double()
    s[bad, torch.tensor([0, -1, -1, 0, -1])] = torch.tensor([INF, NAN, INF, NAN, INF], device="cuda").to(dtype)
    ref, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    out = gnt.linear_w4(x, q, s, z, group=group, path=path)
    good = torch.ones(2 * n, dtype=torch.bool, device="cuda")
    good[bad] = False
    assert not out[:, bad].isfinite().any()
    check(out[:, good], ref[:, good], rounded(sum_error(mag, k), ref, dtype)[:, good])
    out = gnt.gated_linear_w4(x, q, s, z, group=group, path=path)
    h, _, eh, _ = gated_bound(x, w, "silu")
    good = good[:n] & good[n:]
    assert not out[:, ~good].isfinite().any()
    check(out[:, good], h[:, good], rounded(eh, h, dtype)[:, good])
    gnt.gemm_nt_check()


def test_weights_beyond_fp16():
    """What the header says of it: exact sums stay finite, weights rounded to fp16 become infinite."""
    k, n = 256, 40
    x = torch.full((20, k), 2.0 ** -10, device="cuda", dtype=F16)
    q = torch.full((n, k // 2), 0xff, dtype=torch.uint8, device="cuda")  # 15: 7 steps above 8
    s = torch.full((n, 2), 8192.0, device="cuda", dtype=F16)
    s[1::2] = 9600.0                                                      # 67200, above 65504
    want = (7 * s[:, 0].double() * 2.0 ** -10 * k).expand(20, n)
    for path, tokens in ((P.SKINNY, 16), (P.MMASYNC, 20)):
        out = gnt.linear_w4(x[:tokens], q, s, path=path)
        check(out, want[:tokens], EPS[F16] * want[:tokens])
    out = gnt.linear_w4(x, q, s, path=P.TC05)
    assert (out[:, 1::2] == INF).all()
    check(out[:, ::2], want[:, ::2], EPS[F16] * want[:, ::2])
