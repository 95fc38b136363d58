"""Scales anywhere in fp32's range, on every kernel: what is inside the range at the
end is right whatever the two scales' product, or a block's sum times one of them,
would be on the way.

Tolerance as in the product's own tests, 2^-17 of the sum of magnitudes and half an
ulp; results below the normal range may lose 2^-149 for each block of K and once more.
"""
import pytest

import dense_fp16_tensor_gemm_gb300 as gnt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_gpu_block128 as product  # noqa: E402

F8 = torch.float8_e4m3fn
INF = float("inf")


def check(out, a, sa, b, sb):
    ref, mag = product.reference(a, sa, b, sb)
    want = ref.float()
    kb = sa.shape[-1]
    lim = 2.0 ** -17 * mag + 2.0 ** -24 * ref.abs() + 2.0 ** -149 * (kb + 1)
    over = want.isinf()
    assert torch.equal(out[over], want[over])
    bad = ~((out.double() - ref).abs() <= lim) & ~over
    assert not bad.any(), "%d of %d off, e.g. %g for %g" % (
        int(bad.sum()), bad.numel(), float(out[bad][0]), float(ref[bad][0]))


def operands(M, N, K, dtype=F8, low=300.0):
    """Codes of large values, so that products of tiny scales come back into range."""
    g = product.gen(M + N)
    a, b = product.codes(g, M, K, dtype=dtype), product.codes(g, N, K, dtype=dtype)
    for t in (a, b):
        t.copy_((low * (1 + 0.4 * torch.rand(t.shape, generator=g, device="cuda"))).to(dtype))
    return g, a, b


def scales(g, rows, K, block_rows, size):
    return product.scales(g, rows, K, block_rows).clamp(0.5, 1.9) * size


SIZES = [(2e-22, 3e-23), (2.0 ** -70, 2.0 ** -75), (2.0 ** -120, 2.0 ** 100), (2.0 ** 100, 2.0 ** -120),
         (2.0 ** -140, 2.0 ** 120), (2.0 ** 120, 2.0 ** -140), (2.0 ** 90, 2.0 ** -100), (2.0 ** -100, 2.0 ** 90),
         (2.0 ** 50, 2.0 ** 55), (1e-3, 2.0 ** -110), (2.0 ** -110, 1e-3)]


@pytest.mark.parametrize("path", product.PATHS)
@pytest.mark.parametrize("M", [20, 300])
@pytest.mark.parametrize("sizes", SIZES)
def test_products_of_extreme_scales(path, M, sizes):
    N, K = 400, 300
    g, a, b = operands(M, N, K)
    for rows_a, rows_b in ((1, 128), (1, 1), (128, 1)):
        sa, sb = scales(g, M, K, rows_a, sizes[0]), scales(g, N, K, rows_b, sizes[1])
        check(product.run(a, sa, b, sb, path), a, sa, b, sb)


@pytest.mark.parametrize("path", product.PATHS)
@pytest.mark.parametrize("M", [20, 300])
def test_large_sums_of_e5m2(path, M):
    """A block's sum of 2^38 times two scales of 2^-76: 2^-114."""
    N, K = 300, 256
    g, a, b = operands(M, N, K, torch.float8_e5m2, 40000.0)
    for rows_b in (1, 128):
        sa, sb = scales(g, M, K, 1, 2.0 ** -76), scales(g, N, K, rows_b, 2.0 ** -76)
        check(product.run(a, sa, b, sb, path), a, sa, b, sb)


@pytest.mark.parametrize("path", product.PATHS)
@pytest.mark.parametrize("M", [20, 300])
def test_zeros_under_large_scales(path, M):
    """A block of zeros gives zero under any finite scales; a tiny sum comes back."""
    N, K = 400, 384
    g, a, b = operands(M, N, K, low=2.0)
    a[:, :128] = 0
    b[:200, 128:256] = 0
    a[:, 256:] = a[:, 256:].float().mul(2.0 ** -10).to(F8)
    for rows_a, rows_b in ((1, 128), (1, 1), (128, 1)):
        sa, sb = scales(g, M, K, rows_a, 1.0), scales(g, N, K, rows_b, 1.0)
        sa[:, 0], sb[:, 0] = 1e20, 1e20
        if rows_b == 1:  # rows of B that are zero in the second block
            sa[:, 1] = 2.0 ** 120
            sb[:200, 1], sb[200:, 1] = 2.0 ** 120, 2.0 ** -120
        sa[:, 2], sb[:, 2] = 2.0 ** 60, 2.0 ** 59
        check(product.run(a, sa, b, sb, path), a, sa, b, sb)


@pytest.mark.parametrize("path", product.PATHS)
@pytest.mark.parametrize("M", [20, 300])
def test_single_rows_among_ordinary_ones(path, M):
    """Tiny, huge, zero, infinite and NaN scales of some rows leave the others alone."""
    N, K = 400, 300
    g, a, b = operands(M, N, K)
    for rows_b in (1, 128):
        sa, sb = scales(g, M, K, 1, 2.0 ** -8), scales(g, N, K, rows_b, 2.0 ** -8)
        sa[3], sa[4], sa[5], sa[6, 0] = 2.0 ** -126, 2.0 ** 110, 0.0, 1e-45
        sa[7, 1], sa[8, 2] = INF, float("nan")
        if rows_b == 1:
            sb[11], sb[130], sb[17] = 2.0 ** -126, 2.0 ** 105, 0.0
        out = product.run(a, sa, b, sb, path)
        keep = torch.ones(M, dtype=torch.bool, device="cuda")
        keep[7:9] = False
        check(out[keep], a[keep], sa[keep], b, sb)
        zero = (sb == 0).all(1).nonzero().flatten() if rows_b == 1 else []
        rest = torch.ones(N, dtype=torch.bool, device="cuda")
        rest[zero] = False
        assert bool((out[7, rest] == INF).all()) and bool(out[8].isnan().all())
        assert bool(out[7, ~rest].isnan().all())


@pytest.mark.parametrize("dtype", [F8, torch.float8_e5m2])
@pytest.mark.parametrize("rows_b", [1, 128])
def test_care_for_some_blocks_of_many_tiles(dtype, rows_b):
    """More tiles than CTA pairs, 6 K blocks a tile, so that tiles begin inside groups of
    scales: blocks of zeros and of tiny or huge scales here and there."""
    M, N, K = 2400, 2400, 700
    g, a, b = operands(M, N, K, dtype)
    sa, sb = scales(g, M, K, 1, 2.0 ** -8), scales(g, N, K, rows_b, 2.0 ** -8)
    sa[::97, 1], sb[::13 if rows_b == 1 else 5, 1] = 2.0 ** -75, 2.0 ** -75
    sa[300:330, 4] = 2.0 ** -126
    sa[700:1000, 0] = 2.0 ** 85
    a[1024:1500, 128:256] = 0
    sa[1024:1500, 1] = 2.0 ** -116
    b[512:900, 512:640] = 0
    if rows_b == 1:
        sb[512:900, 4], sb[2000:2050, 3] = 2.0 ** -116, 2.0 ** 105
    for path in (gnt.Path.TC05_PAIR, gnt.Path.SKINNY):
        check(product.run(a, sa, b, sb, path), a, sa, b, sb)
