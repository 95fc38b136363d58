"""Argument checks of the gated product, its gradient and the products with
4-bit weights: all decided on the host, before any CUDA call (no GPU here)."""
import pytest
import torch

import dense_fp16_tensor_gemm_gb300 as gnt
from dense_fp16_tensor_gemm_gb300 import _build

X, W, H, GU, S, Z = (i << 28 for i in range(1, 7))
OK, INVALID, OVERLAP = gnt.Status.OK, gnt.Status.INVALID_VALUE, gnt.Status.OVERLAP
D = gnt.DType
NEVER = (OK, INVALID, OVERLAP, gnt.Status.NOT_SUPPORTED)  # what valid arguments do not give without a device
HUGE = 2 ** 63 - 1


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gnt.load()


def gated(lib, x=X, ldx=512, w=W, ldw=512, h=H, ldh=256, gu=0, ldgu=512, t=D.BF16, act=0, tokens=64, hidden=512,
          inner=256, path=0):
    return lib.gemm_nt_gated(x, ldx, w, ldw, h, ldh, gu, ldgu, t, act, tokens, hidden, inner, path, None)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), INVALID), (dict(hidden=2 ** 31), INVALID), (dict(inner=2 ** 30), INVALID),
    (dict(inner=HUGE), INVALID), (dict(x=0), INVALID), (dict(w=0), INVALID), (dict(h=0), INVALID),
    (dict(x=X + 1), INVALID), (dict(h=H + 1), INVALID), (dict(gu=GU + 1), INVALID), (dict(t=D.F32), INVALID),
    (dict(t=D.E4M3), INVALID), (dict(act=3), INVALID), (dict(act=-1), INVALID), (dict(ldx=511), INVALID),
    (dict(ldw=511), INVALID), (dict(ldh=255), INVALID), (dict(gu=GU, ldgu=511), INVALID), (dict(ldx=HUGE), INVALID),
    (dict(path=99), INVALID), (dict(path=-1), INVALID),
    (dict(h=X + 2), OVERLAP), (dict(h=W + 2 * 511 * 512), OVERLAP), (dict(gu=H + 2), OVERLAP), (dict(gu=X), OVERLAP),
    (dict(gu=W), OVERLAP),
    (dict(tokens=0, x=0, w=0, h=0), OK), (dict(inner=0, h=0), OK),
])
def test_gated_refusals(lib, change, status):
    assert gated(lib, **change) == status


def test_gated_valid_arguments_reach_the_device(lib):
    assert gated(lib) not in NEVER
    assert gated(lib, gu=GU) not in NEVER
    assert gated(lib, hidden=0, x=0, w=0, ldx=0, ldw=0) not in NEVER


def grad(lib, d=H, ldd=256, gu=GU, ldgu=512, o=X, ldo=512, t=D.F16, act=1, tokens=64, inner=256):
    return lib.gemm_nt_gated_grad(d, ldd, gu, ldgu, o, ldo, t, act, tokens, inner, None)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=2 ** 31), INVALID), (dict(inner=-1), INVALID), (dict(inner=HUGE), INVALID), (dict(d=0), INVALID),
    (dict(gu=0), INVALID), (dict(o=0), INVALID), (dict(o=X + 1), INVALID), (dict(ldd=255), INVALID),
    (dict(ldgu=511), INVALID), (dict(ldo=511), INVALID), (dict(t=D.F32), INVALID), (dict(act=7), INVALID),
    (dict(o=GU), OVERLAP), (dict(o=H + 2 * 255), OVERLAP),
    (dict(tokens=0, d=0), OK), (dict(inner=0, o=0), OK),
])
def test_grad_refusals(lib, change, status):
    assert grad(lib, **change) == status


def test_grad_valid_arguments_reach_the_device(lib):
    assert grad(lib) not in NEVER


def w4(codes=W, ldc=256, scales=S, lds=4, zeros=0, ldz=4, group=128):
    return gnt.Weights4(codes, ldc, scales, lds, zeros, ldz, group)


WEIGHTS = [
    (dict(codes=0), INVALID), (dict(ldc=255), INVALID), (dict(scales=0), INVALID), (dict(scales=S + 1), INVALID),
    (dict(lds=3), INVALID), (dict(zeros=Z, ldz=3), INVALID), (dict(group=0), INVALID), (dict(group=16), INVALID),
    (dict(group=-32), INVALID), (dict(group=64), INVALID),  # more groups than the pitch holds
]


def product(lib, x=X, ldx=512, w=None, out=H, ldo=1024, t=D.F16, m=8, n=1024, k=512, path=0):
    return lib.gemm_nt_w4(x, ldx, w, out, ldo, t, m, n, k, path, None)


@pytest.mark.parametrize("change,status", [(dict(w=w4(**c)), s) for c, s in WEIGHTS] + [
    (dict(), INVALID),  # no weights
    (dict(w=w4(), m=-1), INVALID), (dict(w=w4(), k=2 ** 31), INVALID), (dict(w=w4(), x=0), INVALID),
    (dict(w=w4(), x=X + 1), INVALID), (dict(w=w4(), ldx=511), INVALID), (dict(w=w4(), ldo=1023), INVALID),
    (dict(w=w4(), t=D.F32), INVALID), (dict(w=w4(), path=77), INVALID),
    (dict(w=w4(), out=X + 2), OVERLAP), (dict(w=w4(), out=W + 256 * 1023), OVERLAP), (dict(w=w4(), out=S), OVERLAP),
    (dict(w=w4(zeros=Z), out=Z), OVERLAP),
    (dict(m=0), OK), (dict(n=0, out=0), OK),
])
def test_w4_refusals(lib, change, status):
    assert product(lib, **change) == status


def test_w4_valid_arguments_reach_the_device(lib):
    assert product(lib, w=w4()) not in NEVER
    assert product(lib, w=w4(zeros=Z)) not in NEVER
    assert product(lib, k=0, x=0, ldx=0) not in NEVER


def w4_gated(lib, x=X, w=None, h=H, t=D.F16, act=0, tokens=8, hidden=512, inner=512, path=0):
    return lib.gemm_nt_w4_gated(x, 512, w, h, 512, t, act, tokens, hidden, inner, path, None)


@pytest.mark.parametrize("change,status", [(dict(w=w4(**c)), s) for c, s in WEIGHTS] + [
    (dict(w=w4(), act=3), INVALID), (dict(w=w4(), inner=HUGE), INVALID), (dict(w=w4(), inner=513), INVALID),
    (dict(w=w4(), h=W + 256 * 1023), OVERLAP), (dict(tokens=0), OK), (dict(inner=0), OK),
])
def test_w4_gated_refusals(lib, change, status):
    assert w4_gated(lib, **change) == status


def test_w4_gated_valid_arguments_reach_the_device(lib):
    assert w4_gated(lib, w=w4()) not in NEVER


def quantize(lib, w=X, wt=D.F32, rows=100, cols=512, ldw=512, q=None, st=D.BF16):
    return lib.gemm_nt_w4_quantize(w, wt, rows, cols, ldw, q, st, None)


@pytest.mark.parametrize("change,status", [(dict(q=w4(**c)), s) for c, s in WEIGHTS] + [
    (dict(), INVALID), (dict(q=w4(), rows=-1), INVALID), (dict(q=w4(), w=0), INVALID), (dict(q=w4(), w=X + 2), INVALID),
    (dict(q=w4(), wt=D.E4M3), INVALID), (dict(q=w4(), st=D.F32), INVALID), (dict(q=w4(), ldw=511), INVALID),
    (dict(q=w4(codes=X)), OVERLAP), (dict(q=w4(scales=W + 256)), OVERLAP), (dict(q=w4(zeros=S + 4)), OVERLAP),
    (dict(q=w4(zeros=W)), OVERLAP), (dict(rows=0), OK), (dict(cols=0, w=0), OK),
])
def test_quantize_refusals(lib, change, status):
    assert quantize(lib, **change) == status


def test_quantize_valid_arguments_reach_the_device(lib):
    assert quantize(lib, q=w4()) not in NEVER
    assert quantize(lib, q=w4(zeros=Z)) not in NEVER


def copy_rows(lib, src=X + 2, lds=500, dst=H, ldd=512, rows=100, nbytes=498):
    return lib.gemm_nt_copy_rows(src, lds, dst, ldd, rows, nbytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(nbytes=-1), INVALID), (dict(nbytes=HUGE), INVALID), (dict(src=0), INVALID),
    (dict(dst=0), INVALID), (dict(dst=H + 8), INVALID), (dict(ldd=504), INVALID), (dict(ldd=496), INVALID),
    (dict(lds=497), INVALID), (dict(dst=X + 16), OVERLAP), (dict(rows=0, src=0), OK), (dict(nbytes=0), OK),
])
def test_copy_rows_refusals(lib, change, status):
    assert copy_rows(lib, **change) == status


def test_copy_rows_valid_arguments_reach_the_device(lib):
    assert copy_rows(lib) not in NEVER
    assert copy_rows(lib, rows=1, ldd=499) not in NEVER


def test_tensor_forms_refuse():
    """What the tensor forms refuse before they look at a device."""
    x, w = torch.zeros(4, 64, dtype=torch.float16), torch.zeros(32, 64, dtype=torch.float16)
    q, s = torch.zeros(32, 32, dtype=torch.uint8), torch.zeros(32, 1, dtype=torch.float16)
    h, gu = torch.zeros(4, 16, dtype=torch.float16), torch.zeros(4, 32, dtype=torch.float16)
    for call in (
        lambda: gnt.gated_linear(x, w[:31]), lambda: gnt.gated_linear(x, w[:, :63]), lambda: gnt.gated_linear(x[0], w),
        lambda: gnt.gated_linear(x, w, activation="relu"), lambda: gnt.gated_linear(x, w),  # not on a GPU
        lambda: gnt.gated_linear_backward(h, gu[:, :31], x, w), lambda: gnt.gated_linear_backward(h[:3], gu, x, w),
        lambda: gnt.gated_linear_backward(h, gu, x, w, activation=0), lambda: gnt.gated_linear_backward(h, gu, x, w),
        lambda: gnt.linear_w4(x, q[:, :31], s), lambda: gnt.linear_w4(x, q, s, group=32), lambda: gnt.linear_w4(x, q, s),
        lambda: gnt.linear_w4(x, q, s, group=16), lambda: gnt.linear_w4(x, q, s[:31]), lambda: gnt.linear_w4(x, q, s[0]),
        lambda: gnt.gated_linear_w4(x, q[:31], s[:31]), lambda: gnt.gated_linear_w4(x, q, s, activation="tanh"),
        lambda: gnt.quantize_w4(w, group=16), lambda: gnt.quantize_w4(w[0]), lambda: gnt.quantize_w4(w),
    ):
        with pytest.raises(ValueError):
            call()
    for call in (
        lambda: gnt.gated_linear(x, w.float()), lambda: gnt.gated_linear(x.float(), w.float()),
        lambda: gnt.gated_linear_backward(h.float(), gu, x, w), lambda: gnt.linear_w4(x, q, s.bfloat16()),
        lambda: gnt.linear_w4(x, q.to(torch.int8), s), lambda: gnt.linear_w4(x.float(), q, s.float()),
        lambda: gnt.linear_w4(x, q, s, s), lambda: gnt.quantize_w4(q), lambda: gnt.quantize_w4(w, scale_dtype=torch.float32),
    ):
        with pytest.raises(TypeError):
            call()


def test_sums_longer_than_the_kernels_step(lib):
    """K is walked in 32 bits: 2^30 is taken, one more is refused before any device call."""
    x, w, h, s = (i << 40 for i in range(1, 5))
    for k, refused in ((2 ** 30, False), (2 ** 30 + 1, True), (2 ** 31 - 1, True)):
        ld = 2 ** 31
        four = w4(codes=w, ldc=ld, scales=s, lds=2 ** 24)
        for status in (gated(lib, x=x, ldx=ld, w=w, ldw=ld, h=h, ldh=8, tokens=1, hidden=k, inner=8),
                       lib.gemm_nt_w4(x, ld, four, h, 8, D.F16, 1, 8, k, 0, None),
                       lib.gemm_nt_w4_gated(x, ld, four, h, 8, D.F16, 0, 1, k, 8, 0, None)):
            assert status == INVALID if refused else status not in NEVER
