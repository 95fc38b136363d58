"""Argument checks of the block-scaled product, its quantiser and the few-token
expert layer: all decided on the host, before any CUDA call (no GPU here)."""
import ctypes

import pytest

import dense_fp16_tensor_gemm_gb300 as gnt
from dense_fp16_tensor_gemm_gb300 import _build

A, B, O, SA, SB, W = (i << 28 for i in range(1, 7))
OK, INVALID, OVERLAP = gnt.Status.OK, gnt.Status.INVALID_VALUE, gnt.Status.OVERLAP
D = gnt.DType
NEVER = (OK, INVALID, OVERLAP, gnt.Status.NOT_SUPPORTED)  # what valid arguments do not give without a device


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gnt.load()


def scale(data, rows=1, row_stride=1, kb_stride=64, batch_stride=0):
    return gnt.Scale128(data, rows, row_stride, kb_stride, batch_stride)


def product(lib, a=A, sa=None, b=B, sb=None, out=O, ab=D.E4M3, ot=D.F32, M=64, N=256, K=512, lda=512, ldb=512, ldo=256,
            s=(0, 0, 0), batch=1, path=0, null_sa=False, null_sb=False):
    sa = None if null_sa else (sa or scale(SA))
    sb = None if null_sb else (sb or scale(SB, 128, 4, 1))
    return lib.gemm_nt_block128(a, sa, b, sb, out, ab, ot, M, N, K, lda, ldb, ldo, *s, batch, path, None)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), INVALID), (dict(K=2 ** 31), INVALID), (dict(a=0), INVALID), (dict(out=0), INVALID),
    (dict(ab=D.F16), INVALID), (dict(ab=D.E2M1), INVALID), (dict(ot=D.E4M3), INVALID), (dict(out=O + 2), INVALID),
    (dict(lda=511), INVALID), (dict(ldb=511), INVALID), (dict(ldo=255), INVALID), (dict(s=(-1, 0, 0)), INVALID),
    (dict(null_sa=True), INVALID), (dict(null_sb=True), INVALID), (dict(sa=scale(0)), INVALID),
    (dict(sa=scale(SA + 2)), INVALID), (dict(sa=scale(SA, 64)), INVALID), (dict(sb=scale(SB, 1, -1)), INVALID),
    (dict(sb=scale(SB, 1, 1, -4)), INVALID), (dict(path=99), INVALID), (dict(path=-1), INVALID),
    (dict(out=A + 1024), OVERLAP), (dict(out=SA), OVERLAP), (dict(out=SB), OVERLAP),
    (dict(s=(0, 0, 64 * 256 - 1), batch=2), OVERLAP),
    (dict(M=0, null_sa=True, a=0), OK), (dict(batch=0), OK),
])
def test_product_refusals(lib, change, status):
    assert product(lib, **change) == status


def test_product_valid_arguments_reach_the_device(lib):
    """The same calls with good arguments fail only for want of a device."""
    assert product(lib) not in NEVER
    assert product(lib, K=0, lda=0, ldb=0, a=0, b=0, null_sa=True, null_sb=True) not in NEVER


def quantize(lib, x=A, xt=D.BF16, rows=100, cols=300, ldx=300, q=B, ldq=304, sq=None, qt=0, ldqt=112, st=None,
             t=D.E4M3):
    sq = sq or scale(SA, 1, 1, 100)
    return lib.gemm_nt_block128_quantize(x, xt, rows, cols, ldx, q, ldq, sq, qt, ldqt, st, t, None)


ST = scale(SB, 1, 1, 300)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(x=0), INVALID), (dict(x=A + 1), INVALID), (dict(xt=D.E4M3), INVALID),
    (dict(t=D.F16), INVALID), (dict(ldx=299), INVALID), (dict(ldq=299), INVALID), (dict(q=0), INVALID),
    (dict(sq=scale(SA, 2)), INVALID), (dict(sq=scale(0)), INVALID), (dict(qt=W), INVALID),  # no scales for QT
    (dict(qt=W, st=ST, ldqt=99), INVALID),
    (dict(qt=W, st=scale(SB, 128, 1, 3)), INVALID),                           # block rows differ
    (dict(sq=scale(SA, 1, 1, 99)), OVERLAP), (dict(sq=scale(SA, 1, 0, 1)), OVERLAP),  # scales share elements
    (dict(q=A + 10), OVERLAP), (dict(qt=B + 50, st=ST), OVERLAP), (dict(sq=scale(B, 1, 1, 100)), OVERLAP),
    (dict(qt=W, st=scale(SA, 1, 1, 300)), OVERLAP),
    (dict(rows=0, x=0, q=0), OK), (dict(cols=0), OK),
])
def test_quantize_refusals(lib, change, status):
    assert quantize(lib, **change) == status


def test_quantize_valid_arguments_reach_the_device(lib):
    assert quantize(lib) not in NEVER
    assert quantize(lib, qt=W, st=ST) not in NEVER
    assert quantize(lib, q=0, qt=W, st=ST) not in NEVER


X, L, W13, W2, WS = A, B, 1 << 32, 1 << 33, 1 << 34


def moe(lib, x=X, ldx=256, l=L, ldl=16, w13=W13, ldw13=256, s13=None, w2=W2, ldw2=128, s2=None, out=O, ldo=256,
        xt=D.BF16, wt=D.BF16, T=4, E=16, k=2, H=256, I=128, ws=WS, nbytes=1 << 20, sw13=2 * 128 * 256, sw2=128 * 256):
    return lib.gemm_nt_moe(x, ldx, l, ldl, w13, ldw13, sw13, s13, w2, ldw2, sw2, s2, out, ldo, xt, wt, T, E, k, H, I, 1,
                           ws, nbytes, None)


S13, S2 = scale(SA, 128, 2, 1, 4), scale(SB, 128, 1, 1, 2)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(x=0), INVALID), (dict(l=0), INVALID), (dict(l=L + 2), INVALID), (dict(out=0), INVALID),
    (dict(w13=0), INVALID), (dict(w2=0), INVALID), (dict(ldx=255), INVALID), (dict(ldl=15), INVALID),
    (dict(ldw13=255), INVALID), (dict(ldw2=127), INVALID), (dict(ldo=255), INVALID), (dict(sw2=-1), INVALID),
    (dict(k=0), INVALID), (dict(k=17), INVALID), (dict(xt=D.F32), INVALID), (dict(wt=D.F16), INVALID),
    (dict(wt=D.E5M2), INVALID), (dict(wt=D.E4M3), INVALID), (dict(wt=D.E4M3, s13=S13), INVALID),
    (dict(s13=S13, s2=S2), INVALID),                                          # scales with 16-bit weights
    (dict(ws=0), INVALID), (dict(ws=WS + 8), INVALID),
    (dict(nbytes=4 * 2 * 128 * 4 - 1), gnt.Status.SCRATCH_TOO_SMALL),
    (dict(T=129, nbytes=1 << 28), gnt.Status.NOT_SUPPORTED), (dict(E=1025, ldl=1025), gnt.Status.NOT_SUPPORTED),
    (dict(E=64, ldl=64, k=33, nbytes=1 << 28), gnt.Status.NOT_SUPPORTED),
    (dict(out=X), OVERLAP), (dict(out=L), OVERLAP), (dict(out=W2 + 64), OVERLAP), (dict(ws=W13), OVERLAP),
    (dict(ws=X), OVERLAP), (dict(ws=O), OVERLAP),
    (dict(T=0), OK), (dict(H=0), OK),
])
def test_moe_refusals(lib, change, status):
    assert moe(lib, **change) == status


def test_moe_valid_arguments_reach_the_device(lib):
    assert moe(lib) not in NEVER
    assert moe(lib, wt=D.E4M3, s13=S13, s2=S2) not in NEVER
    assert moe(lib, I=0, w13=0, w2=0, ws=0, nbytes=0) not in NEVER


def test_moe_workspace_bytes(lib):
    f = lib.gemm_nt_moe_workspace_bytes
    assert f(4, 2, 128) == 4 * 2 * 128 * 4
    assert f(1, 1, 1) == 64 and f(0, 2, 5) == 0 and f(-1, 2, 5) == -1


def test_scale_struct_layout():
    """The binding's struct mirrors gemm_scale128_t: pointer, int32, three int64."""
    offsets = [getattr(gnt.Scale128, n).offset for n, _ in gnt.Scale128._fields_]
    assert offsets == [0, 8, 16, 24, 32] and ctypes.sizeof(gnt.Scale128) == 40


def test_tensor_forms_refuse_shapes_and_types():
    import torch
    f8 = torch.float8_e4m3fn
    a = torch.zeros(8, 256, dtype=torch.uint8).view(f8)
    s = torch.ones(8, 2)
    with pytest.raises(ValueError):
        gnt.gemm_nt_block128_tensors(a, s, a[:, :128], s)
    with pytest.raises(TypeError):
        gnt.gemm_nt_block128_tensors(a, s, a.view(torch.float8_e5m2), s)
    with pytest.raises(TypeError):
        gnt.gemm_nt_block128_tensors(a, s.double(), a, s)
    with pytest.raises(ValueError):
        gnt.gemm_nt_block128_tensors(a, s[:, :1], a, s)
    with pytest.raises(TypeError):
        gnt.gemm_nt_block128_tensors(a, s, a, s, out_dtype=torch.int32)
    with pytest.raises(ValueError):
        gnt.quantize_block128(torch.zeros(4, 4), block_rows=64)
    with pytest.raises(TypeError):
        gnt.quantize_block128(torch.zeros(4, 4, dtype=torch.float64))
    with pytest.raises(TypeError):
        gnt.quantize_block128(torch.zeros(4, 4), q_dtype=torch.float16)
    x, l = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 4)
    w13, w2 = torch.zeros(4, 32, 64, dtype=torch.bfloat16), torch.zeros(4, 64, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        gnt.moe_few_tokens(x, l, w13, w2[:, :, :8], 2)
    with pytest.raises(TypeError):
        gnt.moe_few_tokens(x, l.half(), w13, w2, 2)
    with pytest.raises(TypeError):
        gnt.moe_few_tokens(x, l, w13.half(), w2.half(), 2)
    with pytest.raises(ValueError):
        gnt.moe_few_tokens(x, l, w13, w2, 2, S13=torch.ones(4, 1, 1), S2=torch.ones(4, 1, 1))


def test_linear_refuses_what_does_not_fit():
    torch = pytest.importorskip("torch")
    f8 = torch.float8_e4m3fn
    x, w, sw = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(8, 256).to(f8), torch.ones(1, 2)
    wt, swt = torch.zeros(256, 8).to(f8), torch.ones(2, 1)
    saved = (torch.zeros(256, 4).to(f8), torch.ones(256, 1))
    dy = torch.zeros(4, 8, dtype=torch.bfloat16)
    for bad in (lambda: gnt.linear_block128(x[0], w, sw), lambda: gnt.linear_block128(x[:, :128], w, sw),
                lambda: gnt.linear_block128(x, w, sw[0]), lambda: gnt.linear_block128(x, w, torch.ones(2, 2)),
                lambda: gnt.linear_block128_backward(dy[:, :4], saved, wt, swt),
                lambda: gnt.linear_block128_backward(dy[:3], saved, wt, swt),
                lambda: gnt.linear_block128_backward(dy, (saved[0], torch.ones(256, 3)), wt, swt),
                lambda: gnt.linear_block128(x.t(), w[:, :4], torch.ones(1, 1))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: gnt.linear_block128(x.double(), w, sw), lambda: gnt.linear_block128(x, w.float(), sw),
                lambda: gnt.linear_block128(x, w, sw.double()),
                lambda: gnt.linear_block128_backward(dy, (saved[0].to(torch.float8_e5m2), saved[1]), wt, swt)):
        with pytest.raises(TypeError):
            bad()
