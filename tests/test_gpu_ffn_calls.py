"""The feed-forward tensor forms' common case as an extension against the Python forms:
the same bits, the same refusals (on the GPU)."""
import pytest
import torch

import dense_fp16_tensor_gemm_gb300 as gnt

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
P = gnt.Path


@pytest.fixture
def both(monkeypatch):
    """Runs a call in the extension and in Python; what each returns or raises."""
    gnt.quantize_w4(torch.zeros(1, 32, device="cuda"))  # (binds it)
    extension = gnt._calls
    assert extension is not None, "the extension has not been built"

    def run(form, *a, **kw):
        out = []
        for calls in (extension, None):
            monkeypatch.setattr(gnt, "_calls", calls)
            try:
                out.append(form(*a, **kw))
            except Exception as e:  # noqa: BLE001
                out.append(e)
        return out
    return run


def same(pair):
    for v in pair:
        if isinstance(v, Exception):
            raise v
    first, second = (v if isinstance(v, tuple) else (v,) for v in pair)
    assert len(first) == len(second)
    for a, b in zip(first, second):
        assert a.shape == b.shape and a.dtype == b.dtype and a.device == b.device
        assert a.numel() == 0 or a.stride() == b.stride()
        ints = torch.uint8 if a.dtype == torch.uint8 else torch.int16
        assert torch.equal(a.contiguous().view(ints), b.contiguous().view(ints))


def refused(pair, kind):
    assert [type(v) for v in pair] == [kind, kind], pair
    assert str(pair[0]) == str(pair[1])


def rand(*shape, dtype=BF16):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(sum(shape)), device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,k,n", [(0, 64, 32), (1, 0, 8), (1, 64, 0), (1, 1000, 77), (16, 256, 96), (17, 1000, 77), (40, 77, 33),
                                   (130, 520, 264)])
def test_gated_and_backward(both, m, k, n, dtype):
    x, w, dh = rand(m, k, dtype=dtype), rand(2 * n, k, dtype=dtype) / 8, rand(m, n, dtype=dtype)
    same(both(gnt.gated_linear, x, w))
    same(both(gnt.gated_linear, x, w, "gelu", keep=True, path=P.MMASYNC))
    wide = rand(m, 2 * k + 8, dtype=dtype)
    same(both(gnt.gated_linear, wide[:, 3:3 + k], w, "gelu_tanh", keep=True))
    gu = gnt.gated_linear(x, w, keep=True)[1]
    same(both(gnt.gated_linear_backward, dh, gu, x, w))


@pytest.mark.parametrize("wt", [torch.float32, BF16, F16])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize(both, group, wt):
    for rows, cols in ((0, 64), (5, 0), (3, 77), (64, 1000)):
        for zeros in (False, True):
            for st in (None, BF16, F16):
                same(both(gnt.quantize_w4, rand(rows, cols, dtype=wt), group, zeros, st))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,k,n", [(0, 64, 32), (1, 1000, 78), (16, 256, 96), (17, 1001, 78), (130, 520, 264)])
def test_products_in_4_bits(both, m, k, n, dtype):
    x = rand(m, k, dtype=dtype)
    for zeros in (False, True):
        q, s, *z = gnt.quantize_w4(rand(n, k, dtype=dtype) / 8, 64, zeros)
        z = z[0] if z else None
        same(both(gnt.linear_w4, x, q, s, z, 64))
        same(both(gnt.linear_w4, x, q, s, z, 64, path=P.MMASYNC))
        same(both(gnt.gated_linear_w4, x, q, s, z, 64, "gelu"))


def test_outputs_that_are_given_come_back(both):
    x, w = rand(4, 256), rand(64, 256)
    q, s = gnt.quantize_w4(w)
    h, y = torch.empty(4, 40, dtype=BF16, device="cuda")[:, :32], torch.empty(4, 64, dtype=BF16, device="cuda")
    assert all(v is h for v in both(gnt.gated_linear, x, w, out=h))
    assert all(v is y for v in both(gnt.linear_w4, x, q, s, out=y))
    assert all(v is h for v in both(gnt.gated_linear_w4, x, q, s, out=h))


def test_refusals(both):
    x, w = rand(4, 256), rand(64, 256)
    q, s = gnt.quantize_w4(w)
    gu, dh = rand(4, 64), rand(4, 32)
    for change, kind in ((dict(W13=rand(64, 255)), ValueError), (dict(W13=rand(63, 256)), ValueError),
                         (dict(W13=w.half()), TypeError), (dict(X=x.float()), TypeError), (dict(activation="relu"), ValueError),
                         (dict(out=rand(4, 31)), ValueError), (dict(out=rand(4, 32, dtype=F16)), ValueError),
                         (dict(W13=rand(256, 64).t()), ValueError), (dict(path=99), gnt.GemmError),
                         (dict(path=P.TC05_PAIR, X=rand(4, 257)[:, :256]), gnt.GemmError), (dict(out=x[:, :32]), gnt.GemmError),
                         (dict(X=x.cpu()), ValueError), (dict(keep=torch.zeros(2)), RuntimeError)):
        refused(both(gnt.gated_linear, **{**dict(X=x, W13=w), **change}), kind)
    for change, kind in ((dict(dH=rand(4, 31)), ValueError), (dict(GU=rand(3, 64)), ValueError), (dict(GU=gu.half()), TypeError),
                         (dict(activation=None), ValueError)):
        refused(both(gnt.gated_linear_backward, **{**dict(dH=dh, GU=gu, X=x, W13=w), **change}), kind)
    for change, kind in ((dict(group=48), ValueError), (dict(W=w.double()), TypeError), (dict(W=w[0]), ValueError),
                         (dict(scale_dtype=torch.float32), TypeError), (dict(zeros=torch.zeros(2)), RuntimeError)):
        refused(both(gnt.quantize_w4, **{**dict(W=w), **change}), kind)
    for change, kind in ((dict(Q=q[:, :127]), ValueError), (dict(S=s.half()), TypeError), (dict(S=s[:63]), ValueError),
                         (dict(Z=s), TypeError), (dict(group=64), ValueError), (dict(out=rand(4, 63)), ValueError),
                         (dict(path=P.TC05_PAIR), gnt.GemmError), (dict(path=-1), gnt.GemmError), (dict(Q=q.cpu()), ValueError)):
        refused(both(gnt.linear_w4, **{**dict(X=x, Q=q, S=s), **change}), kind)


def test_an_operand_copy_without_memory_is_an_exception(both):
    """The copy onto 16-byte boundaries is allocated inside the call: an allocator that refuses
    it raises, from the extension as from Python, and the next call works."""
    torch.cuda.empty_cache()
    x, w = rand(2, 4095), torch.zeros(32768, 4095, dtype=BF16, device="cuda")   # a copy of 268 MB
    gnt.gated_linear(x, w[:8])
    dh, gu = rand(2, 16384), rand(2, 32768)
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    try:
        torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (128 << 20)) / total)
        refused_by = [type(v) for v in both(gnt.gated_linear, x, w) + both(gnt.gated_linear_backward, dh, gu, x, w)]
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert refused_by == [torch.cuda.OutOfMemoryError] * 4
    same(both(gnt.gated_linear, x, w))
