"""The plain, MX and packed tensor forms with `stream` given: memory comes from that
stream's pool (stand-ins as in test_block128_streams.py, no GPU)."""
import pytest

import dense_fp16_tensor_gemm_gb300 as gnt
from test_block128_streams import Stream, fake, flat  # noqa: F401

torch = pytest.importorskip("torch")

A, B = torch.zeros(8, 128, dtype=torch.float16), torch.zeros(16, 128, dtype=torch.float16)
A8, B8 = (torch.zeros(n, 128, dtype=torch.uint8).view(torch.float8_e4m3fn) for n in (8, 16))
SA, SB = (torch.full((n, 4), 127, dtype=torch.uint8) for n in (8, 16))
A4, B4 = (torch.zeros(n, 64, dtype=torch.uint8) for n in (8, 16))

CALLS = {
    "plain": lambda **kw: gnt.gemm_nt(A, B, **kw),
    "batched": lambda **kw: gnt.gemm_nt_batched(A[None], B[None], **kw),
    "mx": lambda **kw: gnt.gemm_nt_mx_tensors(A8, SA, B8, SB, **kw),
    "packed": lambda **kw: gnt.gemm_nt_packed(A4, B4, 128, gnt.DType.E2M1, **kw),
    "packed mx": lambda **kw: gnt.gemm_nt_packed(A4, B4, 128, gnt.DType.E2M1, SA, SB, **kw),
    "scales": lambda **kw: gnt.pack_mx_scales(SA, 128, **kw),
}


@pytest.fixture
def forms(fake, monkeypatch):  # noqa: F811
    f, lib, recorded = fake
    # these functions import torch themselves
    monkeypatch.setattr(torch, "empty", lambda *a, real=torch.empty, **kw: (f.pools.append(f.cuda.now.cuda_stream),
                                                                           real(*a, **kw))[1])
    monkeypatch.setattr(f, "empty", torch.empty, raising=False)
    handle = gnt._stream_handle
    monkeypatch.setattr(gnt, "_stream_handle", lambda s: handle(f.cuda.now if s is None else s))
    return f, lib, recorded


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_another_stream(forms, name, as_handle):
    f, lib, recorded = forms
    out = flat(CALLS[name](stream=7 if as_handle else Stream(7)))
    assert f.pools and set(f.pools) == {7} and set(lib.launched) == {7}
    for t in out:
        assert (t.data_ptr(), 1) in recorded


@pytest.mark.parametrize("stream", [None, 1])
@pytest.mark.parametrize("name", CALLS)
def test_the_current_stream(forms, name, stream):
    f, lib, recorded = forms
    CALLS[name](stream=stream)
    assert set(f.pools) == {1} and set(lib.launched) == {1} and not recorded
