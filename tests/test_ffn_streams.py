"""The gated and 4-bit tensor forms with `stream` given: memory belongs to the stream
that uses it and results are recorded for the caller's.  With tensors that are not
on the current CUDA device: refused before anything is called.  (Stand-ins for the
allocator, the streams and the library: no GPU.)"""
import pytest

import dense_fp16_tensor_gemm_gb300 as gnt

torch = pytest.importorskip("torch")
from test_block128_streams import Stream, fake, flat  # noqa: E402,F401

BF16 = torch.bfloat16
X, W13 = torch.zeros(8, 256, dtype=BF16), torch.zeros(64, 256, dtype=BF16)
GU, DH = torch.zeros(8, 64, dtype=BF16), torch.zeros(8, 32, dtype=BF16)
Q, S, Z = torch.zeros(64, 128, dtype=torch.uint8), torch.zeros(64, 2, dtype=BF16), torch.zeros(64, 2, dtype=torch.uint8)

CALLS = {
    "gated": lambda **k: gnt.gated_linear(X, W13, **k),
    "gated, kept": lambda **k: gnt.gated_linear(X, W13, keep=True, **k),
    "backward": lambda **k: gnt.gated_linear_backward(DH, GU, X, W13, **k),
    "quantise": lambda **k: gnt.quantize_w4(W13, zeros=True, **k),
    "4 bits": lambda **k: gnt.linear_w4(X, Q, S, Z, **k),
    "gated, 4 bits": lambda **k: gnt.gated_linear_w4(X, Q, S, **k),
}


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_another_stream(fake, name, as_handle):  # noqa: F811
    f, lib, recorded = fake
    out = flat(CALLS[name](stream=7 if as_handle else Stream(7)))
    assert f.pools and set(f.pools) == {7}
    assert lib.launched and set(lib.launched) == {7}
    assert f.cuda.now.cuda_stream == 1
    for t in out:
        assert (t.data_ptr(), 1) in recorded


@pytest.mark.parametrize("stream", [None, 1])
@pytest.mark.parametrize("name", CALLS)
def test_the_current_stream(fake, name, stream):  # noqa: F811
    f, lib, recorded = fake
    CALLS[name](stream=stream)
    assert set(f.pools) == {1} and set(lib.launched) == {1} and not recorded


def test_what_was_kept_stays_until_the_backward_pass_has_read_it(fake):  # noqa: F811
    CALLS["backward"](stream=Stream(7))
    assert (GU.data_ptr(), 7) in fake[2]


def test_given_outputs_are_the_callers(fake):  # noqa: F811
    f, _, recorded = fake
    h, y = torch.empty(8, 32, dtype=BF16), torch.empty(8, 64, dtype=BF16)
    assert gnt.gated_linear(X, W13, out=h, stream=Stream(7)) is h
    assert gnt.gated_linear_w4(X, Q, S, out=h, stream=Stream(7)) is h
    assert gnt.linear_w4(X, Q, S, out=y, stream=Stream(7)) is y
    assert not f.pools and not recorded


@pytest.mark.parametrize("name", CALLS)
def test_host_tensors_are_refused(name, monkeypatch):
    class Library:
        def __getattr__(self, name):
            raise AssertionError("%s was called" % name)
    monkeypatch.setattr(gnt, "_lib", Library())
    with pytest.raises(ValueError, match="CUDA device"):
        CALLS[name]()


@pytest.mark.gpu
def test_one_operand_on_the_host_is_refused(monkeypatch):
    class Library:
        def __getattr__(self, name):
            raise AssertionError("%s was called" % name)
    monkeypatch.setattr(gnt, "_lib", Library())
    calls = {
        "gated": (gnt.gated_linear, dict(X=X, W13=W13, out=DH)),
        "backward": (gnt.gated_linear_backward, dict(dH=DH, GU=GU, X=X, W13=W13)),
        "4 bits": (gnt.linear_w4, dict(X=X, Q=Q, S=S, Z=Z, out=GU)),
        "gated, 4 bits": (gnt.gated_linear_w4, dict(X=X, Q13=Q, S13=S, Z13=Z, out=DH)),
    }
    for call, tensors in calls.values():
        for one in tensors:
            with pytest.raises(ValueError):
                call(**{k: v if k == one else v.cuda() for k, v in tensors.items()})


@pytest.mark.parametrize("name", CALLS)
def test_host_tensors_are_refused_by_the_first_call_of_all(name, monkeypatch):
    """Before torch has been looked at, too, nothing asks the library for anything."""
    class Library:
        def __getattr__(self, name):
            raise AssertionError("%s was called" % name)
    monkeypatch.setattr(gnt, "_torch", None)
    monkeypatch.setattr(gnt, "_calls", None)
    monkeypatch.setattr(gnt, "_lib", Library())
    with pytest.raises(ValueError, match="CUDA device"):
        CALLS[name]()
    assert gnt._calls is None


def test_the_extension_is_bound_once_torch_and_the_library_are_there(monkeypatch):
    from dense_fp16_tensor_gemm_gb300 import _build
    _build.build()
    for first, second in ((gnt._init_torch, gnt.load), (gnt.load, gnt._init_torch)):
        monkeypatch.setattr(gnt, "_torch", None)
        monkeypatch.setattr(gnt, "_calls", None)
        monkeypatch.setattr(gnt, "_lib", None)
        first()
        assert gnt._calls is None
        second()
        assert gnt._calls is not None


def test_an_extension_that_does_not_load_leaves_the_python_forms(monkeypatch):
    def refuse(*a):
        raise ImportError("built for another torch")
    import importlib.machinery
    lib = gnt.load()
    monkeypatch.setattr(importlib.machinery, "ExtensionFileLoader", refuse)
    monkeypatch.setattr(gnt, "_calls", None)
    gnt._bind_calls()
    assert gnt._calls is None and gnt.load() is lib


def test_an_extension_of_another_torch_stays_unbound(monkeypatch):
    """Where it has been built: under its own release it is bound, under another one not."""
    from dense_fp16_tensor_gemm_gb300 import _build
    if _build._calls_command("") is None:
        pytest.skip("no extension here")
    _build.build()
    gnt.load()
    torch = gnt._init_torch()
    release = torch.__version__
    for version, bound in ((release, True), ("2.0.1+cu118", False), (release, True)):
        monkeypatch.setattr(gnt, "_calls", None)
        monkeypatch.setattr(torch, "__version__", version)
        gnt._bind_calls()
        assert (gnt._calls is not None) == bound
