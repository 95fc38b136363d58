"""With `stream` given, memory belongs to the stream that uses it: whatever a call
allocates comes from that stream's pool (a block of the current stream's pool may
still be read or written by work queued there, which the other stream does not
wait for), and what it returns is recorded for the caller's stream as well.  The
allocator, the streams and the library are stand-ins here (no GPU)."""
import contextlib
import ctypes

import pytest

import dense_fp16_tensor_gemm_gb300 as gnt

torch = pytest.importorskip("torch")


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Cuda:
    Stream = Stream

    def __init__(self):
        self.now = Stream(1)

    def ExternalStream(self, handle):
        """As torch's: handle 0 makes a stream of its own, not the default one."""
        return Stream(handle or 99)

    def default_stream(self, device=None):
        return Stream(0)

    def current_stream(self, device=None):
        return self.now

    @contextlib.contextmanager
    def stream(self, s):
        before, self.now = self.now, s
        yield
        self.now = before


class Torch:
    """torch, with a note of the stream that was current at each allocation."""

    def __init__(self):
        self.cuda, self.pools = Cuda(), []

    def __getattr__(self, name):
        return getattr(torch, name)

    def empty(self, *args, **kw):
        self.pools.append(self.cuda.now.cuda_stream)
        return torch.empty(*args, **kw)

    def empty_strided(self, *args, **kw):
        self.pools.append(self.cuda.now.cuda_stream)
        return torch.empty_strided(*args, **kw)


class Library:
    """Every entry point returns GEMM_OK; `launched`: the handles of the streams."""

    def __init__(self):
        self.launched = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 4096
            self.launched.append(ctypes.c_void_p(args[-1]).value or 0)
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    gnt._init_torch()
    f, lib, recorded = Torch(), Library(), []
    monkeypatch.setattr(gnt, "_torch", f)
    monkeypatch.setattr(gnt, "_lib", lib)
    monkeypatch.setattr(gnt, "_stream_of", lambda index: f.cuda.now.cuda_stream)
    monkeypatch.setattr(gnt, "_same_device", lambda *a: 0)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: recorded.append((t.data_ptr(), s.cuda_stream)), raising=False)
    return f, lib, recorded


F8 = torch.float8_e4m3fn
X = torch.zeros(8, 256, dtype=torch.bfloat16)
W, SW = torch.zeros(128, 256, dtype=torch.uint8).view(F8), torch.ones(1, 2)
WT, SWT = torch.zeros(256, 128, dtype=torch.uint8).view(F8), torch.ones(2, 1)
A, SA = torch.zeros(8, 256, dtype=torch.uint8).view(F8), torch.ones(8, 2)
SAVED = (torch.zeros(256, 8, dtype=torch.uint8).view(F8), torch.ones(256, 1))
DY = torch.zeros(8, 128, dtype=torch.bfloat16)
W13, W2 = torch.zeros(4, 32, 256, dtype=torch.bfloat16), torch.zeros(4, 256, 16, dtype=torch.bfloat16)
LOGITS = torch.zeros(8, 4)

CALLS = {
    "product": lambda s: gnt.gemm_nt_block128_tensors(A, SA, W, SW, stream=s),
    "quantise": lambda s: gnt.quantize_block128(X, transposed=True, stream=s),
    "forward": lambda s: gnt.linear_block128(X, W, SW, stream=s),
    "backward": lambda s: gnt.linear_block128_backward(DY, SAVED, WT, SWT, stream=s),
    "experts": lambda s: gnt.moe_few_tokens(X, LOGITS, W13, W2, 2, stream=s),
}


def flat(r):
    return [r] if isinstance(r, torch.Tensor) else [t for v in r for t in flat(v)]


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_another_stream(fake, name, as_handle):
    f, lib, recorded = fake
    out = flat(CALLS[name](7 if as_handle else Stream(7)))
    assert f.pools and set(f.pools) == {7}, "allocated for streams %s" % f.pools
    assert lib.launched and set(lib.launched) == {7}
    assert f.cuda.now.cuda_stream == 1
    for t in out:
        assert (t.data_ptr(), 1) in recorded, "a result is not recorded for the caller's stream"


def test_saved_codes_stay_until_the_backward_pass_has_read_them(fake):
    recorded = fake[2]
    CALLS["backward"](Stream(7))
    for t in SAVED:
        assert (t.data_ptr(), 7) in recorded


@pytest.mark.parametrize("stream", [None, 1])
@pytest.mark.parametrize("name", CALLS)
def test_the_current_stream(fake, name, stream):
    f, lib, recorded = fake
    CALLS[name](stream)
    assert set(f.pools) == {1} and set(lib.launched) == {1} and not recorded


def test_given_outputs_and_workspace_are_the_callers(fake):
    f, _, recorded = fake
    out, ws = torch.empty_like(X), torch.empty(4096, dtype=torch.uint8)
    assert gnt.moe_few_tokens(X, LOGITS, W13, W2, 2, out=out, workspace=ws, stream=Stream(7)) is out
    assert not f.pools and not recorded


@pytest.mark.parametrize("name", CALLS)
def test_the_default_stream_by_its_handle(fake, name):
    f, lib, _ = fake
    CALLS[name](0)
    assert set(f.pools) == {0} and set(lib.launched) == {0}
