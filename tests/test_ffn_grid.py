"""Operands off 16-byte boundaries: which of them the tensor forms copy first (stand-ins for
the library and the device, no GPU), and that the calls then take the kernels that the same
operands on those boundaries take (on the GPU, bit for bit)."""
import ctypes

import pytest

import dense_fp16_tensor_gemm_gb300 as gnt

torch = pytest.importorskip("torch")
from test_block128_streams import fake  # noqa: E402,F401

BF16 = torch.bfloat16
P = gnt.Path


class Library:
    """Every entry point returns GEMM_OK; `copied`: the rows and bytes of each copy."""

    def __init__(self):
        self.copied = []

    def __getattr__(self, name):
        def call(*args):
            if name == "gemm_nt_copy_rows":
                self.copied.append(tuple(ctypes.c_int64(a).value for a in args[4:6]))
            return 0
        return call


# tokens, columns, whether the stream of 16-bit and of 4-bit weights takes them
TOKENS = [(1, 1001, True, True), (16, 1001, True, True), (17, 1001, False, False), (16, 4097, False, False),
          (16, 4095, True, True), (15, 4351, True, True), (14, 4651, True, False), (12, 6001, False, False),
          (8, 8191, True, True), (8, 8193, False, False), (10, 8191, False, False), (1, 65535, True, True)]


@pytest.mark.parametrize("tokens,cols,few,few4", TOKENS)
def test_tokens_are_copied_unless_the_stream_takes_them(fake, monkeypatch, tokens, cols, few, few4):  # noqa: F811
    x, w = torch.zeros(tokens, cols, dtype=BF16), torch.zeros(4, (cols + 7) // 8 * 8, dtype=BF16)[:, :cols]
    # a single row lies off the grid only where it starts off it
    x = torch.zeros(tokens * cols + 9, dtype=BF16)[1:1 + tokens * cols].view(tokens, cols) if tokens == 1 else x
    q = torch.zeros(4, ((cols + 1) // 2 + 15) // 16 * 16, dtype=torch.uint8)[:, :(cols + 1) // 2]
    s = torch.zeros(4, (cols + 127) // 128, dtype=BF16)
    for call, takes in ((lambda: gnt.gated_linear(x, w), few), (lambda: gnt.linear_w4(x, q, s), few4),
                        (lambda: gnt.gated_linear_w4(x, q, s), few4)):
        lib = Library()
        monkeypatch.setattr(gnt, "_lib", lib)
        call()
        assert lib.copied == ([] if takes else [(tokens, 2 * cols)])
    for call in (lambda: gnt.gated_linear(x, w, path=P.MMASYNC), lambda: gnt.linear_w4(x, q, s, path=P.MMASYNC)):
        lib = Library()
        monkeypatch.setattr(gnt, "_lib", lib)
        call()
        assert lib.copied == []


@pytest.fixture
def forms(monkeypatch):
    """Runs a call in the extension and in Python."""
    gnt.quantize_w4(torch.zeros(1, 32, device="cuda"))  # (binds it)
    extension = gnt._calls
    assert extension is not None, "the extension has not been built"

    def run(call):
        out = []
        for calls in (extension, None):
            monkeypatch.setattr(gnt, "_calls", calls)
            out.append(call())
        return out
    return run


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(BF16)


def on_grid(t):
    rows, cols = t.shape
    unit = 16 // t.element_size()
    out = torch.zeros(rows, (cols + unit - 1) // unit * unit, dtype=t.dtype, device=t.device)[:, :cols]
    out.copy_(t)
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,cols,few,few4", TOKENS)
def test_calls_off_the_grid_take_the_kernels_of_those_on_it(forms, tokens, cols, few, few4):
    g = torch.Generator("cuda").manual_seed(cols)
    x, n = normal(g, tokens * cols + 1)[1:].view(tokens, cols), 160
    w = normal(g, 2 * n, cols) / 64
    q, s = gnt.quantize_w4(w)
    xs = on_grid(x)
    # the stream, and tcgen05 where it refuses
    want = gnt.gated_linear(xs, on_grid(w), path=P.SKINNY if few else P.TC05)
    for out in forms(lambda: gnt.gated_linear(x, w)):
        assert torch.equal(out, want)
    way = P.SKINNY if few4 else P.TC05
    want = gnt.linear_w4(xs, q, s, path=way)
    for out in forms(lambda: gnt.linear_w4(x, q, s)):
        assert torch.equal(out, want)
    want = gnt.gated_linear_w4(xs, q, s, path=way)
    for out in forms(lambda: gnt.gated_linear_w4(x, q, s)):
        assert torch.equal(out, want)
    # the rule is the library's: the stream takes those tokens and no others
    for take, call in ((few, lambda: gnt.gated_linear(x, on_grid(w), path=P.SKINNY)),
                       (few4, lambda: gnt.linear_w4(x, q, s, path=P.SKINNY))):
        if take:
            call()
        else:
            with pytest.raises(gnt.GemmError):
                call()
    gnt.gemm_nt_check()
