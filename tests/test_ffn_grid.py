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


# columns of 4-bit weights, bytes between the rows' starts, of what the storage starts with
CODES = [(1000, 500, 0), (1000, 512, 1), (999, 500, 16), (4100, 2050, 0), (256, 130, 2)]


def codes_off(cols, pitch, offset, rows, device):
    width = (cols + 1) // 2
    store = torch.zeros(offset + rows * pitch + 16, dtype=torch.uint8, device=device)
    return store[offset:offset + rows * pitch].view(rows, pitch)[:, :width]


@pytest.mark.parametrize("cols,pitch,offset", CODES)
def test_codes_off_the_grid_are_copied(fake, monkeypatch, cols, pitch, offset):  # noqa: F811
    for tokens, rows in ((1, 6), (40, 6)):
        x = torch.zeros(tokens, (cols + 7) // 8 * 8, dtype=BF16)[:, :cols]
        q, s = codes_off(cols, pitch, offset, rows, "cpu"), torch.zeros(rows, (cols + 127) // 128, dtype=BF16)
        for call in (gnt.linear_w4, gnt.gated_linear_w4):
            for path, copies in ((P.AUTO, [(rows, (cols + 1) // 2)]), (P.MMASYNC, [])):
                lib = Library()
                monkeypatch.setattr(gnt, "_lib", lib)
                call(x, q, s, path=path)
                assert lib.copied == copies
    # an output that lies on them is refused before that, whatever the library sees
    lib = Library()
    monkeypatch.setattr(gnt, "_lib", lib)
    monkeypatch.setattr(gnt, "error_string", lambda status: "overlap")
    store = torch.zeros(4096, dtype=torch.uint8)
    q, out = store[1:1 + 6 * 500].view(6, 500), store[3000:3012].view(BF16).view(1, 6)
    for at, refused in ((out, True), (store[3002:3014].view(BF16).view(1, 6), False)):
        x, s = torch.zeros(1, 1000, dtype=BF16), torch.zeros(6, 8, dtype=BF16)
        if refused:
            with pytest.raises(gnt.GemmError) as e:
                gnt.linear_w4(x, q, s, out=at)
            assert e.value.status == gnt.Status.OVERLAP and not lib.copied
        else:
            assert gnt.linear_w4(x, q, s, out=at) is at


@pytest.mark.gpu
@pytest.mark.parametrize("cols,pitch,offset", CODES)
def test_codes_off_the_grid_take_the_kernels_of_those_on_it(forms, cols, pitch, offset):
    g = torch.Generator("cuda").manual_seed(cols + pitch)
    for tokens in (1, 7, 40, 200):
        x = on_grid(normal(g, tokens, cols))
        for zeros in (False, True):
            q, s, *z = gnt.quantize_w4(normal(g, 320, cols) / 32, 64, zeros)
            off = codes_off(cols, pitch, offset, 320, "cuda")
            off.copy_(q)
            for call in (gnt.linear_w4, gnt.gated_linear_w4):
                want = call(x, q, s, *z, group=64)
                for out in forms(lambda: call(x, off, s, *z, group=64)):
                    assert torch.equal(out, want)
    gnt.gemm_nt_check()


@pytest.mark.gpu
def test_a_single_row_of_codes_takes_the_same_kernels(forms):
    """Its pitch is never stepped by, so any will do."""
    g = torch.Generator("cuda").manual_seed(1)
    for tokens in (1, 40):
        for cols in (1001, 1000):
            x = on_grid(normal(g, tokens, cols))
            q, s = gnt.quantize_w4(normal(g, 1, cols) / 32)
            for out in forms(lambda: gnt.linear_w4(x, q, s)):
                assert torch.equal(out, gnt.linear_w4(x, q, s, path=P.SKINNY if tokens == 1 else P.TC05))
    gnt.gemm_nt_check()
