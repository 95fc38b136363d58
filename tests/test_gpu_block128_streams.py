"""The 8-bit layers and the expert layer on a stream of their own while the current
stream still has work queued on memory it has given back: results are those of the
same calls on an idle GPU, bit for bit."""
import pytest

import dense_fp16_tensor_gemm_gb300 as gnt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def operands():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)
    x, dy = normal(1024, 2048), normal(1024, 1536)
    w = gnt.quantize_block128(normal(1536, 2048), block_rows=128, transposed=True)
    saved = gnt.linear_block128(x, w[0], w[1])[1]
    a, sa = gnt.quantize_block128(x)
    t, logits, w13, w2 = normal(64, 1024), normal(64, 16, dtype=torch.float32), normal(16, 1024, 1024), normal(16, 1024, 512)
    return {
        "product": lambda **kw: gnt.gemm_nt_block128_tensors(a, sa, w[0], w[1], **kw),
        "quantise": lambda **kw: gnt.quantize_block128(x, transposed=True, **kw),
        "forward": lambda **kw: gnt.linear_block128(x, w[0], w[1], **kw),
        "backward": lambda **kw: gnt.linear_block128_backward(dy, saved, w[2], w[3], **kw),
        "experts": lambda **kw: gnt.moe_few_tokens(t, logits, w13, w2, 4, **kw),
    }


def flat(r):
    return [r] if isinstance(r, torch.Tensor) else [t for v in r for t in flat(v)]


def bits(r):
    return [t.contiguous().view(torch.uint8).clone() for t in flat(r)]


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", ["product", "quantise", "forward", "backward", "experts"])
def test_beside_a_busy_current_stream(name, as_handle):
    call, side = operands()[name], torch.cuda.Stream()
    want = bits(call())
    sizes = sorted({t.untyped_storage().nbytes() for t in flat(call())})
    sizes += [gnt.gemm_nt_moe_workspace_bytes(64, 4, 512), 1024 * 2048, 1024 * 1536, 4 << 10, 64 << 10]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # about 50 ms; then memory that is already given back is written
    for n in sizes * 2:
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x7f)
    got = call(stream=side.cuda_stream if as_handle else side)
    side.synchronize()
    torch.cuda.synchronize()
    gnt.gemm_nt_check(side.cuda_stream)
    for p, q in zip(bits(got), want):
        assert torch.equal(p, q)


def test_dropped_results_are_not_handed_out_while_they_are_written():
    """A forward pass whose results nobody keeps: what the caller's stream allocates
    next is not what the other stream still writes."""
    call, side = operands()["forward"], torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    sizes = [t.untyped_storage().nbytes() for t in flat(call(stream=side))]
    mine = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in sizes * 2]
    torch.cuda.synchronize()
    for t in mine:
        assert bool((t == 0x55).all())


def test_the_default_stream_by_its_handle():
    """Handle 0 under another current stream is the default stream: what it wrote is
    there for work on the default stream without further ado."""
    call = operands()["forward"]
    want = bits(call())
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        with torch.cuda.stream(torch.cuda.default_stream()):
            torch.cuda._sleep(50_000_000)
        got = call(stream=0)
    got = bits(got)  # copies on the default stream
    for p, q in zip(got, want):
        assert torch.equal(p, q)
