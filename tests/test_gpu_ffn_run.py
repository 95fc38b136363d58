"""The gated and 4-bit operators as they are used together: beside busy streams, in
captured graphs, in a chain, and behind one another (on the GPU).  Their results do not
depend on the run, so a call's are compared bit for bit."""
import importlib.util
import os

import pytest

import dense_fp16_tensor_gemm_gb300 as gnt
from ffn_util import EPS, act64, check, gated_bound, rounded, sum_error, w4_values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")


def operands(seed=1, tokens=(1, 12, 40, 300)):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF16)
    w13, w = normal(1200, 1024, scale=1 / 32), normal(520, 1024, scale=1 / 32)
    q13, s13, z13 = gnt.quantize_w4(w13, group=64, zeros=True)
    q, s = gnt.quantize_w4(w)
    calls = {}
    for m in tokens:
        x, dh = normal(m, 1024), normal(m, 600)
        gu = gnt.gated_linear(x, w13, keep=True)[1]
        calls["gated", m] = lambda x=x, **kw: gnt.gated_linear(x, w13, **kw)
        calls["kept", m] = lambda x=x, **kw: gnt.gated_linear(x, w13, "gelu", keep=True, **kw)
        calls["backward", m] = lambda x=x, dh=dh, gu=gu, **kw: gnt.gated_linear_backward(dh, gu, x, w13, **kw)
        calls["w4", m] = lambda x=x, **kw: gnt.linear_w4(x, q, s, **kw)
        calls["w4 gated", m] = lambda x=x, **kw: gnt.gated_linear_w4(x, q13, s13, z13, group=64, **kw)
    calls["quantise", 0] = lambda **kw: gnt.quantize_w4(w13, group=32, zeros=True, **kw)
    return calls


def flat(r):
    return [r] if isinstance(r, torch.Tensor) else [t for v in r for t in flat(v)]


def bits(r):
    return [t.contiguous().view(torch.uint8).clone() for t in flat(r)]


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_beside_a_busy_current_stream():
    for name, call in operands().items():
        side = torch.cuda.Stream()
        want = bits(call())
        sizes = sorted({t.untyped_storage().nbytes() for t in flat(call())})
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        for n in sizes * 3:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x7f)
        got = call(stream=side)
        side.synchronize()
        torch.cuda.synchronize()
        gnt.gemm_nt_check(side.cuda_stream)
        assert same(bits(got), want), name


def test_two_streams_at_once():
    calls = operands()
    want = {k: bits(c()) for k, c in calls.items()}
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):
        for k, c in calls.items():
            got.append((k, c(stream=a), c(stream=b)))
    torch.cuda.synchronize()
    gnt.gemm_nt_check()
    for k, p, q in got:
        assert same(bits(p), want[k]) and same(bits(q), want[k]), k


def test_two_graphs():
    """Every call in two graphs, replayed in turns and at once, with inputs that change."""
    calls = operands()
    want = {k: bits(c()) for k, c in calls.items()}
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g, out = torch.cuda.CUDAGraph(), {}
        with torch.cuda.graph(g):
            for k, c in calls.items():
                out[k] = c()
        graphs.append((g, out))
    for t in [t for _, out in graphs for r in out.values() for t in flat(r)]:
        t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    gnt.gemm_nt_check()
    for _, out in graphs:
        for k, r in out.items():
            assert same(bits(r), want[k]), k


def test_a_captured_backward_pass_beside_an_eager_one():
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x, w, dh = (torch.randn(*s, generator=g, device="cuda").to(BF16) / 8 for s in ((300, 512), (800, 512), (300, 400)))
    eager = gnt.gated_linear(x, w, keep=True)[1]  # kept across the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, gu = gnt.gated_linear(x, w, keep=True)
        dx, dw = gnt.gated_linear_backward(dh, gu, x, w)
    want = bits(gnt.gated_linear_backward(dh, eager, x, w))
    graph.replay()
    assert same(bits((dx, dw)), want)
    x.mul_(-0.5)
    graph.replay()
    h2, gu2 = gnt.gated_linear(x, w, keep=True)
    assert same(bits((h, dx, dw)), bits((h2, *gnt.gated_linear_backward(dh, gu2, x, w))))
    gnt.gemm_nt_check()


def test_each_call_reads_what_the_one_before_it_wrote():
    """A chain on one stream, nothing waited for: quantise, multiply, multiply, and so on
    with weights that are written anew each time."""
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    for m in (1, 9, 48, 200):
        x0 = torch.randn(m, 512, generator=g, device="cuda").to(BF16)
        ws = [torch.randn(1024, 512, generator=g, device="cuda").to(BF16) / 16 for _ in range(6)]
        runs = []
        for wait in (True, False):
            w = torch.empty_like(ws[0])
            x = x0
            for one in ws:
                w.copy_(one)
                q, s = gnt.quantize_w4(w, group=128)
                if wait:
                    torch.cuda.synchronize()
                x = gnt.gated_linear_w4(x, q, s, out=torch.empty(m, 512, dtype=BF16, device="cuda"))
                if wait:
                    torch.cuda.synchronize()
                x = gnt.gated_linear(x, w)
                if wait:
                    torch.cuda.synchronize()
                del q, s
            runs.append(bits(x))
        assert same(*runs), m
    gnt.gemm_nt_check()


def test_a_run_of_them():
    """Training step and decoding of one block, each operator on what the last one gave,
    each against the formula on the same inputs."""
    g = torch.Generator(device="cuda")
    g.manual_seed(11)

    def normal(*shape, scale):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF16)
    x, w13, w2 = normal(200, 512, scale=1), normal(1376, 512, scale=512 ** -0.5), normal(512, 688, scale=688 ** -0.5)
    h, gu = gnt.gated_linear(x, w13, keep=True)
    ref, y, eh, ey = gated_bound(x, w13, "silu")
    check(h, ref, rounded(eh, ref, BF16))
    check(gu, y, rounded(ey, y, BF16))
    out = gnt.gemm_nt(h, w2, out_dtype=BF16)
    dh = torch.empty(200, 688, dtype=BF16, device="cuda")
    gnt.gemm_nt_batched_major(out.data_ptr(), 0, w2.data_ptr(), 1, dh.data_ptr(), 1, 1, 200, 688, 512, 512, 688, 688, 0, 0, 0, 1,
                              0, torch.cuda.current_stream().cuda_stream)
    dx, dw = gnt.gated_linear_backward(dh, gu, x, w13)
    gate, up = gu.double().chunk(2, 1)
    value, slope = act64(gate, "silu")
    d = torch.cat((dh.double() * up * slope, dh.double() * value), 1)
    # the products' operands are rounded to bf16 (and computed to 2^-19 of their terms)
    ed = rounded(2.0 ** -19 * torch.cat(((dh.double() * up).abs() * (1 + gate.abs()), (dh.double() * gate).abs()), 1), d, BF16)
    rx, rw = d @ w13.double(), d.t() @ x.double()
    mag = d.abs() + ed
    check(dx, rx, rounded(ed @ w13.double().abs() + sum_error(mag @ w13.double().abs(), 1376), rx, BF16))
    check(dw, rw, rounded(ed.t() @ x.double().abs() + sum_error(mag.t() @ x.double().abs(), 200), rw, BF16))
    # decoding with the updated weights in 4 bits
    w13 = (w13.float() - 0.01 * dw.float()).to(BF16)
    q13, s13, z13 = gnt.quantize_w4(w13, zeros=True)
    q2, s2 = gnt.quantize_w4(w2, group=32)
    v13, v2 = w4_values(q13, s13, z13, 128, 512), w4_values(q2, s2, None, 32, 688)
    for m in (1, 5, 33):
        t = x[:m]
        h = gnt.gated_linear_w4(t, q13, s13, z13)
        eps = EPS[BF16] if m > 16 else 0.0
        ref, _, eh, _ = gated_bound(t, v13, "silu", eps)
        check(h, ref, rounded(3 * eh, ref, BF16))  # (zeros multiplied apart: 3 times the magnitudes)
        y = gnt.linear_w4(h, q2, s2, group=32)
        ref, mag = h.double() @ v2.t(), h.double().abs() @ v2.abs().t()
        check(y, ref, rounded(3 * sum_error(mag, 688) + eps * mag, ref, BF16))
    gnt.gemm_nt_check()


def test_example():
    spec = importlib.util.spec_from_file_location("feed_forward", EXAMPLE)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    w13, w2, errors = mod.train()
    # bf16 throughout: h rounded before Y, gradients through g, u, dh and [dg du], each by
    # 2^-9 of a value or less (its largest half step is 2^-8): at most four of them deep
    assert all(e < 4 * 2.0 ** -8 for e in errors.values()), errors
    # 4 bits: half a step of 2/15 to 2/7 of a group's largest weight, two layers deep
    assert mod.decode(w13, w2) < 0.3
