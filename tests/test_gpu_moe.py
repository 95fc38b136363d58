"""The few-token expert layer against its formula in 64 bits.

Tolerance: operands enter exactly (h to 22 bits), sums run in fp32 over at most
hidden / 8 MMA steps split over 8 warps.  With eps = 2^-16 for a dot product
relative to its sum of magnitudes G = |Wg| |x|, U = |Wu| |x| and |silu'| <= 1.1,
  |dh| <= eps * (1.1 G |u| + |silu(g)| U + |h|),
  |dOut| <= sum_j p_j |W2| (|dh| + eps |h|) + half an ulp of Out.
"""
import math

import pytest

import dense_fp16_tensor_gemm_gb300 as gnt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF_ULP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
SMALLEST = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
EPS = 2.0 ** -16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def routing(row, topk, renorm):
    """(expert, weight) pairs of one token, from the definition."""
    order = [e for e in sorted(range(len(row)), key=lambda e: (-row[e], e)) if row[e] > -math.inf]
    picks = order[:topk]
    total = math.fsum(math.exp(row[e] - row[order[0]]) for e in (picks if renorm else order))
    return [(e, math.exp(row[e] - row[order[0]]) / total) for e in picks]


def reference(x, logits, w13, w2, topk, renorm):
    """Out and the tolerance before the last rounding, weights already in 64 bits."""
    out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    xd = x.double()
    for t, row in enumerate(logits.double().cpu().tolist()):
        for e, p in routing(row, topk, renorm):
            g, u = (w13[e] @ xd[t]).chunk(2)
            G, U = (w13[e].abs() @ xd[t].abs()).chunk(2)
            s = g * torch.sigmoid(g)
            h = s * u
            dh = EPS * (1.1 * G * u.abs() + s.abs() * U + h.abs())
            out[t] += p * (w2[e] @ h)
            tol[t] += p * (w2[e].abs() @ (dh + EPS * h.abs()))
    return out, tol


def check(out, ref, tol):
    err = (out.double() - ref).abs()
    lim = tol + HALF_ULP[out.dtype] * ref.abs() + SMALLEST[out.dtype]
    bad = ~(err <= lim)
    assert not bad.any(), "%d of %d off, worst %.3g times the tolerance" % (
        int(bad.sum()), bad.numel(), float((err / lim).max()))


def weights(g, E, H, I, dtype):
    w13 = torch.randn(E, 2 * I, H, generator=g, device="cuda") * H ** -0.5
    w2 = torch.randn(E, H, I, generator=g, device="cuda") * I ** -0.5
    if dtype != torch.float8_e4m3fn:
        w13, w2 = w13.to(dtype), w2.to(dtype)
        return w13, w2, None, None, w13.double(), w2.double()

    def quant(w):
        qs = [gnt.quantize_block128(m, block_rows=128) for m in w]
        return torch.stack([q.view(torch.uint8) for q, _ in qs]).view(dtype), torch.stack([s for _, s in qs])

    def values(q, s):
        full = s.double().repeat_interleave(128, -2)[:, :q.shape[1]].repeat_interleave(128, -1)[:, :, :q.shape[2]]
        return q.double() * full
    (q13, s13), (q2, s2) = quant(w13), quant(w2)
    return q13, q2, s13, s2, values(q13, s13), values(q2, s2)


def run(x, logits, w13, w2, topk, s13, s2, renorm=True, **kw):
    out = gnt.moe_few_tokens(x, logits, w13, w2, topk, S13=s13, S2=s2, renormalize=renorm, **kw)
    gnt.gemm_nt_check(torch.cuda.current_stream().cuda_stream)
    return out


@pytest.mark.parametrize("T,E,k,H,I", [
    (1, 8, 2, 256, 128), (1, 1, 1, 8, 8), (2, 64, 8, 512, 256), (8, 16, 4, 640, 136), (9, 16, 4, 640, 136),
    (17, 4, 2, 264, 72), (40, 4, 4, 128, 64), (64, 33, 3, 200, 96), (65, 8, 2, 320, 64), (128, 300, 6, 64, 40),
    (5, 600, 32, 72, 24), (64, 1024, 32, 48, 16), (128, 1024, 32, 48, 16)])
@pytest.mark.parametrize("xt,wt", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                                   (torch.bfloat16, torch.float8_e4m3fn), (torch.float16, torch.float8_e4m3fn)])
def test_layer(T, E, k, H, I, xt, wt):
    g = gen(T + E + H)
    x = torch.randn(T, H, generator=g, device="cuda").to(xt)
    logits = torch.randn(T, E, generator=g, device="cuda") * 2
    w13, w2, s13, s2, d13, d2 = weights(g, E, H, I, wt)
    for renorm in (True, False):
        out = run(x, logits, w13, w2, k, s13, s2, renorm)
        check(out, *reference(x, logits, d13, d2, k, renorm))


@pytest.mark.parametrize("wt", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("H,I", [(100, 50), (37, 129), (129, 3)])
def test_odd_sizes_and_pitches(wt, H, I):
    """Rows that start anywhere, in larger allocations filled with NaN."""
    g = gen(H)
    T, E, k = 6, 5, 2
    w13, w2, s13, s2, d13, d2 = weights(g, E, H, I, wt)

    def inside(v, extra):
        nan = torch.full((*v.shape[:-1], v.shape[-1] + extra), float("nan"), device="cuda").to(v.dtype)
        nan[..., 1:1 + v.shape[-1]].copy_(v)
        return nan[..., 1:1 + v.shape[-1]]
    x = inside(torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16), 3)
    logits = inside(torch.randn(T, E, generator=g, device="cuda"), 2)
    buf = torch.full((T, H + 5), float("nan"), dtype=torch.bfloat16, device="cuda")
    run(x, logits, inside(w13, 7), inside(w2, 5), k, s13, s2, out=buf[:, 2:2 + H])
    check(buf[:, 2:2 + H], *reference(x, logits, d13, d2, k, True))
    assert bool(buf[:, :2].isnan().all()) and bool(buf[:, 2 + H:].isnan().all())


def test_row_scales():
    """8-bit weights with a scale for each 128 elements of every row."""
    g = gen(2)
    T, E, k, H, I = 3, 4, 2, 300, 140
    w13 = torch.randn(E, 2 * I, H, generator=g, device="cuda")
    w2 = torch.randn(E, H, I, generator=g, device="cuda") * 0.1
    q13, q2 = w13.to(torch.float8_e4m3fn), w2.to(torch.float8_e4m3fn)
    s13 = torch.exp2(torch.randn(E, 2 * I, 3, generator=g, device="cuda")) * 0.05
    s2 = torch.exp2(torch.randn(E, H, 2, generator=g, device="cuda"))
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device="cuda")
    d13 = q13.double() * s13.double().repeat_interleave(128, -1)[..., :H]
    d2 = q2.double() * s2.double().repeat_interleave(128, -1)[..., :I]
    check(run(x, logits, q13, q2, k, s13, s2), *reference(x, logits, d13, d2, k, True))


def test_masks_ties_and_not_a_number():
    g = gen(5)
    T, E, k, H, I = 7, 40, 4, 64, 32
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.float16)
    w13, w2, _, _, d13, d2 = weights(g, E, H, I, torch.float16)
    logits = torch.randn(T, E, generator=g, device="cuda")
    inf = float("inf")
    logits[0] = -inf                       # no expert at all
    logits[1] = -inf
    logits[1, 33] = -3.0                   # one expert, fewer than topk
    logits[2] = 0.5                        # all tied: experts 0..3
    logits[3] = torch.finfo(torch.float32).min  # the lowest value is a value: tied, taken
    logits[4, ::2] = -inf
    logits[5, 7] = float("nan")
    logits[6, 3], logits[6, 2], logits[6, 9:] = 0.0, -0.0, -1.0  # -0 and 0 tie: 2 before 3
    logits[6, :2] = -5.0
    logits[6, 4:9] = -5.0
    # an expert nobody takes may hold anything
    w13[39] = float("nan")
    w2[39] = float("nan")
    logits[4, 39] = -inf
    logits[6, 39] = -inf
    logits[5, 39] = -inf
    for renorm in (True, False):
        out = run(x, logits, w13, w2, k, None, None, renorm)
        rows = [0, 1, 2, 3, 4, 6]
        check(out[rows], *reference(x[rows], logits[rows], d13, d2, k, renorm))
        assert bool((out[0] == 0).all())
        assert bool(out[5].isnan().all())


def test_not_a_number_in_one_expert_reaches_its_tokens_only():
    g = gen(6)
    T, E, k, H, I = 12, 6, 2, 96, 40
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    w13, w2, _, _, d13, d2 = weights(g, E, H, I, torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device="cuda")
    clean = run(x, logits, w13, w2, k, None, None)
    w13[2, 5, 7] = float("nan")
    x[3, 0] = float("inf")
    out = run(x, logits, w13, w2, k, None, None)
    takes = logits.topk(k, dim=1).indices.eq(2).any(1)
    takes[3] = True
    assert bool(out[takes].isnan().any(1).all())
    assert torch.equal(out[~takes], clean[~takes])


def test_runs_agree_and_other_streams_and_workspaces():
    g = gen(7)
    T, E, k, H, I = 24, 16, 4, 512, 256
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device="cuda")
    w13, w2, *_ = weights(g, E, H, I, torch.bfloat16)
    first = run(x, logits, w13, w2, k, None, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.full((gnt.gemm_nt_moe_workspace_bytes(T, k, I),), 0xff, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(first)
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        gnt.moe_few_tokens(x, logits, w13, w2, k, out=out, workspace=ws, stream=side)
    gnt.gemm_nt_check(side.cuda_stream)
    assert torch.equal(first, out)
    with pytest.raises(gnt.GemmError) as e:
        gnt.moe_few_tokens(x, logits, w13, w2, k, workspace=ws[:-16])
    assert e.value.status == gnt.Status.SCRATCH_TOO_SMALL


def test_captured_in_a_graph_with_the_router():
    """Router product, layer: captured once, replayed on new tokens."""
    g = gen(8)
    T, E, k, H, I = 4, 8, 2, 256, 128
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    router = torch.randn(E, H, generator=g, device="cuda").to(torch.bfloat16)
    w13, w2, _, _, d13, d2 = weights(g, E, H, I, torch.bfloat16)
    ws = torch.empty(gnt.gemm_nt_moe_workspace_bytes(T, k, I), dtype=torch.uint8, device="cuda")
    logits = torch.empty(T, E, device="cuda")
    out = torch.empty_like(x)

    def step():
        gnt.gemm_nt(x, router, out=logits)
        gnt.moe_few_tokens(x, logits, w13, w2, k, out=out, workspace=ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        x.copy_(torch.randn(T, H, generator=gen(seed), device="cuda").to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        check(out, *reference(x, logits, d13, d2, k, True))
