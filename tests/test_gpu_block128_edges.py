"""Edges of the block-scaled product and the expert layer: Out at every alignment
with its surroundings untouched, operands past 4 GB, even row shares of single
CTAs, experts with many tokens, waits that run out.

Values are small integers and scales powers of two where a result is compared
bit for bit: every sum then fits fp32, and the 16-bit ones are kept below 256.
Other tolerances are those of the formulas' own tests.
"""
import pytest

import dense_fp16_tensor_gemm_gb300 as gnt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_gpu_block128 as product  # noqa: E402
import test_gpu_moe as moe  # noqa: E402

F8 = torch.float8_e4m3fn


def integers(g, rows, k, low, high):
    pitch = (k + 15) // 16 * 16
    v = torch.zeros(rows, pitch, device="cuda").to(F8)[:, :k]
    v.copy_(torch.randint(low, high, (rows, k), generator=g, device="cuda").to(F8))
    return v


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("N,pitch,first", [(300, 301, 0), (255, 256, 0), (255, 256, 1), (513, 521, 3), (130, 137, 5),
                                           (256, 264, 8), (384, 388, 4), (257, 270, 2), (1, 7, 6), (127, 136, 15)])
def test_out_at_any_alignment_and_nothing_beside_it(dtype, N, pitch, first):
    """Rows of Out that start anywhere, on the pair kernel (whole sectors leave
    from a staging area) and on single CTAs."""
    g = product.gen(N + first)
    M, K = 290, 200
    # bf16 holds integers to 256: at most 64 non-zero products of 1 times a scale of 1 or 2
    a = integers(g, M, K, 0, 2)
    a[:, 64:] = 0
    b = integers(g, N, K, -1, 2)
    sa, sb = torch.ones(M, 2, device="cuda"), torch.full((N, 2), 2.0, device="cuda")
    ref = 2 * (a.double() @ b.double().t())
    for path in (gnt.Path.TC05_PAIR, gnt.Path.SKINNY):
        buf = torch.full((first + M * pitch + 64,), -77.0, device="cuda").to(dtype)
        view = buf[first:first + M * pitch].view(M, pitch)
        product.run(a, sa, b, sb, path, out=view[:, :N])
        assert torch.equal(view[:, :N].double(), ref)
        assert bool((view[:, N:] == -77).all()) and bool((buf[:first] == -77).all())
        assert bool((buf[first + M * pitch:] == -77).all())


@pytest.mark.parametrize("M", [5, 64])
@pytest.mark.parametrize("N", [10001, 19300])
def test_even_row_shares(M, N):
    """More rows of B than 64 for every SM, fewer than 128: one wave of CTAs with
    even shares that are no multiple of anything."""
    g = product.gen(M + N)
    a, b = product.codes(g, M, 300), product.codes(g, N, 300)
    sa = product.scales(g, M, 300, 1)
    for rows in (1, 128):
        sb = product.scales(g, N, 300, rows)
        product.check(product.run(a, sa, b, sb, gnt.Path.AUTO), *product.reference(a, sa, b, sb))


@pytest.mark.parametrize("path,M", [(gnt.Path.TC05_PAIR, 300), (gnt.Path.SKINNY, 20), (gnt.Path.MMASYNC, 20)])
def test_product_past_4_gb(path, M):
    """The batch's second half lies past 2^32 bytes in A, B and Out."""
    g = product.gen(M)
    N, K, far = 260, 260, 2 ** 32 + 4096
    a, b = (torch.empty(far + n * 272, dtype=torch.uint8, device="cuda") for n in (M, N))
    out = torch.empty(far // 4 + M * N, device="cuda")
    av, bv = (torch.as_strided(t.view(F8), (2, n, K), (far, 272, 1)) for t, n in ((a, M), (b, N)))
    for v in (av, bv):
        v.copy_((torch.randn(v.shape, generator=g, device="cuda") * 8).to(F8))
    ov = torch.as_strided(out, (2, M, N), (far // 4, N, 1))
    sa, sb = product.scales(g, M, K, 1, 2), product.scales(g, N, K, 128, 2)
    product.run(av, sa, bv, sb, path, out=ov)
    product.check(ov, *product.reference(av, sa, bv, sb))


def test_quantise_past_4_gb():
    """A matrix whose last rows lie past 2^32 bytes."""
    rows, pitch, cols = 4, 2 ** 29 + 64, 300
    x = torch.empty(3 * pitch + cols, dtype=torch.float32, device="cuda")
    v = torch.as_strided(x, (rows, cols), (pitch, 1))
    v.copy_(torch.randn(rows, cols, device="cuda"))
    got = gnt.quantize_block128(v, transposed=True)
    want = gnt.quantize_block128(v.contiguous(), transposed=True)
    gnt.gemm_nt_check(torch.cuda.current_stream().cuda_stream)
    for p, q in zip(got, want):
        p, q = (t.view(torch.uint8) if t.dtype == F8 else t for t in (p, q))
        assert torch.equal(p, q)


@pytest.mark.parametrize("T,E,k,H,I", [(128, 4, 4, 96, 640), (33, 2, 1, 64, 1024), (20, 64, 8, 256, 128),
                                       (100, 5, 3, 130, 200), (24, 3, 3, 40, 2000)])
@pytest.mark.parametrize("xt,wt", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                                   (torch.bfloat16, F8)])
def test_experts_with_many_tokens(T, E, k, H, I, xt, wt):
    """Several groups of 16 tokens on an expert, experts cut along K, few warps' worth
    of work and much; the same bits every time."""
    g = moe.gen(T + H + I)
    x = torch.randn(T, H, generator=g, device="cuda").to(xt)
    logits = torch.randn(T, E, generator=g, device="cuda") * 2
    w13, w2, s13, s2, d13, d2 = moe.weights(g, E, H, I, wt)
    out = moe.run(x, logits, w13, w2, k, s13, s2)
    moe.check(out, *moe.reference(x, logits, d13, d2, k, True))
    for _ in range(5):
        assert torch.equal(moe.run(x, logits, w13, w2, k, s13, s2), out)


def test_experts_past_4_gb():
    """The second expert's weights lie past 2^32 bytes."""
    g = moe.gen(1)
    T, E, H, I, far = 3, 2, 64, 32, 2 ** 31 + 64
    bufs = [torch.empty(far + n, dtype=torch.bfloat16, device="cuda") for n in (2 * I * H, H * I)]
    w13, w2 = (torch.as_strided(b, (E, *s), (far, s[1], 1)) for b, s in zip(bufs, ((2 * I, H), (H, I))))
    for w in (w13, w2):
        w.copy_((torch.randn(w.shape, generator=g, device="cuda") / 8).to(torch.bfloat16))
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device="cuda")
    out = moe.run(x, logits, w13, w2, 2, None, None)
    moe.check(out, *moe.reference(x, logits, w13.double(), w2.double(), 2, True))


@pytest.mark.parametrize("fault", [1, 2])
@pytest.mark.parametrize("path,M,N,K", [(gnt.Path.TC05_PAIR, 512, 512, 4096), (gnt.Path.SKINNY, 64, 16384, 4096),
                                        (gnt.Path.SKINNY, 16, 512, 16384)])
def test_waits_that_run_out_are_reported(path, M, N, K, fault):
    """A load that the producer leaves out (1), a stage that is not released (2):
    every wait ends, the status says so and the next call is right.  K is long
    enough that every CTA, one of 8 that split K included, fills a stage twice."""
    g = product.gen(M)
    a, b = product.codes(g, M, K), product.codes(g, N, K)
    sa, sb = product.scales(g, M, K, 1), product.scales(g, N, K, 128)
    stream = torch.cuda.current_stream().cuda_stream
    gnt.gemm_nt_check(stream)
    gnt.gemm_nt_debug_set_wait_limit(50_000_000)  # cycles, about 25 ms
    gnt.gemm_nt_debug_set_fault(fault)
    try:
        gnt.gemm_nt_block128_tensors(a, sa, b, sb, path=path)
        with pytest.raises(gnt.GemmError) as e:
            gnt.gemm_nt_check(stream)
        assert e.value.status == gnt.Status.DEVICE_TIMEOUT
    finally:
        gnt.gemm_nt_debug_set_fault(0)
        gnt.gemm_nt_debug_set_wait_limit(0)
    gnt.gemm_nt_check(stream)
    product.check(product.run(a, sa, b, sb, path), *product.reference(a, sa, b, sb))
