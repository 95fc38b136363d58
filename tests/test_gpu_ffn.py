"""The gated feed-forward product, its gradient and products with 4-bit weights
against their formulas in 64 bits (on the GPU)."""
import math

import pytest
import torch

import dense_fp16_tensor_gemm_gb300 as gnt
from ffn_util import ACTS, EPS, act64, check, gated_bound, rounded, sum_error, w4_values

pytestmark = pytest.mark.gpu
P = gnt.Path
F16, BF16 = torch.float16, torch.bfloat16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, scale=1.0, dtype=BF16, pitch=0, offset=0):
    """Rows of random values, `pitch` elements apart, `offset` elements into their
    storage; what lies between the rows is NaN."""
    rows, cols = shape
    pitch = pitch or cols
    store = torch.full((offset + rows * pitch,), math.nan, device="cuda", dtype=dtype)
    out = store[offset:].view(rows, pitch)[:, :cols]
    out.copy_(torch.randn(rows, cols, generator=g, device="cuda") * scale)
    return out


# tokens, hidden, inner, and the pitch's excess over the row
SHAPES = [(1, 1, 1, 0), (1, 64, 8, 0), (1, 2048, 1024, 0), (2, 8, 300, 8), (3, 1000, 77, 0), (7, 1000, 520, 0),
          (8, 4096, 256, 0), (9, 264, 129, 8), (16, 1024, 2048, 0), (17, 520, 64, 0), (33, 136, 1000, 24), (64, 2048, 512, 0),
          (65, 256, 96, 0), (100, 333, 55, 1), (128, 640, 384, 0), (129, 72, 130, 0), (256, 512, 128, 0),
          (300, 1000, 260, 0), (520, 1032, 1048, 8), (1000, 64, 2047, 0)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", SHAPES)
def test_gated(shape, dtype):
    m, k, n, extra = shape
    g = gen(m + k + n)
    x = normal(g, m, k, dtype=dtype, pitch=k + extra)
    w = normal(g, 2 * n, k, scale=k ** -0.5, dtype=dtype, pitch=k + extra)
    for i, act in enumerate(ACTS):
        h, y, eh, ey = gated_bound(x, w, act)
        out, gu = gnt.gated_linear(x, w, activation=act, keep=True)
        check(out, h, rounded(eh, h, dtype), act)
        check(gu, y, rounded(ey, y, dtype), act + " gu")
        assert torch.equal(gnt.gated_linear(x, w, activation=act), out) or m <= 64
        into = torch.full((m, n + 3), 7.0, dtype=dtype, device="cuda")
        gnt.gated_linear(x, w, activation=act, out=into[:, :n])
        check(into[:, :n], h, rounded(eh, h, dtype), act + " out")
        assert (into[:, n:] == 7).all()
    gnt.gemm_nt_check()


@pytest.mark.parametrize("path", [P.MMASYNC, P.TC05_PAIR, P.SKINNY, P.TC05])
@pytest.mark.parametrize("offset", [0, 8, 1])
def test_gated_paths_and_alignments(path, offset):
    for m, k, n, dtype in ((5, 264, 72, BF16), (70, 520, 200, F16), (300, 136, 513, BF16)):
        m = min(m, {P.SKINNY: 16, P.TC05: 64}.get(path, m))
        g = gen(m + offset)
        x = normal(g, m, k, dtype=dtype, pitch=k + offset, offset=offset)
        w = normal(g, 2 * n, k, scale=k ** -0.5, dtype=dtype, pitch=k + offset, offset=offset)
        h, y, eh, ey = gated_bound(x, w, "silu")
        store = torch.zeros(offset + m * (n + 5), dtype=dtype, device="cuda")
        out = store[offset:].view(m, n + 5)[:, :n]
        if offset == 1 and path != P.MMASYNC:
            with pytest.raises(gnt.GemmError):
                gnt.gated_linear(x, w, out=out, path=path)
            continue
        _, gu = gnt.gated_linear(x, w, out=out, keep=True, path=path)
        check(out, h, rounded(eh, h, dtype))
        check(gu, y, rounded(ey, y, dtype))
        assert (store[offset:].view(m, n + 5)[:, n:] == 0).all()
    gnt.gemm_nt_check()


def test_gated_values():
    """Large, infinite and NaN gates, and nothing to sum."""
    x = torch.zeros(6, 8, dtype=BF16, device="cuda")
    x[:, 0] = torch.tensor([0.0, 100.0, -100.0, 3e38, -3e38, math.nan], device="cuda")
    x[:, 1] = 1
    w = torch.zeros(2, 8, dtype=BF16, device="cuda")
    w[0, 0], w[1, 1] = 1, 2
    for act in ACTS:
        h = gnt.gated_linear(x, w, activation=act).flatten().float().tolist()
        assert h[0] == 0 and h[1] == 200 and h[2] == 0 and h[3] == math.inf and h[4] == 0 and math.isnan(h[5])
        assert (gnt.gated_linear(x[:, :0], w[:, :0], activation=act) == 0).all()
    assert gnt.gated_linear(x[:0], w).shape == (0, 1) and gnt.gated_linear(x, w[:0]).shape == (6, 0)


def backward_case(m, k, n, dtype, act, seed=0, extra=0):
    g = gen(m + k + n + seed)
    x = normal(g, m, k, dtype=dtype, pitch=k + extra)
    w = normal(g, 2 * n, k, scale=k ** -0.5, dtype=dtype, pitch=k + extra)
    gu = normal(g, m, 2 * n, scale=1.5, dtype=dtype, pitch=2 * n + extra)
    dh = normal(g, m, n, scale=0.1, dtype=dtype, pitch=n + extra)
    return x, w, gu, dh


def check_backward(x, w, gu, dh, act, dx, dw):
    dtype, n = x.dtype, dh.shape[1]
    g, u, d = gu[:, :n].double(), gu[:, n:].double(), dh.double()
    value, slope = act64(g, act)
    ref = torch.cat((d * u * slope, d * value), 1)
    # P and P' to 2^-19 of 1 (see gated_bound), |slope| < 1.13, and the rounding to dtype
    err = torch.cat(((d * u).abs() * (1 + g.abs()), (d * g).abs()), 1) * 2.0 ** -19
    err = rounded(err, ref, dtype)
    mag, xd, wd = ref.abs() + err, x.double(), w.double()
    rx, rw = ref @ wd, ref.t() @ xd
    check(dx, rx, rounded(err @ wd.abs() + sum_error(mag @ wd.abs(), 2 * n), rx, dtype), "dX")
    check(dw, rw, rounded(err.t() @ xd.abs() + sum_error(mag.t() @ xd.abs(), x.shape[0]), rw, dtype), "dW13")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", [(1, 1, 1, 0), (1, 64, 40, 0), (7, 1000, 77, 0), (64, 256, 96, 8), (130, 333, 51, 1),
                                   (300, 1000, 520, 0), (1025, 512, 264, 0), (520, 264, 1031, 8)])
def test_backward(shape, dtype):
    m, k, n, extra = shape
    for act in ACTS:
        x, w, gu, dh = backward_case(m, k, n, dtype, act, extra=extra)
        dx, dw = gnt.gated_linear_backward(dh, gu, x, w, activation=act)
        assert dx.dtype == dw.dtype == dtype and dx.shape == x.shape and dw.shape == w.shape
        check_backward(x, w, gu, dh, act, dx, dw)
    gnt.gemm_nt_check()


def test_backward_empty():
    x, w, gu, dh = backward_case(5, 24, 8, BF16, "silu")
    dx, dw = gnt.gated_linear_backward(dh[:0], gu[:0], x[:0], w)
    assert dx.shape == (0, 24) and (dw == 0).all()
    dx, dw = gnt.gated_linear_backward(dh[:, :0], gu[:, :0], x, w[:0])
    assert (dx == 0).all() and dw.shape == (0, 24)
    dx, dw = gnt.gated_linear_backward(dh, gu, x[:, :0], w[:, :0])
    assert dx.shape == (5, 0) and dw.shape == (16, 0)


def test_backward_of_ends():
    """Gates where the activation is flat, up to infinity."""
    gate = torch.tensor([[0.0, 60.0, -60.0, 3e38, -3e38, math.inf, -math.inf, 1e-30]], dtype=BF16, device="cuda")
    n = gate.shape[1]
    gu = torch.cat((gate, torch.full_like(gate, 2.0)), 1)
    dgu = torch.zeros_like(gu)
    dh = torch.ones_like(gate)
    for i, act in enumerate(ACTS):
        gnt.gemm_nt_gated_grad(dh.data_ptr(), n, gu.data_ptr(), 2 * n, dgu.data_ptr(), 2 * n, gnt.DType.BF16, i, 1, n,
                               torch.cuda.current_stream().cuda_stream)
        got = dgu[0].float().tolist()
        # at -60 silu is -60 / (1 + e^60), not nothing: its slope is 59 e^-60 < 1e-24 in magnitude
        assert got[:2] == [1, 2] and abs(got[2]) < 2e-24 and got[3:8] == [2, 0, 2, 0, 1]
        assert got[8:10] == [0, 60] and abs(got[10]) < 1e-24 and got[11:14] == [gate[0, 3].item(), 0, math.inf]


def test_gradient_against_differences():
    """g and u that 16 bits hold exactly: the kernel's gradients against the
    differences of the kernel-free formula."""
    g = gen(3)
    x = (torch.randint(-4, 5, (5, 16), generator=g, device="cuda") / 4).to(F16)
    w = (torch.randint(-4, 5, (12, 16), generator=g, device="cuda") / 8).to(F16)
    dh = (torch.randint(-8, 9, (5, 6), generator=g, device="cuda") / 8).to(F16)
    for act in ACTS:
        def loss(xd, wd):
            a, b = (xd @ wd.t()).chunk(2, 1)
            return (act64(a, act)[0] * b * dh.double()).sum()

        _, gu = gnt.gated_linear(x, w, activation=act, keep=True)
        assert torch.equal(gu.double(), x.double() @ w.double().t())
        dx, dw = gnt.gated_linear_backward(dh, gu, x, w, activation=act)
        for got, of in ((dx, 0), (dw, 1)):
            base = [x.double(), w.double()]
            for idx in [(0, 0), (1, 3), (4, 15), (2, 8)]:
                lo, hi = base[of].clone(), base[of].clone()
                step = 1e-5
                lo[idx] -= step
                hi[idx] += step
                at = lambda t: loss(t, base[1]) if of == 0 else loss(base[0], t)  # noqa: E731
                diff = float((at(hi) - at(lo)) / (2 * step))
                # sums of at most 12 terms below 4 in magnitude, each factor rounded to
                # fp16 by 2^-11, the result again; the difference is good to 1e-7
                assert abs(float(got[idx]) - diff) <= 2.0 ** -11 * (12 * 4 + abs(diff)) + 1e-6


def quantize_ref(w, group, zeros, kind):
    """Codes, scales and zero points on the CPU: fp32, each step rounded."""
    w = w.float().cpu()
    n, k = w.shape
    groups = -(-k // group)
    full = torch.zeros(n, groups * group)
    full[:, :k] = w
    full = full.view(n, groups, group)
    seventh, fifteenth = torch.tensor(1 / 7), torch.tensor(1 / 15)
    lo, hi = full.amin(2).clamp(max=0), full.amax(2).clamp(min=0)
    s = ((hi - lo) * fifteenth if zeros else torch.maximum(hi, -lo) * seventh).to(kind)
    f = s.float()
    inv = torch.where(f > 0, torch.ones(()) / f, torch.zeros(()))
    q = torch.round(full * inv[..., None])
    if zeros:
        z = torch.round(-lo * inv).clamp(0, 15)
        q = (q + z[..., None]).clamp(0, 15)
    else:
        z, q = None, q.clamp(-8, 7) + 8
    return q.reshape(n, -1)[:, :k].to(torch.uint8), s, None if z is None else z.to(torch.uint8)


def unpack(q, k):
    return torch.stack((q & 15, q >> 4), -1).reshape(q.shape[0], -1)[:, :k]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("wt,st", [(torch.float32, BF16), (torch.float32, F16), (BF16, BF16), (F16, F16), (F16, BF16)])
def test_quantize(wt, st, group, zeros):
    for n, k, extra in ((1, 1, 0), (1, 31, 0), (3, 32, 0), (5, 33, 3), (17, 520, 0), (9, 1000, 1), (40, 2049, 0), (300, 256, 8)):
        g = gen(n + k)
        w = normal(g, n, k, scale=0.02, dtype=wt, pitch=k + extra)
        w[0] = 0
        if n > 4:
            w[1] = w[1].abs()          # zero points at the ends
            w[2] = -w[2].abs()
            w[3] = (w[3] * 350).round() / 2  # ties
            w[4] *= 1e-30 if wt != F16 else 0
        ref = quantize_ref(w, group, zeros, st)
        got = gnt.quantize_w4(w, group=group, zeros=zeros, scale_dtype=st)
        assert torch.equal(unpack(got[0].cpu(), k), ref[0])
        assert torch.equal(got[1].cpu(), ref[1])
        if zeros:
            assert torch.equal(got[2].cpu(), ref[2])
        if k % 2:
            assert (got[0][:, -1] >> 4 == 0).all()
    assert gnt.quantize_w4(w[:0])[0].shape == (0, 128) and gnt.quantize_w4(w[:, :0])[1].shape == (300, 0)

@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("wt", [torch.float32, BF16, F16])
@pytest.mark.parametrize("pitch,offset", [(1000, 0), (1004, 0), (1004, 4), (1002, 0), (1002, 2), (1001, 0), (1000, 1), (1008, 12)])
def test_quantize_alignments(pitch, offset, wt, zeros):
    """Rows on boundaries of 16, 8, 4 and 2 bytes, and columns that end inside a thread's 32."""
    for cols in (32, 96, 999, 1000):
        w = normal(gen(cols + pitch), 37, cols, dtype=wt, pitch=pitch, offset=offset)
        out = gnt.quantize_w4(w, 64, zeros, BF16)
        ref = quantize_ref(w, 64, zeros, BF16)
        assert torch.equal(unpack(out[0], cols).cpu(), ref[0]) and torch.equal(out[1].cpu(), ref[1])
        assert not zeros or torch.equal(out[2].cpu(), ref[2])
    gnt.gemm_nt_check()



def test_quantize_of_infinities():
    w = torch.ones(4, 128, device="cuda")
    w[0, 5], w[1, 40], w[2, 3] = math.inf, math.nan, -math.inf
    for zeros in (False, True):
        out = gnt.quantize_w4(w, group=32, zeros=zeros)
        bad = torch.zeros(4, 4, dtype=torch.bool)
        bad[0, 0] = bad[1, 1] = bad[2, 0] = True
        assert torch.equal(out[1].isnan().cpu(), bad)
        assert (unpack(out[0], 128).view(4, 4, 32)[bad.cuda()] == (0 if zeros else 8)).all()


def test_quantize_leaves_the_bytes_between_rows():
    w = normal(gen(1), 20, 77, dtype=torch.float32)
    codes = torch.full((20, 50), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((20, 5), 9.0, dtype=BF16, device="cuda")
    z = torch.full((20, 6), 99, dtype=torch.uint8, device="cuda")
    gnt.gemm_nt_w4_quantize(w.data_ptr(), gnt.DType.F32, 20, 77, 77,
                            gnt.Weights4(codes.data_ptr(), 50, s.data_ptr(), 5, z.data_ptr(), 6, 32), gnt.DType.BF16,
                            torch.cuda.current_stream().cuda_stream)
    ref = quantize_ref(w, 32, True, BF16)
    assert torch.equal(unpack(codes[:, :39], 77).cpu(), ref[0]) and (codes[:, 39:] == 0xA5).all()
    assert torch.equal(s[:, :3].cpu(), ref[1]) and (s[:, 3:] == 9).all()
    assert torch.equal(z[:, :3].cpu(), ref[2]) and (z[:, 3:] == 99).all()


def weights4(g, rows, k, group, zeros, dtype, pitch=0, offset=0):
    """Random codes, with scales of different sizes from group to group."""
    width, groups = (k + 1) // 2, -(-k // group)
    pitch = pitch or (width + 15) // 16 * 16
    store = torch.randint(0, 256, (offset + rows * pitch,), generator=g, device="cuda", dtype=torch.uint8)
    q = store[offset:].view(rows, pitch)[:, :width]
    s = (torch.rand(rows, groups, generator=g, device="cuda") * 2 + 0.1) * k ** -0.5 / 4
    z = torch.randint(0, 16, (rows, groups), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return q, s.to(dtype), z


def weight_eps(tokens, dtype):
    """How far kernels may round a weight's value: not at all up to 16 tokens."""
    return 0.0 if tokens <= 16 else EPS[dtype]


@pytest.mark.parametrize("dtype,group,zeros", [(BF16, 128, False), (BF16, 32, True), (F16, 64, True), (F16, 128, False)])
@pytest.mark.parametrize("shape", SHAPES)
def test_w4(shape, dtype, group, zeros):
    m, k, n, extra = shape
    g = gen(m + k + n)
    x = normal(g, m, k, dtype=dtype, pitch=k + extra)
    q, s, z = weights4(g, n, k, group, zeros, dtype)
    w = w4_values(q, s, z, group, k)
    ref, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    # code and zero may be multiplied apart: their sums are up to 3 times |code - zero|'s share of 15
    wide = x.double().abs() @ (w.abs() + 31 * s.double()[:, torch.arange(k, device="cuda") // group]).t()
    bound = sum_error(wide, k) + weight_eps(m, dtype) * mag
    out = gnt.linear_w4(x, q, s, z, group=group)
    check(out, ref, rounded(bound, ref, dtype))
    into = torch.full((m, n + 3), 7.0, dtype=dtype, device="cuda")
    gnt.linear_w4(x, q, s, z, group=group, out=into[:, :n])
    check(into[:, :n], ref, rounded(bound, ref, dtype))
    assert (into[:, n:] == 7).all()
    gnt.gemm_nt_check()


@pytest.mark.parametrize("dtype,group,zeros", [(BF16, 128, True), (F16, 32, False), (BF16, 64, False)])
@pytest.mark.parametrize("shape", SHAPES)
def test_w4_gated(shape, dtype, group, zeros):
    m, k, n, extra = shape
    g = gen(m + k + n)
    x = normal(g, m, k, dtype=dtype, pitch=k + extra)
    q, s, z = weights4(g, 2 * n, k, group, zeros, dtype)
    w = w4_values(q, s, z, group, k)
    wide = w.abs() + 31 * s.double()[:, torch.arange(k, device="cuda") // group]
    for act in ACTS:
        h, y, _, _ = gated_bound(x, w, act)
        err = sum_error(x.double().abs() @ wide.t(), k) + weight_eps(m, dtype) * (x.double().abs() @ w.abs().t())
        gate, up, eg, eu = y[:, :n], y[:, n:], err[:, :n], err[:, n:]
        ea = 1.13 * eg + 2.0 ** -19 * gate.abs()
        bound = ea * up.abs() + act64(gate, act)[0].abs() * eu + ea * eu
        out = gnt.gated_linear_w4(x, q, s, z, group=group, activation=act)
        check(out, h, rounded(bound, h, dtype), act)
    gnt.gemm_nt_check()


@pytest.mark.parametrize("m", [1, 5, 40, 200])
@pytest.mark.parametrize("offset,pitch", [(0, 0), (0, 263), (1, 264), (4, 260), (16, 272)])
def test_w4_alignments(offset, pitch, m):
    """Rows of codes anywhere, what lies between them random."""
    g = gen(offset + m)
    k, n = 520, 72
    x = normal(g, m, k, dtype=F16, pitch=k + offset, offset=offset)
    q, s, z = weights4(g, n, k, 64, True, F16, pitch, offset)
    w = w4_values(q, s, z, 64, k)
    ref, wide = x.double() @ w.t(), x.double().abs() @ (w.abs() + 31 * s.double()[:, torch.arange(k, device="cuda") // 64]).t()
    check(gnt.linear_w4(x, q, s, z, group=64), ref,
          rounded(sum_error(wide, k) + weight_eps(m, F16) * (x.double().abs() @ w.abs().t()), ref, F16))
    gnt.gemm_nt_check()


@pytest.mark.parametrize("path", [P.SKINNY, P.TC05, P.MMASYNC])
@pytest.mark.parametrize("m,k,n", [(1, 4096, 64), (4, 8192, 96), (13, 2050, 40), (40, 6000, 200), (64, 4104, 136), (257, 1000, 300),
                                   (600, 264, 1030), (1, 32, 2000), (130, 8, 16)])
def test_w4_paths(path, m, k, n):
    """Every kernel, with and without a split of K."""
    m = min(m, 16, 65536 // ((k + 127) // 128 * 128)) if path == P.SKINNY else m  # the tokens lie in shared memory
    for dtype, group, zeros in ((BF16, 128, True), (F16, 32, False)):
        g = gen(m + k)
        x = normal(g, m, k, dtype=dtype, pitch=(k + 7) // 8 * 8)
        q, s, z = weights4(g, 2 * n, k, group, zeros, dtype)
        w = w4_values(q, s, z, group, k)
        wide = w.abs() + 31 * s.double()[:, torch.arange(k, device="cuda") // group]
        err = sum_error(x.double().abs() @ wide.t(), k) + EPS[dtype] * (path == P.TC05) * (x.double().abs() @ w.abs().t())
        y = x.double() @ w.t()
        check(gnt.linear_w4(x, q, s, z, group=group, path=path), y, rounded(err, y, dtype))
        gate, up, eg, eu = y[:, :n], y[:, n:], err[:, :n], err[:, n:]
        a, ea = act64(gate, "silu")[0], 1.13 * eg + 2.0 ** -19 * gate.abs()
        check(gnt.gated_linear_w4(x, q, s, z, group=group, path=path), a * up,
              rounded(ea * up.abs() + a.abs() * eu + ea * eu, a * up, dtype))
    gnt.gemm_nt_check()


def test_w4_of_what_was_quantised():
    """Weights through the quantiser and the product: off by half a step of their
    group at most, and a clamped end's."""
    g = gen(9)
    w = normal(g, 96, 1000, scale=0.03)
    for zeros in (False, True):
        got = gnt.quantize_w4(w, group=64, zeros=zeros)
        v = w4_values(got[0], got[1], got[2] if zeros else None, 64, 1000)
        step = got[1].double()[:, torch.arange(1000, device="cuda") // 64]
        # half a step; the scale's rounding (2^-9 of 7 or 15 steps) may clamp the ends, the zero point's moves them by half a step
        assert ((v - w.double()).abs() <= (0.5 + 15 * 2.0 ** -8 + 0.5 * zeros) * step).all()


def test_empty_sums():
    x = torch.zeros(4, 0, dtype=BF16, device="cuda")
    q, s = torch.zeros(6, 0, dtype=torch.uint8, device="cuda"), torch.zeros(6, 0, dtype=BF16, device="cuda")
    assert (gnt.linear_w4(x, q, s) == 0).all() and (gnt.gated_linear_w4(x, q, s) == 0).all()
    x, (q, s, z) = torch.zeros(0, 64, dtype=BF16, device="cuda"), weights4(gen(1), 6, 64, 32, False, BF16)
    assert gnt.linear_w4(x, q, s, group=32).shape == (0, 6)
    assert gnt.linear_w4(torch.zeros(3, 64, dtype=BF16, device="cuda"), q[:0], s[:0], group=32).shape == (3, 0)


@pytest.mark.parametrize("offset", [0, 1, 2, 4, 16, 30])
def test_copy_rows(offset):
    """Every unit that a source's alignment allows, and bytes between the rows left alone."""
    for rows, width, pitch in ((1, 1, 1), (3, 15, 16), (7, 16, 17), (70, 1001, 1002), (40, 4096, 4100), (2, 70000, 70016)):
        src = torch.randint(0, 256, (offset + rows * pitch,), dtype=torch.uint8, device="cuda")
        ldd = (width + 15) // 16 * 16 + 16
        dst = torch.full((rows, ldd), 0xA5, dtype=torch.uint8, device="cuda")
        gnt.gemm_nt_copy_rows(src.data_ptr() + offset, pitch, dst.data_ptr(), ldd, rows, width,
                              torch.cuda.current_stream().cuda_stream)
        assert torch.equal(dst[:, :width], src[offset:].view(rows, pitch)[:, :width])
        assert (dst[:, width:] == 0xA5).all()


@pytest.mark.parametrize("m", [1, 16, 17, 70, 300])
@pytest.mark.parametrize("k,offset", [(1001, 0), (1002, 3), (1000, 1), (1004, 4)])
def test_rows_off_the_grid(k, offset, m):
    """Operands that are copied first, and the same calls on the warp kernel."""
    n = 300
    g = gen(k + m)
    x = normal(g, m, k, dtype=F16, pitch=k + offset, offset=offset)
    w = normal(g, 2 * n, k, scale=k ** -0.5, dtype=F16, pitch=k + offset, offset=offset)
    h, y, eh, ey = gated_bound(x, w, "gelu")
    for path in (P.AUTO, P.MMASYNC):
        out, gu = gnt.gated_linear(x, w, "gelu", keep=True, path=path)
        check(out, h, rounded(eh, h, F16))
        check(gu, y, rounded(ey, y, F16))
    dh = normal(g, m, n, scale=0.1, dtype=F16)
    check_backward(x, w, gu, dh, "gelu", *gnt.gated_linear_backward(dh, gu, x, w, "gelu"))
    q, s, z = weights4(g, n, k, 32, True, F16)
    v = w4_values(q, s, z, 32, k)
    wide = x.double().abs() @ (v.abs() + 31 * s.double()[:, torch.arange(k, device="cuda") // 32]).t()
    ref, mag = x.double() @ v.t(), x.double().abs() @ v.abs().t()
    check(gnt.linear_w4(x, q, s, z, group=32), ref, rounded(sum_error(wide, k) + weight_eps(m, F16) * mag, ref, F16))
    gnt.gemm_nt_check()
