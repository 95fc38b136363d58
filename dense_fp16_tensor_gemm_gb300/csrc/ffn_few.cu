// ffn_few.cu -- gated products, and plain and gated products with 4-bit weights,
// for up to 16 tokens on the warp MMA: a stream of the weights.
//
// Bound by memory: every weight is read once and meets at most 16 tokens, so the
// kernel is built around its loads.  The weights are the MMA's A operand (16 rows
// by 16 of K), the tokens its 8 columns.  A CTA of 8 warps owns 16 or 32 rows (of
// a gated product half of them the gate's and half the same rows of the up
// projection, so that a thread ends with g and u of its outputs) and its warps
// take turns along K, 64 bytes of every row at a step: each keeps a ring of
// asynchronous 16-byte copies of its own ahead of it and waits for nobody.
// Sums meet in shared memory at the end, in the warps' order.
//
// Which of K's elements a thread multiplies is free as long as weights and tokens
// agree.  16-bit weights: thread t of a quad has elements [8t, 8t+8) of a step's
// 32, one 16-byte load of either operand and two MMAs.  4-bit weights: of each 32
// of a step's 128 (a group has at least 32) it has [8t, 8t+8), one word of codes;
// an `and` of the word shifted by 4i gives elements i and i + 4 as two small whole
// numbers in the low bits of 1024 + code (fp16) or 128 + code (bf16), from which
// 1024 + zero or 128 + zero is subtracted: exact, so the MMA sums
// (code - zero) x, and a group's sum is scaled in fp32.
#include <algorithm>

#include "ffn.h"
#include "ptx.cuh"

namespace gnt {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    const uint32_t a[4] = {a0, a1, a2, a3};
    if (BF16)
        mma_m16n8k16_bf16(d, a, b0, b1, d);
    else
        mma_m16n8k16(d, a, b0, b1, d);
}

template <bool BF16>
__device__ __forceinline__ float value_of(uint32_t bits)
{
    return BF16 ? __uint_as_float(bits << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}

// Elements i and i + 4 of a word of codes, less the zero in `magic_zero` (twice).
template <bool BF16>
__device__ __forceinline__ uint32_t codes_at(uint32_t word, int i, uint32_t magic_zero)
{
    constexpr uint32_t magic = BF16 ? 0x43004300u : 0x64006400u;
    const uint32_t v = ((word >> (4 * i)) & 0x000f000fu) | magic;
    if (BF16) {
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&magic_zero));
        return *reinterpret_cast<const uint32_t*>(&d);
    }
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&magic_zero));
    return *reinterpret_cast<const uint32_t*>(&d);
}

// Elements [k, k + 8) of a token, zeros past K.
__device__ __forceinline__ uint4 load_x(const uint16_t* row, int k, int K, bool vec)
{
    uint4 v = make_uint4(0, 0, 0, 0);
    if (!row || k >= K)
        return v;
    if (vec && K - k >= 8)
        return __ldg(reinterpret_cast<const uint4*>(row + k));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < K)
            w[i >> 1] |= static_cast<uint32_t>(__ldg(row + k + i)) << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// MT: sets of 16 rows per CTA; NT: sets of 8 tokens.
template <bool BF16, bool W4, bool GATED, int NT, int MT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2) ffn_few_kernel(const FfnParams p, int vec_x)
{
    using S = OutStore<BF16 ? kOutBF16 : kOutF16>;
    constexpr int kDepth = 8 / MT;              // steps in flight per warp
    constexpr int kStep = MT * 1024;            // bytes
    constexpr int kRows = GATED ? 8 : 16;       // outputs per set of rows
    constexpr int XV = W4 ? 4 : 1;              // 16-byte pieces of a token per step
    constexpr int kStepK = W4 ? 128 : 32;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * (kDepth * kStep);
    const int out0 = blockIdx.x * (MT * kRows);

    pdl_launch_dependents();
    pdl_wait();

    const int row_bytes = W4 ? (p.k >> 1) + (p.k & 1) : 2 * p.k;
    const int steps = (row_bytes + 63) >> 6;
    const int count = steps > warp ? (steps - warp + kWarps - 1) / kWarps : 0;

    // this lane's copies of a step: 16 bytes of rows (lane + 32 i) / 4
    const uint8_t* src[2 * MT];
    uint32_t dst[2 * MT];
    const int c16 = (lane & 3) * 16;
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
        const int r = (lane >> 2) + 8 * (i & 1), o = out0 + (i >> 1) * kRows + (GATED ? (r & 7) : r);
        const int64_t row = o + (GATED && r >= 8 ? static_cast<int64_t>(p.n) : 0);
        src[i] = o < p.n ? static_cast<const uint8_t*>(p.w) + row * p.ldw * (W4 ? 1 : 2) : nullptr;
        dst[i] = (i >> 1) * 1024 + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4);
    }
    const auto issue = [&](int i) {
        if (i < count) {
            const int off = (warp + i * kWarps) * 64 + c16;
            const uint32_t slot = ring + (i % kDepth) * kStep;
#pragma unroll
            for (int c = 0; c < 2 * MT; ++c) {
                const int bytes = src[c] ? max(0, min(16, row_bytes - off)) : 0;
                // (nothing is read of an address with 0 bytes)
                cp_async16(slot + dst[c], bytes ? src[c] + off : p.w, bytes);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth; ++i)
        issue(i);

    const uint16_t* xrow[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
        xrow[n] = 8 * n + g < p.tokens ? static_cast<const uint16_t*>(p.x) + (8 * n + g) * p.ldx : nullptr;
    // the scale (low half) and zero of the 32 elements 32 t of a step, for rows g and g + 8 of each set
    const uint16_t* srow[2 * MT];
    const uint8_t* zrow[2 * MT];
    if (W4) {
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            const int r = g + 8 * (i & 1), o = out0 + (i >> 1) * kRows + (GATED ? g : r);
            const int64_t row = o + (GATED && (i & 1) ? static_cast<int64_t>(p.n) : 0);
            srow[i] = o < p.n ? static_cast<const uint16_t*>(p.scales) + row * p.lds : nullptr;
            zrow[i] = o < p.n && p.zeros ? p.zeros + row * p.ldz : nullptr;
        }
    }
    uint4 x[NT][XV];
    uint32_t sz[2 * MT];
    const auto fetch = [&](int i, uint4 (&xv)[NT][XV], uint32_t (&s)[2 * MT]) {
        const int k0 = (warp + i * kWarps) * kStepK;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < XV; ++j)
                xv[n][j] = load_x(i < count ? xrow[n] : nullptr, k0 + 32 * j + 8 * t, p.k, vec_x);
        if (W4) {
            const int k = k0 + 32 * t;
#pragma unroll
            for (int c = 0; c < 2 * MT; ++c) {
                s[c] = 8u << 16;
                if (i < count && srow[c]) {
                    // (past K: the last group's, whose end may lie there)
                    const int grp = min(k, p.k - 1) >> p.group_shift;
                    s[c] = __ldg(srow[c] + grp) | (zrow[c] ? static_cast<uint32_t>(__ldg(zrow[c] + grp)) : 8u) << 16;
                }
            }
        }
    };
    fetch(0, x, sz);

    float acc[MT][NT][4] = {};
    float part[MT][NT][4] = {};
    const uint32_t mask = (1u << p.group_shift) - 1;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
        uint4 xn[NT][XV];
        uint32_t szn[2 * MT];
        fetch(i + 1, xn, szn);
        cp_async_wait<kDepth - 1>();
        __syncwarp();
        const uint32_t slot = ring + (i % kDepth) * kStep;
        if constexpr (W4) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t b[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 v = x[n][j];
                    b[n][0] = __byte_perm(v.x, v.z, 0x5410);
                    b[n][1] = __byte_perm(v.x, v.z, 0x7632);
                    b[n][2] = __byte_perm(v.y, v.w, 0x5410);
                    b[n][3] = __byte_perm(v.y, v.w, 0x7632);
                }
                float f[2 * MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    uint32_t a[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t pair = __shfl_sync(0xffffffffu, sz[2 * m + h], (lane & ~3) | j);
                        f[2 * m + h] = value_of<BF16>(pair & 0xffffu);
                        const uint32_t zero = __byte_perm((pair >> 16) | (BF16 ? 0x4300u : 0x6400u), 0, 0x1010);
                        const uint32_t word = lds32(slot + m * 1024 + (g + 8 * h) * 64 + ((j ^ ((g >> 1) & 3)) << 4) + t * 4);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            a[h][e] = codes_at<BF16>(word, e, zero);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma<BF16>(part[m][n], a[0][0], a[1][0], a[0][1], a[1][1], b[n][0], b[n][1]);
                        mma<BF16>(part[m][n], a[0][2], a[1][2], a[0][3], a[1][3], b[n][2], b[n][3]);
                    }
                }
                if ((((j + 1) << 5) & mask) == 0) {  // a group's end
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                acc[m][n][e] = fmaf(part[m][n][e], f[2 * m + (e >> 1)], acc[m][n][e]);
                                part[m][n][e] = 0.f;
                            }
                }
            }
        } else {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint32_t at = slot + m * 1024 + g * 64 + ((t ^ ((g >> 1) & 3)) << 4);
                const uint4 lo = lds128(at), hi = lds128(at + 512);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma<BF16>(acc[m][n], lo.x, hi.x, lo.y, hi.y, x[n][0].x, x[n][0].y);
                    mma<BF16>(acc[m][n], lo.z, hi.z, lo.w, hi.w, x[n][0].z, x[n][0].w);
                }
            }
        }
        __syncwarp();
        issue(i + kDepth);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < XV; ++j)
                x[n][j] = xn[n][j];
#pragma unroll
        for (int c = 0; c < 2 * MT; ++c)
            sz[c] = szn[c];
    }
    cp_async_wait<0>();
    __syncthreads();  // the rings are read out: their memory takes the sums
    float4* red = reinterpret_cast<float4*>(smem);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            red[(warp * (MT * NT) + m * NT + n) * 32 + lane] = make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
    __syncthreads();
    if (threadIdx.x < MT * NT * 32) {
        const int set = threadIdx.x >> 5, m = set / NT, n = set % NT;
        float v[4] = {};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 a = red[(w * (MT * NT) + set) * 32 + lane];
            v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        }
        typename S::T* out = static_cast<typename S::T*>(p.out);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int tok = 8 * n + 2 * t + e;
            if (tok >= p.tokens)
                continue;
            if (GATED) {
                const int o = out0 + m * 8 + g;
                if (o < p.n) {
                    S::st1(out + tok * p.ldo + o, act_value(v[e], p.act) * v[2 + e]);
                    if (!W4 && p.gu) {
                        typename S::T* gu = static_cast<typename S::T*>(p.gu) + tok * p.ldgu;
                        S::st1(gu + o, v[e]);
                        S::st1(gu + p.n + o, v[2 + e]);
                    }
                }
            } else {
                const int o = out0 + m * 16 + g;
                if (o < p.n)
                    S::st1(out + tok * p.ldo + o, v[e]);
                if (o + 8 < p.n)
                    S::st1(out + tok * p.ldo + o + 8, v[2 + e]);
            }
        }
    }
}

constexpr int kSmem = kWarps * 8 * 1024;

template <bool BF16, bool W4, bool GATED, int NT, int MT>
cudaError_t run(const FfnParams& p, int vec_x, cudaStream_t stream, bool configure)
{
    auto* kernel = ffn_few_kernel<BF16, W4, GATED, NT, MT>;
    if (configure)
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    constexpr int per = MT * (GATED ? 8 : 16);
    cfg.gridDim = dim3(static_cast<unsigned>((int64_t(p.n) + per - 1) / per));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, vec_x);
}

template <bool BF16, bool W4, bool GATED>
cudaError_t by_tokens(const FfnParams& p, int vec_x, cudaStream_t stream, bool configure)
{
    if (configure) {
        const cudaError_t e = run<BF16, W4, GATED, 1, 1>(p, vec_x, stream, true);
        return e == cudaSuccess ? run<BF16, W4, GATED, 2, 2>(p, vec_x, stream, true) : e;
    }
    if (p.tokens <= 8)
        return run<BF16, W4, GATED, 1, 1>(p, vec_x, stream, false);
    return run<BF16, W4, GATED, 2, 2>(p, vec_x, stream, false);
}

template <bool BF16>
cudaError_t by_kind(const FfnParams& p, int vec_x, cudaStream_t stream, bool configure)
{
    if (configure) {
        cudaError_t e = by_tokens<BF16, true, false>(p, vec_x, stream, true);
        if (e == cudaSuccess) e = by_tokens<BF16, true, true>(p, vec_x, stream, true);
        if (e == cudaSuccess) e = by_tokens<BF16, false, true>(p, vec_x, stream, true);
        return e;
    }
    if (!p.scales)
        return by_tokens<BF16, false, true>(p, vec_x, stream, false);
    return p.gated ? by_tokens<BF16, true, true>(p, vec_x, stream, false) : by_tokens<BF16, true, false>(p, vec_x, stream, false);
}

}  // namespace

cudaError_t ffn_few_configure()
{
    const FfnParams p{};
    const cudaError_t e = by_kind<true>(p, 0, nullptr, true);
    return e == cudaSuccess ? by_kind<false>(p, 0, nullptr, true) : e;
}

cudaError_t ffn_few_launch(const FfnParams& p, cudaStream_t stream)
{
    const int vec_x = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ldx % 8 == 0;
    return p.bf16 ? by_kind<true>(p, vec_x, stream, false) : by_kind<false>(p, vec_x, stream, false);
}

}  // namespace gnt
