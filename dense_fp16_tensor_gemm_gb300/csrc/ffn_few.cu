// ffn_few.cu -- gated products, and plain and gated products with 4-bit weights,
// for up to 16 tokens on the warp MMA: a stream of the weights.
//
// Bound by memory, and with 4-bit weights by the instructions that turn codes into
// operands: every weight is read once and meets at most 16 tokens.  The weights are
// the MMA's A operand (16 rows by 16 of K), the tokens its 8 columns.  A CTA of 16
// warps walks over tiles of 16 rows (of a gated product 8 of the gate and the same 8
// of the up projection, so that a thread ends with g and u of its outputs); its warps
// take turns along K, 64 bytes of every row at a step, and each keeps a ring of
// asynchronous 16-byte copies of its own, running on into the next tile, so that
// a tile's end costs no bandwidth.  A tile's sums meet in shared memory and one
// warp, another each time, adds them in the warps' order.  The tokens lie in shared
// memory for all tiles, in the order in which the MMA's lanes read them.
//
// Which of K's elements a thread multiplies is free as long as weights and tokens
// agree.  16-bit weights: thread t of a quad has elements [8t, 8t+8) of a step's
// 32, one 16-byte load of either operand and two MMAs.  4-bit weights: a step is
// 128 of K; in groups of 128 thread t has [32t, 32t+32), one 16-byte load, else
// [8t, 8t+8) of each 32, so that an MMA stays inside a group.  An `and` of a word of
// codes shifted by 4i gives elements i and i + 4 as small whole numbers in the low
// bits of 1024 + code (fp16) or 128 + code (bf16), from which 1024 + zero or 128 +
// zero is subtracted: exact, so the MMA sums (code - zero) x, and a group's sum is
// scaled in fp32.
#include <algorithm>

#include "ffn.h"
#include "ptx.cuh"

namespace gnt {

namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kDepth = 4;       // steps in flight per warp
constexpr int kStep = 1024;     // bytes: 16 rows of 64

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
    if (vec && K - k >= 8)
        return __ldg(reinterpret_cast<const uint4*>(row + k));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < K)
            w[i >> 1] |= static_cast<uint32_t>(__ldg(row + k + i)) << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Bytes of the tokens in shared memory.
int64_t x_bytes(const FfnParams& p)
{
    const int step = p.scales ? 128 : 32;
    return (int64_t(p.k) + step - 1) / step * step * 2 * p.tokens;
}
constexpr int red_bytes(int nt) { return 2 * kWarps * nt * 512; }
constexpr int kMaxSmem = 227 * 1024;

// NT: sets of 8 tokens.  G128: groups of 128.
template <bool BF16, bool W4, bool GATED, int NT, bool G128>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) ffn_few_kernel(const FfnParams p, int vec_x, int tiles)
{
    using S = OutStore<BF16 ? kOutBF16 : kOutF16>;
    constexpr int kRows = GATED ? 8 : 16;  // outputs per tile
    constexpr int XV = W4 ? 4 : 1;         // 16-byte pieces of a token per step
    constexpr int kStepK = W4 ? 128 : 32;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * (kDepth * kStep);
    float4* const red = reinterpret_cast<float4*>(smem + kWarps * kDepth * kStep);
    uint4* const xs = reinterpret_cast<uint4*>(smem + kWarps * kDepth * kStep + red_bytes(NT));

    pdl_launch_dependents();
    pdl_wait();

    const int row_bytes = W4 ? (p.k >> 1) + (p.k & 1) : 2 * p.k;
    const int steps = (row_bytes + 63) >> 6;
    const int count = steps > warp ? (steps - warp + kWarps - 1) / kWarps : 0;  // of this warp, per tile

    // What is fetched next: step `fi` of tile `ft`.  This lane copies 16 bytes of rows
    // lane / 4 and lane / 4 + 8, and fetches the scales and zeros of those rows for the 32
    // elements 32 t of the step.
    int ft = blockIdx.x, fi = 0;
    const uint8_t* src[2];
    const uint16_t* srow[2];
    const uint8_t* zrow[2];
    int valid = 0;
    const auto open = [&] {
        valid = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int o = ft * kRows + (GATED ? g : g + 8 * h);
            const bool in = ft < tiles && o < p.n;
            // (rows past the weights: the first one's scales, and zeros for codes)
            const int64_t row = in ? o + (GATED && h ? static_cast<int64_t>(p.n) : 0) : 0;
            valid |= in ? 1 << h : 0;
            src[h] = static_cast<const uint8_t*>(p.w) + row * p.ldw * (W4 ? 1 : 2);
            if (W4) {
                srow[h] = static_cast<const uint16_t*>(p.scales) + row * p.lds;
                zrow[h] = p.zeros + row * p.ldz;
            }
        }
    };
    const uint32_t dst = g * 64 + ((t ^ ((g >> 1) & 3)) << 4);  // (row g + 8: 512 bytes on)
    const auto fetch = [&](int slot, uint32_t (&sc)[2], uint32_t (&ze)[2]) {
        if (ft < tiles) {
            const int step = warp + fi * kWarps, off = step * 64 + t * 16;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int bytes = valid & (1 << h) ? max(0, min(16, row_bytes - off)) : 0;
                // (nothing is read of an address with 0 bytes)
                cp_async16(ring + slot * kStep + dst + 512 * h, bytes ? src[h] + off : p.w, bytes);
                if (W4) {
                    // (past K: the last group's, whose end may lie there)
                    const int grp = min(step * kStepK + 32 * t, p.k - 1) >> p.group_shift;
                    sc[h] = __ldg(srow[h] + grp);
                    if (p.zeros)
                        ze[h] = __ldg(zrow[h] + grp);
                }
            }
            if (++fi == count) {
                fi = 0;
                ft += gridDim.x;
                open();
            }
        }
        cp_async_commit();
    };
    uint32_t sc[kDepth][2], ze[kDepth][2];
#pragma unroll
    for (int i = 0; i < kDepth; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sc[i][h] = 0;
            ze[i][h] = 8;
        }
    if (count > 0) {
        open();
#pragma unroll
        for (int i = 0; i < kDepth; ++i)
            fetch(i, sc[i], ze[i]);
    }

    // the tokens: [step][piece][token][t], 8 elements each, paired as the codes are
    for (int e = threadIdx.x; e < steps * XV * p.tokens * 4; e += kThreads) {
        // consecutive threads on consecutive elements of a token
        const int tok = e / (steps * XV * 4), r = e - tok * (steps * XV * 4);
        const int k = r * 8, step = r / (XV * 4), in = r % (XV * 4);
        const int j = !W4 ? 0 : (G128 ? in & 3 : in >> 2), tt = !W4 ? in : (G128 ? in >> 2 : in & 3);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (k < p.k)
            v = load_x(static_cast<const uint16_t*>(p.x) + tok * p.ldx, k, p.k, vec_x);
        if (W4)
            v = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                           __byte_perm(v.y, v.w, 0x7632));
        xs[((step * XV + j) * p.tokens + tok) * 4 + tt] = v;
    }
    __syncthreads();
    uint32_t xat[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
        xat[n] = smem_u32(xs) + (8 * n + g) * 64 + t * 16;
    const int xpiece = p.tokens * 64;  // bytes
    const uint32_t mask = G128 ? 127u : (1u << p.group_shift) - 1;

    int buf = 0, slot0 = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
        float acc[NT][4] = {};
        // one step: its codes or weights in `slot`, its scales and zeros in s and z
        const auto step = [&](int i, int slot, uint32_t (&s)[2], uint32_t (&z)[2]) {
            const int xoff = (warp + i * kWarps) * XV * xpiece;
            cp_async_wait<kDepth - 1>();
            __syncwarp();
            const uint32_t at = ring + slot * kStep;
            if constexpr (W4) {
                float f[2];
                uint32_t zero[2], words[2][4];
                if (G128) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        f[h] = value_of<BF16>(s[h]);
                        zero[h] = __byte_perm(z[h] | (BF16 ? 0x4300u : 0x6400u), 0, 0x1010);
                        const uint4 w = lds128(at + dst + 512 * h);
                        words[h][0] = w.x, words[h][1] = w.y, words[h][2] = w.z, words[h][3] = w.w;
                    }
                }
                float part[NT][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t a[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (!G128) {
                            f[h] = value_of<BF16>(__shfl_sync(0xffffffffu, s[h], (lane & ~3) | j));
                            zero[h] = __byte_perm(__shfl_sync(0xffffffffu, z[h], (lane & ~3) | j) | (BF16 ? 0x4300u : 0x6400u), 0, 0x1010);
                            words[h][j] = lds32(at + (g + 8 * h) * 64 + ((j ^ ((g >> 1) & 3)) << 4) + t * 4);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            a[h][e] = codes_at<BF16>(words[h][j], e, zero[h]);
                    }
                    const bool start = ((j << 5) & mask) == 0;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        uint4 b = make_uint4(0, 0, 0, 0);
                        if (8 * n + g < p.tokens)
                            b = lds128(xat[n] + xoff + j * xpiece);
                        if (start)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                part[n][e] = 0.f;
                        mma<BF16>(part[n], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
                        mma<BF16>(part[n], a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
                        if ((((j + 1) << 5) & mask) == 0) {  // a group's end
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                acc[n][e] = fmaf(part[n][e], f[e >> 1], acc[n][e]);
                        }
                    }
                }
            } else {
                const uint4 lo = lds128(at + dst), hi = lds128(at + dst + 512);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint4 b = make_uint4(0, 0, 0, 0);
                    if (8 * n + g < p.tokens)
                        b = lds128(xat[n] + xoff);
                    mma<BF16>(acc[n], lo.x, hi.x, lo.y, hi.y, b.x, b.y);
                    mma<BF16>(acc[n], lo.z, hi.z, lo.w, hi.w, b.z, b.w);
                }
            }
            __syncwarp();
            fetch(slot, s, z);
        };
        // (the ring's slots, and with them the scales' registers, run on from tile to tile)
        int i = 0;
        while (i < count) {
            switch (slot0) {
            case 0: step(i, 0, sc[0], ze[0]); if (++i == count) { slot0 = 1; break; }
            case 1: step(i, 1, sc[1], ze[1]); if (++i == count) { slot0 = 2; break; }
            case 2: step(i, 2, sc[2], ze[2]); if (++i == count) { slot0 = 3; break; }
            default: step(i, 3, sc[3], ze[3]); ++i; slot0 = 0;
            }
        }
        // the tile's sums
        float4* const mine = red + (buf * kWarps + warp) * (NT * 32) + lane;
#pragma unroll
        for (int n = 0; n < NT; ++n)
            mine[n * 32] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
        __syncthreads();
        if (warp != tile / static_cast<int>(gridDim.x) % kWarps)
            continue;
        typename S::T* out = static_cast<typename S::T*>(p.out);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float v[4] = {};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 a = red[(buf * kWarps + w) * (NT * 32) + n * 32 + lane];
                v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int tok = 8 * n + 2 * t + e;
                if (tok >= p.tokens)
                    continue;
                const int o = tile * kRows + g;
                if (GATED) {
                    if (o < p.n) {
                        S::st1(out + tok * p.ldo + o, act_value(v[e], p.act) * v[2 + e]);
                        if (!W4 && p.gu) {
                            typename S::T* gu = static_cast<typename S::T*>(p.gu) + tok * p.ldgu;
                            S::st1(gu + o, v[e]);
                            S::st1(gu + p.n + o, v[2 + e]);
                        }
                    }
                } else {
                    if (o < p.n)
                        S::st1(out + tok * p.ldo + o, v[e]);
                    if (o + 8 < p.n)
                        S::st1(out + tok * p.ldo + o + 8, v[2 + e]);
                }
            }
        }
    }
    cp_async_wait<0>();
}

template <bool BF16, bool W4, bool GATED, int NT, bool G128>
cudaError_t run(const FfnParams& p, int num_sms, cudaStream_t stream, bool configure)
{
    auto* kernel = ffn_few_kernel<BF16, W4, GATED, NT, G128>;
    if (configure)
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    const int vec_x = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ldx % 8 == 0;
    const int smem = kWarps * kDepth * kStep + red_bytes(NT) + static_cast<int>(x_bytes(p));
    constexpr int per = GATED ? 8 : 16;
    const int tiles = static_cast<int>((int64_t(p.n) + per - 1) / per);
    const int resident = NT == 1 && 2 * (smem + 1024) <= kMaxSmem + 1024 ? 2 : 1;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min(tiles, resident * num_sms)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, vec_x, tiles);
}

template <bool BF16, bool W4, bool GATED>
cudaError_t by_tokens(const FfnParams& p, int num_sms, cudaStream_t stream, bool configure)
{
    cudaError_t e = cudaSuccess;
    const bool g128 = p.group_shift == 7;
    if constexpr (W4) {
        if (configure || (p.tokens <= 8 && g128)) e = run<BF16, W4, GATED, 1, true>(p, num_sms, stream, configure);
        if (e == cudaSuccess && (configure || (p.tokens > 8 && g128))) e = run<BF16, W4, GATED, 2, true>(p, num_sms, stream, configure);
    }
    if (e == cudaSuccess && (configure || (p.tokens <= 8 && !g128))) e = run<BF16, W4, GATED, 1, false>(p, num_sms, stream, configure);
    if (e == cudaSuccess && (configure || (p.tokens > 8 && !g128))) e = run<BF16, W4, GATED, 2, false>(p, num_sms, stream, configure);
    return e;
}

template <bool BF16>
cudaError_t by_kind(const FfnParams& p, int num_sms, cudaStream_t stream, bool configure)
{
    cudaError_t e = cudaSuccess;
    if (configure || (p.scales && !p.gated)) e = by_tokens<BF16, true, false>(p, num_sms, stream, configure);
    if (e == cudaSuccess && (configure || (p.scales && p.gated))) e = by_tokens<BF16, true, true>(p, num_sms, stream, configure);
    if (e == cudaSuccess && (configure || !p.scales)) e = by_tokens<BF16, false, true>(p, num_sms, stream, configure);
    return e;
}

}  // namespace

bool ffn_few_fits(const FfnParams& p)
{
    return p.tokens <= kFewTokens && x_bytes(p) <= 128 * 1024;
}

cudaError_t ffn_few_configure()
{
    const FfnParams p{};
    const cudaError_t e = by_kind<true>(p, 0, nullptr, true);
    return e == cudaSuccess ? by_kind<false>(p, 0, nullptr, true) : e;
}

cudaError_t ffn_few_launch(const FfnParams& p, int num_sms, cudaStream_t stream)
{
    return p.bf16 ? by_kind<true>(p, num_sms, stream, false) : by_kind<false>(p, num_sms, stream, false);
}

}  // namespace gnt
