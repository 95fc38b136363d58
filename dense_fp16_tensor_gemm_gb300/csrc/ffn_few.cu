// ffn_few.cu -- gated products, and plain and gated products with 4-bit weights,
// for up to 16 tokens on the warp MMA: a stream of the weights.
//
// Bound by memory, and with 4-bit weights by the latency of its loads: every weight is read once
// and meets at most 16 tokens.  The weights are
// the MMA's A operand (16 rows by 16 of K), the tokens its 8 columns.  A CTA walks
// over tiles of 16 rows (of a gated product 8 of the gate and the same 8 of the up
// projection, so that a thread ends with g and u of its outputs); its warps take turns
// along K, 128 bytes of every row at a step, and each keeps a ring of asynchronous
// 16-byte copies of its own, running on into the next tile, so that a tile's end costs
// no bandwidth.  A tile's sums meet in shared memory and one warp, another each time,
// adds them in the warps' order.  The tokens lie in shared memory for all tiles, in the
// order in which the MMA's lanes read them.
//
// Which of K's elements a thread multiplies is free as long as weights and tokens
// agree.  16-bit weights: thread t of a quad has elements [8t, 8t+8) of each 32, one
// 16-byte load of either operand and two MMAs.  4-bit weights: in groups of 128 it has
// [32t, 32t+32) of each 128, one 16-byte load, else [8t, 8t+8) of each 32, so that an MMA
// stays inside a group.  An `and` of a word of codes shifted by 4i gives elements i and
// i + 4 as small whole numbers in the low bits of 1024 + code (fp16) or 128 + code
// (bf16), from which 1024 + zero or 128 + zero is subtracted: exact, so the MMA sums
// (code - zero) x, and a group's sum is scaled in fp32.
//
// One token x 4096 x 8192 gated: 23.7 us in bf16 (134 MB, 5.7 TB/s), 13.4 in 4 bits (35 MB);
// x 4096 x 4096 in 4 bits 6.4, x 8192 x 16384 22.0.  About 4 us of each are launch, first loads
// and the last sums.  In 4 bits a step of 4096 codes takes some 400 instructions, 112 of them the
// codes' shifts and logical operations, on the ALU, the busiest pipe at 45 to 49 % of active cycles
// (issue slots 54 to 57 %); of the 10 cycles between two instructions of a warp 3 to 4 go to waiting
// for loads.  Rings of two steps
// (4-bit 12.8 and 21.6, but 4 tokens 9.0 for 8.3) and two CTAs an SM (5.4 for 4096 x 4096, 25 for
// 8192 x 16384) were measured beside three and three.
#include <algorithm>

#include "ffn.h"
#include "ptx.cuh"

namespace gnt {

namespace {

constexpr int kStep = 2048;  // bytes: 16 rows of 128

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
// The same, from zero.
template <bool BF16>
__device__ __forceinline__ void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    const uint32_t a[4] = {a0, a1, a2, a3};
    const float none[4] = {0.f, 0.f, 0.f, 0.f};
    if (BF16)
        mma_m16n8k16_bf16(d, a, b0, b1, none);
    else
        mma_m16n8k16(d, a, b0, b1, none);
}

// The scale in half `hi` of a pair.
template <bool BF16>
__device__ __forceinline__ float scale_of(uint32_t pair, int hi)
{
    if (BF16)
        return __uint_as_float(hi ? pair & 0xffff0000u : pair << 16);
    const __half2 h = *reinterpret_cast<const __half2*>(&pair);
    return hi ? __high2float(h) : __low2float(h);
}
// 1024 + zero or 128 + zero, twice, from byte `hi` of a pair of zeros.
template <bool BF16>
__device__ __forceinline__ uint32_t zero_of(uint32_t pair, int hi)
{
    return __byte_perm(pair, BF16 ? 0x43 : 0x64, hi ? 0x4141 : 0x4040);
}

// Elements i and i + 4 of a word of codes, less the zero in `magic_zero` (twice).
template <bool BF16>
__device__ __forceinline__ uint32_t codes_at(uint32_t word, int i, uint32_t magic_zero)
{
    constexpr uint32_t magic = BF16 ? 0x43004300u : 0x64006400u;
    // (word >> 4 i) & 0x000f000f | magic: one logical operation after the shift
    uint32_t v;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(word >> (4 * i)), "r"(0x000f000fu), "r"(magic));
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

int64_t x_bytes(const FfnParams& p) { return few_token_bytes(p.tokens, p.k, p.scales != nullptr); }
constexpr int kMaxSmem = 227 * 1024;

// What the tokens' memory leaves: CTAs of 8 warps, three or two to an SM, or one of 16.
template <int NT, int WARPS>
struct Cfg {
    static constexpr int kThreads = 32 * WARPS;
    static constexpr int kDepth = WARPS == 8 ? 3 : 2;  // steps in flight per warp
    static constexpr int kRing = WARPS * kDepth * kStep;
    static constexpr int kRed = 2 * WARPS * NT * 512;
};

// NT: sets of 8 tokens; 0: a single token.  G128: groups of 128.
template <bool BF16, bool W4, bool GATED, int NTOK, int WARPS, bool G128>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 8 ? 3 : 1) ffn_few_kernel(const FfnParams p, int vec_x, int vec_s, int vec_z, int tiles)
{
    using S = OutStore<BF16 ? kOutBF16 : kOutF16>;
    constexpr int NT = NTOK ? NTOK : 1;
    using C = Cfg<NT, WARPS>;
    const int tokens = NTOK ? p.tokens : 1;
    constexpr int kDepth = C::kDepth;
    constexpr int kRows = GATED ? 8 : 16;  // outputs per tile
    constexpr int kStepK = W4 ? 256 : 64;
    constexpr int XV = W4 ? 8 : 2;         // 16-byte pieces of a token per step
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * (kDepth * kStep);
    float4* const red = reinterpret_cast<float4*>(smem + C::kRing);
    uint4* const xs = reinterpret_cast<uint4*>(smem + C::kRing + C::kRed);

    pdl_launch_dependents();
    const int row_bytes = W4 ? (p.k >> 1) + (p.k & 1) : 2 * p.k;
    const int steps = (row_bytes + 127) >> 7;
    const int count = steps > warp ? (steps - warp + WARPS - 1) / WARPS : 0;  // of this warp, per tile

    // What is fetched next: step `fi` of tile `ft`.  This lane copies piece lane % 8 of rows
    // lane / 8 + 4 i, and fetches scales and zeros of rows g and g + 8: those of the step's
    // two groups, or, in shorter groups, those at 64 t and 64 t + 32 of it.
    int ft = blockIdx.x, fi = 0;
    const uint8_t* src[2];  // rows i = 0 and 2, of step fi
    const uint16_t* srow[2];
    const uint8_t* zrow[2];
    int valid = 0;
    bool full = false;  // a tile of 16 rows
    const int64_t four = p.ldw * (W4 ? 4 : 8);  // bytes from a row to the fourth after it
    const auto open = [&] {
        valid = 0;
        full = static_cast<int64_t>(ft + 1) * kRows <= p.n;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (lane >> 3) + 4 * i, o = ft * kRows + (GATED ? r & 7 : r);
            valid |= ft < tiles && o < p.n ? 1 << i : 0;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t up = GATED && h ? p.n : 0;
            const int o = ft * kRows + (lane >> 3) + (GATED ? 0 : 8 * h);
            src[h] = static_cast<const uint8_t*>(p.w) + (valid & (1 << 2 * h) ? o + up : 0) * p.ldw * (W4 ? 1 : 2) + (lane & 7) * 16 +
                     warp * 128;
            if (W4) {
                // (rows past the weights: the last one's scales, and zeros for codes)
                const int64_t row = min(ft * kRows + (GATED ? g : g + 8 * h), p.n - 1) + up;
                srow[h] = static_cast<const uint16_t*>(p.scales) + row * p.lds;
                zrow[h] = p.zeros ? p.zeros + row * p.ldz : nullptr;
            }
        }
    };
    uint32_t dst[2];  // rows i = 0, 1; rows 2 and 3 lie 1024 bytes on
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = (lane >> 3) + 4 * i;
        dst[i] = ring + r * 128 + (((lane & 7) ^ ((r & 1) << 2 | ((r >> 1) & 3))) << 4);
    }
    const auto fetch = [&](int slot, uint32_t (&sc)[2], uint32_t (&ze)[2]) {
        if (ft < tiles) {
            const int step = warp + fi * WARPS;
            if (full && (step + 1) * 128 <= row_bytes) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    cp_async16(dst[i & 1] + slot * kStep + 1024 * (i >> 1), src[i >> 1] + (i & 1 ? four : 0));
            } else {
                const int left = max(0, min(16, row_bytes - step * 128 - (lane & 7) * 16));
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    // (nothing is read where 0 bytes are copied)
                    cp_async16(dst[i & 1] + slot * kStep + 1024 * (i >> 1), src[i >> 1] + (i & 1 ? four : 0),
                               valid & (1 << i) ? left : 0);
            }
            src[0] += WARPS * 128;
            src[1] += WARPS * 128;
            if (W4) {
                const int k = step * kStepK + (G128 ? 0 : 64 * t);
                const int g0 = k >> p.group_shift, g1 = (k + (G128 ? 128 : 32)) >> p.group_shift;
                // Nothing is done here with what is loaded that would have to wait for it: a
                // pair comes in one load, and of groups of 64, both elements 64 t and 64 t + 32
                // of which are in one, the lower half alone is looked at.
                const bool single = !G128 && p.group_shift == 6;
                const bool inside = (step + 1) * kStepK <= p.k;
                // past K: the last group's, whose end may lie there
                const int last = (p.k - 1) >> p.group_shift;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (inside && !single && vec_s)
                        sc[h] = __ldg(reinterpret_cast<const uint32_t*>(srow[h] + g0));
                    else if (inside && single)
                        sc[h] = __ldg(srow[h] + g0);
                    else
                        sc[h] = __ldg(srow[h] + min(g0, last)) | static_cast<uint32_t>(__ldg(srow[h] + min(g1, last))) << 16;
                }
                if (p.zeros) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (inside && !single && vec_z)
                            ze[h] = __ldg(reinterpret_cast<const uint16_t*>(zrow[h] + g0));
                        else if (inside && single)
                            ze[h] = __ldg(zrow[h] + g0);
                        else
                            ze[h] = __ldg(zrow[h] + min(g0, last)) | static_cast<uint32_t>(__ldg(zrow[h] + min(g1, last))) << 8;
                    }
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
            ze[i][h] = 0x0808;
        }
    if (count > 0) {
        open();
        // The first steps' weights come into L2 while the preceding grids finish: a prefetch
        // reads no value, so it may run ahead of the wait for them.
        if (lane % 8 == 0) {
#pragma unroll
            for (int i = 0; i < kDepth; ++i)
                if (i < count && (warp + i * WARPS) * 128 < row_bytes)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (valid & (1 << r))
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(src[r >> 1] + (r & 1 ? four : 0) + i * (WARPS * 128)));
        }
        pdl_wait();
#pragma unroll
        for (int i = 0; i < kDepth; ++i)
            fetch(i, sc[i], ze[i]);
    } else {
        pdl_wait();
    }

    // the tokens: [step][piece][token][t], 8 elements each, paired as the codes are
    for (int e = threadIdx.x; e < steps * XV * tokens * 4; e += C::kThreads) {
        // consecutive threads on consecutive elements of a token
        const int tok = e / (steps * XV * 4), r = e - tok * (steps * XV * 4);
        const int k = r * 8, step = r / (XV * 4), in = r % (XV * 4);
        const int j = W4 && G128 ? (in >> 4) * 4 + (in & 3) : in >> 2, tt = W4 && G128 ? (in >> 2) & 3 : in & 3;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (k < p.k)
            v = load_x(static_cast<const uint16_t*>(p.x) + tok * p.ldx, k, p.k, vec_x);
        if (W4)
            v = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                           __byte_perm(v.y, v.w, 0x7632));
        xs[((step * XV + j) * tokens + tok) * 4 + tt] = v;
    }
    __syncthreads();
    const uint32_t xpiece = tokens * 64;  // bytes
    uint32_t xat[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
        // (lanes of tokens that are not there read the last one: their columns are not stored)
        xat[n] = smem_u32(xs) + min(8 * n + g, tokens - 1) * 64 + t * 16 + warp * XV * xpiece;
    const uint32_t swz = (g & 1) << 2 | ((g >> 1) & 3);  // of rows g and g + 8
    // 16-byte piece c of row g of a step
    const auto piece = [&](int c) { return ring + g * 128 + ((static_cast<uint32_t>(c) ^ swz) << 4); };
    const uint32_t half0 = piece(t), half1 = piece(4 + t);
    const uint32_t mask = G128 ? 127u : (1u << p.group_shift) - 1;

    int buf = 0, slot0 = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
        float acc[NT][4] = {};
        // one step: its codes or weights in `slot`, its scales and zeros in s and z
        const auto step = [&](int i, int slot, uint32_t (&s)[2], uint32_t (&z)[2]) {
            const uint32_t xoff = static_cast<uint32_t>(i) * (WARPS * XV) * xpiece;
            cp_async_wait<kDepth - 1>();
            __syncwarp();
            if constexpr (W4) {
                float f[2], part[NT][4];
                uint32_t zero[2], words[2][4];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (G128 && j % 4 == 0) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            f[h] = scale_of<BF16>(s[h], j >> 2);
                            zero[h] = zero_of<BF16>(z[h], j >> 2);
                            const uint4 w = lds128((j ? half1 : half0) + slot * kStep + 1024 * h);
                            words[h][0] = w.x, words[h][1] = w.y, words[h][2] = w.z, words[h][3] = w.w;
                        }
                    }
                    uint32_t a[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (!G128) {
                            const uint32_t sv = __shfl_sync(0xffffffffu, s[h], (lane & ~3) | (j >> 1));
                            const uint32_t zv = __shfl_sync(0xffffffffu, z[h], (lane & ~3) | (j >> 1));
                            const bool high = j & 1 && p.group_shift == 5;
                            f[h] = high ? scale_of<BF16>(sv, 1) : scale_of<BF16>(sv, 0);
                            zero[h] = high ? zero_of<BF16>(zv, 1) : zero_of<BF16>(zv, 0);
                            words[h][j & 3] = lds32(piece(j) + slot * kStep + 1024 * h + t * 4);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            a[h][e] = codes_at<BF16>(words[h][j & 3], e, zero[h]);
                    }
                    const bool start = ((j << 5) & mask) == 0;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 b = lds128(xat[n] + xoff + j * xpiece);
                        if (start)
                            mma0<BF16>(part[n], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
                        else
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
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t at = (j ? half1 : half0) + slot * kStep;
                    const uint4 lo = lds128(at), hi = lds128(at + 1024);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 b = lds128(xat[n] + xoff + j * xpiece);
                        mma<BF16>(acc[n], lo.x, hi.x, lo.y, hi.y, b.x, b.y);
                        mma<BF16>(acc[n], lo.z, hi.z, lo.w, hi.w, b.z, b.w);
                    }
                }
            }
            __syncwarp();
            fetch(slot, s, z);
        };
        // (the ring's slots, and with them the scales' registers, run on from tile to tile)
        int i = 0;
        while (i < count) {
            switch (slot0) {
            case 0:
                step(i, 0, sc[0], ze[0]);
                if (++i == count) {
                    slot0 = 1 % kDepth;
                    break;
                }
                [[fallthrough]];
            case 1:
                step(i, 1, sc[1], ze[1]);
                if (++i == count || kDepth == 2) {
                    slot0 = 2 % kDepth;
                    break;
                }
                [[fallthrough]];
            default:
                if constexpr (kDepth == 3) {
                    step(i, 2, sc[2], ze[2]);
                    ++i;
                    slot0 = 0;
                }
            }
        }
        // the tile's sums
        float4* const mine = red + (buf * WARPS + warp) * (NT * 32) + lane;
#pragma unroll
        for (int n = 0; n < NT; ++n)
            mine[n * 32] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
        __syncthreads();
        if (warp != tile / static_cast<int>(gridDim.x) % WARPS)
            continue;
        typename S::T* out = static_cast<typename S::T*>(p.out);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float v[4] = {};
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float4 a = red[(buf * WARPS + w) * (NT * 32) + n * 32 + lane];
                v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int tok = 8 * n + 2 * t + e;
                if (tok >= tokens)
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

template <bool BF16, bool W4, bool GATED, int NTOK, int WARPS, bool G128>
cudaError_t run(const FfnParams& p, int device, int num_sms, cudaStream_t stream)
{
    using C = Cfg<NTOK ? NTOK : 1, WARPS>;
    auto* kernel = ffn_few_kernel<BF16, W4, GATED, NTOK, WARPS, G128>;
    static SmemLimit limit;
    const cudaError_t e = limit.allow(kernel, kMaxSmem, device);
    if (e != cudaSuccess)
        return e;
    const int vec_x = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ldx % 8 == 0;
    const int vec_s = reinterpret_cast<uintptr_t>(p.scales) % 4 == 0 && p.lds % 2 == 0;  // pairs of scales
    const int vec_z = reinterpret_cast<uintptr_t>(p.zeros) % 2 == 0 && p.ldz % 2 == 0;
    const int smem = C::kRing + C::kRed + static_cast<int>(x_bytes(p));
    constexpr int per = GATED ? 8 : 16;
    const int tiles = static_cast<int>((int64_t(p.n) + per - 1) / per);
    const int resident = WARPS == 8 ? std::min(3, (kMaxSmem + 1024) / (smem + 1024)) : 1;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min(tiles, resident * num_sms)));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, vec_x, vec_s, vec_z, tiles);
}

template <bool BF16, bool W4, bool GATED, bool G128>
cudaError_t by_tokens(const FfnParams& p, int device, int num_sms, cudaStream_t stream)
{
    if (p.tokens > 8)
        return run<BF16, W4, GATED, 2, 16, G128>(p, device, num_sms, stream);
    // two CTAs of 8 warps have to fit
    if (2 * (Cfg<1, 8>::kRing + Cfg<1, 8>::kRed + x_bytes(p) + 1024) <= kMaxSmem + 1024)
        return p.tokens == 1 ? run<BF16, W4, GATED, 0, 8, G128>(p, device, num_sms, stream)
                             : run<BF16, W4, GATED, 1, 8, G128>(p, device, num_sms, stream);
    return run<BF16, W4, GATED, 1, 16, G128>(p, device, num_sms, stream);
}

template <bool BF16, bool W4, bool GATED>
cudaError_t by_group(const FfnParams& p, int device, int num_sms, cudaStream_t stream)
{
    if constexpr (W4)
        if (p.group_shift == 7)
            return by_tokens<BF16, W4, GATED, true>(p, device, num_sms, stream);
    return by_tokens<BF16, W4, GATED, false>(p, device, num_sms, stream);
}

template <bool BF16>
cudaError_t by_kind(const FfnParams& p, int device, int num_sms, cudaStream_t stream)
{
    if (!p.scales)
        return by_group<BF16, false, true>(p, device, num_sms, stream);
    return p.gated ? by_group<BF16, true, true>(p, device, num_sms, stream)
                   : by_group<BF16, true, false>(p, device, num_sms, stream);
}

}  // namespace

cudaError_t ffn_few_launch(const FfnParams& p, int device, int num_sms, cudaStream_t stream)
{
    return p.bf16 ? by_kind<true>(p, device, num_sms, stream) : by_kind<false>(p, device, num_sms, stream);
}

}  // namespace gnt
