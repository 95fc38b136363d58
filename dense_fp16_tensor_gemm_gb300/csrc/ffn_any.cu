// ffn_any.cu -- gated products and products with 4-bit weights on the warp MMA,
// any layout.
//
//   Out[t][j] = sum_k x[t][k] w[j][k], or act(g) u of the rows j and n + j of w
//
// The form for operands the tensor maps cannot describe (bases or pitches off
// the 16-byte grid).  A CTA of 4 warps owns 64 tokens by 64 rows of the weights,
// each warp 32 x 32; of a gated product a warp's 32 rows are 16 of the gate and
// the same 16 of the up projection, so that a thread holds g and u of its
// outputs.  K is staged 64 at a time as 16-bit values, 4-bit weights as their
// whole numbers code - zero (exact), whose sums over 32 elements (no group is
// shorter) are scaled in fp32.  Rows are padded to 144 bytes (9 x 16), so
// the 8 rows an ldmatrix reads fall on different banks.  Bound by its scalar loads (2048 x
// 4097 x 8192 gated 4.2 ms, 65 TFLOP/s; copied onto the grid first, 0.26).
#include <algorithm>

#include "ffn.h"
#include "ptx.cuh"

namespace gnt {

namespace {

constexpr int kT = 64, kKB = 64, kPitch = kKB + 8, kThreads = 128;

template <bool BF16>
__device__ __forceinline__ uint16_t bits_of(float v)
{
    return BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}
template <bool BF16>
__device__ __forceinline__ float value_of(uint16_t v)
{
    return BF16 ? __bfloat162float(__ushort_as_bfloat16(v)) : __half2float(__ushort_as_half(v));
}

// Row of the weights that row r of a staged tile holds.
__device__ __forceinline__ int64_t weight_row(const FfnParams& p, int j0, int r, bool& inside)
{
    if (!p.gated) {
        inside = j0 + r < p.n;
        return j0 + r;
    }
    const int j = j0 + (r >> 5) * 16 + (r & 15);
    inside = j < p.n;
    return j + (r & 16 ? static_cast<int64_t>(p.n) : 0);
}

template <bool BF16, bool W4>
__global__ void __launch_bounds__(kThreads) ffn_any_kernel(const FfnParams p, int tiles_t, int64_t tiles)
{
    using S = OutStore<BF16 ? kOutBF16 : kOutF16>;
    __shared__ __align__(16) uint16_t xs[kT * kPitch];
    __shared__ __align__(16) uint16_t ws[kT * kPitch];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wt = (warp >> 1) * 32, wc = (warp & 1) * 32;  // the warp's 32 x 32 corner of the tile
    const uint16_t* x = static_cast<const uint16_t*>(p.x);
    const int per = p.gated ? kT / 2 : kT;  // columns of Out per tile
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int t0 = static_cast<int>(t % tiles_t) * kT, j0 = static_cast<int>(t / tiles_t) * per;
        float acc[2][4][4] = {};
        for (int k0 = 0; k0 < p.k; k0 += kKB) {
            __syncthreads();
            // every load of the block is in flight before the first is stored
            const int c = threadIdx.x % kKB, r0 = threadIdx.x / kKB;  // 16-bit values: a column, every other row
            uint16_t xv[kT / 2], wv[kT / 2];
            const bool kin = k0 + c < p.k;
#pragma unroll
            for (int i = 0; i < kT / 2; ++i) {
                const int r = r0 + 2 * i;
                xv[i] = kin && t0 + r < p.tokens ? __ldg(x + (t0 + r) * p.ldx + k0 + c) : uint16_t(0);
            }
            if (W4) {
                // a byte is two neighbours of K: a column of bytes, every fourth row
                const int cb = threadIdx.x % (kKB / 2), rb = threadIdx.x / (kKB / 2), k = k0 + 2 * cb;
                uint8_t zv[kT / 4];
#pragma unroll
                for (int i = 0; i < kT / 4; ++i) {
                    bool inside;
                    const int64_t row = weight_row(p, j0, rb + 4 * i, inside);
                    const bool in = inside && k < p.k;
                    wv[i] = in ? __ldg(static_cast<const uint8_t*>(p.w) + row * p.ldw + (k >> 1)) : 0;
                    zv[i] = in && p.zeros ? __ldg(p.zeros + row * p.ldz + (k >> p.group_shift)) : 8;
                }
#pragma unroll
                for (int i = 0; i < kT / 4; ++i) {
                    // (x is zero past K: what stands there, and an odd K's last high half, counts for nothing)
                    uint16_t* dst = ws + (rb + 4 * i) * kPitch + 2 * cb;
                    dst[0] = bits_of<BF16>(static_cast<float>((wv[i] & 15) - zv[i]));
                    dst[1] = bits_of<BF16>(static_cast<float>((wv[i] >> 4) - zv[i]));
                }
            } else {
#pragma unroll
                for (int i = 0; i < kT / 2; ++i) {
                    bool inside;
                    const int64_t row = weight_row(p, j0, r0 + 2 * i, inside);
                    wv[i] = kin && inside ? __ldg(static_cast<const uint16_t*>(p.w) + row * p.ldw + k0 + c) : uint16_t(0);
                }
#pragma unroll
                for (int i = 0; i < kT / 2; ++i)
                    ws[(r0 + 2 * i) * kPitch + c] = wv[i];
            }
#pragma unroll
            for (int i = 0; i < kT / 2; ++i)
                xs[(r0 + 2 * i) * kPitch + c] = xv[i];
            __syncthreads();
#pragma unroll
            for (int kh = 0; kh < kKB; kh += 32) {
                if (k0 + kh >= p.k)
                    break;
                float part[2][4][4] = {};
#pragma unroll
                for (int k = kh; k < kh + 32; k += 16) {
                    uint32_t a[2][4], b[2][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        ldmatrix_x4(smem_u32(xs + (wt + 16 * i + (lane & 15)) * kPitch + k + (lane >> 4) * 8), a[i][0],
                                    a[i][1], a[i][2], a[i][3]);
#pragma unroll
                    for (int j = 0; j < 2; ++j)  // words 0, 2 and 1, 3 are the two n8 tiles of 16 rows
                        ldmatrix_x4(smem_u32(ws + (wc + 16 * j + (lane & 15)) * kPitch + k + (lane >> 4) * 8), b[j][0],
                                    b[j][1], b[j][2], b[j][3]);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float(&d)[4] = W4 ? part[i][j] : acc[i][j];
                            if (BF16)
                                mma_m16n8k16_bf16(d, a[i], b[j >> 1][j & 1], b[j >> 1][(j & 1) + 2], d);
                            else
                                mma_m16n8k16(d, a[i], b[j >> 1][j & 1], b[j >> 1][(j & 1) + 2], d);
                        }
                }
                if (W4) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            bool inside;
                            const int64_t row = weight_row(p, j0, wc + 8 * j + 2 * (lane & 3) + e, inside);
                            const float s = !inside ? 0.f
                                                    : value_of<BF16>(__ldg(static_cast<const uint16_t*>(p.scales) +
                                                                           row * p.lds + ((k0 + kh) >> p.group_shift)));
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                acc[i][j][e] = fmaf(part[i][j][e], s, acc[i][j][e]);
                                acc[i][j][e + 2] = fmaf(part[i][j][e + 2], s, acc[i][j][e + 2]);
                            }
                        }
                }
            }
        }
        typename S::T* out = static_cast<typename S::T*>(p.out);
        typename S::T* gu = static_cast<typename S::T*>(p.gu);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int64_t tok = t0 + wt + 16 * i + (lane >> 2) + 8 * (e >> 1);
                    if (tok >= p.tokens)
                        continue;
                    if (!p.gated) {
                        const int col = j0 + wc + 8 * j + 2 * (lane & 3) + (e & 1);
                        if (col < p.n)
                            S::st1(out + tok * p.ldo + col, acc[i][j][e]);
                    } else if (j < 2) {
                        const int col = j0 + wc / 2 + 8 * j + 2 * (lane & 3) + (e & 1);
                        if (col < p.n) {
                            const float g = acc[i][j][e], u = acc[i][j + 2][e];
                            S::st1(out + tok * p.ldo + col, act_value(g, p.act) * u);
                            if (gu) {
                                S::st1(gu + tok * p.ldgu + col, g);
                                S::st1(gu + tok * p.ldgu + p.n + col, u);
                            }
                        }
                    }
                }
    }
}

}  // namespace

cudaError_t ffn_any_launch(const FfnParams& p, int num_sms, cudaStream_t stream)
{
    const int per = p.gated ? kT / 2 : kT;
    const int tiles_t = static_cast<int>((int64_t(p.tokens) + kT - 1) / kT);
    const int64_t tiles = tiles_t * ((int64_t(p.n) + per - 1) / per);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(tiles, static_cast<int64_t>(num_sms) * 8));
    if (p.scales) {
        if (p.bf16)
            ffn_any_kernel<true, true><<<grid, kThreads, 0, stream>>>(p, tiles_t, tiles);
        else
            ffn_any_kernel<false, true><<<grid, kThreads, 0, stream>>>(p, tiles_t, tiles);
    } else if (p.bf16) {
        ffn_any_kernel<true, false><<<grid, kThreads, 0, stream>>>(p, tiles_t, tiles);
    } else {
        ffn_any_kernel<false, false><<<grid, kThreads, 0, stream>>>(p, tiles_t, tiles);
    }
    return cudaGetLastError();
}

}  // namespace gnt
