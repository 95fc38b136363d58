// block128_any.cu -- block-scaled 8-bit product on the warp MMA, any layout.
//
//   Out[i,j] = sum_c sa[i,c] sb[j,c] sum_{k in block c} A[i,k] B[j,k]
//
// The form for operands the tensor maps cannot describe (bases or pitches off
// the 16-byte grid).  A CTA of 4 warps owns a 64 x 64 tile of Out, each warp 32
// x 32; a K block of 128 is staged as fp16 (every E4M3 and E5M2 value is an fp16
// value), eight m16n8k16 steps give its fp32 partial sums, and the tile's
// accumulators take them times the two scales.  Bound by the warp MMA and by the
// staging between barriers (8192 x 8192 x 8192: 10.1 ms, 109 TFLOP/s).  Rows are padded to 272 bytes
// (17 x 16), so the 8 rows an ldmatrix reads fall on different banks.
#include <cuda_fp8.h>

#include "block128.h"
#include "ptx.cuh"

namespace gnt {

namespace {

constexpr int kT = 64, kKB = 128, kPitch = kKB + 8, kThreads = 128;

// 64 rows x 128 bytes of one operand into fp16, zeros outside rows and K.
template <bool E5M2>
__device__ __forceinline__ void stage_block(uint16_t* dst, const uint8_t* src, int64_t ld, int row0, int nrows, int k0,
                                            int K, bool vec)
{
    constexpr __nv_fp8_interpretation_t kind = E5M2 ? __NV_E5M2 : __NV_E4M3;
    if (vec) {  // 16-byte aligned rows
#pragma unroll
        for (int i = 0; i < kT * 8 / kThreads; ++i) {
            const int e = threadIdx.x + i * kThreads, r = e >> 3, c = (e & 7) * 16;
            uint32_t w[4] = {0, 0, 0, 0};
            if (row0 + r < nrows && k0 + c < K) {
                const uint8_t* g = src + static_cast<int64_t>(row0 + r) * ld + k0 + c;
                if (K - (k0 + c) >= 16) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(g));
                    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                } else {
                    for (int b = 0; b < K - (k0 + c); ++b)
                        w[b >> 2] |= static_cast<uint32_t>(g[b]) << (8 * (b & 3));
                }
            }
            uint32_t h[8];
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                const __half2_raw p =
                    __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[b >> 1] >> (16 * (b & 1))), kind);
                h[b] = p.x | static_cast<uint32_t>(p.y) << 16;
            }
            uint4* d = reinterpret_cast<uint4*>(dst + r * kPitch + c);
            d[0] = make_uint4(h[0], h[1], h[2], h[3]);
            d[1] = make_uint4(h[4], h[5], h[6], h[7]);
        }
    } else {
#pragma unroll 4
        for (int i = 0; i < kT * kKB / kThreads; ++i) {
            const int r = i, c = threadIdx.x;  // one row per step, consecutive threads on consecutive bytes
            uint16_t v = 0;
            if (row0 + r < nrows && k0 + c < K)
                v = __nv_cvt_fp8_to_halfraw(src[static_cast<int64_t>(row0 + r) * ld + k0 + c], kind).x;
            dst[r * kPitch + c] = v;
        }
    }
}

template <bool E5M2, int OT>
__global__ void __launch_bounds__(kThreads) block128_any_kernel(const BlkParams p, int vec_a, int vec_b)
{
    using S = OutStore<OT>;
    __shared__ __align__(16) uint16_t as[kT * kPitch];
    __shared__ __align__(16) uint16_t bs[kT * kPitch];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wr = (warp >> 1) * 32, wc = (warp & 1) * 32;  // the warp's 32 x 32 corner of the tile
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    for (int64_t t = blockIdx.x; t < tiles * p.batch; t += gridDim.x) {
        const int b = static_cast<int>(t / tiles);
        const int m0 = static_cast<int>(t % tiles % p.tiles_m) * kT, n0 = static_cast<int>(t % tiles / p.tiles_m) * kT;
        const uint8_t* A = static_cast<const uint8_t*>(p.A) + b * p.stride_a;
        const uint8_t* B = static_cast<const uint8_t*>(p.B) + b * p.stride_b;
        float acc[2][4][4] = {};
        for (int kb = 0; kb < p.num_kb; ++kb) {
            __syncthreads();
            stage_block<E5M2>(as, A, p.lda, m0, p.M, kb * kKB, p.K, vec_a != 0);
            stage_block<E5M2>(bs, B, p.ldb, n0, p.N, kb * kKB, p.K, vec_b != 0);
            __syncthreads();
            float part[2][4][4] = {};
#pragma unroll
            for (int k = 0; k < kKB; k += 16) {
                uint32_t a[2][4], w[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    ldmatrix_x4(smem_u32(as + (wr + 16 * i + (lane & 15)) * kPitch + k + (lane >> 4) * 8), a[i][0],
                                a[i][1], a[i][2], a[i][3]);
#pragma unroll
                for (int j = 0; j < 2; ++j)  // rows 16j..16j+15 of B: words 0, 2 and 1, 3 are its two n8 tiles
                    ldmatrix_x4(smem_u32(bs + (wc + 16 * j + (lane & 15)) * kPitch + k + (lane >> 4) * 8), w[j][0],
                                w[j][1], w[j][2], w[j][3]);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_m16n8k16(part[i][j], a[i], w[j >> 1][j & 1], w[j >> 1][(j & 1) + 2], part[i][j]);
            }
            // rows and columns outside Out hold zeros and are not stored: their scales are read as the last ones
            float fa[4], fb[8];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                fa[r] = scale_at(p.sa, b, min(m0 + wr + 8 * r + (lane >> 2), p.M - 1), kb);
#pragma unroll
            for (int c = 0; c < 8; ++c)
                fb[c] = scale_at(p.sb, b, min(n0 + wc + 8 * (c >> 1) + 2 * (lane & 3) + (c & 1), p.N - 1), kb);
            const auto add = [&](auto factors) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const Factors f = factors(fa[2 * i + (e >> 1)], fb[2 * j + (e & 1)]);
                            acc[i][j][e] = fmaf(part[i][j][e] * f.first, f.second, acc[i][j][e]);
                        }
            };
            const uint32_t from = plain_from(E5M2);
            if (__all_sync(0xffffffffu, plain_scale(fa[0], from) && plain_scale(fa[1], from) && plain_scale(fa[2], from) &&
                                            plain_scale(fa[3], from)))
                add([](float s, float w) { return Factors{s, w}; });
            else
                add([](float s, float w) { return scale_factors(s, w); });
        }
        typename S::T* out = static_cast<typename S::T*>(p.out) + b * p.stride_o;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = m0 + wr + 16 * i + 8 * (e >> 1) + (lane >> 2);
                    const int col = n0 + wc + 8 * j + 2 * (lane & 3) + (e & 1);
                    if (row < p.M && col < p.N)
                        S::st1(out + static_cast<int64_t>(row) * p.ldo + col, acc[i][j][e]);
                }
    }
}

template <bool E5M2>
void launch(const BlkParams& p, int grid, int va, int vb, cudaStream_t stream)
{
    if (p.out_type == kOutF16)
        block128_any_kernel<E5M2, kOutF16><<<grid, kThreads, 0, stream>>>(p, va, vb);
    else if (p.out_type == kOutBF16)
        block128_any_kernel<E5M2, kOutBF16><<<grid, kThreads, 0, stream>>>(p, va, vb);
    else
        block128_any_kernel<E5M2, kOutF32><<<grid, kThreads, 0, stream>>>(p, va, vb);
}

bool rows_on_16(const void* base, int64_t ld, int64_t stride, int batch)
{
    return reinterpret_cast<uintptr_t>(base) % 16 == 0 && ld % 16 == 0 && (batch == 1 || stride % 16 == 0);
}

}  // namespace

cudaError_t block128_any_launch(const BlkParams& prm, cudaStream_t stream)
{
    BlkParams p = prm;
    p.tiles_m = (p.M - 1) / kT + 1;
    p.tiles_n = (p.N - 1) / kT + 1;
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n * p.batch;
    const int grid = static_cast<int>(tiles < (1 << 20) ? tiles : (1 << 20));
    const int va = rows_on_16(p.A, p.lda, p.stride_a, p.batch), vb = rows_on_16(p.B, p.ldb, p.stride_b, p.batch);
    if (p.e5m2)
        launch<true>(p, grid, va, vb, stream);
    else
        launch<false>(p, grid, va, vb, stream);
    return cudaGetLastError();
}

}  // namespace gnt
