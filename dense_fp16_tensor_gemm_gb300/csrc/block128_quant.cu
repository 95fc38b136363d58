// block128_quant.cu -- 8-bit quantisation with one scale for each block of 128.
//
//   a = max(max |x|, 2^-100) over the block,  s = a * (1/F),  q = rn8(x * (F * (1/a)))
//
// with F the largest value of the 8-bit type, each step rounded to fp32: 2^-100
// keeps the factors finite and normal for blocks of zeros or of tiny values.  Bound by
// memory (one read, one or two quarter- or half-size writes).  A CTA takes 128
// columns of R x 16 rows and holds them in registers, 8 columns x R rows a
// thread, 16-byte loads; a row's largest value is then a 16-lane shuffle, a
// column's an 8-warp exchange in shared memory, and both orders of the result
// come from one read.  The transposed codes pass through shared memory so that
// they leave as whole rows of 128 bytes.  R = 8 (a 128 x 128 tile) when a
// column or tile maximum is needed, else 2: four times the CTAs when few rows
// are quantised for the next product.
#include <cuda_fp8.h>

#include "gemm_nt.h"
#include "block128.h"

namespace gnt {

namespace {

constexpr float kFloor = 7.888609052210118e-31f;  // 2^-100

// max that keeps a NaN, as |x| of the block's elements must
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <int XT>
__device__ __forceinline__ float load1(const void* x, int64_t i)
{
    if constexpr (XT == GEMM_DTYPE_F32)
        return static_cast<const float*>(x)[i];
    else if constexpr (XT == GEMM_DTYPE_F16)
        return __half2float(static_cast<const __half*>(x)[i]);
    else
        return __bfloat162float(static_cast<const __nv_bfloat16*>(x)[i]);
}

// 8 consecutive elements from a 16-byte aligned place.
template <int XT>
__device__ __forceinline__ void load8(const void* x, int64_t i, float (&v)[8])
{
    if constexpr (XT == GEMM_DTYPE_F32) {
        const float4* g = reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
        const float4 a = __ldcs(g), b = __ldcs(g + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 w = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + i));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (XT == GEMM_DTYPE_F16) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
                v[2 * j] = f.x, v[2 * j + 1] = f.y;
            } else {
                v[2 * j] = __uint_as_float(u[j] << 16);
                v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
            }
        }
    }
}

template <bool E5M2>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d)
{
    constexpr __nv_fp8_interpretation_t kind = E5M2 ? __NV_E5M2 : __NV_E4M3;
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, kind);
    return lo | static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, kind)) << 16;
}

__device__ __forceinline__ void store_bytes(uint8_t* d, const uint32_t* w, int n)
{
    for (int i = 0; i < n; ++i)
        d[i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
}

// R: rows per thread (the CTA holds 16 R rows x 128 columns).  TILE: one scale
// for the whole 128 x 128 tile.  Q / T: which orders are written.
template <int XT, bool E5M2, int R, bool TILE, bool Q, bool T>
__global__ void __launch_bounds__(256) quantize_kernel(const QuantParams p)
{
    static_assert(R == 8 || (!TILE && !T), "column and tile maxima need all 128 rows");
    constexpr float F = E5M2 ? 57344.f : 448.f;
    constexpr float kInvF = 1.f / F;
    constexpr int kPitchT = 128 + 16;
    __shared__ __align__(16) uint8_t tq[T ? 128 * kPitchT : 16];
    __shared__ float cmax[T || TILE ? 8 : 1][128];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, warp = threadIdx.x >> 5;
    const int64_t col0 = static_cast<int64_t>(blockIdx.x) * 128;
    const int64_t col = col0 + tx * 8;
    const int ncol = col < p.cols ? static_cast<int>(min(static_cast<int64_t>(8), p.cols - col)) : 0;
    for (int64_t row0 = static_cast<int64_t>(blockIdx.y) * (16 * R); row0 < p.rows;
         row0 += static_cast<int64_t>(gridDim.y) * (16 * R)) {
        const int64_t row = row0 + ty * R;
        float v[R][8];
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] = 0.f;
            if (row + i < p.rows) {
                if (p.vec_x && ncol == 8) {
                    load8<XT>(p.x, (row + i) * p.ldx + col, v[i]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < ncol)
                            v[i][j] = load1<XT>(p.x, (row + i) * p.ldx + col + j);
                }
            }
        }
        float ra[R];  // largest of each row's 128 columns, in every lane that holds the row
        if (Q && !TILE) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float a = kFloor;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    a = max_nan(a, fabsf(v[i][j]));
                ra[i] = a;
            }
#pragma unroll
            for (int s = 1; s < 16; s *= 2)
#pragma unroll
                for (int i = 0; i < R; ++i)
                    ra[i] = max_nan(ra[i], __shfl_xor_sync(0xffffffffu, ra[i], s));
        }
        float ca[8];  // largest of each of the thread's 8 columns (TILE: all the same)
        if (T || TILE) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float a = kFloor;
#pragma unroll
                for (int i = 0; i < R; ++i)
                    a = max_nan(a, fabsf(v[i][j]));
                ca[j] = max_nan(a, __shfl_xor_sync(0xffffffffu, a, 16));
            }
            if ((threadIdx.x & 16) == 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    cmax[warp][tx * 8 + j] = ca[j];
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int w = 0; w < 8; ++w)
                    ca[j] = max_nan(ca[j], cmax[w][tx * 8 + j]);
            if (TILE) {
                float a = ca[0];
#pragma unroll
                for (int j = 1; j < 8; ++j)
                    a = max_nan(a, ca[j]);
#pragma unroll
                for (int s = 1; s < 16; s *= 2)
                    a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, s));
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    ca[j] = a;
            }
        }
        if (Q) {
            float r = TILE ? F * (1.f / ca[0]) : 0.f;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (!TILE)
                    r = F * (1.f / ra[i]);
                const uint32_t w[2] = {pack4<E5M2>(v[i][0] * r, v[i][1] * r, v[i][2] * r, v[i][3] * r),
                                       pack4<E5M2>(v[i][4] * r, v[i][5] * r, v[i][6] * r, v[i][7] * r)};
                if (row + i < p.rows && ncol > 0) {
                    uint8_t* d = p.q + (row + i) * p.ldq + col;
                    if (p.vec_q && ncol == 8)
                        *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
                    else
                        store_bytes(d, w, ncol);
                }
                if (!TILE && tx == 0 && row + i < p.rows)
                    p.sq[(row + i) * p.sq_rs + blockIdx.x * p.sq_ks] = ra[i] * kInvF;
            }
            if (TILE && threadIdx.x == 0)
                p.sq[row0 / 128 * p.sq_rs + blockIdx.x * p.sq_ks] = ca[0] * kInvF;
        }
        if (T) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float r = F * (1.f / ca[j]);
                const uint2 w = make_uint2(pack4<E5M2>(v[0][j] * r, v[1 % R][j] * r, v[2 % R][j] * r, v[3 % R][j] * r),
                                           pack4<E5M2>(v[4 % R][j] * r, v[5 % R][j] * r, v[6 % R][j] * r, v[7 % R][j] * r));
                *reinterpret_cast<uint2*>(tq + (tx * 8 + j) * kPitchT + ty * 8) = w;
                if (!TILE && ty == 0 && j < ncol)
                    p.st[(col + j) * p.st_rs + row0 / 128 * p.st_ks] = ca[j] * kInvF;
            }
            if (TILE && threadIdx.x == 0)
                p.st[blockIdx.x * p.st_rs + row0 / 128 * p.st_ks] = ca[0] * kInvF;
            __syncthreads();
            const int nrow = static_cast<int>(min(static_cast<int64_t>(128), p.rows - row0));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = (threadIdx.x >> 3) + 32 * e, r = (threadIdx.x & 7) * 16;
                if (col0 + c < p.cols && r < nrow) {
                    const uint4 w = *reinterpret_cast<const uint4*>(tq + c * kPitchT + r);
                    uint8_t* d = p.qt + (col0 + c) * p.ldqt + row0 + r;
                    if (p.vec_qt && r + 16 <= nrow) {
                        *reinterpret_cast<uint4*>(d) = w;
                    } else {
                        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
                        store_bytes(d, u, min(16, nrow - r));
                    }
                }
            }
        }
        if (T || TILE)
            __syncthreads();  // cmax and tq are rewritten by the next rows
    }
}

template <int XT, bool E5M2>
cudaError_t launch(const QuantParams& p, bool tile, cudaStream_t stream)
{
    const bool q = p.q != nullptr, t = p.qt != nullptr;
    const int rows = tile || t ? 128 : 32;
    const int64_t gy = (p.rows + rows - 1) / rows;
    const dim3 grid(static_cast<unsigned>((p.cols + 127) / 128), static_cast<unsigned>(gy < 65535 ? gy : 65535));
    if (tile) {
        if (q && t)
            quantize_kernel<XT, E5M2, 8, true, true, true><<<grid, 256, 0, stream>>>(p);
        else if (q)
            quantize_kernel<XT, E5M2, 8, true, true, false><<<grid, 256, 0, stream>>>(p);
        else
            quantize_kernel<XT, E5M2, 8, true, false, true><<<grid, 256, 0, stream>>>(p);
    } else {
        if (q && t)
            quantize_kernel<XT, E5M2, 8, false, true, true><<<grid, 256, 0, stream>>>(p);
        else if (q)
            quantize_kernel<XT, E5M2, 2, false, true, false><<<grid, 256, 0, stream>>>(p);
        else
            quantize_kernel<XT, E5M2, 8, false, false, true><<<grid, 256, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t block128_quantize_launch(const QuantParams& p, bool tile, cudaStream_t stream)
{
    switch (p.x_type) {
    case GEMM_DTYPE_F32:
        return p.e5m2 ? launch<GEMM_DTYPE_F32, true>(p, tile, stream) : launch<GEMM_DTYPE_F32, false>(p, tile, stream);
    case GEMM_DTYPE_F16:
        return p.e5m2 ? launch<GEMM_DTYPE_F16, true>(p, tile, stream) : launch<GEMM_DTYPE_F16, false>(p, tile, stream);
    case GEMM_DTYPE_BF16:
        return p.e5m2 ? launch<GEMM_DTYPE_BF16, true>(p, tile, stream)
                      : launch<GEMM_DTYPE_BF16, false>(p, tile, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace gnt
