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
//
// 16-bit inputs stay packed, two to a register, and their maxima are taken on
// pairs (exact: a maximum rounds nothing); the registers saved make room for
// half as many CTAs again, which is what keeps enough bytes in flight.  A block's factor
// is computed by one lane and passed on: an fp32 reciprocal costs as much as
// quantising 8 elements.
//
// Measured, bf16: 8192 x 8192 both orders 58 us (4.7 TB/s; 150 with the inputs
// widened to fp32 in registers, 72 with a padded transposed tile, whose stores met
// 16 to a bank), rows only 42 us, 64 x 8192 rows only 1.7 us.  A third of the SM's
// warps fit (80 registers), 56 % of the issue slots are used: latency is what is left.
#include <cuda_fp8.h>

#include "gemm_nt.h"
#include "block128.h"
#include "ptx.cuh"

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

// max of two pairs of 16-bit floats, keeping NaN; the arguments are magnitudes.
template <int XT>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
{
    uint32_t r;
    if constexpr (XT == GEMM_DTYPE_F16)
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <int XT>
__device__ __forceinline__ float2 widen(uint32_t w)
{
    if constexpr (XT == GEMM_DTYPE_F16)
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// A thread's R rows x 8 columns: fp32 values as they are, 16-bit ones packed.
template <int XT, int R>
struct Tile {
    static constexpr bool WIDE = XT == GEMM_DTYPE_F32;
    static constexpr int W = WIDE ? 8 : 4;  // words of a row
    uint32_t v[R][W];

    __device__ __forceinline__ void load(const QuantParams& p, int64_t row, int64_t col, int ncol)
    {
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j)
                v[i][j] = 0;
            if (row + i < p.rows) {
                const int64_t at = (row + i) * p.ldx + col;
                if (p.vec_x && ncol == 8) {
                    const uint4* g = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.x) + at * (WIDE ? 4 : 2));
#pragma unroll
                    for (int j = 0; j < W / 4; ++j) {
                        const uint4 w = __ldcs(g + j);
                        v[i][4 * j] = w.x, v[i][4 * j + 1] = w.y, v[i][4 * j + 2] = w.z, v[i][4 * j + 3] = w.w;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < ncol) {
                            if constexpr (WIDE)
                                v[i][j] = static_cast<const uint32_t*>(p.x)[at + j];
                            else
                                v[i][j / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p.x)[at + j]) << (16 * (j & 1));
                        }
                }
            }
        }
    }

    __device__ __forceinline__ float get(int i, int j) const
    {
        if constexpr (WIDE) {
            return __uint_as_float(v[i][j]);
        } else {
            const float2 f = widen<XT>(v[i][j / 2]);
            return j & 1 ? f.y : f.x;
        }
    }

    // Largest magnitude of each row over the 16 lanes that hold it.
    __device__ __forceinline__ void row_max(float (&a)[R]) const
    {
        if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                a[i] = 0.f;
#pragma unroll
                for (int j = 0; j < W; ++j)
                    a[i] = max_nan(a[i], fabsf(__uint_as_float(v[i][j])));
#pragma unroll
                for (int s = 1; s < 16; s *= 2)
                    a[i] = max_nan(a[i], __shfl_xor_sync(0xffffffffu, a[i], s));
            }
        } else {
            constexpr uint32_t M = 0x7fff7fffu;
#pragma unroll
            for (int i = 0; i < R; i += 2) {  // two rows' maxima in one word
                const uint32_t m0 = max2<XT>(max2<XT>(v[i][0] & M, v[i][1] & M), max2<XT>(v[i][2] & M, v[i][3] & M));
                const uint32_t m1 =
                    max2<XT>(max2<XT>(v[i + 1][0] & M, v[i + 1][1] & M), max2<XT>(v[i + 1][2] & M, v[i + 1][3] & M));
                uint32_t m = max2<XT>(__byte_perm(m0, m1, 0x5410), __byte_perm(m0, m1, 0x7632));
#pragma unroll
                for (int s = 1; s < 16; s *= 2)
                    m = max2<XT>(m, __shfl_xor_sync(0xffffffffu, m, s));
                const float2 f = widen<XT>(m);
                a[i] = f.x;
                a[i + 1] = f.y;
            }
        }
    }

    // Largest magnitude of each column over the warp's rows, as stored: a word a
    // column (fp32) or two columns.
    __device__ __forceinline__ void col_max(uint32_t (&a)[W]) const
    {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            if constexpr (WIDE) {
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < R; ++i)
                    m = max_nan(m, fabsf(__uint_as_float(v[i][j])));
                a[j] = __float_as_uint(max_nan(m, __shfl_xor_sync(0xffffffffu, m, 16)));
            } else {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < R; ++i)
                    m = max2<XT>(m, v[i][j] & 0x7fff7fffu);
                a[j] = max2<XT>(m, __shfl_xor_sync(0xffffffffu, m, 16));
            }
        }
    }
};

__host__ __device__ constexpr int ctas_per_sm(int xt, int r) { return xt == GEMM_DTYPE_F32 ? 2 : (r == 8 ? 3 : 4); }

// Brings the tile that a CTA will take when as many as run at once have ended into
// L2, a row a thread.  For fp32 inputs, whose registers leave two CTAs an SM: 8192 x
// 8192 both orders 73 us (80), in 128 x 128 blocks 63 (71).  With 16-bit inputs it
// gave 2 % at most, and rows alone took 47 us for 42.
template <int ROWS>
__device__ __forceinline__ void prefetch(const QuantParams& p, int64_t row0)
{
    const unsigned bx = blockIdx.x + p.ahead;
    const int64_t row = row0 + static_cast<int64_t>(bx / gridDim.x) * ROWS + threadIdx.x;
    const int64_t col = static_cast<int64_t>(bx % gridDim.x) * 128;
    if (threadIdx.x < ROWS && p.vec_x && row < p.rows && col + 128 <= p.cols)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const float*>(p.x) + row * p.ldx + col),
                     "n"(128 * 4)
                     : "memory");
}

// R: rows per thread (the CTA holds 16 R rows x 128 columns).  TILE: one scale
// for the whole 128 x 128 tile.  Q / T: which orders are written.
template <int XT, bool E5M2, int R, bool TILE, bool Q, bool T>
__global__ void __launch_bounds__(256, ctas_per_sm(XT, R)) quantize_kernel(const QuantParams p)
{
    static_assert(R == 8 || (!TILE && !T), "column and tile maxima need all 128 rows");
    constexpr float F = E5M2 ? 57344.f : 448.f;
    constexpr float kInvF = 1.f / F;
    using D = Tile<XT, R>;
    constexpr int CW = 16 * D::W;  // words of a warp's column maxima
    __shared__ __align__(16) uint8_t tq[T ? 128 * 128 : 16];  // column c's 128 codes, swizzled (below)
    __shared__ __align__(16) uint32_t cmax[T || TILE ? 8 : 1][T || TILE ? CW : 1];
    __shared__ __align__(16) float cfac[T || TILE ? 128 : 4];  // columns' factors (TILE: their maxima)
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t col0 = static_cast<int64_t>(blockIdx.x) * 128;
    const int64_t col = col0 + tx * 8;
    const int ncol = col < p.cols ? static_cast<int>(min(static_cast<int64_t>(8), p.cols - col)) : 0;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t row0 = static_cast<int64_t>(blockIdx.y) * (16 * R); row0 < p.rows;
         row0 += static_cast<int64_t>(gridDim.y) * (16 * R)) {
        const int64_t row = row0 + ty * R;
        D d;
        d.load(p, row, col, ncol);
        if constexpr (D::WIDE)
            prefetch<16 * R>(p, row0);
        if (T || TILE) {
            uint32_t m[D::W];
            d.col_max(m);
            if (lane < 16) {
#pragma unroll
                for (int j = 0; j < D::W; j += 4)
                    *reinterpret_cast<uint4*>(&cmax[warp][tx * D::W + j]) = make_uint4(m[j], m[j + 1], m[j + 2], m[j + 3]);
            }
            __syncthreads();
            if (threadIdx.x < CW) {  // a word's columns: their maxima, factors and scales
                uint32_t w = cmax[0][threadIdx.x];
#pragma unroll
                for (int k = 1; k < 8; ++k) {
                    const uint32_t u = cmax[k][threadIdx.x];
                    if constexpr (D::WIDE)
                        w = __float_as_uint(max_nan(__uint_as_float(w), __uint_as_float(u)));
                    else
                        w = max2<XT>(w, u);
                }
                float a[2];
                if constexpr (D::WIDE) {
                    a[0] = __uint_as_float(w);
                } else {
                    const float2 f = widen<XT>(w);
                    a[0] = f.x, a[1] = f.y;
                }
#pragma unroll
                for (int e = 0; e < 128 / CW; ++e) {
                    const int c = threadIdx.x * (128 / CW) + e;
                    const float m1 = max_nan(a[e], kFloor);
                    cfac[c] = TILE ? m1 : F * (1.f / m1);
                    if (T && !TILE && col0 + c < p.cols)
                        p.st[(col0 + c) * p.st_rs + row0 / 128 * p.st_ks] = m1 * kInvF;
                }
            }
            __syncthreads();
        }
        float tile_factor = 0.f;
        if (TILE) {
            float a = max_nan(max_nan(cfac[lane], cfac[lane + 32]), max_nan(cfac[lane + 64], cfac[lane + 96]));
#pragma unroll
            for (int s = 1; s < 32; s *= 2)
                a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, s));
            tile_factor = F * (1.f / a);
            if (threadIdx.x == 0) {
                if (Q)
                    p.sq[row0 / 128 * p.sq_rs + blockIdx.x * p.sq_ks] = a * kInvF;
                if (T)
                    p.st[blockIdx.x * p.st_rs + row0 / 128 * p.st_ks] = a * kInvF;
            }
        }
        if (Q) {
            float mine = tile_factor;
            if (!TILE) {
                float a[R];
                d.row_max(a);
                float m = a[0];  // lane tx looks after row tx % R
#pragma unroll
                for (int i = 1; i < R; ++i)
                    m = tx % R == i ? a[i] : m;
                m = max_nan(m, kFloor);
                mine = F * (1.f / m);
                if (tx < R && row + tx < p.rows)
                    p.sq[(row + tx) * p.sq_rs + blockIdx.x * p.sq_ks] = m * kInvF;
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float r = TILE ? tile_factor : __shfl_sync(0xffffffffu, mine, (lane & 16) + i);
                const uint32_t w[2] = {
                    pack4<E5M2>(d.get(i, 0) * r, d.get(i, 1) * r, d.get(i, 2) * r, d.get(i, 3) * r),
                    pack4<E5M2>(d.get(i, 4) * r, d.get(i, 5) * r, d.get(i, 6) * r, d.get(i, 7) * r)};
                if (row + i < p.rows && ncol > 0) {
                    uint8_t* o = p.q + (row + i) * p.ldq + col;
                    if (p.vec_q && ncol == 8)
                        *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
                    else
                        store_bytes(o, w, ncol);
                }
            }
        }
        if (T) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float r = TILE ? tile_factor : cfac[tx * 8 + j];
                const uint2 w = make_uint2(
                    pack4<E5M2>(d.get(0, j) * r, d.get(1 % R, j) * r, d.get(2 % R, j) * r, d.get(3 % R, j) * r),
                    pack4<E5M2>(d.get(4 % R, j) * r, d.get(5 % R, j) * r, d.get(6 % R, j) * r, d.get(7 % R, j) * r));
                // 16-byte chunk ty / 2 of column 8 tx + j at chunk ^ (tx % 8), its halves
                // exchanged for tx >= 8: the 16 lanes of a row of threads fill 128 bytes
                *reinterpret_cast<uint2*>(tq + (tx * 8 + j) * 128 + (((ty >> 1) ^ (tx & 7)) << 4) +
                                          (((ty ^ (tx >> 3)) & 1) << 3)) = w;
            }
            __syncthreads();
            const int nrow = static_cast<int>(min(static_cast<int64_t>(128), p.rows - row0));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = (threadIdx.x >> 3) + 32 * e, r = (threadIdx.x & 7) * 16;
                if (col0 + c < p.cols && r < nrow) {
                    uint4 w = *reinterpret_cast<const uint4*>(tq + c * 128 + (r ^ ((c >> 3 & 7) << 4)));
                    if (c >= 64)
                        w = make_uint4(w.z, w.w, w.x, w.y);
                    uint8_t* o = p.qt + (col0 + c) * p.ldqt + row0 + r;
                    if (p.vec_qt && r + 16 <= nrow) {
                        *reinterpret_cast<uint4*>(o) = w;
                    } else {
                        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
                        store_bytes(o, u, min(16, nrow - r));
                    }
                }
            }
        }
        if (T || TILE)
            __syncthreads();  // cmax, cfac and tq are rewritten by the next rows
    }
}

template <auto KERNEL>
cudaError_t start(const QuantParams& p, dim3 grid, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, KERNEL, p);
}

template <int XT, bool E5M2>
cudaError_t launch(const QuantParams& prm, bool tile, cudaStream_t stream)
{
    QuantParams p = prm;
    const bool q = p.q != nullptr, t = p.qt != nullptr;
    p.ahead = static_cast<unsigned>(p.num_sms * ctas_per_sm(XT, tile || t ? 8 : 2));
    const int rows = tile || t ? 128 : 32;
    const int64_t gy = (p.rows + rows - 1) / rows;
    const dim3 grid(static_cast<unsigned>((p.cols + 127) / 128), static_cast<unsigned>(gy < 65535 ? gy : 65535));
    if (tile) {
        if (q && t)
            return start<quantize_kernel<XT, E5M2, 8, true, true, true>>(p, grid, stream);
        return q ? start<quantize_kernel<XT, E5M2, 8, true, true, false>>(p, grid, stream)
                 : start<quantize_kernel<XT, E5M2, 8, true, false, true>>(p, grid, stream);
    }
    if (q && t)
        return start<quantize_kernel<XT, E5M2, 8, false, true, true>>(p, grid, stream);
    return q ? start<quantize_kernel<XT, E5M2, 2, false, true, false>>(p, grid, stream)
             : start<quantize_kernel<XT, E5M2, 8, false, false, true>>(p, grid, stream);
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
