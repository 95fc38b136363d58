// w4_quant.cu -- 4-bit codes of a weight matrix, with one 16-bit scale (and
// optionally a zero point) for each group of 32, 64 or 128 elements of a row.
//
//   symmetric   a = max |w|, s = round16(a * (1/7)), code = clamp(rint(w * (1/s)), -8, 7) + 8
//   with zeros  lo = min(w, 0), hi = max(w, 0), s = round16((hi - lo) * (1/15)),
//               z = clamp(rint(-lo * (1/s)), 0, 15), code = clamp(rint(w * (1/s)) + z, 0, 15)
//
// in fp32, each step rounded, with the rounded s, so that codes and scales
// together stand for the weights as nearly as they can.  A thread holds 32
// consecutive elements (four 16-byte loads of 16-bit weights, one 16-byte store of
// codes); a group's 1, 2 or 4 threads share its extremes by shuffles.  Bound by
// memory, one read of the weights, as long as the instructions stay below it: w * (1/s)
// is rounded to a whole number by adding 1.5 * 2^23, whose low bits then hold it
// (|w / s| stays below 32), and a saturating pack clamps and joins two codes.  8192 x 8192
// bf16 in 28.8 us, 5.9 TB/s (16 elements a thread 33.6: the scale's arithmetic is per thread;
// 8 elements, comparisons and shifts in the place of the pack 80).
#include <algorithm>
#include <cfloat>

#include "ffn.h"
#include "gemm_nt.h"

namespace gnt {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 32;  // elements per thread

// Elements of a 32-bit word of weights.  WT: 0 fp16, 1 bf16, 2 fp32.
template <int WT>
__device__ __forceinline__ void unpack(uint32_t w, float* v)
{
    if constexpr (WT == 2) {
        v[0] = __uint_as_float(w);
    } else if constexpr (WT == 1) {
        v[0] = __uint_as_float(w << 16);
        v[1] = __uint_as_float(w & 0xffff0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        v[0] = f.x;
        v[1] = f.y;
    }
}

// U: bytes on whose boundaries all rows of weights start, and of a load: 16, 8, of 16-bit
// weights 4, or 0 for single elements.  A thread's elements lie apart from its neighbours', so
// every load of a warp touches 32 lines, and their number is the time: 8192 x 8192 bf16 28.5 us,
// x 8188 47.8, x 8190 76, x 8191 119; fp32 10227 x 1250 26.8, x 1251 43.
template <int WT, int U>
__device__ __forceinline__ void load_piece(const Quant4Params& p, int64_t row, int64_t col, float (&v)[kPer])
{
    constexpr int kWords = WT == 2 ? kPer : kPer / 2, kOf = WT == 2 ? 1 : 2;
    const uint8_t* at = static_cast<const uint8_t*>(p.w) + (row * p.ldw + col) * (WT == 2 ? 4 : 2);
    if (U > 0 && col + kPer <= p.cols) {
        uint32_t w[kWords];
        if constexpr (U == 16) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 a = __ldcs(reinterpret_cast<const uint4*>(at) + i);
                w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
            }
        } else if constexpr (U == 8) {
#pragma unroll
            for (int i = 0; i < kWords / 2; ++i) {
                const uint2 a = __ldg(reinterpret_cast<const uint2*>(at) + i);
                w[2 * i] = a.x, w[2 * i + 1] = a.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[i] = __ldg(reinterpret_cast<const uint32_t*>(at) + i);
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            unpack<WT>(w[i], v + kOf * i);
        return;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        v[i] = 0.f;
        if (col + i < p.cols) {
            if constexpr (WT == 2)
                v[i] = reinterpret_cast<const float*>(at)[i];
            else if constexpr (WT == 1)
                v[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(at)[i]);
            else
                v[i] = __half2float(reinterpret_cast<const __half*>(at)[i]);
        }
    }
}

// max, a NaN if either is one
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// {hi, lo} as two 4-bit numbers, clamped to 0..15, below c's bits
__device__ __forceinline__ uint32_t pack_u4(int hi, int lo, uint32_t c)
{
    uint32_t d;
    asm("cvt.pack.sat.u4.s32.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(hi), "r"(lo), "r"(c));
    return d;
}

template <int WT, int U, bool ZEROS>
__global__ void __launch_bounds__(kThreads) w4_quantize_kernel(const Quant4Params p, int per_row, int64_t total, int step_rows,
                                                               int step_pieces)
{
    const int lanes = 1 << (p.group_shift - 5);  // threads of a group
    int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    int64_t row = i / per_row;
    int piece = static_cast<int>(i - row * per_row);
    // (a warp goes on as a whole: its groups share by shuffles)
    for (; (i & ~31ll) < total; i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t col = static_cast<int64_t>(piece) * kPer;
        float v[kPer];
        if (i < total) {
            load_piece<WT, U>(p, row, col, v);
        } else {
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                v[k] = 0.f;
        }
        // the largest of w and of -w, or of |w|
        float hi = 0.f, low = 0.f;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            hi = max_nan(hi, ZEROS ? v[k] : fabsf(v[k]));
            if (ZEROS)
                low = max_nan(low, -v[k]);
        }
        for (int o = 1; o < lanes; o <<= 1) {
            hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
            if (ZEROS)
                low = max_nan(low, __shfl_xor_sync(0xffffffffu, low, o));
        }
        float s = ZEROS ? __fmul_rn(__fadd_rn(hi, low), 1.f / 15.f) : __fmul_rn(hi, 1.f / 7.f);
        const bool bad = !(hi < INFINITY) || !(low < INFINITY);  // an infinity or NaN
        if (bad)
            s = __uint_as_float(0x7fc00000u);
        uint16_t s16;
        if (p.s_bf16) {
            s16 = __bfloat16_as_ushort(__float2bfloat16_rn(s));
            s = __bfloat162float(__ushort_as_bfloat16(s16));
        } else {
            s16 = __half_as_ushort(__float2half_rn(s));
            s = __half2float(__ushort_as_half(s16));
        }
        float inv = 0.f;
        if (s >= FLT_MIN)
            inv = __frcp_rn(s);
        else if (s > 0.f)
            s16 = 0;  // 1/s could be infinite: such a group is zero
        int z = 8;
        if (ZEROS)
            z = bad ? 0 : static_cast<int>(fminf(rintf(__fmul_rn(low, inv)), 15.f));
        uint32_t word[kPer / 8];
        if (bad) {
#pragma unroll
            for (int h = 0; h < kPer / 8; ++h)
                word[h] = 0x11111111u * static_cast<uint32_t>(z);
        } else {
            const int bias = z - 0x4b400000;
#pragma unroll
            for (int h = 0; h < kPer / 8; ++h) {
                int q[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    q[k] = __float_as_int(__fadd_rn(__fmul_rn(v[8 * h + k], inv), 12582912.f)) + bias;
                word[h] = pack_u4(q[1], q[0], pack_u4(q[3], q[2], pack_u4(q[5], q[4], pack_u4(q[7], q[6], 0u))));
            }
        }
        if (i < total && col < p.cols) {
            if ((threadIdx.x & (lanes - 1)) == 0) {
                const int64_t group = col >> p.group_shift;
                static_cast<uint16_t*>(p.scales)[row * p.lds + group] = s16;
                if (ZEROS)
                    p.zeros[row * p.ldz + group] = static_cast<uint8_t>(z);
            }
            uint8_t* dst = p.codes + row * p.ldc + (col >> 1);
            if (col + kPer <= p.cols && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
                *reinterpret_cast<uint4*>(dst) = make_uint4(word[0], word[1], word[2], word[3]);
            } else {
#pragma unroll
                for (int k = 0; k < kPer / 2; ++k) {
                    const int64_t left = p.cols - col - 2 * k;  // elements from this byte on
                    const uint32_t byte = word[k >> 2] >> (8 * (k & 3)) & 0xffu;
                    if (left > 0)
                        dst[k] = static_cast<uint8_t>(left == 1 ? byte & 15u : byte);  // an odd row's last high half is zero
                }
            }
        }
        row += step_rows;
        piece += step_pieces;
        if (piece >= per_row) {
            piece -= per_row;
            ++row;
        }
    }
}

template <int WT, int U>
void launch(const Quant4Params& p, unsigned grid, int per_row, int64_t total, cudaStream_t stream)
{
    const int64_t step = static_cast<int64_t>(grid) * kThreads;
    const int rows = static_cast<int>(step / per_row), pieces = static_cast<int>(step % per_row);
    if (p.zeros)
        w4_quantize_kernel<WT, U, true><<<grid, kThreads, 0, stream>>>(p, per_row, total, rows, pieces);
    else
        w4_quantize_kernel<WT, U, false><<<grid, kThreads, 0, stream>>>(p, per_row, total, rows, pieces);
}

template <int WT>
void launch(const Quant4Params& p, uintptr_t at, unsigned grid, int per_row, int64_t total, cudaStream_t stream)
{
    if (at % 16 == 0)
        launch<WT, 16>(p, grid, per_row, total, stream);
    else if (at % 8 == 0)
        launch<WT, 8>(p, grid, per_row, total, stream);
    else if (WT != 2 && at % 4 == 0)
        launch<WT, WT != 2 ? 4 : 0>(p, grid, per_row, total, stream);
    else
        launch<WT, 0>(p, grid, per_row, total, stream);
}

}  // namespace

cudaError_t w4_quantize_launch(const Quant4Params& p, int num_sms, cudaStream_t stream)
{
    const int esize = p.w_type == GEMM_DTYPE_F32 ? 4 : 2;
    // the boundary that every row starts on
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.w) | static_cast<uintptr_t>(p.rows > 1 ? p.ldw * esize : 0);
    // pieces of 32 elements, whole groups of them: a group's threads are neighbours
    const int64_t groups = (p.cols + (int64_t(1) << p.group_shift) - 1) >> p.group_shift;
    const int per_row = static_cast<int>(groups << (p.group_shift - 5));
    const int64_t total = per_row * p.rows;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((total + kThreads - 1) / kThreads, int64_t(num_sms) * 32));
    if (p.w_type == GEMM_DTYPE_F32)
        launch<2>(p, at, grid, per_row, total, stream);
    else if (p.w_type == GEMM_DTYPE_BF16)
        launch<1>(p, at, grid, per_row, total, stream);
    else
        launch<0>(p, at, grid, per_row, total, stream);
    return cudaGetLastError();
}

}  // namespace gnt
