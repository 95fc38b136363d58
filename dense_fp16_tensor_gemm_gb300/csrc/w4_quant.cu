// w4_quant.cu -- 4-bit codes of a weight matrix, with one 16-bit scale (and
// optionally a zero point) for each group of 32, 64 or 128 elements of a row.
//
//   symmetric   a = max |w|, s = round16(a * (1/7)), code = clamp(rint(w * (1/s)), -8, 7) + 8
//   with zeros  lo = min(w, 0), hi = max(w, 0), s = round16((hi - lo) * (1/15)),
//               z = clamp(rint(-lo * (1/s)), 0, 15), code = clamp(rint(w * (1/s)) + z, 0, 15)
//
// in fp32, each step rounded, with the rounded s, so that codes and scales
// together stand for the weights as nearly as they can.  A thread holds 8
// consecutive elements (one 16-byte load of 16-bit weights, one 4-byte store of
// codes); a group's 4, 8 or 16 threads share its extremes by shuffles.  Bound by
// memory: one read of the weights.
#include <algorithm>
#include <cfloat>

#include "ffn.h"
#include "gemm_nt.h"

namespace gnt {

namespace {

constexpr int kThreads = 256;

// WT: 0 fp16, 1 bf16, 2 fp32.  VEC: 16-byte aligned rows of weights.
template <int WT, bool VEC>
__device__ __forceinline__ void load8(const Quant4Params& p, int64_t row, int64_t col, float (&v)[8])
{
    if (VEC && col + 8 <= p.cols) {
        if constexpr (WT == 2) {
            const float4* g = reinterpret_cast<const float4*>(static_cast<const float*>(p.w) + row * p.ldw + col);
            const float4 a = __ldcs(g), b = __ldcs(g + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 a = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.w) + row * p.ldw + col));
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 f;
                if constexpr (WT == 1)
                    f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
                else
                    f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = 0.f;
        if (col + i < p.cols) {
            if constexpr (WT == 2)
                v[i] = static_cast<const float*>(p.w)[row * p.ldw + col + i];
            else if constexpr (WT == 1)
                v[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.w)[row * p.ldw + col + i]);
            else
                v[i] = __half2float(static_cast<const __half*>(p.w)[row * p.ldw + col + i]);
        }
    }
}

template <int WT, bool VEC>
__global__ void __launch_bounds__(kThreads) w4_quantize_kernel(const Quant4Params p, int64_t per_row, int64_t total)
{
    const int lane = threadIdx.x & 31;
    const int lanes = 1 << (p.group_shift - 3);  // threads of a group
    // 32 threads take 256 consecutive elements of a row
    for (int64_t i = (blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x) >> 5; i < total;
         i += static_cast<int64_t>(gridDim.x) * (kThreads / 32)) {
        const int64_t row = i / per_row, col = (i - row * per_row) * 256 + lane * 8;
        float v[8];
        load8<WT, VEC>(p, row, col, v);
        float lo = 0.f, hi = 0.f;
        int bad = 0;  // an infinity or NaN
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            lo = fminf(lo, v[k]);
            hi = fmaxf(hi, v[k]);
            bad |= (__float_as_uint(v[k]) & 0x7f800000u) == 0x7f800000u;
        }
        for (int o = 1; o < lanes; o <<= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
            bad |= __shfl_xor_sync(0xffffffffu, bad, o);
        }
        float s = p.zeros ? __fmul_rn(__fsub_rn(hi, lo), 1.f / 15.f) : __fmul_rn(fmaxf(hi, -lo), 1.f / 7.f);
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
        float inv = 0.f;  // also of a NaN: the group's codes are its zero's
        if (s >= FLT_MIN)
            inv = __frcp_rn(s);
        else if (s > 0.f)
            s16 = 0;  // 1/s could be infinite: such a group is zero
        const float z = !p.zeros ? 8.f : (bad ? 0.f : fminf(fmaxf(rintf(__fmul_rn(-lo, inv)), 0.f), 15.f));
        uint32_t word = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float q = bad ? 0.f : rintf(__fmul_rn(v[k], inv));
            word |= static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(q + z, 0.f), 15.f))) << (4 * k);
        }
        if (col < p.cols) {
            const int64_t group = col >> p.group_shift;
            if ((lane & (lanes - 1)) == 0) {
                static_cast<uint16_t*>(p.scales)[row * p.lds + group] = s16;
                if (p.zeros)
                    p.zeros[row * p.ldz + group] = static_cast<uint8_t>(z);
            }
            uint8_t* dst = p.codes + row * p.ldc + (col >> 1);
            const int64_t left = (p.cols - col + 1) >> 1;  // bytes
            if ((p.cols & 1) && left <= 4)
                word &= (1u << (4 * (p.cols - col))) - 1;  // an odd row's last high half is zero
            if (left >= 4 && (reinterpret_cast<uintptr_t>(dst) & 3) == 0) {
                *reinterpret_cast<uint32_t*>(dst) = word;
            } else {
                for (int k = 0; k < 4 && k < left; ++k)
                    dst[k] = static_cast<uint8_t>(word >> (8 * k));
            }
        }
    }
}

template <int WT>
void launch(const Quant4Params& p, bool vec, unsigned grid, int64_t per_row, int64_t total, cudaStream_t stream)
{
    if (vec)
        w4_quantize_kernel<WT, true><<<grid, kThreads, 0, stream>>>(p, per_row, total);
    else
        w4_quantize_kernel<WT, false><<<grid, kThreads, 0, stream>>>(p, per_row, total);
}

}  // namespace

cudaError_t w4_quantize_launch(const Quant4Params& p, int num_sms, cudaStream_t stream)
{
    const int esize = p.w_type == GEMM_DTYPE_F32 ? 4 : 2;
    const bool vec = reinterpret_cast<uintptr_t>(p.w) % 16 == 0 && p.ldw * esize % 16 == 0;
    const int64_t per_row = (p.cols + 255) / 256, total = per_row * p.rows;
    const unsigned grid =
        static_cast<unsigned>(std::min<int64_t>((total + kThreads / 32 - 1) / (kThreads / 32), int64_t(num_sms) * 64));
    if (p.w_type == GEMM_DTYPE_F32)
        launch<2>(p, vec, grid, per_row, total, stream);
    else if (p.w_type == GEMM_DTYPE_BF16)
        launch<1>(p, vec, grid, per_row, total, stream);
    else
        launch<0>(p, vec, grid, per_row, total, stream);
    return cudaGetLastError();
}

}  // namespace gnt
