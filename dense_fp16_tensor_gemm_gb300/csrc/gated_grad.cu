// gated_grad.cu -- the gradient at a gated product's two projections:
//   dg = dh u act'(g),  du = dh act(g)
// from dh and the g and u that the forward pass kept.  Each of dg and du is
// rounded once to 16 bits, the operands' type of the two products that follow.
// Bound by memory: 6 bytes read and 4 written per element (4096 x 8192 silu in 50 us, 6.7 TB/s;
// 55 where the activation was chosen per element), with gelu by erfc's and exp's instructions
// (81 us).  At an odd width, where nothing but single elements can be read, 3001 x 2047 silu
// in 16 us.
#include <algorithm>

#include "ffn.h"

namespace gnt {

namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ float2 unpack(uint32_t v)
{
    if (BF16)
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

template <int ACT>
__device__ __forceinline__ void grad(float dh, float g, float u, float& dg, float& du)
{
    const ActP a = act_p<true>(g, ACT);
    // (where P' is 0 the slope is P, also for an infinite g)
    dg = dh * u * (a.d == 0.f ? a.p : fmaf(g, a.d, a.p));
    du = dh * (g * a.p);
}

// 8 elements per thread and operand, rows that allow 16-byte loads and stores.
template <bool BF16, int ACT>
__global__ void __launch_bounds__(kThreads) gated_grad_kernel(const GradParams p, int64_t per_row, int64_t total)
{
    using S = OutStore<BF16 ? kOutBF16 : kOutF16>;
    const uint16_t* dh = static_cast<const uint16_t*>(p.dh);
    const uint16_t* gu = static_cast<const uint16_t*>(p.gu);
    typename S::T* out = static_cast<typename S::T*>(p.out);
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t row = i / per_row, col = (i - row * per_row) * 8;
        const uint4 d = __ldcs(reinterpret_cast<const uint4*>(dh + row * p.ldd + col));
        const uint4 g = __ldcs(reinterpret_cast<const uint4*>(gu + row * p.ldgu + col));
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(gu + row * p.ldgu + p.n + col));
        const uint32_t dw[4] = {d.x, d.y, d.z, d.w}, gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
        uint32_t og[4], ou[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 fd = unpack<BF16>(dw[k]), fg = unpack<BF16>(gw[k]), fu = unpack<BF16>(uw[k]);
            float2 a, b;
            grad<ACT>(fd.x, fg.x, fu.x, a.x, b.x);
            grad<ACT>(fd.y, fg.y, fu.y, a.y, b.y);
            og[k] = S::pack(a.x, a.y);
            ou[k] = S::pack(b.x, b.y);
        }
        // (kept in L2 where it fits: the products read it next)
        *reinterpret_cast<uint4*>(out + row * p.ldo + col) = make_uint4(og[0], og[1], og[2], og[3]);
        *reinterpret_cast<uint4*>(out + row * p.ldo + p.n + col) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
    }
}

// Any layout (an odd number of columns puts u's and du's rows off every boundary): single
// elements, four of a row in flight per thread, blockDim.y rows to a CTA.
template <bool BF16, int ACT>
__global__ void __launch_bounds__(kThreads) gated_grad_any_kernel(const GradParams p)
{
    using S = OutStore<BF16 ? kOutBF16 : kOutF16>;
    const auto at = [](uint16_t v) {
        return BF16 ? __bfloat162float(__ushort_as_bfloat16(v)) : __half2float(__ushort_as_half(v));
    };
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; row < p.tokens;
         row += static_cast<int64_t>(gridDim.x) * blockDim.y) {
        const uint16_t* dh = static_cast<const uint16_t*>(p.dh) + row * p.ldd;
        const uint16_t* gu = static_cast<const uint16_t*>(p.gu) + row * p.ldgu;
        typename S::T* out = static_cast<typename S::T*>(p.out) + row * p.ldo;
        for (int64_t c = threadIdx.x; c < p.n; c += 4 * blockDim.x) {
            uint16_t d[4], g[4], u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t col = c + k * blockDim.x;
                if (col < p.n) {
                    d[k] = __ldcs(dh + col);
                    g[k] = __ldcs(gu + col);
                    u[k] = __ldcs(gu + p.n + col);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t col = c + k * blockDim.x;
                if (col < p.n) {
                    float a, b;
                    grad<ACT>(at(d[k]), at(g[k]), at(u[k]), a, b);
                    out[col] = S::pack(a, 0.f) & 0xffffu;
                    out[p.n + col] = S::pack(b, 0.f) & 0xffffu;
                }
            }
        }
    }
}

template <bool BF16, int ACT>
void launch(const GradParams& p, int num_sms, cudaStream_t stream)
{
    const auto on16 = [](const void* q, int64_t ld) { return reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld % 8 == 0; };
    if (p.n % 8 == 0 && on16(p.dh, p.ldd) && on16(p.gu, p.ldgu) && on16(p.out, p.ldo)) {
        const int64_t per_row = p.n / 8, total = per_row * p.tokens;
        const unsigned grid = static_cast<unsigned>(std::min<int64_t>((total + kThreads - 1) / kThreads, int64_t(num_sms) * 64));
        gated_grad_kernel<BF16, ACT><<<grid, kThreads, 0, stream>>>(p, per_row, total);
        return;
    }
    unsigned x = 32;
    while (x < kThreads && x * 4 < p.n)
        x *= 2;
    const dim3 block(x, kThreads / x);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((p.tokens + block.y - 1) / block.y, int64_t(num_sms) * 64));
    gated_grad_any_kernel<BF16, ACT><<<grid, block, 0, stream>>>(p);
}

template <bool BF16>
void by_act(const GradParams& p, int num_sms, cudaStream_t stream)
{
    switch (p.act) {
    case kActSilu: return launch<BF16, kActSilu>(p, num_sms, stream);
    case kActGelu: return launch<BF16, kActGelu>(p, num_sms, stream);
    default: return launch<BF16, kActGeluTanh>(p, num_sms, stream);
    }
}

}  // namespace

cudaError_t gated_grad_launch(const GradParams& p, int num_sms, cudaStream_t stream)
{
    if (p.bf16)
        by_act<true>(p, num_sms, stream);
    else
        by_act<false>(p, num_sms, stream);
    return cudaGetLastError();
}

}  // namespace gnt
