// block128.h -- declarations shared by the block-scaled (one fp32 scale per 128
// elements of K) product, its quantiser and the few-token expert layer.  Not
// part of the public ABI.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace gnt {

// The scales of one operand: element (batch b, row r, K block c) at
// data[b*bs + (r >> shift)*rs + c*ks]; shift is 0 or 7.
struct ScaleView {
    const float* data;
    int shift;
    int64_t rs, ks, bs;
};

#ifdef __CUDACC__
__device__ __forceinline__ float scale_at(const ScaleView& s, int b, int row, int kb)
{
    return __ldg(s.data + b * s.bs + static_cast<int64_t>(row >> s.shift) * s.rs + static_cast<int64_t>(kb) * s.ks);
}

// A block's sum p times its two scales, which may hold any fp32 values: nothing on
// the way may leave the normal range while the result is inside.  p is zero or, in
// E4M3, from 2^-18 to 2^25, in E5M2 from 2^-32 to 2^39: p * s is zero or normal (or
// has 22 bits left), and the other scale may follow, if |s| lies between 2^-109 or
// 2^-94 and 2^80; zero, infinity and NaN decide the result alone.  2^-109 takes in
// what the quantiser gives a block of zeros, 2^-100 / 448.
__device__ __forceinline__ uint32_t plain_from(int e5m2) { return e5m2 ? (127u - 94) << 23 : (127u - 109) << 23; }
constexpr uint32_t kPlainTo = (127u + 80) << 23;
__device__ __forceinline__ bool plain_scale(float s, uint32_t from)
{
    const uint32_t u = __float_as_uint(s) & 0x7fffffffu;
    return u - from <= kPlainTo - from || u == 0 || u >= 0x7f800000u;
}
__device__ __forceinline__ bool is_normal(float f)
{
    return (__float_as_uint(f) & 0x7fffffffu) - 0x00800000u < 0x7f000000u;
}

// p * s * w as (p * first) * second.  The scales' product where that is normal or
// exact; else both scales are below 1, or both above it: the one nearer to 1 first.
struct Factors {
    float first, second;
};
__device__ __forceinline__ Factors scale_factors(float s, float w)
{
    const float f = s * w, as = fabsf(s), aw = fabsf(w);
    if (is_normal(f) || as == 0.f || aw == 0.f || !(as < INFINITY) || !(aw < INFINITY))
        return {f, 1.f};
    const bool swap = (as > aw) == (fabsf(f) < 1.f);
    return swap ? Factors{s, w} : Factors{w, s};
}
#endif

// One block-scaled product, for every kernel.
struct BlkParams {
    const void* A;
    const void* B;
    void* out;
    int out_type;  // kOutF32, kOutF16, kOutBF16
    int e5m2;      // element type of A and B
    int M, N, K, batch, num_kb;
    int64_t lda, ldb, ldo;
    int64_t stride_a, stride_b, stride_o;
    ScaleView sa, sb;
    // tcgen05 kernels
    int tiles_m, tiles_n, num_tiles, group_m;
    int a_bmul, b_bmul;       // 1 if the tensor map has a batch dimension
    int row_share, x_box;     // swapped kernel: an even share of B's rows per CTA; rows of a B box
    int vec;                  // elements per store that Out's base, pitch and batch stride allow: 8, 4 or 1
    uint32_t idesc_bits;
    uint32_t* status;
    unsigned long long wait_limit;
    int fault;
};

// What a launch needs to know about the current device.
struct DeviceInfo {
    int num_sms;
    int block_pairs;  // CTA pairs of block128_pair resident at once
    int device;       // its index, below 64
    uint32_t* status;
    unsigned long long wait_limit;
    int fault;
};
// Per-device set-up as for every entry point; returns a gemm_status_t value.
int device_info(DeviceInfo* out);

// 3-D tensor map of a K-major operand (see make_map of the API unit).
bool operand_map(CUtensorMap* map, const void* base, int64_t rows, int64_t K, int64_t ld, int64_t batch,
                 int64_t stride, int box_rows, int* bmul, int dtype);

cudaError_t block128_any_launch(const BlkParams& p, cudaStream_t stream);

// CTA pairs, 256 x 256 tiles.
cudaError_t block128_pair_configure(int* max_pairs);  // one-time per device
cudaError_t block128_pair_launch(const BlkParams& p, int max_pairs, cudaStream_t stream);
// Single CTAs, 128 rows of B by up to 128 rows of A, K split over clusters.
cudaError_t block128_swap_configure();  // one-time per device
cudaError_t block128_swap_launch(const BlkParams& p, int num_sms, cudaStream_t stream);

// Quantiser: block (1 x 128 or 128 x 128) scales of X, in X's order (q) and / or
// transposed (qt).
struct QuantParams {
    const void* x;
    int x_type;  // gemm_dtype_t value
    int64_t rows, cols, ldx;
    uint8_t* q;
    int64_t ldq;
    float* sq;
    int64_t sq_rs, sq_ks;
    uint8_t* qt;
    int64_t ldqt;
    float* st;
    int64_t st_rs, st_ks;
    int e5m2;
    int vec_x, vec_q, vec_qt;  // rows allow 16-byte loads / 8-byte stores / 16-byte stores
    int num_sms;
    unsigned ahead;  // set by the launch: CTAs that run at once
};
cudaError_t block128_quantize_launch(const QuantParams& p, bool tile, cudaStream_t stream);

// Mixture-of-experts layer for a few tokens.
constexpr int kMoeMaxTokens = 128, kMoeMaxExperts = 1024, kMoeMaxTopk = 32;
struct MoeParams {
    const void* x;        // tokens x hidden, fp16 or bf16
    int64_t ldx;
    const float* logits;  // tokens x experts
    int64_t ldl;
    const void* w13;      // experts x 2*inner x hidden: gate rows, then up rows
    int64_t ldw13, stride_w13;
    ScaleView s13;        // 8-bit weights only; bs is the expert stride
    const void* w2;       // experts x hidden x inner
    int64_t ldw2, stride_w2;
    ScaleView s2;
    void* out;            // tokens x hidden, x's type
    int64_t ldo;
    float* h;             // workspace: (tokens * topk) x ldh
    int64_t ldh;
    int tokens, experts, topk, hidden, inner, renorm;
    int bf16, w8;         // types: x and Out; weights E4M3 (else x's type)
    int vec_x, vec_13, vec_2;  // rows start on 16-byte boundaries
    uint32_t* status;
    unsigned long long wait_limit;
};
cudaError_t moe_configure();  // one-time per device
cudaError_t moe_launch(const MoeParams& p, int num_sms, cudaStream_t stream);
inline int64_t moe_ldh(int64_t inner) { return (inner + 15) / 16 * 16; }

}  // namespace gnt
