// ffn.h -- declarations shared by the gated feed-forward product, its backward
// pass and the products with 4-bit weights.  Not part of the public ABI.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "few_tokens.h"
#include "internal.h"

namespace gnt {

constexpr int kActSilu = 0, kActGelu = 1, kActGeluTanh = 2;

#ifdef __CUDACC__
// act(g) = g P(g) and its slope P(g) + g P'(g), with P the logistic function
// (silu), the normal distribution function (gelu), or the logistic function of
// 2 sqrt(2/pi) (g + 0.044715 g^3) (gelu_tanh: (1 + tanh v)/2 is the logistic
// function of 2v, which keeps its relative precision where 1 + tanh v cancels;
// so does erfc on the normal one's lower tail).  A quotient below 2^-126 is 0: silu of -88 is
// -0, not -5e-37.
struct ActP {
    float p, d;  // P and P'
};
__device__ __forceinline__ float logistic(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

template <bool SLOPE>
__device__ __forceinline__ ActP act_p(float g, int act)
{
    ActP r;
    r.d = 0.f;
    if (act == kActGelu) {
        r.p = 0.5f * erfcf(g * -0.70710678f);
        if (SLOPE)
            r.d = 0.39894228f * __expf(-0.5f * g * g);
    } else {
        const float v = act == kActSilu ? g : 1.59576912f * (g + 0.044715f * g * g * g);
        r.p = logistic(v);
        if (SLOPE) {
            r.d = r.p - r.p * r.p;
            // past the ends P' is 0, whatever the polynomial's own slope overflows to
            if (act == kActGeluTanh && r.d != 0.f)
                r.d *= 1.59576912f * (1.f + 0.134145f * g * g);
        }
    }
    return r;
}

__device__ __forceinline__ float act_value(float g, int act) { return g * act_p<false>(g, act).p; }
#endif

// One product of tokens with weights, plain or gated:
//   plain  Out[t][j] = sum_k x[t][k] w[j][k]
//   gated  Out[t][j] = act(g) u, g and u the sums with rows j and n + j of w
// Weights are 16-bit (x's type), or 4-bit codes (element 2b in the low half of
// byte b of a row) that stand for (code - zero) * scale, one scale and zero for
// each `1 << group_shift` elements of a row.
struct FfnParams {
    const void* x;
    int64_t ldx;
    const void* w;
    int64_t ldw;           // elements; bytes for 4-bit weights
    const void* scales;    // x's type; null: 16-bit weights
    int64_t lds;
    const uint8_t* zeros;  // null: 8
    int64_t ldz;
    int group_shift;
    void* out;
    int64_t ldo;
    void* gu;  // gated, 16-bit weights: [g u] of every token; null: not kept
    int64_t ldgu;
    int tokens, n, k;
    int gated, act, bf16;
    uint32_t* status;
    unsigned long long wait_limit;
    int fault;
};

// A kernel's limit of dynamic shared memory, set by its first launch on a device.  (The 93
// kernels here and their device memory, 6 MB, are not brought in by the first product of a
// program that launches none of them: 19.8 ms of host time where they were, 13.4 without.)
class SmemLimit {
public:
    template <typename K>
    cudaError_t allow(K* kernel, int bytes, int device)
    {
        const uint64_t bit = uint64_t(1) << device;
        if (done_.load(std::memory_order_acquire) & bit)
            return cudaSuccess;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess)
            done_.fetch_or(bit, std::memory_order_release);
        return e;
    }

private:
    std::atomic<uint64_t> done_{0};  // a bit per device
};

// Launches take the current device's index and SMs.
// Any layout, on the warp MMA.
cudaError_t ffn_any_launch(const FfnParams& p, int num_sms, cudaStream_t stream);

// The gated product with 16-bit weights on CTA pairs; X and W on the 16-byte grid.
cudaError_t gated_pairs(int act, int device, int* pairs);  // pairs that can be resident at once
cudaError_t gated_pair_launch(const FfnParams& p, int pairs, cudaStream_t stream);

// Up to 16 tokens that fit (few_tokens_fit), on the warp MMA; rows of the weights on the
// 16-byte grid.
cudaError_t ffn_few_launch(const FfnParams& p, int device, int num_sms, cudaStream_t stream);

// The weights as the MMA's rows; X and W on the 16-byte grid.  16-bit weights: up to
// kSwapTokens tokens.
constexpr int kSwapTokens = 64;
// 3-D tensor map of a K-major operand (see encode_map of the API unit), and that of gate
// and up rows in turns.  Each call encodes its own and none is kept:
// 0.1 to 0.6 us of a call's 4 on the host.
bool call_map(CUtensorMap* map, const void* base, int64_t rows, int64_t K, int64_t ld, int64_t batch, int64_t stride,
              int box_rows, int dtype);
bool interleaved_map(CUtensorMap* map, const void* base, int64_t n, int64_t K, int64_t ld, int dtype);
cudaError_t ffn_swap_launch(const FfnParams& p, int device, int num_sms, cudaStream_t stream);

// dGU = [dh u act'(g), dh act(g)]
struct GradParams {
    const void* dh;
    int64_t ldd;
    const void* gu;
    int64_t ldgu;
    void* out;
    int64_t ldo;
    int64_t tokens, n;
    int act, bf16;
};
cudaError_t gated_grad_launch(const GradParams& p, int num_sms, cudaStream_t stream);

// 4-bit quantiser.
struct Quant4Params {
    const void* w;
    int w_type;  // gemm_dtype_t value
    int64_t rows, cols, ldw;
    uint8_t* codes;
    int64_t ldc;
    void* scales;
    int64_t lds;
    uint8_t* zeros;  // null: symmetric
    int64_t ldz;
    int group_shift, s_bf16;
};
cudaError_t w4_quantize_launch(const Quant4Params& p, int num_sms, cudaStream_t stream);

// Rows of `bytes` bytes onto 16-byte boundaries (dst and ldd; pitches in bytes).
cudaError_t copy_rows_launch(const void* src, int64_t lds, void* dst, int64_t ldd, int64_t rows, int64_t bytes, cudaStream_t stream);

}  // namespace gnt
