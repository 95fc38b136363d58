// moe.cu -- a mixture-of-experts layer for a few tokens, in two kernels.
//
//   up    h[t,j]  = silu(Wg x_t) * (Wu x_t)        for the experts e_j of token t
//   down  Out[t]  = sum_j p_j W2[e_j] h[t,j]
//
// With few tokens both are bound by reading the chosen experts' weights once
// (6 * hidden * inner bytes an expert in 16 bits), so the kernels are built
// around keeping bytes in flight.  Weights go straight to the warps that use
// them: each warp owns a ring in shared memory, filled with 16-byte cp.async by
// the very lanes that read it back, so that no barrier stands between a load
// and its use.  A warp item is 16 (or 32) weight rows by 64 elements of K; the
// warps of a CTA split K.
//
// Products use mma.sync with fp32 accumulation within an item, items added to
// nearest in fp32 registers (add_item), weights on the 16-row side and 8
// tokens on the other.  The up kernel multiplies x as it is, m16n8k16 in x's
// type, with weights of that type or E4M3 ones widened to it (exact).  h is fp32;
// for bf16 and E4M3 weights it is stored as the sum of two bf16 values (16
// significant bits, fp32's range; the error, 2^-18 of a value at most, is 1/500 of what
// rounding Out to bf16 adds, and 1/60 in fp16) and multiplied as two bf16 operands.  fp16
// weights do not fit bf16 and fp16 does not hold h's range, so there the down
// kernel multiplies in tf32 (m16n8k8), which holds every fp16 value, h in two
// parts again.  The order of K inside an item is free as long as both operands
// share it: a lane takes 16 contiguous bytes of a row, and its consecutive
// elements feed the slots of the MMA that are its own.
//
// With 64 tokens the warps' own time on an item bounds the kernels, not memory: an
// item of 2 KB of E4M3 weights costs a warp 380 instructions in the up kernel and 460
// in the down kernel (counted, with their part of the routing), and rings and sums
// leave an SM 16 warps.  So an item's loads and loop are kept to running pointers
// and immediate offsets, and the next item's load goes out before the arithmetic.
// (Widening E4M3 through fp16 costs little: leaving it out took 7 % off 64 tokens.)
//
// Measured, 64 experts of 2048 x 1024, 8 a token: one token 28 us in bf16 (100 MB,
// 15 us at the memory's rate; two launches and their first loads take 7.5), 64 tokens
// 142 us in E4M3 (403 MB, 60 us), 178 in bf16 (805 MB, 119 us).  16 tokens on 8
// experts of 4096 x 8192, 2 a token: 253 to 276 us (1.6 GB, 235 us).
//
// Routing is recomputed by every CTA from the logits, a few thousand
// instructions; that spares a kernel and a round trip through memory.
#include <algorithm>

#include "gemm_nt.h"
#include "block128.h"
#include "internal.h"
#include "ptx.cuh"

namespace gnt {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kItem = 64;  // elements of K per warp item

// ---------------------------------------------------------------- small PTX
// 16 bytes global -> shared; bytes past `n` (0..16) of the source are zeros
// and are not read.  .cg: past L1, for data read once; .ca: through L1.
__device__ __forceinline__ void cp_async_cg(uint32_t dst, const void* src, int n)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_ca(uint32_t dst, const void* src, int n)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_tf32(float (&c)[4], float a0, float a1, float a2, float a3, float b0, float b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
          "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

// m16n8k16 in fp16 or bf16: a and b as packed pairs.
template <bool BF16>
__device__ __forceinline__ void mma_16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1)
{
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The tf32 value that is left of v when its low 13 bits are dropped.
__device__ __forceinline__ float tf32_head(float v) { return __uint_as_float(__float_as_uint(v) & 0xffffe000u); }

__device__ __forceinline__ float ld_cluster(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// v - head, exact; nothing for an infinity, which its head holds whole.
__device__ __forceinline__ float tf32_rest(float v, float head) { return fabsf(v) < INFINITY ? v - head : 0.f; }

// Two E4M3 bytes -> a pair of fp16 or bf16 values (exact; NaN stays NaN).
template <bool BF16>
__device__ __forceinline__ uint32_t widen_e4m3(uint32_t w)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
    if constexpr (BF16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
        h = *reinterpret_cast<const uint32_t*>(&b);
    }
    return h;
}

// ---------------------------------------------------------------- routing
// Per CTA, in shared memory.  A slot is token * topk + j.
struct Route {
    uint32_t* mask;    // [experts][words]: bit t of an expert's mask: token t takes it
    float* p;          // [slots]
    uint16_t* chosen;  // [slots] expert, 0xffff: none
    uint16_t* list;    // [slots] slots by expert, then token
    uint16_t* off;     // [experts] start of each expert's part of list
    uint16_t* act;     // [active + 1] experts with tokens, ascending, one entry for every `group` of them
    uint16_t* aoff;    // [active + 1] their starts in list; the last entry closes it
    uint8_t* bad;      // [tokens] the token's logits hold a NaN
    int* nact;
};

// Most entries of Route::act: a group has 8 tokens at least, but for an expert's last.
__host__ __device__ constexpr int route_entries(int experts, int slots)
{
    return (experts < slots ? experts : slots) + slots / 8;
}

__host__ __device__ constexpr int route_bytes(int tokens, int experts, int topk)
{
    const int words = (tokens + 31) / 32, slots = tokens * topk, act = route_entries(experts, slots);
    const int b = 4 * (experts * words + slots + 1) + 2 * (2 * slots + experts + 2 * (act + 1)) + tokens;
    return (b + 15) / 16 * 16;
}

__device__ __forceinline__ Route route_carve(uint8_t* s, const MoeParams& p)
{
    const int words = (p.tokens + 31) / 32, slots = p.tokens * p.topk;
    const int act = route_entries(p.experts, slots);
    Route r;
    r.mask = reinterpret_cast<uint32_t*>(s);
    r.p = reinterpret_cast<float*>(r.mask + p.experts * words);
    r.nact = reinterpret_cast<int*>(r.p + slots);
    r.chosen = reinterpret_cast<uint16_t*>(r.nact + 1);
    r.list = r.chosen + slots;
    r.off = r.list + slots;
    r.act = r.off + p.experts;
    r.aoff = r.act + act + 1;
    r.bad = reinterpret_cast<uint8_t*>(r.aoff + act + 1);
    return r;
}

// Unsigned keys in the order of the floats; 0 marks what cannot be taken (NaN,
// or taken already), and a -inf is below kAbove.
constexpr uint32_t kAbove = 0x00800000u;
__device__ __forceinline__ uint32_t order_key(float v)
{
    const uint32_t u = __float_as_uint(v);
    return v != v ? 0u : (u & 0x80000000u ? ~u : u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// One warp, one token: topk rounds of a warp-wide maximum over keys held in
// registers (VPL experts a lane), the lowest index among equals; lane j keeps
// round j's result.
template <int VPL>
__device__ __forceinline__ void route_token(const MoeParams& p, const Route& r, int t, int lane)
{
    const float* l = p.logits + t * p.ldl;
    const int words = (p.tokens + 31) / 32;
    uint32_t key[VPL];
    bool nan = false;  // + 0 below makes -0 and 0 the tie they are
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        const float v = e < p.experts ? __fadd_rn(l[e], 0.f) : -INFINITY;
        nan |= v != v;
        key[i] = order_key(v);
    }
    nan = __any_sync(0xffffffffu, nan);
    float all = 0.f;  // sum of exponentials over every expert (softmax before the choice)
    uint32_t top = 0, mine = 0;
    int at = -1;
    for (int j = 0; j < p.topk; ++j) {
        uint32_t best = 0;
        int idx = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (key[i] > best) {
                best = key[i];
                idx = lane + 32 * i;
            }
        const uint32_t m = __reduce_max_sync(0xffffffffu, best);
        if (m < kAbove)
            break;
        const int e = static_cast<int>(__reduce_min_sync(0xffffffffu, best == m ? static_cast<uint32_t>(idx) : ~0u));
        if (j == 0) {
            top = m;
            if (!p.renorm) {
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if (key[i] >= kAbove)
                        all += expf(key_value(key[i]) - key_value(m));
            }
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (e == lane + 32 * i)
                key[i] = 0;
        if (lane == j) {
            mine = m;
            at = e;
        }
    }
    const float ev = at >= 0 ? expf(key_value(mine) - key_value(top)) : 0.f;
    float sum = p.renorm ? ev : all;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, s);
    if (lane < p.topk) {
        r.chosen[t * p.topk + lane] = at >= 0 ? static_cast<uint16_t>(at) : uint16_t(0xffff);
        r.p[t * p.topk + lane] = nan ? NAN : ev / sum;
        if (at >= 0)
            atomicOr(&r.mask[at * words + t / 32], 1u << (t & 31));
    }
    if (lane == 0)
        r.bad[t] = nan;
}

// One warp, 32 / L tokens at once, L lanes and VPL keys a lane for each: topk
// rounds of a maximum over a token's keys, the lowest index among equals.  With
// many tokens few lanes each are best (64 tokens of 64 experts took 9 thousand
// cycles a token and warp at a time); with few, whole warps.
template <int VPL, int L>
__device__ __forceinline__ void route_tokens(const MoeParams& p, const Route& r, int t0, int lane)
{
    const int words = (p.tokens + 31) / 32, sub = lane % L, t = t0 + lane / L;
    const bool live = t < p.tokens;
    const float* l = p.logits + (live ? t : 0) * p.ldl;
    uint32_t key[VPL];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = sub + L * i;
        const float v = live && e < p.experts ? __fadd_rn(l[e], 0.f) : -INFINITY;  // -0 and 0 tie
        nan |= v != v;
        key[i] = order_key(v);
    }
    uint32_t top = 0;
    float all = 0.f;  // sum of exponentials over every expert (softmax before the choice)
    int taken = 0;
    float* out_p = r.p + t * p.topk;
    for (int j = 0; j < p.topk; ++j) {
        uint32_t best = 0, idx = ~0u;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (key[i] > best) {
                best = key[i];
                idx = sub + L * i;
            }
        uint32_t m = best;
#pragma unroll
        for (int s = 1; s < L; s *= 2)
            m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
        uint32_t e = best == m ? idx : ~0u;
#pragma unroll
        for (int s = 1; s < L; s *= 2)
            e = min(e, __shfl_xor_sync(0xffffffffu, e, s));
        if (m >= kAbove) {
            if (j == 0) {
                top = m;
                if (!p.renorm) {
#pragma unroll
                    for (int i = 0; i < VPL; ++i)
                        if (key[i] >= kAbove)
                            all += expf(key_value(key[i]) - key_value(m));
                }
            }
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (e == static_cast<uint32_t>(sub + L * i))
                    key[i] = 0;
            taken = j + 1;
        }
        if (live && sub == 0) {
            const bool has = m >= kAbove;
            r.chosen[t * p.topk + j] = has ? static_cast<uint16_t>(e) : uint16_t(0xffff);
            out_p[j] = key_value(m);
            if (has)
                atomicOr(&r.mask[e * words + t / 32], 1u << (t & 31));
        }
    }
    __syncwarp();
    float sum = all;
    if (p.renorm)
        for (int j = sub; live && j < taken; j += L)
            sum += expf(out_p[j] - key_value(top));
#pragma unroll
    for (int s = 1; s < L; s *= 2) {
        sum += __shfl_xor_sync(0xffffffffu, sum, s);
        nan |= __shfl_xor_sync(0xffffffffu, static_cast<int>(nan), s) != 0;
    }
    if (live) {
        for (int j = sub; j < taken; j += L)
            out_p[j] = nan ? NAN : expf(out_p[j] - key_value(top)) / sum;
        if (sub == 0)
            r.bad[t] = nan;
    }
}

__device__ __forceinline__ void route_all(const MoeParams& p, const Route& r, int group)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int words = (p.tokens + 31) / 32, slots = p.tokens * p.topk;
    for (int i = threadIdx.x; i < p.experts * words; i += kThreads)
        r.mask[i] = 0;
    __syncthreads();
    if (p.tokens > kWarps && p.experts <= 64) {
        for (int t = warp * 8; t < p.tokens; t += kWarps * 8)
            route_tokens<16, 4>(p, r, t, lane);
    } else if (p.tokens > kWarps && p.experts <= 256) {
        for (int t = warp * 2; t < p.tokens; t += kWarps * 2)
            route_tokens<16, 16>(p, r, t, lane);
    } else {
        for (int t = warp; t < p.tokens; t += kWarps) {
            if (p.experts <= 64)
                route_token<2>(p, r, t, lane);
            else
                route_token<32>(p, r, t, lane);
        }
    }
    __syncthreads();
    if (warp == 0) {
        int total = 0, nact = 0;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            const int e = e0 + lane;
            int n = 0;
            if (e < p.experts)
                for (int w = 0; w < words; ++w)
                    n += __popc(r.mask[e * words + w]);
            const int parts = (n + group - 1) / group;
            int incl = n | parts << 16;  // tokens and entries so far, summed in one word
#pragma unroll
            for (int s = 1; s < 32; s *= 2) {
                const int v = __shfl_up_sync(0xffffffffu, incl, s);
                if (lane >= s)
                    incl += v;
            }
            const int start = total + (incl & 0xffff) - n, a = nact + (incl >> 16) - parts;
            if (e < p.experts)
                r.off[e] = static_cast<uint16_t>(start);
            for (int i = 0; i < parts; ++i) {
                r.act[a + i] = static_cast<uint16_t>(e);
                r.aoff[a + i] = static_cast<uint16_t>(start + i * group);
            }
            const int last = __shfl_sync(0xffffffffu, incl, 31);
            nact += last >> 16;
            total += last & 0xffff;
        }
        if (lane == 0) {
            r.aoff[nact] = static_cast<uint16_t>(total);
            *r.nact = nact;
        }
    }
    __syncthreads();
    for (int s = threadIdx.x; s < slots; s += kThreads) {
        const int e = r.chosen[s], t = s / p.topk;
        if (e != 0xffff) {
            int pos = r.off[e] + __popc(r.mask[e * words + t / 32] & ((1u << (t & 31)) - 1));
            for (int w = 0; w < t / 32; ++w)
                pos += __popc(r.mask[e * words + w]);
            r.list[pos] = static_cast<uint16_t>(s);
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------- items
// Shared-memory layout of one ring stage, in 512-byte lines (32 lanes x 16
// bytes): first the weights, then the tokens' side.  A lane holds 16 elements
// of K per row: two chunks of 8 (16-bit weights: k = 32*half + 8*t, t = lane %
// 4), or one of 16 (8-bit: k = 16*t).  TB: bytes of a token's element, 2 (x) or
// 4 (h: 8 fp32 values, or 8 bf16 heads and then their 8 rests).
template <bool W8, int MT, int NT, int TB>
struct Stage {
    static constexpr int PER_ROW = W8 ? 1 : 2;
    static constexpr int W_LINES = MT * 2 * PER_ROW;  // [mt][row half][chunk]
    static constexpr int B_PER_TOKEN = TB;            // 16 elements
    static constexpr int LINES = W_LINES + NT * B_PER_TOKEN;
    static constexpr int BYTES = LINES * 512;
};

// First of the 8 elements of K that a lane's half `hf` covers within an item.
template <bool W8>
__host__ __device__ constexpr int half_k(int t, int hf)
{
    return W8 ? 16 * t + 8 * hf : 32 * hf + 8 * t;
}

__device__ __forceinline__ int clamp16(int bytes) { return bytes < 0 ? 0 : (bytes > 16 ? 16 : bytes); }

// A 16-byte chunk of a row that starts anywhere: byte by byte, zeros past n.
__device__ __noinline__ void copy_bytes(uint32_t dst, const uint8_t* src, int n)
{
    uint32_t w[4] = {0, 0, 0, 0};
    for (int i = 0; i < n; ++i)
        w[i >> 2] |= static_cast<uint32_t>(src[i]) << (8 * (i & 3));
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
}

// One lane's N chunks of one row of an item, chunk c from byte (c / PAIR) * STEP +
// (c % PAIR) * 16 of src to line c.  `bytes` is 16, or 0 for a row that gives
// zeros (src is then any readable row).  `inside`: the whole item lies within the
// row; else ends[c / PAIR] bytes from there are the row's.
template <int N, int PAIR, int STEP, bool STREAM>
__device__ __forceinline__ void load_chunks(uint32_t dst, const uint8_t* src, int bytes, bool inside, int end0, int end1,
                                            bool vec)
{
    if (vec && inside) {
#pragma unroll
        for (int c = 0; c < N; ++c) {
            if (STREAM)
                cp_async_cg(dst + c * 512, src + c / PAIR * STEP + c % PAIR * 16, bytes);
            else
                cp_async_ca(dst + c * 512, src + c / PAIR * STEP + c % PAIR * 16, bytes);
        }
    } else {
#pragma unroll
        for (int c = 0; c < N; ++c) {
            const int n = bytes ? clamp16((c / PAIR ? end1 : end0) - c % PAIR * 16) : 0;
            const uint8_t* from = src + (n ? c / PAIR * STEP + c % PAIR * 16 : 0);
            if (vec)
                cp_async_ca(dst + c * 512, from, n);
            else
                copy_bytes(dst + c * 512, from, n);
        }
    }
}

__device__ __forceinline__ uint4 lds16(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// The 16 weights of a lane's row, as they lie in shared memory: one 16-byte line
// (8 bits) or two (16 bits); and those of one half as 4 packed pairs of the MMA's type.
template <bool W8>
struct RowWeights {
    uint4 v[W8 ? 1 : 2];

    __device__ __forceinline__ void read(uint32_t line, int hf)
    {
        if (!W8)
            v[hf] = lds16(line + 512 * hf);
        else if (hf == 0)
            v[0] = lds16(line);
    }

    template <bool BF16>
    __device__ __forceinline__ void half(int hf, uint32_t (&o)[4]) const
    {
        if constexpr (W8) {
            const uint32_t a = hf ? v[0].z : v[0].x, b = hf ? v[0].w : v[0].y;
            o[0] = widen_e4m3<BF16>(a);
            o[1] = widen_e4m3<BF16>(a >> 16);
            o[2] = widen_e4m3<BF16>(b);
            o[3] = widen_e4m3<BF16>(b >> 16);
        } else {
            o[0] = v[hf].x, o[1] = v[hf].y, o[2] = v[hf].z, o[3] = v[hf].w;
        }
    }
};

__device__ __forceinline__ float2 halves(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// How an item is multiplied: x as it is; h as bf16 heads and rests; h as fp32 on
// tf32 (fp16 weights).
enum { kPlain, kSplit, kTf32 };

// Multiplies one landed item into c: `st` is the lane's own stage address (+ 16 *
// lane), nt token tiles of 8 are in use.
template <int HOW, bool BF16, bool W8, int MT, int NT>
__device__ __forceinline__ void multiply_item(uint32_t st, int nt, float (&c)[MT][NT][4])
{
    using S = Stage<W8, MT, NT, HOW == kPlain ? 2 : 4>;
    RowWeights<W8> raw[2 * MT];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        uint32_t lo[MT][4], hi[MT][4];
#pragma unroll
        for (int m = 0; m < 2 * MT; ++m)
            raw[m].read(st + m * S::PER_ROW * 512, hf);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            raw[2 * m].template half<BF16>(hf, lo[m]);
            raw[2 * m + 1].template half<BF16>(hf, hi[m]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n < nt) {
                const uint32_t line = st + (S::W_LINES + n * S::B_PER_TOKEN) * 512;
                if constexpr (HOW == kTf32) {
                    const uint4 x = lds16(line + 1024 * hf), y = lds16(line + 1024 * hf + 512);
                    const float b[8] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z),
                                        __uint_as_float(x.w), __uint_as_float(y.x), __uint_as_float(y.y),
                                        __uint_as_float(y.z), __uint_as_float(y.w)};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float b0 = tf32_head(b[2 * j]), b1 = tf32_head(b[2 * j + 1]);
                        const float d0 = tf32_rest(b[2 * j], b0), d1 = tf32_rest(b[2 * j + 1], b1);
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const float2 l = halves(lo[m][j]), h = halves(hi[m][j]);
                            mma_tf32(c[m][n], l.x, h.x, l.y, h.y, b0, b1);
                            mma_tf32(c[m][n], l.x, h.x, l.y, h.y, d0, d1);
                        }
                    }
                } else {
#pragma unroll
                    for (int part = 0; part < (HOW == kSplit ? 2 : 1); ++part) {
                        const uint4 w = lds16(line + (HOW == kSplit ? 1024 * hf + 512 * part : 512 * hf));
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            mma_16<BF16>(c[m][n], lo[m][0], hi[m][0], lo[m][1], hi[m][1], w.x, w.y);
                            mma_16<BF16>(c[m][n], lo[m][2], hi[m][2], lo[m][3], hi[m][3], w.z, w.w);
                        }
                    }
                }
            }
        }
    }
}

// Adds an item's products to the sums, times the rows' scales (8-bit weights).  Every
// item starts from zero: an MMA cuts its sums off rather than rounding them, so a
// chain of them over all of K ends low, by 1e-4 of the result at K = 65536; here 4
// to 16 MMAs are chained, and the items are added in fp32 to nearest.
template <bool W8, int MT, int NT>
__device__ __forceinline__ void add_item(float (&c)[MT][NT][4], const float (&part)[MT][NT][4], const float (&s)[2 * MT])
{
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                c[m][n][v] = W8 ? fmaf(part[m][n][v], s[2 * m + (v >> 1)], c[m][n][v]) : c[m][n][v] + part[m][n][v];
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// ---------------------------------------------------------------- up
// A unit is 8*MT gate rows and the 8*MT up rows that go with them (MT m16 tiles:
// an accumulator's lower rows are the gates, its upper ones their ups), over all
// of K, for up to 8*NT of the expert's tokens.  An expert with more tokens has as many
// entries among the active ones, so that CTAs and warps share out work, not experts:
// 64 tokens of which 17 meet on one of 64 experts in E4M3 149 us, 182 with whole
// experts; 128 tokens 226 and 381.  CTAs take even ranges of the units of all entries.
//
// KS warps share a unit and split its K: one, where there are many units for every SM
// (a warp then ends a unit in its own registers; 8 warps meeting after every 4 items
// of K took half of 64 tokens' time); two, where a warp each would leave warps
// without one; all 8, where there are few and a unit's latency counts.  One token on
// 8 of 64 experts of 2048 x I, layer in us:
//   units an SM   2     3     4     5     6.7   10    13    16    21
//   bf16   8     16.3  20.8  22.1  24.9  28.5
//          2     21.7  23.8  21.9  24.4  28.3  38.9  45.1  50.6  64.9
//          1                 25.6        30.0  41.7  45.6  50.5  65.0
//   E4M3   8     15.9  19.4  21.2  23.4  25.5
//          2     21.9  22.2  21.2  23.4  25.6  34.9  40.3  43.5  55.1
//          1                 24.2        27.9  34.5  38.8  41.5  55.9
// hence 8 below 4, 2 up to 16 (E4M3: 8), then 1.
template <bool W8, int MT, int NT, int KS>
struct UpCfg {
    using S = Stage<W8, MT, NT, 2>;
    // A warp alone on 16-bit weights is all latency: one CTA an SM and deep rings (D
    // stages).  E4M3's items are half as long and cost a warp as much: two CTAs
    // (8 tokens on 64 experts 85 us, 97 with one).
    static constexpr int CTAS = KS == 1 && !W8 ? 1 : 2;
    static constexpr int D = KS > 1 ? (NT == 1 || W8 ? 4 : 3) : (NT == 1 ? (W8 ? 6 : 8) : 3);
    static constexpr int RBUF = KS == 1 ? 0 : (NT == 1 ? 2 : 1);  // buffers for the warps' sums
    static constexpr int RING = kWarps * D * S::BYTES;
    static constexpr int FIXED = RING + RBUF * kWarps * NT * 4 * 32 * 4;
    static_assert(kWarps % KS == 0 && (KS == 1 || MT == 1), "unit shapes");
};

// Barrier of the KS warps that share a unit.
template <int KS>
__device__ __forceinline__ void unit_sync(int group)
{
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(32 * KS) : "memory");
}

// h of one element: where it goes in a row's groups of 8 columns (bf16 heads,
// then their rests; or, for fp16 weights, fp32).
template <bool SPLIT>
__device__ __forceinline__ void store_h(float* row, int i0, int j, float gate, float up)
{
    const float h = gate / (1.f + expf(-gate)) * up;
    if constexpr (SPLIT) {
        // the nearest bf16 value to a finite h may be an infinity: the largest one then
        const bool finite = fabsf(h) < INFINITY;
        constexpr float kMax = 3.3895313892515355e38f;
        const __nv_bfloat16 head = __float2bfloat16_rn(finite ? fminf(fmaxf(h, -kMax), kMax) : h);
        const float rest = finite ? h - __bfloat162float(head) : 0.f;
        __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(row + i0) + j;
        o[0] = head;
        o[8] = __float2bfloat16_rn(rest);
    } else {
        row[i0 + j] = h;
    }
}

template <bool BF16, bool W8, int MT, int NT, int KS>
__global__ void __launch_bounds__(kThreads, UpCfg<W8, MT, NT, KS>::CTAS) moe_up_kernel(const MoeParams p)
{
    using C = UpCfg<W8, MT, NT, KS>;
    using S = typename C::S;
    constexpr int D = C::D;
    constexpr bool SPLIT = BF16 || W8;
    extern __shared__ __align__(16) uint8_t smem[];
    float* red = reinterpret_cast<float*>(smem + C::RING);
    const Route r = route_carve(smem + C::FIXED, p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

    pdl_wait();
    // After the wait: the down kernel may start early and read the logits, which
    // are then complete.
    pdl_launch_dependents();
    route_all(p, r, 8 * NT);

    const int tiles = ceil_div(p.inner, 8 * MT), nit = ceil_div(p.hidden, kItem);
    const int64_t units = static_cast<int64_t>(*r.nact) * tiles;
    // this warp's units: u0, u0 + step, ... < u1, K items [ks0, ks1)
    constexpr int step = kWarps / KS;
    const int u0 = static_cast<int>(units * blockIdx.x / gridDim.x) + warp / KS;
    const int u1 = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x);
    const int ks0 = nit * (warp % KS) / KS, ks1 = nit * (warp % KS + 1) / KS;
    const uint32_t ring = smem_u32(smem) + warp * D * S::BYTES + lane * 16;
    constexpr int ES = W8 ? 1 : 2;
    const uint8_t* xb = static_cast<const uint8_t*>(p.x);
    const uint8_t* wb = static_cast<const uint8_t*>(p.w13);

    // Loader: the items (unit, token group, K item) of this warp in order, by
    // pointers to the lane's own bytes.  Rows outside the matrix, and tokens past
    // the group, read nothing of row 0.
    int lu = u0, lk = ks0, lslot = 0;
    const uint8_t* wr[2 * MT];  // gate and up row of each m16 tile
    const uint8_t* xr[NT];
    uint32_t wbytes = 0, xbytes = 0;  // bit m: tile m's rows are inside; bit q: token of tile q
    auto load_next = [&] {
        if (ks0 < ks1 && lu < u1) {
            if (lk == ks0) {
                const int a = lu / tiles, i0 = (lu - a * tiles) * (8 * MT) + g;
                const int n = r.aoff[a + 1] - r.aoff[a];
                const uint8_t* we = wb + static_cast<int64_t>(r.act[a]) * p.stride_w13 * ES + ks0 * (kItem * ES) + t * 16;
                wbytes = xbytes = 0;
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const int i = i0 + 8 * m;
                    wr[2 * m] = wr[2 * m + 1] = we;
                    if (i < p.inner) {
                        wr[2 * m] += static_cast<int64_t>(i) * p.ldw13 * ES;
                        wr[2 * m + 1] += static_cast<int64_t>(p.inner + i) * p.ldw13 * ES;
                        wbytes |= 1u << m;
                    }
                }
#pragma unroll
                for (int q = 0; q < NT; ++q) {
                    const int j = q * 8 + g;
                    xr[q] = xb + ks0 * (kItem * 2) + half_k<W8>(t, 0) * 2;
                    if (j < n) {
                        xr[q] += static_cast<int64_t>(r.list[r.aoff[a] + j] / p.topk) * p.ldx * 2;
                        xbytes |= 1u << q;
                    }
                }
            }
            const uint32_t st = ring + lslot * S::BYTES;
            const bool inside = (lk + 1) * kItem <= p.hidden;
            const int left = p.hidden - lk * kItem, w0 = (left - half_k<W8>(t, 0)) * ES, w1 = (left - half_k<W8>(t, 1)) * ES;
#pragma unroll
            for (int m = 0; m < 2 * MT; ++m) {
                load_chunks<S::PER_ROW, 1, 64, true>(st + m * S::PER_ROW * 512, wr[m], wbytes >> (m / 2) & 1 ? 16 : 0,
                                                     inside, w0, w1, p.vec_13);
                wr[m] += kItem * ES;
            }
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                load_chunks<2, 1, W8 ? 16 : 64, false>(st + (S::W_LINES + q * 2) * 512, xr[q], xbytes >> q & 1 ? 16 : 0,
                                                       inside, (left - half_k<W8>(t, 0)) * 2,
                                                       (left - half_k<W8>(t, 1)) * 2, p.vec_x);
                xr[q] += kItem * 2;
            }
            if (++lk == ks1) {
                lk = ks0;
                lu += step;
            }
        }
        cp_async_commit();
        lslot = lslot + 1 == D ? 0 : lslot + 1;
    };
#pragma unroll 1
    for (int i = 0; i < D - 1; ++i)
        load_next();

    int slot = 0, parity = 0;
#pragma unroll 1
    for (int u = u0; u < u1; u += step) {
        const int a = u / tiles, i0 = (u - a * tiles) * (8 * MT);
        const int first = r.aoff[a], n = r.aoff[a + 1] - first;
        const float* ps[2 * MT];  // the lane's rows' scales
        if (W8) {
            const float* se = p.s13.data + r.act[a] * p.s13.bs;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int i = min(i0 + 8 * m + g, p.inner - 1);
                ps[2 * m] = se + static_cast<int64_t>(i >> p.s13.shift) * p.s13.rs;
                ps[2 * m + 1] = se + static_cast<int64_t>((p.inner + i) >> p.s13.shift) * p.s13.rs;
            }
        }
        const int nt = ceil_div(n, 8);
        float c[MT][NT][4] = {};
#pragma unroll 1
        for (int k = ks0; k < ks1; ++k) {
            float s[2 * MT] = {};
            if (W8) {
                const int64_t kb = static_cast<int64_t>(k >> 1) * p.s13.ks;  // an item is half a block of 128
#pragma unroll
                for (int m = 0; m < 2 * MT; ++m)
                    s[m] = __ldg(ps[m] + kb);
            }
            cp_async_wait<D - 2>();
            load_next();  // into the slot of the item before, which is in registers
            float part[MT][NT][4] = {};
            multiply_item<kPlain, BF16, W8, MT, NT>(ring + slot * S::BYTES, nt, part);
            add_item<W8, MT, NT>(c, part, s);
            slot = slot + 1 == D ? 0 : slot + 1;
        }
        // Columns past inner, to the end of their 8, get zeros (their rows were).
        if constexpr (KS == 1) {
#pragma unroll
            for (int q = 0; q < NT; ++q)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const int j = q * 8 + 2 * t + v;
                    if (j < n) {
                        float* row = p.h + r.list[first + j] * p.ldh;
#pragma unroll
                        for (int m = 0; m < MT; ++m)
                            if (i0 + 8 * m < p.inner)
                                store_h<SPLIT>(row, i0 + 8 * m, g, c[m][q][v], c[m][q][2 + v]);
                    }
                }
        } else {
            float* rd = red + parity * (kWarps * NT * 4 * 32);
            if (C::RBUF == 2)
                parity ^= 1;  // the other buffer is rewritten only after the next unit's barrier
            else
                unit_sync<KS>(warp / KS);
#pragma unroll
            for (int q = 0; q < NT; ++q)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    rd[((warp * NT + q) * 4 + v) * 32 + lane] = c[0][q][v];
            unit_sync<KS>(warp / KS);
            const int w0 = warp / KS * KS;
            for (int idx = threadIdx.x - 32 * w0; idx < nt * 64; idx += 32 * KS) {
                const int l = idx & 31, wh = (idx >> 5) & 1, q = idx >> 6;
                float gate = 0.f, up = 0.f;
#pragma unroll
                for (int w = w0; w < w0 + KS; ++w) {
                    gate += rd[((w * NT + q) * 4 + wh) * 32 + l];
                    up += rd[((w * NT + q) * 4 + 2 + wh) * 32 + l];
                }
                const int j = q * 8 + 2 * (l & 3) + wh;
                if (j < n)
                    store_h<SPLIT>(p.h + r.list[first + j] * p.ldh, i0, l >> 2, gate, up);
            }
        }
    }
    cp_async_wait<0>();
}

// ---------------------------------------------------------------- down
// A cluster of C CTAs owns 16*MT rows of Out and shares the experts' K items.
//
// One token tile (NT == 1): the cluster's warps take even ranges of the items.  A
// warp adds each expert's share, times the tokens' weights, to sums of its own in
// shared memory, so that nothing synchronises until the end, when the warps' and
// then the CTAs' sums are added in a fixed order.
//
// Two token tiles: a warp's own sums would be most of shared memory (64 KB of 211
// at 64 tokens, one CTA an SM).  There a CTA has one set of sums, its items are cut
// into units of one expert, warp w takes units w, w + 8, ..., and adds to the
// sums when the units before have: a fixed order again, and with more units than
// warps nobody waits long.
template <bool W8, int NT, int MT>
struct DownCfg {
    using S = Stage<W8, MT, NT, 4>;
    static constexpr bool TURNS = NT > 1;
    // CTAs an SM, and ring stages within what they leave each other
    static constexpr int CTAS = TURNS ? (W8 ? 2 : 1) : (MT == 1 ? 2 : 1);
    static constexpr int D = NT == 1 ? (W8 ? 4 : 3) : (MT == 2 && !W8 ? 3 : 2);
    static constexpr int RING = kWarps * D * S::BYTES;
    static __host__ __device__ constexpr int sum_bytes(int tokens)
    {
        return (TURNS ? 1 : kWarps) * tokens * 16 * MT * 4 + 16;  // 16: whose turn it is, and whether one gave up
    }
};

__device__ __forceinline__ int turn_word(uint32_t a)
{
    int v;
    asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void set_turn_word(uint32_t a, int v)
{
    asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
// Waits until the word at `turn` is at least `unit`; false after `limit` cycles, or
// once another warp has given up, which the word behind it says and keeps saying.
__device__ __forceinline__ bool wait_turn(uint32_t turn, int unit, unsigned long long limit)
{
    const long long t0 = clock64();
    while (!__all_sync(0xffffffffu, turn_word(turn) >= unit))
        if (__any_sync(0xffffffffu, turn_word(turn + 4) != 0 || static_cast<unsigned long long>(clock64() - t0) > limit))
            return false;
    return true;
}

template <bool BF16, bool W8, int NT, int MT>
__global__ void __launch_bounds__(kThreads, DownCfg<W8, NT, MT>::CTAS) moe_down_kernel(const MoeParams p, int cluster)
{
    using C = DownCfg<W8, NT, MT>;
    using S = typename C::S;
    constexpr int D = C::D, ROWS = 16 * MT, HOW = BF16 || W8 ? kSplit : kTf32;
    constexpr bool TURNS = C::TURNS;
    extern __shared__ __align__(16) uint8_t smem[];
    float* sums = reinterpret_cast<float*>(smem + C::RING);  // [warp][token][row], or [token][row]
    const uint32_t turn = smem_u32(smem) + C::RING + C::sum_bytes(p.tokens) - 16;
    const Route r = route_carve(smem + C::RING + C::sum_bytes(p.tokens), p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rank = static_cast<int>(blockIdx.x % cluster);
    const int r0 = static_cast<int>(blockIdx.x / cluster) * ROWS;

    const int nout = p.tokens * ROWS;
    for (int i = threadIdx.x; i < (TURNS ? 1 : kWarps) * nout; i += kThreads)
        sums[i] = 0.f;
    if (TURNS && threadIdx.x == 0) {
        set_turn_word(turn, 0);
        set_turn_word(turn + 4, 0);
    }
    route_all(p, r, 8 * NT);  // the logits were complete before the up kernel let this one start
    pdl_wait();       // h

    const int nit = ceil_div(p.inner, kItem);
    // The warp's positions [q0, q1): K items of all experts, one after the other; or
    // units of `len` items of an expert, two for every warp where there are enough.
    int len = nit;
    if (TURNS)
        while (len > 4 && *r.nact * ceil_div(nit, len) < 2 * kWarps * cluster)
            len = (len + 1) / 2;
    const int per = TURNS ? ceil_div(nit, len) : nit;  // positions of an expert
    const int64_t all = static_cast<int64_t>(*r.nact) * per;
    const int share = TURNS ? rank : rank * kWarps + warp, shares = TURNS ? cluster : cluster * kWarps;
    const int u0 = static_cast<int>(all * share / shares), q1 = static_cast<int>(all * (share + 1) / shares);
    const int q0 = TURNS ? u0 + warp : u0;
    // Position q: active expert a, K items [k0, k1).
    auto segment = [&](int q, int& a, int& k0, int& k1) {
        a = q / per;
        k0 = TURNS ? (q - a * per) * len : q - a * per;
        k1 = min(nit, k0 + (TURNS ? len : q1 - q));
    };
    const uint32_t ring = smem_u32(smem) + warp * D * S::BYTES + lane * 16;
    constexpr int ES = W8 ? 1 : 2;
    const uint8_t* wb = static_cast<const uint8_t*>(p.w2);
    const uint8_t* hb = reinterpret_cast<const uint8_t*>(p.h);

    // Loader: per expert of the range, per token group, its K items (pointers as in
    // the up kernel; h's rows are whole groups of 8 columns, zeros past inner).
    const int kpad = (p.inner + 7) / 8 * 8;
    int lq = q0, lk = 0, lend = 0, lslot = 0;
    const uint8_t* wr[2 * MT];
    const uint8_t* hr[NT];
    uint32_t wbytes = 0, hbytes = 0;  // bit m: row m is inside; bit q: token of tile q
    bool fresh = true;
    auto load_next = [&] {
        if (lq < q1) {
            if (fresh) {
                int a;
                segment(lq, a, lk, lend);
                const int n = r.aoff[a + 1] - r.aoff[a];
                const uint8_t* we = wb + static_cast<int64_t>(r.act[a]) * p.stride_w2 * ES + lk * (kItem * ES) + t * 16;
                wbytes = hbytes = 0;
#pragma unroll
                for (int m = 0; m < 2 * MT; ++m) {
                    const int row = r0 + 8 * m + g;
                    wr[m] = we;
                    if (row < p.hidden) {
                        wr[m] += static_cast<int64_t>(row) * p.ldw2 * ES;
                        wbytes |= 1u << m;
                    }
                }
#pragma unroll
                for (int q = 0; q < NT; ++q) {
                    const int j = q * 8 + g;
                    hr[q] = hb + lk * (kItem * 4) + half_k<W8>(t, 0) * 4;
                    if (j < n) {
                        hr[q] += static_cast<int64_t>(r.list[r.aoff[a] + j]) * p.ldh * 4;
                        hbytes |= 1u << q;
                    }
                }
                fresh = false;
            }
            const uint32_t st = ring + lslot * S::BYTES;
            const bool inside = (lk + 1) * kItem <= p.inner;
            const int left = p.inner - lk * kItem, w0 = (left - half_k<W8>(t, 0)) * ES, w1 = (left - half_k<W8>(t, 1)) * ES;
            const int h0 = (kpad - lk * kItem - half_k<W8>(t, 0)) * 4, h1 = (kpad - lk * kItem - half_k<W8>(t, 1)) * 4;
#pragma unroll
            for (int m = 0; m < 2 * MT; ++m) {
                load_chunks<S::PER_ROW, 1, 64, true>(st + m * S::PER_ROW * 512, wr[m], wbytes >> m & 1 ? 16 : 0, inside, w0,
                                                     w1, p.vec_2);
                wr[m] += kItem * ES;
            }
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                load_chunks<4, 2, W8 ? 32 : 128, false>(st + (S::W_LINES + q * 4) * 512, hr[q], hbytes >> q & 1 ? 16 : 0,
                                                        inside, h0, h1, true);
                hr[q] += kItem * 4;
            }
            if (++lk == lend) {
                fresh = true;
                lq += TURNS ? kWarps : lend - lq % nit;
            }
        }
        cp_async_commit();
        lslot = lslot + 1 == D ? 0 : lslot + 1;
    };
#pragma unroll 1
    for (int i = 0; i < D - 1; ++i)
        load_next();

    float* mine = sums + (TURNS ? 0 : warp * nout);
    int slot = 0;
#pragma unroll 1
    for (int q = q0; q < q1;) {
        int a, k0, k1;
        segment(q, a, k0, k1);
        const int first = r.aoff[a], n = r.aoff[a + 1] - first;
        const float* ps[2 * MT];  // the lane's rows' scales
        if (W8) {
#pragma unroll
            for (int m = 0; m < 2 * MT; ++m)
                ps[m] = p.s2.data + r.act[a] * p.s2.bs +
                        static_cast<int64_t>(min(r0 + 8 * m + g, p.hidden - 1) >> p.s2.shift) * p.s2.rs;
        }
        const int nt = ceil_div(n, 8);
        float c[MT][NT][4] = {};
#pragma unroll 1
        for (int k = k0; k < k1; ++k) {
            float s[2 * MT] = {};
            if (W8) {
                const int64_t kb = static_cast<int64_t>(k >> 1) * p.s2.ks;  // an item is half a block of 128
#pragma unroll
                for (int m = 0; m < 2 * MT; ++m)
                    s[m] = __ldg(ps[m] + kb);
            }
            cp_async_wait<D - 2>();
            load_next();  // into the slot of the item before, which is in registers
            float part[MT][NT][4] = {};
            multiply_item<HOW, BF16 || W8, W8, MT, NT>(ring + slot * S::BYTES, nt, part);
            add_item<W8, MT, NT>(c, part, s);
            slot = slot + 1 == D ? 0 : slot + 1;
        }
        if (TURNS && !wait_turn(turn, q - u0, p.wait_limit)) {  // nothing is added out of turn
            if (lane == 0) {
                set_turn_word(turn + 4, 1);
                atomicOr(p.status, kStatusTimeout);
            }
            break;
        }
#pragma unroll
        for (int w = 0; w < NT; ++w)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int j = w * 8 + 2 * t + v;
                if (w < nt && j < n) {
                    const int sl = r.list[first + j];
                    const float pw = r.p[sl];
                    float* d = mine + (sl / p.topk) * ROWS + g;
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        d[16 * m] = fmaf(pw, c[m][w][v], d[16 * m]);
                        d[16 * m + 8] = fmaf(pw, c[m][w][2 + v], d[16 * m + 8]);
                    }
                }
            }
        __syncwarp();
        if (TURNS && lane == 0)
            set_turn_word(turn, q - u0 + 1);
        q += TURNS ? kWarps : k1 - k0;
    }
    cp_async_wait<0>();
    __syncthreads();
    if (!TURNS) {
        for (int i = threadIdx.x; i < nout; i += kThreads) {
            float s = sums[i];
#pragma unroll
            for (int w = 1; w < kWarps; ++w)
                s += sums[w * nout + i];
            sums[i] = s;
        }
    }
    cluster_sync();
    const int o0 = static_cast<int>(static_cast<int64_t>(nout) * rank / cluster);
    const int o1 = static_cast<int>(static_cast<int64_t>(nout) * (rank + 1) / cluster);
    const uint32_t base = smem_u32(sums);
    for (int i = o0 + threadIdx.x; i < o1; i += kThreads) {
        float s = 0.f;
        for (int q = 0; q < cluster; ++q)
            s += ld_cluster(mapa_shared(base + 4 * i, q));
        const int tok = i / ROWS, row = r0 + i % ROWS;
        if (r.bad[tok])
            s = NAN;
        if (row < p.hidden) {
            using O = OutStore<BF16 ? kOutBF16 : kOutF16>;
            O::st1(static_cast<typename O::T*>(p.out) + tok * p.ldo + row, s);
        }
    }
    cluster_sync();  // no CTA leaves while another may still read its sums
}

// ---------------------------------------------------------------- host
constexpr int kMaxSmem = 232448;

template <bool BF16, bool W8, int NT, int MT>
cudaError_t configure_one()
{
    constexpr auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(moe_up_kernel<BF16, W8, 1, NT, kWarps>, attr, kMaxSmem);
    if (e == cudaSuccess && NT == 1)
        e = cudaFuncSetAttribute(moe_up_kernel<BF16, W8, 1, 1, 2>, attr, kMaxSmem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(moe_up_kernel<BF16, W8, NT, NT, 1>, attr, kMaxSmem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(moe_down_kernel<BF16, W8, NT, MT>, attr, kMaxSmem);
    return e;
}

template <bool BF16, bool W8, int MT, int NT, int KS>
cudaError_t launch_up(const MoeParams& p, int64_t reach, int num_sms, cudaStream_t stream)
{
    using C = UpCfg<W8, MT, NT, KS>;
    const int64_t units = reach * ((p.inner + 8 * MT - 1) / (8 * MT));
    constexpr int AT_ONCE = kWarps / KS;  // units a CTA works on
    const int64_t ctas = (units + AT_ONCE - 1) / AT_ONCE;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    // every SM in use before a CTA takes as many units as it can
    cfg.gridDim = dim3(static_cast<unsigned>(
        std::min<int64_t>(C::CTAS * num_sms, std::max<int64_t>(ctas, std::min<int64_t>(units, num_sms)))));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::FIXED + route_bytes(p.tokens, p.experts, p.topk);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_up_kernel<BF16, W8, MT, NT, KS>, p);
}

template <bool BF16, bool W8, int NT, int MT>
cudaError_t launch_one(const MoeParams& p, int num_sms, cudaStream_t stream)
{
    const int rb = route_bytes(p.tokens, p.experts, p.topk);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    const int64_t reach = std::min<int64_t>(p.experts, int64_t(p.tokens) * p.topk);  // most experts in use
    // Units of 8*NT columns for a warp alone, two warps or all eight of a CTA (above).
    const int64_t units = reach * ((p.inner + 8 * NT - 1) / (8 * NT));
    cudaError_t e;
    if (NT == 1 && units >= 4 * num_sms && units < (W8 ? 8 : 16) * num_sms)
        e = launch_up<BF16, W8, 1, 1, 2>(p, reach, num_sms, stream);
    else
        e = units >= 4 * num_sms ? launch_up<BF16, W8, NT, NT, 1>(p, reach, num_sms, stream)
                                 : launch_up<BF16, W8, 1, NT, kWarps>(p, reach, num_sms, stream);
    if (e != cudaSuccess)
        return e;
    // The largest clusters whose CTAs are all resident at once, two on an SM where
    // two fit, as long as each warp keeps a few items: a second wave of 512 CTAs after 304 cost one token 9 of 26 us.
    const int tiles = (p.hidden + 16 * MT - 1) / (16 * MT);
    const int64_t items = reach * ((p.inner + kItem - 1) / kItem);
    using Down = DownCfg<W8, NT, MT>;
    const int smem = Down::RING + Down::sum_bytes(p.tokens) + rb;
    const int want = num_sms * (Down::CTAS == 2 && smem <= kMaxSmem / 2 - 2048 ? 2 : 1);
    int c = 1;
    while (c < 8 && 2 * tiles * c <= want && items >= 2 * 2 * c * kWarps)
        c *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * c));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(c);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, moe_down_kernel<BF16, W8, NT, MT>, p, c);
}

// One token tile and 16 rows a warp where an expert hardly ever has more than 8
// tokens: up to 8 of them, or up to 4 on average for an expert (16 tokens on 2 of
// 8 experts); an expert that has more reads its weights again, from L2.  Else two
// token tiles, and 32 rows a warp, which halves how often x and h are read; in
// the down kernel only while the sums of 32 rows fit beside the rings.
template <bool BF16, bool W8>
cudaError_t launch_typed(const MoeParams& p, int num_sms, cudaStream_t stream)
{
    const int rb = route_bytes(p.tokens, p.experts, p.topk);
    if ((p.tokens <= 8 || p.tokens * p.topk <= 4 * p.experts) && UpCfg<W8, 1, 1, 1>::FIXED + rb <= kMaxSmem &&
        DownCfg<W8, 1, 1>::RING + DownCfg<W8, 1, 1>::sum_bytes(p.tokens) + rb <= kMaxSmem)
        return launch_one<BF16, W8, 1, 1>(p, num_sms, stream);
    if (DownCfg<W8, 2, 2>::RING + DownCfg<W8, 2, 2>::sum_bytes(p.tokens) + rb <= kMaxSmem)
        return launch_one<BF16, W8, 2, 2>(p, num_sms, stream);
    return launch_one<BF16, W8, 2, 1>(p, num_sms, stream);
}

// The last form takes anything within the limits.
static_assert(UpCfg<false, 2, 2, 1>::FIXED + route_bytes(kMoeMaxTokens, kMoeMaxExperts, kMoeMaxTopk) <= kMaxSmem &&
                  UpCfg<false, 1, 2, kWarps>::FIXED + route_bytes(kMoeMaxTokens, kMoeMaxExperts, kMoeMaxTopk) <= kMaxSmem &&
                  UpCfg<true, 2, 2, 1>::FIXED + route_bytes(kMoeMaxTokens, kMoeMaxExperts, kMoeMaxTopk) <= kMaxSmem &&
                  UpCfg<true, 1, 2, kWarps>::FIXED + route_bytes(kMoeMaxTokens, kMoeMaxExperts, kMoeMaxTopk) <= kMaxSmem &&
                  DownCfg<false, 2, 1>::RING + DownCfg<false, 2, 1>::sum_bytes(kMoeMaxTokens) +
                          route_bytes(kMoeMaxTokens, kMoeMaxExperts, kMoeMaxTopk) <= kMaxSmem &&
                  DownCfg<true, 2, 1>::RING + DownCfg<true, 2, 1>::sum_bytes(kMoeMaxTokens) +
                          route_bytes(kMoeMaxTokens, kMoeMaxExperts, kMoeMaxTopk) <= kMaxSmem,
              "shared memory at the limits");

template <bool BF16, bool W8>
cudaError_t configure_typed()
{
    cudaError_t e = configure_one<BF16, W8, 1, 1>();
    if (e == cudaSuccess) e = configure_one<BF16, W8, 2, 2>();
    if (e == cudaSuccess) e = configure_one<BF16, W8, 2, 1>();
    return e;
}

}  // namespace

cudaError_t moe_configure()
{
    cudaError_t e = configure_typed<false, false>();
    if (e == cudaSuccess) e = configure_typed<false, true>();
    if (e == cudaSuccess) e = configure_typed<true, false>();
    if (e == cudaSuccess) e = configure_typed<true, true>();
    return e;
}

cudaError_t moe_launch(const MoeParams& p, int num_sms, cudaStream_t stream)
{
    if (p.bf16)
        return p.w8 ? launch_typed<true, true>(p, num_sms, stream) : launch_typed<true, false>(p, num_sms, stream);
    return p.w8 ? launch_typed<false, true>(p, num_sms, stream) : launch_typed<false, false>(p, num_sms, stream);
}

}  // namespace gnt
