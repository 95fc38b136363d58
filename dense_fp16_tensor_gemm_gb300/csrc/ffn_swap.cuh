// ffn_swap.cuh -- gated products, and plain and gated products with 4-bit weights,
// on tcgen05 with the weights as the MMA's 128 rows and the tokens as its columns.
//
// A CTA owns 128 rows of the weights by up to 256 tokens, over all of K or a
// cluster CTA's share of it.  The accumulator's lane is a row of the weights, so a
// warp stores neighbouring outputs of one token.  Of a gated product each 32 lanes
// hold 16 rows of the gate and the same 16 of the up projection: g and u of an
// output sit 16 lanes apart in one warp, and one exchange per two tokens brings
// them together.
//
// 16-bit weights reach the MMA's shared memory by TMA.  4-bit ones land by TMA as
// they lie (256 of K, 128 bytes a row, at a stage) and sixteen warps turn them into
// 16-bit values (code - zero) * scale, rounded once to the tokens' type, and write
// them to Tensor Memory, 128 x 64 at a time, from where the MMA takes its A operand:
// that needs no shared memory and leaves room for a ring as deep as the round trip
// conversion - MMA - release is long (from four stages in shared memory the
// conversion and the MMAs waited for each other's signals: 64 x 16384 x 8192 65 us).
// A `prmt` puts two neighbours' bytes into the halves of a word, one logical
// operation turns them into small whole numbers on top of 1024 (fp16) or 128 (bf16),
// and subtracting that plus the zero is exact.  The rounding is what lets one MMA run
// over all groups; fewer tokens than the tensor cores need take ffn_few.cu, which has
// none.
//
// 16-bit weights: bound by their bytes (64 tokens x 4096 x 8192 gated 26.0 us, x 2048 x 8192
// 15.0, 6 TB/s between the two and 4 us that every call takes).  4-bit ones, up to 128
// tokens: by no one thing (64 x 16384 x 8192 27.9 us, x 4096 x 4096 12.0; 25.4 without the
// conversion's arithmetic, 20.5 without the scales either, of which 6.6 are launch and ends and
// 13.9 the codes, 5.0 TB/s on 128 of 152 SMs; there the ALU is busy 71 % of the time, issue
// slots 78 %.  Half the tokens' loads change nothing, so pairs of CTAs would not
// either).  More tokens: by the tensor cores and the last round of tiles (2048 x 8192 x 4096
// in bf16, groups of 128, no zero points, 87 us, four rounds of 152 tiles for 3.4; in fp16, groups
// of 64 and zero points, 102).
//
// Roles (768 threads): warp 0 TMA of the weights, warp 1 MMA issue, warp 2 TMA of
// the tokens, warp 3 TMEM allocation, warps 4-19 conversion, warps 20-23 epilogue.
// Every wait is bounded, and a warp that goes on as a whole waits as a whole: all its
// lanes see the same outcome.
#pragma once
#include <algorithm>

#include "block128_tc.cuh"
#include "ffn.h"
#include "gemm_nt.h"

namespace gnt {
namespace swp {

using namespace tc;

constexpr int kThreads = 768;
constexpr int kRowsW = 128;                  // rows of the weights per tile
constexpr int kABytes = kRowsW * BK * 2;     // one k-block of 16-bit weights
constexpr int kRawK = 256;                   // K per stage of codes: 128 bytes a row
constexpr int kRawBytes = kRowsW * kRawK / 2;
constexpr int kRawKb = kRawK / BK;
constexpr int kConvWarps = 8, kConvSets = 2, kEpiWarps = 4;

// NT: tokens per tile.
template <bool W4, int NT>
struct Cfg {
    // k-blocks per stage.  A wait that finds its barrier done still takes a warp about
    // 135 cycles and a commit 60, while the four MMAs of a k-block run 127 at 64 tokens, 254
    // at 128 and 508 at 256: k-blocks share them, as many as leave room for a ring.
    static constexpr int kKb = NT == 256 ? 1 : (W4 && NT <= 64 ? 4 : 2);
    static constexpr int kXBytes = NT * BK * 2;                            // of one k-block
    static constexpr int kStage = kKb * ((W4 ? 0 : kABytes) + kXBytes);  // of shared memory
    static constexpr int kRaw = W4 ? (NT == 256 ? 3 : (NT == 128 ? 5 : 6)) : 0;
    static constexpr int kStages = W4 ? (NT == 256 ? 5 : (NT == 128 ? 4 : 3)) : 4;
    static constexpr int kSmem = 1024 + kStages * kStage + kRaw * kRawBytes + 512;
    // Tensor Memory: the accumulators (one of 256 columns, where the converted
    // weights leave no room for two), then 32 columns of weights a stage
    static constexpr int kAccs = W4 && NT == 256 ? 1 : 2;
    static constexpr int kACol = kAccs * NT;
    static constexpr int kTmem = W4 ? 512 : 2 * NT;
    static_assert(!W4 || kACol + 32 * kKb * kStages <= 512, "weights fit Tensor Memory");
    static_assert(kSmem <= 232448, "shared memory budget");
    static_assert(kStages * kStage >= kRowsW * NT * 4, "a split's sums fit the stages");
    static_assert((2 * kStages + 2 * kRaw + 5) * 8 + 8 <= 512, "barrier area");
    static_assert(kRawKb % kKb == 0, "stages of codes are whole stages");
    // A wait tells a phase from the next, not from the one after that, so no set may come
    // two turns of a ring ahead of the slowest.  From one stage that a set writes to its
    // next one lie at most 1 + (kConvSets - 1) * kPer others.  When it wrote the former, the
    // stage kStages before that had been multiplied, and with it everything before: the
    // latter's last use but one is among that if the gap is at most kStages.  In the ring of
    // codes the fill before last of a set's next stage has to have landed: it has if a
    // stage of its has been multiplied.
    static constexpr int kPer = kRawKb / kKb;
    static_assert(!W4 || 1 + (kConvSets - 1) * kPer <= kStages, "conversion stays within one turn of the ring");
    static_assert(!W4 || (kRaw - kConvSets + 1) * kPer >= kStages + 1, "and of the ring of codes");
};

struct SwapParams {
    FfnParams f;
    int tiles_w, tiles_t, num_tiles, num_kb, splits;
    int vec_s, vec_z;  // rows of scales and zeros on 16- and 8-byte boundaries
    int whole;  // gated: tiles whose outputs end here are whole boxes of the interleaved map
    uint32_t idesc;
};

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
// 32 lanes x 16 columns of 32 bits, from 16 registers of each thread.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D[tmem] (+)= A[tmem] * B[smem desc]^T, 16-bit operands: row i of A is lane i, two
// neighbours of K a column.
__device__ __forceinline__ void tc_mma_ta(uint32_t d, uint32_t a, uint32_t blo, uint32_t bhi, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 db, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(blo), "r"(bhi), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
__device__ __forceinline__ void tma_prefetch_l2_4d(const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2, int32_t c3)
{
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                 : "memory");
}
__device__ __forceinline__ float lds_cluster(uint32_t a)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// 8 codes of a word as 16-bit values, neighbours in one word.
template <bool BF16>
__device__ __forceinline__ void convert8(uint32_t word, uint32_t zero2, uint32_t scale2, uint32_t* out)
{
    constexpr uint32_t magic = BF16 ? 0x43004300u : 0x64006400u;
    const uint32_t high = word >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // bytes: word's i-th and high's i-th, each the low byte of a half
        const uint32_t sel = static_cast<uint32_t>(i) | static_cast<uint32_t>(i) << 4 | static_cast<uint32_t>(4 + i) << 8 |
                             static_cast<uint32_t>(4 + i) << 12;
        uint32_t q;  // bytes & 0x000f000f | magic, in one logical operation
        asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(q) : "r"(__byte_perm(word, high, sel)), "r"(0x000f000fu), "r"(magic));
        if (BF16) {
            __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&q), *reinterpret_cast<const __nv_bfloat162*>(&zero2));
            d = __hmul2(d, *reinterpret_cast<const __nv_bfloat162*>(&scale2));
            out[i] = *reinterpret_cast<const uint32_t*>(&d);
        } else {
            __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&q), *reinterpret_cast<const __half2*>(&zero2));
            d = __hmul2(d, *reinterpret_cast<const __half2*>(&scale2));
            out[i] = *reinterpret_cast<const uint32_t*>(&d);
        }
    }
}

// Where a CTA's work lies: its tile's first output and first token, and its k-blocks.
struct Piece {
    int o0, t0, kb0, kb1;
    int end;  // kb1, or with 4-bit weights the end of its last stage of codes: the ring's
              // stages up to there are passed on too, without k-blocks, so that every stage
              // of codes is as many of the ring's (what keeps the conversion's sets together)
};
// The i-th piece of this CTA; false if there is none.
template <bool W4, bool GATED>
__device__ __forceinline__ bool piece_at(const SwapParams& p, int i, int nt, int rank, Piece& c)
{
    const int t = static_cast<int>(blockIdx.x) / p.splits + i * (static_cast<int>(gridDim.x) / p.splits);
    if (t >= p.num_tiles)
        return false;
    // neighbouring CTAs take the token tiles of one tile of the weights
    c.o0 = t / p.tiles_t * (GATED ? kRowsW / 2 : kRowsW);
    c.t0 = t % p.tiles_t * nt;
    // shares of whole stages of codes
    const int groups = (p.num_kb + kRawKb - 1) / kRawKb;
    c.kb0 = static_cast<int>(static_cast<int64_t>(groups) * rank / p.splits) * kRawKb;
    c.end = static_cast<int>(static_cast<int64_t>(groups) * (rank + 1) / p.splits) * kRawKb;
    c.kb1 = min(p.num_kb, c.end);
    if (!W4)
        c.end = c.kb1;
    return true;
}

// The outputs of 32 tokens in a lane pair of a gated product: lanes 16-31 (`up`) hold rows of the
// up projection, and store the odd tokens.
template <int ACT>
__device__ __forceinline__ void store_gated(const FfnParams& p, int o, int up, int tok0, const float (&v)[32])
{
    float h[16];
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
        const float other = __shfl_xor_sync(0xffffffffu, up ? v[j] : v[j + 1], 16);
        const float g = up ? other : v[j], u = up ? v[j + 1] : other;
        h[j / 2] = act_value(g, ACT) * u;
    }
    unsigned short* dst = static_cast<unsigned short*>(p.out) + static_cast<int64_t>(tok0 + up) * p.ldo + o;
    const int left = o < p.n ? p.tokens - tok0 - up : 0;
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
        if (j < left)
            *dst = p.bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(h[j / 2])) : __half_as_ushort(__float2half_rn(h[j / 2]));
        dst += 2 * p.ldo;
    }
}

// This lane's row of the weights, 32 tokens: its outputs (plain), or with the lane that
// holds the other projection's row the outputs of half the tokens each (gated).
template <bool GATED>
__device__ __forceinline__ void store_tokens(const FfnParams& p, int o0, int row, int tok0, const float (&v)[32], int lane)
{
    const auto bits = [&](float f) {
        return p.bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(f)) : __half_as_ushort(__float2half_rn(f));
    };
    if constexpr (!GATED) {
        const int o = o0 + row;
        if (o < p.n) {
            unsigned short* dst = static_cast<unsigned short*>(p.out) + static_cast<int64_t>(tok0) * p.ldo + o;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                if (tok0 + j < p.tokens)
                    *dst = bits(v[j]);
                dst += p.ldo;
            }
        }
    } else {
        const int up = lane >> 4;
        const int o = o0 + (row >> 5) * 16 + (lane & 15);
        if (p.gu && o < p.n) {
            unsigned short* dst = static_cast<unsigned short*>(p.gu) + static_cast<int64_t>(tok0) * p.ldgu + o + (up ? p.n : 0);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                if (tok0 + j < p.tokens)
                    *dst = bits(v[j]);
                dst += p.ldgu;
            }
        }
        // (the activation is chosen once: a choice per output is a branch behind which the next
        // output's arithmetic waits: 2048 tokens x 2048 x 8192 in 4 bits 171 us, 98 so; 8 outputs
        // at a time 113)
        switch (p.act) {
        case kActSilu: store_gated<kActSilu>(p, o, up, tok0, v); break;
        case kActGelu: store_gated<kActGelu>(p, o, up, tok0, v); break;
        default: store_gated<kActGeluTanh>(p, o, up, tok0, v);
        }
    }
}

// GS: the group's length, as a shift.
template <bool W4, bool BF16, bool GATED, int NT, int GS>
__global__ void __launch_bounds__(kThreads, 1)
    ffn_swap_kernel(const __grid_constant__ CUtensorMap tmw, const __grid_constant__ CUtensorMap tmi,
                    const __grid_constant__ CUtensorMap tmx, const SwapParams p)
{
    using C = Cfg<W4, NT>;
    constexpr int kStages = C::kStages, kRaw = W4 ? C::kRaw : 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* as = smem;
    uint8_t* xs = smem + (W4 ? 0 : kStages * C::kKb * kABytes);
    uint8_t* raw = smem + kStages * C::kStage;
    uint64_t* full = reinterpret_cast<uint64_t*>(raw + C::kRaw * kRawBytes);  // tokens have landed, weights have or are converted
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint64_t* raw_full = drain + 1;
    uint64_t* raw_empty = raw_full + kRaw;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(raw_empty + kRaw);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const FfnParams& f = p.f;
    const unsigned long long limit = f.wait_limit;
    const auto gave_up = [&] {
        *abort_flag = 1;
        atomicOr(f.status, kStatusTimeout);
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1 + (W4 ? kConvWarps : 1));  // the tokens' copy, and the weights' or their conversion
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&tfull[b]), 1);
            mbar_init(smem_u32(&tempty[b]), kEpiWarps);
        }
        mbar_init(smem_u32(drain), 1);
        for (int s = 0; s < kRaw; ++s) {
            mbar_init(smem_u32(&raw_full[s]), 1);
            mbar_init(smem_u32(&raw_empty[s]), kConvWarps);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_map(&tmw);
        tma_prefetch_map(&tmx);
    }
    if (warp == 3) {
        tmem_alloc<C::kTmem>(smem_u32(tmem_slot));
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_launch_dependents();
    if (warp == 0 && lane == 0) {
        // the first ring of weights comes into L2 while the preceding grids finish
        Piece c;
        if (piece_at<W4, GATED>(p, 0, NT, rank, c)) {
            constexpr int step = W4 ? kRawKb : 1;
            for (int i = 0, kb = c.kb0; i < (W4 ? C::kRaw : C::kKb * kStages) && kb < c.kb1; ++i, kb += step) {
                const int x = W4 ? kb * (BK / 2) : kb * BK;
                if (GATED && c.o0 + kRowsW / 2 <= p.whole)
                    tma_prefetch_l2_4d(&tmi, x, 0, 0, c.o0 / 16);
                else if (!GATED)
                    tma_prefetch_l2_3d(&tmw, x, c.o0, 0);
            }
        }
    }
    pdl_wait();

    // waits (bounded) until the copies last posted on each of n barriers have landed
    const auto settle = [&](uint64_t* bars, int n, uint32_t filled, uint32_t parity) {
        for (int s = 0; s < n; ++s) {
            if (filled & (1u << s)) {
                const long long t0 = clock64();
                while (!mbar_try_wait(smem_u32(&bars[s]), (parity >> s) & 1u) &&
                       static_cast<unsigned long long>(clock64() - t0) <= limit) {
                }
            }
        }
    };

    if (warp == 0) {
        // ------------------------------------------------------------ the weights
        if (lane == 0) {
            constexpr int ring = W4 ? kRaw : kStages, kbs = W4 ? kRawKb : C::kKb, bytes = W4 ? kRawBytes : kABytes;
            uint64_t* const fb = W4 ? raw_full : full;
            uint64_t* const eb = W4 ? raw_empty : empty;
            uint8_t* const base = W4 ? raw : as;
            int s = 0;
            uint32_t phase = 0, filled = 0, parity = 0;
            bool first = true, ok = true;
            Piece c;
            for (int i = 0; ok && piece_at<W4, GATED>(p, i, NT, rank, c); ++i) {
                for (int kb = c.kb0; kb < c.kb1; kb += kbs) {
                    if (!wait_bounded(smem_u32(&eb[s]), phase ^ 1, abort_flag, limit)) {
                        gave_up();
                        ok = false;
                        break;
                    }
                    const bool drop = f.fault == 1 && blockIdx.x == 0 && first;
                    first = false;
                    if (!drop) {
                        const uint32_t bar = smem_u32(&fb[s]);
                        const int n = W4 ? 1 : min(kbs, c.kb1 - kb);
                        mbar_arrive_expect_tx(bar, n * bytes);
                        filled |= 1u << s;
                        parity = (parity & ~(1u << s)) | (phase << s);
                        for (int b = 0; b < n; ++b) {
                            const uint32_t dst = smem_u32(base) + (W4 ? s : s * kbs + b) * bytes;
                            const int x = W4 ? kb * (BK / 2) : (kb + b) * BK;
                            if (GATED && c.o0 + kRowsW / 2 <= p.whole) {
                                // (eight boxes a k-block held 64 tokens x 2048 x 8192 to 24.0 us, one 18)
                                tma_load_4d(dst, &tmi, bar, x, 0, 0, c.o0 / 16);
                            } else if (GATED) {
                                // the last tile, where it ends inside 16 rows
#pragma unroll 1
                                for (int q = 0; q < 8; ++q)  // 16 rows of the gate, the same of the up projection
                                    tma_load_3d(dst + q * (bytes / 8), &tmw, bar, x, c.o0 + (q >> 1) * 16, q & 1);
                            } else {
                                tma_load_3d(dst, &tmw, bar, x, c.o0, 0);
                            }
                        }
                    }
                    if (++s == ring) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            settle(fb, ring, filled, parity);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ the tokens
        if (lane == 0) {
            int s = 0;
            uint32_t phase = 0, filled = 0, parity = 0;
            bool ok = true;
            Piece c;
            for (int i = 0; ok && piece_at<W4, GATED>(p, i, NT, rank, c); ++i) {
                for (int kb = c.kb0; kb < c.end; kb += C::kKb) {
                    if (!wait_bounded(smem_u32(&empty[s]), phase ^ 1, abort_flag, limit)) {
                        gave_up();
                        ok = false;
                        break;
                    }
                    const uint32_t bar = smem_u32(&full[s]);
                    const int n = max(0, min(C::kKb, c.kb1 - kb));
                    mbar_arrive_expect_tx(bar, n * C::kXBytes);
                    filled |= 1u << s;
                    parity = (parity & ~(1u << s)) | (phase << s);
                    for (int b = 0; b < n; ++b)
                        tma_load_3d(smem_u32(xs + (s * C::kKb + b) * C::kXBytes), &tmx, bar, (kb + b) * BK, c.t0, 0);
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            settle(full, kStages, filled, parity);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issue
        // The whole warp walks the loop and one lane issues: addresses and descriptors
        // then stay in uniform registers, where the instructions want them (a loop of one
        // thread issues an MMA every 56 cycles, this one every 32 or less).
        {
            const bool one = blk::elect_one();
            const DescWords da = desc_words(smem_u32(as), false), dx = desc_words(smem_u32(xs), false);
            int s = 0;
            uint32_t phase = 0;
            bool skip_release = f.fault == 2 && blockIdx.x == 0;  // test hook: lose one stage release
            bool ok = true;
            Piece c;
            for (int i = 0; ok && piece_at<W4, GATED>(p, i, NT, rank, c); ++i) {
                const int buf = i % C::kAccs;
                if (!blk::wait_lanes(smem_u32(&tempty[buf]), ((i / C::kAccs) & 1) ^ 1, abort_flag, limit)) {
                    gave_up();
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + static_cast<uint32_t>(buf * NT);
                for (int kb = c.kb0; kb < c.end; kb += C::kKb) {
                    if (!blk::wait_lanes(smem_u32(&full[s]), phase, abort_flag, limit)) {
                        gave_up();
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (one) {
#pragma unroll
                        for (int b = 0; b < C::kKb; ++b) {
                            if (kb + b >= c.kb1)
                                break;
                            const int slot = s * C::kKb + b;
                            const uint32_t alo = da.lo + slot * (kABytes >> 4), blo = dx.lo + slot * (C::kXBytes >> 4);
#pragma unroll
                            for (int k = 0; k < BK / 16; ++k) {
                                const uint32_t more = (k > 0 || b > 0 || kb > c.kb0) ? 1u : 0u;
                                if (W4)
                                    tc_mma_ta(d, tmem_base + C::kACol + 32 * slot + 8 * k, blo + k * dx.kstep, dx.hi, p.idesc,
                                              more);
                                else
                                    tc_mma_w<false>(d, alo + k * da.kstep, da.hi, blo + k * dx.kstep, dx.hi, p.idesc, more);
                            }
                        }
                        if (!skip_release)
                            tc_commit(smem_u32(&empty[s]));
                    }
                    __syncwarp();
                    skip_release = false;
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
                if (!ok)
                    break;
                if (one)
                    tc_commit(smem_u32(&tfull[buf]));
                __syncwarp();
            }
            if (one)
                tc_commit(smem_u32(drain));
            __syncwarp();
            const long long t0 = clock64();
            while (!mbar_try_wait(smem_u32(drain), 0) && static_cast<unsigned long long>(clock64() - t0) <= limit) {
            }
        }
    } else if (W4 && warp >= 4 && warp < 4 + kConvSets * kConvWarps) {
        // ------------------------------------------------------------ 4-bit weights to 16 bits
        // A thread converts 32 of K of one row of each k-block.  Two sets of eight warps
        // take the stages of codes in turns.
        const int r = (threadIdx.x - 128) & 127, half = ((threadIdx.x - 128) >> 7) & 1, set = (threadIdx.x - 128) >> 8;
        const uint32_t swz = static_cast<uint32_t>(r & 7);
        const uint32_t raw0 = smem_u32(raw) + r * 128;
        const uint32_t a0 = tmem_base + C::kACol + 16 * half + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        int s = 0, rs = 0, turn = 0;
        uint32_t phase = 0, rphase = 0;
        bool ok = true;
        Piece c;
        for (int i = 0; ok && piece_at<W4, GATED>(p, i, NT, rank, c); ++i) {
            const int o = GATED ? c.o0 + (r >> 5) * 16 + (r & 15) : c.o0 + r;
            const int64_t row = o + (GATED && (r & 16) ? static_cast<int64_t>(f.n) : 0);
            // (rows past the weights are converted with the last one's scales and not stored)
            const int64_t at = o < f.n ? row : static_cast<int64_t>(f.n) - 1;
            const uint16_t* srow = static_cast<const uint16_t*>(f.scales) + at * f.lds;
            const uint8_t* zrow = f.zeros ? f.zeros + at * f.ldz : nullptr;
            // Scales and zeros come eight groups at a time, those of one, two or four stages of
            // codes, in one 16-byte and one 8-byte load a thread, a turn of this set ahead of
            // their use: each load of a warp touches 32 rows, and two of single scales a stage
            // cost 64 x 16384 x 8192 5 us.
            const int chunks = ((f.k - 1) >> (GS + 3)) + 1, last = (f.k - 1) >> GS;
            const auto chunk_of = [&](int kb) { return min(kb * BK >> (GS + 3), chunks - 1); };
            const auto fetch = [&](int ch, uint4& sc, uint2& ze) {
                const bool whole = 8 * ch + 8 <= last + 1;  // (no element past a row's last is read)
                if (whole && p.vec_s) {
                    sc = __ldg(reinterpret_cast<const uint4*>(srow) + ch);
                } else {
                    uint32_t v[8];
#pragma unroll
                    for (int b = 0; b < 8; ++b)
                        v[b] = __ldg(srow + min(8 * ch + b, last));
                    sc = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
                }
                ze = make_uint2(0x08080808u, 0x08080808u);
                if (zrow && whole && p.vec_z) {
                    ze = __ldg(reinterpret_cast<const uint2*>(zrow) + ch);
                } else if (zrow) {
                    uint32_t v[8];
#pragma unroll
                    for (int b = 0; b < 8; ++b)
                        v[b] = __ldg(zrow + min(8 * ch + b, last));
                    ze = make_uint2(v[0] | v[1] << 8 | v[2] << 16 | v[3] << 24, v[4] | v[5] << 8 | v[6] << 16 | v[7] << 24);
                }
            };
            // (the whole piece's come into L2 first: a turn is shorter than a load from memory)
            if (set == 0 && half == 0) {
                const int g1 = min(c.end * BK >> GS, last + 1);
                for (int g = c.kb0 * BK >> GS; g < g1; g += 64)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(srow + g));
                if (zrow)
                    for (int g = c.kb0 * BK >> GS; g < g1; g += 128)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(zrow + g));
            }
            uint4 scales, scales1;
            uint2 zeros, zeros1;
            int chunk = chunk_of(c.kb0 + (set + kConvSets - turn) % kConvSets * kRawKb);
            fetch(chunk, scales, zeros);
            for (int kb = c.kb0; ok && kb < c.kb1; kb += kRawKb) {
                if (turn == set) {
                    const int chunk1 = chunk_of(kb + kConvSets * kRawKb);
                    if (chunk1 != chunk)
                        fetch(chunk1, scales1, zeros1);
                    // the groups of this stage's k-blocks, first of them `first` of the eight
                    const int first = kb * BK >> GS & 7;
                    uint32_t sw[2], zw;  // scales 0-3 and zeros 0-3 of the stage (of shorter groups: this half's)
                    if (GS == 7) {
                        sw[0] = first & 4 ? (first & 2 ? scales.w : scales.z) : (first & 2 ? scales.y : scales.x);
                        sw[1] = 0;
                        zw = (first & 4 ? zeros.y : zeros.x) >> (first & 2 ? 16 : 0);
                    } else if (GS == 6) {
                        sw[0] = first & 4 ? scales.z : scales.x;
                        sw[1] = first & 4 ? scales.w : scales.y;
                        zw = first & 4 ? zeros.y : zeros.x;
                    } else {
                        sw[0] = __byte_perm(scales.x, scales.y, half ? 0x7632 : 0x5410);
                        sw[1] = __byte_perm(scales.z, scales.w, half ? 0x7632 : 0x5410);
                        zw = __byte_perm(zeros.x, zeros.y, half ? 0x7531 : 0x6420);
                    }
                    if (!blk::wait_lanes(smem_u32(&raw_full[rs]), rphase, abort_flag, limit)) {
                        gave_up();
                        ok = false;
                        break;
                    }
                    const int left = f.k - (kb * BK + half * 32);  // elements inside K
#pragma unroll
                    for (int j = 0; j < kRawKb; j += C::kKb) {
                        if (!blk::wait_lanes(smem_u32(&empty[s]), phase ^ 1, abort_flag, limit)) {
                            gave_up();
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll
                        for (int b = 0; b < C::kKb; ++b) {
                            const int jb = j + b;  // (past the last k-block: zeros, which nothing reads)
                            const uint4 w = lds128(raw0 + rs * kRawBytes + (((2 * jb + half) ^ swz) << 4));
                            const uint32_t words[4] = {w.x, w.y, w.z, w.w};
                            const int at = GS == 7 ? jb >> 1 : jb;
                            const uint32_t scale2 = __byte_perm(sw[at >> 1], 0, at & 1 ? 0x3232 : 0x1010);
                            const uint32_t zero2 = __byte_perm(zw, BF16 ? 0x43 : 0x64, 0x4040 | at | at << 8);
                            uint32_t out[16];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                convert8<BF16>(words[e], zero2, scale2, out + 4 * e);
                            if (left < 32 + jb * BK) {
                                // past K: zeros, whatever the scale
#pragma unroll
                                for (int h = 0; h < 16; ++h) {
                                    const int l = left - jb * BK - 2 * h;
                                    out[h] &= l >= 2 ? 0xffffffffu : (l == 1 ? 0xffffu : 0u);
                                }
                            }
                            tmem_st16(a0 + 32 * (s * C::kKb + b), out);
                        }
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(smem_u32(&full[s]));
                        if (++s == kStages) {
                            s = 0;
                            phase ^= 1;
                        }
                    }
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_u32(&raw_empty[rs]));
                    if (chunk1 != chunk) {
                        scales = scales1;
                        zeros = zeros1;
                        chunk = chunk1;
                    }
                } else {  // the other set's
                    s += C::kPer;
                    if (s >= kStages) {
                        s -= kStages;
                        phase ^= 1;
                    }
                }
                if (++rs == kRaw) {
                    rs = 0;
                    rphase ^= 1;
                }
                turn = turn + 1 == kConvSets ? 0 : turn + 1;
            }
        }
    } else if (warp >= 20) {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;
        Piece c;
        for (int i = 0; piece_at<W4, GATED>(p, i, NT, rank, c); ++i) {
            const int buf = i % C::kAccs;
            if (!blk::wait_lanes(smem_u32(&tfull[buf]), (i / C::kAccs) & 1, abort_flag, limit)) {
                gave_up();
                break;
            }
            tc_fence_after();
            const uint32_t tacc = tmem_base + static_cast<uint32_t>(buf * NT) + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
            for (int n = 0; n < NT; n += 32) {
                if (c.t0 + n >= f.tokens)
                    break;
                uint32_t r[32];
                tmem_ld32_wait(tacc + static_cast<uint32_t>(n), r);
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = __uint_as_float(r[j]);
                if (p.splits == 1) {
                    store_tokens<GATED>(f, c.o0, q * 32 + lane, c.t0 + n, v, lane);
                } else {
                    // every MMA has read its operands: the stages take the sums, [token][row]
                    float* sums = reinterpret_cast<float*>(smem) + n * kRowsW + q * 32 + lane;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        sums[j * kRowsW] = v[j];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&tempty[buf]));
        }
    }

    tc_fence_before();
    __syncthreads();
    if (p.splits > 1) {
        // A split has one tile per cluster.  Each CTA sums 32 tokens at a time, in the CTAs' order.
        cluster_sync();
        Piece c;
        if (warp >= 20 && piece_at<W4, GATED>(p, 0, NT, rank, c)) {
            const int row = (warp & 3) * 32 + lane;
            for (int n = rank * 32; n < NT && c.t0 + n < f.tokens; n += p.splits * 32) {
                float v[32] = {};
                for (int k = 0; k < p.splits; ++k) {
                    const uint32_t at = mapa_shared(smem_u32(smem), static_cast<uint32_t>(k)) + (n * kRowsW + row) * 4;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] += lds_cluster(at + j * (kRowsW * 4));
                }
                store_tokens<GATED>(f, c.o0, row, c.t0 + n, v, lane);
            }
        }
        cluster_sync();  // nobody leaves while its sums are read
    }
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc<C::kTmem>(tmem_base);
    }
}

struct Launch {
    int device, grid;
    cudaStream_t stream;
};

template <bool W4, bool BF16, bool GATED, int NT, int GS>
cudaError_t run(const CUtensorMap* maps, const SwapParams& p, const Launch& l)
{
    auto* kernel = ffn_swap_kernel<W4, BF16, GATED, NT, GS>;
    static SmemLimit limit;
    const cudaError_t e = limit.allow(kernel, Cfg<W4, NT>::kSmem, l.device);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.splits);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(l.grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<W4, NT>::kSmem;
    cfg.stream = l.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, maps[0], maps[1], maps[2], p);
}

template <bool W4, bool BF16, bool GATED, int GS>
cudaError_t by_tokens(int nt, const CUtensorMap* maps, const SwapParams& p, const Launch& l)
{
    if (nt == 32)
        return run<W4, BF16, GATED, 32, GS>(maps, p, l);
    if constexpr (W4) {
        if (nt == 256)
            return run<W4, BF16, GATED, 256, GS>(maps, p, l);
        if (nt == 128)
            return run<W4, BF16, GATED, 128, GS>(maps, p, l);
    }
    return run<W4, BF16, GATED, 64, GS>(maps, p, l);
}

template <bool BF16, bool GATED>
cudaError_t by_group(int shift, int nt, const CUtensorMap* maps, const SwapParams& p, const Launch& l)
{
    switch (shift) {
    case 5: return by_tokens<true, BF16, GATED, 5>(nt, maps, p, l);
    case 6: return by_tokens<true, BF16, GATED, 6>(nt, maps, p, l);
    default: return by_tokens<true, BF16, GATED, 7>(nt, maps, p, l);
    }
}

}  // namespace swp
}  // namespace gnt
