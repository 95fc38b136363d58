// block128_pair.cu -- block-scaled 8-bit product on CTA pairs (tcgen05,
// cta_group::2).
//
//   Out[i,j] = sum_c sa[i,c] sb[j,c] P_c[i,j],   P_c = sum_{k in block c} A[i,k] B[j,k]
//
// The scales change with every 128 elements of K, so the tensor core cannot
// accumulate over blocks: each block's P_c is a fresh accumulator in Tensor
// Memory, and "promotion" warps take it out, scale it and add it to sums they
// hold in registers.  A pair owns a 256 x 256 tile; per block the MMAs take 512
// cycles (four 256x256x32 instructions at 8192 multiply-adds an SM and cycle),
// in which each SM's 8 promotion warps must read 128 x 256 values from Tensor
// Memory and do one (or, with scales per row of B, two) packed fp32 operations
// for every two of them: 128 or 256 issue cycles of the 512 a scheduler has.
// Two accumulators of 256 columns fill Tensor Memory and let block c + 1's MMAs
// run while block c is promoted.
//
// Roles per CTA (384 threads): warp 0 TMA producer; warp 1 Tensor Memory and,
// in the leader, MMA issue; warp 2 brings the scales into a ring of their own
// (plain loads: any strides); warps 4-11 promotion, 128 sums per thread, which
// take over registers from warps 0-3.  Warps 4-11 read Tensor Memory in the
// 16x256b shape: a quad of lanes holds 8 consecutive columns of a row, so a
// thread needs 4 row scales and, for scales per row of B, 32 column scales
// instead of 128, and Out leaves in row segments.
// Synchronisation:
//   full[s], empty[s]    operand ring, as in the unscaled pair kernel
//   tfull[b], tempty[b]  accumulators: leader's commit to both CTAs / one
//                        arrival per promotion warp of both, at the leader
//   sfull[r], sempty[r]  scale ring, within the CTA
// Every wait is bounded.
#include <algorithm>

#include "block128_tc.cuh"

namespace gnt {

namespace {

using namespace blk;
using tc::BM;

constexpr int kTile = 256;                  // rows and columns of a pair's tile
constexpr int kStages = 6;
constexpr int kOpBytes = BM * kRowBytes;    // one CTA's half of A, and of B
constexpr int kScaleRing = 8;
constexpr int kScaleFloats = 128 + 256;     // rows' scales, columns' scales (or rows' times each column block's)
constexpr int kScaleBatch = 4;              // K blocks whose scale loads are in flight together
constexpr int kTmemCols = 512;
constexpr int kBarBytes = 512;
constexpr int kSmem = 1024 + kStages * 2 * kOpBytes + kScaleRing * kScaleFloats * 4 + kBarBytes;
static_assert(kSmem <= 232448, "shared memory budget");

// Tile t of this pair's walk -> batch and tile origin; tiles go down groups of
// group_m row tiles, column by column, so that pairs at work share operands in L2.
__device__ __forceinline__ void decode(const BlkParams& p, int t, int& b, int& m0, int& n0)
{
    const int per = p.tiles_m * p.tiles_n;
    b = t / per;
    t -= b * per;
    const int g = t / (p.group_m * p.tiles_n), first = g * p.group_m;
    const int gm = min(p.group_m, p.tiles_m - first), r = t - g * p.group_m * p.tiles_n;
    m0 = (first + r % gm) * kTile;
    n0 = r / gm * kTile;
}

// 4 x 4 words across a quad of lanes: lane i ends with word i of lanes 0..3.
__device__ __forceinline__ void quad_transpose(uint32_t (&v)[4], int lane)
{
    const bool odd = lane & 1, high = lane & 2;
    const uint32_t a = __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[1], 1);
    const uint32_t b = __shfl_xor_sync(0xffffffffu, odd ? v[2] : v[3], 1);
    if (odd) {
        v[0] = a;
        v[2] = b;
    } else {
        v[1] = a;
        v[3] = b;
    }
    const uint32_t c = __shfl_xor_sync(0xffffffffu, high ? v[0] : v[2], 2);
    const uint32_t d = __shfl_xor_sync(0xffffffffu, high ? v[1] : v[3], 2);
    if (high) {
        v[0] = c;
        v[1] = d;
    } else {
        v[2] = c;
        v[3] = d;
    }
}

// Stores a promotion warp's 32 rows x 128 columns: acc[c][h][half][j] holds
// columns 32c + 8j + 2(lane % 4) + {0, 1} of row 16h + 8*half + lane / 4.
template <int OT>
__device__ __forceinline__ void store_tile(const BlkParams& p, const uint64_t (&acc)[4][2][2][4], int b, int row0,
                                           int col0, int lane)
{
    using S = OutStore<OT>;
    typename S::T* out = static_cast<typename S::T*>(p.out) + b * p.stride_o;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = row0 + 16 * h + 8 * half + (lane >> 2);
            typename S::T* d = out + static_cast<int64_t>(row) * p.ldo;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    unpack2(acc[c][h][half][j], v[2 * j], v[2 * j + 1]);
                if constexpr (OT != kOutF32) {
                    if (p.vec == 8) {  // 16-byte stores: each lane takes 8 consecutive columns
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = S::pack(v[2 * j], v[2 * j + 1]);
                        quad_transpose(w, lane);
                        const int col = col0 + 32 * c + 8 * (lane & 3);
                        if (row < p.M && col + 8 <= p.N) {
                            __stcs(reinterpret_cast<uint4*>(d + col), make_uint4(w[0], w[1], w[2], w[3]));
                        } else if (row < p.M) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (col + e < p.N)
                                    d[col + e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
                        }
                        continue;
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int col = col0 + 32 * c + 8 * j + 2 * (lane & 3);
                    if (row < p.M) {
                        if (p.vec >= 2 && col + 2 <= p.N) {
                            S::st2(d + col, v[2 * j], v[2 * j + 1]);
                        } else {
                            if (col < p.N)
                                S::st1(d + col, v[2 * j]);
                            if (col + 1 < p.N)
                                S::st1(d + col + 1, v[2 * j + 1]);
                        }
                    }
                }
            }
        }
}

// BROW: a scale for each row of B (each column of the tile), else one for each
// 128 of them.
template <bool BROW>
__global__ void __launch_bounds__(kThreads, 1)
    block128_pair_kernel(const __grid_constant__ CUtensorMap tma, const __grid_constant__ CUtensorMap tmb,
                         const BlkParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* as = smem;
    uint8_t* bs = smem + kStages * kOpBytes;
    float* scales = reinterpret_cast<float*>(smem + 2 * kStages * kOpBytes);
    uint64_t* full = reinterpret_cast<uint64_t*>(scales + kScaleRing * kScaleFloats);
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* sfull = tempty + 2;
    uint64_t* sempty = sfull + kScaleRing;
    uint64_t* drain = sempty + kScaleRing;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((2 * kStages + 4 + 2 * kScaleRing + 1) * 8 + 8 <= kBarBytes, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&tfull[b]), 1);
            mbar_init(smem_u32(&tempty[b]), 2 * kPromoWarps);
        }
        for (int r = 0; r < kScaleRing; ++r) {
            mbar_init(smem_u32(&sfull[r]), 32);
            mbar_init(smem_u32(&sempty[r]), kPromoWarps);
        }
        mbar_init(smem_u32(drain), 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_map(&tma);
        tma_prefetch_map(&tmb);
    }
    if (warp == 1) {
        tmem_alloc_pair<kTmemCols>(smem_u32(tmem_slot));
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_launch_dependents();
    pdl_wait();  // global memory only after the preceding grids are done

    if (warp < 4) {
        regs_utility();
        if (warp == 0 && lane == 0) {
            // -------------------------------------------------------- producer (both CTAs)
            int stage = 0;
            uint32_t phase = 0, filled = 0, fill_parity = 0;
            bool ok = true, drop = p.fault == 1 && blockIdx.x == 0;
            for (int t = pair; ok && t < p.num_tiles; t += pairs) {
                int b, m0, n0;
                decode(p, t, b, m0, n0);
                const int xa = m0 + static_cast<int>(rank) * BM, xb = n0 + static_cast<int>(rank) * BM;
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!wait_bounded(smem_u32(&empty[stage]), phase ^ 1, abort_flag, p.wait_limit)) {
                        raise(p, abort_flag);
                        ok = false;
                        break;
                    }
                    if (!drop) {
                        const uint32_t fb = smem_u32(&full[stage]), fb_leader = mapa_shared(fb, 0);
                        if (leader) {
                            mbar_arrive_expect_tx(fb, 4 * kOpBytes);
                            filled |= 1u << stage;
                            fill_parity = (fill_parity & ~(1u << stage)) | (phase << stage);
                        }
                        tma_load_3d_pair(smem_u32(as + stage * kOpBytes), &tma, fb_leader, kb * kRowBytes, xa, b * p.a_bmul);
                        tma_load_3d_pair(smem_u32(bs + stage * kOpBytes), &tmb, fb_leader, kb * kRowBytes, xb, b * p.b_bmul);
                    }
                    drop = false;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // every load of the pair lands before either CTA leaves
            for (int s = 0; s < kStages; ++s)
                if (filled & (1u << s))
                    drain_wait(smem_u32(&full[s]), (fill_parity >> s) & 1u, p.wait_limit);
        } else if (warp == 1 && lane == 0 && leader) {
            // -------------------------------------------------------- MMA issue (leader)
            const uint32_t idesc = idesc_f16_f32(kTile, kTile) | p.idesc_bits;
            const DescWords da = desc_words(smem_u32(as), false), db = desc_words(smem_u32(bs), false);
            int stage = 0, buf = 0;
            uint32_t phase = 0, tphase = 0;
            bool ok = true, skip_release = p.fault == 2 && blockIdx.x == 0;
            for (int t = pair; ok && t < p.num_tiles; t += pairs) {
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!wait_bounded(smem_u32(&tempty[buf]), tphase ^ 1, abort_flag, p.wait_limit) ||
                        !wait_bounded(smem_u32(&full[stage]), phase, abort_flag, p.wait_limit)) {
                        raise(p, abort_flag);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem_base + static_cast<uint32_t>(buf * kTile);
                    const uint32_t alo = da.lo + stage * (kOpBytes >> 4), blo = db.lo + stage * (kOpBytes >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_pair_w<true>(d, alo + k * da.kstep, da.hi, blo + k * db.kstep, db.hi, idesc, k > 0);
                    if (!skip_release)
                        tc_commit_pair_mc(smem_u32(&empty[stage]), 0x3);
                    skip_release = false;
                    tc_commit_pair_mc(smem_u32(&tfull[buf]), 0x3);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                    buf ^= 1;
                    tphase ^= buf == 0;
                }
            }
            // no MMA may still be running when Tensor Memory is released
            tc_commit_pair(smem_u32(drain));
            drain_wait(smem_u32(drain), 0, p.wait_limit);
        } else if (warp == 2) {
            // -------------------------------------------------------- scales (each CTA its rows)
            // Rows and columns outside Out multiply zeros and are not stored;
            // they take the last row's scale.  The loads of kScaleBatch K blocks
            // are in flight together.
            constexpr int NB = BROW ? 8 : 2;
            int slot = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = pair; ok && t < p.num_tiles; t += pairs) {
                int b, m0, n0;
                decode(p, t, b, m0, n0);
                m0 += static_cast<int>(rank) * BM;
                for (int kb0 = 0; ok && kb0 < p.num_kb; kb0 += kScaleBatch) {
                    float va[kScaleBatch][4], vb[kScaleBatch][NB];
#pragma unroll
                    for (int i = 0; i < kScaleBatch; ++i) {
                        const int kb = min(kb0 + i, p.num_kb - 1);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            va[i][r] = scale_at(p.sa, b, min(m0 + 32 * r + lane, p.M - 1), kb);
#pragma unroll
                        for (int r = 0; r < NB; ++r)
                            vb[i][r] = scale_at(p.sb, b, min(BROW ? n0 + 32 * r + lane : n0 + 128 * r, p.N - 1), kb);
                    }
#pragma unroll
                    for (int i = 0; i < kScaleBatch; ++i) {
                        if (ok && kb0 + i < p.num_kb) {
                            if (!wait_bounded(smem_u32(&sempty[slot]), phase ^ 1, abort_flag, p.wait_limit)) {
                                raise(p, abort_flag);
                                ok = false;
                            } else {
                                float* s = scales + slot * kScaleFloats;
#pragma unroll
                                for (int r = 0; r < 4; ++r) {
                                    if (BROW) {
                                        s[32 * r + lane] = va[i][r];
                                    } else {
                                        s[128 + 32 * r + lane] = va[i][r] * vb[i][0];
                                        s[256 + 32 * r + lane] = va[i][r] * vb[i][1];
                                    }
                                }
                                if (BROW) {
#pragma unroll
                                    for (int r = 0; r < NB; ++r)
                                        s[128 + 32 * r + lane] = vb[i][r];
                                }
                                mbar_arrive(smem_u32(&sfull[slot]));
                                if (++slot == kScaleRing) {
                                    slot = 0;
                                    phase ^= 1;
                                }
                            }
                        }
                    }
                }
            }
        }
    } else {
        // ------------------------------------------------------------ promotion (both CTAs)
        regs_promotion();
        const int q = warp & 3, ch = (warp - 4) >> 2;  // lane quadrant, column half
        int slot = 0, buf = 0;
        uint32_t sphase = 0, tphase = 0;
        bool ok = true;
        for (int t = pair; ok && t < p.num_tiles; t += pairs) {
            uint64_t acc[4][2][2][4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int v = 0; v < 2; ++v)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[c][h][v][j] = 0;
            for (int kb = 0; kb < p.num_kb; ++kb) {
                if (!wait_bounded(smem_u32(&sfull[slot]), sphase, abort_flag, p.wait_limit)) {
                    raise(p, abort_flag);
                    ok = false;
                    break;
                }
                const float* s = scales + slot * kScaleFloats;
                uint64_t sr[2][2];  // the thread's 4 rows' scales, twice each
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const float f = s[(BROW ? 0 : 128 + 128 * ch) + 32 * q + 16 * h + 8 * v + (lane >> 2)];
                        sr[h][v] = pack2(f, f);
                    }
                const uint64_t* sc = reinterpret_cast<const uint64_t*>(s + 128 + 128 * ch) + (lane & 3);
                if (!wait_bounded(smem_u32(&tfull[buf]), tphase, abort_flag, p.wait_limit)) {
                    raise(p, abort_flag);
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t ta = tmem_base + static_cast<uint32_t>(buf * kTile + 128 * ch) +
                                    (static_cast<uint32_t>(32 * q) << 16);
                // the next 16 x 32 chunk's load runs under the arithmetic of this one
                uint32_t x[2][16];
                tmem_ld16x256_x4(ta, x[0]);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int c = u >> 1, h = u & 1;
                    tmem_wait(x[u & 1]);
                    if (u < 7) {
                        tmem_ld16x256_x4(ta + 32 * ((u + 1) >> 1) + (((u + 1) & 1) ? 16u << 16 : 0u), x[(u + 1) & 1]);
                    } else {
                        // the accumulator is in registers: free it for block kb + 2
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[buf]), 0));
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint64_t cs = BROW ? sc[16 * c + 4 * j] : 0;
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            uint64_t part = pack2u(x[u & 1][4 * j + 2 * v], x[u & 1][4 * j + 2 * v + 1]);
                            if (BROW)
                                part = mul2(part, cs);
                            acc[c][h][v][j] = fma2(part, sr[h][v], acc[c][h][v][j]);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sempty[slot]));
                if (++slot == kScaleRing) {
                    slot = 0;
                    sphase ^= 1;
                }
                buf ^= 1;
                tphase ^= buf == 0;
            }
            if (!ok)
                break;
            int b, m0, n0;
            decode(p, t, b, m0, n0);
            const int row0 = m0 + static_cast<int>(rank) * BM + 32 * q, col0 = n0 + 128 * ch;
            if (p.out_type == kOutF16)
                store_tile<kOutF16>(p, acc, b, row0, col0, lane);
            else if (p.out_type == kOutBF16)
                store_tile<kOutBF16>(p, acc, b, row0, col0, lane);
            else
                store_tile<kOutF32>(p, acc, b, row0, col0, lane);
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no CTA leaves while its peer may still touch its memory
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair<kTmemCols>(tmem_base);
    }
}

cudaLaunchConfig_t pair_config(int pairs, cudaStream_t stream, cudaLaunchAttribute* attr)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

template <bool BROW>
cudaError_t configure(int* max_pairs)
{
    cudaError_t e = cudaFuncSetAttribute(block128_pair_kernel<BROW>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = pair_config(1, nullptr, attr);
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, block128_pair_kernel<BROW>, &cfg);
    *max_pairs = std::min(*max_pairs, n);
    return e;
}

}  // namespace

cudaError_t block128_pair_configure(int* max_pairs)
{
    int n = 1 << 30;
    cudaError_t e = configure<false>(&n);
    if (e == cudaSuccess)
        e = configure<true>(&n);
    *max_pairs = n;
    return e;
}

cudaError_t block128_pair_launch(const BlkParams& prm, int max_pairs, cudaStream_t stream)
{
    BlkParams p = prm;
    CUtensorMap tma, tmb;
    const int type = p.e5m2 ? 4 : 3;  // gemm_dtype_t
    if (!operand_map(&tma, p.A, p.M, p.K, p.lda, p.batch, p.stride_a, BM, &p.a_bmul, type) ||
        !operand_map(&tmb, p.B, p.N, p.K, p.ldb, p.batch, p.stride_b, BM, &p.b_bmul, type))
        return cudaErrorInvalidValue;
    p.tiles_m = (p.M + kTile - 1) / kTile;
    p.tiles_n = (p.N + kTile - 1) / kTile;
    p.num_tiles = p.tiles_m * p.tiles_n * p.batch;
    p.group_m = 8;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = pair_config(std::min(p.num_tiles, max_pairs), stream, attr);
    return p.sb.shift ? cudaLaunchKernelEx(&cfg, block128_pair_kernel<false>, tma, tmb, p)
                      : cudaLaunchKernelEx(&cfg, block128_pair_kernel<true>, tma, tmb, p);
}

}  // namespace gnt
