// block128_swap.cu -- block-scaled 8-bit product on single CTAs (tcgen05), for
// few rows of A or few tiles.
//
// The operands are swapped: 128 rows of B (weights) are the MMA's row side and
// BN = 16, 32, 64 or 128 rows of A its column side, so a decode batch pays for
// no padding beyond its next power of two.  Bound by reading B once: a K block
// brings 16 KB of B a tile, 700 cycles at an SM's share of memory bandwidth,
// against 64 cycles of MMA at BN = 32.  What matters is bytes in flight, hence a
// ring of up to 200 KB, and enough CTAs: with fewer tiles than SMs a cluster of
// up to 8 CTAs splits K of one tile and adds its sums through distributed
// shared memory, in CTA order, so the result never depends on timing.
//
// As in the pair kernel each K block is a fresh accumulator (four of them in
// Tensor Memory) that promotion warps scale and add to sums in registers; here
// a thread holds one row of B (32x32b loads) and half of the columns, its row's
// scale in a register and the columns' scales broadcast from shared memory.  The
// row's goes first; where it is tiny or huge (a vote per K block) each product's order
// is chosen by itself.
//
// Measured: 64 x 16384 x 8192 25.5 us (5.5 TB/s; one wave of 152 CTAs with even row
// shares; 27.5 with one warp issuing the MMAs), 1 x 4096 x 4096 7.2 us, of which the
// 16.8 MB take 2.5: launch, the first loads and the cluster's exchange are the rest.
#include <algorithm>

#include "block128_tc.cuh"

namespace gnt {

namespace {

using namespace blk;
using tc::BM;

constexpr int kThreads = 384;   // warps 0-3: producer, MMA, scales, MMA; warps 4-11: promotion
constexpr int kPromoWarps = 8;
constexpr int kAcc = 4;         // accumulators in Tensor Memory
constexpr int kScaleRing = 4;   // slots of kScaleGroup K blocks
constexpr int kScaleGroup = 4;
constexpr int kMaxCluster = 8;

constexpr int max_int(int a, int b) { return a > b ? a : b; }
constexpr int min_int(int a, int b) { return a < b ? a : b; }

template <int BN>
struct Cfg {
    static constexpr int X_BYTES = BM * kRowBytes, Y_BYTES = BN * kRowBytes;
    static constexpr int STAGE = X_BYTES + Y_BYTES;
    static constexpr int SCALE_FLOATS = 128 + max_int(32, BN);
    static constexpr int BAR_BYTES = 512;
    static constexpr int REST = 1024 + kScaleRing * kScaleGroup * SCALE_FLOATS * 4 + BAR_BYTES;
    static constexpr int STAGES = min_int(12, (232448 - REST) / STAGE);
    static constexpr int SMEM = REST + STAGES * STAGE;
    static constexpr int TMEM_COLS = max_int(32, kAcc * BN);
    static constexpr int COLS = BN / 2;  // columns of a promotion thread
    static_assert(BM * BN * 4 <= STAGES * STAGE, "a tile's sums fit in the ring");
    static_assert((2 * STAGES + 2 * kAcc + 2 * kScaleRing + 2) * 8 + 8 <= BAR_BYTES, "barrier area");
    static_assert(STAGES > 2 && kAcc % 2 == 0, "two warps take turns");
};

__device__ __forceinline__ float ld_cluster(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Tiles: rows of B first, so that neighbours share A.  With p.row_share each CTA
// has one tile, an even share of B's rows (at most 128) that starts anywhere.
__device__ __forceinline__ void decode(const BlkParams& p, int t, int bn, int& b, int& x0, int& xend, int& y0)
{
    if (p.row_share) {
        b = y0 = 0;
        x0 = static_cast<int>(static_cast<int64_t>(p.N) * t / p.num_tiles);
        xend = static_cast<int>(static_cast<int64_t>(p.N) * (t + 1) / p.num_tiles);
        return;
    }
    const int per = p.tiles_m * p.tiles_n;
    b = t / per;
    t -= b * per;
    y0 = t / p.tiles_n * bn;
    x0 = t % p.tiles_n * BM;
    xend = x0 + min(BM, p.N - x0);
}

template <int BN>
__global__ void __launch_bounds__(kThreads, 1)
    block128_swap_kernel(const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tmy,
                         const BlkParams p, int cluster)
{
    using C = Cfg<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* xs = smem;
    uint8_t* ys = smem + C::STAGES * C::X_BYTES;
    float* scales = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE);
    uint64_t* full = reinterpret_cast<uint64_t*>(scales + kScaleRing * kScaleGroup * C::SCALE_FLOATS);
    uint64_t* empty = full + C::STAGES;
    uint64_t* tfull = empty + C::STAGES;
    uint64_t* tempty = tfull + kAcc;
    uint64_t* sfull = tempty + kAcc;
    uint64_t* sempty = sfull + kScaleRing;
    uint64_t* drain = sempty + kScaleRing;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x) % cluster;
    const int first = static_cast<int>(blockIdx.x) / cluster, step = static_cast<int>(gridDim.x) / cluster;
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.num_kb) * rank / cluster);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.num_kb) * (rank + 1) / cluster);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int b = 0; b < kAcc; ++b) {
            mbar_init(smem_u32(&tfull[b]), 1);
            mbar_init(smem_u32(&tempty[b]), kPromoWarps);
        }
        for (int r = 0; r < kScaleRing; ++r) {
            mbar_init(smem_u32(&sfull[r]), 32);
            mbar_init(smem_u32(&sempty[r]), kPromoWarps);
        }
        mbar_init(smem_u32(&drain[0]), 1);
        mbar_init(smem_u32(&drain[1]), 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_map(&tmx);
        tma_prefetch_map(&tmy);
    }
    if (warp == 1) {
        tmem_alloc<C::TMEM_COLS>(smem_u32(tmem_slot));
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_launch_dependents();
    pdl_wait();  // global memory only after the preceding grids are done

    uint64_t acc[C::COLS / 2];  // promotion threads: pairs of columns
#pragma unroll
    for (int j = 0; j < C::COLS / 2; ++j)
        acc[j] = 0;
    const int q = warp & 3, ch = (warp - 4) >> 2;  // promotion: lane quadrant, column half

    if (warp == 0) {
        if (lane == 0) {
            // -------------------------------------------------------- producer
            int stage = 0;
            uint32_t phase = 0, filled = 0, fill_parity = 0;
            // B is read once, A by every tile row: keep A in L2 under the stream
            const uint64_t pol_x = l2_policy_evict_first(), pol_y = l2_policy_evict_last();
            bool ok = true, drop = p.fault == 1 && blockIdx.x == 0;
            for (int t = first; ok && t < p.num_tiles; t += step) {
                int b, x0, xend, y0;
                decode(p, t, BN, b, x0, xend, y0);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!wait_bounded(smem_u32(&empty[stage]), phase ^ 1, abort_flag, p.wait_limit)) {
                        raise(p, abort_flag);
                        ok = false;
                        break;
                    }
                    if (!drop) {
                        const uint32_t fb = smem_u32(&full[stage]);
                        mbar_arrive_expect_tx(fb, static_cast<uint32_t>(p.x_box * kRowBytes + C::Y_BYTES));
                        filled |= 1u << stage;
                        fill_parity = (fill_parity & ~(1u << stage)) | (phase << stage);
                        tma_load_3d_hint(smem_u32(xs + stage * C::X_BYTES), &tmx, fb, kb * kRowBytes, x0, b * p.b_bmul, pol_x);
                        tma_load_3d_hint(smem_u32(ys + stage * C::Y_BYTES), &tmy, fb, kb * kRowBytes, y0, b * p.a_bmul, pol_y);
                    }
                    drop = false;
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            for (int s = 0; s < C::STAGES; ++s)
                if (filled & (1u << s))
                    drain_wait(smem_u32(&full[s]), (fill_parity >> s) & 1u, p.wait_limit);
        }
    } else if (warp == 1 || warp == 3) {
        // ------------------------------------------------------------ MMA issue
        // As in the pair kernel: one warp for the even K blocks and one for the odd ones,
        // each paying its waits and commits while the other's MMAs run.
        const int par = warp >> 1;
        const uint32_t idesc = idesc_f16_f32(BM, BN) | p.idesc_bits;
        const DescWords dx = desc_words(smem_u32(xs), false), dy = desc_words(smem_u32(ys), false);
        const int blocks = (p.num_tiles - first + step - 1) / step * (kb1 - kb0);
        int stage = par, buf = par;
        uint32_t phase = 0, tphase = 0;
        bool skip_release = p.fault == 2 && blockIdx.x == 0 && par == 0;
        const bool chosen = elect_one();
#pragma unroll 1
        for (int n = par; n < blocks; n += 2) {
            const uint32_t fa = smem_u32(&full[stage]), te = smem_u32(&tempty[buf]);
            // even lanes: the accumulator is free; odd lanes: the operands are here
            if (!wait_lanes(lane & 1 ? fa : te, lane & 1 ? phase : tphase ^ 1, abort_flag, p.wait_limit)) {
                raise(p, abort_flag);
                break;
            }
            tc_fence_after();
            if (chosen) {
                const uint32_t d = tmem_base + static_cast<uint32_t>(buf * BN);
                const uint32_t xlo = dx.lo + stage * (C::X_BYTES >> 4), ylo = dy.lo + stage * (C::Y_BYTES >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc_mma_w<true>(d, xlo + k * dx.kstep, dx.hi, ylo + k * dy.kstep, dy.hi, idesc, k > 0);
                tc_commit(smem_u32(&tfull[buf]));
                if (!skip_release)
                    tc_commit(smem_u32(&empty[stage]));
            }
            __syncwarp();
            skip_release = false;
            stage += 2;
            if (stage >= C::STAGES) {
                stage -= C::STAGES;
                phase ^= 1;
            }
            buf += 2;
            if (buf >= kAcc) {
                buf -= kAcc;
                tphase ^= 1;
            }
        }
        // no MMA may still be running when Tensor Memory is released
        if (chosen) {
            tc_commit(smem_u32(&drain[par]));
            drain_wait(smem_u32(&drain[par]), 0, p.wait_limit);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ scales: 128 rows of B, BN rows of A
        const uint32_t ring = smem_u32(scales);
        int n = 0;  // K blocks so far
        bool ok = true;
        for (int t = first; ok && t < p.num_tiles; t += step) {
            int b, x0, xend, y0;
            decode(p, t, BN, b, x0, xend, y0);
            ScaleRun<4> x(p.sb, b, x0, p.N);
            ScaleRun<(BN + 31) / 32> y(p.sa, b, y0, p.M);
            x.skip(kb0);
            y.skip(kb0);
#pragma unroll 1
            for (int kb = kb0; kb < kb1; ++kb, ++n) {
                const int slot = n / kScaleGroup % kScaleRing;
                if (n % kScaleGroup == 0 && !wait_bounded(smem_u32(&sempty[slot]), (n / (kScaleGroup * kScaleRing) & 1) ^ 1,
                                                          abort_flag, p.wait_limit)) {
                    raise(p, abort_flag);
                    ok = false;
                    break;
                }
                const uint32_t s = ring + n % (kScaleGroup * kScaleRing) * (C::SCALE_FLOATS * 4);
                x.copy(s);
                y.copy(s + 128 * 4);
                if (n % kScaleGroup == kScaleGroup - 1)
                    cp_async_arrive(smem_u32(&sfull[slot]));
            }
        }
        if (n % kScaleGroup != 0)  // the last group, short
            cp_async_arrive(smem_u32(&sfull[n / kScaleGroup % kScaleRing]));
        cp_async_wait_all();
    } else if (warp >= 4) {
        // ------------------------------------------------------------ promotion
        const uint32_t row_scale = smem_u32(scales) + (32 * q + lane) * 4;
        const uint32_t col_scales = smem_u32(scales) + (128 + C::COLS * ch) * 4;
        const uint32_t tf0 = smem_u32(tfull), te0 = smem_u32(tempty), sf0 = smem_u32(sfull);
        const uint32_t ta0 = tmem_base + static_cast<uint32_t>(C::COLS * ch) + (static_cast<uint32_t>(32 * q) << 16);
        const uint32_t from = plain_from(p.e5m2);
        int n = 0;  // K blocks so far: ring positions and phases follow from it
        bool ok = true;
        for (int t = first; ok && t < p.num_tiles; t += step) {
#pragma unroll 1
            for (int kb = kb0; kb < kb1; ++kb, ++n) {
                if (n % kScaleGroup == 0)
                    ok &= wait_bounded(sf0 + n / kScaleGroup % kScaleRing * 8, n / (kScaleGroup * kScaleRing) & 1, abort_flag,
                                       p.wait_limit);
                const uint32_t so = n % (kScaleGroup * kScaleRing) * (C::SCALE_FLOATS * 4);
                const float fx = lds_f32(row_scale + so);
                ok &= wait_bounded(tf0 + n % kAcc * 8, n / kAcc & 1, abort_flag, p.wait_limit);
                if (!ok) {
                    raise(p, abort_flag);
                    break;
                }
                tc_fence_after();
                uint32_t x[C::COLS];
#pragma unroll
                for (int c = 0; c < C::COLS; c += 8)
                    tmem_ld32x8(ta0 + n % kAcc * BN + c, x + c);
#pragma unroll
                for (int c = 0; c < C::COLS; c += 8)
                    tmem_wait8(x + c);
                tc_fence_before();
                mbar_arrive_if(te0 + n % kAcc * 8, lane == 0);
                if (__any_sync(0xffffffffu, !plain_scale(fx, from)) && any_set(x)) {
                    add_careful(acc, x, fx, col_scales + so);
                } else {
                    const uint64_t sx = pack2(fx, fx);
#pragma unroll
                    for (int j = 0; j < C::COLS / 4; ++j) {
                        const ulonglong2 w = lds_f32x4(col_scales + so + 16 * j);
                        acc[2 * j] = fma2(mul2(pack2u(x[4 * j], x[4 * j + 1]), sx), w.x, acc[2 * j]);
                        acc[2 * j + 1] = fma2(mul2(pack2u(x[4 * j + 2], x[4 * j + 3]), sx), w.y, acc[2 * j + 1]);
                    }
                }
                if (n % kScaleGroup == kScaleGroup - 1) {
                    __syncwarp();
                    mbar_arrive_if(smem_u32(&sempty[n / kScaleGroup % kScaleRing]), lane == 0);
                }
            }
            if (!ok || cluster > 1)
                break;  // a cluster has one tile, finished below
            int b, x0, xend, y0;
            decode(p, t, BN, b, x0, xend, y0);
            const int x = x0 + 32 * q + lane, y = y0 + C::COLS * ch;
            const auto store = [&](auto ot) {
                using S = OutStore<decltype(ot)::value>;
                typename S::T* d = static_cast<typename S::T*>(p.out) + b * p.stride_o + static_cast<int64_t>(y) * p.ldo + x;
#pragma unroll
                for (int j = 0; j < C::COLS; j += 2) {
                    float v0, v1;
                    unpack2(acc[j / 2], v0, v1);
                    acc[j / 2] = 0;
                    if (x < xend) {
                        if (y + j < p.M)
                            S::st1(d, v0);
                        if (y + j + 1 < p.M)
                            S::st1(d + p.ldo, v1);
                    }
                    d += 2 * p.ldo;
                }
            };
            if (p.out_type == kOutF16)
                store(std::integral_constant<int, kOutF16>());
            else if (p.out_type == kOutBF16)
                store(std::integral_constant<int, kOutBF16>());
            else
                store(std::integral_constant<int, kOutF32>());
        }
        if (cluster > 1) {
            // Every MMA has read its operands (the last accumulator is here), so the
            // ring can take the sums: column j of the tile at [j][row].
            float* d = reinterpret_cast<float*>(smem) + C::COLS * ch * BM + 32 * q + lane;
#pragma unroll
            for (int j = 0; j < C::COLS; j += 2) {
                float v0, v1;
                unpack2(acc[j / 2], v0, v1);
                d[j * BM] = v0;
                d[(j + 1) * BM] = v1;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (cluster > 1) {
        cluster_sync();
        int b, x0, xend, y0;
        decode(p, first, BN, b, x0, xend, y0);
        const int n = min(BN, p.M - y0) * BM;
        const int lo = static_cast<int>(static_cast<int64_t>(n) * rank / cluster);
        const int hi = static_cast<int>(static_cast<int64_t>(n) * (rank + 1) / cluster);
        const uint32_t base = smem_u32(smem);
        for (int i = lo + static_cast<int>(threadIdx.x); i < hi; i += kThreads) {
            float s = 0.f;
            for (int r = 0; r < cluster; ++r)
                s += ld_cluster(mapa_shared(base + 4 * i, r));
            const int x = x0 + i % BM, y = y0 + i / BM;
            if (x < xend) {
                const int64_t o = b * p.stride_o + static_cast<int64_t>(y) * p.ldo + x;
                if (p.out_type == kOutF16)
                    OutStore<kOutF16>::st1(static_cast<uint16_t*>(p.out) + o, s);
                else if (p.out_type == kOutBF16)
                    OutStore<kOutBF16>::st1(static_cast<uint16_t*>(p.out) + o, s);
                else
                    OutStore<kOutF32>::st1(static_cast<float*>(p.out) + o, s);
            }
        }
        cluster_sync();  // no CTA leaves while another may still read its sums
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<C::TMEM_COLS>(tmem_base);
    }
}

template <int BN>
cudaError_t launch(BlkParams p, int num_sms, cudaStream_t stream)
{
    CUtensorMap tmx, tmy;
    const int type = p.e5m2 ? 4 : 3;  // gemm_dtype_t
    // One wave of shares of 64 to 128 rows, with boxes just as tall (the MMA's other
    // rows hold what a slot last held and are not stored): 64 x 16384 x 8192 on all
    // SMs instead of 128 of them, 64 x 18000 x 8192 28.4 us.  Above 128 rows an SM whole
    // tiles take two rounds: 48.5 to 50 us from 20000 to 32768 rows.
    p.row_share = p.batch == 1 && p.M <= BN && p.N >= 64 * num_sms && p.N <= 128 * num_sms;
    p.x_box = p.row_share ? std::min(BM, ((p.N + num_sms - 1) / num_sms + 7) / 8 * 8) : BM;
    if (!operand_map(&tmx, p.B, p.N, p.K, p.ldb, p.batch, p.stride_b, p.x_box, &p.b_bmul, type) ||
        !operand_map(&tmy, p.A, p.M, p.K, p.lda, p.batch, p.stride_a, BN, &p.a_bmul, type))
        return cudaErrorInvalidValue;
    p.tiles_m = (p.M - 1) / BN + 1;
    p.tiles_n = (p.N - 1) / BM + 1;
    p.num_tiles = p.row_share ? num_sms : p.tiles_m * p.tiles_n * p.batch;
    // split K while whole clusters still fit the GPU and a CTA keeps 4 K blocks
    int c = 1;
    while (c < kMaxCluster && p.num_tiles * 2 * c <= num_sms && p.num_kb >= 8 * c)
        c *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(c > 1 ? p.num_tiles * c : std::min(p.num_tiles, num_sms)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<BN>::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(c);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, block128_swap_kernel<BN>, tmx, tmy, p, c);
}

template <int BN>
cudaError_t configure()
{
    return cudaFuncSetAttribute(block128_swap_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<BN>::SMEM);
}

}  // namespace

cudaError_t block128_swap_configure()
{
    cudaError_t e = configure<16>();
    if (e == cudaSuccess) e = configure<32>();
    if (e == cudaSuccess) e = configure<64>();
    if (e == cudaSuccess) e = configure<128>();
    return e;
}

cudaError_t block128_swap_launch(const BlkParams& p, int num_sms, cudaStream_t stream)
{
    if (p.M <= 16)
        return launch<16>(p, num_sms, stream);
    if (p.M <= 32)
        return launch<32>(p, num_sms, stream);
    if (p.M <= 64)
        return launch<64>(p, num_sms, stream);
    return launch<128>(p, num_sms, stream);
}

}  // namespace gnt
