// gated_pair.cu -- the gated product h = act(x Wg^T) (x Wu^T) on CTA pairs
// (tcgen05 cta_group::2).
//
// A pair owns 256 tokens by 128 columns of h.  CTA r stages its 128 tokens and,
// as its half of the MMA's 256 rows of B, 128 rows of projection r: CTA 0 those
// of the gate, CTA 1 the same rows of the up projection (W13 is described to
// TMA as two matrices, so a tile at the end of the gate reads zeros and not
// up rows).  The 256-column accumulator of either CTA then holds, for its
// tokens, g in columns 0-127 and u of the same outputs in columns 128-255, and a
// thread that reads a column of each computes h in registers: g and u go to
// memory only when they are kept.
//
// Bound by the tensor cores: 4 tokens x hidden x inner flop, and two
// accumulators let a tile's epilogue run under the next one's MMAs.  8192 x 4096 x
// 8192 bf16 with g and u kept: 548 us in a burst (2.0 PFLOP/s), 628-645 back to back at
// the power cap (1.7); 661 when one thread walked the issue loop.  Full rows are stored as
// whole 32-byte sectors straight from registers, since a thread holds 64 consecutive
// bytes of its token; rows off 16-byte boundaries (u's, of an odd width) go through shared
// memory.
//
// Roles per CTA (320 threads): warp 0 TMA producer, warp 1 TMEM allocation and
// (CTA 0) MMA issue, warps 2-9 epilogue; barriers as in tc05_pair.cu.  Every
// wait is bounded.
#include <algorithm>

#include "block128_tc.cuh"
#include "ffn.h"
#include "gemm_nt.h"

namespace gnt {

namespace {

using namespace tc;

constexpr int kThreads = 320;
constexpr int kStages = 6;
constexpr int kCols = 128;                    // columns of h per tile
constexpr int kOpBytes = 128 * BK * 2;        // one operand's share of a stage
constexpr int kStageBytes = 2 * kOpBytes;
constexpr int kTmemCols = 512;                // two accumulators
constexpr int kStagePitch = 34;               // 16-bit elements per staged row: 17 words, no bank conflicts
constexpr int kWarpStage = 32 * kStagePitch;  // elements per epilogue warp
constexpr int kSmem = 1024 + kStages * kStageBytes + 8 * kWarpStage * 2 + 256;
static_assert(kSmem <= 232448, "shared memory budget");

struct PairParams {
    void* out;
    int64_t ldo;
    void* gu;  // null: not kept
    int64_t ldgu;
    int tokens, n;
    int tiles_x, tiles_y, num_tiles, num_kb, group_x;
    int bf16;
    int vec_h, vec_g, vec_u;  // rows allow stores of 16 elements (32 bytes), 8, or 1
    uint32_t idesc;
    uint32_t* status;
    unsigned long long wait_limit;
    int fault;
};

__device__ __forceinline__ void tile_at(const PairParams& p, int t, int& tx, int& ty)
{
    const int span = p.group_x * p.tiles_y;
    const int g = t / span, first = g * p.group_x;
    const int gx = min(p.tiles_x - first, p.group_x);
    const int r = t - g * span;
    tx = first + r % gx;
    ty = r / gx;
}

__device__ __forceinline__ uint32_t pack16(float a, float b, bool bf16)
{
    return bf16 ? OutStore<kOutBF16>::pack(a, b) : OutStore<kOutF16>::pack(a, b);
}

__device__ __forceinline__ void st_global_32(void* dst, const uint32_t* w)
{
    asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// 32 consecutive elements (as 16 words) of this lane's row, columns col..col+31
// of `cols`.  vec 16 or 8: whole sectors or half ones straight from registers
// (a row per lane); 1, or a tile's ragged end: through the warp's staging area, so
// that a warp stores 64 consecutive bytes of one row at a time.
__device__ __forceinline__ void store32(uint16_t* base, int64_t ld, int64_t row0, int nrows, int col, int cols,
                                        const uint32_t (&w)[16], int vec, int lane, uint16_t* stage)
{
    if (vec > 1 && col + 32 <= cols) {
        if (lane < nrows) {
            uint16_t* dst = base + (row0 + lane) * ld + col;
            if (vec == 16) {
                st_global_32(dst, w);
                st_global_32(dst + 16, w + 8);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    __stcs(reinterpret_cast<uint4*>(dst) + i, make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
            }
        }
        return;
    }
    uint32_t* mine = reinterpret_cast<uint32_t*>(stage + lane * kStagePitch);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        mine[i] = w[i];
    __syncwarp();
    if (col + lane < cols) {
        uint16_t* dst = base + row0 * ld + col + lane;
        for (int r = 0; r < nrows; ++r, dst += ld)
            *dst = stage[r * kStagePitch + lane];
    }
    __syncwarp();
}

template <int ACT>
__global__ void __launch_bounds__(kThreads, 1)
    gated_pair_kernel(const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tmw, const PairParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* as = smem;
    uint8_t* bs = smem + kStages * kOpBytes;
    uint16_t* staging = reinterpret_cast<uint16_t*>(smem + kStages * kStageBytes);
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + 8 * kWarpStage);
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&tfull[b]), 1);
            mbar_init(smem_u32(&tempty[b]), 2 * 8);  // the epilogue warps of both CTAs
        }
        mbar_init(smem_u32(drain), 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_map(&tmx);
        tma_prefetch_map(&tmw);
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
    pdl_wait();

    if (warp == 0) {
        // ------------------------------------------------------------ producer (both CTAs)
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, filled = 0, fill_parity = 0;
            bool first = true, ok = true;
            for (int t = pair; ok && t < p.num_tiles; t += pairs) {
                int tx, ty;
                tile_at(p, t, tx, ty);
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!wait_bounded(smem_u32(&empty[stage]), phase ^ 1, abort_flag, p.wait_limit)) {
                        *abort_flag = 1;
                        atomicOr(p.status, kStatusTimeout);
                        ok = false;
                        break;
                    }
                    const bool drop = p.fault == 1 && blockIdx.x == 0 && first;
                    first = false;
                    if (!drop) {
                        const uint32_t bar = smem_u32(&full[stage]);
                        if (leader) {
                            mbar_arrive_expect_tx(bar, 2 * kStageBytes);
                            filled |= 1u << stage;
                            fill_parity = (fill_parity & ~(1u << stage)) | (phase << stage);
                        }
                        const uint32_t lead = mapa_shared(bar, 0);
                        tma_load_3d_pair(smem_u32(as + stage * kOpBytes), &tmx, lead, kb * BK, tx * 256 + rank * 128, 0);
                        tma_load_3d_pair(smem_u32(bs + stage * kOpBytes), &tmw, lead, kb * BK, ty * kCols, rank);
                    }
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // the leader's barriers count both CTAs' bytes: every load lands before either exits
            for (int st = 0; st < kStages; ++st) {
                if (filled & (1u << st)) {
                    const long long t0 = clock64();
                    while (!mbar_try_wait(smem_u32(&full[st]), (fill_parity >> st) & 1u) &&
                           static_cast<unsigned long long>(clock64() - t0) <= p.wait_limit) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (leader)
        // The whole warp walks the loop and one lane issues, so that descriptors stay in
        // uniform registers.
        if (leader) {
            const bool one = blk::elect_one();
            const DescWords da = desc_words(smem_u32(as), false), db = desc_words(smem_u32(bs), false);
            int stage = 0, local = 0;
            uint32_t phase = 0;
            bool skip_release = p.fault == 2 && blockIdx.x == 0;  // test hook: lose one stage release
            bool ok = true;
            for (int t = pair; ok && t < p.num_tiles; t += pairs, ++local) {
                const int buf = local & 1;
                if (!blk::wait_lanes(smem_u32(&tempty[buf]), ((local >> 1) & 1) ^ 1, abort_flag, p.wait_limit)) {
                    *abort_flag = 1;
                    atomicOr(p.status, kStatusTimeout);
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + static_cast<uint32_t>(buf * 256);
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!blk::wait_lanes(smem_u32(&full[stage]), phase, abort_flag, p.wait_limit)) {
                        *abort_flag = 1;
                        atomicOr(p.status, kStatusTimeout);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t alo = da.lo + stage * (kOpBytes >> 4), blo = db.lo + stage * (kOpBytes >> 4);
                    if (one) {
#pragma unroll
                        for (int k = 0; k < BK / 16; ++k)
                            tc_mma_pair_w<false>(d, alo + k * da.kstep, da.hi, blo + k * db.kstep, db.hi, p.idesc,
                                                 (k > 0 || kb > 0) ? 1u : 0u);
                        if (!skip_release)
                            tc_commit_pair_mc(smem_u32(&empty[stage]), 0x3);
                    }
                    __syncwarp();
                    skip_release = false;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok)
                    break;
                if (one)
                    tc_commit_pair_mc(smem_u32(&tfull[buf]), 0x3);
                __syncwarp();
            }
            if (one)
                tc_commit_pair(smem_u32(drain));
            __syncwarp();
            const long long t0 = clock64();
            while (!mbar_try_wait(smem_u32(drain), 0) && static_cast<unsigned long long>(clock64() - t0) <= p.wait_limit) {
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue (both CTAs)
        const int ew = warp - 2, q = warp & 3, c0 = (ew >> 2) * (kCols / 2);
        uint16_t* stage_buf = staging + ew * kWarpStage;
        uint16_t* out = static_cast<uint16_t*>(p.out);
        uint16_t* gu = static_cast<uint16_t*>(p.gu);
        int local = 0;
        for (int t = pair; t < p.num_tiles; t += pairs, ++local) {
            int tx, ty;
            tile_at(p, t, tx, ty);
            const int buf = local & 1;
            if (!blk::wait_lanes(smem_u32(&tfull[buf]), (local >> 1) & 1, abort_flag, p.wait_limit)) {
                *abort_flag = 1;
                atomicOr(p.status, kStatusTimeout);
                break;
            }
            tc_fence_after();
            const uint32_t tacc = tmem_base + static_cast<uint32_t>(buf * 256) + (static_cast<uint32_t>(q * 32) << 16);
            const int64_t row0 = static_cast<int64_t>(tx) * 256 + rank * 128 + q * 32;
            const int nrows = static_cast<int>(min(static_cast<int64_t>(32), p.tokens - row0));
#pragma unroll 1
            for (int c = c0; c < c0 + kCols / 2; c += 32) {
                const int col = ty * kCols + c;
                if (nrows <= 0 || col >= p.n)
                    break;  // warp-uniform
                uint32_t g[32], u[32], w[16];
                tmem_ld32_wait(tacc + static_cast<uint32_t>(c), g);
                tmem_ld32_wait(tacc + static_cast<uint32_t>(c + kCols), u);
                if (gu) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        w[i] = pack16(__uint_as_float(g[2 * i]), __uint_as_float(g[2 * i + 1]), p.bf16);
                    store32(gu, p.ldgu, row0, nrows, col, p.n, w, p.vec_g, lane, stage_buf);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        w[i] = pack16(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]), p.bf16);
                    store32(gu + p.n, p.ldgu, row0, nrows, col, p.n, w, p.vec_u, lane, stage_buf);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float a = act_value(__uint_as_float(g[2 * i]), ACT) * __uint_as_float(u[2 * i]);
                    const float b = act_value(__uint_as_float(g[2 * i + 1]), ACT) * __uint_as_float(u[2 * i + 1]);
                    w[i] = pack16(a, b, p.bf16);
                }
                store32(out, p.ldo, row0, nrows, col, p.n, w, p.vec_h, lane, stage_buf);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[buf]), 0));
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

cudaLaunchConfig_t config(int grid, cudaStream_t stream, cudaLaunchAttribute* attr)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

// Asked once per device, by the kernel's first launch there.
template <int ACT>
cudaError_t resident(int device, int* pairs)
{
    static SmemLimit limit;
    static std::atomic<int> known[64];  // 1 + their number
    int n = known[device].load(std::memory_order_relaxed);
    if (n == 0) {
        cudaError_t e = limit.allow(gated_pair_kernel<ACT>, kSmem, device);
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = config(2, nullptr, attr);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, gated_pair_kernel<ACT>, &cfg);
        if (e != cudaSuccess)
            return e;
        known[device].store(++n, std::memory_order_relaxed);
    }
    *pairs = n - 1;
    return cudaSuccess;
}

}  // namespace

cudaError_t gated_pairs(int act, int device, int* pairs)
{
    switch (act) {
    case kActSilu: return resident<kActSilu>(device, pairs);
    case kActGelu: return resident<kActGelu>(device, pairs);
    default: return resident<kActGeluTanh>(device, pairs);
    }
}

cudaError_t gated_pair_launch(const FfnParams& f, int pairs, cudaStream_t stream)
{
    PairParams p{};
    const int dtype = f.bf16 ? GEMM_DTYPE_BF16 : GEMM_DTYPE_F16;
    CUtensorMap tmx, tmw;
    if (!call_map(&tmx, f.x, f.tokens, f.k, f.ldx, 1, 0, 128, dtype) ||
        !call_map(&tmw, f.w, f.n, f.k, f.ldw, 2, int64_t(f.n) * f.ldw, kCols, dtype))
        return cudaErrorInvalidValue;
    p.out = f.out;
    p.ldo = f.ldo;
    p.gu = f.gu;
    p.ldgu = f.ldgu;
    p.tokens = f.tokens;
    p.n = f.n;
    p.tiles_x = static_cast<int>((int64_t(f.tokens) + 255) / 256);
    p.tiles_y = static_cast<int>((int64_t(f.n) + kCols - 1) / kCols);
    p.num_tiles = p.tiles_x * p.tiles_y;  // (the caller's bound)
    p.num_kb = static_cast<int>((int64_t(f.k) + BK - 1) / BK);
    p.group_x = 8;
    p.bf16 = f.bf16;
    const auto width = [](const void* q, int64_t ld) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(q);
        return a % 32 == 0 && ld % 16 == 0 ? 16 : (a % 16 == 0 && ld % 8 == 0 ? 8 : 1);
    };
    p.vec_h = width(f.out, f.ldo);
    p.vec_g = width(f.gu, f.ldgu);
    p.vec_u = width(static_cast<const uint16_t*>(f.gu) + f.n, f.ldgu);
    p.idesc = idesc_f16_f32(256, 256) | (f.bf16 ? (1u << 7) | (1u << 10) : 0u);
    p.status = f.status;
    p.wait_limit = f.wait_limit;
    p.fault = f.fault;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config(2 * std::min(p.num_tiles, pairs), stream, attr);
    switch (f.act) {
    case kActSilu: return cudaLaunchKernelEx(&cfg, gated_pair_kernel<kActSilu>, tmx, tmw, p);
    case kActGelu: return cudaLaunchKernelEx(&cfg, gated_pair_kernel<kActGelu>, tmx, tmw, p);
    default: return cudaLaunchKernelEx(&cfg, gated_pair_kernel<kActGeluTanh>, tmx, tmw, p);
    }
}

}  // namespace gnt
