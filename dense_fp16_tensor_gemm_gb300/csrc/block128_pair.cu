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
// as does shared memory (64 KB in and out at 128 bytes a cycle), and each SM's
// promotion warps read 128 x 256 values from Tensor Memory and do one packed fp32
// operation for every two of them (300 cycles; two, where B has a scale for
// every row).  Two accumulators of 256 columns fill Tensor Memory; what bounds
// the kernel is the round trip of one: MMA, commit to both CTAs, loads and
// arithmetic, release to the leader.  Measured per block (4864 x 4096, K from
// 2048 to 8192): 430 ns, 645 where B has a scale for every row; before the scales were
// looked at (below) 410 and 620, and against those 310 with the
// arithmetic left out, 345 with the loads left out.  Halves of 128 columns, which
// shorten the trip, are slower (A is read twice and shared memory fills up), as
// are 16 warps with 64 sums each (490 and 670), scalar arithmetic (452) and loads of
// 16 rows x 64 columns, which let a column's scale serve two rows (510 and 655).  A tile's
// epilogue adds 1.5 us (16-bit Out) to 3 us (fp32): its registers are the sums.
// 8192 x 8192 x 8192 into bf16: 440-452 us among other calls, 407-414 from a graph
// (2430-2700 TFLOP/s).
//
// Roles per CTA (384 threads): warp 0 TMA producer; warps 1 and 3 in the leader
// MMA issue; warp 2 brings the scales into a ring of their own (any strides);
// warps 4-11 promotion, 128 sums per thread, which take over registers from
// warps 0-3.  A thread holds 128 columns of one row (32x32b loads), so a block
// takes two scales from shared memory, or 1 + 128; Out passes through a small
// staging area to leave in row segments.
// Synchronisation:
//   full[s], empty[s]    operand ring, as in the unscaled pair kernel
//   tfull[b], tempty[b]  accumulators: leader's commit to both CTAs / one
//                        arrival per promotion warp of both, at the leader
//   sfull[r], sempty[r]  scale ring, within the CTA
// The scales may hold any fp32 values.  Where their product (by row: a block's sum
// times the column's scale) may leave the normal range on the way, the scale warp
// marks the group, and its blocks are scaled in another order, or in two steps inside
// Tensor Memory: 3-4 % for the check, at 8192 x 8192 x 8192 407 us for 393.
// Every wait is bounded.
#include <algorithm>

#include "block128_tc.cuh"

namespace gnt {

namespace {

using namespace blk;
using tc::BM;

constexpr int kTile = 256;                  // rows and columns of a pair's tile
constexpr int kThreads = 384;
constexpr int kPromoWarps = 8;
constexpr int kCols = 128;                  // columns of a promotion thread
constexpr int kPiece = 32;                  // columns of one accumulator load
constexpr int kAcc = 2;                     // accumulators in Tensor Memory, one per K block parity
constexpr int kStages = 5;
constexpr int kOpBytes = BM * kRowBytes;    // one CTA's half of A, and of B
constexpr int kScaleRing = 4;               // slots of kScaleGroup K blocks
constexpr int kScaleGroup = 4;
constexpr int kScaleFloats = 128 + 256;     // rows' scales, then columns' (or the two column blocks')
constexpr int kStagePitch = 40;             // words of a staging row: 8 of the piece before, then 32
constexpr int kStageWords = 32 * kStagePitch;  // a promotion warp's staging area
constexpr int kTmemCols = 512;
constexpr int kBarBytes = 512;
constexpr int kSmem = 1024 + kStages * 2 * kOpBytes + kScaleRing * kScaleGroup * kScaleFloats * 4 + kPromoWarps * kStageWords * 4 + kBarBytes;
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

// K blocks of all of a pair's tiles.
__device__ __forceinline__ int blocks_of(const BlkParams& p, int pair, int pairs)
{
    return (p.num_tiles - pair + pairs - 1) / pairs * p.num_kb;
}

// Word w of row r of a staging area.  16-byte slots change places in pairs in rows
// 4-7 of every 8, so that the 8 rows a phase of 16-byte stores writes fall on
// different banks.
__device__ __forceinline__ int staged(int r, int w) { return r * kStagePitch + (w ^ (r & 4)); }

// Stores a promotion warp's 32 rows x 128 columns, a row per thread, through its
// staging area.  128 bytes of every row at a time leave as whole row segments:
// 16-byte words where Out's rows lie on 16-byte boundaries; else each row's
// segments start on its own 32-byte boundary, up to 8 words back in the piece
// before (which are staged again), so that memory gets whole sectors whatever
// the pitch, and what is left of a row follows the last piece.  Reads of the
// staging area go ahead of a batch's stores: one at a time the two latencies add up.
template <int OT, int C = 0>
__device__ __forceinline__ void store_tile(const BlkParams& p, const uint64_t (&acc)[kCols / 2], uint32_t* stage, int b,
                                           int row0, int col0, int lane)
{
    using S = OutStore<OT>;
    using T = typename S::T;
    constexpr int PER_WORD = OT == kOutF32 ? 1 : 2, SEG = 32 * PER_WORD, BACK = 8 * PER_WORD;  // elements
    T* out = static_cast<T*>(p.out) + b * p.stride_o + static_cast<int64_t>(row0) * p.ldo + col0;
    const int rows = min(p.M - row0, 32), cols = min(kCols, p.N - col0);
    // rows on 16-byte boundaries: half sectors at a piece's ends cost less than the other
    // route (16 x 3001 x 2052 x 1000 into fp32 201 us for 236; 2056 into bf16 170 for 203)
    const bool wide = p.vec >= 4 * PER_WORD;
#pragma unroll
    for (int w = C ? 0 : 8; w < kStagePitch; w += 4) {
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = C - BACK + (w + i) * PER_WORD;
            if constexpr (OT == kOutF32) {
                float f[2];
                unpack2(acc[e / 2], f[0], f[1]);
                v[i] = __float_as_uint(f[i & 1]);
            } else {
                float f0, f1;
                unpack2(acc[e / 2], f0, f1);
                v[i] = S::pack(f0, f1);
            }
        }
        *reinterpret_cast<uint4*>(stage + staged(lane, w)) = make_uint4(v[0], v[1], v[2], v[3]);
    }
    __syncwarp();
    if (wide && C + SEG <= cols) {
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = *reinterpret_cast<const uint4*>(stage + staged(4 * i + (lane >> 3), 8 + 4 * (lane & 7)));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3);
            if (r < rows)
                __stcs(reinterpret_cast<uint4*>(out + r * p.ldo + C) + (lane & 7), v[i]);
        }
    } else if (C < cols + BACK) {
        constexpr int FOUR = 4 * PER_WORD, BATCH = 4;
        // Of rows r0, r0 + step, ... the 16 bytes at column c, less the way back to
        // the row's boundary: four words off the staging area, one store inside Out.
        auto batch = [&](int r0, int step, int c) {
            uint32_t v[BATCH][4];
            int k[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int r = r0 + i * step;
                k[i] = c - (static_cast<int>(reinterpret_cast<uintptr_t>(out + r * p.ldo) / sizeof(T)) & (BACK - 1));
                const int e = k[i] - (C - BACK), w = e / PER_WORD;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[i][j] = stage[staged(r, min(w + j, kStagePitch - 1))];
                if (PER_WORD == 2 && (e & 1)) {
                    const uint32_t next = stage[staged(r, min(w + 4, kStagePitch - 1))];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[i][j] = __funnelshift_r(v[i][j], j < 3 ? v[i][(j + 1) & 3] : next, 16);
                }
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int r = r0 + i * step, lo = max(0, -k[i]), hi = r < rows ? min(FOUR, cols - k[i]) : 0;
                T* d = out + r * p.ldo + k[i];
                if (lo == 0 && hi == FOUR) {
                    // not streamed: a sector shared with the neighbour tile waits for it in L2
                    *reinterpret_cast<uint4*>(d) = make_uint4(v[i][0], v[i][1], v[i][2], v[i][3]);
                } else {
#pragma unroll
                    for (int j = 0; j < FOUR; ++j)
                        if (j >= lo && j < hi)
                            d[j] = OT == kOutF32 ? static_cast<T>(__uint_as_float(v[i][j & 3]))
                                                 : static_cast<T>(v[i][j / PER_WORD] >> (16 * (j & 1)));
                }
            }
        };
#pragma unroll 1
        for (int r = 0; r < rows; r += 4 * BATCH)
            batch(r + (lane >> 3), 4, C + FOUR * (lane & 7));
        if (C + SEG == kCols && lane < 16)  // what is left of the rows
            batch(lane >> 1, 8, kCols + FOUR * (lane & 1));
    }
    __syncwarp();
    if constexpr (C + SEG < kCols)
        store_tile<OT, C + SEG>(p, acc, stage, b, row0, col0, lane);
}

// Whether the scales of a group's K blocks 0 to `last`, landed at shared address `s`,
// need no care: the smallest and the largest of the rows' times those of the column
// blocks' are normal, or (BROW) every column's is one to multiply by first.  For the
// whole warp, four rows or eight columns a lane; few instructions, which promotion
// warps wait for (200 a group cost 3 % of 8192 x 8192 x 8192).
template <bool BROW>
__device__ __forceinline__ bool plain_group(uint32_t s, int last, uint32_t from)
{
    const uint32_t lane = threadIdx.x & 31;
    bool plain;
    if (BROW) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kScaleGroup; ++i) {
            const uint32_t at = s + min(i, last) * (kScaleFloats * 4) + 512 + 16 * lane;
            top = max(top, max(beyond(lds_f32x4(at), from), beyond(lds_f32x4(at + 512), from)));
        }
        plain = top <= 2u * (kPlainTo - from);
    } else {
        float lo = INFINITY, hi = 0.f, blo = INFINITY, bhi = 0.f;
#pragma unroll
        for (int i = 0; i < kScaleGroup; ++i) {
            const uint32_t at = s + min(i, last) * (kScaleFloats * 4);
            float v[4];
            const ulonglong2 w = lds_f32x4(at + 16 * lane);
            unpack2(w.x, v[0], v[1]);
            unpack2(w.y, v[2], v[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                lo = fminf(lo, fabsf(v[e]));
                hi = fmaxf(hi, fabsf(v[e]));
            }
            const float f = fabsf(lds_f32(at + 512 + 4 * (lane & 1)));
            blo = fminf(blo, f);
            bhi = fmaxf(bhi, f);
        }
        blo = fminf(blo, __shfl_xor_sync(0xffffffffu, blo, 1));
        bhi = fmaxf(bhi, __shfl_xor_sync(0xffffffffu, bhi, 1));
        plain = is_normal(lo * blo) && is_normal(hi * bhi);
    }
    return __all_sync(0xffffffffu, plain);
}

// The scale warp: for every K block of the pair's tiles, this CTA's 128 row scales
// of A and the tile's 256 (BROW) or 2 of B into the scale ring, by asynchronous
// copies.  A slot is handed on once its copies have landed, with the word that says
// whether care is needed; the ring keeps the warp three slots ahead.  (One arrival: 32
// of them, though off the critical path, made 397 us 447 at 8192 x 8192 x 8192.)
// Rows outside Out multiply zeros and are not stored; they take the last row's scale.
template <bool BROW>
__device__ __forceinline__ void load_scales(const BlkParams& p, int rank, float* scales, uint32_t* careful, uint64_t* sfull,
                                            uint64_t* sempty, volatile int* abort_flag, int pair, int pairs)
{
    const uint32_t ring = smem_u32(scales), from = plain_from(p.e5m2);
    const int blocks = blocks_of(p, pair, pairs);
    int n = 0;  // K blocks so far
    for (int t = pair; t < p.num_tiles; t += pairs) {
        int b, m0, n0;
        decode(p, t, b, m0, n0);
        ScaleRun<4> a(p.sa, b, m0 + rank * BM, p.M);
        ScaleRun<BROW ? 8 : 1> w(p.sb, b, n0, p.N, BROW ? 1 : 128);
#pragma unroll 1
        for (int kb = 0; kb < p.num_kb; ++kb) {
            const int slot = n / kScaleGroup % kScaleRing, at = n % kScaleGroup;
            if (at == 0 &&
                !wait_bounded(smem_u32(&sempty[slot]), (n / (kScaleGroup * kScaleRing) & 1) ^ 1, abort_flag, p.wait_limit)) {
                raise(p, abort_flag);
                cp_async_wait_all();
                return;
            }
            const uint32_t first = ring + slot * kScaleGroup * (kScaleFloats * 4), s = first + at * (kScaleFloats * 4);
            a.copy(s);
            w.copy(s + 128 * 4);
            ++n;
            if (at == kScaleGroup - 1 || n == blocks) {
                cp_async_wait_all();
                __syncwarp();  // every lane's copies are here
                const bool plain = plain_group<BROW>(first, at, from);
                if ((threadIdx.x & 31) == 0) {
                    careful[slot] = !plain;
                    mbar_arrive(smem_u32(&sfull[slot]));
                }
                __syncwarp();
            }
        }
    }
}

// Multiplies a warp's 32 rows x 128 columns of the accumulator at `ta` in place by
// their rows' two factors, where those leave the normal range on the way.
__device__ __forceinline__ void scale_accumulator(uint32_t ta, Factors f)
{
#pragma unroll 1
    for (int c = 0; c < kCols; c += 16) {
        uint32_t x[16];
        tmem_ld(ta + c, x);
        tmem_wait(x);
#pragma unroll
        for (int j = 0; j < 16; ++j)
            x[j] = __float_as_uint(__uint_as_float(x[j]) * f.first * f.second);
        tmem_st(ta + c, x);
    }
    tmem_st_wait();
}

// By row: one K block, a warp's 32 rows x 128 columns of the accumulator at `ta` times
// the row's scale fa and the columns' at shared address `cols`, added to its sums; with
// care where some scales may leave the normal range on the way and there is something
// to scale (a block of zeros has tiny scales).  16 columns at a time: few registers
// beside the sums.
__device__ __forceinline__ void promote_careful(uint64_t (&acc)[kCols / 2], uint32_t ta, float fa, uint32_t cols, bool care)
{
    const uint64_t sr = pack2(fa, fa);
#pragma unroll
    for (int c = 0; c < kCols; c += 16) {
        uint32_t x[16];
        tmem_ld(ta + c, x);
        tmem_wait(x);
        uint64_t* d = acc + c / 2;
        if (care && any_set(x)) {
            add_careful(d, x, fa, cols + 4 * c);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const ulonglong2 w = lds_f32x4(cols + 4 * c + 16 * j);
                d[2 * j] = fma2(mul2(pack2u(x[4 * j], x[4 * j + 1]), w.x), sr, d[2 * j]);
                d[2 * j + 1] = fma2(mul2(pack2u(x[4 * j + 2], x[4 * j + 3]), w.y), sr, d[2 * j + 1]);
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
    uint32_t* staging = reinterpret_cast<uint32_t*>(scales + kScaleRing * kScaleGroup * kScaleFloats);
    uint64_t* tfull = reinterpret_cast<uint64_t*>(staging + kPromoWarps * kStageWords);
    uint64_t* tempty = tfull + kAcc;
    uint64_t* full = tempty + kAcc;
    uint64_t* empty = full + kStages;
    uint64_t* sfull = empty + kStages;
    uint64_t* sempty = sfull + kScaleRing;
    uint64_t* drain = sempty + kScaleRing;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    uint32_t* careful_slot = tmem_slot + 2;  // one word for each slot of the scale ring
    static_assert((2 * kStages + 2 * kAcc + 2 * kScaleRing + 2) * 8 + 8 + 4 * kScaleRing <= kBarBytes, "barrier area");

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int b = 0; b < kAcc; ++b) {
            mbar_init(smem_u32(&tfull[b]), 1);
            mbar_init(smem_u32(&tempty[b]), 2 * kPromoWarps);
        }
        for (int r = 0; r < kScaleRing; ++r) {
            mbar_init(smem_u32(&sfull[r]), 1);
            mbar_init(smem_u32(&sempty[r]), kPromoWarps);
        }
        mbar_init(smem_u32(&drain[0]), 1);
        mbar_init(smem_u32(&drain[1]), 1);
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
        regs_give<72>();
        if (warp == 0 && lane == 0) {
            // -------------------------------------------------------- producer (both CTAs)
            int stage = 0;
            uint32_t phase = 0, filled = 0, fill_parity = 0;
            bool ok = true, drop = p.fault == 1 && blockIdx.x == 0;
            for (int t = pair; ok && t < p.num_tiles; t += pairs) {
                int b, m0, n0;
                decode(p, t, b, m0, n0);
                const int xa = m0 + static_cast<int>(rank) * BM, xb = n0 + static_cast<int>(rank) * BM;
#pragma unroll 1
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
#pragma unroll 1
            for (int s = 0; s < kStages; ++s)
                if (filled & (1u << s))
                    drain_wait(smem_u32(&full[s]), (fill_parity >> s) & 1u, p.wait_limit);
        } else if ((warp == 1 || warp == 3) && leader) {
            // -------------------------------------------------------- MMA issue (leader)
            // Warps 1 and 3 take the even and odd K blocks (counted over the pair's
            // tiles).  What a block costs its warp beside the MMAs (waits, commits,
            // loop) is longer than the 128 cycles that the tensor core's queue covers,
            // so each warp pays it while the other's MMAs run.  The whole warp runs the
            // loop, lanes polling different barriers at once and operands in uniform
            // registers; one lane issues.
            const int par = warp >> 1;
            const uint32_t idesc = idesc_f16_f32(kTile, kTile) | p.idesc_bits;
            const DescWords da = desc_words(smem_u32(as), false), db = desc_words(smem_u32(bs), false);
            const uint32_t d = tmem_base + static_cast<uint32_t>(par * kTile);
            const uint32_t te = smem_u32(&tempty[par]), tf = smem_u32(&tfull[par]);
            int stage = par;
            uint32_t phase = 0, tphase = 0;
            bool skip_release = p.fault == 2 && blockIdx.x == 0 && par == 0;
            const bool chosen = elect_one();
#pragma unroll 1
            for (int n = blocks_of(p, pair, pairs) - par; n > 0; n -= 2) {
                const uint32_t fa = smem_u32(&full[stage]), ea = smem_u32(&empty[stage]);
                const uint32_t alo = da.lo + static_cast<uint32_t>(stage * (kOpBytes >> 4));
                const uint32_t blo = db.lo + static_cast<uint32_t>(stage * (kOpBytes >> 4));
                // even lanes: the accumulator is free; odd lanes: the operands are here
                if (!wait_lanes(lane & 1 ? fa : te, lane & 1 ? phase : tphase ^ 1, abort_flag, p.wait_limit)) {
                    raise(p, abort_flag);
                    break;
                }
                tc_fence_after();
                if (chosen) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_pair_w<true>(d, alo + k * da.kstep, da.hi, blo + k * db.kstep, db.hi, idesc, k > 0);
                    tc_commit_pair_mc(tf, 0x3);
                    if (!skip_release)
                        tc_commit_pair_mc(ea, 0x3);
                }
                __syncwarp();
                skip_release = false;
                tphase ^= 1;
                stage += 2;
                if (stage >= kStages) {
                    stage -= kStages;
                    phase ^= 1;
                }
            }
            // no MMA may still be running when Tensor Memory is released
            if (chosen) {
                tc_commit_pair(smem_u32(&drain[par]));
                drain_wait(smem_u32(&drain[par]), 0, p.wait_limit);
            }
        } else if (warp == 2) {
            load_scales<BROW>(p, static_cast<int>(rank), scales, careful_slot, sfull, sempty, abort_flag, pair, pairs);
        }
    } else {
        // ------------------------------------------------------------ promotion (both CTAs)
        regs_take<216>();
        // Lane quadrant q, columns [128cq, 128cq + 128): pieces of 32 columns in two
        // register buffers, a piece's load under the arithmetic of the piece before.
        const int q = warp & 3, cq = (warp - 4) >> 2;
        const uint32_t tmem_warp = tmem_base + static_cast<uint32_t>(128 * cq) + (static_cast<uint32_t>(32 * q) << 16);
        const uint32_t my_scales = smem_u32(scales) + (32 * q + lane) * 4;
        const uint32_t col_scales = smem_u32(scales) + (128 + (BROW ? 128 * cq : cq)) * 4;
        const uint32_t tf0 = smem_u32(tfull), sf0 = smem_u32(sfull), careful0 = smem_u32(careful_slot);
        const uint32_t te0 = mapa_shared(smem_u32(tempty), 0);
        const int blocks = blocks_of(p, pair, pairs);
        int n = 0;  // K blocks so far: ring positions and phases follow from it
        bool ok = true, careful = false;  // careful: of the group that block n is in
        auto enter_group = [&](int at, bool& care) {
            const int slot = at / kScaleGroup % kScaleRing;
            const bool here = wait_bounded(sf0 + slot * 8, at / (kScaleGroup * kScaleRing) & 1, abort_flag, p.wait_limit);
            care = lds_u32(careful0 + slot * 4) != 0;
            return here;
        };
        while (ok && n < blocks) {
            uint64_t acc[kCols / 2];
#pragma unroll
            for (int j = 0; j < kCols / 2; ++j)
                acc[j] = 0;
            int left = p.num_kb;
            // Blocks in whose groups all scales are plain; by row, from the first other one
            // on, the rest of the tile in a loop that can take care.  No way leads back to this loop inside a tile: a
            // branch around its arithmetic keeps loads from going ahead (490 us for 397 at
            // 8192 x 8192 x 8192), and so do two bodies in one loop (545).
#pragma unroll 1
            do {
                if (n % kScaleGroup == 0)
                    ok &= enter_group(n, careful);
                if (BROW && careful)
                    break;
                const uint32_t so = n % (kScaleGroup * kScaleRing) * (kScaleFloats * 4);
                float fa = lds_f32(my_scales + so), fb = BROW ? 1.f : lds_f32(col_scales + so);
                ok &= wait_bounded(tf0 + (n & 1) * 8, n >> 1 & 1, abort_flag, p.wait_limit);
                tc_fence_after();
                const uint32_t ta = tmem_warp + (n & 1) * kTile;
                if (!BROW && careful) {
                    scale_accumulator(ta, scale_factors(fa, fb));
                    fa = fb = 1.f;
                }
                uint64_t sr = 0;
#pragma unroll
                for (int g = 0; g < kCols / kPiece; g += 2) {
                    uint32_t x[2][kPiece];
                    tmem_ld(ta + kPiece * g, x[0]);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t(&z)[kPiece] = x[c];
                        tmem_wait(z);
                        if (c == 0) {
                            tmem_ld(ta + kPiece * (g + 1), x[1]);
                        } else if (g + 2 == kCols / kPiece) {
                            // the accumulator is in registers: free it for block n + 2
                            tc_fence_before();
                            if (lane == 0)
                                mbar_arrive_cluster(te0 + (n & 1) * 8);
                        }
                        if (g == 0 && c == 0) {
                            const float f = BROW ? fa : fa * fb;
                            sr = pack2(f, f);
                        }
#pragma unroll
                        for (int j = 0; j < kPiece / 4; ++j) {
                            uint64_t p0 = pack2u(z[4 * j], z[4 * j + 1]), p1 = pack2u(z[4 * j + 2], z[4 * j + 3]);
                            uint64_t* d = acc + kPiece / 2 * (g + c) + 2 * j;
                            if (BROW) {
                                const ulonglong2 w = lds_f32x4(col_scales + so + (kPiece * (g + c) + 4 * j) * 4);
                                d[0] = fma2(mul2(p0, w.x), sr, d[0]);
                                d[1] = fma2(mul2(p1, w.y), sr, d[1]);
                            } else {
                                d[0] = fma2(p0, sr, d[0]);
                                d[1] = fma2(p1, sr, d[1]);
                            }
                        }
                    }
                }
                if (n % kScaleGroup == kScaleGroup - 1) {
                    __syncwarp();
                    mbar_arrive_if(smem_u32(&sempty[n / kScaleGroup % kScaleRing]), lane == 0);
                }
                ++n;
            } while (--left > 0 && ok);
            if (BROW && left > 0 && ok) {
#pragma unroll 1
                do {
                    const uint32_t so = n % (kScaleGroup * kScaleRing) * (kScaleFloats * 4);
                    ok &= wait_bounded(tf0 + (n & 1) * 8, n >> 1 & 1, abort_flag, p.wait_limit);
                    tc_fence_after();
                    promote_careful(acc, tmem_warp + (n & 1) * kTile, lds_f32(my_scales + so), col_scales + so, careful);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_cluster(te0 + (n & 1) * 8);
                    if (n % kScaleGroup == kScaleGroup - 1)
                        mbar_arrive_if(smem_u32(&sempty[n / kScaleGroup % kScaleRing]), lane == 0);
                    ++n;
                    if (--left > 0 && n % kScaleGroup == 0)
                        ok &= enter_group(n, careful);
                } while (left > 0 && ok);
            }
            if (!ok) {
                raise(p, abort_flag);
                break;
            }
            int b, m0, n0;
            decode(p, pair + (n / p.num_kb - 1) * pairs, b, m0, n0);
            const int row0 = m0 + static_cast<int>(rank) * BM + 32 * q, col0 = n0 + 128 * cq;
            uint32_t* stage_buf = staging + (warp - 4) * kStageWords;
            if (p.out_type == kOutF16)
                store_tile<kOutF16>(p, acc, stage_buf, b, row0, col0, lane);
            else if (p.out_type == kOutBF16)
                store_tile<kOutBF16>(p, acc, stage_buf, b, row0, col0, lane);
            else
                store_tile<kOutF32>(p, acc, stage_buf, b, row0, col0, lane);
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
    p.tiles_m = (p.M - 1) / kTile + 1;
    p.tiles_n = (p.N - 1) / kTile + 1;
    p.num_tiles = p.tiles_m * p.tiles_n * p.batch;
    p.group_m = 8;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = pair_config(std::min(p.num_tiles, max_pairs), stream, attr);
    return p.sb.shift ? cudaLaunchKernelEx(&cfg, block128_pair_kernel<false>, tma, tmb, p)
                      : cudaLaunchKernelEx(&cfg, block128_pair_kernel<true>, tma, tmb, p);
}

}  // namespace gnt
