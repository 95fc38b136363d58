// block128_tc.cuh -- pieces shared by the tcgen05 kernels of the block-scaled
// product: packed fp32 arithmetic, Tensor Memory loads without a wait, register
// hand-over between warpgroups, bounded waits.
#pragma once
#include "block128.h"
#include "ptx.cuh"
#include "tc05_common.cuh"

namespace gnt {
namespace blk {

constexpr int kRowBytes = 128;    // one K block of an operand row

// Two fp32 operations in one instruction (each rounded to nearest even).
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t pack2u(uint32_t a, uint32_t b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The load alone: r may be used only after tmem_wait(r), which waits for all of this
// thread's loads and names the registers so that no use of them is scheduled before it.  32 lanes x 16
// or 32 columns: thread i of the warp receives TMEM lane (lane field) + i.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
          "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
        :
        : "memory");
}
// The way back, to be waited for by tmem_st_wait.
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        :
        : "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
          "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
          "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
          "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
        :
        : "memory");
}

// Shared-memory loads by 32-bit address.
__device__ __forceinline__ float lds_f32(uint32_t a)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ ulonglong2 lds_f32x4(uint32_t a)
{
    ulonglong2 v;
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "r"(a) : "memory");
    return v;
}

// mbar_arrive of the lanes whose predicate holds, without a branch.
__device__ __forceinline__ void mbar_arrive_if(uint32_t bar, bool pred)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"(static_cast<uint32_t>(pred))
        : "memory");
}

// 32 lanes x 8 columns: thread i of the warp receives TMEM lane (lane field) + i.
__device__ __forceinline__ void tmem_ld32x8(uint32_t taddr, uint32_t* r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait8(uint32_t* r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}

// Register hand-over between the warpgroups of a CTA: what the takers gain must
// come from what the givers return of the registers the CTA was launched with.
template <int N>
__device__ __forceinline__ void regs_give()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_take()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void raise(const BlkParams& p, volatile int* abort_flag)
{
    *abort_flag = 1;
    atomicOr(p.status, kStatusTimeout);
}

// As tc::wait_bounded, in line: ptxas does not allocate registers across a call
// in a kernel that hands registers over.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, const volatile int* abort_flag,
                                             unsigned long long limit)
{
    if (__builtin_expect(mbar_try_wait(bar, parity), 1))
        return true;
    const long long t0 = clock64();
    while (!mbar_try_wait_sleep(bar, parity, 1000000u))
        if (*abort_flag || static_cast<unsigned long long>(clock64() - t0) > limit)
            return false;
    return true;
}

// A whole warp waits, each lane on a barrier and phase of its own; true once all
// have completed.
__device__ __forceinline__ bool wait_lanes(uint32_t bar, uint32_t parity, const volatile int* abort_flag,
                                           unsigned long long limit)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
        return true;
    const long long t0 = clock64();
    while (!__all_sync(0xffffffffu, mbar_try_wait_sleep(bar, parity, 1000000u)))
        if (__any_sync(0xffffffffu, *abort_flag || static_cast<unsigned long long>(clock64() - t0) > limit))
            return false;
    return true;
}

// One lane of a converged warp, the same at every call.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// ---------------------------------------------------------------- scales
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const float* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// One of the barrier's expected arrivals, made when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The scales of 32*R rows from `first` (or, step 128, of one in 128 rows in the
// first lanes), copied K block by K block by one warp.  Where the rows' scales
// are adjacent and on 16-byte boundaries (as the quantiser leaves them when the
// number of rows is a multiple of 4), 128 rows take one instruction, else four.
template <int R>
struct ScaleRun {
    const float* src[R];
    int64_t step;
    bool wide;
    uint32_t off;

    __device__ __forceinline__ ScaleRun(const ScaleView& v, int b, int first, int rows, int every = 1)
    {
        const int lane = threadIdx.x & 31;
        const float* base = v.data + b * v.bs;
        step = v.ks;
        wide = R % 4 == 0 && every == 1 && v.shift == 0 && v.rs == 1 && v.ks % 4 == 0 && rows - first >= 32 * R &&
               (reinterpret_cast<uintptr_t>(base + first) & 15) == 0;
        off = static_cast<uint32_t>(wide ? 16 * lane : 4 * lane);
        if (wide) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                src[r] = base + first + 128 * r + 4 * lane;  // only the first R / 4 are used
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = min(first + (every == 1 ? 32 * r + lane : every * (lane & 1)), rows - 1);
                src[r] = base + static_cast<int64_t>(row >> v.shift) * v.rs;
            }
        }
    }

    // Starts at K block kb instead of 0.
    __device__ __forceinline__ void skip(int kb)
    {
#pragma unroll
        for (int r = 0; r < R; ++r)
            src[r] += kb * step;
    }

    // The next K block's scales to shared address `dst`.
    __device__ __forceinline__ void copy(uint32_t dst)
    {
        dst += off;
        if (wide) {
#pragma unroll
            for (int r = 0; r < R / 4; ++r) {
                cp_async16(dst + 512 * r, src[r]);
                src[r] += step;
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                cp_async4(dst + 128 * r, src[r]);
                src[r] += step;
            }
        }
    }
};

// Twice how far the largest of four scales' magnitudes lies above `from`, as a word
// (doubling drops the signs; a smaller one wraps to the top): plain_scale but for zero,
// infinity and NaN, which may as well be treated with care.
__device__ __forceinline__ uint32_t beyond(ulonglong2 w, uint32_t from)
{
    const uint32_t a = 2u * static_cast<uint32_t>(w.x) - 2u * from, b = 2u * static_cast<uint32_t>(w.x >> 32) - 2u * from;
    const uint32_t c = 2u * static_cast<uint32_t>(w.y) - 2u * from, d = 2u * static_cast<uint32_t>(w.y >> 32) - 2u * from;
    return max(max(a, b), max(c, d));
}

// Whether any of the warp's values is not zero.
template <int N>
__device__ __forceinline__ bool any_set(const uint32_t (&x)[N])
{
    uint32_t u = 0;
#pragma unroll
    for (int j = 0; j < N; ++j)
        u |= x[j];
    return __any_sync(0xffffffffu, u != 0);
}

// acc += x times the thread's scale and the columns' (at shared address `w`), where
// the thread's leaves the range that needs no care.  Blocks of zeros, whose scales
// are tiny, do not come here: their products are zero in any order.
template <int N>
__device__ __forceinline__ void add_careful(uint64_t* acc, const uint32_t (&x)[N], float s, uint32_t w)
{
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        float a[2];
        unpack2(acc[j / 2], a[0], a[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const Factors f = scale_factors(s, lds_f32(w + 4 * (j + e)));
            a[e] = fmaf(__uint_as_float(x[j + e]) * f.first, f.second, a[e]);
        }
        acc[j / 2] = pack2(a[0], a[1]);
    }
}

// Waits (with the limit) without giving up early: for drains before exit.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, unsigned long long limit)
{
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity) && static_cast<unsigned long long>(clock64() - t0) <= limit) {
    }
}

}  // namespace blk
}  // namespace gnt
