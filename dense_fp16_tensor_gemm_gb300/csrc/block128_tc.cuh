// block128_tc.cuh -- pieces shared by the tcgen05 kernels of the block-scaled
// product: packed fp32 arithmetic, Tensor Memory loads without a wait, register
// hand-over between warpgroups, bounded waits.
#pragma once
#include "block128.h"
#include "ptx.cuh"
#include "tc05_common.cuh"

namespace gnt {
namespace blk {

constexpr int kThreads = 384;     // warps 0-3: producer, MMA, scales, idle; warps 4-11: promotion
constexpr int kPromoWarps = 8;
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

// tcgen05.ld 16x256b.x4 as tmem_ld16x256_x4_wait, without the wait: r may be
// used only after tmem_wait(r).
__device__ __forceinline__ void tmem_ld16x256_x4(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Waits for this thread's Tensor Memory loads; names the registers so that no
// use of them is scheduled before it.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
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

// Register hand-over: the kernels launch 384 threads with 168 registers each;
// the utility warpgroup keeps 104 and the two promotion warpgroups take 200:
// 104 + 2 * 200 = 504 = 3 * 168.
__device__ __forceinline__ void regs_utility() { asm volatile("setmaxnreg.dec.sync.aligned.u32 104;"); }
__device__ __forceinline__ void regs_promotion() { asm volatile("setmaxnreg.inc.sync.aligned.u32 200;"); }

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
    if (mbar_try_wait(bar, parity))
        return true;
    const long long t0 = clock64();
    while (!mbar_try_wait_sleep(bar, parity, 1000000u))
        if (*abort_flag || static_cast<unsigned long long>(clock64() - t0) > limit)
            return false;
    return true;
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
