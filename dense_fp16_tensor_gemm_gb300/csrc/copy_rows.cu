// copy_rows.cu -- a matrix's rows onto 16-byte boundaries, for kernels that read by TMA
// or 16 bytes at a time.  A thread writes 16 bytes, gathered in the widest units that the
// source's base and pitch allow (neighbouring threads share their lines in L1).  Bound by
// memory, one read and one write, and at 2-byte units by the loads' lines in L1 (4000 x
// 4097 16-bit elements 16 us).
#include <algorithm>

#include "ffn.h"

namespace gnt {

namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads) copy_rows_kernel(const uint8_t* src, int64_t lds, uint8_t* dst, int64_t ldd,
                                                             int64_t rows, int64_t bytes)
{
    constexpr int kUnits = 16 / sizeof(T);
    const int64_t pieces = (bytes + 15) / 16;
    // a block walks along a row, blockIdx.y's and further ones in steps
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        for (int64_t p = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; p < pieces;
             p += static_cast<int64_t>(gridDim.x) * kThreads) {
            const uint8_t* s = src + row * lds + p * 16;
            uint8_t* d = dst + row * ldd + p * 16;
            if (bytes - p * 16 >= 16) {
                union {
                    T t[kUnits];
                    uint4 v;
                } u;
#pragma unroll
                for (int i = 0; i < kUnits; ++i)
                    u.t[i] = __ldg(reinterpret_cast<const T*>(s) + i);
                *reinterpret_cast<uint4*>(d) = u.v;
            } else {
                for (int i = 0; i < bytes - p * 16; ++i)
                    d[i] = s[i];
            }
        }
    }
}

}  // namespace

cudaError_t copy_rows_launch(const void* src, int64_t lds, void* dst, int64_t ldd, int64_t rows, int64_t bytes, cudaStream_t stream)
{
    const uint8_t* s = static_cast<const uint8_t*>(src);
    uint8_t* d = static_cast<uint8_t*>(dst);
    const int64_t pieces = (bytes + 15) / 16;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((pieces + kThreads - 1) / kThreads, 1024)),
                    static_cast<unsigned>(std::min<int64_t>(rows, 65535)));
    const uintptr_t at = reinterpret_cast<uintptr_t>(src) | static_cast<uintptr_t>(rows > 1 ? lds : 0);
    if (at % 16 == 0)
        copy_rows_kernel<uint4><<<grid, kThreads, 0, stream>>>(s, lds, d, ldd, rows, bytes);
    else if (at % 4 == 0)
        copy_rows_kernel<uint32_t><<<grid, kThreads, 0, stream>>>(s, lds, d, ldd, rows, bytes);
    else if (at % 2 == 0)
        copy_rows_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(s, lds, d, ldd, rows, bytes);
    else
        copy_rows_kernel<uint8_t><<<grid, kThreads, 0, stream>>>(s, lds, d, ldd, rows, bytes);
    return cudaGetLastError();
}

}  // namespace gnt
