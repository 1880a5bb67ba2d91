// What the kernels that plan moves of pages share: one workgroup that passes over
// the page table, its counters in LDS where the pool's pages fit and in the
// scratch otherwise.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hr {
namespace {

constexpr int kScan = 1024;        // threads of the planning workgroup
constexpr int kPlanPages = 12288;  // pages whose three counters fit LDS

// exclusive sum of v over the workgroup's kScan threads, and the total
__device__ __forceinline__ int scan_wg(int v, int* total, int* lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int inc = v;
#pragma unroll
    for (int x = 1; x < 64; x *= 2) {
        const int y = __shfl_up(inc, x);
        if (lane >= x) inc += y;
    }
    __syncthreads();
    if (lane == 63) lds[wave] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int x = 0; x < kScan / 64; ++x) {
        const int y = lds[x];
        if (x < wave) before += y;
        all += y;
    }
    *total = all;
    return before + inc - v;
}

__device__ __forceinline__ int page_in(int32_t page, int64_t n) {
    return page >= 0 && page < n ? page : -1;
}

// Entries of the table are taken by groups of 16 lanes, a row each at a time.
constexpr int kRowLanes = 16;

// Launches a planning kernel: in LDS if its counters fit, else in the scratch.
template <class A, class... P>
int plan(void (*in_lds)(A, P...), void (*in_scratch)(A, P...), int words, const A& a, hipStream_t s, P... args) {
    const size_t bytes = static_cast<size_t>(words) * a.n_pages * 4;
    if (a.n_pages <= kPlanPages) {
        if (bytes > 65536) {
            const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(in_lds), hipFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(bytes));
            if (e != hipSuccess) return static_cast<int>(e);
        }
        hipLaunchKernelGGL(in_lds, dim3(1), dim3(kScan), bytes, s, a, args...);
    } else {
        hipLaunchKernelGGL(in_scratch, dim3(1), dim3(kScan), 0, s, a, args...);
    }
    return static_cast<int>(hipGetLastError());
}

}  // namespace
}  // namespace hr
