// Global loads of kernels that start while the one before them still writes what they read.
#pragma once

#include <stdint.h>

namespace q8 {

// ld.global.nc, which __ldg and const __restrict__ stand for, is for data that nothing writes during the whole kernel: it need not see
// the writes of the kernel before, and the compiler may move it ahead of the wait for that kernel. These are coherent loads and
// stay behind the wait.
__device__ __forceinline__ uint32_t load8(const void* p) {
    uint32_t v;
    asm volatile("ld.global.u8 %0, [%1];\n" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t load32(const void* p) {
    uint32_t v;
    asm volatile("ld.global.b32 %0, [%1];\n" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint2 load64(const void* p) {
    uint2 v;
    asm volatile("ld.global.v2.b32 {%0, %1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint4 load128(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ int load_int(const int32_t* p) { return (int)load32(p); }
__device__ __forceinline__ float load_float(const float* p) { return __uint_as_float(load32(p)); }

}  // namespace q8
