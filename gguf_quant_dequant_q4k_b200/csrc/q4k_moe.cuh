// q4k_moe.cuh -- device helpers of the mixture-of-experts kernels: loads of memory
// that an earlier kernel may have written. They are ordinary (coherent) loads that
// stay where they are written: neither moved in front of pdl_wait() nor behind the
// work that is meant to cover their latency.
#pragma once

#include <cuda_runtime.h>

namespace q4k {

__device__ __forceinline__ int load_i32(const int* p) {
    int v;
    asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ float4 load_f4(const float4* p) {
    float4 v;
    asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// load_f4 of data that is read once.
__device__ __forceinline__ float4 load_f4_once(const float4* p) {
    float4 v;
    asm volatile("ld.global.cs.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

}  // namespace q4k
