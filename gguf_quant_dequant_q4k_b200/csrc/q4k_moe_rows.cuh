// q4k_moe_rows.cuh -- expert-grouped product, one warp per (output row, up to
// four slots of an expert): every weight decoded once per four slots.
#pragma once

#include <cuda_fp16.h>

#include "q4k_internal.h"
#include "q4k_moe.h"
#include "q4k_superblock.cuh"
#include "q4k_swiglu.cuh"

namespace q4k {

constexpr int kMoeRowsThreads = 256;
constexpr int kMoeRowsSlots = 4;

__device__ __forceinline__ float moe_to_f32(float v) { return v; }
__device__ __forceinline__ float moe_to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void moe_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void moe_store(__half* p, float v) { *p = __float2half_rn(v); }

template <typename XT, bool MIRROR>
__device__ __forceinline__ void moe_rows_dot(const uint8_t* __restrict__ wr, const XT* const (&x)[kMoeRowsSlots],
                                             int cnt, int nsb, int lane, float (&acc)[kMoeRowsSlots]) {
    const int g = lane >> 3, r = (lane & 7) * 8, high = r >= 32, l0 = r & 31;
    for (int b = 0; b < nsb; ++b) {
        const uint8_t* sb = wr + static_cast<size_t>(b) * kBlockBytes;
        const Header hd = decode_header(ldg_nc_v4(sb));
        const uint2 qb = ldg_nc_v2(sb + kQsOffset + 32 * g + l0);
        float dsc, dm;
        subblock_coeffs(hd, 2 * g + high, dsc, dm);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t word = (e < 4) ? qb.x : qb.y;
            float v = weight_value(dsc, dm, (word >> (8 * (e & 3) + (high ? 4 : 0))) & 15u);
            if (MIRROR) v = __half2float(__float2half_rn(v));
#pragma unroll
            for (int i = 0; i < kMoeRowsSlots; ++i)
                if (i < cnt) acc[i] = fmaf(v, moe_to_f32(x[i][b * kQK + 8 * lane + e]), acc[i]);
        }
    }
}

template <typename XT, typename YT, bool SWIGLU, bool MIRROR>
__global__ void __launch_bounds__(kMoeRowsThreads)
q4k_moe_rows_kernel(const uint8_t* __restrict__ w, const uint8_t* __restrict__ w2, const XT* __restrict__ x,
                    MoeGroups gr, YT* __restrict__ y, int n, int k, unsigned* fault) {
    const int nsb = k / kQK, lane = threadIdx.x & 31;
    const int e = blockIdx.y;
    const int s0 = gr.offsets[e], s1 = gr.offsets[e + 1];
    if (s0 < 0 || s1 < s0 || s1 > gr.pairs) {
        if (threadIdx.x == 0) atomicOr(fault, Q4K_FAULT_ROUTE_RANGE);
        return;
    }
    for (int row = (blockIdx.x * kMoeRowsThreads + threadIdx.x) >> 5; row < n; row += (gridDim.x * kMoeRowsThreads) >> 5) {
        const size_t off = (static_cast<size_t>(e) * n + row) * nsb * kBlockBytes;
        for (int s = s0; s < s1; s += kMoeRowsSlots) {
            const int cnt = min(kMoeRowsSlots, s1 - s);
            const XT* xr[kMoeRowsSlots];
            int pair[kMoeRowsSlots];
            float acc[kMoeRowsSlots], acc2[kMoeRowsSlots];
#pragma unroll
            for (int i = 0; i < kMoeRowsSlots; ++i) {
                pair[i] = i < cnt ? gr.order[s + i] : -1;
                const bool ok = pair[i] >= 0 && pair[i] < gr.pairs;
                if (i < cnt && !ok) atomicOr(fault, Q4K_FAULT_ROUTE_RANGE);
                if (!ok) pair[i] = -1;
                const int xrow = !ok ? 0 : gr.per_row == 0 ? s + i : pair[i] / gr.per_row;
                xr[i] = x + static_cast<size_t>(xrow) * k;
                acc[i] = acc2[i] = 0.f;
            }
            moe_rows_dot<XT, MIRROR>(w + off, xr, cnt, nsb, lane, acc);
            if (SWIGLU) moe_rows_dot<XT, MIRROR>(w2 + off, xr, cnt, nsb, lane, acc2);
#pragma unroll
            for (int i = 0; i < kMoeRowsSlots; ++i) {
                float a = acc[i], b = acc2[i];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
                    if (SWIGLU) b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
                }
                if (lane == 0 && pair[i] >= 0) {
                    if (SWIGLU) moe_store(y + static_cast<size_t>(s + i) * n + row, silu_mul(a, b));
                    else moe_store(y + static_cast<size_t>(pair[i]) * n + row, a);
                }
            }
        }
    }
}

}  // namespace q4k
