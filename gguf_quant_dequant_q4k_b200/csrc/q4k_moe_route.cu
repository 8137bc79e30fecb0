// q4k_moe_route.cu -- the router of a mixture-of-experts layer (q4k_moe_route):
// each token's top_k experts and their softmax weights, and the pairs (token,
// choice) grouped by expert.
//
// Two launches, no workspace, no atomics (the lists do not depend on timing):
// * choose: a warp per token. A lane holds experts lane, lane + 32, ... as
//   order-preserving integer keys; each of the top_k rounds takes the warp's
//   maximum (redux) and, among equal keys, the lowest expert. The weights are
//   exp(l - l_max) over the sum of the chosen (or of all) in f32.
// * group: a CTA per expert reads all ids once, counts those below its expert
//   (the first slot of its range) and writes its own pairs in ascending order
//   at the positions a block-wide scan gives.
// Bound: reading the logits (choose), E passes over the ids from L2 (group).
#include <cfloat>
#include <cstdint>

#include "q4k_internal.h"
#include "q4k_moe.h"

namespace q4k {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kChooseThreads = 256;
constexpr int kGroupThreads = 512;

// Larger float, larger key; NaN and -inf get 0 (never chosen), +inf the key of
// FLT_MAX.
__device__ __forceinline__ uint32_t logit_key(float v) {
    if (!(v > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(fminf(v, FLT_MAX));
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_logit(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}

// S: keys per lane, experts <= 32 S.
template <int S>
__global__ void __launch_bounds__(kChooseThreads)
q4k_moe_choose_kernel(const float* __restrict__ logits, int* __restrict__ ids, float* __restrict__ weights,
                      int n_tokens, int n_experts, int top_k, bool renorm) {
    const int lane = threadIdx.x & 31;
    const int warp0 = (blockIdx.x * kChooseThreads + threadIdx.x) >> 5;
    const int nwarps = (gridDim.x * kChooseThreads) >> 5;
    for (int t = warp0; t < n_tokens; t += nwarps) {
        const float* row = logits + static_cast<size_t>(t) * n_experts;
        uint32_t key[S];
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const int e = 32 * i + lane;
            key[i] = e < n_experts ? logit_key(__ldg(row + e)) : 0u;
        }
        float top = 0.f, all = 0.f, mine = 0.f;   // lane j keeps the j-th choice
        int chosen = -1;
        for (int j = 0; j < top_k; ++j) {
            uint32_t best = 0u;
            int at = 0;
#pragma unroll
            for (int i = 0; i < S; ++i)
                if (key[i] > best) {   // the lane's first among equals
                    best = key[i];
                    at = 32 * i + lane;
                }
            const uint32_t m = __reduce_max_sync(kFull, best);
            if (m == 0u) break;        // no expert left
            const int e = static_cast<int>(
                __reduce_min_sync(kFull, best == m ? static_cast<unsigned>(at) : 0xFFFFFFFFu));
            const float l = key_logit(m);
            if (j == 0) {
                top = l;
                if (!renorm) {
                    float s = 0.f;
#pragma unroll
                    for (int i = 0; i < S; ++i) s += key[i] != 0u ? expf(key_logit(key[i]) - top) : 0.f;
                    all = warp_sum(s);
                }
            }
            if (lane == j) {
                chosen = e;
                mine = expf(l - top);
            }
#pragma unroll
            for (int i = 0; i < S; ++i)
                if (32 * i + lane == e) key[i] = 0u;
        }
        const float total = renorm ? warp_sum(mine) : all;
        if (lane < top_k) {
            ids[static_cast<size_t>(t) * top_k + lane] = chosen;
            weights[static_cast<size_t>(t) * top_k + lane] = chosen >= 0 ? __fdiv_rn(mine, total) : 0.f;
        }
    }
}

// CTA e < n_experts: expert e's offset and pairs; the last CTA: the total and
// the -1 behind the last slot.
__global__ void __launch_bounds__(kGroupThreads)
q4k_moe_group_kernel(const int* __restrict__ ids, int* __restrict__ offsets, int* __restrict__ order, int n_pairs,
                     int n_experts) {
    __shared__ int warp_less[kGroupThreads / 32], warp_eq[kGroupThreads / 32];
    const int e = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // thread t's contiguous share of the pairs
    const int per = (n_pairs + kGroupThreads - 1) / kGroupThreads;
    const int p0 = min(n_pairs, tid * per), p1 = min(n_pairs, p0 + per);
    int less = 0, eq = 0;
    for (int p = p0; p < p1; ++p) {
        const int id = __ldg(ids + p);
        less += id >= 0 && id < e;
        eq += id == e;
    }
    int scan = eq;   // inclusive scan of eq over the block
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(kFull, scan, off);
        if (lane >= off) scan += v;
    }
    less = __reduce_add_sync(kFull, less);
    if (lane == 31) {
        warp_less[warp] = less;
        warp_eq[warp] = scan;
    }
    __syncthreads();
    int base = 0, before = 0;
    for (int w = 0; w < kGroupThreads / 32; ++w) {
        base += warp_less[w];
        if (w < warp) before += warp_eq[w];
    }
    if (tid == 0) offsets[e] = base;
    if (e < n_experts) {
        int s = base + before + scan - eq;
        for (int p = p0; p < p1; ++p)
            if (__ldg(ids + p) == e) order[s++] = p;
    } else {
        for (int s = base + tid; s < n_pairs; s += kGroupThreads) order[s] = -1;
    }
}

template <int S>
void launch_choose(const float* logits, int* ids, float* weights, int n_tokens, int n_experts, int top_k, bool renorm,
                   int num_sms, cudaStream_t stream) {
    const int per_cta = kChooseThreads / 32;
    int blocks = (n_tokens + per_cta - 1) / per_cta;
    if (blocks > num_sms * 8) blocks = num_sms * 8;
    q4k_moe_choose_kernel<S><<<blocks, kChooseThreads, 0, stream>>>(logits, ids, weights, n_tokens, n_experts, top_k,
                                                                    renorm);
}

}  // namespace

int launch_moe_route(const float* logits, int* ids, float* weights, int* offsets, int* order, int n_tokens,
                     int n_experts, int top_k, bool renorm, int num_sms, cudaStream_t stream) {
    if (n_tokens > 0) {
        if (n_experts <= 32)
            launch_choose<1>(logits, ids, weights, n_tokens, n_experts, top_k, renorm, num_sms, stream);
        else if (n_experts <= 64)
            launch_choose<2>(logits, ids, weights, n_tokens, n_experts, top_k, renorm, num_sms, stream);
        else if (n_experts <= 128)
            launch_choose<4>(logits, ids, weights, n_tokens, n_experts, top_k, renorm, num_sms, stream);
        else
            launch_choose<8>(logits, ids, weights, n_tokens, n_experts, top_k, renorm, num_sms, stream);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_failure(e);
    }
    q4k_moe_group_kernel<<<n_experts + 1, kGroupThreads, 0, stream>>>(ids, offsets, order, n_tokens * top_k, n_experts);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? Q4K_OK : cuda_failure(e);
}

}  // namespace q4k
