// q4k_moe_route.cu -- the router of a mixture-of-experts layer (q4k_moe_route):
// each token's top_k experts and their softmax weights, and the pairs (token,
// choice) grouped by expert.
//
// No workspace; the lists do not depend on timing. Small batches (one_launch): one
// CTA does both steps in one launch. Others: two launches.
// * choose: a warp per token. A lane holds experts lane, lane + 32, ... as
//   order-preserving integer keys; each of the top_k rounds takes the warp's
//   maximum (redux) and, among equal keys, the lowest expert. The weights are
//   exp(l - l_max) over the sum of the chosen (or of all) in f32.
// * group: one cluster of eight CTAs; every CTA, and every warp of it, owns a
//   contiguous piece of the pairs. A warp counts its pairs per expert, the
//   counts are scanned over warps, CTAs (distributed shared memory) and experts,
//   and a second pass over the piece places each pair behind the equal ones
//   before it (32 at a time by match).
// Bound: the launches for a small batch; reading the logits, and the two passes'
// latency, for a large one (8191 tokens, 128 experts, top 8: 78.5 us with a CTA
// per expert that read all ids).
#include <cfloat>
#include <cstdint>

#include "q4k_internal.h"
#include "q4k_moe.h"
#include "q4k_pair.cuh"

namespace q4k {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kChooseThreads = 256;
constexpr int kGroupThreads = 1024;
constexpr int kGroupWarps = kGroupThreads / 32;
constexpr int kGroupCtas = 8;        // portable cluster size
constexpr int kGroupBatch = 8;       // ids per lane in flight
constexpr int kSmallTokens = 64;     // two tokens per warp of the one CTA
static_assert(kSmallTokens * Q4K_MOE_MAX_TOP_K <= 1024, "one pass of 32 pairs per warp");

// One launch or two. A warp's second token costs as much again, the more the more
// rounds (top_k) and keys per lane (s). Measured, one launch against two, us:
//   8 experts, top 2:    16 tokens 3.0 / 4.7    32: 3.3 / 4.7     64: 4.3 / 4.7
//   8 experts, top 4:                           33: 4.7 / 5.0     64: 5.2 / 5.1
//   64 experts, top 2:                          33: 4.7 / 5.2     64: 5.2 / 5.2
//   64 experts, top 8:   16: 4.5 / 5.9          32: 5.6 / 6.2     64: 8.4 / 6.4
//   128 experts, top 2:                         33: 5.5 / 5.7     64: 6.1 / 5.7
//   256 experts, top 16: 16: 9.0 / 9.2          32: 12.8 / 9.5    64: 23.1 / 10.6
bool one_launch(int n_tokens, int top_k, int s) {
    return n_tokens <= 32 || (n_tokens <= kSmallTokens && top_k + s <= 5);
}

// Larger float, larger key; equal floats, equal keys (-0.0 + 0.0 is +0.0); NaN
// and -inf get 0 (never chosen), +inf the key of FLT_MAX.
__device__ __forceinline__ uint32_t logit_key(float v) {
    if (!(v > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(__fadd_rn(fminf(v, FLT_MAX), 0.0f));
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

// Token t's choices and weights, by one warp. S: keys per lane, experts <= 32 S.
template <int S>
__device__ __forceinline__ void choose_token(const float* logits, int* __restrict__ ids,
                                             float* __restrict__ weights, long long t, int n_experts, int top_k,
                                             bool renorm, int lane) {
    const float* row = logits + t * n_experts;
    uint32_t key[S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const int e = 32 * i + lane;
        key[i] = e < n_experts ? logit_key(row[e]) : 0u;
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
        const int e = static_cast<int>(__reduce_min_sync(kFull, best == m ? static_cast<unsigned>(at) : 0xFFFFFFFFu));
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
        ids[t * top_k + lane] = chosen;
        weights[t * top_k + lane] = chosen >= 0 ? __fdiv_rn(mine, total) : 0.f;
    }
}

struct GroupShared {
    int count[kGroupWarps][Q4K_MOE_MAX_EXPERTS];   // pairs of a warp's piece; then those of the warps before it
    int total[Q4K_MOE_MAX_EXPERTS];                // of the CTA
    int base[Q4K_MOE_MAX_EXPERTS];                 // the expert's first slot plus the CTAs before
    int scan[Q4K_MOE_MAX_EXPERTS / 32];
    int slots;
};

// offsets and order of ids [n_pairs], by a cluster of CTAS CTAs of kGroupThreads threads.
template <int CTAS>
__device__ __forceinline__ void group_pairs(GroupShared& sh, const int* ids, int* __restrict__ offsets,
                                            int* __restrict__ order, int n_pairs, int n_experts) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = CTAS > 1 ? static_cast<int>(cluster_rank()) : 0;
    // whole groups of 32 pairs per warp; 64-bit: rounding up may pass 2^31
    const long long per_warp = (static_cast<long long>(n_pairs) + CTAS * kGroupThreads - 1) / (CTAS * kGroupThreads) * 32;
    const long long p0 = (static_cast<long long>(rank) * kGroupWarps + warp) * per_warp;
    const long long p1 = min(p0 + per_warp, static_cast<long long>(n_pairs));
    for (int e = lane; e < n_experts; e += 32) sh.count[warp][e] = 0;
    __syncwarp();
    constexpr int kBatch = CTAS > 1 ? kGroupBatch : 1;   // one CTA: at most 32 pairs per warp
    // kBatch loads at a time are in flight; the first batch stays in registers for the second pass
    int kept[kBatch];
    auto fetch = [&](long long p, int (&id)[kBatch]) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) id[i] = p + 32 * i + lane < p1 ? ids[p + 32 * i + lane] : -1;
    };
    fetch(p0, kept);
    for (long long p = p0; p < p1; p += 32 * kBatch) {
        int id[kBatch];
        if (p > p0) fetch(p, id);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int v = p > p0 ? id[i] : kept[i];
            if (v >= 0) atomicAdd(&sh.count[warp][v], 1);     // a count: the order does not matter
        }
    }
    __syncthreads();
    int all = 0, before = 0;
    if (tid < n_experts) {
        int s = 0;
#pragma unroll 8
        for (int w = 0; w < kGroupWarps; ++w) {
            const int c = sh.count[w][tid];
            sh.count[w][tid] = s;
            s += c;
        }
        sh.total[tid] = all = s;
    }
    if (CTAS > 1) {
        cluster_sync();
        if (tid < n_experts) {
            all = 0;
            for (int c = 0; c < CTAS; ++c) {
                int v;
                asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(map_to_rank(&sh.total[tid], static_cast<uint32_t>(c))) : "memory");
                all += v;
                before += c < rank ? v : 0;
            }
        }
    }
    int scan = all;   // over the experts: 32 per warp, then the warps
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(kFull, scan, off);
        if (lane >= off) scan += v;
    }
    if (warp < Q4K_MOE_MAX_EXPERTS / 32 && lane == 31) sh.scan[warp] = scan;
    __syncthreads();
    if (tid < n_experts) {
        int first = scan - all;
        for (int w = 0; w < warp; ++w) first += sh.scan[w];
        sh.base[tid] = first + before;
        if (rank == 0) offsets[tid] = first;
        if (tid == n_experts - 1) {
            sh.slots = first + all;
            if (rank == 0) offsets[n_experts] = first + all;
        }
    }
    __syncthreads();
    for (long long p = p0; p < p1; p += 32 * kBatch) {
        int id[kBatch];
        if (p > p0) fetch(p, id);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int v = p > p0 ? id[i] : kept[i];
            const unsigned same = __match_any_sync(kFull, v);
            if (v >= 0)
                order[sh.base[v] + sh.count[warp][v] + __popc(same & ((1u << lane) - 1u))] =
                    static_cast<int>(p) + 32 * i + lane;
            __syncwarp();
            if (v >= 0 && lane == __ffs(same) - 1) sh.count[warp][v] += __popc(same);
            __syncwarp();
        }
    }
    for (long long s = static_cast<long long>(sh.slots) + rank * kGroupThreads + tid; s < n_pairs; s += CTAS * kGroupThreads)
        order[s] = -1;
    if (CTAS > 1) cluster_sync();   // no CTA still reads this one's totals
}

template <int S>
__global__ void __launch_bounds__(kChooseThreads)
q4k_moe_choose_kernel(const float* logits, int* __restrict__ ids, float* __restrict__ weights,
                      int n_tokens, int n_experts, int top_k, bool renorm) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int warp0 = (blockIdx.x * kChooseThreads + threadIdx.x) >> 5;
    const int nwarps = (gridDim.x * kChooseThreads) >> 5;
    for (long long t = warp0; t < n_tokens; t += nwarps)   // 64-bit: n_tokens + nwarps may pass 2^31
        choose_token<S>(logits, ids, weights, t, n_experts, top_k, renorm, lane);
}

__global__ void __cluster_dims__(kGroupCtas, 1, 1) __launch_bounds__(kGroupThreads)
q4k_moe_group_kernel(const int* ids, int* __restrict__ offsets, int* __restrict__ order, int n_pairs, int n_experts) {
    __shared__ GroupShared sh;
    pdl_launch_dependents();
    pdl_wait();
    group_pairs<kGroupCtas>(sh, ids, offsets, order, n_pairs, n_experts);
}

template <int S>
__global__ void __launch_bounds__(kGroupThreads)
q4k_moe_route_small_kernel(const float* logits, int* ids, float* __restrict__ weights,
                           int* __restrict__ offsets, int* __restrict__ order, int n_tokens, int n_experts, int top_k,
                           bool renorm) {
    __shared__ GroupShared sh;
    pdl_launch_dependents();
    pdl_wait();
    for (int t = threadIdx.x >> 5; t < n_tokens; t += kGroupWarps)
        choose_token<S>(logits, ids, weights, t, n_experts, top_k, renorm, threadIdx.x & 31);
    __syncthreads();
    group_pairs<1>(sh, ids, offsets, order, n_tokens * top_k, n_experts);
}

struct RouteArgs {
    const float* logits;
    int* ids;
    float* weights;
    int *offsets, *order;
    int n_tokens, n_experts, top_k;
    bool renorm;
};

template <int S>
cudaError_t launch_route(const RouteArgs& a, int num_sms, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (one_launch(a.n_tokens, a.top_k, S)) {
        cfg.gridDim = dim3(1);
        cfg.blockDim = dim3(kGroupThreads);
        return cudaLaunchKernelEx(&cfg, q4k_moe_route_small_kernel<S>, a.logits, a.ids, a.weights, a.offsets, a.order,
                                  a.n_tokens, a.n_experts, a.top_k, a.renorm);
    }
    const int per_cta = kChooseThreads / 32;
    const long long blocks = (static_cast<long long>(a.n_tokens) + per_cta - 1) / per_cta;
    cfg.gridDim = dim3(static_cast<unsigned>(blocks < num_sms * 8 ? blocks : num_sms * 8));
    cfg.blockDim = dim3(kChooseThreads);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, q4k_moe_choose_kernel<S>, a.logits, a.ids, a.weights, a.n_tokens,
                                             a.n_experts, a.top_k, a.renorm);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(kGroupCtas);
    cfg.blockDim = dim3(kGroupThreads);
    return cudaLaunchKernelEx(&cfg, q4k_moe_group_kernel, static_cast<const int*>(a.ids), a.offsets, a.order,
                              a.n_tokens * a.top_k, a.n_experts);
}

}  // namespace

int launch_moe_route(const float* logits, int* ids, float* weights, int* offsets, int* order, int n_tokens,
                     int n_experts, int top_k, bool renorm, int num_sms, cudaStream_t stream) {
    const RouteArgs a{logits, ids, weights, offsets, order, n_tokens, n_experts, top_k, renorm};
    const cudaError_t e = n_experts <= 32    ? launch_route<1>(a, num_sms, stream)
                          : n_experts <= 64  ? launch_route<2>(a, num_sms, stream)
                          : n_experts <= 128 ? launch_route<4>(a, num_sms, stream)
                                             : launch_route<8>(a, num_sms, stream);
    return e == cudaSuccess ? Q4K_OK : cuda_failure(e);
}

}  // namespace q4k
