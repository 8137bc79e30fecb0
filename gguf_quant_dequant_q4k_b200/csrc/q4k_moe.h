// q4k_moe.h -- host-side interface of the mixture-of-experts operators: the
// router (q4k_moe_route.cu), the expert-grouped Q4_K products
// (q4k_moe_gemv.cu, q4k_moe_gemm.cu) and the weighted combination
// (q4k_moe_combine.cu). Arguments are validated by the callers (q4k_api.cu).
//
// The kernels are launched programmatically and let their successors start before
// their own wait for their predecessor: what an earlier kernel may write (logits,
// ids, weights, offsets, order, x, z) is read by plain loads behind pdl_wait() (or
// by TMA), never by non-coherent ones, which need data that nothing writes while
// the grid lives; no pointer to it is const __restrict__.
#pragma once

#include <cuda_runtime.h>

namespace q4k {

struct DeviceInfo;

// The routed pairs of a batch and the product's sizes.
struct MoeGroups {
    const int* offsets;   // [experts + 1]: slots offsets[e] .. offsets[e + 1] - 1 are expert e's
    const int* order;     // [pairs]: the pair of each slot
    int experts;
    int pairs;
    int per_row;          // x row of slot s: s if 0, else order[s] / per_row
};

int launch_moe_route(const float* logits, int* ids, float* weights, int* offsets, int* order, int n_tokens,
                     int n_experts, int top_k, bool renorm, int num_sms, cudaStream_t stream);

// w2 != null: gate w, up w2, y = silu(w x) * (w2 x), rows in slot order; else
// y = w x, rows in pair order.
int launch_moe_gemv(const DeviceInfo& dev, const void* w, const void* w2, const float* x, const MoeGroups& g,
                    float* y, int n, int k, cudaStream_t stream);
int launch_moe_gemm(const DeviceInfo& dev, const void* w, const void* w2, const void* x_f16, const MoeGroups& g,
                    void* y, int n, int k, cudaStream_t stream);

int launch_moe_combine(const float* z, const int* ids, const float* weights, const float* residual, float* y,
                       int n_tokens, int top_k, int hidden, int num_sms, cudaStream_t stream);

int read_moe_gemv_fault_flags(unsigned* flags);
int read_moe_gemm_fault_flags(unsigned* flags);

}  // namespace q4k
