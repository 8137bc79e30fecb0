// q4k_moe_combine.cu -- y[t] = residual[t] + sum_j weights[t][j] * z[t*k + j],
// over the choices j with an expert (ids[t][j] >= 0), in f32, j ascending
// (q4k_moe_combine).
//
// Bound: HBM. Each z row is read once and y written once; a thread owns four
// columns of a token and requests its z rows, up to eight, before it adds the
// first (16-byte loads that keep their place), so the loads are in flight together.
// Measured, 4096 tokens, 4096 columns, with the residual: top 4 60.8 us, 6.6 TB/s
// (68.7 with loads that the compiler may move); top 8 97 us. A kernel per top_k: one
// for any top_k, its loops cut off at run time, takes 85 us for top 3 (55) and 106
// for top 6 (79). From five choices on, four CTAs per SM are asked for (top 6 79 us,
// else 90); for fewer the compiler chooses (top 1 31 us, with the bound 39).
#include <utility>

#include "q4k_internal.h"
#include "q4k_moe.cuh"
#include "q4k_moe.h"
#include "q4k_sm100.cuh"

namespace q4k {

namespace {

constexpr int kCombineThreads = 256;
constexpr int kCombineBatch = 8;   // rows in flight

template <int K>
__global__ void __launch_bounds__(kCombineThreads, K > 4 ? 4 : 0)
q4k_moe_combine_kernel(const float* z, const int* ids, const float* weights, const float* residual, float* y,
                       long long n_tokens, int cols4) {
    pdl_launch_dependents();
    pdl_wait();
    const long long total = n_tokens * cols4;
    const long long stride = static_cast<long long>(gridDim.x) * kCombineThreads;
    for (long long i = static_cast<long long>(blockIdx.x) * kCombineThreads + threadIdx.x; i < total; i += stride) {
        const long long t = i / cols4;
        const int c = static_cast<int>(i - t * cols4);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (residual != nullptr) acc = reinterpret_cast<const float4*>(residual)[i];
        bool live[K];
        float wt[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            live[j] = ids[t * K + j] >= 0;   // a row without an expert is never read
            wt[j] = live[j] ? weights[t * K + j] : 0.f;
        }
#pragma unroll
        for (int j0 = 0; j0 < K; j0 += kCombineBatch) {
            float4 v[kCombineBatch];
#pragma unroll
            for (int j = j0; j < K && j < j0 + kCombineBatch; ++j)
                v[j - j0] = live[j] ? load_f4_once(reinterpret_cast<const float4*>(z) + (t * K + j) * cols4 + c)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int j = j0; j < K && j < j0 + kCombineBatch; ++j) {
                acc.x = fmaf(wt[j], v[j - j0].x, acc.x);
                acc.y = fmaf(wt[j], v[j - j0].y, acc.y);
                acc.z = fmaf(wt[j], v[j - j0].z, acc.z);
                acc.w = fmaf(wt[j], v[j - j0].w, acc.w);
            }
        }
        reinterpret_cast<float4*>(y)[i] = acc;
    }
}

using CombineKernel = void (*)(const float*, const int*, const float*, const float*, float*, long long, int);

template <int... J>
CombineKernel combine_kernel(int top_k, std::integer_sequence<int, J...>) {
    static const CombineKernel kernels[] = {q4k_moe_combine_kernel<J + 1>...};
    return kernels[top_k - 1];
}

}  // namespace

int launch_moe_combine(const float* z, const int* ids, const float* weights, const float* residual, float* y,
                       int n_tokens, int top_k, int hidden, int num_sms, cudaStream_t stream) {
    const int cols4 = hidden / 4;
    const long long total = static_cast<long long>(n_tokens) * cols4;
    long long blocks = (total + kCombineThreads - 1) / kCombineThreads;
    const long long cap = static_cast<long long>(num_sms) * 8;
    if (blocks > cap) blocks = cap;
    const CombineKernel kernel = combine_kernel(top_k, std::make_integer_sequence<int, Q4K_MOE_MAX_TOP_K>());
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kCombineThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, z, ids, weights, residual, y, static_cast<long long>(n_tokens),
                                             cols4);
    return e == cudaSuccess ? Q4K_OK : cuda_failure(e);
}

}  // namespace q4k
