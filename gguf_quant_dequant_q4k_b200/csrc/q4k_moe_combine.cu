// q4k_moe_combine.cu -- y[t] = residual[t] + sum_j weights[t][j] * z[t*k + j],
// over the choices j with an expert (ids[t][j] >= 0), in f32, j ascending
// (q4k_moe_combine).
//
// Bound: HBM. Each z row is read once and y written once; a thread owns four
// columns of a token and requests all the token's z rows (up to kCombineMaxK
// 16-byte loads that keep their place) before it adds the first, so the loads are
// in flight together: 4096 tokens, top 4, 4096 columns in 60.5 us, 6.6 TB/s (68 us
// with loads that the compiler may move).
#include "q4k_internal.h"
#include "q4k_moe.cuh"
#include "q4k_moe.h"
#include "q4k_sm100.cuh"

namespace q4k {

namespace {

constexpr int kCombineThreads = 256;
constexpr int kCombineMaxK = 16;   // Q4K_MOE_MAX_TOP_K

template <int K>
__global__ void __launch_bounds__(kCombineThreads)
q4k_moe_combine_kernel(const float* z, const int* ids, const float* weights,
                       const float* residual, float* y, long long n_tokens, int top_k, int cols4) {
    pdl_launch_dependents();
    pdl_wait();
    const long long total = n_tokens * cols4;
    const long long stride = static_cast<long long>(gridDim.x) * kCombineThreads;
    const int kk = K > 0 ? K : top_k;
    constexpr int kMax = K > 0 ? K : kCombineMaxK;
    for (long long i = static_cast<long long>(blockIdx.x) * kCombineThreads + threadIdx.x; i < total; i += stride) {
        const long long t = i / cols4;
        const int c = static_cast<int>(i - t * cols4);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (residual != nullptr) acc = reinterpret_cast<const float4*>(residual)[i];
        float4 v[kMax];
        float wt[kMax];
        bool live[kMax];
#pragma unroll
        for (int j = 0; j < kMax; ++j) {
            if (j >= kk) break;
            live[j] = ids[t * kk + j] >= 0;           // a row without an expert is never read
            wt[j] = live[j] ? weights[t * kk + j] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kMax; ++j) {
            if (j >= kk) break;
            v[j] = live[j] ? load_f4_once(reinterpret_cast<const float4*>(z) + (t * kk + j) * cols4 + c)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int j = 0; j < kMax; ++j) {
            if (j >= kk) break;
            acc.x = fmaf(wt[j], v[j].x, acc.x);
            acc.y = fmaf(wt[j], v[j].y, acc.y);
            acc.z = fmaf(wt[j], v[j].z, acc.z);
            acc.w = fmaf(wt[j], v[j].w, acc.w);
        }
        reinterpret_cast<float4*>(y)[i] = acc;
    }
}

}  // namespace

int launch_moe_combine(const float* z, const int* ids, const float* weights, const float* residual, float* y,
                       int n_tokens, int top_k, int hidden, int num_sms, cudaStream_t stream) {
    const int cols4 = hidden / 4;
    const long long total = static_cast<long long>(n_tokens) * cols4;
    long long blocks = (total + kCombineThreads - 1) / kCombineThreads;
    const long long cap = static_cast<long long>(num_sms) * 8;
    if (blocks > cap) blocks = cap;
    auto* kernel = top_k == 1   ? q4k_moe_combine_kernel<1>
                   : top_k == 2 ? q4k_moe_combine_kernel<2>
                   : top_k == 4 ? q4k_moe_combine_kernel<4>
                   : top_k == 8 ? q4k_moe_combine_kernel<8>
                                : q4k_moe_combine_kernel<0>;
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
                                             top_k, cols4);
    return e == cudaSuccess ? Q4K_OK : cuda_failure(e);
}

}  // namespace q4k
