// q4k_moe_gemm.cu -- Q4_K products grouped by expert (fp16 x, weights rounded to the fp16 mirror).
#include "q4k_moe_rows.cuh"

namespace q4k {

__device__ unsigned int g_moe_gemm_fault_flags = 0;

int launch_moe_gemm(const DeviceInfo& dev, const void* w, const void* w2, const void* xv, const MoeGroups& g,
                    void* y, int n, int k, cudaStream_t stream) {
    void* flags = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&flags, g_moe_gemm_fault_flags);
    if (e != cudaSuccess) return cuda_failure(e);
    const __half* x = static_cast<const __half*>(xv);
    const dim3 grid((n + 7) / 8, g.experts);
    const uint8_t* a = static_cast<const uint8_t*>(w);
    const uint8_t* b = static_cast<const uint8_t*>(w2);
    if (w2 != nullptr)
        q4k_moe_rows_kernel<__half, __half, true, true><<<grid, kMoeRowsThreads, 0, stream>>>(
            a, b, x, g, static_cast<__half*>(y), n, k, static_cast<unsigned*>(flags));
    else
        q4k_moe_rows_kernel<__half, float, false, true><<<grid, kMoeRowsThreads, 0, stream>>>(
            a, b, x, g, static_cast<float*>(y), n, k, static_cast<unsigned*>(flags));
    e = cudaGetLastError();
    return e == cudaSuccess ? Q4K_OK : cuda_failure(e);
}

int moe_gemm_set_attributes() { return Q4K_OK; }

int read_moe_gemm_fault_flags(unsigned* flags) {
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_moe_gemm_fault_flags, sizeof(v));
    if (e != cudaSuccess) return cuda_failure(e);
    const unsigned zero = 0;
    e = cudaMemcpyToSymbol(g_moe_gemm_fault_flags, &zero, sizeof(zero));
    if (e != cudaSuccess) return cuda_failure(e);
    *flags = v;
    return Q4K_OK;
}

}  // namespace q4k
