// Paired-CTA tensor-core GEMM: the instances that store C, and the launcher
// (the kernel is in umma_pair_kernel.cuh).
#include <atomic>

#include "umma_pair_kernel.cuh"

namespace dg {

size_t umma_pair_smem_bytes(int bn, int stages, bool epi_tma, int ksub, int epi_warps) {
    return pair_layout(bn, stages, epi_tma, ksub, epi_warps).total;
}

int umma_pair_max_stages(int bn, bool epi_tma, int ksub, int epi_warps) {
    int s = 2;
    while (s < 12 && pair_layout(bn, s + 1, epi_tma, ksub, epi_warps).total <= 227 * 1024) ++s;
    return s;
}

cudaError_t launch_umma_pair(const UmmaParams &p, const CUtensorMap *tp, const CUtensorMap *tq,
                             const CUtensorMap *tc, bool fp8, int grid, size_t smem, cudaStream_t s) {
    void (*kern)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const UmmaParams);
    if (p.ksub != 1 && p.ksub != 2) return cudaErrorInvalidValue;
    const bool deep = p.ksub == 2;
    kern = fp8 ? (deep ? umma_pair_kernel<true, 2, EPI_STORE> : umma_pair_kernel<true, 1, EPI_STORE>)
               : (deep ? umma_pair_kernel<false, 2, EPI_STORE> : umma_pair_kernel<false, 1, EPI_STORE>);
    static SmemLimit s_limit[4];
    const cudaError_t e = s_limit[(fp8 ? 2 : 0) + (deep ? 1 : 0)].ensure(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_ex(kern, dim3(grid), dim3(192), smem, s, dim3(2, 1, 1), p.pdl, *tp, *tq, *tc, p);
}

}  // namespace dg
