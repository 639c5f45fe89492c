// Paired-CTA tensor-core kernel: the instances that serve the linear cross
// entropy and its gradient (the kernel is in umma_pair_kernel.cuh).
#include <atomic>

#include "umma_pair_kernel.cuh"

namespace dg {

namespace {

template <int KSUB, int EPI>
cudaError_t run_pair(const UmmaParams &p, const CUtensorMap *tp, const CUtensorMap *tq, const CUtensorMap *tc,
                     int grid, size_t smem, cudaStream_t s) {
    static SmemLimit limit;
    auto kern = umma_pair_kernel<false, KSUB, EPI>;
    const cudaError_t e = limit.ensure(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_ex(kern, dim3(grid), dim3(pair_threads(EPI)), smem, s, dim3(2, 1, 1), p.pdl, *tp, *tq, *tc, p);
}

template <int KSUB>
cudaError_t run_use(const UmmaParams &p, const CUtensorMap *tp, const CUtensorMap *tq, const CUtensorMap *tc,
                    PairUse use, int grid, size_t smem, cudaStream_t s) {
    switch (use) {
    case kPairStats:
        if (p.k_chunk < p.kb_total) return run_pair<KSUB, EPI_CE_STATS_LONG>(p, tp, tq, tc, grid, smem, s);
        return run_pair<KSUB, EPI_CE_STATS>(p, tp, tq, tc, grid, smem, s);
    case kPairGrad:
        if (p.k_chunk < p.kb_total) return run_pair<KSUB, EPI_CE_GRAD_LONG>(p, tp, tq, tc, grid, smem, s);
        return run_pair<KSUB, EPI_CE_GRAD>(p, tp, tq, tc, grid, smem, s);
    case kPairWide: return run_pair<KSUB, EPI_STORE_WIDE>(p, tp, tq, tc, grid, smem, s);
    default: return run_pair<KSUB, EPI_PARTIAL>(p, tp, tq, tc, grid, smem, s);
    }
}

}  // namespace

cudaError_t launch_umma_pair_use(const UmmaParams &p, const CUtensorMap *tp, const CUtensorMap *tq,
                                 const CUtensorMap *tc, PairUse use, int grid, size_t smem, cudaStream_t s) {
    if (p.bn != 256 || p.k_chunk < 1 || (use == kPairStats) == (p.epi_tma != 0)) return cudaErrorInvalidValue;
    if (p.ksub == 1) return run_use<1>(p, tp, tq, tc, use, grid, smem, s);
    if (p.ksub == 2) return run_use<2>(p, tp, tq, tc, use, grid, smem, s);
    return cudaErrorInvalidValue;
}

}  // namespace dg
