// The linear cross entropy's GEMM kernels.
#include "gemm_ce.cuh"
#include "host.cuh"

namespace lgb {

template <int KIND, bool LONG>
static cudaError_t launch_kind(const CeGemmParams& p, int grid, cudaStream_t st) {
  auto* k = ce_gemm_kernel<KIND, LONG>;
  constexpr int smem = PairCfg<kCeStages, kCeWarps>::kSmemBytes;
  static std::atomic<unsigned long long> configured{0};
  const cudaError_t e = ensure_smem_limit(k, smem, configured);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(grid), dim3(pair_threads(kCeWarps)), smem, st, p);  // grid: a multiple of 2
}

cudaError_t launch_ce_gemm(int kind, const CeGemmParams& p, int grid, cudaStream_t st) {
  const bool parts = p.kb_range < p.kb_total;
  switch (kind) {
    case CE_STATS: return parts ? launch_kind<CE_STATS, true>(p, grid, st) : launch_kind<CE_STATS, false>(p, grid, st);
    case CE_GRAD: return parts ? launch_kind<CE_GRAD, true>(p, grid, st) : launch_kind<CE_GRAD, false>(p, grid, st);
    case CE_PART: return parts ? launch_kind<CE_PART, true>(p, grid, st) : launch_kind<CE_PART, false>(p, grid, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace lgb
