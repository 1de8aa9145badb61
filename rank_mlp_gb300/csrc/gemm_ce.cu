// The linear cross entropy's GEMM kernels.
#include "gemm_ce.cuh"
#include "host.cuh"

namespace lgb {

template <int KIND, int WARPS>
static cudaError_t launch_kind(const CeGemmParams& p, int grid, cudaStream_t st) {
  auto* k = ce_gemm_kernel<KIND, WARPS>;
  constexpr int smem = PairCfg<kCeStages, WARPS>::kSmemBytes;
  static std::atomic<unsigned long long> configured{0};
  const cudaError_t e = ensure_smem_limit(k, smem, configured);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(grid), dim3(pair_threads(WARPS)), smem, st, p);  // grid: a multiple of 2
}

cudaError_t launch_ce_gemm(int kind, const CeGemmParams& p, int grid, cudaStream_t st) {
  const bool wide = ce_warps(p.kb_total) == 8;
  switch (kind) {
    case CE_STATS: return wide ? launch_kind<CE_STATS, 8>(p, grid, st) : launch_kind<CE_STATS, 4>(p, grid, st);
    case CE_GRAD: return wide ? launch_kind<CE_GRAD, 8>(p, grid, st) : launch_kind<CE_GRAD, 4>(p, grid, st);
    case CE_PART: return launch_kind<CE_PART, 8>(p, grid, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace lgb
