// GEMM instantiations of the layer operators.
#include <atomic>

#include "block_epilogues.cuh"
#include "block_internal.h"

namespace flce {

// Co-resident clusters of the kernel on the current device, asked once per device
// and HALVES (whose instantiations share one footprint).
template <int HALVES>
static int max_clusters(const void* kernel) {
  constexpr int kMaxDev = 64;
  static std::atomic<int> cache[kMaxDev];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return 0;
  int v = cache[dev].load(std::memory_order_relaxed);
  if (v > 0) return v;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kLThreads, 1, 1);
  cfg.dynamicSmemBytes = PairShape<HALVES>::kSmem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&v, kernel, &cfg) != cudaSuccess || v <= 0) {
    cudaGetLastError();
    return 0;
  }
  cache[dev].store(v, std::memory_order_relaxed);
  return v;
}

template <class Epi, int HALVES, bool SPLIT>
static cudaError_t launch_form(const PairArgs& g, const typename Epi::Args& ea, int sms,
                               cudaStream_t st) {
  auto kernel = pair_gemm_kernel<Epi, HALVES, SPLIT>;
  constexpr size_t smem = PairShape<HALVES>::kSmem;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  int clusters = g.tiles_m * g.tiles_n;
  if constexpr (!SPLIT) {
    int most = max_clusters<HALVES>(reinterpret_cast<const void*>(kernel));
    if (most <= 0) most = sms / 2;
    if (clusters > most) clusters = most;
  }
  const int ctas = SPLIT ? 2 * g.slices : 2;
  return launch_dependent(kernel, dim3(static_cast<unsigned>(ctas * clusters)), kLThreads, smem,
                          ctas, st, g, ea);
}

template <class Epi>
static cudaError_t launch(const PairArgs& g, const typename Epi::Args& ea, int sms,
                          cudaStream_t st) {
  if (g.slices > 1) return launch_form<Epi, 1, true>(g, ea, sms, st);
  if constexpr (Epi::kBMN) {  // the gradients
    if (g.halves == 2) return launch_form<Epi, 2, false>(g, ea, sms, st);
  }
  return launch_form<Epi, 1, false>(g, ea, sms, st);
}

cudaError_t launch_linear(const PairArgs& g, const LinearArgs& ea, int sms, cudaStream_t st) {
  return launch<LinearEpi>(g, ea, sms, st);
}
cudaError_t launch_gated(const PairArgs& g, const GatedArgs& ea, int sms, cudaStream_t st) {
  return launch<GatedEpi>(g, ea, sms, st);
}
cudaError_t launch_grad_x(bool two, const PairArgs& g, const GradXArgs& ea, int sms,
                          cudaStream_t st) {
  return two ? launch<GradXEpi<kTwoK>>(g, ea, sms, st) : launch<GradXEpi<kOneEach>>(g, ea, sms, st);
}
cudaError_t launch_grad_w(bool two, const PairArgs& g, const GradWArgs& ea, int sms,
                          cudaStream_t st) {
  return two ? launch<GradWEpi<kTwoA>>(g, ea, sms, st) : launch<GradWEpi<kOneEach>>(g, ea, sms, st);
}

}  // namespace flce
