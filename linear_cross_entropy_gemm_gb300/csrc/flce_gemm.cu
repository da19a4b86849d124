// Instantiations and launchers of the persistent tcgen05 GEMMs.
#include <cuda_runtime.h>

#include "epilogues.cuh"
#include "flce_internal.h"
#include "gemm_launch.cuh"

namespace flce {

template <bool KEEP>
static cudaError_t launch_fwd_lse_t(GemmKind kind, const CUtensorMap& a, const CUtensorMap& b,
                                    const GemmGeom& g, const FwdLseArgs& ea, bool has_bias,
                                    bool has_smooth, int* dev_err, int grid, cudaStream_t st) {
  if (has_bias)
    return has_smooth
               ? launch_any<FwdLseEpi<true, true, KEEP>>(kind, a, b, g, ea, dev_err, grid, st)
               : launch_any<FwdLseEpi<true, false, KEEP>>(kind, a, b, g, ea, dev_err, grid, st);
  return has_smooth
             ? launch_any<FwdLseEpi<false, true, KEEP>>(kind, a, b, g, ea, dev_err, grid, st)
             : launch_any<FwdLseEpi<false, false, KEEP>>(kind, a, b, g, ea, dev_err, grid, st);
}

cudaError_t launch_fwd_lse(GemmKind kind, const CUtensorMap& a, const CUtensorMap& b,
                           const GemmGeom& g, const FwdLseArgs& ea, bool has_bias,
                           bool has_smooth, bool keep, int* dev_err, int grid, cudaStream_t st) {
  return keep ? launch_fwd_lse_t<true>(kind, a, b, g, ea, has_bias, has_smooth, dev_err, grid, st)
              : launch_fwd_lse_t<false>(kind, a, b, g, ea, has_bias, has_smooth, dev_err, grid,
                                        st);
}

cudaError_t launch_dlogits(GemmKind kind, const CUtensorMap& a, const CUtensorMap& b,
                           const GemmGeom& g, const DlogitsArgs& ea, bool has_bias, int* dev_err,
                           int grid, cudaStream_t st) {
  return has_bias ? launch_any<DlogitsEpi<true>>(kind, a, b, g, ea, dev_err, grid, st)
                  : launch_any<DlogitsEpi<false>>(kind, a, b, g, ea, dev_err, grid, st);
}

cudaError_t launch_dw(GemmKind kind, const CUtensorMap& a, const CUtensorMap& b, const GemmGeom& g,
                      const DwArgs& ea, int* dev_err, int grid, cudaStream_t st) {
  return launch_any<DwEpi>(kind, a, b, g, ea, dev_err, grid, st);
}

// dx has few output tiles (N/256 x H/256) and a long K: 256 x 512 tiles would
// leave most of the GPU idle in the last wave, so the wide form runs it as pairs.
cudaError_t launch_dx(GemmKind kind, const CUtensorMap& a, const CUtensorMap& b, const GemmGeom& g,
                      const DxArgs& ea, int* dev_err, int grid, cudaStream_t st) {
  return launch_any<DxEpi>(kind == kGemmWide ? kGemmPair : kind, a, b, g, ea, dev_err, grid, st);
}

}  // namespace flce
