// GEMM instantiations of the layer operators.
#include "block_epilogues.cuh"
#include "block_internal.h"
#include "gemm_launch.cuh"

namespace flce {

template <class Epi>
static cudaError_t launch_pairs(GemmKind kind, const CUtensorMap& a, const CUtensorMap& b,
                                const GemmGeom& g, const typename Epi::Args& ea, int* dev_err,
                                int sms, cudaStream_t st) {
  return kind == kGemmWide ? launch_wide<Epi>(a, b, g, ea, dev_err, sms, st)
                           : launch_pair<Epi>(a, b, g, ea, dev_err, sms, st);
}

cudaError_t launch_linear(GemmKind kind, const CUtensorMap& a, const CUtensorMap& b,
                          const GemmGeom& g, const LinearArgs& ea, int* dev_err, int sms,
                          cudaStream_t st) {
  return launch_pairs<LinearEpi>(kind, a, b, g, ea, dev_err, sms, st);
}

cudaError_t launch_gated(GemmKind kind, const CUtensorMap& a, const CUtensorMap& b,
                         const GemmGeom& g, const GatedArgs& ea, int* dev_err, int sms,
                         cudaStream_t st) {
  return launch_pairs<GatedEpi>(kind, a, b, g, ea, dev_err, sms, st);
}

cudaError_t launch_grad_x(GemmKind kind, bool two, const CUtensorMap& a, const CUtensorMap& b,
                          const GemmGeom& g, const GradXArgs& ea, int* dev_err, int sms,
                          cudaStream_t st) {
  return two ? launch_pairs<GradXEpi<kTwoK>>(kind, a, b, g, ea, dev_err, sms, st)
             : launch_pairs<GradXEpi<kOneEach>>(kind, a, b, g, ea, dev_err, sms, st);
}

cudaError_t launch_grad_w(GemmKind kind, bool two, const CUtensorMap& a, const CUtensorMap& b,
                          const GemmGeom& g, const GradWArgs& ea, int* dev_err, int sms,
                          cudaStream_t st) {
  return two ? launch_pairs<GradWEpi<kTwoA>>(kind, a, b, g, ea, dev_err, sms, st)
             : launch_pairs<GradWEpi<kOneEach>>(kind, a, b, g, ea, dev_err, sms, st);
}

}  // namespace flce
