// C ABI of the layer operators (declared in include/flce.h): argument checks,
// workspace carving, TMA descriptors and the launch sequence.
//
// Linear  forward   one GEMM, x W^T with bias, activation and residual in its epilogue
//         backward  dz = dy a'(z) with the bias gradient's column sums (no kernel
//                   without an activation and a bias: dz is dy), then the GEMMs
//                   dx = dz W and dW = dz^T x
// Gated   forward   one GEMM whose tiles hold both projections of the same outputs
//         backward  dg and du in one element-wise pass, then dx as one GEMM whose sum
//                   runs over both, and dWg and dWu as one GEMM over both
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "block_epilogues.cuh"
#include "block_internal.h"
#include "flce_host.h"

using namespace flce;

namespace {

constexpr int64_t kMaxTokens = 1LL << 30, kMaxFeatures = 1LL << 24;

bool act_ok(int32_t a) { return a >= FLCE_ACT_NONE && a <= FLCE_ACT_SIGMOID; }
bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1) == 0; }
bool flag_ok(int32_t f) { return f == 0 || f == 1; }
// A row pitch as given (0: dense).
int64_t pitch(int64_t ld, int64_t dense) { return ld == 0 ? dense : ld; }
bool pitch_ok(int64_t ld, int64_t dense) { return ld == 0 || ld >= dense; }

flce_status_t check_sizes(int64_t M, int64_t K, int64_t N) {
  if (M < 0 || K <= 0 || N <= 0) return FLCE_ERR_INVALID_ARG;
  if (K % 8 != 0) return FLCE_ERR_ALIGNMENT;  // 16-byte rows of x and W
  if (M > kMaxTokens || K > kMaxFeatures || N > kMaxFeatures) return FLCE_ERR_UNSUPPORTED;
  // Tile indices are int32: the 128 x 128 grids of the three products stay below 2^31.
  const int64_t m = (M + 127) / 128, k = (K + 127) / 128, n = 2 * ((N + 127) / 128);
  if (m * n >= (1LL << 31) || m * k >= (1LL << 31) || n * k >= (1LL << 31))
    return FLCE_ERR_UNSUPPORTED;
  return FLCE_OK;
}

flce_status_t check(const flce_linear_params_t* p) {
  if (!p) return FLCE_ERR_INVALID_ARG;
  const flce_status_t st = check_sizes(p->M, p->K, p->N);
  if (st != FLCE_OK) return st;
  if (!act_ok(p->activation) || !flag_ok(p->has_bias) || !flag_ok(p->has_residual) ||
      !flag_ok(p->input_fp16) || !flag_ok(p->dW_fp32) || !flag_ok(p->db_fp32))
    return FLCE_ERR_INVALID_ARG;
  if (!pitch_ok(p->ld_x, p->K) || !pitch_ok(p->ld_res, p->N) || !pitch_ok(p->ld_y, p->N))
    return FLCE_ERR_INVALID_ARG;
  return p->ld_x % 8 == 0 ? FLCE_OK : FLCE_ERR_ALIGNMENT;
}

flce_status_t check(const flce_gated_params_t* p) {
  if (!p) return FLCE_ERR_INVALID_ARG;
  const flce_status_t st = check_sizes(p->M, p->K, p->F);
  if (st != FLCE_OK) return st;
  if (p->F % 8 != 0) return FLCE_ERR_ALIGNMENT;
  if (!act_ok(p->activation) || !flag_ok(p->input_fp16) || !flag_ok(p->dW_fp32))
    return FLCE_ERR_INVALID_ARG;
  if (!pitch_ok(p->ld_x, p->K) || !pitch_ok(p->ld_h, p->F)) return FLCE_ERR_INVALID_ARG;
  return p->ld_x % 8 == 0 && p->ld_h % 8 == 0 ? FLCE_OK : FLCE_ERR_ALIGNMENT;
}

// An output and, where its rows start on 16-byte boundaries, its store map.
bool out16(Out16* o, void* ptr, int64_t rows, int64_t cols, int64_t ld) {
  std::memset(o, 0, sizeof(*o));
  o->ptr = static_cast<uint16_t*>(ptr);
  o->ld = ld;
  o->use_map = aligned16(ptr) && ld % 8 == 0 ? 1 : 0;
  return !o->use_map || encode_store_2d(&o->map, ptr, cols, rows, static_cast<uint64_t>(ld) * 2,
                                        false);
}

// K-major operand [rows, k]: boxes of 64 x 128. MN-major operand, the transpose
// of a row-major [k, rows] array: boxes of 64 x 64.
bool k_major(CUtensorMap* m, const void* p, int64_t rows, int64_t k, int64_t ld, bool f16) {
  return encode_2d(m, p, k, rows, static_cast<uint64_t>(ld) * 2, kBK, kBM, f16);
}
bool mn_major(CUtensorMap* m, const void* p, int64_t rows, int64_t k, int64_t ld, bool f16) {
  return encode_2d(m, p, rows, k, static_cast<uint64_t>(ld) * 2, 64, kBK, f16);
}

// Backward scratch of the linear layer: dz where it is not dy itself, and the
// bias gradient's partial sums.
struct LinearWs {
  uint16_t* dz;
  float* part;
  int64_t ld_dz;
};
size_t carve(const flce_linear_params_t* p, void* base, LinearWs* w) {
  Carver c(base, 0);
  w->ld_dz = (p->N + 7) / 8 * 8;
  // dy off the 16-byte boundaries also needs a copy: sized for it, since the
  // pointer is not known here.
  w->dz = c.take<uint16_t>(static_cast<size_t>(p->M) * w->ld_dz);
  w->part = p->has_bias ? c.take<float>(static_cast<size_t>(dz_parts(p->M, p->N)) * p->N) : nullptr;
  return c.used() + kAlign;
}

struct GatedWs {
  uint16_t *dg, *du;
};
size_t carve(const flce_gated_params_t* p, void* base, GatedWs* w) {
  Carver c(base, 0);
  w->dg = c.take<uint16_t>(static_cast<size_t>(p->M) * p->F);
  w->du = c.take<uint16_t>(static_cast<size_t>(p->M) * p->F);
  return c.used() + kAlign;
}

bool zero(void* p, size_t bytes, cudaStream_t s) {
  return !p || cudaMemsetAsync(p, 0, bytes, s) == cudaSuccess;
}

}  // namespace

extern "C" {

size_t flce_linear_workspace_size(const flce_linear_params_t* p, int which) {
  if (check(p) != FLCE_OK || p->M == 0 || which != 1) return 0;
  LinearWs w;
  return carve(p, nullptr, &w);
}

flce_status_t flce_linear_forward(const flce_linear_params_t* p, const void* x, const void* W,
                                  const void* b, const void* residual, void* y, void* pre,
                                  void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                  void* stream) {
  NvtxRange nvtx_range("flce_linear_forward");
  (void)workspace;
  (void)workspace_bytes;
  flce_status_t st = check(p);
  if (st != FLCE_OK) return st;
  if (p->M == 0) return FLCE_OK;
  if (!x || !W || !y || (p->has_bias && !b) || (p->has_residual && !residual))
    return FLCE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(W) || (p->has_bias && !aligned16(b)) || !aligned16(pre) ||
      !aligned2(y) || (p->has_residual && !aligned2(residual)))
    return FLCE_ERR_ALIGNMENT;
  int sms = 0;
  if ((st = device_info(&sms)) != FLCE_OK) return st;
  const bool f16 = p->input_fp16 != 0;
  const int M = static_cast<int>(p->M), K = static_cast<int>(p->K), N = static_cast<int>(p->N);

  LinearArgs ea;
  std::memset(&ea, 0, sizeof(ea));
  ea.bias = static_cast<const uint16_t*>(p->has_bias ? b : nullptr);
  ea.res = static_cast<const uint16_t*>(p->has_residual ? residual : nullptr);
  ea.ld_res = pitch(p->ld_res, N);
  ea.res_vec = aligned16(residual) && ea.ld_res % 8 == 0 ? 1 : 0;
  ea.act = p->activation;
  ea.fp16 = f16 ? 1 : 0;
  ea.keep = pre ? 1 : 0;
  ea.M = M;
  ea.N = N;
  CUtensorMap mx, mw;
  if (!out16(&ea.y, y, M, N, pitch(p->ld_y, N)) || (pre && !out16(&ea.z, pre, M, N, N)) ||
      !k_major(&mx, x, M, K, pitch(p->ld_x, K), f16) || !k_major(&mw, W, N, K, K, f16))
    return FLCE_ERR_CUDA;
  const GemmGeom g = geom(M, N, K, f16);
  return launch_linear(kGemmPair, mx, mw, g, ea, reinterpret_cast<int*>(dev_err), sms,
                       static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FLCE_OK
             : FLCE_ERR_CUDA;
}

flce_status_t flce_linear_backward(const flce_linear_params_t* p, const void* dy, const void* x,
                                   const void* W, const void* pre, void* dx, void* dW, void* db,
                                   void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                   void* stream) {
  NvtxRange nvtx_range("flce_linear_backward");
  flce_status_t st = check(p);
  if (st != FLCE_OK) return st;
  if (db && !p->has_bias) return FLCE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p->M == 0)
    return zero(dW, static_cast<size_t>(p->N) * p->K * (p->dW_fp32 ? 4 : 2), s) &&
                   zero(db, static_cast<size_t>(p->N) * (p->db_fp32 ? 4 : 2), s)
               ? FLCE_OK
               : FLCE_ERR_CUDA;
  if (!dx && !dW && !db) return FLCE_OK;
  const bool act = p->activation != FLCE_ACT_NONE;
  if (!dy || (dW && !x) || (dx && !W) || (act && !pre)) return FLCE_ERR_INVALID_ARG;
  if ((dW && !aligned16(x)) || (dx && !aligned16(W)) || (act && !aligned16(pre)) ||
      !aligned16(dx) || !aligned16(dW) || !aligned2(dy) ||
      (db && (reinterpret_cast<uintptr_t>(db) & (p->db_fp32 ? 3 : 1)) != 0))
    return FLCE_ERR_ALIGNMENT;
  LinearWs w;
  if (!workspace) return FLCE_ERR_INVALID_ARG;
  if (workspace_bytes < carve(p, nullptr, &w)) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  carve(p, workspace, &w);
  int sms = 0;
  if ((st = device_info(&sms)) != FLCE_OK) return st;
  const bool f16 = p->input_fp16 != 0;
  const int M = static_cast<int>(p->M), K = static_cast<int>(p->K), N = static_cast<int>(p->N);
  int* derr = reinterpret_cast<int*>(dev_err);

  const int64_t ld_dy = pitch(p->ld_y, N);
  const bool dy_rows16 = aligned16(dy) && ld_dy % 8 == 0;
  const bool copy = (act || !dy_rows16) && (dx || dW);
  if (copy || db) {
    DzArgs za;
    za.dy = static_cast<const uint16_t*>(dy);
    za.ld_dy = ld_dy;
    za.z = static_cast<const uint16_t*>(act ? pre : nullptr);
    za.dz = copy ? w.dz : nullptr;
    za.ld_dz = w.ld_dz;
    za.part = db ? w.part : nullptr;
    za.M = M;
    za.N = N;
    za.act = p->activation;
    za.fp16 = f16 ? 1 : 0;
    za.vec = dy_rows16 && (!act || N % 8 == 0) ? 1 : 0;
    if (launch_dz(za, s) != cudaSuccess) return FLCE_ERR_CUDA;
    if (db && launch_db_finalize(w.part, dz_parts(M, N), N, 0, N, db, p->db_fp32 != 0, f16, s) !=
                  cudaSuccess)
      return FLCE_ERR_CUDA;
  }
  const void* dz = copy ? static_cast<const void*>(w.dz) : dy;
  const int64_t ld_dz = copy ? w.ld_dz : ld_dy;
  if (dx) {
    GradXArgs ea;
    std::memset(&ea, 0, sizeof(ea));
    ea.fp16 = f16 ? 1 : 0;
    ea.M = M;
    ea.K = K;
    CUtensorMap ma, mb;
    if (!out16(&ea.dx, dx, M, K, K) || !k_major(&ma, dz, M, N, ld_dz, f16) ||
        !mn_major(&mb, W, K, N, K, f16))
      return FLCE_ERR_CUDA;
    const GemmGeom g = geom(M, K, N, f16);
    if (launch_grad_x(kGemmPair, false, ma, mb, g, ea, derr, sms, s) != cudaSuccess)
      return FLCE_ERR_CUDA;
  }
  if (dW) {
    GradWArgs ea;
    std::memset(&ea, 0, sizeof(ea));
    ea.out16 = p->dW_fp32 ? 0 : 1;
    ea.fp16 = f16 ? 1 : 0;
    ea.N = N;
    ea.K = K;
    CUtensorMap ma, mb;
    if (!encode_store_2d(&ea.out, dW, K, N, static_cast<uint64_t>(K) * (p->dW_fp32 ? 4 : 2),
                         p->dW_fp32 != 0) ||
        !mn_major(&ma, dz, N, M, ld_dz, f16) || !mn_major(&mb, x, K, M, pitch(p->ld_x, K), f16))
      return FLCE_ERR_CUDA;
    const GemmGeom g = geom(N, K, M, f16);
    if (launch_grad_w(kGemmPair, false, ma, mb, g, ea, derr, sms, s) != cudaSuccess)
      return FLCE_ERR_CUDA;
  }
  return FLCE_OK;
}

size_t flce_gated_workspace_size(const flce_gated_params_t* p, int which) {
  if (check(p) != FLCE_OK || p->M == 0 || which != 1) return 0;
  GatedWs w;
  return carve(p, nullptr, &w);
}

flce_status_t flce_gated_forward(const flce_gated_params_t* p, const void* x, const void* Wg,
                                 const void* Wu, void* h, void* pre, void* workspace,
                                 size_t workspace_bytes, int32_t* dev_err, void* stream) {
  NvtxRange nvtx_range("flce_gated_forward");
  (void)workspace;
  (void)workspace_bytes;
  flce_status_t st = check(p);
  if (st != FLCE_OK) return st;
  if (p->M == 0) return FLCE_OK;
  if (!x || !Wg || !Wu || !h) return FLCE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(Wg) || !aligned16(Wu) || !aligned16(h) || !aligned16(pre))
    return FLCE_ERR_ALIGNMENT;
  int sms = 0;
  if ((st = device_info(&sms)) != FLCE_OK) return st;
  const bool f16 = p->input_fp16 != 0;
  const int M = static_cast<int>(p->M), K = static_cast<int>(p->K), F = static_cast<int>(p->F);

  GatedArgs ea;
  std::memset(&ea, 0, sizeof(ea));
  ea.act = p->activation;
  ea.fp16 = f16 ? 1 : 0;
  ea.keep = pre ? 1 : 0;
  ea.M = M;
  ea.F = F;
  uint16_t* keep = static_cast<uint16_t*>(pre);
  CUtensorMap mx, mg;
  if (!out16(&ea.h, h, M, F, pitch(p->ld_h, F)) ||
      (pre && (!out16(&ea.g, keep, M, F, F) ||
               !out16(&ea.u, keep + static_cast<size_t>(M) * F, M, F, F))) ||
      !k_major(&mx, x, M, K, pitch(p->ld_x, K), f16) || !k_major(&mg, Wg, F, K, K, f16) ||
      !k_major(&ea.second.b2, Wu, F, K, K, f16))
    return FLCE_ERR_CUDA;
  GemmGeom g = geom(M, F, K, f16);
  g.tiles_n = cdiv(F, kBN / 2);  // a 256 x 256 pair tile holds 128 outputs
  return launch_gated(kGemmPair, mx, mg, g, ea, reinterpret_cast<int*>(dev_err), sms,
                      static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FLCE_OK
             : FLCE_ERR_CUDA;
}

flce_status_t flce_gated_backward(const flce_gated_params_t* p, const void* dh, const void* x,
                                  const void* Wg, const void* Wu, const void* pre, void* dx,
                                  void* dWg, void* dWu, void* workspace, size_t workspace_bytes,
                                  int32_t* dev_err, void* stream) {
  NvtxRange nvtx_range("flce_gated_backward");
  flce_status_t st = check(p);
  if (st != FLCE_OK) return st;
  if ((dWg == nullptr) != (dWu == nullptr)) return FLCE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p->M == 0) {
    const size_t bytes = static_cast<size_t>(p->F) * p->K * (p->dW_fp32 ? 4 : 2);
    return zero(dWg, bytes, s) && zero(dWu, bytes, s) ? FLCE_OK : FLCE_ERR_CUDA;
  }
  if (!dx && !dWg) return FLCE_OK;
  if (!dh || !pre || (dWg && !x) || (dx && (!Wg || !Wu)) || !workspace)
    return FLCE_ERR_INVALID_ARG;
  if (!aligned16(dh) || !aligned16(pre) || (dWg && !aligned16(x)) ||
      (dx && (!aligned16(Wg) || !aligned16(Wu))) || !aligned16(dx) || !aligned16(dWg) ||
      !aligned16(dWu))
    return FLCE_ERR_ALIGNMENT;
  GatedWs w;
  if (workspace_bytes < carve(p, nullptr, &w)) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  carve(p, workspace, &w);
  int sms = 0;
  if ((st = device_info(&sms)) != FLCE_OK) return st;
  const bool f16 = p->input_fp16 != 0;
  const int M = static_cast<int>(p->M), K = static_cast<int>(p->K), F = static_cast<int>(p->F);
  int* derr = reinterpret_cast<int*>(dev_err);

  GatedGradArgs ga;
  ga.dh = static_cast<const uint16_t*>(dh);
  ga.ld_dh = pitch(p->ld_h, F);
  ga.g = static_cast<const uint16_t*>(pre);
  ga.u = ga.g + static_cast<size_t>(M) * F;
  ga.dg = w.dg;
  ga.du = w.du;
  ga.M = M;
  ga.F = F;
  ga.act = p->activation;
  ga.fp16 = f16 ? 1 : 0;
  if (launch_gated_grad(ga, s) != cudaSuccess) return FLCE_ERR_CUDA;
  if (dx) {
    GradXArgs ea;
    std::memset(&ea, 0, sizeof(ea));
    ea.fp16 = f16 ? 1 : 0;
    ea.M = M;
    ea.K = K;
    CUtensorMap ma, mb;
    if (!out16(&ea.dx, dx, M, K, K) || !k_major(&ma, w.dg, M, F, F, f16) ||
        !k_major(&ea.second.a2, w.du, M, F, F, f16) || !mn_major(&mb, Wg, K, F, K, f16) ||
        !mn_major(&ea.second.b2, Wu, K, F, K, f16))
      return FLCE_ERR_CUDA;
    GemmGeom g = geom(M, K, F, f16);
    ea.second.k_split = g.k_blocks;
    g.k_blocks *= 2;
    if (launch_grad_x(kGemmPair, true, ma, mb, g, ea, derr, sms, s) != cudaSuccess)
      return FLCE_ERR_CUDA;
  }
  if (dWg) {
    GradWArgs ea;
    std::memset(&ea, 0, sizeof(ea));
    ea.out16 = p->dW_fp32 ? 0 : 1;
    ea.fp16 = f16 ? 1 : 0;
    ea.N = F;
    ea.K = K;
    const uint64_t row = static_cast<uint64_t>(K) * (p->dW_fp32 ? 4 : 2);
    CUtensorMap ma, mb;
    if (!encode_store_2d(&ea.out, dWg, K, F, row, p->dW_fp32 != 0) ||
        !encode_store_2d(&ea.out2, dWu, K, F, row, p->dW_fp32 != 0) ||
        !mn_major(&ma, w.dg, F, M, F, f16) || !mn_major(&ea.second.a2, w.du, F, M, F, f16) ||
        !mn_major(&mb, x, K, M, pitch(p->ld_x, K), f16))
      return FLCE_ERR_CUDA;
    GemmGeom g = geom(F, K, M, f16);
    ea.second.m_split = cdiv(F, 2 * kBM);
    g.tiles_m = 4 * ea.second.m_split;  // both gradients, in 128-row units
    if (launch_grad_w(kGemmPair, true, ma, mb, g, ea, derr, sms, s) != cudaSuccess)
      return FLCE_ERR_CUDA;
  }
  return FLCE_OK;
}

}  // extern "C"
