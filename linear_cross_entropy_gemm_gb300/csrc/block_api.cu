// C ABI of the layer operators (declared in include/flce.h): argument checks,
// workspace carving, TMA descriptors and the launch sequence.
//
// Linear  forward   one GEMM, x W^T with bias, activation and residual in its epilogue
//         backward  dz = dy a'(z) from the kept slopes, with the bias gradient's column sums (no kernel
//                   without an activation and a bias: dz is dy), then the GEMMs
//                   dx = dz W and dW = dz^T x
// Gated   forward   one GEMM whose tiles hold both projections of the same outputs
//         backward  dg and du in one element-wise pass, then dx as one GEMM whose sum
//                   runs over both, and dWg and dWu as one GEMM over both
#include <algorithm>
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
bool keep_ok(int32_t k) { return k == FLCE_KEEP_FIXED || k == FLCE_KEEP_RELATIVE; }
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
      !flag_ok(p->input_fp16) || !flag_ok(p->dW_fp32) || !flag_ok(p->db_fp32) ||
      !keep_ok(p->keep))
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
  if (!act_ok(p->activation) || !flag_ok(p->input_fp16) || !flag_ok(p->dW_fp32) ||
      !keep_ok(p->keep))
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

// K-major operand [rows, k]: boxes of 64 x 128 (or fewer rows). MN-major operand, the
// transpose of a row-major [k, rows] array: boxes of 64 x 128, or 64 x 64 for the
// few-token kernel.
bool k_major(CUtensorMap* m, const void* p, int64_t rows, int64_t k, int64_t ld, bool f16,
             int box = kBM) {
  return encode_2d(m, p, k, rows, static_cast<uint64_t>(ld) * 2, kBK, static_cast<uint32_t>(box),
                   f16);
}
bool mn_major(CUtensorMap* m, const void* p, int64_t rows, int64_t k, int64_t ld, bool f16,
              int box) {
  return encode_2d(m, p, rows, k, static_cast<uint64_t>(ld) * 2, 64, static_cast<uint32_t>(box),
                   f16);
}

// The parts of a few-token product's arguments that do not depend on the operator.
// x: [M, k] with pitch ld_x; the sum runs over `segments` times k.
bool small_args(SmallArgs* a, const void* x, int64_t ld_x, int64_t M, int64_t k, int segments,
                int64_t N, void* y, int64_t ld_y, bool two, bool f16, int32_t* dev_err) {
  std::memset(a, 0, sizeof(*a));
  a->y = static_cast<uint16_t*>(y);
  a->ld_y = ld_y;
  a->y_vec = aligned16(y) && ld_y % 8 == 0 ? 1 : 0;
  a->fp16 = f16 ? 1 : 0;
  a->M = static_cast<int>(M);
  a->N = static_cast<int>(N);
  a->k_split = cdiv(k, kBK);
  a->k_blocks = segments * a->k_split;
  a->slices = small_slices(M, N, a->k_blocks, two);
  a->dev_err = reinterpret_cast<int*>(dev_err);
  a->xp = static_cast<const uint16_t*>(x);
  a->ld_x = ld_x;
  a->k_len = static_cast<int>(k);
  return small_tokens(M) <= 32 || k_major(&a->x, x, M, k, ld_x, f16, small_tokens(M));
}

// ------------------------------------------------- tile width of a pair GEMM
// A tile shape (pair_engine.cuh) and the ns it takes for 64 sum elements with a K-major
// and with an MN-major B, whose boxes are 64 columns wide, so that only widths in
// multiples of 128 load nothing twice.
//
// The numbers below are fitted to the choice they are for: about 1300 products of 140 to
// 4096 rows, 64 to 5000 sum elements and 256 to 12800 columns, of all kinds, each timed in
// every shape. Of 500 others the choice (with the one below) is 2.0 % slower than the
// fastest shape on average, none above 21 %; with rates of single waves and an epilogue
// priced by its activation it was 6 % (gated 9 %, up to 81 %). Widths of 160, 208 and 240
// gained less than 0.2 %.
struct TileShape {
  int halves, bn, slices;
  float ns, ns_mn;  // 0: not used with that B
};
constexpr TileShape kTileShapes[] = {
    {1, 256, 1, 296.f, 296.f}, {1, 224, 1, 290.f, 0.f},   {1, 192, 1, 285.f, 0.f},
    {1, 128, 1, 192.f, 200.f}, {1, 64, 1, 186.f, 280.f},  {2, 256, 1, 0.f, 555.f},
    {2, 192, 1, 0.f, 505.f},   {1, 256, 2, 296.f, 296.f}, {1, 128, 2, 192.f, 200.f},
    {1, 192, 3, 285.f, 0.f},
};
// Clusters of 2, 4 and 6 CTAs of 225 KiB that run at once on 152 SMs, as the runtime
// says (of 8 CTAs it is 15).
constexpr int kClusters[] = {76, 36, 23};
constexpr float kSustained[] = {1.66e6f, 1.75e6f};  // flop/ns under the power cap, by halves
constexpr float kWaveNs = 1400.f;   // of a wave of tiles, beside their sums
constexpr float kWideNs = 600.f;    // the same of two-half tiles
constexpr float kJoinNs = 3900.f;   // exchange of a split tile
constexpr float kSetUpNs = 3600.f;  // start and drain of each further wave of split tiles
// Epilogue ns of an output column; of the gated forward's, which are two sums.
constexpr float kColumnNs = 9.5f, kGatedColumnNs = 16.5f;

// ns of a whole product: its waves of tiles, each as long as the sum or (where it
// runs beside the next tile's sum) the epilogue; the last epilogue; and no less than
// the padded flops take under the power cap. The two-half form, whose epilogue is not
// overlapped, is kept to the weight and input gradients: at 8192 x 28672 x 4096 (gated)
// it took 1213 us against 1133 us, for dW 4096 x 14336 x 8192 549 us against 579 us.
// Split sums pay where the tiles are few: 512 x 4096 x 14336 46 us against 61 us.
float tile_ns(const TileShape& t, bool mn, int64_t tiles_m, int64_t N, int64_t k64, bool two_b) {
  const int cols = pair_cols(two_b ? kTwoB : kOneEach, t.halves, t.bn);
  const int64_t tiles = tiles_m * ((N + cols - 1) / cols);
  const int at_once = kClusters[t.slices - 1];
  const float waves = static_cast<float>((tiles + at_once - 1) / at_once);
  const float sum = static_cast<float>(k64) * (mn ? t.ns_mn : t.ns) / static_cast<float>(t.slices);
  const float epi = (two_b ? kGatedColumnNs : kColumnNs) *
                    static_cast<float>(std::min<int64_t>(cols, N)) / static_cast<float>(t.slices);
  const float busy = t.slices > 1    ? waves * (sum + kJoinNs + epi) + (waves - 1.f) * kSetUpNs
                     : t.halves == 1 ? waves * std::max(sum + kWaveNs, epi) + epi
                                     : waves * (sum + epi + kWideNs);
  const float flops = 2.f * 256.f * 64.f * t.halves * t.bn * static_cast<float>(tiles) * k64;
  return std::max(busy, flops / kSustained[t.halves - 1]);
}

// Whether the shape can compute the product: every slice has a stage of the sum, and every
// pair of a split tile output columns.
bool tile_fits(const TileShape& t, bool mn, int64_t k64, bool two_b) {
  if ((mn ? t.ns_mn : t.ns) == 0.f) return false;
  if (t.slices == 1) return true;
  return (k64 + 1) / 2 >= t.slices && t.bn / 32 % (t.slices * (two_b ? 2 : 1)) == 0;
}

const TileShape& best_tile(bool mn, int64_t M, int64_t N, int64_t k64, bool two_b) {
  const TileShape* best = nullptr;
  float least = 0.f;
  for (const TileShape& t : kTileShapes) {
    if (!tile_fits(t, mn, k64, two_b)) continue;
    const float ns = tile_ns(t, mn, (M + 255) / 256, N, k64, two_b);
    if (!best || ns < least) {
      best = &t;
      least = ns;
    }
  }
  return *best;
}

// Products of at most this many tokens go to the few-token kernel: of 130 products of 33 to 64
// tokens it takes 1.03 of the faster kernel's time on average, CTA pairs 1.28 to 1.39. (Of 230
// of 65 to 128 tokens 1.09 to 1.13 and 1.15 to 1.21, the choice below 1.004 to 1.02.)
constexpr int64_t kSmallTokens = 64;

// And larger ones with few tiles of a long sum, which that kernel cuts into eight slices:
// 267 x 376 x 12800 25 us by CTA pairs (four tiles, three slices), 13 us. Its ns for 64 sum
// elements and the rest of it are fitted like the shapes' above: of 300 products of 70 to
// 1024 rows, sums of 720 to 16384 and 128 to 2900 columns the choice is 0.5 % slower than the
// faster kernel on average, CTA pairs for all of them 13 %. In one wave of clusters only: of
// eight CTAs 15 run at once, and a second wave of them doubled 251 x 1032 x 1312's time.
constexpr float kSmallNs = 300.f, kSmallRestNs = 4500.f;
bool few_tokens(bool mn, int64_t M, int64_t N, int64_t k64, bool two_b) {
  if (M <= kSmallTokens) return true;
  const int slices = small_slices(M, N, static_cast<int>(k64), two_b);
  if (small_tiles(M, N, two_b) > small_clusters(M, slices)) return false;
  const float ns = static_cast<float>((k64 + slices - 1) / slices) * kSmallNs + kSmallRestNs;
  const TileShape& t = best_tile(mn, M, N, k64, two_b);
  return ns < tile_ns(t, mn, (M + 255) / 256, N, k64, two_b);
}

// The geometry of a pair GEMM D[M, N] with a sum of K (`segments` of them): tile shape and
// raster. Bands of 16 row tiles keep 4096 rows of A in L2 while B streams: at 8192 x
// 4096 x 14336, 573 us against 596 us with bands of 8 column tiles.
PairArgs pair_args(int M, int N, int K, int segments, bool mn, bool two_b, bool f16,
                   int32_t* dev_err) {
  PairArgs g;
  std::memset(&g, 0, sizeof(g));
  const TileShape& t = best_tile(mn, M, N, static_cast<int64_t>(segments) * cdiv(K, 64), two_b);
  g.halves = t.halves;
  g.slices = t.slices;
  g.bn = t.bn;
  g.band_m = 16;
  g.tiles_m = cdiv(M, 256);
  g.tiles_n = cdiv(N, pair_cols(two_b ? kTwoB : kOneEach, g.halves, g.bn));
  g.k_split = cdiv(K, pair_lk(g.halves));
  g.k_stages = segments * g.k_split;
  g.fp16 = f16 ? 1 : 0;
  g.dev_err = reinterpret_cast<int*>(dev_err);
  return g;
}

flce_status_t done(cudaError_t e) { return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA; }

// ----------------------------------------------- operands in scratch memory
// The pair GEMM takes an operand from a repacked copy where its own pitch costs more
// than the copy:
//   - Loads through a TMA map whose tensor spans less than 128 KiB run up to several times
//     slower when many SMs share it (measured with the same boxes and bytes: 94 us with
//     15 rows of 8 KiB, 20 us with 16; a dW of 8 x 4096 over 2048 tokens 32 us, 13 us with
//     both operands spread): the copy's rows lie far enough apart.
//   - Rows that start between 32-byte sectors (a pitch of 8 elements modulo 16) cost an
//     operand about a third of the product's time: 2048 x 4096 x 4104 70 us, 54 us with
//     x repacked, against 42 us at 4096. (A pitch of 16 modulo 32 costs a tenth: left.)
constexpr int64_t kSpreadElems = 131072 / 2;  // from a tensor's first element to its last
constexpr int64_t kManyTiles = 32;            // SMs enough to slow a narrow tensor's loads
constexpr float kOddRowsShare = 0.3f;
constexpr float kCopyNs = 2500.f, kCopyBytesNs = 5500.f;  // a launch; bytes read and written a ns

bool is_narrow(int64_t rows, int64_t cols, int64_t ld) {
  return rows > 1 && (rows - 1) * ld + cols < kSpreadElems;
}
// A pitch for rows in scratch memory: whole 128-byte lines, and not narrow.
int64_t scratch_ld(int64_t rows, int64_t cols) {
  int64_t ld = (cols + 63) / 64 * 64;
  if (is_narrow(rows, cols, ld)) {
    const int64_t apart = (kSpreadElems - cols + rows - 2) / (rows - 1);
    ld = (apart + 63) / 64 * 64;
  }
  return ld;
}
// A product that reads an operand: what it takes, and its tiles.
struct Product {
  float ns;
  int64_t tiles;
};
// The pitch of a repacked copy of [rows, cols] with pitch ld; 0: read it as it is.
int64_t repack_ld(int64_t rows, int64_t cols, int64_t ld, const Product& by) {
  const bool narrow = by.tiles >= kManyTiles && is_narrow(rows, cols, ld);
  const float copy = kCopyNs + 4.f * static_cast<float>(rows) * static_cast<float>(cols) / kCopyBytesNs;
  const bool odd = rows > 1 && ld % 16 != 0 && kOddRowsShare * by.ns > copy;
  return narrow || odd ? scratch_ld(rows, cols) : 0;
}
Product product_of(bool mn, int64_t M, int64_t N, int64_t k64, bool two_b) {
  const TileShape& t = best_tile(mn, M, N, k64, two_b);
  const int cols = pair_cols(two_b ? kTwoB : kOneEach, t.halves, t.bn);
  return {tile_ns(t, mn, (M + 255) / 256, N, k64, two_b),
          (M + 255) / 256 * ((N + cols - 1) / cols) * t.slices};
}

// p [rows, cols] with pitch *ld, or its copy in `buf` with the pitch `to` (0: none).
const void* repacked(const void* p, int64_t rows, int64_t cols, int64_t* ld, int64_t to,
                     uint16_t* buf, cudaStream_t s, cudaError_t* e) {
  if (*e != cudaSuccess || to == 0) return p;
  *e = launch_repack(static_cast<const uint16_t*>(p), *ld, buf, to, static_cast<int>(rows),
                     static_cast<int>(cols), s);
  *ld = to;
  return buf;
}

// The bytes of a workspace that `c` has carved, at whatever address it lies.
size_t bytes_of(const Carver& c) { return c.cur - (c.base + kAlign - 1) / kAlign * kAlign + kAlign; }

uint16_t* take_rows(Carver* c, int64_t rows, int64_t ld) {
  return ld > 0 ? c->take<uint16_t>(static_cast<size_t>(rows) * static_cast<size_t>(ld)) : nullptr;
}

// Scratch of the linear layer. Forward: repacked x and W. Backward: dz where it is not dy
// itself, the bias gradient's partial sums, and x and W repacked. The pitches (0: no
// copy) depend on the parameters alone.
struct LinearWs {
  uint16_t *dz, *x, *W;
  float* part;
  int64_t ld_dz, ld_x, ld_w;
  bool repack_dy;  // dy is better copied, even where dz is dy
  bool copy;       // dz is not dy itself
  bool few;        // forward, dx: by the few-token kernel
};
size_t carve_forward(const flce_linear_params_t* p, void* base, LinearWs* w) {
  std::memset(w, 0, sizeof(*w));
  const int64_t k64 = (p->K + 63) / 64;
  if ((w->few = few_tokens(false, p->M, p->N, k64, false))) return 0;
  const Product by = product_of(false, p->M, p->N, k64, false);
  w->ld_x = repack_ld(p->M, p->K, pitch(p->ld_x, p->K), by);
  w->ld_w = repack_ld(p->N, p->K, p->K, by);
  if (w->ld_x == 0 && w->ld_w == 0) return 0;
  Carver c(base, 0);
  w->x = take_rows(&c, p->M, w->ld_x);
  w->W = take_rows(&c, p->N, w->ld_w);
  return bytes_of(c);
}
size_t carve(const flce_linear_params_t* p, void* base, bool dy_aligned, LinearWs* w) {
  std::memset(w, 0, sizeof(*w));
  const int64_t n64 = (p->N + 63) / 64;
  w->few = few_tokens(true, p->M, p->K, n64, false);
  const Product dx = w->few ? Product{0.f, 0} : product_of(true, p->M, p->K, n64, false);
  const Product dw = product_of(true, p->N, p->K, (p->M + 63) / 64, false);
  w->ld_w = repack_ld(p->N, p->K, p->K, dx);
  w->ld_x = repack_ld(p->M, p->K, pitch(p->ld_x, p->K), dw);
  w->ld_dz = scratch_ld(p->M, p->N);
  w->repack_dy = repack_ld(p->M, p->N, pitch(p->ld_y, p->N),
                           {dx.ns + dw.ns, std::max(dx.tiles, dw.tiles)}) != 0;
  w->copy = p->activation != FLCE_ACT_NONE || w->repack_dy || !dy_aligned ||
            pitch(p->ld_y, p->N) % 8 != 0;
  Carver c(base, 0);
  w->dz = take_rows(&c, p->M, w->copy ? w->ld_dz : 0);
  w->part = p->has_bias ? c.take<float>(static_cast<size_t>(dz_parts(p->M, p->N)) * p->N) : nullptr;
  w->x = take_rows(&c, p->M, w->ld_x);
  w->W = take_rows(&c, p->N, w->ld_w);
  return bytes_of(c);
}

// Scratch of the gated projection. Forward: repacked x, Wg and Wu. Backward: dg and du,
// and the operands repacked.
struct GatedWs {
  uint16_t *dg, *du, *x, *Wg, *Wu;
  int64_t ld, ld_x, ld_w;  // ld: of dg and du
  bool few;                // forward, dx: by the few-token kernel
};
size_t carve_forward(const flce_gated_params_t* p, void* base, GatedWs* w) {
  std::memset(w, 0, sizeof(*w));
  const int64_t k64 = (p->K + 63) / 64;
  if ((w->few = few_tokens(false, p->M, p->F, k64, true))) return 0;
  const Product by = product_of(false, p->M, p->F, k64, true);
  w->ld_x = repack_ld(p->M, p->K, pitch(p->ld_x, p->K), by);
  w->ld_w = repack_ld(2 * p->F, p->K, p->K, by) != 0 ? scratch_ld(p->F, p->K) : 0;
  if (w->ld_x == 0 && w->ld_w == 0) return 0;
  Carver c(base, 0);
  w->x = take_rows(&c, p->M, w->ld_x);
  w->Wg = take_rows(&c, p->F, w->ld_w);
  w->Wu = take_rows(&c, p->F, w->ld_w);
  return bytes_of(c);
}
size_t carve(const flce_gated_params_t* p, void* base, GatedWs* w) {
  std::memset(w, 0, sizeof(*w));
  const int64_t f64 = 2 * ((p->F + 63) / 64);
  w->few = few_tokens(true, p->M, p->K, f64, false);
  const Product dx = w->few ? Product{0.f, 0} : product_of(true, p->M, p->K, f64, false);
  const Product dw = product_of(true, 2 * p->F, p->K, (p->M + 63) / 64, false);
  w->ld = scratch_ld(p->M, p->F);
  w->ld_w = repack_ld(2 * p->F, p->K, p->K, dx) != 0 ? scratch_ld(p->F, p->K) : 0;
  w->ld_x = repack_ld(p->M, p->K, pitch(p->ld_x, p->K), dw);
  Carver c(base, 0);
  w->dg = take_rows(&c, p->M, w->ld);
  w->du = take_rows(&c, p->M, w->ld);
  w->x = take_rows(&c, p->M, w->ld_x);
  w->Wg = take_rows(&c, p->F, w->ld_w);
  w->Wu = take_rows(&c, p->F, w->ld_w);
  return bytes_of(c);
}

// What launch of D[M, N] (pair_args, small_args) a product takes.
flce_plan_t plan_of(bool few, bool mn, int64_t M, int64_t N, int64_t k64, bool two_b) {
  flce_plan_t r;
  std::memset(&r, 0, sizeof(r));
  if (few) {
    r.few_tokens = small_tokens(M);
    r.slices = small_slices(M, N, static_cast<int>(k64), two_b);
    return r;
  }
  const TileShape& t = best_tile(mn, M, N, k64, two_b);
  r.halves = t.halves;
  r.columns = t.bn;
  r.slices = t.slices;
  return r;
}

bool zero(void* p, size_t bytes, cudaStream_t s) {
  return !p || cudaMemsetAsync(p, 0, bytes, s) == cudaSuccess;
}

}  // namespace

extern "C" {

size_t flce_linear_workspace_size(const flce_linear_params_t* p, int which) {
  if (check(p) != FLCE_OK || p->M == 0 || which < 0 || which > 2) return 0;
  LinearWs w;
  return which == 0 ? carve_forward(p, nullptr, &w) : carve(p, nullptr, which == 2, &w);
}

flce_status_t flce_linear_plan(const flce_linear_params_t* p, int product, flce_plan_t* plan) {
  const flce_status_t st = check(p);
  if (st != FLCE_OK) return st;
  if (!plan || product < 0 || product > 2 || p->M == 0) return FLCE_ERR_INVALID_ARG;
  const int64_t m64 = (p->M + 63) / 64, k64 = (p->K + 63) / 64, n64 = (p->N + 63) / 64;
  *plan = product == 0 ? plan_of(few_tokens(false, p->M, p->N, k64, false), false, p->M, p->N, k64, false)
        : product == 1 ? plan_of(few_tokens(true, p->M, p->K, n64, false), true, p->M, p->K, n64, false)
                       : plan_of(false, true, p->N, p->K, m64, false);
  return FLCE_OK;
}

flce_status_t flce_linear_forward(const flce_linear_params_t* p, const void* x, const void* W,
                                  const void* b, const void* residual, void* y, void* pre,
                                  void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                  void* stream) {
  NvtxRange nvtx_range("flce_linear_forward");
  flce_status_t st = check(p);
  if (st != FLCE_OK) return st;
  if (p->M == 0) return FLCE_OK;
  if (!x || !W || !y || (p->has_bias && !b) || (p->has_residual && !residual))
    return FLCE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(W) || (p->has_bias && !aligned16(b)) || !aligned16(pre) ||
      !aligned2(y) || (p->has_residual && !aligned2(residual)))
    return FLCE_ERR_ALIGNMENT;
  LinearWs w;
  const size_t need = carve_forward(p, workspace, &w);
  if (need > 0 && !workspace) return FLCE_ERR_INVALID_ARG;
  if (workspace_bytes < need) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  if ((st = device_info(&sms)) != FLCE_OK) return st;
  const bool f16 = p->input_fp16 != 0;
  const int M = static_cast<int>(p->M), K = static_cast<int>(p->K), N = static_cast<int>(p->N);
  if (w.few) {
    SmallArgs sa;
    if (!small_args(&sa, x, pitch(p->ld_x, K), M, K, 1, N, y, pitch(p->ld_y, N), false, f16, dev_err) ||
        !k_major(&sa.w, W, N, K, K, f16))
      return FLCE_ERR_CUDA;
    sa.bias = static_cast<const uint16_t*>(p->has_bias ? b : nullptr);
    sa.res = static_cast<const uint16_t*>(p->has_residual ? residual : nullptr);
    sa.ld_res = pitch(p->ld_res, N);
    sa.res_vec = aligned16(residual) && sa.ld_res % 8 == 0 ? 1 : 0;
    sa.keep = static_cast<uint16_t*>(pre);
    sa.relative = p->keep == FLCE_KEEP_RELATIVE ? 1 : 0;
    sa.wp = static_cast<const uint16_t*>(W);
    sa.act = p->activation;
    return done(launch_small(false, false, sa, static_cast<cudaStream_t>(stream)));
  }

  LinearArgs ea;
  std::memset(&ea, 0, sizeof(ea));
  ea.bias = static_cast<const uint16_t*>(p->has_bias ? b : nullptr);
  ea.res = static_cast<const uint16_t*>(p->has_residual ? residual : nullptr);
  ea.ld_res = pitch(p->ld_res, N);
  ea.res_vec = aligned16(residual) && ea.ld_res % 8 == 0 ? 1 : 0;
  ea.act = p->activation;
  ea.fp16 = f16 ? 1 : 0;
  ea.keep = !pre ? 0 : p->keep == FLCE_KEEP_RELATIVE ? 2 : 1;
  ea.M = M;
  ea.N = N;
  ea.sign = {static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(W), ea.bias,
             pitch(p->ld_x, K), K};
  PairArgs g = pair_args(M, N, K, 1, false, false, f16, dev_err);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  int64_t ld_x = pitch(p->ld_x, K), ld_w = K;
  const void* xn = repacked(x, M, K, &ld_x, w.ld_x, w.x, s, &e);
  const void* Wn = repacked(W, N, K, &ld_w, w.ld_w, w.W, s, &e);
  if (e != cudaSuccess || !out16(&ea.y, y, M, N, pitch(p->ld_y, N)) ||
      (pre && !out16(&ea.slope, pre, M, N, N)) || !k_major(&g.a, xn, M, K, ld_x, f16) ||
      !k_major(&g.b, Wn, N, K, ld_w, f16, g.bn / 2))
    return FLCE_ERR_CUDA;
  return done(launch_linear(g, ea, sms, s));
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
  if (workspace_bytes < carve(p, workspace, aligned16(dy), &w))
    return FLCE_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  if ((st = device_info(&sms)) != FLCE_OK) return st;
  const bool f16 = p->input_fp16 != 0;
  const int M = static_cast<int>(p->M), K = static_cast<int>(p->K), N = static_cast<int>(p->N);

  const int64_t ld_dy = pitch(p->ld_y, N);
  const bool dy_rows16 = aligned16(dy) && ld_dy % 8 == 0;
  const bool copy = w.copy && (dx || dW);
  if (copy || db) {
    DzArgs za;
    za.dy = static_cast<const uint16_t*>(dy);
    za.ld_dy = ld_dy;
    za.slope = static_cast<const uint16_t*>(act ? pre : nullptr);
    za.dz = copy ? w.dz : nullptr;
    za.ld_dz = w.ld_dz;
    za.part = db ? w.part : nullptr;
    za.M = M;
    za.N = N;
    za.fp16 = f16 ? 1 : 0;
    za.tail = p->activation == FLCE_ACT_SIGMOID ? 0x1p82f : -0x1p82f;
    za.vec = dy_rows16 && (!act || N % 8 == 0) ? 1 : 0;
    if (launch_dz(za, s) != cudaSuccess) return FLCE_ERR_CUDA;
    if (db && launch_db_sum(w.part, dz_parts(M, N), N, db, p->db_fp32 != 0, f16, s) != cudaSuccess)
      return FLCE_ERR_CUDA;
  }
  const void* dz = copy ? static_cast<const void*>(w.dz) : dy;
  const int64_t ld_dz = copy ? w.ld_dz : ld_dy;
  cudaError_t e = cudaSuccess;
  if (dx && w.few) {
    SmallArgs sa;
    if (!small_args(&sa, dz, ld_dz, M, N, 1, K, dx, K, false, f16, dev_err) ||
        !mn_major(&sa.w, W, K, N, K, f16, kBK) || launch_small(false, true, sa, s) != cudaSuccess)
      return FLCE_ERR_CUDA;
  } else if (dx) {
    GradXArgs ea;
    std::memset(&ea, 0, sizeof(ea));
    ea.fp16 = f16 ? 1 : 0;
    ea.M = M;
    ea.K = K;
    PairArgs g = pair_args(M, K, N, 1, true, false, f16, dev_err);
    int64_t ld_w = K;
    const void* Wn = repacked(W, N, K, &ld_w, w.ld_w, w.W, s, &e);
    if (!out16(&ea.dx, dx, M, K, K) || !k_major(&g.a, dz, M, N, ld_dz, f16) ||
        !mn_major(&g.b, Wn, K, N, ld_w, f16, pair_lk(g.halves)) || e != cudaSuccess ||
        launch_grad_x(false, g, ea, sms, s) != cudaSuccess)
      return FLCE_ERR_CUDA;
  }
  if (dW) {
    GradWArgs ea;
    std::memset(&ea, 0, sizeof(ea));
    ea.out16 = p->dW_fp32 ? 0 : 1;
    ea.fp16 = f16 ? 1 : 0;
    ea.N = N;
    ea.K = K;
    PairArgs g = pair_args(N, K, M, 1, true, false, f16, dev_err);
    int64_t ld_x = pitch(p->ld_x, K);
    const void* xn = repacked(x, M, K, &ld_x, w.ld_x, w.x, s, &e);
    if (!encode_store_2d(&ea.out, dW, K, N, static_cast<uint64_t>(K) * (p->dW_fp32 ? 4 : 2),
                         p->dW_fp32 != 0) ||
        !mn_major(&g.a, dz, N, M, ld_dz, f16, pair_lk(g.halves)) ||
        !mn_major(&g.b, xn, K, M, ld_x, f16, pair_lk(g.halves)) || e != cudaSuccess ||
        launch_grad_w(false, g, ea, sms, s) != cudaSuccess)
      return FLCE_ERR_CUDA;
  }
  return FLCE_OK;
}

size_t flce_gated_workspace_size(const flce_gated_params_t* p, int which) {
  if (check(p) != FLCE_OK || p->M == 0 || which < 0 || which > 1) return 0;
  GatedWs w;
  return which == 0 ? carve_forward(p, nullptr, &w) : carve(p, nullptr, &w);
}

flce_status_t flce_gated_plan(const flce_gated_params_t* p, int product, flce_plan_t* plan) {
  const flce_status_t st = check(p);
  if (st != FLCE_OK) return st;
  if (!plan || product < 0 || product > 2 || p->M == 0) return FLCE_ERR_INVALID_ARG;
  const int64_t m64 = (p->M + 63) / 64, k64 = (p->K + 63) / 64, f64 = 2 * ((p->F + 63) / 64);
  const int64_t rows = 2 * ((p->F + 255) / 256) * 256;  // of dWg and dWu, each to whole tiles
  *plan = product == 0 ? plan_of(few_tokens(false, p->M, p->F, k64, true), false, p->M, p->F, k64, true)
        : product == 1 ? plan_of(few_tokens(true, p->M, p->K, f64, false), true, p->M, p->K, f64, false)
                       : plan_of(false, true, rows, p->K, m64, false);
  return FLCE_OK;
}

flce_status_t flce_gated_forward(const flce_gated_params_t* p, const void* x, const void* Wg,
                                 const void* Wu, void* h, void* pre, void* workspace,
                                 size_t workspace_bytes, int32_t* dev_err, void* stream) {
  NvtxRange nvtx_range("flce_gated_forward");
  flce_status_t st = check(p);
  if (st != FLCE_OK) return st;
  if (p->M == 0) return FLCE_OK;
  if (!x || !Wg || !Wu || !h) return FLCE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(Wg) || !aligned16(Wu) || !aligned16(h) || !aligned16(pre))
    return FLCE_ERR_ALIGNMENT;
  GatedWs w;
  const size_t need = carve_forward(p, workspace, &w);
  if (need > 0 && !workspace) return FLCE_ERR_INVALID_ARG;
  if (workspace_bytes < need) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  if ((st = device_info(&sms)) != FLCE_OK) return st;
  const bool f16 = p->input_fp16 != 0;
  const int M = static_cast<int>(p->M), K = static_cast<int>(p->K), F = static_cast<int>(p->F);
  if (w.few) {
    SmallArgs sa;
    if (!small_args(&sa, x, pitch(p->ld_x, K), M, K, 1, F, h, pitch(p->ld_h, F), true, f16, dev_err) ||
        !k_major(&sa.w, Wg, F, K, K, f16, 64) || !k_major(&sa.w2, Wu, F, K, K, f16, 64))
      return FLCE_ERR_CUDA;
    sa.keep = static_cast<uint16_t*>(pre);
    sa.relative = p->keep == FLCE_KEEP_RELATIVE ? 1 : 0;
    sa.wp = static_cast<const uint16_t*>(Wg);
    sa.act = p->activation;
    return done(launch_small(true, false, sa, static_cast<cudaStream_t>(stream)));
  }

  GatedArgs ea;
  std::memset(&ea, 0, sizeof(ea));
  ea.act = p->activation;
  ea.fp16 = f16 ? 1 : 0;
  ea.keep = !pre ? 0 : p->keep == FLCE_KEEP_RELATIVE ? 2 : 1;
  ea.M = M;
  ea.F = F;
  ea.sign = {static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(Wg), nullptr,
             pitch(p->ld_x, K), K};
  uint16_t* keep = static_cast<uint16_t*>(pre);
  PairArgs g = pair_args(M, F, K, 1, false, true, f16, dev_err);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  int64_t ld_x = pitch(p->ld_x, K), ld_g = K, ld_u = K;
  const void* xn = repacked(x, M, K, &ld_x, w.ld_x, w.x, s, &e);
  const void* Wgn = repacked(Wg, F, K, &ld_g, w.ld_w, w.Wg, s, &e);
  const void* Wun = repacked(Wu, F, K, &ld_u, w.ld_w, w.Wu, s, &e);
  if (e != cudaSuccess || !out16(&ea.h, h, M, F, pitch(p->ld_h, F)) ||
      (pre && (!out16(&ea.val, keep, M, F, F) ||
               !out16(&ea.cross, keep + static_cast<size_t>(M) * F, M, F, F))) ||
      !k_major(&g.a, xn, M, K, ld_x, f16) || !k_major(&g.b, Wgn, F, K, ld_g, f16, g.bn / 2) ||
      !k_major(&g.b2, Wun, F, K, ld_u, f16, g.bn / 2))
    return FLCE_ERR_CUDA;
  return done(launch_gated(g, ea, sms, s));
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
  if (workspace_bytes < carve(p, workspace, &w)) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  if ((st = device_info(&sms)) != FLCE_OK) return st;
  const bool f16 = p->input_fp16 != 0;
  const int M = static_cast<int>(p->M), K = static_cast<int>(p->K), F = static_cast<int>(p->F);

  GatedGradArgs ga;
  ga.dh = static_cast<const uint16_t*>(dh);
  ga.ld_dh = pitch(p->ld_h, F);
  ga.val = static_cast<const uint16_t*>(pre);
  ga.cross = ga.val + static_cast<size_t>(M) * F;
  ga.ld = w.ld;
  ga.dg = w.dg;
  ga.du = w.du;
  ga.M = M;
  ga.F = F;
  ga.fp16 = f16 ? 1 : 0;
  ga.relative = p->keep == FLCE_KEEP_RELATIVE ? 1 : 0;
  if (launch_gated_grad(ga, s) != cudaSuccess) return FLCE_ERR_CUDA;
  cudaError_t e = cudaSuccess;
  if (dx && w.few) {
    SmallArgs sa;
    const bool ok = small_args(&sa, w.dg, w.ld, M, F, 2, K, dx, K, false, f16, dev_err);
    sa.xp2 = w.du;
    if (!ok || (small_tokens(M) > 32 && !k_major(&sa.x2, w.du, M, F, w.ld, f16, small_tokens(M))) ||
        !mn_major(&sa.w, Wg, K, F, K, f16, kBK) || !mn_major(&sa.w2, Wu, K, F, K, f16, kBK) ||
        launch_small(false, true, sa, s) != cudaSuccess)
      return FLCE_ERR_CUDA;
  } else if (dx) {
    GradXArgs ea;
    std::memset(&ea, 0, sizeof(ea));
    ea.fp16 = f16 ? 1 : 0;
    ea.M = M;
    ea.K = K;
    PairArgs g = pair_args(M, K, F, 2, true, false, f16, dev_err);
    int64_t ld_g = K, ld_u = K;
    const void* Wgn = repacked(Wg, F, K, &ld_g, w.ld_w, w.Wg, s, &e);
    const void* Wun = repacked(Wu, F, K, &ld_u, w.ld_w, w.Wu, s, &e);
    const int lk = pair_lk(g.halves);
    if (!out16(&ea.dx, dx, M, K, K) || !k_major(&g.a, w.dg, M, F, w.ld, f16) ||
        !k_major(&g.a2, w.du, M, F, w.ld, f16) || !mn_major(&g.b, Wgn, K, F, ld_g, f16, lk) ||
        !mn_major(&g.b2, Wun, K, F, ld_u, f16, lk) || e != cudaSuccess ||
        launch_grad_x(true, g, ea, sms, s) != cudaSuccess)
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
    PairArgs g = pair_args(2 * cdiv(F, 256) * 256, K, M, 1, true, false, f16, dev_err);
    g.m_split = g.tiles_m / 2;
    int64_t ld_x = pitch(p->ld_x, K);
    const void* xn = repacked(x, M, K, &ld_x, w.ld_x, w.x, s, &e);
    const int lk = pair_lk(g.halves);
    if (!encode_store_2d(&ea.out, dWg, K, F, row, p->dW_fp32 != 0) ||
        !encode_store_2d(&ea.out2, dWu, K, F, row, p->dW_fp32 != 0) ||
        !mn_major(&g.a, w.dg, F, M, w.ld, f16, lk) || !mn_major(&g.a2, w.du, F, M, w.ld, f16, lk) ||
        !mn_major(&g.b, xn, K, M, ld_x, f16, lk) || e != cudaSuccess ||
        launch_grad_w(true, g, ea, sms, s) != cudaSuccess)
      return FLCE_ERR_CUDA;
  }
  return FLCE_OK;
}

}  // extern "C"
