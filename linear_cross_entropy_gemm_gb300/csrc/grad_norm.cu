// The global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum_t sum_i g_t[i]^2),   out_t = min(1, max_norm / (norm + eps)) g_t
//
// Both passes cut every tensor into 32 KiB chunks and spread the chunks of all
// tensors over one wave of blocks, so a hundred small tensors and one large
// one load the memory alike. Chunks start on 128-byte lines wherever the tensor does,
// so that a warp's load touches four lines, not five (2.1 GB of fp32 gradients 32
// bytes off a line: 324 us from the tensor's start, 296 us = 7.1 TB/s so). The table of
// tensors travels in the kernel's parameters (no copy to the device, nothing to keep
// alive). Bound by HBM: the norm reads every element once, clipping reads it again and
// writes it (60 tensors, 683 MB: 335 us = 6.1 TB/s; chunks of 16 and 64 KiB and blocks of
// 512 threads took 338 to 390).
//
// The norm pass leaves one fp64 sum per block; whoever needs the norm adds those
// in one fixed order, so the result does not depend on the blocks' timing.
// The clip pass walks the chunks backwards: what the norm pass read last is
// what the L2 still holds.
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/flce.h"
#include "block_internal.h"
#include "flce_host.h"

namespace flce {
namespace {

constexpr int kThreadsN = 256;
constexpr int kBlocksPerSm = 4;
constexpr int kChunkBytes = 32768;
constexpr int kVecs = kChunkBytes / 16 / kThreadsN;  // 16-byte loads of a thread per chunk
constexpr int kLine = 128;                           // chunks start at multiples of this
constexpr int kMaxPartials = 4096;                   // blocks of one launch
constexpr int kTableMax = 1024;                      // tensors of one launch

template <int CAP>
struct Table {
  const void* ptr[CAP];
  void* out[CAP];             // clip only
  int64_t numel_type[CAP];    // numel * 4 + flce_dtype_t
  uint32_t begin[CAP + 1];    // first chunk of each tensor; [count]: all chunks
  int count;
};

__device__ __forceinline__ int type_bytes(int type) { return type == FLCE_DTYPE_FP32 ? 4 : 2; }

__device__ __forceinline__ float load_one(const uint8_t* p, int type) {
  if (type == FLCE_DTYPE_FP32) return *reinterpret_cast<const float*>(p);
  return unpack_16(*reinterpret_cast<const uint16_t*>(p), type == FLCE_DTYPE_FP16);
}
__device__ __forceinline__ void store_one(uint8_t* p, float v, int type) {
  if (type == FLCE_DTYPE_FP32)
    *reinterpret_cast<float*>(p) = v;
  else
    *reinterpret_cast<uint16_t*>(p) =
        static_cast<uint16_t>(pack_16x2(v, 0.f, type == FLCE_DTYPE_FP16) & 0xFFFFu);
}

__device__ __forceinline__ float square_16b(const uint4& u, int type) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  float a = 0.f, b = 0.f;
  if (type == FLCE_DTYPE_FP32) {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const float x = __uint_as_float(w[e]), y = __uint_as_float(w[e + 1]);
      a = fmaf(x, x, a);
      b = fmaf(y, y, b);
    }
  } else {
    const bool f16 = type == FLCE_DTYPE_FP16;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = unpack_16(w[e] & 0xFFFFu, f16), y = unpack_16(w[e] >> 16, f16);
      a = fmaf(x, x, a);
      b = fmaf(y, y, b);
    }
  }
  return a + b;
}

__device__ __forceinline__ uint4 scale_16b(const uint4& u, float c, int type) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t r[4];
  if (type == FLCE_DTYPE_FP32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = __float_as_uint(__uint_as_float(w[e]) * c);
  } else {
    const bool f16 = type == FLCE_DTYPE_FP16;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      r[e] = pack_16x2(unpack_16(w[e] & 0xFFFFu, f16) * c, unpack_16(w[e] >> 16, f16) * c, f16);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// The tensor that holds chunk c: the last one that begins at or before it.
template <int CAP>
__device__ __forceinline__ int find_tensor(const Table<CAP>& t, uint32_t c) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.begin[mid] <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Chunk c: bytes [lo, hi) from p, a kLine boundary that may lie before the tensor (whose
// out starts as far before its own). Whole 16-byte words [v_lo, v_hi), and `edge` elements,
// fewer than eight before and after them each.
struct Chunk {
  const uint8_t* p;
  int64_t off;  // of p from the tensor's first byte
  int tensor, type, esize, lo, hi, v_lo, v_hi, head, edge;
  __device__ __forceinline__ int edge_byte(int e) const {
    return e < head ? lo + e * esize : hi - (edge - e) * esize;
  }
};
template <int CAP>
__device__ __forceinline__ Chunk chunk_of(const Table<CAP>& t, uint32_t c) {
  Chunk k;
  k.tensor = find_tensor(t, c);
  const int64_t nt = t.numel_type[k.tensor];
  const uintptr_t first = reinterpret_cast<uintptr_t>(t.ptr[k.tensor]);
  k.type = static_cast<int>(nt & 3);
  k.esize = type_bytes(k.type);
  k.off = static_cast<int64_t>(c - t.begin[k.tensor]) * kChunkBytes -
          static_cast<int64_t>(first % kLine);
  k.p = reinterpret_cast<const uint8_t*>(first + k.off);
  const int64_t left = (nt >> 2) * k.esize - k.off;
  k.lo = k.off < 0 ? static_cast<int>(-k.off) : 0;
  k.hi = static_cast<int>(left < kChunkBytes ? left : kChunkBytes);
  k.v_lo = (k.lo + 15) / 16;
  k.v_hi = k.hi / 16;
  const int head_end = min(k.v_lo * 16, k.hi);
  k.head = (head_end - k.lo) / k.esize;
  k.edge = k.head + (k.hi - max(k.v_hi * 16, head_end)) / k.esize;
  return k;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sum over the block in a fixed order, in every thread.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double s[kThreadsN / 32];
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < kThreadsN / 32; ++w) t += s[w];
  return t;
}

// This thread's 16-byte words of a chunk, all loads in flight; those outside it are zero.
__device__ __forceinline__ bool has_word(const Chunk& k, int j) {
  const int i = j * kThreadsN + static_cast<int>(threadIdx.x);
  return i >= k.v_lo && i < k.v_hi;
}
__device__ __forceinline__ void load_words(const Chunk& k, uint4 (&u)[kVecs]) {
  const uint4* v = reinterpret_cast<const uint4*>(k.p) + threadIdx.x;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    u[j] = make_uint4(0, 0, 0, 0);
    if (has_word(k, j)) u[j] = v[j * kThreadsN];
  }
}

// This thread's share of a chunk's squares.
__device__ __forceinline__ float chunk_squares(const Chunk& k) {
  uint4 u[kVecs];
  load_words(k, u);
  float s = 0.f;
  const int e = threadIdx.x;
  if (e < k.edge) {
    const float x = load_one(k.p + k.edge_byte(e), k.type);
    s = x * x;
  }
#pragma unroll
  for (int j = 0; j < kVecs; ++j) s += square_16b(u[j], k.type);
  return s;
}

// This thread's share of out = c chunk.
__device__ __forceinline__ void scale_chunk(const Chunk& k, void* tensor_out, float c) {
  uint8_t* out = reinterpret_cast<uint8_t*>(reinterpret_cast<uintptr_t>(tensor_out) + k.off);
  if (c == 1.f && out == k.p) return;
  if (((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(k.p)) & 15) != 0) {
    // Source and destination differ in alignment: element by element.
    for (int b = k.lo + static_cast<int>(threadIdx.x) * k.esize; b < k.hi; b += kThreadsN * k.esize)
      store_one(out + b, load_one(k.p + b, k.type) * c, k.type);
    return;
  }
  uint4 u[kVecs];
  load_words(k, u);
  const int e = threadIdx.x;
  if (e < k.edge)
    store_one(out + k.edge_byte(e), load_one(k.p + k.edge_byte(e), k.type) * c, k.type);
  uint4* o = reinterpret_cast<uint4*>(out) + threadIdx.x;
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
    if (has_word(k, j)) __stcs(o + j * kThreadsN, scale_16b(u[j], c, k.type));
}

__device__ __forceinline__ float clip_scale(float norm, float max_norm, float eps) {
  const float q = max_norm / (norm + eps);
  return q > 1.f ? 1.f : q;  // a NaN stays one
}

template <int CAP>
__global__ void __launch_bounds__(kThreadsN, kBlocksPerSm)
    square_sums_kernel(const __grid_constant__ Table<CAP> t, double* part) {
  griddep_launch();
  griddep_wait();
  double total = 0.0;
  const uint32_t chunks = t.begin[t.count];
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x)
    total += static_cast<double>(chunk_squares(chunk_of(t, c)));
  total = block_sum(total);
  if (threadIdx.x == 0) part[blockIdx.x] = total;
}

// The norm from the blocks' sums, in every thread of a block.
__device__ __forceinline__ float norm_of(const double* part, int parts) {
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreadsN) v += part[i];
  return static_cast<float>(sqrt(block_sum(v)));
}

__global__ void __launch_bounds__(kThreadsN) norm_kernel(const double* part, int parts,
                                                         float* norm) {
  griddep_launch();
  griddep_wait();
  const float n = norm_of(part, parts);
  if (threadIdx.x == 0) *norm = n;
}

template <int CAP>
__global__ void __launch_bounds__(kThreadsN, kBlocksPerSm)
    clip_kernel(const __grid_constant__ Table<CAP> t, const double* part, int parts, float max_norm,
                float eps, float* norm) {
  griddep_launch();
  griddep_wait();
  const float n = norm_of(part, parts);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  const float c = clip_scale(n, max_norm, eps);
  const uint32_t chunks = t.begin[t.count];
  for (uint32_t i = blockIdx.x; i < chunks; i += gridDim.x) {
    const Chunk k = chunk_of(t, chunks - 1 - i);
    scale_chunk(k, t.out[k.tensor], c);
  }
}

// The caller's HOST arrays.
struct Grads {
  int64_t count;
  const void* const* ptrs;
  void* const* out;  // null: in place
  const int64_t* numel;
  const int32_t* dtypes;
};

uint64_t chunks_of(const void* p, int64_t bytes) {
  const uint64_t all = reinterpret_cast<uintptr_t>(p) % kLine + static_cast<uint64_t>(bytes);
  return (all + kChunkBytes - 1) / kChunkBytes;
}

flce_status_t check_grads(const Grads& g) {
  if (g.count < 0 || (g.count > 0 && (!g.ptrs || !g.numel || !g.dtypes)))
    return FLCE_ERR_INVALID_ARG;
  uint64_t chunks = 0;
  for (int64_t i = 0; i < g.count; ++i) {
    if (g.numel[i] < 0 || g.dtypes[i] < FLCE_DTYPE_BF16 || g.dtypes[i] > FLCE_DTYPE_FP32)
      return FLCE_ERR_INVALID_ARG;
    if (g.numel[i] == 0) continue;
    if (g.numel[i] > (1LL << 48)) return FLCE_ERR_UNSUPPORTED;
    const uintptr_t mask = g.dtypes[i] == FLCE_DTYPE_FP32 ? 3 : 1;
    const void* o = g.out ? g.out[i] : g.ptrs[i];
    if (!g.ptrs[i] || !o) return FLCE_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(g.ptrs[i]) | reinterpret_cast<uintptr_t>(o)) & mask) != 0)
      return FLCE_ERR_ALIGNMENT;
    chunks += chunks_of(g.ptrs[i], g.numel[i] * static_cast<int64_t>(mask + 1));
    if (chunks >= (1ULL << 31)) return FLCE_ERR_UNSUPPORTED;
  }
  return FLCE_OK;
}

template <int CAP>
int fill(Table<CAP>* t, const Grads& g, int64_t* next) {
  uint32_t chunks = 0;
  int n = 0;
  for (; *next < g.count && n < CAP; ++*next) {
    const int64_t i = *next;
    if (g.numel[i] == 0) continue;
    t->ptr[n] = g.ptrs[i];
    t->out[n] = g.out ? g.out[i] : const_cast<void*>(g.ptrs[i]);
    t->numel_type[n] = g.numel[i] * 4 + g.dtypes[i];
    t->begin[n] = chunks;
    const int64_t bytes = g.numel[i] * (g.dtypes[i] == FLCE_DTYPE_FP32 ? 4 : 2);
    chunks += static_cast<uint32_t>(chunks_of(g.ptrs[i], bytes));
    ++n;
  }
  t->begin[n] = chunks;
  t->count = n;
  return n;
}

template <int CAP>
uint32_t grid_of(const Table<CAP>& t, int sms) {
  const uint32_t most = static_cast<uint32_t>(sms) * kBlocksPerSm;
  const uint32_t n = t.begin[t.count] < most ? t.begin[t.count] : most;
  return n < static_cast<uint32_t>(kMaxPartials) ? n : kMaxPartials;
}

// One launch for each CAP tensors; the norm passes leave their sums one after another.
template <int CAP>
cudaError_t run_passes(const Grads& g, bool clip, float max_norm, float eps, float* norm,
                       double* part, int sms, cudaStream_t st) {
  Table<CAP> t;
  int64_t next = 0;
  int parts = 0;
  cudaError_t e = cudaSuccess;
  for (next = 0; next < g.count && e == cudaSuccess;) {
    if (fill(&t, g, &next) == 0) break;
    const uint32_t grid = grid_of(t, sms);
    e = launch_dependent(square_sums_kernel<CAP>, dim3(grid), kThreadsN, 0, 1, st, t, part + parts);
    parts += static_cast<int>(grid);
  }
  // Without elements there is no clip pass to write the norm, 0.
  if ((!clip || parts == 0) && e == cudaSuccess)
    return launch_dependent(norm_kernel, dim3(1), kThreadsN, 0, 1, st, part, parts, norm);
  for (next = 0; next < g.count && e == cudaSuccess;) {
    if (fill(&t, g, &next) == 0) break;
    e = launch_dependent(clip_kernel<CAP>, dim3(grid_of(t, sms)), kThreadsN, 0, 1, st, t, part,
                         parts, max_norm, eps, norm);
  }
  return e;
}

size_t workspace_of(int64_t count) {
  const int64_t launches = count > 0 ? (count + kTableMax - 1) / kTableMax : 1;
  return static_cast<size_t>(launches) * kMaxPartials * sizeof(double) + kAlign;
}

flce_status_t run(const Grads& g, bool clip, float max_norm, float eps, float* norm,
                  void* workspace, size_t workspace_bytes, cudaStream_t st) {
  const flce_status_t bad = check_grads(g);
  if (bad != FLCE_OK) return bad;
  if (!norm || !workspace) return FLCE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(norm) & 3) != 0) return FLCE_ERR_ALIGNMENT;
  if (workspace_bytes < workspace_of(g.count)) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  const flce_status_t ds = device_info(&sms);
  if (ds != FLCE_OK) return ds;
  Carver cv(workspace, workspace_bytes);
  double* part = cv.take<double>(0);
  // The smallest table that holds the tensors: a launch copies its parameters.
  const cudaError_t e =
      g.count <= 64    ? run_passes<64>(g, clip, max_norm, eps, norm, part, sms, st)
      : g.count <= 256 ? run_passes<256>(g, clip, max_norm, eps, norm, part, sms, st)
                       : run_passes<kTableMax>(g, clip, max_norm, eps, norm, part, sms, st);
  return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

}  // namespace
}  // namespace flce

extern "C" {

size_t flce_grad_norm_workspace_size(int64_t count) {
  return count < 0 ? 0 : flce::workspace_of(count);
}

flce_status_t flce_grad_norm(int64_t count, const void* const* ptrs, const int64_t* numel,
                             const int32_t* dtypes, float* norm, void* workspace,
                             size_t workspace_bytes, void* stream) {
  flce::NvtxRange nvtx_range("flce_grad_norm");
  const flce::Grads g{count, ptrs, nullptr, numel, dtypes};
  return flce::run(g, false, 0.f, 0.f, norm, workspace, workspace_bytes,
                   static_cast<cudaStream_t>(stream));
}

flce_status_t flce_clip_grads(int64_t count, const void* const* ptrs, void* const* out,
                              const int64_t* numel, const int32_t* dtypes, float max_norm,
                              float eps, float* norm, void* workspace, size_t workspace_bytes,
                              void* stream) {
  flce::NvtxRange nvtx_range("flce_clip_grads");
  if (!(max_norm >= 0.f) || !(eps >= 0.f) || !(eps < INFINITY)) return FLCE_ERR_INVALID_ARG;
  const flce::Grads g{count, ptrs, out, numel, dtypes};
  return flce::run(g, true, max_norm, eps, norm, workspace, workspace_bytes,
                   static_cast<cudaStream_t>(stream));
}

}  // extern "C"
