// flce_clip.cu — the global 2-norm of many gradient tensors, and their clipping:
// kernels and C entry points.
//
//   norm = sqrt(sum g^2),  c = min(1, max_norm / (norm + 1e-6)),  out = rn(g c)
//
// Two passes over the gradients, both bound by memory.  The tensors' pointers
// and sizes travel in the kernels' parameters (no copy to the device, nothing
// for the caller to keep), and the tensors are cut into chunks that the blocks
// take in turn, so that many small tensors cost no more than a few large ones.
#include <algorithm>
#include <cmath>

#include "flce_elem.cuh"
#include "flce_host.h"

namespace flce {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;          // elements per chunk
constexpr int kMaxGrid = 1024;        // blocks of a launch at most: partial sums per launch
constexpr int kSmallTable = 32;       // tensors per launch: the small table is copied faster
constexpr int kLargeTable = 960;      // (28.9 KB of the 32 KB of kernel parameters)

// One launch's tensors: chunk_end[i] is the number of chunks of tensors 0..i.
template <int N>
struct GradTable {
  const void* src[N];
  void* dst[N];
  int64_t numel[N];
  int32_t chunk_end[N];
  uint8_t dtype[N];
  int32_t count;
  int32_t chunks;
};

template <int N>
__device__ __forceinline__ int find_tensor(const GradTable<N>& t, int chunk) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (chunk < t.chunk_end[mid]) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Sum of squares of up to 8 values: in fp32 where that is safe, in fp64 where a
// square could overflow fp32 or the sum is so small that squares may have
// underflowed (fp32 squares vanish below about 1e-23; 2^-100 leaves 24 bits of
// head-room above the subnormals for every term that matters to the sum).
template <int V>
__device__ __forceinline__ double sum_squares(const float (&x)[V]) {
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) s = fmaf(x[k], x[k], s);
  if (s > 0x1p-100f && s < INFINITY) return double(s);
  double d = 0.0;
  bool any = false;
#pragma unroll
  for (int k = 0; k < V; ++k) any |= x[k] != 0.f;  // a NaN is not 0 either
  if (any) {
#pragma unroll
    for (int k = 0; k < V; ++k) d = fma(double(x[k]), double(x[k]), d);
  }
  return d;
}

constexpr int kVec = 8;

template <class T>
__device__ __forceinline__ double chunk_norm(const T* p, int n) {
  double sum = 0.0;
  const bool vec = reinterpret_cast<uintptr_t>(p) % 16 == 0;
  const int full = vec ? n / kVec * kVec : 0;
  for (int i = threadIdx.x * kVec; i < full; i += kThreads * kVec) {
    const Vec<T, kVec> v = load_vec<T, kVec>(p + i);
    float x[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) x[k] = to_f32(v.v[k]);
    sum += sum_squares<kVec>(x);
  }
  for (int i = full + threadIdx.x; i < n; i += kThreads) {
    const float x[1] = {to_f32(p[i])};
    sum += sum_squares<1>(x);
  }
  return sum;
}

template <int N>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ GradTable<N> t, double* part) {
  __shared__ double red[32];
  double sum = 0.0;
  for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const int i = find_tensor(t, c);
    const int64_t begin = int64_t(c - (i ? t.chunk_end[i - 1] : 0)) * kChunk;
    const int n = int(min(int64_t(kChunk), t.numel[i] - begin));
    if (t.dtype[i] == FLCE_F32) {
      sum += chunk_norm(static_cast<const float*>(t.src[i]) + begin, n);
    } else if (t.dtype[i] == FLCE_BF16) {
      sum += chunk_norm(static_cast<const __nv_bfloat16*>(t.src[i]) + begin, n);
    } else {
      sum += chunk_norm(static_cast<const __half*>(t.src[i]) + begin, n);
    }
  }
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// Sum of the blocks' partial sums, the same in every block.
__device__ __forceinline__ double total(const double* part, int n, double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += part[i];
  return block_sum(s, red);
}

__global__ void __launch_bounds__(kThreads) norm_total_kernel(const double* part, int n, float* norm) {
  __shared__ double red[32];
  const double s = total(part, n, red);
  if (threadIdx.x == 0) *norm = float(sqrt(s));
}

template <class T>
__device__ __forceinline__ void chunk_scale(const T* src, T* dst, int n, float c) {
  const bool vec = reinterpret_cast<uintptr_t>(src) % 16 == 0 && reinterpret_cast<uintptr_t>(dst) % 16 == 0;
  const int full = vec ? n / kVec * kVec : 0;
  for (int i = threadIdx.x * kVec; i < full; i += kThreads * kVec) {
    Vec<T, kVec> v = load_vec<T, kVec>(src + i);
#pragma unroll
    for (int k = 0; k < kVec; ++k) v.v[k] = from_f32<T>(to_f32(v.v[k]) * c);
    store_vec<T, kVec>(dst + i, v);
  }
  for (int i = full + threadIdx.x; i < n; i += kThreads) dst[i] = from_f32<T>(to_f32(src[i]) * c);
}

// min(1, max / (norm + 1e-6)) that keeps a NaN.
__device__ __forceinline__ float clip_factor(float norm, float max_norm) {
  const float c = max_norm / (norm + 1e-6f);
  return c > 1.0f ? 1.0f : c;
}

template <int N>
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ GradTable<N> t,
                                                             const double* part, int n_part, float max_norm,
                                                             float* norm) {
  __shared__ double red[32];
  const float nm = float(sqrt(total(part, n_part, red)));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = nm;
  const float f = clip_factor(nm, max_norm);
  // an infinite limit over an infinite norm is NaN; such a limit clips nothing
  const float c = max_norm == INFINITY && nm == nm ? 1.0f : f;
  // last chunks first: the norm's pass has just read them
  for (int c0 = t.chunks - 1 - int(blockIdx.x); c0 >= 0; c0 -= gridDim.x) {
    const int i = find_tensor(t, c0);
    if (c == 1.0f && t.src[i] == t.dst[i]) continue;
    const int64_t begin = int64_t(c0 - (i ? t.chunk_end[i - 1] : 0)) * kChunk;
    const int n = int(min(int64_t(kChunk), t.numel[i] - begin));
    if (t.dtype[i] == FLCE_F32) {
      chunk_scale(static_cast<const float*>(t.src[i]) + begin, static_cast<float*>(t.dst[i]) + begin, n, c);
    } else if (t.dtype[i] == FLCE_BF16) {
      chunk_scale(static_cast<const __nv_bfloat16*>(t.src[i]) + begin, static_cast<__nv_bfloat16*>(t.dst[i]) + begin,
                  n, c);
    } else {
      chunk_scale(static_cast<const __half*>(t.src[i]) + begin, static_cast<__half*>(t.dst[i]) + begin, n, c);
    }
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
constexpr int64_t kMaxChunks = INT32_MAX / 2;  // of all tensors together: 8.8e12 elements

struct Grads {
  const void* const* src;
  void* const* dst;  // nullptr: norm only
  const int64_t* numel;
  const int32_t* dtypes;
  int64_t count;
};

int validate(const Grads& g, bool clip) {
  if (g.count < 0 || g.count > (int64_t(1) << 24)) return FLCE_ERR_INVALID_ARG;
  if (g.count > 0 && (!g.src || !g.numel || !g.dtypes || (clip && !g.dst))) return FLCE_ERR_INVALID_ARG;
  int64_t chunks = 0;
  for (int64_t i = 0; i < g.count; ++i) {
    if (!known_dtype(g.dtypes[i])) return FLCE_ERR_UNSUPPORTED_DTYPE;
    if (g.numel[i] < 0 || g.numel[i] / kChunk >= kMaxChunks) return FLCE_ERR_INVALID_ARG;
    chunks += (g.numel[i] + kChunk - 1) / kChunk;
    if (chunks > kMaxChunks) return FLCE_ERR_INVALID_ARG;
    if (g.numel[i] == 0) continue;
    if (!g.src[i] || (clip && !g.dst[i])) return FLCE_ERR_INVALID_ARG;
    const size_t e = elem_size(g.dtypes[i]);
    if (!aligned_to(g.src[i], e) || (clip && !aligned_to(g.dst[i], e))) return FLCE_ERR_MISALIGNED;
  }
  return FLCE_OK;
}

// Fills `t` with tensors from index *next on, as many as fit.
template <int N>
void fill(GradTable<N>& t, const Grads& g, int64_t* next) {
  t.count = 0;
  t.chunks = 0;
  for (; *next < g.count && t.count < N; ++*next) {
    const int64_t i = *next;
    if (g.numel[i] == 0) continue;
    t.src[t.count] = g.src[i];
    t.dst[t.count] = g.dst ? g.dst[i] : nullptr;
    t.numel[t.count] = g.numel[i];
    t.dtype[t.count] = uint8_t(g.dtypes[i]);
    t.chunks += int32_t((g.numel[i] + kChunk - 1) / kChunk);
    t.chunk_end[t.count++] = t.chunks;
  }
}

int grid_for(int chunks, int num_sms) { return std::max(1, std::min({chunks, 4 * num_sms, kMaxGrid})); }

template <int N>
int run_tables(const Grads& g, bool clip, float max_norm, float* norm, double* part, int num_sms, cudaStream_t st) {
  GradTable<N> t;
  int parts = 0;
  for (int64_t next = 0; next < g.count;) {
    fill(t, g, &next);
    if (t.count == 0) continue;  // only empty tensors were left
    const int grid = grid_for(t.chunks, num_sms);
    FLCE_TRY(logged(FLCE_LAUNCH_OTHER, st, [&] {
      grad_norm_kernel<N><<<grid, kThreads, 0, st>>>(t, part + parts);
      return cudaGetLastError();
    }));
    parts += grid;
  }
  if (!clip || parts == 0)
    return logged(FLCE_LAUNCH_OTHER, st, [&] {
      norm_total_kernel<<<1, kThreads, 0, st>>>(part, parts, norm);
      return cudaGetLastError();
    });
  bool first = true;
  for (int64_t next = 0; next < g.count;) {
    fill(t, g, &next);
    if (t.count == 0) continue;
    FLCE_TRY(logged(FLCE_LAUNCH_OTHER, st, [&] {
      grad_scale_kernel<N><<<grid_for(t.chunks, num_sms), kThreads, 0, st>>>(t, part, parts, max_norm,
                                                                            first ? norm : nullptr);
      return cudaGetLastError();
    }));
    first = false;
  }
  return FLCE_OK;
}

int run(const Grads& g, bool clip, float max_norm, float* norm, void* workspace, size_t workspace_bytes,
        flce_stream_t stream) {
  FLCE_TRY(validate(g, clip));
  if (!norm || !workspace) return FLCE_ERR_INVALID_ARG;
  if (!aligned_to(norm, 4) || !aligned_to(workspace, 16)) return FLCE_ERR_MISALIGNED;
  size_t need = 0;
  FLCE_TRY(flce_grad_norm_workspace_size(g.count, &need));
  if (workspace_bytes < need) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  DeviceInfo dev;
  FLCE_TRY(get_device(&dev));
  FLCE_TRY(check_local(dev, norm, workspace));
  for (int64_t i = 0; i < g.count; ++i) {
    if (g.numel[i] == 0) continue;
    FLCE_TRY(check_local(dev, g.src[i]));
    if (clip && g.dst[i] != g.src[i]) FLCE_TRY(check_local(dev, g.dst[i]));
  }
  double* part = static_cast<double*>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return g.count <= kSmallTable ? run_tables<kSmallTable>(g, clip, max_norm, norm, part, dev.num_sms, st)
                                : run_tables<kLargeTable>(g, clip, max_norm, norm, part, dev.num_sms, st);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_grad_norm_workspace_size(int64_t count, size_t* bytes) {
  if (!bytes || count < 0 || count > (int64_t(1) << 24)) return FLCE_ERR_INVALID_ARG;
  // one partial sum per block and launch
  const int64_t launches = std::max<int64_t>(1, (count + kLargeTable - 1) / kLargeTable);
  *bytes = size_t(launches) * kMaxGrid * sizeof(double);
  return FLCE_OK;
}

int flce_grad_norm(const void* const* grads, const int64_t* numel, const int32_t* dtypes, int64_t count, float* norm,
                   void* workspace, size_t workspace_bytes, flce_stream_t stream) {
  const Grads g = {grads, nullptr, numel, dtypes, count};
  return run(g, false, 0.f, norm, workspace, workspace_bytes, stream);
}

int flce_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* numel, const int32_t* dtypes,
                        int64_t count, float max_norm, float* norm, void* workspace, size_t workspace_bytes,
                        flce_stream_t stream) {
  if (!(max_norm >= 0.f)) return FLCE_ERR_INVALID_ARG;
  const Grads g = {grads, outs, numel, dtypes, count};
  return run(g, true, max_norm, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
