// flce_clip.cu — the global 2-norm of many gradient tensors, and their clipping:
// kernels and C entry points.
//
//   norm = sqrt(sum g^2),  c = min(1, max_norm / (norm + 1e-6)),  out = rn(g c)
//
// Two passes over the gradients, both bound by memory: 622 M bf16 elements of a
// head's gradients take 548 us, where reading twice and writing once at the copy
// rate takes 557.  The second pass may find the end of what the first read in L2,
// so it goes backwards.  The tensors' pointers and sizes travel in the kernels'
// parameters (no copy to the device, nothing for the caller to keep), and the
// tensors of a type are cut into chunks of one size, a block each, so that many
// small tensors cost no more than a few large ones and blocks go where earlier ones
// end.
//
// fp64 is slow on this part (two lanes per SM and clock): with an fp64 addition
// per 32 elements and fp64 sums over the block the first pass ran at half the
// memory's rate (head: 1021 us; 34 M fp32 elements: 95, now 70).  So a chunk is
// summed in fp32, compensated over its rounds, and only chunks with squares outside
// fp32's safe range are summed again in fp64, element by element: with the head's
// last 1500 rows below 1e-18 the call takes 710 us, with half of its rows 1620.
#include <cmath>

#include "flce_device.cuh"
#include "flce_elem.cuh"
#include "flce_host.h"

namespace flce {
namespace {

constexpr int kGradThreads = 256;
constexpr int kTotalThreads = 1024;
constexpr int kUnroll = 4;            // 16-byte loads under way per thread
constexpr int kMinChunk = 8192;       // elements per chunk: this times a power of two,
constexpr int64_t kWantChunks = 8000; // so that there are about this many at most
constexpr int kFewParts = 512;        // up to here every block of the second pass adds the partial sums itself
constexpr int kSmallTable = 32;       // tensors per launch: the small table is copied faster
constexpr int kMediumTable = 240;
constexpr int kLargeTable = 960;      // (27.9 KB of the 32 KB of kernel parameters)

// One launch's tensors: chunk_end[i] is the number of chunks of tensors 0..i.
template <int N>
struct GradTable {
  const void* src[N];
  void* dst[N];
  int64_t numel[N];
  int32_t chunk_end[N];
  int32_t count;
  int32_t chunks;
  int32_t chunk;  // elements
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

// Sum of the squares of N values in fp32.  *safe is cleared where a square may
// have overflowed, or the sum is so small that squares may have underflowed
// (fp32 squares vanish below about 1e-23; 2^-100 leaves 24 bits of head-room
// above the subnormals for every term that matters to the sum).
template <int N>
__device__ __forceinline__ float sum_squares(const float (&x)[N], bool* safe) {
  constexpr int kChains = N < 8 ? N : 8;
  float s[kChains];
#pragma unroll
  for (int k = 0; k < kChains; ++k) s[k] = x[k] * x[k];
#pragma unroll
  for (int k = kChains; k < N; ++k) s[k % kChains] = fmaf(x[k], x[k], s[k % kChains]);
#pragma unroll
  for (int w = kChains / 2; w > 0; w /= 2)
#pragma unroll
    for (int k = 0; k < w; ++k) s[k] += s[k + w];
  if (!(s[0] > 0x1p-100f && s[0] < 0x1p100f)) {
    bool any = false;
#pragma unroll
    for (int k = 0; k < N; ++k) any |= x[k] != 0.f;  // a NaN is not 0 either
    if (any) *safe = false;
  }
  return s[0];
}

// A sum that keeps what its additions round off.
struct Compensated {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float t = hi + x, b = t - hi;
    lo += (hi - (t - b)) + (x - b);
    hi = t;
  }
};

template <class T>
struct Loads {
  static constexpr int kVec = 16 / sizeof(T);                   // elements per load
  static constexpr int kRound = kGradThreads * kVec * kUnroll;  // elements a block has under way
};
// Elements before the first 16-byte boundary.
template <class T>
__device__ __forceinline__ int head_of(const T* p, int n) {
  return min(n, int((16 - reinterpret_cast<uintptr_t>(p) % 16) % 16 / sizeof(T)));
}

template <class T>
__device__ __forceinline__ float chunk_norm(const T* p, int n, bool* safe) {
  constexpr int kVec = Loads<T>::kVec, kRound = Loads<T>::kRound;
  Compensated sum;
  const int head = head_of(p, n);
  const T* q = p + head;
  const int m = n - head, full = m / kRound * kRound;
  for (int base = threadIdx.x * kVec; base < full; base += kRound) {
    Vec<T, kVec> v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) v[u] = load_vec<T, kVec>(q + base + u * kGradThreads * kVec);
    float x[kUnroll * kVec];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int k = 0; k < kVec; ++k) x[u * kVec + k] = to_f32(v[u].v[k]);
    sum.add(sum_squares(x, safe));
  }
  int i = full + threadIdx.x * kVec;
  for (; i + kVec <= m; i += kGradThreads * kVec) {
    const Vec<T, kVec> v = load_vec<T, kVec>(q + i);
    float x[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) x[k] = to_f32(v.v[k]);
    sum.add(sum_squares(x, safe));
  }
  // what is left: the head, and less than a vector at the end
  const int tail = full + (m - full) / kVec * kVec;
  for (i = threadIdx.x; i < head + m - tail; i += kGradThreads) {
    const float x[1] = {to_f32(i < head ? p[i] : q[tail + i - head])};
    sum.add(sum_squares(x, safe));
  }
  return sum.hi + sum.lo;
}

// Sum over the block in fp64 with as few additions as there are values (a
// butterfly would make every lane add); every thread gets it.
__device__ __forceinline__ double block_tree(double x, double* red) {
  __syncthreads();  // `red` may still be read from the call before
  red[threadIdx.x] = x;
  for (int w = blockDim.x / 2; w > 0; w /= 2) {
    __syncthreads();
    if (int(threadIdx.x) < w) red[threadIdx.x] += red[threadIdx.x + w];
  }
  __syncthreads();
  return red[0];
}

// The first pass: each block adds up a chunk and writes one partial sum.  kUnroll
// loads per thread under way and blocks of one chunk keep it at the copy rate;
// with about 8000 chunks per call, and one more for each tensor, the partial sums
// stay few.
template <int N, class T>
__global__ void __launch_bounds__(kGradThreads) grad_norm_kernel(const __grid_constant__ GradTable<N> t, double* part) {
  __shared__ double red[kGradThreads];
  __shared__ float red32[32];
  griddep_release();  // the next kernel may be set up
  const int c = blockIdx.x, i = find_tensor(t, c);
  const int64_t begin = int64_t(c - (i ? t.chunk_end[i - 1] : 0)) * t.chunk;
  const int n = int(min(int64_t(t.chunk), t.numel[i] - begin));
  const T* p = static_cast<const T*>(t.src[i]) + begin;
  bool safe = true;
  const float s = chunk_norm(p, n, &safe);
  double all;  // of the chunk's squares
  if (!__syncthreads_or(!safe)) {
    all = double(block_sum(s, red32));
  } else {
    double d = 0.0;
    for (int k = threadIdx.x; k < n; k += kGradThreads) {
      const double x = double(to_f32(p[k]));
      d = fma(x, x, d);
    }
    all = block_tree(d, red);
  }
  if (threadIdx.x == 0) part[c] = all;
}

// Sum of the blocks' partial sums; `red` has blockDim.x values.
__device__ __forceinline__ double total(const double* part, int n, double* red) {
  double s = 0.0;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += blockDim.x) s += part[i];
  return block_tree(s, red);
}

// The partial sums' total where there are many, or where nothing is clipped: one
// block, in fp64 and in a fixed order.  It is latency: about 5 us behind 8000
// partial sums (34 M fp32 elements), 1 % of the head's two passes.
__global__ void __launch_bounds__(kTotalThreads) norm_total_kernel(const double* part, int n, float* norm) {
  __shared__ double red[kTotalThreads];
  griddep_release();
  griddep_wait();  // the partial sums are there
  const double s = total(part, n, red);
  if (threadIdx.x == 0) *norm = float(sqrt(s));
}

template <class T>
__device__ __forceinline__ void chunk_scale(const T* src, T* dst, int n, float c) {
  constexpr int kVec = Loads<T>::kVec, kRound = Loads<T>::kRound;
  // 16-byte loads and stores where both sides reach a boundary together
  if ((reinterpret_cast<uintptr_t>(src) - reinterpret_cast<uintptr_t>(dst)) % 16 == 0) {
    const int head = head_of(src, n), m = n - head;
    const T* q = src + head;
    T* o = dst + head;
    for (int base = threadIdx.x * kVec; base < m; base += kRound) {
      Vec<T, kVec> v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = base + u * kGradThreads * kVec;
        if (i + kVec <= m) v[u] = load_vec<T, kVec>(q + i);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = base + u * kGradThreads * kVec;
        if (i + kVec <= m) {
#pragma unroll
          for (int k = 0; k < kVec; ++k) v[u].v[k] = from_f32<T>(to_f32(v[u].v[k]) * c);
          store_vec<T, kVec>(o + i, v[u]);
        }
      }
    }
    const int tail = m / kVec * kVec;
    for (int i = threadIdx.x; i < head + m - tail; i += kGradThreads) {
      const int at = i < head ? i : head + tail + i - head;
      dst[at] = from_f32<T>(to_f32(src[at]) * c);
    }
    return;
  }
  constexpr int kSingles = 16;  // loads under way
  for (int base = threadIdx.x; base < n; base += kGradThreads * kSingles) {
    T x[kSingles];
#pragma unroll
    for (int u = 0; u < kSingles; ++u)
      if (base + u * kGradThreads < n) x[u] = src[base + u * kGradThreads];
#pragma unroll
    for (int u = 0; u < kSingles; ++u)
      if (base + u * kGradThreads < n) dst[base + u * kGradThreads] = from_f32<T>(to_f32(x[u]) * c);
  }
}

// min(1, max / (norm + 1e-6)) that keeps a NaN.
__device__ __forceinline__ float clip_factor(float norm, float max_norm) {
  const float c = max_norm / (norm + 1e-6f);
  return c > 1.0f ? 1.0f : c;
}

// The second pass.  Up to kFewParts partial sums every block adds up itself
// rather than wait for one more launch: 112 tensors of adapters (3.7 M bf16 elements)
// take 11.7 us for both passes.
template <int N, class T>
__global__ void __launch_bounds__(kGradThreads, 4) grad_scale_kernel(const __grid_constant__ GradTable<N> t,
                                                             const double* part, int n_part, float max_norm,
                                                             float* norm) {
  // n_part > 0: the norm is still to be added up, else *norm has it
  __shared__ double red[kGradThreads];
  griddep_release();
  griddep_wait();  // the partial sums, or the norm, are there
  float nm;
  if (n_part > 0) {
    nm = float(sqrt(total(part, n_part, red)));
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = nm;
  } else {
    nm = *norm;
  }
  const float f = clip_factor(nm, max_norm);
  // an infinite limit over an infinite norm is NaN; such a limit clips nothing
  const float c = max_norm == INFINITY && nm == nm ? 1.0f : f;
  // last chunks first: the norm's pass has just read them
  const int c0 = t.chunks - 1 - int(blockIdx.x), i = find_tensor(t, c0);
  if (c == 1.0f && t.src[i] == t.dst[i]) return;
  const int64_t begin = int64_t(c0 - (i ? t.chunk_end[i - 1] : 0)) * t.chunk;
  const int n = int(min(int64_t(t.chunk), t.numel[i] - begin));
  chunk_scale(static_cast<const T*>(t.src[i]) + begin, static_cast<T*>(t.dst[i]) + begin, n, c);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
constexpr int64_t kMaxElements = int64_t(1) << 42;  // of all tensors together

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
  int64_t elements = 0;
  for (int64_t i = 0; i < g.count; ++i) {
    if (!known_dtype(g.dtypes[i])) return FLCE_ERR_UNSUPPORTED_DTYPE;
    if (g.numel[i] < 0 || g.numel[i] > kMaxElements) return FLCE_ERR_INVALID_ARG;
    elements += g.numel[i];
    if (elements > kMaxElements) return FLCE_ERR_INVALID_ARG;
    if (g.numel[i] == 0) continue;
    if (!g.src[i] || (clip && !g.dst[i])) return FLCE_ERR_INVALID_ARG;
    const size_t e = elem_size(g.dtypes[i]);
    if (!aligned_to(g.src[i], e) || (clip && !aligned_to(g.dst[i], e))) return FLCE_ERR_MISALIGNED;
  }
  return FLCE_OK;
}

// Fills `t` with tensors of a type from index *next on, as many as fit.
template <int N>
void fill(GradTable<N>& t, const Grads& g, int32_t dtype, int64_t* next, int32_t chunk) {
  t.count = 0;
  t.chunks = 0;
  t.chunk = chunk;
  for (; *next < g.count && t.count < N; ++*next) {
    const int64_t i = *next;
    if (g.numel[i] == 0 || g.dtypes[i] != dtype) continue;
    t.src[t.count] = g.src[i];
    t.dst[t.count] = g.dst ? g.dst[i] : nullptr;
    t.numel[t.count] = g.numel[i];
    t.chunks += int32_t((g.numel[i] + chunk - 1) / chunk);
    t.chunk_end[t.count++] = t.chunks;
  }
}

// Calls launch(table, type) for tables that hold all tensors.
template <int N, class F>
int for_tables(const Grads& g, int32_t chunk, cudaStream_t st, F&& launch) {
  GradTable<N> t;
  auto of = [&](int32_t dtype, auto type) {
    for (int64_t next = 0; next < g.count;) {
      fill(t, g, dtype, &next, chunk);
      if (t.count) FLCE_TRY(logged(FLCE_LAUNCH_OTHER, st, [&] { return launch(t, type); }));
    }
    return int(FLCE_OK);
  };
  FLCE_TRY(of(FLCE_F32, float()));
  FLCE_TRY(of(FLCE_BF16, __nv_bfloat16()));
  return of(FLCE_F16, __half());
}

template <int N>
int run_tables(const Grads& g, bool clip, float max_norm, float* norm, double* part, cudaStream_t st) {
  int64_t elements = 0;
  for (int64_t i = 0; i < g.count; ++i) elements += g.numel[i];
  int32_t chunk = kMinChunk;  // at most 2^30 elements, for 2^42
  while (elements / chunk > kWantChunks) chunk *= 2;
  int parts = 0;
  FLCE_TRY(for_tables<N>(g, chunk, st, [&](const GradTable<N>& t, auto type) {
    grad_norm_kernel<N, decltype(type)><<<t.chunks, kGradThreads, 0, st>>>(t, part + parts);
    parts += t.chunks;
    return cudaGetLastError();
  }));
  const bool alone = !clip || parts == 0 || parts > kFewParts;
  if (alone)
    FLCE_TRY(logged(FLCE_LAUNCH_OTHER, st, [&] {
      return launch_dependent(norm_total_kernel, 1, kTotalThreads, st, static_cast<const double*>(part), parts, norm);
    }));
  if (!clip || parts == 0) return FLCE_OK;
  return for_tables<N>(g, chunk, st, [&](const GradTable<N>& t, auto type) {
    return launch_dependent(grad_scale_kernel<N, decltype(type)>, unsigned(t.chunks), kGradThreads, st, t,
                            static_cast<const double*>(part), alone ? 0 : parts, max_norm, norm);
  });
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
  LocalRanges src, dst;
  for (int64_t i = 0; i < g.count; ++i) {
    if (g.numel[i] == 0) continue;
    FLCE_TRY(check_local(dev, g.src[i], &src));
    if (clip && g.dst[i] != g.src[i]) FLCE_TRY(check_local(dev, g.dst[i], &dst));
  }
  double* part = static_cast<double*>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (g.count <= kSmallTable) return run_tables<kSmallTable>(g, clip, max_norm, norm, part, st);
  if (g.count <= kMediumTable) return run_tables<kMediumTable>(g, clip, max_norm, norm, part, st);
  return run_tables<kLargeTable>(g, clip, max_norm, norm, part, st);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_grad_norm_workspace_size(int64_t count, size_t* bytes) {
  if (!bytes || count < 0 || count > (int64_t(1) << 24)) return FLCE_ERR_INVALID_ARG;
  // one partial sum per block: at most kWantChunks + one for each tensor
  *bytes = size_t(kWantChunks + count + 32) * sizeof(double);
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
