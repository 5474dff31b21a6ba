// flce_logits.cu — logits of a batch of requests made ready for choosing a token
// (penalties for repeated tokens, biases, a grammar mask), with the greedy
// choice and the log-sum-exp from the same pass: kernels and the C entry point.
//
//   seen:  z = z > 0 ? z / rep : z * rep;   n > 0 times answered: z -= freq n, z -= pres
//   z += bias;   masked: z = -inf;   out = rn(z)
//   token = lowest argmax out,  lse = log sum exp out
//
// The bound is memory: logits read once, out written once.  A block takes a
// tile of one row's vocabulary; it counts the row's history into a table of the
// tile in shared memory (integer atomics: the order does not matter), so that
// the penalties are applied while the tile streams through registers.
#include <algorithm>
#include <cmath>

#include "flce_device.cuh"
#include "flce_elem.cuh"
#include "flce_host.h"

namespace flce {
namespace {

constexpr int kRowThreads = 256;
constexpr int64_t kMinTile = 1024;
constexpr int64_t kMaxTile = 16384;     // 64 KB of counts (and 64 KB of biases)
constexpr int64_t kWantBlocks = 608;    // four blocks on each of 152 SMs
constexpr uint32_t kPromptBit = 0x80000000u;

struct Partial {
  float m;       // largest out of the tile (NaN above all)
  float s;       // sum of e^(out - m)
  int32_t idx;   // lowest index of m
  int32_t pad;
};

struct LogitsParams {
  const void* logits;
  const void* tokens;
  const int64_t *lens, *prompt_lens;
  const float *repetition, *presence, *frequency;
  const void* bias_ids;
  const float* bias;
  const uint32_t* mask;
  void* out;
  Partial* part;   // [rows][tiles]
  int64_t ls, os, ts, bis, bs, ms;
  int64_t history;
  int32_t n_bias;
  int32_t vocab, tile, tiles;
  int32_t tokens_i64, bias_ids_i64;
};

// Running softmax statistics of one thread: indexes come in ascending order, so
// a strict comparison keeps the lowest.
struct Stat {
  float m = -INFINITY, s = 0.f;
  int idx = INT32_MAX;
};

// Whether (m, idx) of b goes before a's: a NaN above all, then the larger
// value, then the lower index.
__device__ __forceinline__ bool before(float bm, int bi, float am, int ai) {
  const bool bn = bm != bm, an = am != am;
  if (bn != an) return bn;
  if (!bn && bm != am) return bm > am;
  return bi < ai;
}

// e^(m - top) of a part of a sum, with nothing for an empty part.
__device__ __forceinline__ float rescale(float m, float top) {
  return m == -INFINITY ? 0.f : ex2_approx((m - top) * kLog2e);
}
__device__ __forceinline__ void merge(Stat& a, const Stat& b) {
  const bool take = before(b.m, b.idx, a.m, a.idx);
  const float top = take ? b.m : a.m;
  a.s = a.s * rescale(a.m, top) + b.s * rescale(b.m, top);
  if (take) a.idx = b.idx;
  a.m = top;
}
__device__ __forceinline__ void warp_merge(Stat& a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat b;
    b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    b.idx = __shfl_xor_sync(0xffffffffu, a.idx, o);
    // both sides of a pair add in the same order
    if ((threadIdx.x & o) == 0) {
      merge(a, b);
    } else {
      merge(b, a);
      a = b;
    }
  }
}

__device__ __forceinline__ int64_t load_id(const void* p, int i64, int64_t i) {
  return i64 ? static_cast<const int64_t*>(p)[i] : int64_t(static_cast<const int32_t*>(p)[i]);
}

// Counts the row's history into the tile's table.
__device__ __forceinline__ void count_history(const LogitsParams& p, int64_t row, int v0, int n, uint32_t* counts) {
  const int64_t len = p.lens ? min(max(p.lens[row], int64_t(0)), p.history) : p.history;
  const int64_t prompt = p.prompt_lens ? min(max(p.prompt_lens[row], int64_t(0)), p.history) : 0;
  for (int64_t i = threadIdx.x; i < len; i += kRowThreads) {
    const int64_t at = load_id(p.tokens, p.tokens_i64, row * p.ts + i) - v0;
    if (at >= 0 && at < n) {
      if (i < prompt) {
        atomicOr(&counts[at], kPromptBit);
      } else {
        atomicAdd(&counts[at], 1u);
      }
    }
  }
}

// Adds the row's biases to the tile's table, entry by entry in order: one warp,
// 32 entries at a time; of the lanes with the same id, the lowest adds all.
__device__ __forceinline__ void add_biases(const LogitsParams& p, int64_t row, int v0, int n, float* biases) {
  const int lane = threadIdx.x & 31;
  for (int base = 0; base < p.n_bias; base += 32) {
    const int i = base + lane;
    int at = -1;
    float b = 0.f;
    if (i < p.n_bias) {
      const int64_t a = load_id(p.bias_ids, p.bias_ids_i64, row * p.bis + i) - v0;
      if (a >= 0 && a < n) {
        at = int(a);
        b = p.bias[row * p.bs + i];
      }
    }
    const uint32_t same = __match_any_sync(0xffffffffu, at);
    const bool lead = at >= 0 && lane == __ffs(same) - 1;
    float sum = lead ? biases[at] : 0.f;
    uint32_t todo = same;
    while (__any_sync(0xffffffffu, lead && todo != 0)) {
      const int src = todo ? __ffs(todo) - 1 : lane;
      const float x = __shfl_sync(0xffffffffu, b, src);
      if (lead && todo) sum += x;
      todo &= todo - 1;
    }
    if (lead) biases[at] = sum;
    __syncwarp();
  }
}

// One step of the chain for an entry of the history.
__device__ __forceinline__ float penalise(float z, uint32_t word, float rep, float pres, float freq, bool has_rep) {
  if (has_rep) z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
  const uint32_t n = word & ~kPromptBit;
  if (n) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, float(n))), pres);
  return z;
}

template <class T, class O, int V>
__global__ void __launch_bounds__(kRowThreads) process_logits_kernel(LogitsParams p) {
  extern __shared__ __align__(16) uint32_t table[];
  __shared__ Stat red[kRowThreads / 32];
  const int64_t row = blockIdx.x / p.tiles;
  const int tile = int(blockIdx.x % p.tiles);
  const int v0 = tile * p.tile;
  const int n = min(p.tile, p.vocab - v0);
  uint32_t* counts = table;
  float* biases = reinterpret_cast<float*>(table + (p.tokens ? p.tile : 0));
  if (p.tokens || p.n_bias) {
    const int words = (p.tokens ? p.tile : 0) + (p.n_bias ? p.tile : 0);
    for (int i = threadIdx.x * 4; i < words; i += kRowThreads * 4) *reinterpret_cast<uint4*>(table + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (p.n_bias && threadIdx.x < 32) add_biases(p, row, v0, n, biases);
    if (p.tokens) count_history(p, row, v0, n, counts);
    __syncthreads();
  }
  const bool has_rep = p.repetition != nullptr;
  const float rep = has_rep ? p.repetition[row] : 1.f;
  const float pres = p.presence ? p.presence[row] : 0.f;
  const float freq = p.frequency ? p.frequency[row] : 0.f;
  const T* logits = static_cast<const T*>(p.logits) + row * p.ls + v0;
  O* out = static_cast<O*>(p.out) + row * p.os + v0;
  const uint32_t* mask = p.mask ? p.mask + row * p.ms + v0 / 32 : nullptr;
  Stat st;
  for (int i = threadIdx.x * V; i < n; i += kRowThreads * V) {
    const Vec<T, V> x = load_vec<T, V>(logits + i);
    // V divides 32 and the tile is a multiple of 32: a vector's bits are in one word
    const uint32_t bits = mask ? mask[i / 32] >> (i % 32) : 0xffffffffu;
    Vec<O, V> o;
    float f[V];
    float top = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float z = to_f32(x.v[k]);
      if (p.tokens) {
        const uint32_t word = counts[i + k];
        if (word) z = penalise(z, word, rep, pres, freq, has_rep);
      }
      if (p.n_bias) {
        const float b = biases[i + k];
        if (b != 0.f) z = __fadd_rn(z, b);
      }
      if (!((bits >> k) & 1u)) z = -INFINITY;
      o.v[k] = from_f32<O>(z);
      f[k] = to_f32(o.v[k]);
      nan |= f[k] != f[k];
      top = fmaxf(top, f[k]);
    }
    store_vec<O, V>(out + i, o);
    if (nan || top > st.m) {  // rare once a large value has been met
      const float old = st.m;
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (before(f[k], v0 + i + k, st.m, st.idx)) {
          st.m = f[k];
          st.idx = v0 + i + k;
        }
      st.s *= rescale(old, st.m);
    }
    if (st.m != -INFINITY) {
      // the difference first: m * log2(e) overflows for values near the type's lowest
#pragma unroll
      for (int k = 0; k < V; ++k) st.s += ex2_approx((f[k] - st.m) * kLog2e);
    }
  }
  warp_merge(st);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = st;
  __syncthreads();
  if (threadIdx.x < 32) {
    if (threadIdx.x < kRowThreads / 32) st = red[threadIdx.x]; else st = Stat();
    warp_merge(st);
    if (threadIdx.x == 0) p.part[row * p.tiles + tile] = Partial{st.m, st.s, st.idx, 0};
  }
}

// One warp per row joins the tiles' statistics.
__global__ void __launch_bounds__(kRowThreads) merge_logits_kernel(const Partial* part, int64_t rows, int tiles,
                                                               int64_t* token, float* lse) {
  const int64_t row = blockIdx.x * int64_t(kRowThreads / 32) + (threadIdx.x >> 5);
  if (row >= rows) return;
  Stat st;
  for (int i = threadIdx.x & 31; i < tiles; i += 32) {
    const Partial q = part[row * tiles + i];
    Stat b;
    b.m = q.m;
    b.s = q.s;
    b.idx = q.idx;
    merge(st, b);
  }
  warp_merge(st);
  if ((threadIdx.x & 31) == 0) {
    const bool none = st.m == -INFINITY;
    if (token) token[row] = none ? -1 : int64_t(st.idx);
    // an infinite or NaN maximum is the sum
    if (lse) lse[row] = none || st.m == INFINITY || st.m != st.m ? st.m : st.m + logf(st.s);
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tile width: enough blocks to fill the GPU, within what shared memory holds.
int64_t plan_tile(int64_t rows, int64_t vocab) {
  const int64_t per_row = std::max<int64_t>(1, cdiv(kWantBlocks, std::max<int64_t>(rows, 1)));
  const int64_t tile = cdiv(cdiv(vocab, per_row), 128) * 128;
  return std::min(std::max(tile, kMinTile), kMaxTile);
}

int validate(const flce_logits_problem* p) {
  if (!p) return FLCE_ERR_INVALID_ARG;
  if (p->rows < 0 || p->vocab < 1 || p->vocab > (int64_t(1) << 30)) return FLCE_ERR_INVALID_ARG;
  if (p->history < 0 || p->history > INT32_MAX || p->n_bias < 0 || p->n_bias > INT32_MAX - 32)
    return FLCE_ERR_INVALID_ARG;
  if (p->rows > INT32_MAX / cdiv(p->vocab, plan_tile(p->rows, p->vocab))) return FLCE_ERR_INVALID_ARG;
  if (p->logits_stride < 0 || p->tokens_stride < 0 || p->bias_ids_stride < 0 || p->bias_stride < 0 ||
      p->mask_stride < 0 || (p->rows > 1 && p->out_stride < p->vocab) || p->out_stride < 0)
    return FLCE_ERR_INVALID_ARG;
  if (!known_dtype(p->logits_dtype) || !known_dtype(p->out_dtype)) return FLCE_ERR_UNSUPPORTED_DTYPE;
  if (p->out_dtype != p->logits_dtype && p->out_dtype != FLCE_F32) return FLCE_ERR_DTYPE_MISMATCH;
  return FLCE_OK;
}

template <class T, class O, int V>
cudaError_t launch(const LogitsParams& p, int64_t rows, cudaStream_t st) {
  const size_t smem = size_t(p.tile) * 4 * ((p.tokens ? 1 : 0) + (p.n_bias ? 1 : 0));
  auto kern = process_logits_kernel<T, O, V>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMaxTile * 8));
  if (e != cudaSuccess) return e;
  kern<<<unsigned(rows * p.tiles), kRowThreads, smem, st>>>(p);
  return cudaGetLastError();
}
template <class T, class O>
cudaError_t launch_types(const LogitsParams& p, int64_t rows, bool vec, cudaStream_t st) {
  // the last vector of a row must be whole
  constexpr int kV = 16 / sizeof(T);
  if (vec && p.vocab % kV == 0) return launch<T, O, kV>(p, rows, st);
  return launch<T, O, 1>(p, rows, st);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_process_logits_workspace_size(const flce_logits_problem* problem, size_t* bytes) {
  if (!bytes) return FLCE_ERR_INVALID_ARG;
  FLCE_TRY(validate(problem));
  *bytes = size_t(problem->rows) * size_t(cdiv(problem->vocab, plan_tile(problem->rows, problem->vocab))) *
               sizeof(Partial) + 256;
  return FLCE_OK;
}

int flce_process_logits(const flce_logits_problem* problem, const void* logits, const void* tokens,
                        const int64_t* lens, const int64_t* prompt_lens, const float* repetition,
                        const float* presence, const float* frequency, const void* bias_ids, const float* bias,
                        const void* mask, void* out, int64_t* token, float* lse, void* workspace,
                        size_t workspace_bytes, flce_stream_t stream) {
  const flce_logits_problem* p = problem;
  size_t need = 0;
  FLCE_TRY(flce_process_logits_workspace_size(p, &need));
  if (p->rows == 0) return FLCE_OK;
  if (!logits || !out || !workspace) return FLCE_ERR_INVALID_ARG;
  if (!tokens && (lens || prompt_lens || repetition || presence || frequency)) return FLCE_ERR_INVALID_ARG;
  if ((bias_ids != nullptr) != (bias != nullptr)) return FLCE_ERR_INVALID_ARG;
  const size_t el = elem_size(p->logits_dtype), eo = elem_size(p->out_dtype);
  if (!aligned_to(logits, el) || !aligned_to(out, eo) || !aligned_to(tokens, p->tokens_i64 ? 8 : 4) ||
      !aligned_to(lens, 8) || !aligned_to(prompt_lens, 8) || !aligned_to(repetition, 4) || !aligned_to(presence, 4) ||
      !aligned_to(frequency, 4) || !aligned_to(bias_ids, p->bias_ids_i64 ? 8 : 4) || !aligned_to(bias, 4) ||
      !aligned_to(mask, 4) || !aligned_to(token, 8) || !aligned_to(lse, 4) || !aligned_to(workspace, 16))
    return FLCE_ERR_MISALIGNED;
  if (workspace_bytes < need) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  DeviceInfo dev;
  FLCE_TRY(get_device(&dev));
  FLCE_TRY(check_local(dev, logits, tokens, lens, prompt_lens, repetition, presence, frequency, bias_ids, bias, mask,
                       out, token, lse, workspace));
  LogitsParams q{};
  q.logits = logits;
  q.tokens = p->history > 0 ? tokens : nullptr;
  q.lens = lens;
  q.prompt_lens = prompt_lens;
  q.repetition = repetition;
  q.presence = presence;
  q.frequency = frequency;
  q.bias_ids = bias_ids;
  q.bias = bias;
  q.mask = static_cast<const uint32_t*>(mask);
  q.out = out;
  q.part = static_cast<Partial*>(workspace);
  q.ls = p->logits_stride;
  q.os = p->out_stride;
  q.ts = p->tokens_stride;
  q.bis = p->bias_ids_stride;
  q.bs = p->bias_stride;
  q.ms = p->mask_stride;
  q.history = p->history;
  q.n_bias = bias ? int32_t(p->n_bias) : 0;
  q.vocab = int32_t(p->vocab);
  q.tile = int32_t(plan_tile(p->rows, p->vocab));
  q.tiles = int32_t(cdiv(p->vocab, q.tile));
  q.tokens_i64 = p->tokens_i64;
  q.bias_ids_i64 = p->bias_ids_i64;
  const bool vec = aligned_to(logits, 16) && aligned_to(out, 16) &&
                   (p->rows == 1 || (p->logits_stride * el % 16 == 0 && p->out_stride * eo % 16 == 0));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  FLCE_TRY(logged(FLCE_LAUNCH_OTHER, st, [&] {
    if (p->logits_dtype == FLCE_F32) return launch_types<float, float>(q, p->rows, vec, st);
    if (p->logits_dtype == FLCE_BF16)
      return p->out_dtype == FLCE_F32 ? launch_types<__nv_bfloat16, float>(q, p->rows, vec, st)
                                      : launch_types<__nv_bfloat16, __nv_bfloat16>(q, p->rows, vec, st);
    return p->out_dtype == FLCE_F32 ? launch_types<__half, float>(q, p->rows, vec, st)
                                    : launch_types<__half, __half>(q, p->rows, vec, st);
  }));
  if (!token && !lse) return FLCE_OK;
  return logged(FLCE_LAUNCH_OTHER, st, [&] {
    merge_logits_kernel<<<unsigned(cdiv(p->rows, kRowThreads / 32)), kRowThreads, 0, st>>>(q.part, p->rows, q.tiles, token,
                                                                                     lse);
    return cudaGetLastError();
  });
}

}  // extern "C"
