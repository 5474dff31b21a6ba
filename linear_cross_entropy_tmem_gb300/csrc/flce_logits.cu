// flce_logits.cu — logits of a batch of requests made ready for choosing a token
// (penalties for repeated tokens, biases, a grammar mask), with the greedy
// choice and the log-sum-exp from the same pass: kernels and the C entry point.
//
//   seen:  z = z > 0 ? z / rep : z * rep;   n > 0 times answered: z -= freq n, z -= pres
//   z += bias;   masked: z = -inf;   out = rn(z)
//   token = lowest argmax out,  lse = log sum exp out
//
// The bound is memory: logits read once, out written once.  A block takes a
// tile of one row's vocabulary and holds it in registers: its loads are issued
// first, and while they are under way the block works on the few entries that
// the row's history and biases name.  It counts the history into a table of the
// tile in shared memory (integer atomics: their order does not matter), then
// one thread per named entry works out its new value, leaves it in the table
// and marks it in a bitmap.  The dense pass only looks at the bitmap: a test per
// vector instead of a table look-up and a division's code per entry.  Rounding,
// maximum and sum come from registers, the maximum before the first exponential.
//
// 256 x 262144 fp32 to fp32: 81 us without options, what the copy rate gives;
// 98 us with a mask and 300 biases, 126 us with histories of up to 2048 as well.
// Each of a row's blocks scans the whole history for its own tile, and that scan
// with its atomics and barriers is what keeps the blocks from their loads.
// Smaller tiles scan more often, larger ones leave fewer blocks to overlap:
// 128 threads 142 us, 16 entries per thread 168, 512 threads 171, four blocks on
// an SM (registers spill) 161, the next ids loaded ahead (they do as well) 142, a
// history shared by a cluster of 8 blocks 199, a kernel of its own for the named
// entries 124 (but 12 us in place of 8 for a single row, 37 in place of 23 for 64).
#include <algorithm>
#include <cmath>

#include "flce_device.cuh"
#include "flce_elem.cuh"
#include "flce_host.h"

namespace flce {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kMaxPerThread = 32;       // entries a thread holds, at most: a tile of 8192
constexpr int kMaxSingles = 16;         // the same without vectors (a mask word per entry takes registers)
constexpr int64_t kWantBlocks = 456;    // three blocks on each of a GB300's 152 SMs: the workspace's size depends on
                                        // it, and that query needs no GPU
constexpr uint32_t kFull = 0xffffffffu;
constexpr int64_t kMaxIds = (int64_t(1) << 30) - 1;  // of a row's history, and of its biases

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
  int32_t vocab, tiles;
  int32_t tokens_i64, bias_ids_i64;
};

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

// e^(m - top) of a part of a sum, with nothing for an empty part.  (The
// difference first: m * log2(e) overflows for values near the type's lowest.)
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
    b.m = __shfl_xor_sync(kFull, a.m, o);
    b.s = __shfl_xor_sync(kFull, a.s, o);
    b.idx = __shfl_xor_sync(kFull, a.idx, o);
    // both sides of a pair add in the same order
    if ((threadIdx.x & o) == 0) {
      merge(a, b);
    } else {
      merge(b, a);
      a = b;
    }
  }
}

// The largest of three values, a NaN if any is one.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Largest value over the warp (NaN above all), by the order of its bits as a
// signed integer; -0 counts as +0.
__device__ __forceinline__ float warp_max(float x) {
  const int bits = x != x ? 0x7fffffff : __float_as_int(x + 0.f);
  const int key = bits >= 0 ? bits : bits ^ 0x7fffffff;
  const int top = __reduce_max_sync(kFull, key);
  return __int_as_float(top >= 0 ? top : top ^ 0x7fffffff);
}

// The entries of a tile: places [0, tile) stand for [first, first + tile), of
// which `count` from `begin` on are in the row.
struct Span {
  int first, begin, count;
};
// An id's place in the tile, or -1 (padding among them).
__device__ __forceinline__ int place(const Span& s, int64_t id) {
  const int lo = int(id);
  return (id >> 32) == 0 && unsigned(lo - s.begin) < unsigned(s.count) ? lo - s.first : -1;
}
__device__ __forceinline__ int place(const Span& s, int32_t id) {
  return unsigned(id - s.begin) < unsigned(s.count) ? id - s.first : -1;
}

// A list of ids read by the block, kIds of them per thread under way at once.
constexpr int kIds = 8;
constexpr int kIdsBlock = kIds * kRowThreads;
constexpr int kBiases = 2;  // biases per thread that are read at the start
struct Ids {
  const void* p;
  int i64;
  __device__ __forceinline__ void load(int base, int n, const Span& s, int (&at)[kIds]) const {
    if (i64) {
      load(static_cast<const int64_t*>(p), base, n, s, at);
    } else {
      load(static_cast<const int32_t*>(p), base, n, s, at);
    }
  }
  template <class Id>
  __device__ __forceinline__ void load(const Id* ids, int base, int n, const Span& s, int (&at)[kIds]) const {
    Id id[kIds];
#pragma unroll
    for (int u = 0; u < kIds; ++u) {
      const int i = base + u * kRowThreads + int(threadIdx.x);
      id[u] = i < n ? ids[i] : Id(-1);
    }
#pragma unroll
    for (int u = 0; u < kIds; ++u) at[u] = place(s, id[u]);
  }
  __device__ __forceinline__ int one(int i, const Span& s) const {
    return i64 ? place(s, static_cast<const int64_t*>(p)[i]) : place(s, static_cast<const int32_t*>(p)[i]);
  }
};

// Sum of a row's biases of vocabulary entry v, in the list's order; whole warps.
__device__ __forceinline__ float bias_sum(const Ids& ids, const float* bias, int n, int v) {
  const Span one = {v, v, 1};
  float sum = 0.f;
  for (int base = 0; base < n; base += 32) {
    const int i = base + int(threadIdx.x & 31);
    const bool hit = i < n && ids.one(i, one) == 0;
    const float b = hit ? bias[i] : 0.f;
    for (uint32_t m = __ballot_sync(kFull, hit); m; m &= m - 1) sum = __fadd_rn(sum, __shfl_sync(kFull, b, __ffs(m) - 1));
  }
  return sum;
}

// Steps 1 and 2 of the chain for an entry of the history, answered n times.
__device__ __forceinline__ float penalise(float z, uint32_t n, float rep, float pres, float freq, bool has_rep) {
  if (has_rep) z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
  if (n) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, float(n))), pres);
  return z;
}

// A tile's marks: bit i of the bitmap for place i.
__device__ __forceinline__ bool marked(const uint32_t* map, int at) { return (map[at >> 5] >> (at & 31)) & 1u; }
// Marks a place; true for the one call that does.
__device__ __forceinline__ bool mark(uint32_t* map, int at) {
  const uint32_t bit = 1u << (at & 31);
  return !(atomicOr(&map[at >> 5], bit) & bit);
}

// What the row's history and biases say of a tile, in shared memory.
template <int kTile>
struct Named {
  uint32_t table[kTile];      // how often an entry was answered; then, at the marked places, new values
  uint32_t map[kTile / 32];   // marks: places of the history, then of the biases too
  uint32_t seen[kTile / 32];  // places that a bias names
  int biased, twice;          // whether a bias names a place, or one twice
  int pad[2];
  uint16_t list[kTile];       // the places that the history names, a part for each warp
};

// Counts the id at place `at` (-1: none): its mark, and if it was answered its
// count.  Predicated rather than branched to, and nothing comes back, so nothing
// waits.
template <int kTile>
__device__ __forceinline__ void count_id(Named<kTile>& s, int at, bool answered) {
  const int to = max(at, 0);
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ge.s32 p, %2, 0;\n\t"
      "setp.ne.and.u32 q, %3, 0, p;\n\t"
      "@p red.shared.or.b32 [%0], %4;\n\t"
      "@q red.shared.add.u32 [%1], 1;\n\t}"
      ::"r"(smem_u32(&s.map[to >> 5])), "r"(smem_u32(&s.table[to])), "r"(at), "r"(uint32_t(answered)),
      "r"(1u << (to & 31))
      : "memory");
}

// 1 x 151936 fp32 with everything: 8 us, of which a launch and its merge are 4.
// A block's tile is kRowThreads * V * NV entries; thread t holds the vectors at
// (t + i * kRowThreads) * V.  Vectors are aligned in memory: a row whose first
// element is `shift` elements past a 16-byte boundary starts `shift` entries
// into its first vector (V = 1: no shift).
template <class T, class O, int V, int NV>
__global__ void __launch_bounds__(kRowThreads, V * NV > 16 ? 3 : 4) process_logits_kernel(LogitsParams p) {
  constexpr int kTile = kRowThreads * V * NV;
  extern __shared__ __align__(16) uint32_t smem[];
  Named<kTile>& s = *reinterpret_cast<Named<kTile>*>(smem);
  __shared__ Stat red[kRowWarps];
  griddep_release();  // the merge may be set up
  const int64_t row = blockIdx.x / unsigned(p.tiles);
  const int tile = int(blockIdx.x % unsigned(p.tiles));
  const T* logits = static_cast<const T*>(p.logits) + row * p.ls;
  O* out = static_cast<O*>(p.out) + row * p.os;
  const int shift = V == 1 ? 0 : int((reinterpret_cast<uintptr_t>(logits) / sizeof(T)) % V);
  Span span;
  span.first = tile * kTile - shift;  // < 0 in a shifted first tile
  span.begin = max(span.first, 0);
  span.count = max(0, min(span.first + kTile, p.vocab) - span.begin);  // 0: the row ends before the tile
  const int first = span.first;

  // The loads of the lists go out before the tile's.  The first ids are loaded
  // whatever the row's length.
  const bool named = p.tokens || p.n_bias;
  const int history = p.tokens ? int(p.history) : 0;
  const Ids ids = {p.tokens_i64 ? static_cast<const void*>(static_cast<const int64_t*>(p.tokens) + row * p.ts)
                                : static_cast<const void*>(static_cast<const int32_t*>(p.tokens) + row * p.ts),
                   p.tokens_i64};
  const Ids bias_ids = {p.bias_ids_i64
                            ? static_cast<const void*>(static_cast<const int64_t*>(p.bias_ids) + row * p.bis)
                            : static_cast<const void*>(static_cast<const int32_t*>(p.bias_ids) + row * p.bis),
                        p.bias_ids_i64};
  int ids_at[kIds];
  int bias_at[kBiases];
  const int64_t len64 = history && p.lens ? p.lens[row] : history;
  const int64_t prompt64 = history && p.prompt_lens ? p.prompt_lens[row] : 0;
  if (history) ids.load(0, history, span, ids_at);
#pragma unroll
  for (int u = 0; u < kBiases; ++u) {
    const int i = u * kRowThreads + int(threadIdx.x);
    bias_at[u] = i < p.n_bias ? bias_ids.one(i, span) : -1;
  }
  Vec<T, V> x[NV];   // as loaded: a conversion here would wait for its load before the next is issued
  uint32_t bits[NV];
  const bool inner = first >= 0 && first + kTile <= p.vocab;
  if (inner) {
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = load_vec<T, V>(logits + first + (int(threadIdx.x) + i * kRowThreads) * V);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = first + (int(threadIdx.x) + i * kRowThreads) * V;
      if (v >= 0 && v + V <= p.vocab) {
        x[i] = load_vec<T, V>(logits + v);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
          x[i].v[k] = v + k >= 0 && v + k < p.vocab ? logits[v + k] : from_f32<T>(-INFINITY);
      }
    }
  }
  if (!p.mask) {
#pragma unroll
    for (int i = 0; i < NV; ++i) bits[i] = kFull;
  } else {
    const uint32_t* m = p.mask + row * p.ms;
    const int words = (p.vocab + 31) >> 5;
    if (shift == 0) {  // V divides 32: a vector's bits are in one word
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int w = (first + (int(threadIdx.x) + i * kRowThreads) * V) >> 5;
        bits[i] = w < words ? m[w] : 0u;
      }
    } else {  // in one word or two
      uint32_t next[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int w = (first + (int(threadIdx.x) + i * kRowThreads) * V) >> 5;  // -1: before the row
        bits[i] = w >= 0 && w < words ? m[w] : 0u;
        next[i] = w + 1 < words ? m[w + 1] : 0u;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = first + (int(threadIdx.x) + i * kRowThreads) * V;
        // kept rotated, as a whole word is
        const uint32_t w = __funnelshift_r(bits[i], next[i], v & 31);
        bits[i] = __funnelshift_l(w, w, v & 31);
      }
    }
  }

  if (named) {
    constexpr int kWords = kTile + 2 * (kTile / 32) + 4;  // up to the list
    for (int i = threadIdx.x * 4; i < kWords; i += kRowThreads * 4)
      *reinterpret_cast<uint4*>(smem + i) = make_uint4(0, 0, 0, 0);
    const int len = int(min(max(len64, int64_t(0)), int64_t(history)));
    const int prompt = int(min(max(prompt64, int64_t(0)), int64_t(history)));
    const bool has_rep = p.repetition != nullptr;
    const float rep = has_rep ? p.repetition[row] : 1.f;
    const float pres = p.presence ? p.presence[row] : 0.f;
    const float freq = p.frequency ? p.frequency[row] : 0.f;
    __syncthreads();

    // Count the history; mark what the biases name.
    for (int base = 0; base < len; base += kIdsBlock) {
      if (base) ids.load(base, len, span, ids_at);
#pragma unroll
      for (int u = 0; u < kIds; ++u) {
        const int i = base + u * kRowThreads + int(threadIdx.x);
        count_id(s, i < len ? ids_at[u] : -1, i >= prompt);
      }
    }
    auto name = [&](int at) {
      if (at >= 0) {
        s.biased = 1;
        if (!mark(s.seen, at)) s.twice = 1;
      }
    };
#pragma unroll
    for (int u = 0; u < kBiases; ++u) name(bias_at[u]);
    for (int i = kBiases * kRowThreads + threadIdx.x; i < p.n_bias; i += kRowThreads) name(bias_ids.one(i, span));
    __syncthreads();

    // A warp lists the places of its words of the map (every eighth, as marks may
    // crowd), and a lane per place works out its value from the logit (in L1: the
    // tile's loads have just passed there).
    const int lane = threadIdx.x & 31, word = lane * kRowWarps + (threadIdx.x >> 5);
    uint32_t places = word < kTile / 32 ? s.map[word] : 0u;
    int upto = __popc(places);  // places of the lanes up to this one
    int pos = -upto;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int other = __shfl_up_sync(kFull, upto, o);
      if (lane >= o) upto += other;
    }
    pos += upto;
    const int n = __shfl_sync(kFull, upto, 31);
    uint16_t* list = s.list + (threadIdx.x >> 5) * (kTile / kRowWarps);
    for (; places; places &= places - 1) list[pos++] = uint16_t(word * 32 + __ffs(places) - 1);
    __syncwarp();
    constexpr int kLoads = 4;  // under way at once
    for (int base = lane; base < n; base += 32 * kLoads) {
      int at[kLoads];
      float z[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        at[u] = base + u * 32 < n ? int(list[base + u * 32]) : -1;
        if (at[u] >= 0) z[u] = to_f32(logits[first + at[u]]);
      }
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
        if (at[u] >= 0) s.table[at[u]] = __float_as_uint(penalise(z[u], s.table[at[u]], rep, pres, freq, has_rep));
    }
    __syncthreads();
    if (s.biased) {
      const float* bias = p.bias + row * p.bs;
      auto add = [&](int at, float b) {
        const float z = marked(s.map, at) ? __uint_as_float(s.table[at]) : to_f32(logits[first + at]);
        s.table[at] = __float_as_uint(__fadd_rn(z, b));
        mark(s.map, at);
      };
      if (!s.twice) {
        for (int i = threadIdx.x; i < p.n_bias; i += kRowThreads) {
          const int at = bias_ids.one(i, span);
          if (at >= 0) add(at, bias[i]);
        }
      } else {  // some entry has several: their sum, in the list's order, once
        for (int i = threadIdx.x >> 5; i < p.n_bias; i += kRowWarps) {
          const int at = bias_ids.one(i, span);
          if (at < 0) continue;
          bool first_one = true;
          for (int j = threadIdx.x & 31; j < i; j += 32) first_one &= bias_ids.one(j, span) != at;
          if (!__all_sync(kFull, first_one)) continue;
          const float sum = bias_sum(bias_ids, bias, p.n_bias, first + at);
          if ((threadIdx.x & 31) == 0) add(at, sum);
        }
      }
      __syncthreads();
    }
  }

  // `at_top` is the lowest vector with the thread's maximum; which of its
  // entries it is, the merge looks up in `out`.
  float top = -INFINITY;
  int at_top = INT32_MAX;
  float f[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (int(threadIdx.x) + i * kRowThreads) * V;
    const int v = first + at;
    const uint32_t allowed = __funnelshift_r(bits[i], bits[i], v & 31);  // rotated: bit k for entry v + k
#pragma unroll
    for (int k = 0; k < V; ++k) f[i][k] = to_f32(x[i].v[k]);
    if (named) {
      const uint32_t w = s.map[at >> 5] >> (at & 31);
      if (w & ((1u << V) - 1)) {
#pragma unroll
        for (int k = 0; k < V; ++k)
          if ((w >> k) & 1u) f[i][k] = __uint_as_float(s.table[at + k]);
      }
    }
    Vec<O, V> o;
    float t = -INFINITY;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (!((allowed >> k) & 1u)) f[i][k] = -INFINITY;
      o.v[k] = from_f32<O>(f[i][k]);
      f[i][k] = to_f32(o.v[k]);
    }
    // entries outside the row are -inf
    if constexpr (V == 1) {
      t = f[i][0];
    } else {
#pragma unroll
      for (int k = 0; k < V; k += 2) t = max3_nan(t, f[i][k], f[i][k + 1]);
    }
    if (t > top || (t != t && top == top)) {
      top = t;
      at_top = v;
    }
    if (inner || (v >= 0 && v + V <= p.vocab)) {
      store_vec<O, V>(out + v, o);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (v + k >= 0 && v + k < p.vocab) out[v + k] = o.v[k];
    }
  }

  Stat st;
  st.m = warp_max(top);
  st.idx = __reduce_min_sync(kFull, top == st.m || (top != top && st.m != st.m) ? at_top : INT32_MAX);
  if (st.m != -INFINITY) {
    if constexpr (V == 1) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) sum += ex2_approx((f[i][0] - st.m) * kLog2e);
      st.s = warp_sum(sum);
    } else {  // two lanes of fp32 per instruction
      const uint64_t neg = f2_splat(-st.m), l2e = f2_splat(kLog2e);
      uint64_t sum = f2_splat(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; k += 2) {
          float a, b;
          f2_unpack(f2_mul(f2_add(f2_pack(f[i][k], f[i][k + 1]), neg), l2e), a, b);
          sum = f2_add(sum, f2_pack(ex2_approx(a), ex2_approx(b)));
        }
      float a, b;
      f2_unpack(sum, a, b);
      st.s = warp_sum(a + b);
    }
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = st;
  __syncthreads();
  if (threadIdx.x < 32) {
    if (threadIdx.x < kRowWarps) st = red[threadIdx.x]; else st = Stat();
    warp_merge(st);
    if (threadIdx.x == 0) p.part[row * p.tiles + tile] = Partial{st.m, st.s, st.idx, 0};
  }
}

// One warp per row joins the tiles' statistics, and finds the first entry of
// the vector of `vec` that holds the maximum.  Set up while the tiles' kernel
// runs: it adds 1.5 us or so of latency and no traffic to speak of.
template <class O>
__global__ void __launch_bounds__(kRowThreads) merge_logits_kernel(const Partial* part, int64_t rows, int tiles,
                                                                  const O* out, int64_t os, int vocab, int vec,
                                                                  int64_t* token, float* lse) {
  const int64_t row = blockIdx.x * int64_t(kRowWarps) + (threadIdx.x >> 5);
  if (row >= rows) return;
  griddep_wait();  // the tiles' statistics are there
  const int lane = threadIdx.x & 31;
  Stat st;
  for (int i = lane; i < tiles; i += 32) {
    const Partial q = part[row * tiles + i];
    Stat b;
    b.m = q.m;
    b.s = q.s;
    b.idx = q.idx;
    merge(st, b);
  }
  warp_merge(st);
  const bool none = st.m == -INFINITY;
  if (token) {
    bool hit = false;
    const int v = st.idx + lane;
    if (!none && lane < vec && v >= 0 && v < vocab) {
      const float x = to_f32(out[row * os + v]);
      hit = x == st.m || (x != x && st.m != st.m);
    }
    const uint32_t hits = __ballot_sync(kFull, hit);
    if (lane == 0) token[row] = hits ? int64_t(st.idx + __ffs(hits) - 1) : -1;
  }
  // an infinite or NaN maximum is the sum
  if (lse && lane == 0) lse[row] = none || st.m == INFINITY || st.m != st.m ? st.m : st.m + logf(st.s);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Entries per thread: as many as the registers hold, fewer where the blocks
// would not fill the GPU.  (A tile of a row may start up to 7 places early.)
int plan_per_thread(int64_t rows, int64_t vocab) {
  int per = kMaxPerThread;
  while (per > 4 && std::max<int64_t>(rows, 1) * cdiv(vocab + 7, kRowThreads * per) < kWantBlocks) per /= 2;
  return per;
}
// Tiles of a row at most, whatever the form below.
int64_t plan_tiles(int64_t rows, int64_t vocab) {
  return cdiv(vocab + 7, int64_t(kRowThreads) * std::min(kMaxSingles, plan_per_thread(rows, vocab)));
}

int validate(const flce_logits_problem* p) {
  if (!p) return FLCE_ERR_INVALID_ARG;
  if (p->rows < 0 || p->vocab < 1 || p->vocab > (int64_t(1) << 30)) return FLCE_ERR_INVALID_ARG;
  if (p->history < 0 || p->history > kMaxIds || p->n_bias < 0 || p->n_bias > kMaxIds)
    return FLCE_ERR_INVALID_ARG;
  if (p->rows > INT32_MAX / plan_tiles(p->rows, p->vocab)) return FLCE_ERR_INVALID_ARG;
  if (p->logits_stride < 0 || p->tokens_stride < 0 || p->bias_ids_stride < 0 || p->bias_stride < 0 ||
      p->mask_stride < 0 || (p->rows > 1 && p->out_stride < p->vocab) || p->out_stride < 0)
    return FLCE_ERR_INVALID_ARG;
  if (!known_dtype(p->logits_dtype) || !known_dtype(p->out_dtype)) return FLCE_ERR_UNSUPPORTED_DTYPE;
  if (p->out_dtype != p->logits_dtype && p->out_dtype != FLCE_F32) return FLCE_ERR_DTYPE_MISMATCH;
  return FLCE_OK;
}

// The kernel's form: vectors of `vec` entries, `nv` of them per thread.
struct Form {
  int vec, nv;
  int32_t tiles;
};
// Vectors of 16 bytes where every row of logits and of out starts equally far
// past a 16-byte boundary, in elements; else single elements.
Form plan_form(const flce_logits_problem* p, const void* logits, const void* out) {
  const int wide = int(16 / elem_size(p->logits_dtype));
  const uint64_t a = reinterpret_cast<uintptr_t>(logits) / elem_size(p->logits_dtype);
  const uint64_t b = reinterpret_cast<uintptr_t>(out) / elem_size(p->out_dtype);
  const bool ok = (a - b) % wide == 0 && (p->rows == 1 || (p->logits_stride - p->out_stride) % wide == 0);
  Form f;
  f.vec = ok ? wide : 1;
  const int per = plan_per_thread(p->rows, p->vocab);
  f.nv = f.vec == 1 ? std::min(kMaxSingles, per) : std::max(1, per / f.vec);
  const bool shifted = a % f.vec != 0 || (p->rows > 1 && p->logits_stride % f.vec != 0);
  f.tiles = int32_t(cdiv(p->vocab + (shifted ? f.vec - 1 : 0), int64_t(kRowThreads) * f.vec * f.nv));
  return f;
}

template <class T, class O, int V, int NV>
cudaError_t launch(const LogitsParams& p, int64_t rows, cudaStream_t st) {
  auto kern = process_logits_kernel<T, O, V, NV>;
  constexpr size_t kBytes = sizeof(Named<kRowThreads * V * NV>);
  const size_t smem = p.tokens || p.n_bias ? kBytes : 0;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kBytes));
  if (e != cudaSuccess) return e;
  kern<<<unsigned(rows * p.tiles), kRowThreads, smem, st>>>(p);
  return cudaGetLastError();
}
template <class T, class O>
cudaError_t launch_types(const LogitsParams& p, int64_t rows, const Form& f, cudaStream_t st) {
  constexpr int kV = 16 / sizeof(T);
  if (f.vec == kV) {
    if (f.nv == 1) return launch<T, O, kV, 1>(p, rows, st);
    if (f.nv == 2) return launch<T, O, kV, 2>(p, rows, st);
    if (f.nv == 4) return launch<T, O, kV, 4>(p, rows, st);
    if constexpr (kV == 4) {
      if (f.nv == 8) return launch<T, O, kV, 8>(p, rows, st);
    }
  } else {
    if (f.nv == 4) return launch<T, O, 1, 4>(p, rows, st);
    if (f.nv == 8) return launch<T, O, 1, 8>(p, rows, st);
    if (f.nv == 16) return launch<T, O, 1, 16>(p, rows, st);
  }
  return cudaErrorInvalidValue;
}

template <class O>
cudaError_t launch_merge(const LogitsParams& q, int64_t rows, const Form& f, int64_t* token, float* lse,
                         cudaStream_t st) {
  return launch_dependent(merge_logits_kernel<O>, unsigned(cdiv(rows, kRowWarps)), kRowThreads, st,
                          static_cast<const Partial*>(q.part), rows, q.tiles, static_cast<const O*>(q.out), q.os,
                          q.vocab, f.vec, token, lse);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_process_logits_workspace_size(const flce_logits_problem* problem, size_t* bytes) {
  if (!bytes) return FLCE_ERR_INVALID_ARG;
  FLCE_TRY(validate(problem));
  *bytes = size_t(problem->rows) * size_t(plan_tiles(problem->rows, problem->vocab)) * sizeof(Partial) + 256;
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
  q.tokens_i64 = p->tokens_i64;
  q.bias_ids_i64 = p->bias_ids_i64;
  const Form form = plan_form(p, logits, out);
  q.tiles = form.tiles;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  FLCE_TRY(logged(FLCE_LAUNCH_OTHER, st, [&] {
    if (p->logits_dtype == FLCE_F32) return launch_types<float, float>(q, p->rows, form, st);
    if (p->logits_dtype == FLCE_BF16)
      return p->out_dtype == FLCE_F32 ? launch_types<__nv_bfloat16, float>(q, p->rows, form, st)
                                      : launch_types<__nv_bfloat16, __nv_bfloat16>(q, p->rows, form, st);
    return p->out_dtype == FLCE_F32 ? launch_types<__half, float>(q, p->rows, form, st)
                                    : launch_types<__half, __half>(q, p->rows, form, st);
  }));
  if (!token && !lse) return FLCE_OK;
  return logged(FLCE_LAUNCH_OTHER, st, [&] {
    if (p->out_dtype == FLCE_F32) return launch_merge<float>(q, p->rows, form, token, lse, st);
    if (p->out_dtype == FLCE_BF16) return launch_merge<__nv_bfloat16>(q, p->rows, form, token, lse, st);
    return launch_merge<__half>(q, p->rows, form, token, lse, st);
  });
}

}  // extern "C"
