// flce_sample.cu — choice of a token from each row of logits: temperature,
// top-k, top-p, min-p and one given uniform number: kernel and C entry point.
//
//   w_i = e^((z_i - max z) / T); entries are ranked by (z descending, index ascending)
//   top-k keeps the first k ranks, top-p of those the ranks before which less than
//   p of their mass lies, min-p the entries with w_i >= min_p
//   token = first kept i, in index order, with sum of kept w_j (j <= i) > u sum of kept w
//
// The bound is memory: the logits are read once.  A cluster takes a row and holds
// it in its CTAs' shared memory, so that every later pass over the row stays on
// chip.
//
// Whole numbers come out of sums here (which entries are kept, which is chosen),
// so weights are integers: w_i in units of 2^-kBits of the largest, from a
// table and a polynomial with an error below 2^-31 of w_i (2^-37 where w_i is
// at least 2^-6 of the largest: those carry the error of the sums).  Integer sums
// do not depend on their order, and equal logits have equal weights.
//
// Top-k and top-p cut the ranking at one place.  The place is found by histograms:
// a first one over the distance from the maximum, in steps of 2^(1/64) of the
// weight, then over ever smaller intervals of (value, index), until one entry is
// left.
#include <algorithm>
#include <cmath>

#include "flce_device.cuh"
#include "flce_elem.cuh"
#include "flce_host.h"

namespace flce {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreadsS = 512;
constexpr int kWarpsS = kThreadsS / 32;
constexpr int kMaxCtas = 16;           // of a cluster
constexpr int kBins = 2048;
constexpr float kBinsPerOctave = 64.f; // of the first histogram: 32 octaves below the largest weight
constexpr int64_t kMaxVocab = 1 << 20; // a CTA's limb sums (65536 entries of 16 bits) fit 32 bits
constexpr int64_t kSliceBytes = 64 << 10;   // of a row in one CTA: two CTAs on an SM
constexpr int64_t kSliceMost = 180 << 10;   // the most that a CTA holds; the rest of its slice is read again

struct SampleParams {
  const void* logits;
  const float *uniform, *temperature;
  const int64_t* top_k;
  const float *top_p, *min_p;
  int64_t* token;
  float* logprob;
  int64_t* kept;
  int64_t stride;
  int32_t vocab;
  int32_t slice;    // entries of a CTA's slice: whole 16-byte vectors
  int32_t cached;   // of which so many places of shared memory hold
  int32_t bits;     // weights are in units of 2^-bits
};

struct Pair {
  uint64_t a, b;
};

struct Shared {
  uint32_t hist[4][kBins];   // entries, and three limbs of 16 bits of their weights
  uint32_t first[kBins];     // the first histogram, of the whole row
  uint64_t table[32];        // 2^(62 - j / 32)
  Pair slots[2][kMaxCtas];   // what the CTAs tell each other, by turns
  uint64_t found[4];         // the interval that holds the cut
  uint64_t wa[kWarpsS], wb[kWarpsS];
  float wf[kWarpsS], wg[kWarpsS];
  int at[2];
};

// Place in the descending order of values, as an unsigned number (-0 is +0; no NaN).
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t u = __float_as_uint(z + 0.f);
  return (u >> 31) ? u : u ^ 0x7fffffffu;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key >> 31) ? key : key ^ 0x7fffffffu);
}
__device__ __forceinline__ uint64_t place_of(float z, int i) { return uint64_t(key_of(z)) << 32 | uint32_t(i); }

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint64_t warp_sum64(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}
template <class N>
__device__ __forceinline__ N warp_scan(N x) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const N v = __shfl_up_sync(kFull, x, o);
    if (int(threadIdx.x & 31) >= o) x += v;
  }
  return x;
}

// Weights of a row.
struct Weigh {
  float top;         // the largest logit
  float c_hi, c_lo;  // log2(e) / temperature
  int bits;
  const uint64_t* table;

  // 2^bits 2^-y for y = (top - z) c >= 0, rounded.  y = p + e in two floats; p is
  // split into n / 32 + r exactly, 2^(-n / 32) is a table's value and a shift, and
  // 2^-(r + e) - 1 a Taylor polynomial of at most 1 / 64 in absolute value: its fourth
  // power leaves 2^-39.
  __device__ __forceinline__ uint64_t operator()(float z) const {
    if (z == top) return 1ull << bits;
    const float d = top - z, b = d - top, d_lo = (top - (d - b)) - (z + b);
    float p = d * c_hi;
    float e = fmaf(d_lo, c_hi, fmaf(d, c_lo, fmaf(d, c_hi, -p)));
    if (d == INFINITY) {  // -inf, or a difference beyond fp32
      const double y = z == -INFINITY || top == INFINITY ? INFINITY : (double(top) - double(z)) * (double(c_hi) + double(c_lo));
      p = float(y);
      e = float(y - double(p));
    }
    if (!(p < float(bits + 1))) return 0ull;  // less than half a unit
    const float t = fmaf(p, 32.f, 12582912.f);  // 1.5 * 2^23: the sum's last bits are the integer
    const int n = __float_as_int(t) - 0x4B400000;
    const float r = fmaf(t - 12582912.f, -0.03125f, p);
    constexpr float kL1 = 0.693147181f, kL2 = 0.240226507f, kL3 = 0.0555041087f, kL4 = 0.00961812911f;  // ln(2)^k / k!
    const uint64_t base = table[n & 31];
    const int shift = n >> 5;
    const float x = -(r + e);
    const float rest = x * x * fmaf(x, fmaf(x, kL4, kL3), kL2);
    uint64_t w;
    if (p < 6.f) {
      // the linear term in two floats, and everything in units of 2^-44
      constexpr float kL1lo = -1.90465421e-9f;  // ln(2) - kL1
      const float x_lo = (-r - x) - e;
      const float m = x * kL1;
      const float m_lo = fmaf(x_lo, kL1, fmaf(x, kL1lo, fmaf(x, kL1, -m)));
      const int64_t q = __float2ll_rn(m * 0x1p44f) + __float2ll_rn((m_lo + rest) * 0x1p44f);
      w = base + uint64_t(__mul64hi(int64_t(base), q << 20));  // q << 20: units of 2^-64
    } else {
      const uint32_t b32 = uint32_t(base >> 31);
      w = uint64_t(uint32_t(int(b32) + __float2int_rn(float(b32) * fmaf(x, kL1, rest)))) << 31;
    }
    return ((w >> (61 - bits + shift)) + 1) >> 1;
  }
};

// A CTA's part of the row.  Places j stand for row entries first + j; those outside
// [lo, hi) are not of the slice and hold -inf.  Warp w has places [w seg, (w + 1) seg).
template <class T>
struct Slice {
  static constexpr int kV = 16 / sizeof(T);
  static constexpr int kStep = 32 * kV;  // places that a warp takes at once
  T* mem;
  const T* row;  // place 0, 16-byte aligned
  int first, lo, hi, cached, seg;

  __device__ __forceinline__ void load(int j, float (&z)[kV]) const {
    if (j + kV <= hi && j >= lo) {
      const Vec<T, kV> v = load_vec<T, kV>(row + j);
#pragma unroll
      for (int e = 0; e < kV; ++e) z[e] = to_f32(v.v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < kV; ++e) z[e] = j + e >= lo && j + e < hi ? to_f32(row[j + e]) : -INFINITY;
    }
  }
  // f(z, j) for the warp's places, kStep at a time; j is the lane's first
  template <class F>
  __device__ __forceinline__ void each(F&& f) const {
    const int begin = int(threadIdx.x >> 5) * seg, end = min(hi, begin + seg), mine = int(threadIdx.x & 31) * kV;
    for (int j0 = begin; j0 < end; j0 += kStep) {
      float z[kV];
      if (j0 < cached) {
        const Vec<T, kV> v = load_vec<T, kV>(mem + j0 + mine);
#pragma unroll
        for (int e = 0; e < kV; ++e) z[e] = to_f32(v.v[e]);
      } else {
        load(j0 + mine, z);
      }
      f(z, j0 + mine);
    }
  }
};

// The row's cluster: its CTAs tell each other two numbers each.
struct Cluster {
  Shared& s;
  int rank, ctas, turn = 0;

  // afterwards slots[i] holds CTA i's pair
  __device__ __forceinline__ const Pair* tell(uint64_t a, uint64_t b) {
    Pair* mine = &s.slots[turn][rank];
    if (int(threadIdx.x) < ctas) {
      const uint32_t to = map_to_cta(smem_u32(mine), threadIdx.x);
      st_cluster(to, a);
      st_cluster(to + 8, b);
    }
    const Pair* all = s.slots[turn];
    turn ^= 1;
    cluster_sync();
    return all;
  }
};

// Sums of two numbers over the block; every thread gets them.
__device__ __forceinline__ void block_sum2(Shared& s, uint64_t& a, uint64_t& b) {
  a = warp_sum64(a);
  b = warp_sum64(b);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    s.wa[threadIdx.x >> 5] = a;
    s.wb[threadIdx.x >> 5] = b;
  }
  __syncthreads();
  a = b = 0;
#pragma unroll
  for (int w = 0; w < kWarpsS; ++w) {
    a += s.wa[w];
    b += s.wb[w];
  }
}

// Inclusive sums over the block of each thread's two numbers.
template <class N>
__device__ __forceinline__ void block_scan2(N* bufa, N* bufb, N& a, N& b) {
  a = warp_scan(a);
  b = warp_scan(b);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  if (lane == 31) {
    bufa[warp] = a;
    bufb[warp] = b;
  }
  __syncthreads();
  for (int w = 0; w < warp; ++w) {
    a += bufa[w];
    b += bufb[w];
  }
}

__device__ __forceinline__ void add_entry(Shared& s, int bin, uint64_t w) {
  atomicAdd(&s.hist[0][bin], 1u);
  atomicAdd(&s.hist[1][bin], uint32_t(w) & 0xffffu);
  atomicAdd(&s.hist[2][bin], uint32_t(w >> 16) & 0xffffu);
  atomicAdd(&s.hist[3][bin], uint32_t(w >> 32));
}
__device__ __forceinline__ void clear_hist(Shared& s) {
  __syncthreads();
  for (int i = threadIdx.x; i < 4 * kBins; i += kThreadsS) s.hist[0][i] = 0u;
  __syncthreads();
}

// An interval [lo, hi) of places in the ranking, with `n` entries, and what stands before it.
struct Interval {
  uint64_t lo, hi, mass;
  uint32_t n, count;
};

// The interval's histogram over all CTAs, and in it the bin where the entries
// (by_mass: the weights) from the ranking's start on reach `target`.
__device__ __forceinline__ void descend(Shared& s, Cluster& cl, Interval& v, int shift, uint64_t target, bool by_mass) {
  cluster_sync();  // the histograms are there
  constexpr int kMost = kBins / kThreadsS;
  const int per = kBins / cl.ctas, each = max(1, per / kThreadsS);  // bins of a CTA, of a thread
  const int bin0 = cl.rank * per + int(threadIdx.x) * each;
  const bool on = int(threadIdx.x) * each < per;
  uint64_t n[kMost], m[kMost], a = 0, b = 0;
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    n[k] = m[k] = 0;
    if (on && k < each) {
      for (int c = 0; c < cl.ctas; ++c) {
        const uint32_t at = map_to_cta(smem_u32(&s.hist[0][bin0 + k]), uint32_t(c));
        n[k] += ld_cluster(at);
        if (by_mass)
          m[k] += ld_cluster(at + kBins * 4) + (uint64_t(ld_cluster(at + kBins * 8)) << 16) +
                  (uint64_t(ld_cluster(at + kBins * 12)) << 32);
      }
    }
    a += n[k];
    b += m[k];
  }
  const uint64_t own_a = a, own_b = b;
  block_scan2(s.wa, s.wb, a, b);
  // the last thread knows the CTA's sums
  __syncthreads();
  if (threadIdx.x == kThreadsS - 1) {
    s.wa[0] = a;
    s.wb[0] = b;
    // if the target lies behind the interval (it does not): everything in it is kept
    s.found[0] = v.hi;
    s.found[1] = v.mass;
    s.found[2] = 0;
  }
  __syncthreads();
  const Pair* all = cl.tell(s.wa[0], s.wb[0]);
  uint64_t ca = v.count, cb = v.mass;
  for (int c = 0; c < cl.rank; ++c) {
    ca += all[c].a;
    cb += all[c].b;
  }
  ca += a - own_a;
  cb += b - own_b;
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    if (on && k < each) {
      const uint64_t before = by_mass ? cb : ca, after = by_mass ? cb + m[k] : ca + n[k];
      if (before < target && after >= target) {  // one thread of the cluster
        const uint64_t lo = v.lo + (uint64_t(bin0 + k) << shift);
        for (int c = 0; c < cl.ctas; ++c) {
          const uint32_t to = map_to_cta(smem_u32(s.found), uint32_t(c));
          st_cluster(to, lo);
          st_cluster(to + 8, cb);
          st_cluster(to + 16, ca << 32 | n[k]);
        }
      }
    }
    ca += n[k];
    cb += m[k];
  }
  cluster_sync();
  const uint64_t hi = v.hi;
  v.lo = s.found[0];
  v.hi = min(hi, v.lo + (uint64_t(1) << shift));
  v.mass = s.found[1];
  v.count = uint32_t(s.found[2] >> 32);
  v.n = uint32_t(s.found[2]);
  __syncthreads();
}

__device__ __forceinline__ int shift_of(const Interval& v) {
  return max(0, 64 - __clzll((v.hi - v.lo - 1) | 1) - 11);
}

// Down to one entry: the ranking is cut behind it.
template <class T>
__device__ __forceinline__ void narrow(Shared& s, Cluster& cl, const Slice<T>& sl, const Weigh& weigh, Interval& v,
                                       uint64_t target, bool by_mass) {
  while (v.n > 1) {
    clear_hist(s);
    const int shift = shift_of(v);
    const uint32_t k_lo = uint32_t(v.lo >> 32), k_hi = uint32_t((v.hi - 1) >> 32);
    sl.each([&](const float (&z)[Slice<T>::kV], int j) {
#pragma unroll
      for (int e = 0; e < Slice<T>::kV; ++e) {
        const uint32_t key = key_of(z[e]);
        if (key < k_lo || key > k_hi || z[e] == -INFINITY) continue;
        const uint64_t at = uint64_t(key) << 32 | uint32_t(sl.first + j + e);
        if (at < v.lo || at >= v.hi) continue;
        const int bin = int((at - v.lo) >> shift);
        if (by_mass) {
          add_entry(s, bin, weigh(z[e]));
        } else {
          atomicAdd(&s.hist[0][bin], 1u);
        }
      }
    });
    descend(s, cl, v, shift, target, by_mass);
  }
}

// Bin of the first histogram, monotone in z.  (Halves: top - z may lie beyond fp32.)
__device__ __forceinline__ int first_bin(float z, float top, float per_unit) {
  return min(kBins - 1, int(fmaf(z, -0.5f, 0.5f * top) * (2.f * per_unit)));
}
// First key, between the maximum's and -inf's, whose value is in bin b or behind it; whole warps.
__device__ __forceinline__ uint32_t bin_edge(int b, float top, float per_unit) {
  uint32_t lo = key_of(top), hi = key_of(-INFINITY);
  while (hi > lo) {
    const uint32_t step = (hi - lo + 31) / 32;
    const uint64_t i = uint64_t(lo) + uint64_t(threadIdx.x & 31) * step;
    const bool before = i < hi && first_bin(value_of(uint32_t(i)), top, per_unit) < b;
    const int c = __popc(__ballot_sync(kFull, before));
    if (step == 1 || c == 0) return lo + c;
    const uint32_t from = lo;
    lo = from + uint32_t(c - 1) * step + 1;
    const uint64_t to = uint64_t(from) + uint64_t(c) * step;
    hi = to < hi ? uint32_t(to) : hi;
  }
  return lo;
}

template <class T>
__global__ void __launch_bounds__(kThreadsS, 2) sample_kernel(SampleParams p) {
  extern __shared__ __align__(16) uint8_t dynamic[];
  Shared& s = *reinterpret_cast<Shared*>(dynamic);
  constexpr int kV = Slice<T>::kV;
  uint32_t ctas;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  Cluster cl{s, int(cluster_ctarank()), int(ctas)};
  const int64_t row = blockIdx.x / ctas;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  // ---- the slice, and the largest logit
  Slice<T> sl;
  {
    const T* base = static_cast<const T*>(p.logits) + row * p.stride;
    const int phase = int(reinterpret_cast<uintptr_t>(base) / sizeof(T) % kV);
    const int begin = min(p.vocab, cl.rank * p.slice), end = min(p.vocab, begin + p.slice);
    sl.mem = reinterpret_cast<T*>(dynamic + (sizeof(Shared) + 15) / 16 * 16);
    sl.first = cl.rank * p.slice - phase;
    sl.row = base + sl.first;
    sl.lo = phase;
    sl.hi = phase + end - begin;
    sl.cached = p.cached;
    sl.seg = ((sl.hi + kWarpsS - 1) / kWarpsS + Slice<T>::kStep - 1) / Slice<T>::kStep * Slice<T>::kStep;
  }
  // every CTA has to run before another one writes to its memory: the wait is below
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (threadIdx.x < 32) s.table[threadIdx.x] = uint64_t(rint(exp2(62.0 - double(threadIdx.x) / 32.0)));
  float top = -INFINITY;
  bool nan = false;
  {
    const int begin = warp * sl.seg, end = min(sl.hi, begin + sl.seg);
#pragma unroll 4
    for (int j0 = begin; j0 < end; j0 += Slice<T>::kStep) {
      const int j = j0 + lane * kV;
      float z[kV];
      sl.load(j, z);
      if (j0 < sl.cached) {
        Vec<T, kV> v;
#pragma unroll
        for (int e = 0; e < kV; ++e) v.v[e] = from_f32<T>(z[e]);
        store_vec<T, kV>(sl.mem + j, v);
      }
#pragma unroll
      for (int e = 0; e < kV; ++e) {
        nan |= z[e] != z[e];
        top = fmaxf(top, z[e]);
      }
    }
    const int key = top >= 0.f ? __float_as_int(top + 0.f) : __float_as_int(top) ^ 0x7fffffff;
    const int most = __reduce_max_sync(kFull, __any_sync(kFull, nan) ? 0x7fffffff : key);
    if (lane == 0) s.wa[warp] = uint64_t(uint32_t(most) ^ 0x80000000u);
    __syncthreads();
    uint64_t best = 0;
#pragma unroll
    for (int w = 0; w < kWarpsS; ++w) best = max(best, s.wa[w]);
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const Pair* all = cl.tell(best, 0);
    for (int c = 0; c < cl.ctas; ++c) best = max(best, all[c].a);
    const int got = int(uint32_t(best) ^ 0x80000000u);
    nan = got == 0x7fffffff;
    top = __int_as_float(got >= 0 ? got : got ^ 0x7fffffff);
  }
  const float temperature = p.temperature ? p.temperature[row] : 1.f;
  const bool out = cl.rank == 0 && threadIdx.x == 0;
  if (!nan && top == -INFINITY) {  // nothing is allowed
    if (out) {
      p.token[row] = -1;
      if (p.logprob) p.logprob[row] = -INFINITY;
      if (p.kept) p.kept[row] = 0;
    }
    cluster_sync();
    return;
  }
  if (nan || !(temperature > 0.f)) {  // greedy: the first of the largest, a NaN before all
    int best = INT32_MAX;
    sl.each([&](const float (&z)[kV], int j) {
#pragma unroll
      for (int e = kV - 1; e >= 0; --e)
        if (nan ? z[e] != z[e] : z[e] == top) best = min(best, sl.first + j + e);
    });
    best = __reduce_min_sync(kFull, best);
    if (lane == 0) s.wb[warp] = uint64_t(best);
    __syncthreads();
    uint64_t low = INT32_MAX;
#pragma unroll
    for (int w = 0; w < kWarpsS; ++w) low = min(low, s.wb[w]);
    const Pair* all = cl.tell(low, 0);
    for (int c = 0; c < cl.ctas; ++c) low = min(low, all[c].a);
    if (out) {
      p.token[row] = int64_t(low);
      if (p.logprob) p.logprob[row] = nan ? NAN : 0.f;
      if (p.kept) p.kept[row] = 1;
    }
    cluster_sync();
    return;
  }

  // ---- where the ranking is cut
  const double c = 1.4426950408889634 / double(temperature);
  Weigh weigh;
  weigh.top = top;
  weigh.c_hi = float(c);
  weigh.c_lo = float(c - double(weigh.c_hi));
  weigh.bits = p.bits;
  weigh.table = s.table;
  const int64_t k_row = p.top_k ? p.top_k[row] : 0;
  const uint32_t k = k_row <= 0 || k_row >= p.vocab ? 0u : uint32_t(k_row);
  const float top_p = p.top_p ? p.top_p[row] : 1.f;
  const bool nucleus = top_p < 1.f;
  uint64_t cut = ~0ull;  // entries at places behind it are dropped
  if (k || nucleus) {
    const float per_unit = weigh.c_hi * kBinsPerOctave;
    clear_hist(s);
    sl.each([&](const float (&z)[kV], int) {
#pragma unroll
      for (int e = 0; e < kV; ++e)
        if (z[e] != -INFINITY) atomicAdd(&s.hist[0][first_bin(z[e], top, per_unit)], 1u);
    });
    cluster_sync();
    for (int b = threadIdx.x; b < kBins / cl.ctas; b += kThreadsS) {
      const int bin = cl.rank * (kBins / cl.ctas) + b;
      uint32_t n = 0;
      for (int i = 0; i < cl.ctas; ++i) n += ld_cluster(map_to_cta(smem_u32(&s.hist[0][bin]), uint32_t(i)));
      for (int i = 0; i < cl.ctas; ++i) st_cluster(map_to_cta(smem_u32(&s.first[bin]), uint32_t(i)), n);
    }
    if (threadIdx.x < 2) s.at[threadIdx.x] = kBins - 1;
    cluster_sync();
    // each thread has four bins: entries, and where k is reached
    constexpr int kPer = kBins / kThreadsS;
    uint32_t n[kPer], sum = 0, dummy = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += n[i] = s.first[threadIdx.x * kPer + i];
    uint32_t upto = sum;
    block_scan2(reinterpret_cast<uint32_t*>(s.wa), reinterpret_cast<uint32_t*>(s.wb), upto, dummy);
    uint32_t before = upto - sum;
    uint32_t total;
    __syncthreads();
    if (threadIdx.x == kThreadsS - 1) s.found[3] = upto;
    __syncthreads();
    total = uint32_t(s.found[3]);
    const uint32_t most = k && k < total ? k : total;
    Interval v{};
    if (k && k < total) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (before < k && before + n[i] >= k) {
          s.at[0] = int(threadIdx.x) * kPer + i;
          s.found[2] = uint64_t(before) << 32 | n[i];
        }
        before += n[i];
      }
      before = upto - sum;
      __syncthreads();
      v.lo = uint64_t(bin_edge(s.at[0], top, per_unit)) << 32;
      v.hi = uint64_t(bin_edge(s.at[0] + 1, top, per_unit)) << 32;
      v.count = uint32_t(s.found[2] >> 32);
      v.n = uint32_t(s.found[2]);
      __syncthreads();
      narrow(s, cl, sl, weigh, v, k, false);
      cut = v.hi - 1;
    }
    if (nucleus) {
      // Bounds on the mass up to each bin, from the entries in it: a bin's weights lie
      // within 2^(1/64) of each other.  They name the bins in which the mass can reach
      // p of the whole; the slack covers the bounds' own rounding.
      constexpr float kSlack = 1e-4f;
      float lo_sum = 0.f, hi_sum = 0.f;
      float lo_n[kPer], hi_n[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t in = min(before + n[i], most) - min(before, most);
        before += n[i];
        const int b = int(threadIdx.x) * kPer + i;
        hi_n[i] = float(in) * exp2f(-float(b) / kBinsPerOctave);
        lo_n[i] = b == kBins - 1 ? 0.f : float(in) * exp2f(-float(b + 1) / kBinsPerOctave);
        lo_sum += lo_n[i];
        hi_sum += hi_n[i];
      }
      float lo_upto = lo_sum, hi_upto = hi_sum;
      block_scan2(s.wf, s.wg, lo_upto, hi_upto);
      __syncthreads();
      if (threadIdx.x == kThreadsS - 1) {
        s.wf[0] = lo_upto;
        s.wg[0] = hi_upto;
      }
      __syncthreads();
      const float p_lo = top_p * s.wf[0] * (1.f - kSlack), p_hi = top_p * s.wg[0] * (1.f + kSlack);
      float lo_at = lo_upto - lo_sum, hi_at = hi_upto - hi_sum;
      __syncthreads();
      if (threadIdx.x < 2) s.at[threadIdx.x] = kBins - 1;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        hi_at += hi_n[i];
        lo_at += lo_n[i];
        if (hi_at * (1.f + kSlack) >= p_lo) atomicMin(&s.at[0], int(threadIdx.x) * kPer + i);
        if (lo_at * (1.f - kSlack) >= p_hi) atomicMin(&s.at[1], int(threadIdx.x) * kPer + i);
      }
      __syncthreads();
      const int b_lo = s.at[0], b_hi = max(s.at[0], s.at[1]);
      v.lo = uint64_t(bin_edge(b_lo, top, per_unit)) << 32;
      v.hi = uint64_t(bin_edge(b_hi + 1, top, per_unit)) << 32;
      if (b_lo == 0) v.lo = 0;
      if (b_hi == kBins - 1) v.hi = uint64_t(key_of(-INFINITY)) << 32;
      // the mass of the whole, of what stands before these bins, and their histogram
      clear_hist(s);
      const int shift = shift_of(v);
      uint64_t whole = 0, ahead = 0;
      sl.each([&](const float (&z)[kV], int j) {
#pragma unroll
        for (int e = 0; e < kV; ++e) {
          const uint64_t at = place_of(z[e], sl.first + j + e);
          if (at > cut || z[e] == -INFINITY) continue;
          const uint64_t w = weigh(z[e]);
          whole += w;
          if (at < v.lo) {
            ahead += w;
          } else if (at < v.hi) {
            add_entry(s, int((at - v.lo) >> shift), w);
          }
        }
      });
      block_sum2(s, whole, ahead);
      const Pair* all = cl.tell(whole, ahead);
      whole = ahead = 0;
      for (int i = 0; i < cl.ctas; ++i) {
        whole += all[i].a;
        ahead += all[i].b;
      }
      // entries are kept while the mass before them is less than p of the whole
      const double goal = ceil(double(top_p) * double(whole));
      const uint64_t target = goal >= 1.0 ? uint64_t(goal) : 1ull;
      v.mass = ahead;
      v.count = 0;
      descend(s, cl, v, shift, target, true);
      // (entries behind top-k's cut are not in the histograms)
      v.hi = min(v.hi, cut == ~0ull ? cut : cut + 1);
      narrow(s, cl, sl, weigh, v, target, true);
      cut = min(cut, v.hi - 1);
    }
  }
  const float min_p = p.min_p ? p.min_p[row] : 0.f;
  const uint64_t least = min_p > 0.f ? uint64_t(ceil(fmin(double(min_p), 1.0) * double(1ull << p.bits))) : 0ull;

  // ---- the kept entries' mass, in index order, and the entry that the number falls on
  auto weight = [&](float z, int i, bool& kept) -> uint64_t {
    kept = z != -INFINITY && place_of(z, i) <= cut;
    if (!kept) return 0ull;
    const uint64_t w = weigh(z);
    kept = w >= least;
    return kept ? w : 0ull;
  };
  uint64_t mass = 0, count = 0;
  sl.each([&](const float (&z)[kV], int j) {
#pragma unroll
    for (int e = 0; e < kV; ++e) {
      bool kept;
      mass += weight(z[e], sl.first + j + e, kept);
      count += kept;
    }
  });
  mass = warp_sum64(mass);
  count = warp_sum64(count);
  __syncthreads();
  if (lane == 0) {
    s.wa[warp] = mass;
    s.wb[warp] = count;
  }
  __syncthreads();
  uint64_t own = 0, own_n = 0, ahead = 0;
  for (int w = 0; w < kWarpsS; ++w) {
    if (w < warp) ahead += s.wa[w];
    own += s.wa[w];
    own_n += s.wb[w];
  }
  const Pair* all = cl.tell(own, own_n);
  uint64_t whole = 0, kept_n = 0;
  for (int i = 0; i < cl.ctas; ++i) {
    if (i < cl.rank) ahead += all[i].a;
    whole += all[i].a;
    kept_n += all[i].b;
  }
  // the first entry up to which there is more than u of the mass: u below 0 counts as 0, from 1 on as just below 1
  const double at = fmax(floor(double(p.uniform[row]) * double(whole)), 0.0);  // a NaN too counts as 0
  const uint64_t goal = at < double(whole) ? min(uint64_t(at), whole - 1) : whole - 1;
  if (goal >= ahead && goal < ahead + mass) {  // one warp of the cluster
    bool done = false;
    uint64_t sum = ahead;
    sl.each([&](const float (&z)[kV], int j) {
      if (done) return;
      uint64_t w[kV], mine = 0;
#pragma unroll
      for (int e = 0; e < kV; ++e) {
        bool kept;
        mine += w[e] = weight(z[e], sl.first + j + e, kept);
      }
      const uint64_t upto = warp_scan(mine);
      const uint32_t hit = __ballot_sync(kFull, sum + upto > goal);
      if (hit) {
        done = true;
        if (lane == __ffs(hit) - 1) {
          uint64_t t = sum + upto - mine;
          bool found = false;
#pragma unroll
          for (int e = 0; e < kV; ++e) {
            t += w[e];
            if (!found && t > goal) {
              found = true;
              p.token[row] = sl.first + j + e;
              if (p.logprob)
                p.logprob[row] = float(z[e] == top ? -log(ldexp(double(whole), -p.bits))
                                                   : (double(z[e]) - double(top)) / double(temperature) -
                                                         log(ldexp(double(whole), -p.bits)));
              if (p.kept) p.kept[row] = int64_t(kept_n);
            }
          }
        }
      }
      sum += __shfl_sync(kFull, upto, 31);
    });
  }
  cluster_sync();  // nobody reads another CTA's memory any more
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
constexpr int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

int validate(const flce_sample_problem* p) {
  if (!p) return FLCE_ERR_INVALID_ARG;
  if (p->rows < 0 || p->rows > INT32_MAX / kMaxCtas || p->vocab < 1 || p->vocab > kMaxVocab || p->logits_stride < 0)
    return FLCE_ERR_INVALID_ARG;
  if (!known_dtype(p->logits_dtype)) return FLCE_ERR_UNSUPPORTED_DTYPE;
  return FLCE_OK;
}

template <class T>
cudaError_t launch_sample(SampleParams& q, int64_t rows, int num_sms, cudaStream_t st) {
  constexpr int kV = Slice<T>::kV, kStep = Slice<T>::kStep;
  // CTAs of a row: as few as hold it in kSliceBytes each; more while SMs are free and a slice is worth a pass
  int ctas = 1;
  while (ctas < kMaxCtas && (cdiv(q.vocab, ctas) * int64_t(sizeof(T)) > kSliceBytes ||
                             (rows * ctas * 2 <= num_sms && q.vocab / ctas > 2 * kThreadsS * kV)))
    ctas *= 2;
  q.slice = int32_t(cdiv(cdiv(q.vocab, ctas), kV) * kV);
  const int64_t places = cdiv(q.slice + kV - 1, int64_t(kStep) * kWarpsS) * kStep * kWarpsS;
  q.cached = int32_t(std::min<int64_t>(places, kSliceMost / int64_t(sizeof(T)) / kStep * kStep));
  int bits = 62;  // the sum of all weights fits 63 bits
  for (int64_t v = 1; v < q.vocab; v *= 2) --bits;
  q.bits = std::min(46, bits);
  const size_t fixed = (sizeof(Shared) + 15) / 16 * 16;
  auto kern = sample_kernel<T>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(fixed + kSliceMost));
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(rows * ctas));
  cfg.blockDim = dim3(kThreadsS);
  cfg.dynamicSmemBytes = fixed + size_t(q.cached) * sizeof(T);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, q);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_sample(const flce_sample_problem* problem, const void* logits, const float* uniform,
                const float* temperature, const int64_t* top_k, const float* top_p, const float* min_p,
                int64_t* token, float* logprob, int64_t* kept, flce_stream_t stream) {
  const flce_sample_problem* p = problem;
  FLCE_TRY(validate(p));
  if (p->rows == 0) return FLCE_OK;
  if (!logits || !uniform || !token) return FLCE_ERR_INVALID_ARG;
  if (!aligned_to(logits, elem_size(p->logits_dtype)) || !aligned_to(uniform, 4) || !aligned_to(temperature, 4) ||
      !aligned_to(top_k, 8) || !aligned_to(top_p, 4) || !aligned_to(min_p, 4) || !aligned_to(token, 8) ||
      !aligned_to(logprob, 4) || !aligned_to(kept, 8))
    return FLCE_ERR_MISALIGNED;
  DeviceInfo dev;
  FLCE_TRY(get_device(&dev));
  FLCE_TRY(check_local(dev, logits, uniform, temperature, top_k, top_p, min_p, token, logprob, kept));
  SampleParams q{};
  q.logits = logits;
  q.uniform = uniform;
  q.temperature = temperature;
  q.top_k = top_k;
  q.top_p = top_p;
  q.min_p = min_p;
  q.token = token;
  q.logprob = logprob;
  q.kept = kept;
  q.stride = p->logits_stride;
  q.vocab = int32_t(p->vocab);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return logged(FLCE_LAUNCH_OTHER, st, [&] {
    if (p->logits_dtype == FLCE_F32) return launch_sample<float>(q, p->rows, dev.num_sms, st);
    if (p->logits_dtype == FLCE_BF16) return launch_sample<__nv_bfloat16>(q, p->rows, dev.num_sms, st);
    return launch_sample<__half>(q, p->rows, dev.num_sms, st);
  });
}

}  // extern "C"
