// flce_sample.cu — choice of a token from each row of logits: temperature,
// top-k, top-p, min-p and one given uniform number: kernel and C entry point.
//
//   w_i = e^((z_i - max z) / T); entries are ranked by (z descending, index ascending)
//   top-k keeps the first k ranks, top-p of those the ranks before which less than
//   p of their mass lies, min-p the entries with w_i >= min_p
//   token = first kept i, in index order, with sum of kept w_j (j <= i) > u sum of kept w
//
// The bound is memory: the logits are read once.  A cluster takes a row and holds as
// much of it as fits in its CTAs' shared memory, so that the later passes over
// the row stay on chip, or nearly.
//
// Whole numbers come out of sums here (which entries are kept, which is chosen),
// so weights are integers: w_i in units of 2^-bits of the largest (bits is 46, or as
// many as leave the sum of all below 2^62), from a table and a polynomial with an
// error below 2^-27 of w_i and a unit (found: 2^-28.6), or 2^-35 (2^-36) where w_i is at
// least 2^-6 of the largest: those carry the error of the sums, mostly.  Integer sums do
// not depend on their order, and equal logits have equal weights.
//
// Top-k and top-p cut the ranking at one place.  A first histogram, over the distance
// from the maximum in steps of 2^(1/64) of the weight, names the bins in which
// it lies.  If few entries stand up to there, one CTA lists and
// finishes them.  Else the entries of those bins are listed, or, where
// they are many (ties), found by histograms over ever smaller intervals of (value,
// index).  The mass that top-p is of takes a pass that forms every weight, which is
// what takes longest in the largest calls: 256 x 262144 fp32 with top-p takes 324 to 337 us,
// of which the first read is 60 and the weights 150.  About 100 instructions per entry fill
// 60 % of the issue slots.  The others are idle: where a row has one CTA, 81 % of it is read
// again in every later pass, one vector per lane at a time (how much of the time that is
// was not measured).  Rows of few different values are slow: their entries add to the same bins
// (256 rows of 262144, all but one equal, 2.9 ms).
#include <algorithm>
#include <atomic>
#include <cmath>

#include "flce_device.cuh"
#include "flce_elem.cuh"
#include "flce_host.h"

namespace flce {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreadsS = 1024;
constexpr int kWarpsS = kThreadsS / 32;
constexpr int kMaxCtas = 16;           // of a cluster
constexpr int kBins = 2048;
constexpr float kBinsPerOctave = 64.f; // of the first histogram: 32 octaves below the largest weight
constexpr uint32_t kList = kThreadsS;  // entries that one block finishes, one per thread
constexpr int64_t kMaxVocab = 1 << 20; // weights are in units of 2^-42 of the largest there

__host__ __device__ constexpr int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

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
  uint32_t hist[3][kBins];   // entries, and the low and the high 32 bits of their weights' sums
  uint32_t first[kBins];     // the first histogram, of the whole row: entries up to each bin's end
  uint64_t table[32];        // 2^(62 - j / 32)
  uint2 pairs[32];           // 2^(31 - j / 32) as an integer and as a float
  uint32_t octaves[64][8];   // what 2^-i makes of an integer: its power of two << 8 | how far it is shifted; eight times
  Pair slots[2][kMaxCtas];   // what the CTAs tell each other, by turns
  uint64_t found[4];         // the interval that holds the cut
  uint64_t wa[kWarpsS], wb[kWarpsS];
  uint64_t extra[kWarpsS];   // what listed entries add to a warp's mass
  unsigned long long last;   // mass of the first histogram's last bin, in units of 2^-32 of the largest weight
  uint32_t listed;           // length of the list
  int at[2];
  // in place of a histogram, when it is not needed: a list of entries
  __device__ __forceinline__ uint64_t* list() { return reinterpret_cast<uint64_t*>(hist[0]); }
};

// 2^(62 - j / 32), rounded.
__constant__ uint64_t kTable[32] = {
    0x4000000000000000ull, 0x3ea0ecb6dc8a80cfull, 0x3d495f454921b30bull, 0x3bf92e66f736bd73ull,
    0x3ab031b9f7490e4cull, 0x396e41b9df20d22aull, 0x383337bb0aa53844ull, 0x36feede5f6bc8dd5ull,
    0x35d13f32b5a75abdull, 0x34aa07647c4ab917ull, 0x3389230547e12039ull, 0x326e6f619b8bc9e9ull,
    0x3159ca845541b6b7ull, 0x304b1332999c2516ull, 0x2f4228e7d6030db0ull, 0x2e3eebd1d8bee7baull,
    0x2d413cccfe779921ull, 0x2c48fd6074ab0964ull, 0x2b560fba90a852b2ull, 0x2a6856ad3a9f03beull,
    0x297fb5aa6c544e3bull, 0x289c10c0c3125a06ull, 0x27bd4c982468446bull, 0x26e34e6e7553954eull,
    0x260dfc14636e2a5cull, 0x253d3bea3fbdc258ull, 0x2470f4dceac470ceull, 0x23a90e62d17354f0ull,
    0x22e57078faa2f5baull, 0x222603a024b6a14aull, 0x216ab0d9f3121ec5ull, 0x20b361a62b0ae876ull};

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

__device__ __forceinline__ uint64_t ld_cluster64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
// A place at the end of a list in CTA 0's memory, whose length stands at `addr`.
__device__ __forceinline__ uint32_t append_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], 1;" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Sum over a warp of numbers whose sum is below 2^63 (in limbs of 21 bits: the hardware adds 32 bits at once).
__device__ __forceinline__ uint64_t warp_total(uint64_t x) {
  const uint32_t a = __reduce_add_sync(kFull, uint32_t(x) & 0x1fffffu);
  const uint32_t b = __reduce_add_sync(kFull, uint32_t(x >> 21) & 0x1fffffu);
  const uint32_t c = __reduce_add_sync(kFull, uint32_t(x >> 42));
  return a + (uint64_t(b) << 21) + (uint64_t(c) << 42);
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
// Over the block: the sum of one number per warp (the same in all its lanes), and that of the warps before.
struct Sums {
  uint64_t all, before;
};
__device__ __forceinline__ Sums block_sums(Shared& s, uint64_t a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  if (lane == 0) s.wa[warp] = a;
  __syncthreads();
  const uint64_t x = s.wa[lane];
  return {warp_total(x), warp_total(lane < warp ? x : uint64_t(0))};
}
// The sums of two.
__device__ __forceinline__ void block_sums(Shared& s, uint64_t& a, uint64_t& b) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  if (lane == 0) {
    s.wa[warp] = a;
    s.wb[warp] = b;
  }
  __syncthreads();
  a = warp_total(s.wa[lane]);
  b = warp_total(s.wb[lane]);
}
// Inclusive sums over the block's threads, and the whole one.
__device__ __forceinline__ uint64_t block_scan(Shared& s, uint64_t& a) {
  a = warp_scan(a);
  const Sums r = block_sums(s, __shfl_sync(kFull, a, 31));
  a += r.before;
  return r.all;
}
__device__ __forceinline__ void block_scan(Shared& s, uint64_t& a, uint64_t& b, uint64_t& all_a, uint64_t& all_b) {
  all_a = block_scan(s, a);
  all_b = block_scan(s, b);
}

// A weight as factor times power of two.
struct Term {
  uint32_t w, power;
  __device__ __forceinline__ uint64_t value() const { return uint64_t(w) * power; }
  __device__ __forceinline__ void add_to(uint64_t& sum) const {
    asm("mad.wide.u32 %0, %1, %2, %0;" : "+l"(sum) : "r"(w), "r"(power));
  }
};

// Weights of a row: 2^bits 2^-y with y = (top - z) log2(e) / T.  No fp64 in here or in
// what every thread does: an SM has two fp64 lanes.  Two entries go side by side in
// packed fp32 pairs; an entry takes about 30 instructions.
struct Weigh {
  float top;         // the largest logit
  float c_hi, c_lo;  // 2 log2(e) / temperature
  float end;         // -(bits + 1): weights behind it are less than half a unit
  int bits;
  const uint64_t* table;
  const uint2* pairs;
  const uint8_t* octaves;  // the lane's copy
  static constexpr float kNear = -6.f;
  static constexpr float kL1 = 0x1.62e43p-1f, kL1lo = -0x1.05c61p-29f;                    // ln(2)
  static constexpr float kL2 = 0.240226507f, kL3 = 0.0555041087f, kL4 = 0.00961812911f;  // ln(2)^k / k!
  static constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: a sum's last bits are the nearest integer

  __device__ __forceinline__ void set(float temperature) {
    constexpr float kHi = 0x1.715476p+1f, kLo = 0x1.4ae0cp-25f;  // 2 log2(e)
    c_hi = __fdiv_rn(kHi, temperature);
    c_lo = c_hi == 0.f ? 0.f : __fdiv_rn(fmaf(-c_hi, temperature, kHi) + kLo, temperature);
    end = -float(bits + 1);
  }
  // -y = np - e in two floats each, for a pair.  (Half of top - z, which may lie beyond fp32, and what its
  // rounding left.)
  __device__ __forceinline__ void distance(uint64_t z, uint64_t& np, uint64_t& e) const {
    const uint64_t ht = f2_splat(0.5f * top), m1 = f2_splat(-1.f);
    const uint64_t d = f2_fma(z, f2_splat(-0.5f), ht);
    const uint64_t b = f2_fma(ht, m1, d);
    const uint64_t d_lo = f2_fma(f2_fma(z, f2_splat(0.5f), b), m1, f2_fma(f2_fma(b, m1, d), m1, ht));
    np = f2_mul(d, f2_splat(-c_hi));
    e = f2_fma(d_lo, f2_splat(c_hi), f2_fma(d, f2_splat(c_lo), f2_fma(d, f2_splat(c_hi), np)));
  }
  // Weights of two entries, 0 where np is not above `end`.  -np = n / 32 + r exactly; 2^-y = 2^(-n / 32) 2^x
  // with x = -(r + e), at most 1 / 64 in size: a table's value, a shift, and a Taylor polynomial
  // whose fourth power leaves 2^-39.  The last bit that stays is set, which makes up for those cut
  // off.  In units of the table's last bit, 2^-30 of w at most: the table is cut by 1; x, q and its
  // product are rounded by 0.7, 1 and 1.5; the last bit adds 1: below 2^-27.  (Above kNear, weights
  // over 2^-6 of the largest, `precise` takes their place.)
  __device__ __forceinline__ void pair(float z0, float z1, Term (&t)[2], float (&np)[2]) const {
    uint64_t p2, e;
    distance(f2_pack(z0, z1), p2, e);
    const uint64_t t2 = f2_fma(p2, f2_splat(-32.f), f2_splat(kMagic));
    const uint64_t nr = f2_fma(f2_add(t2, f2_splat(-kMagic)), f2_splat(0.03125f), p2);
    const uint64_t x = f2_fma(e, f2_splat(-1.f), nr);
    const uint64_t u = f2_fma(x, f2_fma(x, f2_splat(kL4), f2_splat(kL3)), f2_splat(kL2));
    const uint64_t q2 = f2_fma(x, f2_splat(kL1), f2_mul(f2_mul(x, x), u));
    float q[2], m[2];
    f2_unpack(q2, q[0], q[1]);
    f2_unpack(t2, m[0], m[1]);
    f2_unpack(p2, np[0], np[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t n = __float_as_uint(m[i]);  // the integer in its last bits
      const uint2 base = pairs[n & 31u];
      const uint32_t octave = *reinterpret_cast<const uint32_t*>(octaves + (n & 0x7e0u));
      const uint32_t w = base.x + uint32_t(__float2int_rn(__uint_as_float(base.y) * q[i]));
      uint32_t cut;
      asm("shr.b32 %0, %1, %2;" : "=r"(cut) : "r"(w), "r"(octave & 31u));
      t[i].w = cut | 1u;
      t[i].power = np[i] > end ? octave >> 8 : 0u;
    }
  }
  // 2^62 2^-(e - np) without whole octaves (which it returns): the linear term in two floats, and
  // everything in units of 2^-44.
  __device__ __forceinline__ uint64_t power(float np, float e, int& octaves) const {
    const float t = fmaf(np, -32.f, kMagic);
    const int n = __float_as_int(t) - 0x4B400000;
    const float nr = fmaf(t - kMagic, 0.03125f, np);
    const float x = nr - e, x_lo = (nr - x) - e;
    const float m = x * kL1;
    const float m_lo = fmaf(x_lo, kL1, fmaf(x, kL1lo, fmaf(x, kL1, -m)));
    const float rest = x * x * fmaf(x, fmaf(x, kL4, kL3), kL2);
    const int64_t q = __float2ll_rn(m * 0x1p44f) + __float2ll_rn((m_lo + rest) * 0x1p44f);
    const uint64_t base = table[n & 31];
    octaves = n >> 5;
    return base + uint64_t(__mul64hi(int64_t(base), q << 20));  // q << 20: units of 2^-64
  }
  __device__ __forceinline__ void distance1(float z, float& np, float& e) const {
    uint64_t a, b;
    float other;
    distance(f2_splat(z), a, b);
    f2_unpack(a, np, other);
    f2_unpack(b, e, other);
  }
  // The weight where np is above kNear (or not a number).
  __device__ __forceinline__ uint64_t precise(float z) const {
    if (z == top) return 1ull << bits;
    float np, e;
    distance1(z, np, e);
    if (np != np) return 0ull;  // inf - inf, inf * 0: -inf, or behind an infinite largest logit
    int octaves;
    const uint64_t w = power(np, e, octaves);
    return ((w >> (61 - bits + octaves)) + 1) >> 1;
  }
  __device__ __forceinline__ uint64_t operator()(float z) const {
    Term t[2];
    float np[2];
    pair(z, z, t, np);
    return !(np[0] <= kNear) ? precise(z) : t[0].value();
  }
  // log of the part that z has of `whole`: -ln(2) (y + log2(whole 2^-bits)).  The logarithm's error
  // (of whole's leading bits, in fp32) is found by 2^-log2: what is missing from 1.
  __device__ __forceinline__ float log_part(float z, uint64_t whole) const {
    float np = 0.f, e = 0.f;
    if (z != top) distance1(z, np, e);
    const int lead = 63 - __clzll(whole);
    const uint64_t m = whole << (63 - lead);            // [2^63, 2^64)
    const float l = log2f(float(m >> 40) * 0x1p-23f);   // [0, 1]
    int octaves;
    const uint64_t inverse = power(-l, 0.f, octaves);   // 2^(62 - l + octaves)
    // m inverse is 2^125 (1 + off) before the octaves
    const int64_t off = int64_t(__umul64hi(m, inverse >> octaves)) - (int64_t(1) << 61);
    const float l_lo = float(off) * (0x1p-61f * 1.44269504f);
    // the sum in two floats, times ln(2) in two floats
    const float i = float(lead - bits), a = i + l, a_lo = l - (a - i), p = -np;
    const float t = p + a, b = t - p, t_lo = (p - (t - b)) + (a - b) + (a_lo + e + l_lo);
    return 0.f - fmaf(t, kL1, fmaf(t, kL1lo, t_lo * kL1));
  }
};

// Element e of a lane's vector, e not known at compile time.
template <int kV>
__device__ __forceinline__ float pick(const float (&z)[kV], int e) {
  float x = z[0];
#pragma unroll
  for (int i = 1; i < kV; ++i) x = i == e ? z[i] : x;
  return x;
}

// floor(x n) and ceil(x n) for 0 <= x < 1: x 2^64 is a whole number (down to x = 2^-41;
// smaller ones are cut off at 2^-64).
__device__ __forceinline__ uint64_t part_floor(float x, uint64_t n) { return __umul64hi(__float2ull_rz(x * 0x1p64f), n); }
__device__ __forceinline__ uint64_t part_ceil(float x, uint64_t n) {
  const uint64_t f = __float2ull_ru(x * 0x1p64f);
  return __umul64hi(f, n) + (f * n != 0);
}

// A CTA's part of the row.  Places j stand for row entries first + j; those outside
// [lo, hi) are not of the slice and hold -inf.  Warp w has places [w seg, (w + 1) seg).
template <class T>
struct Slice {
  static constexpr int kV = 16 / sizeof(T);
  static constexpr int kStep = 32 * kV;  // places that a warp takes at once
  T* mem;
  const T* row;  // place 0, 16-byte aligned
  int first, lo, hi, cached, seg;

  // the lane's vector of the places from j0 on, from global memory
  __device__ __forceinline__ Vec<T, kV> load(int j0) const {
    const int j = j0 + int(threadIdx.x & 31) * kV;
    if (j + kV <= hi && j >= lo) return load_vec<T, kV>(row + j);
    Vec<T, kV> v;
#pragma unroll
    for (int e = 0; e < kV; ++e) v.v[e] = j + e >= lo && j + e < hi ? row[j + e] : from_f32<T>(-INFINITY);
    return v;
  }
  __device__ __forceinline__ Vec<T, kV> fetch(int j0) const {
    return j0 < cached ? load_vec<T, kV>(mem + j0 + int(threadIdx.x & 31) * kV) : load(j0);
  }
  // f(z, j) for the places [begin, end), kStep at a time, the next ones under way; j is the lane's first
  template <class F>
  __device__ __forceinline__ void each(int begin, int end, F&& f) const {
    if (begin >= end) return;
    Vec<T, kV> next = fetch(begin);
    for (int j0 = begin; j0 < end; j0 += kStep) {
      float z[kV];
#pragma unroll
      for (int e = 0; e < kV; ++e) z[e] = to_f32(next.v[e]);
      if (j0 + kStep < end) next = fetch(j0 + kStep);
      f(z, j0 + int(threadIdx.x & 31) * kV);
    }
  }
  // the same for the warp's places
  template <class F>
  __device__ __forceinline__ void each(F&& f) const {
    const int begin = int(threadIdx.x >> 5) * seg;
    each(begin, min(hi, begin + seg), f);
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
  // sums of two numbers over all CTAs
  __device__ __forceinline__ void total(uint64_t& a, uint64_t& b) {
    const Pair* all = tell(a, b);
    a = b = 0;
    for (int i = 0; i < ctas; ++i) {
      a += all[i].a;
      b += all[i].b;
    }
  }
};

// A bin can hold a whole row (equal logits), whose mass is below 2^62.  The addition that takes the low word past 2^32
// sees it, and carries: no number of entries is too many.  (One 64-bit atomic would be a loop of compare-and-swap.)
__device__ __forceinline__ void add_entry(Shared& s, int bin, uint64_t w) {
  const uint32_t lo = uint32_t(w);
  atomicAdd(&s.hist[0][bin], 1u);
  const uint32_t sum = atomicAdd(&s.hist[1][bin], lo) + lo;
  const uint32_t hi = uint32_t(w >> 32) + (sum < lo);
  if (hi) atomicAdd(&s.hist[2][bin], hi);
}
__device__ __forceinline__ void clear_hist(Shared& s, int parts) {
  __syncthreads();
  for (int i = threadIdx.x; i < parts * kBins; i += kThreadsS) s.hist[0][i] = 0u;
  __syncthreads();
}

// An interval [lo, hi) of places in the ranking, with `n` entries, and what stands before it.
struct Interval {
  uint64_t lo, hi, mass;
  uint32_t n, count;
};

// The interval's histogram over all CTAs, and in it the bin where the entries
// (kMass: the weights) from the ranking's start on reach `target`; n = 0 where
// none does.
template <bool kMass>
__device__ __forceinline__ void descend(Shared& s, Cluster& cl, Interval& v, int shift, uint64_t target) {
  constexpr int kMost = kBins / kThreadsS;
  const int per = kBins / cl.ctas, each = max(1, per / kThreadsS);  // bins of a CTA, of a thread
  const int bin0 = cl.rank * per + int(threadIdx.x) * each;
  const bool on = int(threadIdx.x) * each < per;
  if (threadIdx.x == 0) {
    s.found[0] = v.hi;
    s.found[1] = v.mass;
    s.found[2] = 0;
  }
  cluster_sync();  // the histograms are there
  uint64_t n[kMost], m[kMost], a = 0, b = 0;
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    n[k] = m[k] = 0;
    if (on && k < each) {
      for (int c = 0; c < cl.ctas; ++c) {
        const uint32_t at = map_to_cta(smem_u32(&s.hist[0][bin0 + k]), uint32_t(c));
        n[k] += ld_cluster(at);
        if (kMass)
          m[k] += ld_cluster(at + kBins * 4) + (uint64_t(ld_cluster(at + kBins * 8)) << 32);
      }
    }
    a += n[k];
    b += m[k];
  }
  const uint64_t own_a = a, own_b = b;
  uint64_t all_a, all_b = 0;
  if (kMass) {
    block_scan(s, a, b, all_a, all_b);
  } else {
    all_a = block_scan(s, a);
  }
  const Pair* all = cl.tell(all_a, all_b);
  uint64_t ca = v.count + a - own_a, cb = v.mass + b - own_b;
  for (int c = 0; c < cl.rank; ++c) {
    ca += all[c].a;
    cb += all[c].b;
  }
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    if (on && k < each) {
      const uint64_t before = kMass ? cb : ca, after = kMass ? cb + m[k] : ca + n[k];
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
}

__device__ __forceinline__ int shift_of(const Interval& v) {
  return max(0, 64 - __clzll((v.hi - v.lo - 1) | 1) - 11);
}

// Down to one entry: the ranking is cut behind it.
template <bool kMass, class T>
__device__ __forceinline__ void narrow(Shared& s, Cluster& cl, const Slice<T>& sl, const Weigh& weigh, Interval& v,
                                       uint64_t target) {
  constexpr int kV = Slice<T>::kV;
  while (v.n > 1) {
    clear_hist(s, kMass ? 3 : 1);
    const int shift = shift_of(v);
    // values outside [lowest, highest] are outside the interval (its end is not of it)
    const float highest = value_of(uint32_t(v.lo >> 32)), lowest = value_of(uint32_t((v.hi - 1) >> 32));
    sl.each([&](const float (&z)[kV], int j) {
      uint32_t mask = 0;
#pragma unroll
      for (int e = 0; e < kV; ++e) mask |= uint32_t(z[e] <= highest && z[e] >= lowest) << e;
      while (mask) {
        const int e = __ffs(mask) - 1;
        mask &= mask - 1;
        const float x = pick(z, e);
        const uint64_t at = place_of(x, sl.first + j + e);
        if (at < v.lo || at >= v.hi) continue;
        const int bin = int((at - v.lo) >> shift);
        if (kMass) {
          add_entry(s, bin, weigh(x));
        } else {
          atomicAdd(&s.hist[0][bin], 1u);
        }
      }
    });
    descend<kMass>(s, cl, v, shift, target);
  }
}

// Distance of a logit from the largest in bins of the first histogram, and the nearest
// bin: both monotone in z.  (Halves: top - z may lie beyond fp32.)  Those over kBins - 1.5,
// and what is not a number, are the last bin's.
__device__ __forceinline__ float first_distance(float z, float top, float per_unit) {
  return fmaf(z, -0.5f, 0.5f * top) * per_unit;
}
__device__ __forceinline__ int first_bin(float x) { return int(__float_as_uint(x + Weigh::kMagic) & uint32_t(kBins - 1)); }
// First key, between the maximum's and -inf's, whose value is in bin b or behind it; whole warps.
__device__ __forceinline__ uint32_t bin_edge(int b, float top, float per_unit) {
  auto before = [&](uint32_t key) {
    const float x = first_distance(value_of(key), top, per_unit);
    return (x < float(kBins) - 1.5f ? first_bin(x) : kBins - 1) < b;
  };
  uint32_t lo = key_of(top), hi = key_of(-INFINITY);
  // near where the border would be without rounding, mostly
  const float at = (0.5f * top - (float(b) - 0.5f) / per_unit) * 2.f;
  if (at > -INFINITY && at < top) {
    const uint32_t near = max(key_of(at), lo + 16u) - 16u + (threadIdx.x & 31);
    const uint32_t m = __ballot_sync(kFull, near < hi && before(near));
    if ((m & 1u) && m != kFull) return near - (threadIdx.x & 31) + __popc(m);
  }
  while (hi > lo) {
    const uint32_t step = (hi - lo + 31) / 32;
    const uint64_t i = uint64_t(lo) + uint64_t(threadIdx.x & 31) * step;
    const int c = __popc(__ballot_sync(kFull, i < hi && before(uint32_t(i))));
    if (step == 1 || c == 0) return lo + c;
    const uint32_t from = lo;
    lo = from + uint32_t(c - 1) * step + 1;
    const uint64_t to = uint64_t(from) + uint64_t(c) * step;
    hi = to < hi ? uint32_t(to) : hi;
  }
  return lo;
}

// Of the threads' numbers x (one each, all different; those of `in` count) within [lo, hi), in ascending order, the
// first up to which there are, with `base`, `target` of them (kMass: of their weights w); ~0 if there is none.
// Histograms over ever smaller intervals: two or three mostly, 1 us each.  (Sorting 1024 of them took 9 us.)
template <bool kMass>
__device__ __forceinline__ uint64_t block_select(Shared& s, uint64_t x, bool in, uint64_t w, uint64_t lo, uint64_t hi,
                                                 uint64_t base, uint64_t target) {
  uint32_t* const number = s.hist[1];
  unsigned long long* const mass = reinterpret_cast<unsigned long long*>(s.hist[2]);
  const uint32_t t = threadIdx.x;
  while (true) {
    const int shift = max(0, 64 - __clzll((hi - lo - 1) | 1) - 10);  // to kList bins
    const bool here = in && x >= lo && x < hi;
    number[t] = 0u;
    if (kMass) mass[t] = 0ull;
    if (t == 0) s.found[2] = 0;
    __syncthreads();
    if (here) {
      const uint32_t b = uint32_t((x - lo) >> shift);
      atomicAdd(&number[b], 1u);
      if (kMass) atomicAdd(&mass[b], static_cast<unsigned long long>(w));
    }
    __syncthreads();
    const uint64_t mine = kMass ? uint64_t(mass[t]) : uint64_t(number[t]);
    uint64_t upto = mine;
    block_scan(s, upto);
    upto += base;
    if (upto - mine < target && upto >= target) {
      s.found[0] = lo + (uint64_t(t) << shift);
      s.found[1] = upto - mine;
      s.found[2] = number[t];
    }
    __syncthreads();
    const uint64_t n = s.found[2];
    if (n == 0) return ~0ull;
    lo = s.found[0];
    hi = min(hi, lo + (uint64_t(1) << shift));
    base = s.found[1];
    if (n == 1 || shift == 0) break;
    __syncthreads();
  }
  if (in && x >= lo && x < hi) s.found[3] = x;
  __syncthreads();
  return s.found[3];
}

// A row's settings, and what it writes.
struct Row {
  uint32_t k;      // 0: all
  float top_p;
  bool nucleus;
  uint64_t least;  // weight, for min-p
  float u;
  // the place within the kept mass `whole` that the uniform number stands for
  __device__ __forceinline__ uint64_t goal(uint64_t whole) const {
    return u >= 1.f ? whole - 1 : u > 0.f ? part_floor(u, whole) : 0ull;  // a NaN counts as 0
  }
  __device__ __forceinline__ uint64_t target(uint64_t whole) const {
    return max(part_ceil(fmaxf(top_p, 0.f), whole), uint64_t(1));
  }
};
__device__ __forceinline__ void write(const SampleParams& p, int64_t row, int64_t token, float logprob, int64_t kept) {
  p.token[row] = token;
  if (p.logprob) p.logprob[row] = logprob;
  if (p.kept) p.kept[row] = kept;
}

// Two numbers per lane, `lane` and `lane + 32`, in ascending order.
__device__ __forceinline__ void warp_sort64(uint64_t (&x)[2], uint32_t n) {
  const uint32_t lane = threadIdx.x & 31;
  for (uint32_t k = 2; k < 2 * n; k *= 2) {
    for (uint32_t j = k / 2; j > 0; j /= 2) {
      if (j == 32) {  // (k = 64)
        const uint64_t lo = min(x[0], x[1]);
        x[1] = max(x[0], x[1]);
        x[0] = lo;
        continue;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint64_t y = __shfl_xor_sync(kFull, x[i], j);
        const bool low = (((lane + 32 * i) & k) == 0) == ((lane & j) == 0);
        x[i] = low ? min(x[i], y) : max(x[i], y);
      }
    }
  }
}
// The row's end where all entries that can stay are listed (n of them, at most kFew, for one warp): sorted by
// rank for the cuts, then by index for the choice.
constexpr uint32_t kFew = 64;
__device__ __forceinline__ void finish_few(Shared& s, const SampleParams& p, int64_t row, const Row& r,
                                           const Weigh& weigh, uint32_t n) {
  const uint32_t lane = threadIdx.x & 31;
  uint64_t x[2], w[2] = {0, 0}, upto[2] = {0, 0};
  bool in[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) x[i] = lane + 32 * i < n ? s.list()[lane + 32 * i] : ~0ull;
  warp_sort64(x, n);
  auto scan = [&] {
    upto[0] = warp_scan(w[0]);
    upto[1] = warp_scan(w[1]) + __shfl_sync(kFull, upto[0], 31);
    return __shfl_sync(kFull, upto[1], 31);
  };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t t = lane + 32 * i;
    in[i] = t < n && (r.k == 0 || t < r.k);
    w[i] = in[i] ? weigh(value_of(uint32_t(x[i] >> 32))) : 0ull;
  }
  uint64_t whole = scan();
  const uint64_t target = r.nucleus ? r.target(whole) : ~0ull;
  uint32_t kept = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    in[i] = in[i] && upto[i] - w[i] < target && w[i] >= r.least;
    kept += __popc(__ballot_sync(kFull, in[i]));
    x[i] = in[i] ? x[i] << 32 | x[i] >> 32 : ~0ull;
  }
  warp_sort64(x, kept);
#pragma unroll
  for (int i = 0; i < 2; ++i) w[i] = lane + 32 * i < kept ? weigh(value_of(uint32_t(x[i]))) : 0ull;
  whole = scan();
  const uint64_t goal = r.goal(whole);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (upto[i] > goal && upto[i] - w[i] <= goal)
      write(p, row, int64_t(x[i] >> 32), weigh.log_part(value_of(uint32_t(x[i])), whole), kept);
}

// The same for more of them (at most kList), one per thread; their places lie before `hi`.  `whole`: the mass
// that top-p is of, if it is known to be more than the list's.  False where top-p's cut lies behind the list.
__device__ __forceinline__ bool finish_list(Shared& s, const SampleParams& p, int64_t row, const Row& r,
                                            const Weigh& weigh, uint32_t n, uint64_t hi, uint64_t whole) {
  const uint32_t t = threadIdx.x;
  const uint64_t lo = uint64_t(key_of(weigh.top)) << 32, x = t < n ? s.list()[t] : ~0ull;
  const float z = value_of(uint32_t(x >> 32));
  bool in = t < n;
  if (r.k && r.k < n) {
    const uint64_t cut = block_select<false>(s, x, in, 0, lo, hi, 0, r.k);  // by all threads: it has barriers
    in = in && x <= cut;
  }
  uint64_t w = in ? weigh(z) : 0ull;
  if (r.nucleus) {
    const uint64_t listed = block_sums(s, warp_total(w)).all, target = r.target(whole ? whole : listed);
    if (listed < target) return false;
    const uint64_t cut = block_select<true>(s, x, in, w, lo, hi, 0, target);
    in = in && x <= cut;
  }
  in = in && w >= r.least;
  const uint32_t kept = __syncthreads_count(in);
  const uint64_t all = block_sums(s, warp_total(in ? w : 0ull)).all, i = uint32_t(x);
  const uint64_t drawn = block_select<true>(s, i, in, w, 0, uint64_t(p.vocab), 0, r.goal(all) + 1);
  if (in && i == drawn) write(p, row, int64_t(i), weigh.log_part(z, all), kept);
  return true;
}

template <class T>
__global__ void __launch_bounds__(kThreadsS, 1) sample_kernel(SampleParams p) {
  extern __shared__ __align__(16) uint8_t dynamic[];
  Shared& s = *reinterpret_cast<Shared*>(dynamic);
  constexpr int kV = Slice<T>::kV, kStep = Slice<T>::kStep;
  uint32_t ctas;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  Cluster cl{s, int(cluster_ctarank()), int(ctas)};
  const int64_t row = blockIdx.x / ctas;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool out = cl.rank == 0 && threadIdx.x == 0;

  // every CTA has to run before another one writes to its memory: the wait is below
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const float temperature = p.temperature ? p.temperature[row] : 1.f;
  const int64_t k_row = p.top_k ? p.top_k[row] : 0;
  const float top_p = p.top_p ? p.top_p[row] : 1.f, min_p = p.min_p ? p.min_p[row] : 0.f, u = p.uniform[row];
  for (int i = threadIdx.x; i < kBins; i += kThreadsS) s.hist[0][i] = 0u;
  if (warp == 0) {
    s.table[lane] = kTable[lane];
    const uint32_t u = uint32_t(kTable[lane] >> 31);
    s.pairs[lane] = make_uint2(u, __float_as_uint(float(u)));
  }
  if (threadIdx.x < 512) {
    const int over = int(threadIdx.x >> 3) - (p.bits - 31);
    s.octaves[threadIdx.x >> 3][threadIdx.x & 7] = (1u << max(-over, 0)) << 8 | uint32_t(min(max(over, 0), 31));
  }
  if (threadIdx.x == 0) {
    s.listed = 0u;
    s.last = 0ull;
  }
  if (threadIdx.x < kWarpsS) s.extra[threadIdx.x] = 0u;

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
    sl.seg = ((sl.hi + kWarpsS - 1) / kWarpsS + kStep - 1) / kStep * kStep;
  }
  Weigh weigh;
  weigh.top = -INFINITY;
  uint32_t total = 0;  // entries above -inf
  {
    const int begin = warp * sl.seg, end = min(sl.hi, begin + sl.seg);
    float top = -INFINITY;  // NaN if there is one
    float finite = 0.f;     // entries above -inf
    auto take = [&](const float (&z)[kV]) {
#pragma unroll
      for (int e = 0; e < kV; e += 2) asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(top) : "f"(top), "f"(z[e]), "f"(z[e + 1]));
#pragma unroll
      for (int e = 0; e < kV; ++e) finite += z[e] > -INFINITY ? 1.f : 0.f;
    };
    auto put = [&](int j0, const Vec<T, kV>& v) {
      if (j0 < sl.cached) store_vec<T, kV>(sl.mem + j0 + lane * kV, v);
      float z[kV];
#pragma unroll
      for (int e = 0; e < kV; ++e) z[e] = to_f32(v.v[e]);
      take(z);
    };
    int j0 = begin;
    if (j0 < sl.lo && j0 < end) {
      put(j0, sl.load(j0));
      j0 += kStep;
    }
    constexpr int kAhead = 4;  // loads under way at once
    for (; j0 + kAhead * kStep <= end; j0 += kAhead * kStep) {
      Vec<T, kV> v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) v[i] = load_vec<T, kV>(sl.row + j0 + i * kStep + lane * kV);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) put(j0 + i * kStep, v[i]);
    }
    for (; j0 < end; j0 += kStep) put(j0, sl.load(j0));
    // the largest by its bits as a signed integer, a NaN above all
    const int bits = top != top ? 0x7fffffff : __float_as_int(top + 0.f);
    const int most = __reduce_max_sync(kFull, bits >= 0 ? bits : bits ^ 0x7fffffff);
    const uint32_t mine = __reduce_add_sync(kFull, uint32_t(finite));
    if (lane == 0) s.wa[warp] = uint64_t(mine) << 32 | (uint32_t(most) ^ 0x80000000u);
    __syncthreads();
    uint32_t best = __reduce_max_sync(kFull, uint32_t(s.wa[lane]));
    const uint32_t count = __reduce_add_sync(kFull, uint32_t(s.wa[lane] >> 32));
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const Pair* all = cl.tell(best, count);
    for (int c = 0; c < cl.ctas; ++c) {
      best = max(best, uint32_t(all[c].a));
      total += uint32_t(all[c].b);
    }
    const int got = int(best ^ 0x80000000u);
    weigh.top = got == 0x7fffffff ? NAN : __int_as_float(got >= 0 ? got : got ^ 0x7fffffff);
  }
  const float top = weigh.top;
  const bool nan = top != top;
  if (top == -INFINITY) {  // nothing is allowed
    if (out) write(p, row, -1, -INFINITY, 0);
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
    __syncthreads();
    if (lane == 0) s.wb[warp] = uint64_t(best);
    __syncthreads();
    uint32_t low = __reduce_min_sync(kFull, uint32_t(s.wb[lane]));
    const Pair* all = cl.tell(low, 0);
    for (int c = 0; c < cl.ctas; ++c) low = min(low, uint32_t(all[c].a));
    if (out) write(p, row, int64_t(low), nan ? NAN : 0.f, 1);
    return;
  }

  weigh.bits = p.bits;
  weigh.table = s.table;
  weigh.pairs = s.pairs;
  weigh.octaves = reinterpret_cast<const uint8_t*>(&s.octaves[0][lane & 7]);
  weigh.set(temperature);
  Row r;
  r.k = k_row <= 0 || k_row >= p.vocab ? 0u : uint32_t(k_row);
  r.top_p = top_p;
  r.nucleus = top_p < 1.f;
  r.least = min_p > 0.f ? __float2ull_ru(fminf(min_p, 1.f) * float(1ull << p.bits)) : 0ull;
  r.u = u;

  // ---- where the ranking is cut: entries of smaller logits than cut_z are dropped, and those of
  // cut_z with an index above cut_i
  float cut_z = -INFINITY;
  int cut_i = INT32_MIN;
  uint64_t cut = ~0ull;
  auto cut_behind = [&](uint64_t place) {
    if (place >= cut) return;
    cut = place;
    cut_z = value_of(uint32_t(place >> 32));
    cut_i = int(min(uint32_t(place), uint32_t(INT32_MAX)));
  };
  // which of a vector's elements stay
  auto staying = [&](const float (&z)[kV], int i) {
    uint32_t mask = 0;
#pragma unroll
    for (int e = 0; e < kV; ++e) mask |= uint32_t(z[e] > cut_z || (z[e] == cut_z && i + e <= cut_i)) << e;
    return mask;
  };
  const uint32_t list_at = map_to_cta(smem_u32(s.list()), 0), listed_at = map_to_cta(smem_u32(&s.listed), 0);
  auto append = [&](float z, int i) {
    const uint32_t at = append_cluster(listed_at);
    if (at < kList) st_cluster(list_at + at * 8, place_of(z, i));
  };

  // What the warp's entries of larger logits than z_hi weigh, if that is known (they all stay, but for min-p),
  // and whether what stays of the others is in s.extra too, and `kept_n` in all.
  bool known = false, listed = false;
  float z_hi = INFINITY;
  uint64_t warp_ahead = 0;
  uint32_t kept_n = 0;
  if (r.k || r.nucleus) {
    // The first histogram, over the distance from the maximum.  Its last bin can hold most of the row: it is counted,
    // and its mass estimated, in registers.
    const float per_unit = weigh.c_hi * kBinsPerOctave;
    float last = 0.f;
    sl.each([&](const float (&z)[kV], int) {
#pragma unroll
      for (int e = 0; e < kV; ++e) {
        const float x = first_distance(z[e], top, per_unit), w = ex2_approx(x * (-1.f / kBinsPerOctave));
        if (x < float(kBins) - 1.5f) {
          atomicAdd(&s.hist[0][first_bin(x)], 1u);
        } else {
          last += w;
        }
      }
    });
    last = fminf(last, 1.f);  // (what is not a number too)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) last += __shfl_xor_sync(kFull, last, o);
    if (lane == 0) atomicAdd(&s.last, __float2ull_rz(last * 0x1p32f));
    cluster_sync();  // the histograms are there
    // each CTA adds up a part of the bins, and tells all others: a thread for one bin and some of the CTAs
    const int per = kBins / cl.ctas;
    if (cl.ctas == 1) {
      for (int b = threadIdx.x; b < kBins; b += kThreadsS) s.first[b] = s.hist[0][b];
    } else {
      const int groups = max(1, kThreadsS / per), share = cl.ctas / groups;  // per <= 1024
      const int b = int(threadIdx.x) % per, bin = cl.rank * per + b, c0 = int(threadIdx.x) / per * share;
      uint32_t n = 0;
      for (int i = 0; i < share; ++i) n += ld_cluster(map_to_cta(smem_u32(&s.hist[0][bin]), uint32_t(c0 + i)));
      // (this CTA's own bins of s.hist[1] collect the groups' parts)
      if (threadIdx.x < per) s.hist[1][b] = 0u;
      __syncthreads();
      atomicAdd(&s.hist[1][b], n);
      __syncthreads();
      n = s.hist[1][b];
      for (int i = 0; i < share; ++i) st_cluster(map_to_cta(smem_u32(&s.first[bin]), uint32_t(c0 + i)), n);
    }
    if (warp == kWarpsS - 1) {
      const uint64_t mass = warp_total(lane < cl.ctas ? ld_cluster64(map_to_cta(smem_u32(&s.last), uint32_t(lane))) : 0ull);
      if (lane == 0) s.found[3] = mass;
    }
    if (threadIdx.x < 2) s.at[threadIdx.x] = kBins - 1;
    cluster_sync();
    // each thread has two bins: their entries, up to their ends
    constexpr int kPer = kBins / kThreadsS;
    const int bin0 = int(threadIdx.x) * kPer;
    uint32_t n[kPer];
    uint64_t upto = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) upto += n[i] = bin0 + i == kBins - 1 ? 0u : s.first[bin0 + i];
    const uint32_t mine = uint32_t(upto);
    const uint32_t binned = uint32_t(block_scan(s, upto));
    const uint32_t before = uint32_t(upto) - mine;
    if (threadIdx.x == kThreadsS - 1) n[kPer - 1] = total - binned;
    const float tail_mass = float(s.found[3]);
    if (r.k >= total) r.k = 0;
    const uint32_t most = r.k ? r.k : total;
    uint64_t est[kPer], e_upto = 0;  // of the mass of the first `most`, in units of 2^-32 of the largest weight
    {
      uint32_t at = before;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t in = min(at + n[i], most) - min(at, most);
        if (r.k && at < r.k && at + n[i] >= r.k) s.at[0] = bin0 + i;
        at += n[i];
        s.first[bin0 + i] = at;
        est[i] = bin0 + i < kBins - 1 ? uint64_t(in) * uint64_t(exp2f(32.f - float(bin0 + i) / kBinsPerOctave))
                                      : uint64_t(tail_mass * (float(in) / fmaxf(float(n[i]), 1.f)));
        e_upto += est[i];
      }
    }
    __syncthreads();
    auto up_to = [&](int b) { return b < 0 ? 0u : s.first[b]; };  // entries of the bins 0 to b
    auto edge = [&](int b) { return uint64_t(b >= kBins ? key_of(-INFINITY) : bin_edge(b, top, per_unit)) << 32; };
    Interval v{};
    if (r.k) {
      const int b = s.at[0];
      v.count = up_to(b - 1);
      v.n = up_to(b) - v.count;
      v.lo = edge(b);
      v.hi = edge(b + 1);
      const bool few = v.count + v.n <= kList;  // one block can finish them
      if (few || v.n <= kList) {
        const float low = value_of(uint32_t(v.hi >> 32)), high = few ? INFINITY : value_of(uint32_t(v.lo >> 32));
        sl.each([&](const float (&z)[kV], int j) {
#pragma unroll
          for (int e = 0; e < kV; ++e)
            if (z[e] > low && z[e] <= high) append(z[e], sl.first + j + e);
        });
        cluster_sync();
        if (few) {
          if (cl.rank == 0) {
            if (v.count + v.n > kFew) {
              finish_list(s, p, row, r, weigh, v.count + v.n, v.hi, 0);
            } else if (warp == 0) {
              finish_few(s, p, row, r, weigh, v.count + v.n);
            }
          }
          return;
        }
        uint64_t place = 0;
        if (cl.rank == 0) {
          const uint64_t x = threadIdx.x < v.n ? s.list()[threadIdx.x] : ~0ull;
          place = block_select<false>(s, x, threadIdx.x < v.n, 0, v.lo, v.hi, v.count, r.k);
          if (threadIdx.x == 0) s.listed = 0u;
        }
        cut_behind(cl.tell(place, 0)[0].a);
      } else {
        narrow<false>(s, cl, sl, weigh, v, r.k);
        cut_behind(v.hi - 1);
      }
    }
    if (r.nucleus) {
      // Estimates of the mass up to each bin name the bins in which it reaches p of the whole.  A
      // bin's weights lie within 2^(1/128) = 1 + 0.0054 of its middle's, and errors before and
      // behind the border count 1 - p and p in their difference: at most 0.0109 p (1 - p) of the
      // whole.  (That it is reached there is seen below, from exact sums.)
      const uint64_t e_mine = e_upto;
      const float e_whole = float(block_scan(s, e_upto)), goal = r.top_p * e_whole;
      const float slack = e_whole * (0.0112f * fmaxf(r.top_p * (1.f - r.top_p), 0.f) + 2e-6f);
      float e_at = float(e_upto - e_mine);
      if (threadIdx.x < 2) s.at[threadIdx.x] = kBins - 1;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        e_at += float(est[i]);
        if (e_at >= goal - slack) atomicMin(&s.at[0], bin0 + i);
        if (e_at >= goal + slack) atomicMin(&s.at[1], bin0 + i);
      }
      __syncthreads();
      const int b_lo = s.at[0], b_hi = s.at[1];
      const uint32_t before_lo = up_to(b_lo - 1), through = up_to(b_hi);
      const bool few = !r.k && through <= kList;  // one block can finish them
      v.lo = edge(b_lo);
      v.hi = edge(b_hi + 1);
      uint64_t target = 0;
      bool found = false;
      known = true;
      for (int round = 0; round < 2 && !found; ++round) {
        // The mass of the whole, of what stands before these bins, and a list of their entries (with `few`, of
        // those before them too), or their histogram where they are many.
        const bool listing = round == 0 && (few || through - before_lo <= kList);
        if (!listing) clear_hist(s, 3);
        const int shift = shift_of(v);
        // (whole keys) larger logits than z_hi stand before the bins, up to z_lo behind them
        z_hi = value_of(uint32_t(v.lo >> 32));
        const float z_lo = value_of(uint32_t(v.hi >> 32)), z_list = listing ? few ? INFINITY : z_hi : -INFINITY;
        uint64_t whole = 0, ahead = 0;
        sl.each([&](const float (&z)[kV], int j) {
          uint32_t stay = ~0u;
          if (cut != ~0ull) stay = staying(z, sl.first + j);
          float np[kV], most = -INFINITY;
          bool any = false;
#pragma unroll
          for (int e = 0; e < kV; e += 2) {
            Term t[2];
            float np2[2];
            weigh.pair(z[e], z[e + 1], t, np2);
            asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(most) : "f"(most), "f"(np2[0]), "f"(np2[1]));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              np[e + i] = np2[i];
              const bool before = z[e + i] > z_hi;
              if (!((stay >> (e + i)) & 1u)) t[i].power = 0u;
              any |= z[e + i] > z_lo && (few || !before);
              t[i].add_to(whole);
              if (!before) t[i].power = 0u;
              t[i].add_to(ahead);
            }
          }
          if (!any && most <= Weigh::kNear) return;
          uint32_t rare = 0;
#pragma unroll
          for (int e = 0; e < kV; ++e) rare |= uint32_t(!(np[e] <= Weigh::kNear) || (z[e] > z_lo && (few || z[e] <= z_hi))) << e;
          rare &= stay;
          while (rare) {
            const int e = __ffs(rare) - 1;
            rare &= rare - 1;
            const float x = pick(z, e);
            const int i = sl.first + j + e;
            if (x == -INFINITY) continue;
            Term t[2];
            float np2[2];
            weigh.pair(x, x, t, np2);
            uint64_t w = t[0].value();
            if (!(np2[0] <= Weigh::kNear)) {
              const uint64_t more = weigh.precise(x) - w;
              w += more;
              whole += more;
              if (x > z_hi) ahead += more;
            }
            if (x <= z_lo) continue;
            if (x <= z_list) {
              append(x, i);
            } else if (x <= z_hi) {
              add_entry(s, int((place_of(x, i) - v.lo) >> shift), w);
            }
          }
        });
        warp_ahead = warp_total(ahead);
        whole = warp_total(whole);
        ahead = warp_ahead;
        block_sums(s, whole, ahead);
        cl.total(whole, ahead);
        target = r.target(whole);
        if (listing && few) {
          bool done = false;
          if (cl.rank == 0) done = finish_list(s, p, row, r, weigh, through, v.hi, whole);
          if (cl.tell(done, 0)[0].a) return;
        } else if (listing) {
          uint64_t place = ~0ull, counts = 0;
          if (cl.rank == 0) {
            const uint32_t t = threadIdx.x, len = s.listed;
            const uint64_t x = t < len ? s.list()[t] : ~0ull;
            const uint64_t w = t < len ? weigh(value_of(uint32_t(x >> 32))) : 0ull;
            if (ahead < target) place = block_select<true>(s, x, t < len, w, v.lo, v.hi, ahead, target);
            counts = uint64_t(len) << 32 | uint32_t(__syncthreads_count(x <= place && t < len));
          }
          const Pair* all = cl.tell(place, counts);
          place = all[0].a;
          found = place != ~0ull;
          if (found) {
            cut_behind(place);
            listed = true;
            kept_n = before_lo + uint32_t(all[0].b);
            // what the listed entries that stay add to the warps in whose parts they lie
            if (threadIdx.x < uint32_t(all[0].b >> 32)) {
              const uint64_t x = ld_cluster64(list_at + threadIdx.x * 8);
              const int j = int(uint32_t(x)) - sl.first;
              if (x <= place && j >= sl.lo && j < sl.hi)
                atomicAdd(reinterpret_cast<unsigned long long*>(&s.extra[j / sl.seg]),
                          static_cast<unsigned long long>(weigh(value_of(uint32_t(x >> 32)))));
            }
            __syncthreads();
          }
        } else {
          v.mass = ahead;
          v.count = 0;
          v.n = 0;
          if (ahead < target) descend<true>(s, cl, v, shift, target);
          found = v.n != 0;
          if (found) {
            narrow<true>(s, cl, sl, weigh, v, target);
            cut_behind(v.hi - 1);
          }
        }
        // else the estimate was too far off: every place (where the sums, which are exact, reach the target)
        v.lo = uint64_t(key_of(top)) << 32;
        v.hi = uint64_t(key_of(-INFINITY)) << 32;
      }
    }
  }

  // ---- the kept entries' mass, in index order, and the entry that the number falls on
  uint64_t mass = 0;
  uint32_t count = 0;
  auto dense = [&](const float (&z)[kV], int j) {
    uint32_t stay = ~0u;
    if (cut != ~0ull) {
      stay = staying(z, sl.first + j);
      count += __popc(stay);
    }
    float np[kV], most = -INFINITY;
#pragma unroll
    for (int e = 0; e < kV; e += 2) {
      Term t[2];
      float np2[2];
      weigh.pair(z[e], z[e + 1], t, np2);
      asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(most) : "f"(most), "f"(np2[0]), "f"(np2[1]));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        np[e + i] = np2[i];
        if (!((stay >> (e + i)) & 1u)) t[i].power = 0u;
        t[i].add_to(mass);
      }
    }
    if (most <= Weigh::kNear) return;
    uint32_t rare = 0;
#pragma unroll
    for (int e = 0; e < kV; ++e) rare |= uint32_t(!(np[e] <= Weigh::kNear) && z[e] > -INFINITY) << e;
    rare &= stay;
    while (rare) {
      const float x = pick(z, __ffs(rare) - 1);
      rare &= rare - 1;
      Term t[2];
      float np2[2];
      weigh.pair(x, x, t, np2);
      mass += weigh.precise(x) - t[0].value();
    }
  };
  // one entry per lane at a time: where few are looked at
  auto sparse = [&](const float (&z)[kV], uint32_t mask) {
    while (mask) {
      const uint64_t w = weigh(pick(z, __ffs(mask) - 1));
      mask &= mask - 1;
      mass += w >= r.least ? w : 0ull;
      count += w >= r.least;
    }
  };
  if (r.least) {
    // min-p's border in logits, roughly: nothing more than two octaves behind it is looked at
    const float near = top - fmaxf(-log2f(min_p) + 2.f, 2.f) * 2.f / weigh.c_hi;
    sl.each([&](const float (&z)[kV], int j) {
      uint32_t mask = staying(z, sl.first + j);
#pragma unroll
      for (int e = 0; e < kV; ++e) mask &= ~(uint32_t(z[e] < near) << e);
      sparse(z, mask);
    });
  } else if (listed) {
    if (lane == 0) mass = warp_ahead + s.extra[warp];
  } else if (known) {
    sl.each([&](const float (&z)[kV], int j) {
      uint32_t mask = 0;
#pragma unroll
      for (int e = 0; e < kV; ++e) {
        count += z[e] > z_hi;
        mask |= uint32_t(z[e] <= z_hi && z[e] >= cut_z) << e;
      }
      if (mask) sparse(z, mask & staying(z, sl.first + j));
    });
    mass += (lane == 0) * warp_ahead;
  } else {
    sl.each(dense);
  }
  mass = warp_total(mass);
  const Sums sums = block_sums(s, mass);
  uint64_t whole = sums.all, kept = total, ahead = 0;
  if (listed && !r.least) {
    kept = kept_n;
  } else if (cut != ~0ull || r.least) {
    kept = block_sums(s, uint64_t(__reduce_add_sync(kFull, count))).all;
  }
  if (cl.ctas > 1) {
    const Pair* all = cl.tell(sums.all, kept);
    whole = 0;
    const bool add = (cut != ~0ull || r.least) && !(listed && !r.least);
    if (add) kept = 0;
    for (int i = 0; i < cl.ctas; ++i) {
      if (i < cl.rank) ahead += all[i].a;
      whole += all[i].a;
      if (add) kept += all[i].b;
    }
  }
  const uint64_t goal = r.goal(whole);
  if (goal < ahead || goal - ahead >= sums.all) return;  // it falls into another CTA's slice
  // the warp's part in which it falls is shared out among all warps
  __syncthreads();
  if (lane == 0 && goal - ahead >= sums.before && goal - ahead - sums.before < mass) {
    s.at[0] = warp;
    s.found[0] = ahead + sums.before;
  }
  __syncthreads();
  const int part0 = s.at[0] * sl.seg, part = cdiv(sl.seg / kStep, kWarpsS) * kStep;
  const int begin = part0 + warp * part, end = min(min(sl.hi, part0 + sl.seg), begin + part);
  const uint64_t from = s.found[0];
  auto weights = [&](const float (&z)[kV], int i, uint64_t (&w)[kV]) {
    const uint32_t stay = staying(z, i);
    uint64_t sum = 0;
#pragma unroll
    for (int e = 0; e < kV; ++e) {
      w[e] = (stay >> e) & 1u ? weigh(z[e]) : 0ull;
      if (w[e] < r.least) w[e] = 0ull;
      sum += w[e];
    }
    return sum;
  };
  uint64_t sum = from;
  if (sl.seg > kStep) {
    mass = 0;
    sl.each(begin, end, [&](const float (&z)[kV], int j) {
      uint64_t w[kV];
      mass += weights(z, sl.first + j, w);
    });
    mass = warp_total(mass);
    sum += block_sums(s, mass).before;
    if (goal < sum || goal - sum >= mass) return;
  } else if (warp > 0) {
    return;  // it is one step, the first warp's
  }
  bool done = false;
  sl.each(begin, end, [&](const float (&z)[kV], int j) {
    if (done) return;
    uint64_t w[kV];
    const uint64_t mine = weights(z, sl.first + j, w);
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
            write(p, row, sl.first + j + e, weigh.log_part(z[e], whole), int64_t(kept));
          }
        }
      }
    }
    sum += __shfl_sync(kFull, upto, 31);
  });
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
constexpr size_t kFixed = (sizeof(Shared) + 15) / 16 * 16;
constexpr size_t kMostSmem = 227 << 10;

int validate(const flce_sample_problem* p) {
  if (!p) return FLCE_ERR_INVALID_ARG;
  if (p->rows < 0 || p->rows > INT32_MAX / kMaxCtas || p->vocab < 1 || p->vocab > kMaxVocab || p->logits_stride < 0)
    return FLCE_ERR_INVALID_ARG;
  if (!known_dtype(p->logits_dtype)) return FLCE_ERR_UNSUPPORTED_DTYPE;
  return FLCE_OK;
}

template <class T>
cudaLaunchConfig_t config(int ctas, cudaLaunchAttribute* attr, size_t smem, cudaStream_t st) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kThreadsS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Clusters of 1, 2, 4, 8 and 16 CTAs that run at once on the current device (one CTA takes an SM), from
// the driver, once per device; in atomics, so that host threads may call at once.
template <class T>
cudaError_t clusters(int device, int (&out)[5]) {
  static std::atomic<int> known[64][5];
  for (int i = 0; i < 5; ++i) {
    int n = known[device][i].load(std::memory_order_relaxed);
    if (n == 0) {
      cudaLaunchAttribute attr[1];
      const cudaLaunchConfig_t cfg = config<T>(1 << i, attr, kMostSmem, nullptr);
      const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, sample_kernel<T>, &cfg);
      if (e != cudaSuccess) return e;
      known[device][i].store(n > 0 ? n : -1, std::memory_order_relaxed);
    }
    out[i] = n;
  }
  return cudaSuccess;
}

template <class T>
cudaError_t launch_sample(SampleParams& q, int64_t rows, int device, cudaStream_t st) {
  constexpr int kV = Slice<T>::kV, kStep = Slice<T>::kStep;
  if (device >= 64) return cudaErrorInvalidDevice;
  auto kern = sample_kernel<T>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMostSmem));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  int at_once[5];
  if (e == cudaSuccess) e = clusters<T>(device, at_once);
  if (e != cudaSuccess) return e;
  // CTAs of a row: the least of rounds of clusters x time of a row, which is about 0.5 ns for each of a
  // CTA's entries and 20 us, 12 without other CTAs (8 x 262144 fp32, top-p: 93, 58 and 44 us with 2, 4 and 8 CTAs; 256 rows of
  // them: 341 and 366 us with 1 and 2)
  int best = 0;
  double least = 0.0;
  for (int i = 0; i < 5; ++i) {
    if (at_once[i] <= 0) continue;
    const double t = double(cdiv(rows, at_once[i])) * (double(cdiv(q.vocab, 1 << i)) * 0.5e-3 + (i ? 20.0 : 12.0));
    if (least == 0.0 || t < least) {
      least = t;
      best = i;
    }
  }
  const int ctas = 1 << best;
  q.slice = int32_t(cdiv(cdiv(q.vocab, ctas), kV) * kV);
  const int64_t places = cdiv(q.slice + kV - 1, int64_t(kStep) * kWarpsS) * kStep * kWarpsS;
  q.cached = int32_t(std::min<int64_t>(places, int64_t(kMostSmem - kFixed) / int64_t(sizeof(T)) / kStep * kStep));
  int bits = 62;  // the sum of all weights fits 63 bits
  for (int64_t v = 1; v < q.vocab; v *= 2) --bits;
  q.bits = std::min(46, bits);
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config<T>(ctas, attr, kFixed + size_t(q.cached) * sizeof(T), st);
  cfg.gridDim = dim3(unsigned(rows * ctas));
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
    if (p->logits_dtype == FLCE_F32) return launch_sample<float>(q, p->rows, dev.index, st);
    if (p->logits_dtype == FLCE_BF16) return launch_sample<__nv_bfloat16>(q, p->rows, dev.index, st);
    return launch_sample<__half>(q, p->rows, dev.index, st);
  });
}

}  // extern "C"
