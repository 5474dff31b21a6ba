// flce_embed.cu — embedding lookup with scaling, and the table's gradient by
// sorted tokens: kernels and the C entry points.
//
//   out_i = rn(W[id_i] s),  0 where id_i is outside [0, V)
//   dW[v] = rn(s sum of dout_i over the tokens i with id_i = v, in order)   (+ dW[v] when accumulating)
//
// Both are bound by memory: the lookup reads and writes a row per token, the
// gradient reads one per token and writes the whole table.
//
// The gradient has three launches.  One cluster sorts the tokens by id (stable,
// so equal ids stay in the tokens' order; 16 us for 16384), while the other SMs clear
// the table's last rows.  Then blocks of kChunk sorted tokens sum their rows in
// registers.  A run of one id that ends in its chunk or the one behind it is the first
// one's block's, and goes straight to the table; the parts of longer runs go to fp32
// slots.  Other blocks of the same launch write zeros to those of the other rows that
// no token names, so that these are written once.  The third launch joins the parts,
// in order.  Nothing depends on the order in which blocks run: same bits every time.
//
// 16384 x 4096 bf16 over 151936 rows, one token in 16 without an id: lookup to fp32 63 us (the
// copy rate gives 58 for the rows of all tokens, 54 for those of 12244 different ones), gradient
// 227 (202).  8 rows: 2.  20011 x 1283 fp32 into 4099 rows: 46 (17), of which the sort takes 18,
// the join and two launches 8.  The sort has eight SMs, whatever the number of tokens.
#include <algorithm>
#include <cmath>

#include "flce_device.cuh"
#include "flce_elem.cuh"
#include "flce_host.h"

namespace flce {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kElems = 8;             // elements of a row that a thread holds
constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxWidth = int64_t(1) << 24;

__host__ __device__ constexpr int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

__device__ __forceinline__ int64_t id_at(const void* ids, int i64, int64_t i) {
  return i64 ? static_cast<const int64_t*>(ids)[i] : int64_t(static_cast<const int32_t*>(ids)[i]);
}

// kElems elements of a row: adjacent ones from `at` on (kVec), or one of every kWide
// from `at` on, of which the row has `count`.
constexpr int kWide = 256;
template <class T>
struct Raw {
  Vec<T, kElems> v;
};
template <class T, bool kVec>
__device__ __forceinline__ void load_elems(const T* at, int count, Raw<T>& r) {
  if constexpr (kVec) {
    if (count > 0) r.v = load_vec<T, kElems>(at);
  } else {
#pragma unroll
    for (int e = 0; e < kElems; ++e)
      if (e < count) r.v.v[e] = at[e * kWide];
  }
}
template <class O, bool kVec>
__device__ __forceinline__ void store_elems(O* at, int count, const float (&x)[kElems]) {
  if constexpr (kVec) {
    if (count <= 0) return;
    Vec<O, kElems> v;
#pragma unroll
    for (int e = 0; e < kElems; ++e) v.v[e] = from_f32<O>(x[e]);
    store_vec<O, kElems>(at, v);
  } else {
#pragma unroll
    for (int e = 0; e < kElems; ++e)
      if (e < count) at[e * kWide] = from_f32<O>(x[e]);
  }
}
// Columns [tile * threads * kElems, ...) of `threads` threads: the t-th's first one, and how many it has.
template <bool kVec>
__device__ __forceinline__ int first_col(int tile, int t, int threads, int cols, int& count) {
  const int at = tile * threads * kElems + t * (kVec ? kElems : 1);
  count = at >= cols ? 0 : kVec ? kElems : min(kElems, (cols - at + kWide - 1) / kWide);
  return at;
}

// ---------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------
struct EmbedParams {
  const void* ids;
  const void* weight;
  void* out;
  int64_t tokens, vocab, ws, os;
  int32_t cols, tiles, ids_i64;
  float scale;
};

// kRows tokens per block and tile of columns: their rows are under way at once.
template <class T, class O, bool kVec, int kRows>
__global__ void __launch_bounds__(256) embed_kernel(EmbedParams p) {
  const int tile = int(blockIdx.x % unsigned(p.tiles));
  const int64_t first = int64_t(blockIdx.x / unsigned(p.tiles)) * kRows;
  int cnt;
  const int at = first_col<kVec>(tile, int(threadIdx.x), int(blockDim.x), p.cols, cnt);
  Raw<T> r[kRows];
  bool there[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t i = first + k;
    const int64_t id = i < p.tokens ? id_at(p.ids, p.ids_i64, i) : -1;
    there[k] = id >= 0 && id < p.vocab;
    if (there[k]) load_elems<T, kVec>(static_cast<const T*>(p.weight) + id * p.ws + at, cnt, r[k]);
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if (first + k >= p.tokens) break;
    float x[kElems];
#pragma unroll
    for (int e = 0; e < kElems; ++e) x[e] = there[k] ? __fmul_rn(to_f32(r[k].v.v[e]), p.scale) : 0.f;
    store_elems<O, kVec>(static_cast<O*>(p.out) + (first + k) * p.os + at, cnt, x);
  }
}

// ---------------------------------------------------------------------------
// Stable sort of the tokens by id
// ---------------------------------------------------------------------------
// (id << 32 | token), ids that have no gradient as `vocab`: they come last.
constexpr int kSortThreads = 1024, kSortWarps = 32;
constexpr int kMaxDigit = 10;          // bits of an id taken in one pass
constexpr int kSortCtas = 8;           // of the cluster
constexpr int64_t kSortOne = 4096;     // up to so many tokens one block does it: 2 us less than a cluster's barriers

// Rows of a table that are cleared: [first, end).
struct ClearParams {
  uint8_t* table;
  int64_t stride, bytes;  // of a row
  int64_t first, end;
};

struct SortParams {
  ClearParams clear;
  const void* ids;
  uint64_t *a, *b;   // pass 0 writes a, pass 1 writes b, ...
  uint32_t* joins;   // counter that the sums start from zero
  int64_t n, vocab, padding;
  int32_t ids_i64, passes, width;  // passes of `width` bits
  int32_t ctas;                    // of the sort: the first ones
};

// Zeros to a row (of elements of 2 or 4 bytes), by `lanes` threads (8 or more) of which this is the `at`-th: single
// units of two bytes up to a 16-byte boundary, whole vectors, the rest.
__device__ __forceinline__ void clear_row(uint8_t* row, int64_t bytes, int at, int lanes) {
  const int head = int(min(bytes, int64_t(-reinterpret_cast<uintptr_t>(row) & 15)));
  const int64_t vecs = (bytes - head) / 16, tail = head + vecs * 16;
  if (2 * at < head) *reinterpret_cast<uint16_t*>(row + 2 * at) = 0;
  for (int64_t i = at; i < vecs; i += lanes) *reinterpret_cast<uint4*>(row + head + i * 16) = make_uint4(0u, 0u, 0u, 0u);
  if (tail + 2 * at < bytes) *reinterpret_cast<uint16_t*>(row + tail + 2 * at) = 0;
}
// Threads for a row: a warp or a part of it.
__device__ __forceinline__ int row_lanes(int64_t bytes) { return bytes > 256 ? 32 : bytes > 128 ? 16 : 8; }

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// The lanes of `among` (this one is of it) with the same `width` bits in d.  (A ballot
// for each bit: a match over the warp takes some 37 cycles of the SM.)
__device__ __forceinline__ uint32_t same_digit(uint32_t among, uint32_t d, int width) {
  for (int b = 0; b < width; ++b) {
    const uint32_t ones = __ballot_sync(kFull, (d >> b) & 1u);
    among &= (d >> b) & 1u ? ones : ~ones;
  }
  return among;
}

// Least significant digit first.  Every warp of the cluster owns a stretch of the
// array: it counts its digits, 32 keys at a time, the counts are summed over warps,
// CTAs (distributed shared memory) and digits, and the warp places its keys, in
// order.  The GPU's other SMs meanwhile clear rows at the table's end, whether a token
// names them or not.
__global__ void __launch_bounds__(kSortThreads, 1) sort_tokens_kernel(SortParams p) {
  extern __shared__ uint32_t smem[];
  const int radix = 1 << p.width;
  uint32_t* count = smem;                          // [warp][digit]
  uint32_t* total = count + kSortWarps * radix;    // [digit] of this CTA
  uint32_t* base = total + radix;                  // [digit] where this CTA's keys go
  __shared__ uint32_t warp_sum_buf[kSortWarps];
  griddep_release();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = int(cluster_ctarank()), ctas = p.ctas;
  if (int(blockIdx.x) >= ctas) {
    const int lanes = row_lanes(p.clear.bytes), per_block = kSortThreads / lanes;
    const int64_t step = int64_t(gridDim.x - ctas) * per_block;
    for (int64_t r = p.clear.first + int64_t(blockIdx.x - ctas) * per_block + int(threadIdx.x) / lanes; r < p.clear.end; r += step)
      clear_row(p.clear.table + r * p.clear.stride, p.clear.bytes, int(threadIdx.x) % lanes, lanes);
    return;
  }
  const int64_t per = cdiv(cdiv(p.n, int64_t(ctas) * kSortWarps), 32) * 32;
  const int64_t lo = min(p.n, (int64_t(rank) * kSortWarps + warp) * per), hi = min(p.n, lo + per);
  if (rank == 0 && threadIdx.x == 0) *p.joins = 0u;
  uint32_t* mine = count + warp * radix;
  const uint64_t* src = nullptr;
  uint64_t* dst = p.a;
  auto key_at = [&](int64_t i) -> uint64_t {
    if (src) return __ldcg(src + i);
    const int64_t id = id_at(p.ids, p.ids_i64, i);
    const bool counts = id >= 0 && id < p.vocab && id != p.padding;
    return uint64_t(counts ? id : p.vocab) << 32 | uint64_t(i);
  };
  constexpr int kBatch = 4;  // keys of a lane under way at once
  uint64_t key[kBatch];
  uint32_t rank_of[kBatch];  // the key's place among the warp's of its digit
  const bool once = per <= 32 * kBatch;  // the warp's keys and ranks stay in registers
  auto fetch = [&](int64_t i0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) key[u] = i0 + u * 32 + lane < hi ? key_at(i0 + u * 32 + lane) : 0ull;
  };
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = 32 + pass * p.width;
    for (int d = lane; d < radix; d += 32) mine[d] = 0u;
    __syncwarp();
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kBatch) {
      fetch(i0);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (i0 + u * 32 >= hi) break;
        const bool in = i0 + u * 32 + lane < hi;
        const uint32_t d = uint32_t(key[u] >> shift) & uint32_t(radix - 1);
        const uint32_t same = same_digit(__ballot_sync(kFull, in), d, p.width);
        rank_of[u] = mine[d] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (in && lane == __ffs(same) - 1) mine[d] += __popc(same);
        __syncwarp();
      }
    }
    __syncthreads();
    const int d = int(threadIdx.x);
    if (d < radix) {
      uint32_t c[kSortWarps], s = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) c[w] = count[w * radix + d];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        count[w * radix + d] = s;
        s += c[w];
      }
      total[d] = s;
    }
    cluster_sync();
    uint32_t before = 0, all = 0;
    if (d < radix) {
      uint32_t v[kSortCtas];  // (all under way at once)
#pragma unroll
      for (int c = 0; c < kSortCtas; ++c) v[c] = c < ctas ? ld_cluster(map_to_cta(smem_u32(total + d), uint32_t(c))) : 0u;
#pragma unroll
      for (int c = 0; c < kSortCtas; ++c) {
        if (c < rank) before += v[c];
        all += v[c];
      }
    }
    // exclusive sum of `all` over the digits
    uint32_t incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum_buf[warp] = incl;
    __syncthreads();
    uint32_t prior = lane < warp ? warp_sum_buf[lane] : 0u;
    prior = __reduce_add_sync(kFull, prior);
    if (d < radix) base[d] = prior + incl - all + before;
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kBatch) {
      if (!once) fetch(i0);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (i0 + u * 32 >= hi) break;
        const bool in = i0 + u * 32 + lane < hi;
        const uint32_t g = uint32_t(key[u] >> shift) & uint32_t(radix - 1), to = base[g] + mine[g];
        if (once) {
          if (in) dst[to + rank_of[u]] = key[u];
          continue;
        }
        const uint32_t same = same_digit(__ballot_sync(kFull, in), g, p.width);
        if (in) dst[to + __popc(same & ((1u << lane) - 1u))] = key[u];
        __syncwarp();
        if (in && lane == __ffs(same) - 1) mine[g] += __popc(same);
        __syncwarp();
      }
    }
    cluster_sync();  // the keys are there, and nobody reads `total` any more
    src = dst;
    dst = dst == p.a ? p.b : p.a;
  }
}

// ---------------------------------------------------------------------------
// Sums over the sorted tokens
// ---------------------------------------------------------------------------
constexpr int kChunk = 32;             // sorted tokens of a block: a warp's worth of keys
constexpr int kMostTeams = 8;          // chunks of a block, where the rows are narrow
constexpr int kZeroBytes = 128 << 10;  // of the table that a block clears, at most
constexpr int kZeroLeast = 16 << 10;
// Bytes that are cleared during the sort, where eight blocks sort and where one does.  (More of them slow the
// sort, which waits for L2: 8192 tokens into 32000 x 2048 bf16 56 us without, 54 with 48 MB, 67 with 96; 16384 into
// 151936 x 4096 230, 225, 225.)
constexpr int64_t kEarly = 48 << 20;
constexpr int64_t kEarlyOne = 16 << 20;
constexpr int kZeroRows = 4096;        // at most

struct EmbedBwdParams {
  const uint64_t* sorted;
  const void* dout;
  void* dweight;
  float* part;        // [chunk][2][cols]: the run that enters a chunk, the run that leaves it
  uint32_t* joins;    // number of runs that cross a border, then the chunks in which they begin
  int64_t n, vocab, ds, ws;
  int32_t cols, tiles, chunks, zero_rows, team;  // threads of a chunk
  float scale;
  int32_t accumulate;
  ClearParams clear;
};

__device__ __forceinline__ uint32_t key_of(uint64_t e) { return uint32_t(e >> 32); }

// First place in the sorted tokens [lo, hi) whose id is at least `id`; whole warps, 32 probes at a time.
__device__ __forceinline__ int64_t lower_bound(const uint64_t* sorted, int64_t lo, int64_t hi, uint32_t id) {
  while (hi > lo) {
    const int64_t step = cdiv(hi - lo, 32), i = lo + int64_t(threadIdx.x & 31) * step;
    const int c = __popc(__ballot_sync(kFull, i < hi && key_of(sorted[i]) < id));
    if (step == 1 || c == 0) return lo + c;
    const int64_t first = lo;
    lo = first + int64_t(c - 1) * step + 1;
    hi = min(hi, first + int64_t(c) * step);
  }
  return lo;
}

// kAdd: to what the row has, `old`.
template <class O, bool kVec, bool kAdd>
__device__ __forceinline__ void write_row(O* to, float scale, int count, const float (&acc)[kElems], const Raw<O>& old) {
  float x[kElems];
#pragma unroll
  for (int e = 0; e < kElems; ++e) x[e] = __fmul_rn(acc[e], scale);
  if constexpr (kAdd) {
#pragma unroll
    for (int e = 0; e < kElems; ++e) x[e] = __fadd_rn(to_f32(old.v.v[e]), x[e]);
  }
  store_elems<O, kVec>(to, count, x);
}

// Zeros to the rows [r0, r1) that no token names.
__device__ __forceinline__ void clear_rows(const EmbedBwdParams& p, int64_t r0, int64_t r1, uint32_t* named, int* range) {
  const int rows = int(r1 - r0), warps = int(blockDim.x >> 5), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < (rows + 31) / 32; i += blockDim.x) named[i] = 0u;
  if (warp < 2) {  // one warp looks for the first token, one for the last
    const int64_t at = lower_bound(p.sorted, 0, p.n, uint32_t(warp == 0 ? r0 : r1));
    if (lane == 0) range[warp] = int(at);
  }
  __syncthreads();
  const int64_t lo = range[0], hi = range[1];
  if (hi - lo <= int64_t(rows) * 16) {
    for (int64_t i = lo + threadIdx.x; i < hi; i += blockDim.x) {
      const int r = int(key_of(p.sorted[i]) - uint32_t(r0));
      atomicOr(&named[r >> 5], 1u << (r & 31));
    }
  } else {  // long runs: look for the rows instead
    for (int r = warp; r < rows; r += warps) {
      const int64_t i = lower_bound(p.sorted, lo, hi, uint32_t(r0 + r));
      if (lane == 0 && i < hi && key_of(p.sorted[i]) == uint32_t(r0 + r)) atomicOr(&named[r >> 5], 1u << (r & 31));
    }
  }
  __syncthreads();
  const int lanes = row_lanes(p.clear.bytes);
  for (int r = int(threadIdx.x) / lanes; r < rows; r += int(blockDim.x) / lanes)
    if (!((named[r >> 5] >> (r & 31)) & 1u))
      clear_row(p.clear.table + (r0 + r) * p.clear.stride, p.clear.bytes, int(threadIdx.x) % lanes, lanes);
}

// kAdd: the sums are added to the table's rows, which are loaded with those of the tokens (28 tokens into 118528 x 64
// bf16: 21.6 us, 16384 into 151936 x 4096 fp32 124; loaded one by one as their sums end, 24 and 136).
template <class T, class O, bool kVec, bool kAdd>
__global__ void __launch_bounds__(256, kAdd || !kVec ? 2 : 3) embed_sum_kernel(EmbedBwdParams p) {
  __shared__ uint32_t named[kZeroRows / 32];
  __shared__ uint32_t all_keys[kMostTeams][2 * kChunk + 2];
  __shared__ uint32_t all_tokens[kMostTeams][2 * kChunk];
  __shared__ int ranges[kMostTeams][4];
  griddep_wait();  // the tokens are sorted
  griddep_release();
  const int teams = int(blockDim.x) / p.team;
  const int64_t sums = cdiv(p.chunks, teams) * p.tiles;
  if (int64_t(blockIdx.x) >= sums) {
    const int64_t r0 = (int64_t(blockIdx.x) - sums) * p.zero_rows;
    clear_rows(p, r0, min(p.clear.end, r0 + p.zero_rows), named, ranges[0]);
    return;
  }
  const int team = int(threadIdx.x) / p.team, t = int(threadIdx.x) % p.team;
  uint32_t* keys = all_keys[team];
  uint32_t* tokens = all_tokens[team];
  int* range = ranges[team];
  const int tile = int(blockIdx.x % unsigned(p.tiles));
  const int chunk = int(blockIdx.x / unsigned(p.tiles)) * teams + team;  // behind the last one: no tokens
  const int64_t begin = int64_t(chunk) * kChunk;
  int count;
  const int at = first_col<kVec>(tile, t, p.team, p.cols, count);
  const T* dout = static_cast<const T*>(p.dout) + at;
  O* dweight = static_cast<O*>(p.dweight) + at;
  if (t < 32) {
    // keys[1 + j] is the chunk's j-th, those of the next one behind them; before and after them, their neighbours
    const int lane = t;
    auto entry = [&](int64_t i) { return i >= 0 && i < p.n ? p.sorted[i] : ~0ull; };
    const uint64_t e0 = entry(begin + lane), e1 = entry(begin + kChunk + lane);
    const uint32_t k0 = key_of(e0), k1 = key_of(e1);
    // lane 0: before the chunk, 1: behind the two, 2: the chunk before's first, 3: before that
    const uint32_t other = lane < 4 ? key_of(entry(lane == 0 ? begin - 1 : lane == 1 ? begin + 2 * kChunk
                                                  : lane == 2 ? begin - kChunk : begin - kChunk - 1)) : 0u;
    const uint32_t before = __shfl_sync(kFull, other, 0), behind = __shfl_sync(kFull, other, 1);
    const uint32_t prior = __shfl_sync(kFull, other, 2), prior2 = __shfl_sync(kFull, other, 3);
    keys[1 + lane] = k0;
    keys[1 + kChunk + lane] = k1;
    tokens[lane] = uint32_t(e0);
    tokens[kChunk + lane] = uint32_t(e1);
    if (lane == 0) keys[0] = before;
    if (lane == 1) keys[2 * kChunk + 1] = behind;
    // The run that enters: how far it goes here, and whether it began in the chunk before and ends
    // here (its block's then).  The one that leaves: how far it goes into the next chunk, and
    // whether it ends there (this block's then).
    const uint32_t first = __shfl_sync(kFull, k0, 0), last = __shfl_sync(kFull, k0, 31);
    const uint32_t m0 = ~__ballot_sync(kFull, k0 == first), m1 = ~__ballot_sync(kFull, k1 == last);
    const int head = m0 ? __ffs(m0) - 1 : 32, ahead = m1 ? __ffs(m1) - 1 : 32;
    const uint32_t next = __shfl_sync(kFull, k1, 0);
    if (lane == 0) {
      const bool enters = before == first;
      const bool ends_here = head < 32 || next != first;
      const bool began = prior != first || prior2 != first;
      const bool skips = enters && ends_here && began;
      const bool leaves = next == last && !(enters && head == 32);
      const bool ends_next = ahead < 32 || behind != last;
      range[0] = skips ? head : 0;
      range[1] = kChunk + (leaves && ends_next ? ahead : 0);
      range[2] = enters && !skips ? head - 1 : -1;       // the entering run's last token, if its part is formed here
      range[3] = leaves && !ends_next ? kChunk - 1 : -1;  // the leaving run's
    }
  }
  __syncthreads();
  const uint32_t none = uint32_t(p.vocab);  // the key of tokens without a gradient; those behind the last are above it
  const int end = range[1], enters = range[2], leaves = range[3];
  float* part = p.part + int64_t(chunk) * 2 * p.cols;
  // rows under way at once; single elements take more registers for them (20011 x 1283 fp32: 47 us, with four rows 49)
  constexpr int kAhead = kVec || kAdd ? 4 : 8;
  float acc[kElems];
#pragma unroll
  for (int e = 0; e < kElems; ++e) acc[e] = 0.f;
  for (int j0 = range[0]; j0 < end; j0 += kAhead) {
    if (keys[1 + j0] >= none) break;
    Raw<T> r[kAhead];
    Raw<O> old[kAdd ? kAhead : 1];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u;
      if (j >= end || keys[1 + j] >= none) break;
      load_elems<T, kVec>(dout + int64_t(tokens[j]) * p.ds, count, r[u]);
      if constexpr (kAdd)
        if ((keys[2 + j] != keys[1 + j] || j + 1 == end) && j != enters && j != leaves)
          load_elems<O, kVec>(dweight + int64_t(keys[1 + j]) * p.ws, count, old[u]);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u;
      if (j >= end) break;
      const uint32_t key = keys[1 + j];
      if (key >= none) break;
#pragma unroll
      for (int e = 0; e < kElems; ++e) acc[e] += to_f32(r[u].v.v[e]);
      if (keys[2 + j] == key && j + 1 < end) continue;
      // the run ends here, or what this block has of it
      if (j == enters || j == leaves) {
        const bool out = j != enters;
        store_elems<float, kVec>(part + (out ? p.cols : 0) + at, count, acc);
        if (out && tile == 0 && t == 0) p.joins[1 + atomicAdd(p.joins, 1u)] = uint32_t(chunk);
      } else {
        write_row<O, kVec, kAdd>(dweight + int64_t(key) * p.ws, p.scale, count, acc, old[kAdd ? u : 0]);
      }
#pragma unroll
      for (int e = 0; e < kElems; ++e) acc[e] = 0.f;
    }
  }
}

// Runs of more than two chunks: the part of the chunk in which the run begins
// and those of the chunks that it enters.  kJoinWarps warps take every kJoinWarps-th
// part each, for 32 columns; their sums are added in order.
constexpr int kJoinWarps = 8;
template <class O>
__global__ void __launch_bounds__(kJoinWarps * 32) embed_join_kernel(EmbedBwdParams p) {
  __shared__ float buf[kJoinWarps][32];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tiles = (p.cols + 31) / 32;
  const int64_t work = int64_t(*p.joins) * tiles;
  for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
    const int chunk = int(p.joins[1 + w / tiles]), c = int(w % tiles) * 32 + lane;
    const uint32_t id = key_of(p.sorted[(int64_t(chunk) + 1) * kChunk - 1]);
    int parts = 1;  // the chunks that begin with the id, from the next one on
    for (uint32_t m = kFull; m == kFull;) {
      const int64_t i = (int64_t(chunk) + parts + lane) * kChunk;
      m = __ballot_sync(kFull, i < p.n && key_of(p.sorted[i]) == id);
      parts += m == kFull ? 32 : __ffs(~m) - 1;
    }
    float s = 0.f;
    if (c < p.cols) {
#pragma unroll 8
      for (int i = warp; i < parts; i += kJoinWarps) s += p.part[(int64_t(chunk + i) * 2 + (i == 0)) * p.cols + c];
    }
    buf[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < p.cols) {
#pragma unroll
      for (int i = 1; i < kJoinWarps; ++i) s += buf[i][lane];
      O* to = static_cast<O*>(p.dweight) + int64_t(id) * p.ws + c;
      s = __fmul_rn(s, p.scale);
      *to = from_f32<O>(p.accumulate ? __fadd_rn(to_f32(*to), s) : s);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
int validate(const flce_embedding_problem* p) {
  if (!p) return FLCE_ERR_INVALID_ARG;
  if (p->tokens < 0 || p->tokens > kMaxTokens || p->vocab < 1 || p->vocab >= INT32_MAX || p->cols < 1 ||
      p->cols > kMaxWidth || p->weight_stride < 0 || p->out_stride < 0)
    return FLCE_ERR_INVALID_ARG;
  if (!known_dtype(p->weight_dtype) || !known_dtype(p->out_dtype)) return FLCE_ERR_UNSUPPORTED_DTYPE;
  if (p->out_dtype != p->weight_dtype && p->out_dtype != FLCE_F32) return FLCE_ERR_DTYPE_MISMATCH;
  if (!std::isfinite(p->scale)) return FLCE_ERR_INVALID_ARG;
  return FLCE_OK;
}

// Threads of a block whose threads hold kElems columns each (kWide where these are apart).
int row_threads(int64_t cols, bool vec) { return vec ? int(std::min<int64_t>(256, cdiv(cdiv(cols, kElems), 32) * 32)) : kWide; }

// Whether all rows start on a boundary of kElems elements, so that vectors do.
bool whole_vectors(int64_t cols, const void* p, int64_t stride, const void* q, int64_t stride2) {
  return cols % kElems == 0 && aligned_to(p, 16) && aligned_to(q, 16) && stride % kElems == 0 && stride2 % kElems == 0;
}

struct BwdLayout {
  size_t a, b, joins, part, bytes;
};
BwdLayout bwd_layout(const flce_embedding_problem* p) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t n = size_t(p->tokens), chunks = size_t(cdiv(p->tokens, kChunk));
  BwdLayout l;
  l.a = 0;
  l.b = up(n * 8);
  l.joins = l.b + up(n * 8);
  l.part = l.joins + up((chunks + 1) * 4);
  l.bytes = l.part + up(chunks * 2 * size_t(p->cols) * 4);
  return l;
}

template <class T, class O, bool kVec>
cudaError_t launch_embed(EmbedParams& q, cudaStream_t st) {
  const int threads = row_threads(q.cols, kVec);
  q.tiles = int32_t(cdiv(q.cols, int64_t(threads) * kElems));
  // Two rows at once where that leaves enough blocks for every SM: 16384 x 4096 bf16 to fp32 63 us (the
  // copy rate gives 58); one at once 65, four 73, eight 97.
  if (cdiv(q.tokens, 2) * q.tiles >= 1024) {
    embed_kernel<T, O, kVec, 2><<<unsigned(cdiv(q.tokens, 2) * q.tiles), threads, 0, st>>>(q);
  } else {
    embed_kernel<T, O, kVec, 1><<<unsigned(q.tokens * q.tiles), threads, 0, st>>>(q);
  }
  return cudaGetLastError();
}
template <class T, class O>
cudaError_t launch_embed(EmbedParams& q, cudaStream_t st) {
  return whole_vectors(q.cols, q.weight, q.ws, q.out, q.os) ? launch_embed<T, O, true>(q, st)
                                                            : launch_embed<T, O, false>(q, st);
}

cudaError_t launch_sort(const SortParams& s, int num_sms, cudaStream_t st) {
  const int radix = 1 << s.width;
  const size_t smem = size_t(kSortWarps + 2) * radix * 4;
  cudaError_t e = cudaFuncSetAttribute(sort_tokens_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (kSortWarps + 2) * (1 << kMaxDigit) * 4);
  if (e != cudaSuccess) return e;
  const unsigned ctas = unsigned(s.ctas), clears = s.clear.end > s.clear.first ? (unsigned(num_sms) - ctas) / ctas * ctas : 0u;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas + clears);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sort_tokens_kernel, s);
}

template <class T, class O, bool kVec>
cudaError_t launch_sum(EmbedBwdParams& q, cudaStream_t st) {
  const int threads = row_threads(q.cols, kVec);
  q.tiles = int32_t(cdiv(q.cols, int64_t(threads) * kElems));
  // blocks of 160 threads or more: narrow rows have several chunks in one
  const int teams = 256 / threads;
  q.team = threads;
  const int64_t clear = cdiv(q.clear.end, q.zero_rows);
  const unsigned grid = unsigned(cdiv(q.chunks, teams) * q.tiles + clear);
  if (grid == 0) return cudaSuccess;  // no tokens, and all is cleared
  return q.accumulate ? launch_dependent(embed_sum_kernel<T, O, kVec, true>, grid, teams * threads, st, q)
                      : launch_dependent(embed_sum_kernel<T, O, kVec, false>, grid, teams * threads, st, q);
}
template <class T, class O>
cudaError_t launch_sum(EmbedBwdParams& q, cudaStream_t st) {
  return whole_vectors(q.cols, q.dout, q.ds, q.dweight, q.ws) ? launch_sum<T, O, true>(q, st)
                                                              : launch_sum<T, O, false>(q, st);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_embedding(const flce_embedding_problem* problem, const void* ids, const void* weight, void* out,
                   flce_stream_t stream) {
  const flce_embedding_problem* p = problem;
  FLCE_TRY(validate(p));
  if (p->tokens == 0) return FLCE_OK;
  if (!ids || !weight || !out || (p->tokens > 1 && p->out_stride < p->cols)) return FLCE_ERR_INVALID_ARG;
  if (!aligned_to(ids, p->ids_i64 ? 8 : 4) || !aligned_to(weight, elem_size(p->weight_dtype)) ||
      !aligned_to(out, elem_size(p->out_dtype)))
    return FLCE_ERR_MISALIGNED;
  if (p->tokens * cdiv(p->cols, 32 * kElems) > INT32_MAX) return FLCE_ERR_INVALID_ARG;
  DeviceInfo dev;
  FLCE_TRY(get_device(&dev));
  FLCE_TRY(check_local(dev, ids, weight, out));
  EmbedParams q{};
  q.ids = ids;
  q.weight = weight;
  q.out = out;
  q.tokens = p->tokens;
  q.vocab = p->vocab;
  q.ws = p->weight_stride;
  q.os = p->out_stride;
  q.cols = int32_t(p->cols);
  q.ids_i64 = p->ids_i64;
  q.scale = p->scale;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return logged(FLCE_LAUNCH_OTHER, st, [&] {
    if (p->weight_dtype == FLCE_F32) return launch_embed<float, float>(q, st);
    if (p->weight_dtype == FLCE_BF16)
      return p->out_dtype == FLCE_F32 ? launch_embed<__nv_bfloat16, float>(q, st)
                                      : launch_embed<__nv_bfloat16, __nv_bfloat16>(q, st);
    return p->out_dtype == FLCE_F32 ? launch_embed<__half, float>(q, st) : launch_embed<__half, __half>(q, st);
  });
}

int flce_embedding_workspace_size(const flce_embedding_problem* problem, size_t* bytes) {
  if (!bytes) return FLCE_ERR_INVALID_ARG;
  FLCE_TRY(validate(problem));
  *bytes = bwd_layout(problem).bytes + 256;
  return FLCE_OK;
}

int flce_embedding_backward(const flce_embedding_problem* problem, const void* ids, const void* dout, void* dweight,
                            void* workspace, size_t workspace_bytes, flce_stream_t stream) {
  const flce_embedding_problem* p = problem;
  size_t need = 0;
  FLCE_TRY(flce_embedding_workspace_size(p, &need));
  if (p->weight_stride < p->cols && p->vocab > 1) return FLCE_ERR_INVALID_ARG;
  if (p->tokens == 0 && p->accumulate) return FLCE_OK;
  if ((p->tokens > 0 && (!ids || !dout)) || !dweight || !workspace) return FLCE_ERR_INVALID_ARG;
  if (!aligned_to(ids, p->ids_i64 ? 8 : 4) || !aligned_to(dout, elem_size(p->out_dtype)) ||
      !aligned_to(dweight, elem_size(p->weight_dtype)) || !aligned_to(workspace, 16))
    return FLCE_ERR_MISALIGNED;
  if (workspace_bytes < need) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  if (cdiv(p->tokens, kChunk) * cdiv(p->cols, 32 * kElems) + p->vocab > INT32_MAX) return FLCE_ERR_INVALID_ARG;
  DeviceInfo dev;
  FLCE_TRY(get_device(&dev));
  FLCE_TRY(check_local(dev, ids, dout, dweight, workspace));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const BwdLayout l = bwd_layout(p);
  SortParams s{};
  s.ids = ids;
  s.a = reinterpret_cast<uint64_t*>(ws + l.a);
  s.b = reinterpret_cast<uint64_t*>(ws + l.b);
  s.joins = reinterpret_cast<uint32_t*>(ws + l.joins);
  s.n = p->tokens;
  s.vocab = p->vocab;
  s.padding = p->padding;
  s.ids_i64 = p->ids_i64;
  int bits = 1;  // of the largest key, vocab
  while ((p->vocab >> bits) != 0) ++bits;
  s.passes = int32_t(cdiv(bits, kMaxDigit));
  s.width = int32_t(cdiv(bits, s.passes));
  s.ctas = p->tokens <= kSortOne ? 1 : kSortCtas;
  // rows that are cleared while the tokens are sorted, from the end (frequent tokens have small numbers, mostly)
  ClearParams& early = s.clear;
  early.table = static_cast<uint8_t*>(dweight);
  early.bytes = p->cols * int64_t(elem_size(p->weight_dtype));
  early.stride = p->weight_stride * int64_t(elem_size(p->weight_dtype));
  early.end = p->accumulate ? 0 : p->vocab;
  early.first = std::max<int64_t>(0, early.end - (s.ctas == 1 ? kEarlyOne : kEarly) / early.bytes);
  FLCE_TRY(logged(FLCE_LAUNCH_OTHER, st, [&] { return launch_sort(s, dev.num_sms, st); }));
  EmbedBwdParams q{};
  q.sorted = s.passes % 2 ? s.a : s.b;
  q.dout = dout;
  q.dweight = dweight;
  q.part = reinterpret_cast<float*>(ws + l.part);
  q.joins = s.joins;
  q.n = p->tokens;
  q.vocab = p->vocab;
  q.ds = p->out_stride;
  q.ws = p->weight_stride;
  q.cols = int32_t(p->cols);
  q.chunks = int32_t(cdiv(p->tokens, kChunk));
  // three blocks to an SM clear the rest, if that makes enough for each and not too much
  q.clear = early;
  q.clear.first = 0;
  q.clear.end = early.first;
  const int64_t clear = std::clamp<int64_t>(q.clear.end * early.bytes / (int64_t(dev.num_sms) * 3), kZeroLeast, kZeroBytes);
  q.zero_rows = int32_t(std::clamp<int64_t>(clear / early.bytes, 1, kZeroRows));
  q.scale = p->scale;
  q.accumulate = p->accumulate;
  FLCE_TRY(logged(FLCE_LAUNCH_OTHER, st, [&] {
    if (p->weight_dtype == FLCE_F32) return launch_sum<float, float>(q, st);
    if (p->weight_dtype == FLCE_BF16)
      return p->out_dtype == FLCE_F32 ? launch_sum<float, __nv_bfloat16>(q, st)
                                      : launch_sum<__nv_bfloat16, __nv_bfloat16>(q, st);
    return p->out_dtype == FLCE_F32 ? launch_sum<float, __half>(q, st) : launch_sum<__half, __half>(q, st);
  }));
  if (q.chunks < 3) return FLCE_OK;  // no run of more than two
  const unsigned grid = unsigned(std::min<int64_t>(int64_t(q.chunks / 3 + 1) * cdiv(q.cols, 32), int64_t(dev.num_sms) * 8));
  return logged(FLCE_LAUNCH_OTHER, st, [&] {
    if (p->weight_dtype == FLCE_F32) return launch_dependent(embed_join_kernel<float>, grid, kJoinWarps * 32, st, q);
    if (p->weight_dtype == FLCE_BF16)
      return launch_dependent(embed_join_kernel<__nv_bfloat16>, grid, kJoinWarps * 32, st, q);
    return launch_dependent(embed_join_kernel<__half>, grid, kJoinWarps * 32, st, q);
  });
}

}  // extern "C"
