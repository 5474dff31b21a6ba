// flce_norm.cuh — residual addition + root-mean-square norm: what its forward
// (flce_norm_fwd.cu, flce_norm_fp8*.cu) and backward (flce_norm_bwd.cu) share.
//
//   h = rn(x + r),  rstd = (mean h^2 + eps)^(-1/2),  y_j = h_j rstd (w_j + o)
//   d_j = rstd (g_j - n_j c) + dh_j  with g_j = dy_j (w_j + o), n_j = h_j rstd,
//   c = mean_j g_j n_j;  dw_j = sum over rows of dy_j n_j
//
// Every element is used once per row, so the bound is memory: the forward reads
// x and r and writes h and y, the backward reads dy, h and dh and writes d.  A
// row is read once and stays in registers between its reduction and its output.
// The rows after it are already being copied into shared memory, each thread's
// own vectors into its own slots (cp.async), so that the bytes under way cost no
// registers and need no barrier (next row in registers instead: 217 us, for too
// few threads fit; three rows ahead: no faster than two).  With that the issue
// slots are the next limit (two thirds busy in the forward), so the arithmetic runs on
// pairs of fp32 lanes (backward 118 -> 94 us), and the weights wait in shared
// memory as fp32 with their offset added.  (Times: 16384 x 4096 bf16.)
//
// Rows need not start on 16-byte boundaries.  A row whose first element is
// `shift` elements past one is laid over threads `shift` places late, so that
// all its vectors but the first and the last are 16 aligned bytes (4099 x 1283
// bf16 with an fp32 residual, backward: 22 us; as single elements 74).  A block (or warp) takes rows a
// multiple of the vector's width apart, which all have the same shift: a thread's
// columns, its weights and its dweight sums are the same for all its rows.
#pragma once

#include <algorithm>
#include <type_traits>

#include "flce_device.cuh"
#include "flce_elem.cuh"

namespace flce {

constexpr int64_t kMaxCols = 131072;
constexpr int kWarpRowBlock = 256;    // threads of a block that gives each warp a row
constexpr int kMaxThreads = 1024;
constexpr int kLoopThreads = 1024;    // rows too wide for registers
constexpr float kE4m3Max = 448.0f;

// Elements of a vector: 16 bytes of the wider of the call's two types, so that
// neighbouring threads' accesses leave no gaps.  (With 8 elements for a 16-bit x
// and an fp32 residual, 32 bytes per thread in two accesses, half of every sector
// asked for was unused.)
inline int vec_of(size_t elem, size_t residual_elem) { return int(16 / std::max(elem, residual_elem)); }
template <class T, class R>
constexpr int kVecOf = 16 / (sizeof(T) > sizeof(R) ? sizeof(T) : sizeof(R));

// How a row is laid over threads, 16 elements per thread at most.
enum RowForm {
  kWarp,    // a warp per row, kWarpRowBlock threads
  kBlock,   // a block of up to 256 threads per row
  kWide,    // a block of up to 512
  kBig,     // a block of up to 1024
  kLoop     // too wide for registers
};
constexpr int row_threads(RowForm form) {
  return form == kWarp || form == kBlock ? kWarpRowBlock : form == kWide ? 512 : kMaxThreads;
}
// Blocks of that many threads on an SM that the registers are shared out for;
// `elems` is what a thread holds of a row.
constexpr int fwd_blocks(RowForm form, bool ragged) {
  return form == kBig || (form == kWide && ragged) ? 1 : form == kWide || ragged ? 2 : 4;
}
constexpr int bwd_blocks(RowForm form, bool ragged, int elems) {
  return form == kBig || form == kWide ? 1 : ragged && elems > 8 ? 2 : 3;
}
constexpr int kRowStages = 2;  // rows under way per block (or warp)
// Single elements are too small to copy; a big row's slots would not fit.
__host__ __device__ constexpr bool copies(RowForm form, int vec) { return vec > 1 && form != kBig; }

struct NormParams {
  const void* x;
  const void* r;
  const void* w;
  void* h;
  void* y;       // y, or the 8-bit q
  float* rstd;
  float* scale;  // 8-bit output
  int64_t rows, xs, rs, hs, ys;
  int32_t cols, w_dtype;
  int32_t group, groups;  // 8-bit output: columns per scale, scales per row
  int32_t lanes;          // lanes whose vectors make up a group, 0 where that is not so
  int32_t slots_at;       // bytes of dynamic shared memory before the weights
  float eps, offset;
};

// w_j + o; without weights 1 + o.
__device__ __forceinline__ float load_weight(const void* w, int dtype, float offset, int col) {
  return (w ? load_as(w, dtype, col) : 1.0f) + offset;
}

// V values in fp32, in pairs (V = 1: the other lane is 0).
template <int V>
struct Floats {
  static constexpr int kPairs = (V + 1) / 2;
  uint64_t p[kPairs];
};
template <class E, int V>
__device__ __forceinline__ Floats<V> widen(const Vec<E, V>& x) {
  Floats<V> f;
#pragma unroll
  for (int j = 0; j < f.kPairs; ++j) f.p[j] = f2_pack(to_f32(x.v[2 * j]), V == 1 ? 0.f : to_f32(x.v[V == 1 ? 0 : 2 * j + 1]));
  return f;
}
__device__ __forceinline__ void narrow2(float lo, float hi, float* out) { out[0] = lo, out[1] = hi; }
__device__ __forceinline__ void narrow2(float lo, float hi, __nv_bfloat16* out) {
  *reinterpret_cast<__nv_bfloat162*>(out) = __floats2bfloat162_rn(lo, hi);
}
__device__ __forceinline__ void narrow2(float lo, float hi, __half* out) {
  *reinterpret_cast<__half2*>(out) = __floats2half2_rn(lo, hi);
}
template <class E, int V>
__device__ __forceinline__ Vec<E, V> narrow(const Floats<V>& f) {
  Vec<E, V> x;
#pragma unroll
  for (int j = 0; j < f.kPairs; ++j) {
    float lo, hi;
    f2_unpack(f.p[j], lo, hi);
    if constexpr (V == 1) {
      x.v[0] = from_f32<E>(lo);
    } else {
      narrow2(lo, hi, &x.v[2 * j]);
    }
  }
  return x;
}
__device__ __forceinline__ float pair_sum(uint64_t p) {
  float lo, hi;
  f2_unpack(p, lo, hi);
  return lo + hi;
}

template <int kBytes>
__device__ __forceinline__ void cp_async(void* dst_smem, const void* src) {
  if constexpr (kBytes == 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst_smem)), "l"(src) : "memory");
  } else {
    static_assert(kBytes == 8 || kBytes == 4, "cp.async takes 4, 8 or 16 bytes");
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst_smem)), "l"(src), "n"(kBytes)
                 : "memory");
  }
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits for all but the last n committed groups of this thread.
template <int n>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory"); }

// The vectors a thread holds of a row: vector i is places (t + i * width) * V,
// columns `shift` lower.
// kRagged: rows may be shifted or end inside a vector.
template <int V, int NV, bool kRagged>
struct RowVectors {
  int first, width, cols, thread;  // first column of vector 0 (may be negative)
  __device__ __forceinline__ int col(int i) const { return first + i * width; }
  __device__ __forceinline__ bool whole(int i) const {
    return kRagged ? col(i) >= 0 && col(i) + V <= cols : col(i) < cols;
  }
  __device__ __forceinline__ bool has(int i, int k) const {
    return kRagged ? col(i) + k >= 0 && col(i) + k < cols : col(i) < cols;
  }

  // What is copied at once of a vector of type E: 16 bytes, or less.
  template <class E>
  static __host__ __device__ constexpr int word_of() {
    return V * sizeof(E) < 16 ? int(V * sizeof(E)) : 16;
  }
  // Bytes of one row's vectors of type E, all threads'.
  template <class E>
  __device__ __forceinline__ int bytes() const { return NV * width * int(sizeof(E)); }

  // Starts copying the thread's whole vectors of a row into its slots.
  template <class E>
  __device__ __forceinline__ void fetch(const E* row, uint8_t* slots) const {
    if constexpr (V > 1) {
      constexpr int kWord = word_of<E>(), kWords = V * sizeof(E) / kWord;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (whole(i))
#pragma unroll
          for (int c = 0; c < kWords; ++c)
            cp_async<kWord>(slot<kWord>(slots, i * kWords + c),
                            reinterpret_cast<const uint8_t*>(row + col(i)) + c * kWord);
    }
  }
  // The vectors that fetch() brought, once its copies have arrived; of the
  // others, a row's ragged ends, `edge` holds the elements.
  template <class E>
  __device__ __forceinline__ Vec<E, V> read(uint8_t* slots, int i, const Vec<E, V> (&edge)[NV]) const {
    if (!whole(i)) return edge[i];
    constexpr int kWord = word_of<E>(), kWords = V * sizeof(E) / kWord;
    using Word = Vec<uint32_t, kWord / 4>;
    Vec<E, V> x;
#pragma unroll
    for (int c = 0; c < kWords; ++c)
      reinterpret_cast<Word*>(&x)[c] = *reinterpret_cast<const Word*>(slot<kWord>(slots, i * kWords + c));
    return x;
  }
  // A row's ragged ends, by element; 0 outside the row.
  template <class E>
  __device__ __forceinline__ void edges(const E* row, Vec<E, V> (&out)[NV]) const {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (!whole(i))
#pragma unroll
        for (int k = 0; k < V; ++k) out[i].v[k] = kRagged && has(i, k) ? row[col(i) + k] : from_f32<E>(0.f);
  }
  // Plain loads of a row, where nothing is copied ahead.
  template <class E>
  __device__ __forceinline__ void load(const E* row, Vec<E, V> (&out)[NV]) const {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (whole(i)) out[i] = load_vec<E, V>(row + col(i));
    edges(row, out);
  }
  template <class E>
  __device__ __forceinline__ void store(E* row, int i, const Vec<E, V>& x) const {
    if (whole(i)) {
      store_vec<E, V>(row + col(i), x);
    } else if (kRagged) {
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (has(i, k)) row[col(i) + k] = x.v[k];
    }
  }
  template <int kWord>
  __device__ __forceinline__ uint8_t* slot(uint8_t* slots, int word) const {
    return slots + (word * (width / V) + thread) * kWord;
  }
  // The thread's weights, offset added, into its slots of a region of
  // bytes<float>(); then vector i's.
  __device__ __forceinline__ void keep_weights(const void* w, int dtype, float offset, uint8_t* slots) const {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k)
        *weight_at(slots, i, k) = has(i, k) ? load_weight(w, dtype, offset, col(i) + k) : 0.f;
  }
  __device__ __forceinline__ float* weight_at(uint8_t* slots, int i, int k) const {
    if constexpr (V == 1) return reinterpret_cast<float*>(slots) + i * width + thread;
    return reinterpret_cast<float*>(slot<16>(slots, i * (V / 4) + k / 4)) + k % 4;
  }
  // Vector i of such a region, for sums.
  __device__ __forceinline__ void put(uint8_t* slots, int i, const Floats<V>& f) const {
    if constexpr (V == 1) {
      float lo, hi;
      f2_unpack(f.p[0], lo, hi);
      *weight_at(slots, i, 0) = lo;
    } else {
#pragma unroll
      for (int c = 0; c < V / 4; ++c) {
        ulonglong2 two = {f.p[2 * c], f.p[2 * c + 1]};
        *reinterpret_cast<ulonglong2*>(slot<16>(slots, i * (V / 4) + c)) = two;
      }
    }
  }
  __device__ __forceinline__ Floats<V> weight(uint8_t* slots, int i) const {
    Vec<float, V> x;
    if constexpr (V == 1) {
      x.v[0] = *weight_at(slots, i, 0);
    } else {
#pragma unroll
      for (int c = 0; c < V / 4; ++c)
        reinterpret_cast<uint4*>(&x)[c] = *reinterpret_cast<const uint4*>(slot<16>(slots, i * (V / 4) + c));
    }
    return widen(x);
  }
};

struct NormBwdParams {
  const void* dy;
  const void* h;
  const void* w;
  const float* rstd;
  const void* dh;
  void* dx;
  void* dr;
  float* part;   // [blocks][cols] partial dweight, or nullptr
  int64_t rows, dys, hs, dhs, dxs, drs;
  int32_t cols, w_dtype;
  float offset;
};

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// A row's layout: vectors of `vec` elements (1 where the call's rows do not all
// have the same shift), `nv` of them per thread.
struct RowPlan {
  RowForm form;
  bool ragged;
  int vec, nv, threads;
};
inline RowPlan plan_row(int64_t cols, int vec, bool shifted) {
  const bool ragged = vec > 1 && (shifted || cols % vec != 0);
  const int64_t vecs = (cols + (shifted ? vec - 1 : 0) + vec - 1) / vec;
  const int most = 16 / vec;  // vectors of 16 elements
  const int warp_nv = std::min(most, 4);
  if (vecs <= 32 * warp_nv) return {kWarp, ragged, vec, warp_nv, kWarpRowBlock};
  // 16 elements per thread, or 8 where a ragged row fits 256 threads that way
  // (its weights take registers) or singles do
  const int nv = vec == 1 || (ragged && vecs <= 256 * (most / 2)) ? most / 2 : most;
  const int64_t threads = ((vecs + nv - 1) / nv + 31) / 32 * 32;
  if (threads <= row_threads(kBlock)) return {kBlock, ragged, vec, nv, int(threads)};
  if (threads <= row_threads(kWide)) return {kWide, ragged, vec, nv, int(threads)};
  const int64_t big = ((vecs + most - 1) / most + 31) / 32 * 32;
  if (big <= row_threads(kBig)) return {kBig, ragged, vec, most, int(big)};
  return {kLoop, false, vec, 0, kLoopThreads};
}

// Dynamic shared memory of a row kernel: weights, and the slots of rows of
// `row_bytes` per element.
inline int row_smem(const RowPlan& pl, size_t row_bytes) {
  const size_t elems = size_t(pl.threads) * pl.nv * pl.vec;
  return int(elems * 4 + (copies(pl.form, pl.vec) ? kRowStages * elems * row_bytes : 0));
}

// The kernel of a plan: make(vectors per thread, form, ragged).
template <int V, class F>
auto pick_form(const RowPlan& pl, F&& make) {
  constexpr int kMost = 16 / V, kHalf = kMost / 2 > 0 ? kMost / 2 : 1, kWarpNv = kMost < 4 ? kMost : 4;
  auto of = [&](auto ragged) {
    using Form = RowForm;
    if (pl.form == kWarp) return make(std::integral_constant<int, kWarpNv>(), std::integral_constant<Form, kWarp>(), ragged);
    if (pl.form == kBig) return make(std::integral_constant<int, kMost>(), std::integral_constant<Form, kBig>(), ragged);
    if constexpr (V == 1 || decltype(ragged)::value) {
      if (pl.nv == kHalf && pl.form == kBlock)
        return make(std::integral_constant<int, kHalf>(), std::integral_constant<Form, kBlock>(), ragged);
    }
    if constexpr (V == 1) {
      return make(std::integral_constant<int, kHalf>(), std::integral_constant<Form, kWide>(), ragged);
    } else {
      if (pl.form == kBlock) return make(std::integral_constant<int, kMost>(), std::integral_constant<Form, kBlock>(), ragged);
      return make(std::integral_constant<int, kMost>(), std::integral_constant<Form, kWide>(), ragged);
    }
  };
  if constexpr (V > 1) {
    if (pl.ragged) return of(std::true_type());
  }
  return of(std::false_type());
}

cudaError_t launch_norm_fwd(const NormParams& p, int32_t dt, int32_t rdt, const RowPlan& pl, int grid, cudaStream_t st);
cudaError_t launch_norm_fwd_fp8_exact(const NormParams& p, int32_t dt, int32_t rdt, const RowPlan& pl, int grid, cudaStream_t st);
cudaError_t launch_norm_fwd_fp8_left(const NormParams& p, int32_t dt, int32_t rdt, const RowPlan& pl, int grid, cudaStream_t st);
cudaError_t launch_norm_bwd(const NormBwdParams& p, int32_t dt, int32_t rdt, const RowPlan& pl, int blocks, cudaStream_t st);

}  // namespace flce
