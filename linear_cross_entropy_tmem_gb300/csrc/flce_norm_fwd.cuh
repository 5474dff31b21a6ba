// flce_norm_fwd.cuh — forward kernels of the norm, with (kFp8) and without an
// 8-bit output.
#pragma once

#include <cuda_fp8.h>

#include "flce_norm.cuh"

namespace flce {
namespace {

// The output: in the input's type, or in 8 bits from exact products or with what is left of them.
enum Output { kSameBits, kFp8Exact, kFp8Left };

// The 8-bit output.  In y_j / s = 448 (h_j w_j) / max |h w| the row's rstd cancels
// (w with its offset), so the quotient is formed from u = (h p) w, with p the power
// of two below rstd, which keeps u within a factor of two of y and rounds nothing.
// u itself is exact where h and the weights have 16 bits and no offset is added;
// else what its rounding left, lo, is carried along, and so the codes are those of
// the exact quotient.  (From y, rounded twice, about two codes in a million fell to
// the other side of a border.)
struct Rstd {
  float pow2, rest;  // rstd = pow2 * rest
};
__device__ __forceinline__ Rstd split(float rstd) {
  const uint32_t bits = __float_as_uint(rstd);
  if (rstd == 0.f || (bits & 0x7f800000u) == 0x7f800000u) return {rstd, 1.0f};  // 0, infinity, NaN
  return {__uint_as_float(bits & 0x7f800000u), __uint_as_float((bits & 0x007fffffu) | 0x3f800000u)};
}
// A group's scale, from the bits of its largest |u|.
__device__ __forceinline__ float scale_of(uint32_t top, float rest) { return __uint_as_float(top) * rest / kE4m3Max; }
// e4m3(448 u / top): t = u / top by the reciprocal, r = what that leaves of u, and
// 448 t + 448 r / top rounded once, which is the fp32 quotient.  Below 2^-100
// (where 1 / top may overflow) values take a factor of 2^64 first.
struct Inverse {
  float first, inv, inv448, minus, minus_lo;  // minus: -top, or 0 where the step would make NaN of 0
};
__device__ __forceinline__ Inverse inverse_of(uint32_t top_bits, float top_lo, float scale) {
  const float first = __uint_as_float(top_bits) < 0x1p-100f ? 0x1p64f : 1.0f, top = __uint_as_float(top_bits) * first;
  const float inv = scale == 0.f ? 0.f : __frcp_rn(top);  // scale 0: codes 0
  const bool finite = top < INFINITY;
  return {first, inv, inv * kE4m3Max, finite ? -top : 0.f, finite ? -top_lo * first : 0.f};
}
// Saturates; NaN stays NaN.
__device__ __forceinline__ uint8_t quantise(float u, float lo, const Inverse& i) {
  u *= i.first;
  const float t = u * i.inv;
  const float r = fmaf(t, i.minus, u) + fmaf(t, i.minus_lo, lo * i.first);
  return uint8_t(__nv_cvt_float_to_fp8(fmaf(t, kE4m3Max, r * i.inv448), __NV_SATFINITE, __NV_E4M3));
}
// What u = a w left, with u's sign taken off.
__device__ __forceinline__ float left_of(float a, float w, float u) { return fmaf(a, w, -u); }
__device__ __forceinline__ float outward(float lo, float u) {
  return __uint_as_float(__float_as_uint(lo) ^ (__float_as_uint(u) & 0x80000000u));
}
// Order-preserving bits, for the atomic maximum of values of either sign.
__device__ __forceinline__ int signed_bits(float x) {
  const int bits = __float_as_int(x);
  return bits >= 0 ? bits : bits ^ 0x7fffffff;
}
__device__ __forceinline__ float from_signed_bits(int key) { return __int_as_float(key >= 0 ? key : key ^ 0x7fffffff); }

// The largest of |a|, |b|, |c|, a NaN if any is one.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Order-preserving bits of |y|: a NaN is above infinity, so that a group with
// one gets a NaN scale.
__device__ __forceinline__ uint32_t abs_bits(float y) { return __float_as_uint(y) & 0x7fffffffu; }

// Rows go to warps (kWarpRow) or to blocks, in turn.  h is rounded to its type
// before its squares are summed, as the backward reads it rounded.
// 16384 x 4096 bf16 with residual: 81.6 us, 6.6 TB/s, what a copy reaches; one
// row of 4096: 3.4 us, a launch.  With the 8-bit output and groups of 128, 8192 x
// 2048 fp16 takes 27.4 us for 118 MB (4.3 TB/s): groups' maxima, the quotient and
// the conversion bring it to 40 instructions per element; 70 % of the issue slots are
// busy, and the rest is latency between a row's reduction and its output.
// Where what is left of the products is carried along, 16384 x 2048 bf16 with an
// fp32 residual takes 86 us (from rounded products 64).  Groups that no power of two
// of lanes makes up, and ragged rows, go through an atomic maximum per element: at
// 8192 x 2048 fp16 83 us with a scale per row, 61 with groups of 48; 4099 x 1283
// bf16 60.
template <class T, class R, int V, int NV, RowForm kForm, bool kRagged, Output kOut>
__global__ void __launch_bounds__(row_threads(kForm), fwd_blocks(kForm, kRagged)) norm_fwd_kernel(NormParams p) {
  constexpr bool kFp8 = kOut != kSameBits, kExact = kOut == kFp8Exact;
  constexpr bool kWarpRow = kForm == kWarp;
  constexpr bool kCopy = copies(kForm, V);  // rows are copied ahead
  // [rows of the block][groups] maxima, and again what is left of them (8-bit output); weights; slots
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red[2][32];
  const int t = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;
  const int width = kWarpRow ? 32 : blockDim.x;
  const int per_block = kWarpRow ? kWarpRowBlock / 32 : 1;
  const int unit = kWarpRow ? threadIdx.x >> 5 : 0;  // the row of the block
  const int64_t step = int64_t(gridDim.x) * per_block;
  int64_t row = blockIdx.x * int64_t(per_block) + unit;
  if (kWarpRow && row >= p.rows) return;
  const T* x = static_cast<const T*>(p.x) + row * p.xs;
  const R* r = static_cast<const R*>(p.r) + row * p.rs;
  const int shift = kRagged ? int((reinterpret_cast<uintptr_t>(x) / sizeof(T)) % V) : 0;
  const RowVectors<V, NV, kRagged> at = {t * V - shift, width * V, p.cols, t};
  const int row_bytes = at.template bytes<T>() + at.template bytes<R>();
  uint8_t* weights = smem + p.slots_at + unit * at.template bytes<float>();
  uint8_t* slots = smem + p.slots_at + per_block * at.template bytes<float>() + unit * kRowStages * row_bytes;
  Vec<T, V> xe[NV];  // ragged ends of the next row, or a whole row where nothing is copied ahead
  Vec<R, V> re[NV];
  auto fetch = [&](int64_t n, int stage) {  // row n, if there is one
    if (n < p.rows) {
      at.fetch(static_cast<const T*>(p.x) + n * p.xs, slots + stage * row_bytes);
      if (p.r) at.fetch(static_cast<const R*>(p.r) + n * p.rs, slots + stage * row_bytes + at.template bytes<T>());
    }
    cp_async_commit();
  };
  if constexpr (kCopy) {
#pragma unroll
    for (int k = 0; k < kRowStages; ++k) fetch(row + k * step, k);
    at.edges(x, xe);
    if (p.r) at.edges(r, re);
  }
  at.keep_weights(p.w, p.w_dtype, p.offset, weights);
  int group[NV];  // 8-bit output: each vector's
#pragma unroll
  for (int i = 0; i < NV; ++i) group[i] = kFp8 && !kRagged ? at.col(i) / p.group : 0;
  int turn = 0, stage = 0;
  for (; row < p.rows; row += step) {
    if constexpr (kCopy) {
      cp_async_wait<kRowStages - 1>();
    } else {
      at.load(x, xe);
      if (p.r) at.load(r, re);
    }
    Floats<V> v[NV];
    uint64_t squares = f2_splat(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Vec<T, V> xv = xe[i];
      if constexpr (kCopy) xv = at.read(slots + stage * row_bytes, i, xe);
      v[i] = widen(xv);
      if (p.r) {
        Vec<R, V> rv = re[i];
        if constexpr (kCopy) rv = at.read(slots + stage * row_bytes + at.template bytes<T>(), i, re);
        const Floats<V> f = widen(rv);
#pragma unroll
        for (int j = 0; j < f.kPairs; ++j) v[i].p[j] = f2_add(v[i].p[j], f.p[j]);
        const Vec<R, V> hv = narrow<R>(v[i]);
        v[i] = widen(hv);
        at.store(static_cast<R*>(p.h) + row * p.hs, i, hv);
      }
#pragma unroll
      for (int j = 0; j < v[i].kPairs; ++j) squares = f2_fma(v[i].p[j], v[i].p[j], squares);
    }
    x += step * p.xs;
    r += step * p.rs;
    if constexpr (kCopy) {
      fetch(row + kRowStages * step, stage);
      if (kRagged && row + step < p.rows) {
        at.edges(x, xe);
        if (p.r) at.edges(r, re);
      }
      stage = stage + 1 == kRowStages ? 0 : stage + 1;
    }
    const float ss = kWarpRow ? warp_sum(pair_sum(squares)) : block_sum(pair_sum(squares), red[turn]);
    turn ^= 1;
    const float rstd = rsqrtf(ss * (1.0f / float(p.cols)) + p.eps);
    if (t == 0 && p.rstd) p.rstd[row] = rstd;
    if constexpr (!kFp8) {
      const uint64_t rstd2 = f2_splat(rstd);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const Floats<V> w = at.weight(weights, i);
#pragma unroll
        for (int j = 0; j < w.kPairs; ++j) v[i].p[j] = f2_mul(f2_mul(v[i].p[j], rstd2), w.p[j]);
        at.store(static_cast<T*>(p.y) + row * p.ys, i, narrow<T>(v[i]));
      }
    }
    if constexpr (kFp8) {
      uint8_t* q = static_cast<uint8_t*>(p.y) + row * p.ys;
      float* scale = p.scale + row * p.groups;
      const Rstd rs = split(rstd);
      const uint64_t pow2 = f2_splat(rs.pow2);
      if (!kRagged && p.lanes) {  // a group is `lanes` neighbouring lanes' vectors of one i
        auto reduce = [&](uint32_t m) {
#pragma unroll
          for (int o = 1; o < 32; o <<= 1)
            if (o < p.lanes) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          return m;
        };
        // h p, u in its place or beside it, and the largest |u| of the vector
        auto product = [&](int i, const Floats<V>& w, Floats<V>& u) {
          float top = 0.f;
#pragma unroll
          for (int j = 0; j < w.kPairs; ++j) {
            v[i].p[j] = f2_mul(v[i].p[j], pow2);
            u.p[j] = f2_mul(v[i].p[j], w.p[j]);
            float f0, f1;
            f2_unpack(u.p[j], f0, f1);
            top = max_abs(top, f0, f1);
          }
          return abs_bits(top);
        };
        uint32_t most[NV];
        if constexpr (kExact) {
#pragma unroll
          for (int i = 0; i < NV; ++i) most[i] = reduce(product(i, at.weight(weights, i), v[i]));
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          Floats<V> u, lo;
          uint32_t m;
          float m_lo = 0.f;
          if constexpr (kExact) {
            u = v[i];
            m = most[i];
          } else {
            const Floats<V> w = at.weight(weights, i);
            const uint32_t own = product(i, w, u);
            m = reduce(own);
            const float top = __uint_as_float(m);
            float best = -INFINITY;  // of equal largest products what is left decides
#pragma unroll
            for (int j = 0; j < w.kPairs; ++j) {
              float a[2], b[2], f[2], l[2];
              f2_unpack(v[i].p[j], a[0], a[1]);
              f2_unpack(w.p[j], b[0], b[1]);
              f2_unpack(u.p[j], f[0], f[1]);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                l[k] = left_of(a[k], b[k], f[k]);
                if (fabsf(f[k]) == top) best = fmaxf(best, outward(l[k], f[k]));
              }
              lo.p[j] = f2_pack(l[0], l[1]);
            }
            // mostly one lane of the group has the largest
            const int lane = threadIdx.x & 31;
            const uint32_t in_group = (p.lanes == 32 ? 0xffffffffu : (1u << p.lanes) - 1) << (lane & ~(p.lanes - 1));
            const uint32_t have = __ballot_sync(0xffffffffu, own == m) & in_group;
            if (!__any_sync(0xffffffffu, have & (have - 1))) {
              m_lo = __shfl_sync(0xffffffffu, best, have ? __ffs(have) - 1 : lane);
            } else {
              m_lo = best;
#pragma unroll
              for (int o = 1; o < 32; o <<= 1)
                if (o < p.lanes) m_lo = fmaxf(m_lo, __shfl_xor_sync(0xffffffffu, m_lo, o));
            }
          }
          const float s = scale_of(m, rs.rest);
          const int col = at.col(i);
          if (col < p.cols) {
            if ((t & (p.lanes - 1)) == 0) scale[group[i]] = s;
            const Inverse inv = inverse_of(m, m_lo, s);
            if (inv.first != 1.0f) {
#pragma unroll
              for (int j = 0; j < u.kPairs; ++j) {
                u.p[j] = f2_mul(u.p[j], f2_splat(inv.first));
                if (!kExact) lo.p[j] = f2_mul(lo.p[j], f2_splat(inv.first));
              }
            }
            Vec<uint8_t, V> qv;
#pragma unroll
            for (int j = 0; j < u.kPairs; ++j) {
              const uint64_t quo = f2_mul(u.p[j], f2_splat(inv.inv));
              uint64_t left = f2_fma(quo, f2_splat(inv.minus), u.p[j]);
              if (!kExact) left = f2_add(f2_fma(quo, f2_splat(inv.minus_lo), left), lo.p[j]);
              float2 y;
              f2_unpack(f2_fma(quo, f2_splat(kE4m3Max), f2_mul(left, f2_splat(inv.inv448))), y.x, y.y);
              if constexpr (V > 1)
                *reinterpret_cast<__nv_fp8x2_storage_t*>(&qv.v[2 * j]) =
                    __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
            }
            store_vec<uint8_t, V>(q + col, qv);
          }
        }
        continue;
      }
      // u, and what is left of it: formed anew where they are used, as both would not fit the registers
      struct Products {
        float u[V + 1], lo[V + 1];
      };
      auto products = [&](int i) {
        Products f;
        if constexpr (kExact) {
#pragma unroll
          for (int j = 0; j < v[i].kPairs; ++j) {
            f2_unpack(v[i].p[j], f.u[2 * j], f.u[2 * j + 1]);
            f.lo[2 * j] = f.lo[2 * j + 1] = 0.f;
          }
        } else {
          const Floats<V> w = at.weight(weights, i);
#pragma unroll
          for (int j = 0; j < w.kPairs; ++j) {
            f2_unpack(f2_mul(v[i].p[j], w.p[j]), f.u[2 * j], f.u[2 * j + 1]);
            float a[2], b[2];
            f2_unpack(v[i].p[j], a[0], a[1]);
            f2_unpack(w.p[j], b[0], b[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) f.lo[2 * j + k] = left_of(a[k], b[k], f.u[2 * j + k]);
          }
        }
        return f;
      };
      auto meet = [] {
        if (kWarpRow) __syncwarp(); else __syncthreads();
      };
      uint32_t* amax = reinterpret_cast<uint32_t*>(smem) + unit * p.groups;
      int* amax_lo = reinterpret_cast<int*>(smem) + (per_block + unit) * p.groups;  // only where not exact
      meet();  // the row before is done with them
      for (int g = t; g < p.groups; g += width) {
        amax[g] = 0u;
        if (!kExact) amax_lo[g] = signed_bits(-INFINITY);
      }
      meet();
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < v[i].kPairs; ++j) v[i].p[j] = f2_mul(v[i].p[j], pow2);
        if constexpr (kExact) {
          const Floats<V> w = at.weight(weights, i);
#pragma unroll
          for (int j = 0; j < w.kPairs; ++j) v[i].p[j] = f2_mul(v[i].p[j], w.p[j]);
        }
        const Products f = products(i);
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (at.has(i, k)) atomicMax(&amax[(at.col(i) + k) / p.group], abs_bits(f.u[k]));
      }
      meet();
      if (!kExact) {  // of equal largest products what is left decides
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const Products f = products(i);
#pragma unroll
          for (int k = 0; k < V; ++k) {
            if (!at.has(i, k)) continue;
            const int g = (at.col(i) + k) / p.group;
            if (abs_bits(f.u[k]) == amax[g]) atomicMax(&amax_lo[g], signed_bits(outward(f.lo[k], f.u[k])));
          }
        }
        meet();
      }
      for (int g = t; g < p.groups; g += width) scale[g] = scale_of(amax[g], rs.rest);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const Products f = products(i);
        Vec<uint8_t, V> qv;
        Inverse inv;
        int last = -1;  // the group that `inv` is of: a vector is in one, or in two
#pragma unroll
        for (int k = 0; k < V; ++k) {
          qv.v[k] = 0;
          if (!at.has(i, k)) continue;
          const int g = (at.col(i) + k) / p.group;
          if (g != last) {
            inv = inverse_of(amax[g], kExact ? 0.f : from_signed_bits(amax_lo[g]), scale_of(amax[g], rs.rest));
            last = g;
          }
          qv.v[k] = quantise(f.u[k], f.lo[k], inv);
        }
        at.store(q, i, qv);
      }
    }
  }
}

// Rows too wide for registers (over 16384 columns): one block per row, which
// reads h (its own writes: each thread returns to the columns it wrote) once more
// per pass, from L2 as a rule.
template <class T, class R, Output kOut>
__global__ void __launch_bounds__(kLoopThreads) norm_fwd_loop_kernel(NormParams p) {
  constexpr bool kFp8 = kOut != kSameBits, kExact = kOut == kFp8Exact;
  extern __shared__ uint32_t amax[];
  __shared__ float red[32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.xs;
  const R* r = static_cast<const R*>(p.r) + row * p.rs;
  R* h = static_cast<R*>(p.h) + row * p.hs;
  float ss = 0.f;
  for (int c = threadIdx.x; c < p.cols; c += kLoopThreads) {
    float f = to_f32(x[c]);
    if (p.r) {
      const R hv = from_f32<R>(f + to_f32(r[c]));
      h[c] = hv;
      f = to_f32(hv);
    }
    ss = fmaf(f, f, ss);
  }
  ss = block_sum(ss, red);
  const float rstd = rsqrtf(ss * (1.0f / float(p.cols)) + p.eps);
  if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
  auto h_at = [&](int c) { return p.r ? to_f32(h[c]) : to_f32(x[c]); };
  auto weight = [&](int c) { return load_weight(p.w, p.w_dtype, p.offset, c); };
  if constexpr (!kFp8) {
    T* y = static_cast<T*>(p.y) + row * p.ys;
    for (int c = threadIdx.x; c < p.cols; c += kLoopThreads) y[c] = from_f32<T>(h_at(c) * rstd * weight(c));
  } else {
    const Rstd rs = split(rstd);
    int* amax_lo = reinterpret_cast<int*>(amax + p.groups);
    auto lo = [&](int c, float u) { return kExact ? 0.f : left_of(h_at(c) * rs.pow2, weight(c), u); };
    auto value = [&](int c) { return h_at(c) * rs.pow2 * weight(c); };
    for (int g = threadIdx.x; g < p.groups; g += kLoopThreads) {
      amax[g] = 0u;
      if (!kExact) amax_lo[g] = signed_bits(-INFINITY);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.cols; c += kLoopThreads) atomicMax(&amax[c / p.group], abs_bits(value(c)));
    __syncthreads();
    if (!kExact) {
      for (int c = threadIdx.x; c < p.cols; c += kLoopThreads) {
        const float u = value(c);
        if (abs_bits(u) == amax[c / p.group]) atomicMax(&amax_lo[c / p.group], signed_bits(outward(lo(c, u), u)));
      }
      __syncthreads();
    }
    for (int g = threadIdx.x; g < p.groups; g += kLoopThreads)
      p.scale[row * p.groups + g] = scale_of(amax[g], rs.rest);
    uint8_t* q = static_cast<uint8_t*>(p.y) + row * p.ys;
    for (int c = threadIdx.x; c < p.cols; c += kLoopThreads) {
      const int g = c / p.group;
      const float u = value(c);
      q[c] = quantise(u, lo(c, u),
                      inverse_of(amax[g], kExact ? 0.f : from_signed_bits(amax_lo[g]), scale_of(amax[g], rs.rest)));
    }
  }
}

template <class T, class R, int V, Output kOut>
cudaError_t launch_fwd(const NormParams& p, const RowPlan& pl, int grid, cudaStream_t st) {
  NormParams q = p;
  // without lanes, a group's maximum, and what is left of it where products are not exact
  const size_t maxima = kOut != kSameBits && !(p.lanes && pl.form != kLoop)
                            ? size_t(p.groups) * (kOut == kFp8Exact ? 4 : 8) * (pl.form == kWarp ? kWarpRowBlock / 32 : 1)
                            : 0;
  if (pl.form == kLoop) {
    auto kern = norm_fwd_loop_kernel<T, R, kOut>;
    if (maxima > 47 * 1024) {  // the kernel also has some of its own
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(maxima));
      if (e != cudaSuccess) return e;
    }
    kern<<<unsigned(p.rows), kLoopThreads, maxima, st>>>(p);
    return cudaGetLastError();
  }
  q.slots_at = int(maxima + 15) / 16 * 16;
  const int smem = q.slots_at + row_smem(pl, sizeof(T) + sizeof(R));
  auto kern = pick_form<V>(pl, [](auto nv, auto form, auto ragged) {
    return &norm_fwd_kernel<T, R, V, decltype(nv)::value, decltype(form)::value, decltype(ragged)::value, kOut>;
  });
  if (smem > 47 * 1024) {  // the kernels also have some of their own
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<grid, pl.threads, smem, st>>>(q);
  return cudaGetLastError();
}

template <class T, class R, Output kOut>
cudaError_t launch_fwd_types(const NormParams& p, const RowPlan& pl, int grid, cudaStream_t st) {
  if (pl.vec == 1) return launch_fwd<T, R, 1, kOut>(p, pl, grid, st);
  return launch_fwd<T, R, kVecOf<T, R>, kOut>(p, pl, grid, st);
}

template <Output kOut>
cudaError_t launch_fwd_any(const NormParams& p, int32_t dt, int32_t rdt, const RowPlan& pl, int grid, cudaStream_t st) {
  if constexpr (kOut != kFp8Exact) {
    if (dt == FLCE_F32) return launch_fwd_types<float, float, kOut>(p, pl, grid, st);
    if (rdt == FLCE_F32)
      return dt == FLCE_BF16 ? launch_fwd_types<__nv_bfloat16, float, kOut>(p, pl, grid, st)
                             : launch_fwd_types<__half, float, kOut>(p, pl, grid, st);
  } else if (rdt == FLCE_F32) {
    return cudaErrorInvalidValue;
  }
  return dt == FLCE_BF16 ? launch_fwd_types<__nv_bfloat16, __nv_bfloat16, kOut>(p, pl, grid, st)
                         : launch_fwd_types<__half, __half, kOut>(p, pl, grid, st);
}

}  // namespace
}  // namespace flce
