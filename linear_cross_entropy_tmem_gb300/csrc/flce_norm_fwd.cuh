// flce_norm_fwd.cuh — forward kernels of the norm, with (kFp8) and without an
// 8-bit output.
#pragma once

#include <cuda_fp8.h>

#include "flce_norm.cuh"

namespace flce {
namespace {

// Division by a group's scale: y times the reciprocal, and one step that makes
// up for its rounding, so that q is e4m3 of the quotient as rounded to fp32.
// Below 2^-100 (where 1 / s may overflow) values take a factor of 2^64 first.
struct Inverse {
  float first, inv, minus;  // minus: -s, or 0 where the step would make NaN of 0
};
__device__ __forceinline__ Inverse inverse_of(float s) {
  const bool small = s < 0x1p-100f;
  if (small) s *= 0x1p64f;
  const float inv = s == 0.f ? 0.f : __frcp_rn(s);
  return {small ? 0x1p64f : 1.0f, inv, s < INFINITY ? -s : 0.f};
}
__device__ __forceinline__ float scale_of(uint32_t amax_bits) { return __uint_as_float(amax_bits) / kE4m3Max; }
// e4m3(y / s); saturates, NaN stays NaN.
__device__ __forceinline__ uint8_t quantise(float y, const Inverse& i) {
  y *= i.first;
  const float q = y * i.inv;
  return uint8_t(__nv_cvt_float_to_fp8(fmaf(fmaf(q, i.minus, y), i.inv, q), __NV_SATFINITE, __NV_E4M3));
}

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
// 2048 fp16 takes 26.7 us for 118 MB (4.4 TB/s): groups' maxima, the division by
// the scale and the conversion bring it to about 35 instructions per element, and
// issue slots are the bound.
template <class T, class R, int V, int NV, RowForm kForm, bool kRagged, bool kFp8>
__global__ void __launch_bounds__(row_threads(kForm), fwd_blocks(kForm, kRagged)) norm_fwd_kernel(NormParams p) {
  constexpr bool kWarpRow = kForm == kWarp;
  constexpr bool kCopy = copies(kForm, V);  // rows are copied ahead
  // [rows of the block][groups] maxima (8-bit output); weights; slots
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red[2][32];
  uint32_t* amax_all = reinterpret_cast<uint32_t*>(smem);
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
    const uint64_t rstd2 = f2_splat(rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Floats<V> w = at.weight(weights, i);
#pragma unroll
      for (int j = 0; j < w.kPairs; ++j) v[i].p[j] = f2_mul(f2_mul(v[i].p[j], rstd2), w.p[j]);
      if (!kFp8) at.store(static_cast<T*>(p.y) + row * p.ys, i, narrow<T>(v[i]));
    }
    if constexpr (kFp8) {
      uint8_t* q = static_cast<uint8_t*>(p.y) + row * p.ys;
      float* scale = p.scale + row * p.groups;
      float f[NV][V];
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < v[i].kPairs; ++j) {
          float hi;
          f2_unpack(v[i].p[j], f[i][2 * j], V == 1 ? hi : f[i][V == 1 ? 0 : 2 * j + 1]);
        }
      if (!kRagged && p.lanes) {  // a group is `lanes` neighbouring lanes' vectors of one i
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float top = 0.f;
#pragma unroll
          for (int k = 0; k + 1 < V; k += 2) top = max_abs(top, f[i][k], f[i][k + 1]);
          uint32_t m = abs_bits(top);
#pragma unroll
          for (int o = 1; o < 32; o <<= 1)
            if (o < p.lanes) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          const float s = scale_of(m);
          const int col = at.col(i);
          if (col < p.cols) {
            if ((t & (p.lanes - 1)) == 0) scale[group[i]] = s;
            const Inverse inv = inverse_of(s);
            if (inv.first != 1.0f) {
#pragma unroll
              for (int j = 0; j < v[i].kPairs; ++j) v[i].p[j] = f2_mul(v[i].p[j], f2_splat(inv.first));
            }
            Vec<uint8_t, V> qv;
#pragma unroll
            for (int j = 0; j < v[i].kPairs; ++j) {
              const uint64_t i2 = f2_splat(inv.inv), quo = f2_mul(v[i].p[j], i2);
              float2 y;
              f2_unpack(f2_fma(f2_fma(quo, f2_splat(inv.minus), v[i].p[j]), i2, quo), y.x, y.y);
              if constexpr (V > 1)
                *reinterpret_cast<__nv_fp8x2_storage_t*>(&qv.v[2 * j]) =
                    __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
            }
            store_vec<uint8_t, V>(q + col, qv);
          }
        }
        continue;
      }
      uint32_t* amax = amax_all + unit * p.groups;
      if (kWarpRow) __syncwarp(); else __syncthreads();  // the row before is done with it
      for (int g = t; g < p.groups; g += width) amax[g] = 0u;
      if (kWarpRow) __syncwarp(); else __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (at.has(i, k)) atomicMax(&amax[(at.col(i) + k) / p.group], abs_bits(f[i][k]));
      if (kWarpRow) __syncwarp(); else __syncthreads();
      for (int g = t; g < p.groups; g += width) scale[g] = scale_of(amax[g]);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        Vec<uint8_t, V> qv;
#pragma unroll
        for (int k = 0; k < V; ++k)
          qv.v[k] = at.has(i, k)
                        ? quantise(f[i][k], inverse_of(scale_of(amax[(at.col(i) + k) / p.group])))
                        : 0;
        at.store(q, i, qv);
      }
    }
  }
}

// Rows too wide for registers (over 16384 columns): one block per row, which
// reads h (its own writes: each thread returns to the columns it wrote) once more
// per pass, from L2 as a rule.
template <class T, class R, bool kFp8>
__global__ void __launch_bounds__(kLoopThreads) norm_fwd_loop_kernel(NormParams p) {
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
  auto value = [&](int c) {
    return (p.r ? to_f32(h[c]) : to_f32(x[c])) * rstd * load_weight(p.w, p.w_dtype, p.offset, c);
  };
  if constexpr (!kFp8) {
    T* y = static_cast<T*>(p.y) + row * p.ys;
    for (int c = threadIdx.x; c < p.cols; c += kLoopThreads) y[c] = from_f32<T>(value(c));
  } else {
    for (int g = threadIdx.x; g < p.groups; g += kLoopThreads) amax[g] = 0u;
    __syncthreads();
    for (int c = threadIdx.x; c < p.cols; c += kLoopThreads) atomicMax(&amax[c / p.group], abs_bits(value(c)));
    __syncthreads();
    for (int g = threadIdx.x; g < p.groups; g += kLoopThreads)
      p.scale[row * p.groups + g] = scale_of(amax[g]);
    uint8_t* q = static_cast<uint8_t*>(p.y) + row * p.ys;
    for (int c = threadIdx.x; c < p.cols; c += kLoopThreads)
      q[c] = quantise(value(c), inverse_of(scale_of(amax[c / p.group])));
  }
}

template <class T, class R, int V, bool kFp8>
cudaError_t launch_fwd(const NormParams& p, const RowPlan& pl, int grid, cudaStream_t st) {
  NormParams q = p;
  const size_t maxima =
      kFp8 && !(p.lanes && pl.form != kLoop) ? size_t(p.groups) * 4 * (pl.form == kWarp ? kWarpRowBlock / 32 : 1) : 0;
  if (pl.form == kLoop) {
    norm_fwd_loop_kernel<T, R, kFp8><<<unsigned(p.rows), kLoopThreads, maxima, st>>>(p);
    return cudaGetLastError();
  }
  q.slots_at = int(maxima + 15) / 16 * 16;
  const int smem = q.slots_at + row_smem(pl, sizeof(T) + sizeof(R));
  auto kern = pick_form<V>(pl, [](auto nv, auto form, auto ragged) {
    return &norm_fwd_kernel<T, R, V, decltype(nv)::value, decltype(form)::value, decltype(ragged)::value, kFp8>;
  });
  if (smem > 47 * 1024) {  // the kernels also have some of their own
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<grid, pl.threads, smem, st>>>(q);
  return cudaGetLastError();
}

template <class T, class R, bool kFp8>
cudaError_t launch_fwd_types(const NormParams& p, const RowPlan& pl, int grid, cudaStream_t st) {
  if (pl.vec == 1) return launch_fwd<T, R, 1, kFp8>(p, pl, grid, st);
  return launch_fwd<T, R, kVecOf<T, R>, kFp8>(p, pl, grid, st);
}

template <bool kFp8>
cudaError_t launch_fwd_any(const NormParams& p, int32_t dt, int32_t rdt, const RowPlan& pl, int grid, cudaStream_t st) {
  if (dt == FLCE_F32) return launch_fwd_types<float, float, kFp8>(p, pl, grid, st);
  if (dt == FLCE_BF16)
    return rdt == FLCE_F32 ? launch_fwd_types<__nv_bfloat16, float, kFp8>(p, pl, grid, st)
                           : launch_fwd_types<__nv_bfloat16, __nv_bfloat16, kFp8>(p, pl, grid, st);
  return rdt == FLCE_F32 ? launch_fwd_types<__half, float, kFp8>(p, pl, grid, st)
                         : launch_fwd_types<__half, __half, kFp8>(p, pl, grid, st);
}

}  // namespace
}  // namespace flce
