// flce_norm.cu — residual addition + root-mean-square norm, forward (also with
// an 8-bit output) and backward: kernels and C entry points.
//
//   h = rn(x + r),  rstd = (mean h^2 + eps)^(-1/2),  y_j = h_j rstd (w_j + o)
//   d_j = rstd (g_j - n_j c) + dh_j  with g_j = dy_j (w_j + o), n_j = h_j rstd,
//   c = mean_j g_j n_j;  dw_j = sum over rows of dy_j n_j
//
// Every element is used once per row, so the bound is memory: the forward reads
// x and r and writes h and y, the backward reads dy, h and dh and writes d.  A
// row is read once and stays in registers between its reduction and its output.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "flce_elem.cuh"
#include "flce_host.h"

namespace flce {
namespace {

constexpr int64_t kMaxCols = 131072;
constexpr int kWarpRowBlock = 256;    // threads of a block that gives each warp a row
constexpr int kMaxThreads = 1024;
constexpr int kLoopThreads = 1024;    // rows too wide for registers
constexpr float kE4m3Max = 448.0f;

// Most threads of a row kernel that holds nv vectors per thread.
constexpr int row_threads(bool warp_row, int nv) { return warp_row ? kWarpRowBlock : nv <= 2 ? 512 : kMaxThreads; }

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
  float eps, offset;
};

template <int V>
__device__ __forceinline__ void load_weight(const void* w, int dtype, float offset, int col, float (&out)[V]) {
  if (w) {
    load_as_f32<V>(w, dtype, col, out);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) out[k] = 1.0f;
  }
#pragma unroll
  for (int k = 0; k < V; ++k) out[k] += offset;
}

// e4m3(y / s), 0 where s is 0; saturates, NaN stays NaN.
__device__ __forceinline__ uint8_t quantise(float y, float s) {
  return s == 0.0f ? uint8_t(0) : uint8_t(__nv_cvt_float_to_fp8(y / s, __NV_SATFINITE, __NV_E4M3));
}

// Order-preserving bits of |y|: a NaN is above infinity, so that a group with
// one gets a NaN scale.
__device__ __forceinline__ uint32_t abs_bits(float y) { return __float_as_uint(y) & 0x7fffffffu; }

// One row per warp (kWarpRow, kWarpRowBlock threads) or per block.  A thread
// holds NV vectors of V elements: vector i is columns (t + i * width) * V.
template <class T, class R, int V, int NV, bool kWarpRow, bool kFp8>
__global__ void __launch_bounds__(row_threads(kWarpRow, NV)) norm_fwd_kernel(NormParams p) {
  extern __shared__ uint32_t amax_all[];  // 8-bit output: [rows of the block][groups]
  __shared__ float red[32];
  const int t = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;
  const int width = kWarpRow ? 32 : blockDim.x;
  const int64_t row = kWarpRow ? blockIdx.x * int64_t(kWarpRowBlock / 32) + (threadIdx.x >> 5) : int64_t(blockIdx.x);
  if (kWarpRow && row >= p.rows) return;
  const T* x = static_cast<const T*>(p.x) + row * p.xs;
  const R* r = static_cast<const R*>(p.r) + row * p.rs;
  R* h = static_cast<R*>(p.h) + row * p.hs;
  float v[NV][V];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (t + i * width) * V;
    if (col < p.cols) {
      const Vec<T, V> xv = load_vec<T, V>(x + col);
      if (p.r) {
        const Vec<R, V> rv = load_vec<R, V>(r + col);
        Vec<R, V> hv;
#pragma unroll
        for (int k = 0; k < V; ++k) {
          hv.v[k] = from_f32<R>(to_f32(xv.v[k]) + to_f32(rv.v[k]));
          v[i][k] = to_f32(hv.v[k]);
        }
        store_vec<R, V>(h + col, hv);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) v[i][k] = to_f32(xv.v[k]);
      }
#pragma unroll
      for (int k = 0; k < V; ++k) ss = fmaf(v[i][k], v[i][k], ss);
    }
  }
  ss = kWarpRow ? warp_sum(ss) : block_sum(ss, red);
  const float rstd = 1.0f / sqrtf(ss / float(p.cols) + p.eps);
  if (t == 0 && p.rstd) p.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (t + i * width) * V;
    if (col < p.cols) {
      float w[V];
      load_weight<V>(p.w, p.w_dtype, p.offset, col, w);
#pragma unroll
      for (int k = 0; k < V; ++k) v[i][k] = v[i][k] * rstd * w[k];
      if (!kFp8) {
        Vec<T, V> yv;
#pragma unroll
        for (int k = 0; k < V; ++k) yv.v[k] = from_f32<T>(v[i][k]);
        store_vec<T, V>(static_cast<T*>(p.y) + row * p.ys + col, yv);
      }
    }
  }
  if (kFp8) {
    uint32_t* amax = amax_all + (kWarpRow ? (threadIdx.x >> 5) * p.groups : 0);
    for (int g = t; g < p.groups; g += width) amax[g] = 0u;
    if (kWarpRow) __syncwarp(); else __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (t + i * width) * V;
      if (col < p.cols) {  // a vector lies within one group (the group is a multiple of V)
        uint32_t m = 0u;
#pragma unroll
        for (int k = 0; k < V; ++k) m = max(m, abs_bits(v[i][k]));
        atomicMax(&amax[col / p.group], m);
      }
    }
    if (kWarpRow) __syncwarp(); else __syncthreads();
    for (int g = t; g < p.groups; g += width) p.scale[row * p.groups + g] = __uint_as_float(amax[g]) / kE4m3Max;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (t + i * width) * V;
      if (col < p.cols) {
        const float s = __uint_as_float(amax[col / p.group]) / kE4m3Max;
        Vec<uint8_t, V> q;
#pragma unroll
        for (int k = 0; k < V; ++k) q.v[k] = quantise(v[i][k], s);
        store_vec<uint8_t, V>(static_cast<uint8_t*>(p.y) + row * p.ys + col, q);
      }
    }
  }
}

// Rows too wide for registers: one block per row, which reads h (its own
// writes: each thread returns to the columns it wrote) once more per pass.
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
  const float rstd = 1.0f / sqrtf(ss / float(p.cols) + p.eps);
  if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
  auto value = [&](int c) {
    float w[1];
    load_weight<1>(p.w, p.w_dtype, p.offset, c, w);
    return (p.r ? to_f32(h[c]) : to_f32(x[c])) * rstd * w[0];
  };
  if (!kFp8) {
    T* y = static_cast<T*>(p.y) + row * p.ys;
    for (int c = threadIdx.x; c < p.cols; c += kLoopThreads) y[c] = from_f32<T>(value(c));
    return;
  }
  for (int g = threadIdx.x; g < p.groups; g += kLoopThreads) amax[g] = 0u;
  __syncthreads();
  for (int c = threadIdx.x; c < p.cols; c += kLoopThreads) atomicMax(&amax[c / p.group], abs_bits(value(c)));
  __syncthreads();
  for (int g = threadIdx.x; g < p.groups; g += kLoopThreads)
    p.scale[row * p.groups + g] = __uint_as_float(amax[g]) / kE4m3Max;
  uint8_t* q = static_cast<uint8_t*>(p.y) + row * p.ys;
  for (int c = threadIdx.x; c < p.cols; c += kLoopThreads)
    q[c] = quantise(value(c), __uint_as_float(amax[c / p.group]) / kE4m3Max);
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
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

// One row at a time per warp (kWarpRow) or per block; dweight is summed in
// registers over the rows of a warp or block and written as one partial row per
// block, which dweight_reduce_kernel adds up in block order.
template <class T, class R, int V, int NV, bool kWarpRow>
__global__ void __launch_bounds__(row_threads(kWarpRow, NV)) norm_bwd_kernel(NormBwdParams p) {
  extern __shared__ float dw_s[];  // kWarpRow: [cols]
  __shared__ float red[2][32];
  const int t = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;
  const int width = kWarpRow ? 32 : blockDim.x;
  const int per_block = kWarpRow ? kWarpRowBlock / 32 : 1;
  const int64_t step = int64_t(gridDim.x) * per_block;
  float acc[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) acc[i][k] = 0.f;
  int turn = 0;
  const float inv_cols = 1.0f / float(p.cols);
  for (int64_t row = int64_t(blockIdx.x) * per_block + (kWarpRow ? (threadIdx.x >> 5) : 0); row < p.rows; row += step) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.dys;
    const R* h = static_cast<const R*>(p.h) + row * p.hs;
    const R* dh = static_cast<const R*>(p.dh) + row * p.dhs;
    const float rstd = p.rstd[row];
    float g[NV][V], n[NV][V];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (t + i * width) * V;
      if (col < p.cols) {
        const Vec<T, V> dyv = load_vec<T, V>(dy + col);
        const Vec<R, V> hv = load_vec<R, V>(h + col);
        float w[V];
        load_weight<V>(p.w, p.w_dtype, p.offset, col, w);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float d = to_f32(dyv.v[k]);
          n[i][k] = to_f32(hv.v[k]) * rstd;
          g[i][k] = d * w[k];
          dot = fmaf(g[i][k], n[i][k], dot);
          acc[i][k] = fmaf(d, n[i][k], acc[i][k]);
        }
      }
    }
    dot = kWarpRow ? warp_sum(dot) : block_sum(dot, red[turn]);
    turn ^= 1;
    const float c = dot * inv_cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (t + i * width) * V;
      if (col < p.cols) {
        float d[V];
#pragma unroll
        for (int k = 0; k < V; ++k) d[k] = rstd * fmaf(-n[i][k], c, g[i][k]);
        if (p.dh) {
          const Vec<R, V> dhv = load_vec<R, V>(dh + col);
#pragma unroll
          for (int k = 0; k < V; ++k) d[k] += to_f32(dhv.v[k]);
        }
        if (p.dx) {
          Vec<T, V> o;
#pragma unroll
          for (int k = 0; k < V; ++k) o.v[k] = from_f32<T>(d[k]);
          store_vec<T, V>(static_cast<T*>(p.dx) + row * p.dxs + col, o);
        }
        if (p.dr) {
          Vec<R, V> o;
#pragma unroll
          for (int k = 0; k < V; ++k) o.v[k] = from_f32<R>(d[k]);
          store_vec<R, V>(static_cast<R*>(p.dr) + row * p.drs + col, o);
        }
      }
    }
  }
  if (!p.part) return;
  float* part = p.part + int64_t(blockIdx.x) * p.cols;
  if (kWarpRow) {  // the warps add their sums in warp order
    for (int wp = 0; wp < per_block; ++wp) {
      if (int(threadIdx.x >> 5) == wp) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int col = (t + i * width) * V;
          if (col < p.cols)
#pragma unroll
            for (int k = 0; k < V; ++k) dw_s[col + k] = wp == 0 ? acc[i][k] : dw_s[col + k] + acc[i][k];
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < p.cols; c += kWarpRowBlock) part[c] = dw_s[c];
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (t + i * width) * V;
      if (col < p.cols)
#pragma unroll
        for (int k = 0; k < V; ++k) part[col + k] = acc[i][k];
    }
  }
}

// Rows too wide for registers: the gradient row by row in two passes ...
template <class T, class R>
__global__ void __launch_bounds__(kLoopThreads) norm_bwd_loop_kernel(NormBwdParams p) {
  __shared__ float red[32];
  const int64_t row = blockIdx.x;
  const T* dy = static_cast<const T*>(p.dy) + row * p.dys;
  const R* h = static_cast<const R*>(p.h) + row * p.hs;
  const R* dh = static_cast<const R*>(p.dh) + row * p.dhs;
  const float rstd = p.rstd[row];
  float dot = 0.f;
  for (int c = threadIdx.x; c < p.cols; c += kLoopThreads) {
    float w[1];
    load_weight<1>(p.w, p.w_dtype, p.offset, c, w);
    dot = fmaf(to_f32(dy[c]) * w[0], to_f32(h[c]) * rstd, dot);
  }
  const float c0 = block_sum(dot, red) / float(p.cols);
  for (int c = threadIdx.x; c < p.cols; c += kLoopThreads) {
    float w[1];
    load_weight<1>(p.w, p.w_dtype, p.offset, c, w);
    float d = rstd * fmaf(-to_f32(h[c]) * rstd, c0, to_f32(dy[c]) * w[0]);
    if (p.dh) d += to_f32(dh[c]);
    if (p.dx) (static_cast<T*>(p.dx) + row * p.dxs)[c] = from_f32<T>(d);
    if (p.dr) (static_cast<R*>(p.dr) + row * p.drs)[c] = from_f32<R>(d);
  }
}
// ... after the column sums (dx may be dy's own memory): block (i, j) sums the
// rows j, j + gridDim.y, ... of columns [256 i, 256 (i + 1)).
template <class T, class R>
__global__ void __launch_bounds__(256) norm_dweight_kernel(NormBwdParams p) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= p.cols) return;
  float s = 0.f;
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y)
    s = fmaf(to_f32(static_cast<const T*>(p.dy)[row * p.dys + c]),
             to_f32(static_cast<const R*>(p.h)[row * p.hs + c]) * p.rstd[row], s);
  p.part[int64_t(blockIdx.y) * p.cols + c] = s;
}

// dw[j] = sum over blocks of part[b][j], in a fixed order: 32 columns per
// block, warp k takes the partial rows k, k + 8, ...
constexpr int kReduceWarps = 8;
__global__ void __launch_bounds__(kReduceWarps * 32) dweight_reduce_kernel(const float* part, int blocks, int cols,
                                                                           void* dw, int dtype) {
  __shared__ float s[kReduceWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < cols)
    for (int b = warp; b < blocks; b += kReduceWarps) a += part[int64_t(b) * cols + c];
  s[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && c < cols) {
#pragma unroll
    for (int k = 1; k < kReduceWarps; ++k) a += s[k][lane];
    store_as(dw, dtype, c, a);
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// How a row is laid over threads: vectors of `vec` elements (1 where rows or
// pointers are not 16-byte aligned, or the width is not a multiple), `nv` of
// them per thread, in a warp or in `threads` threads; nv = 0: the row is too
// wide for registers.
struct RowPlan {
  int vec, nv, threads;
  bool warp_row;
};
RowPlan plan_row(int64_t cols, int vec) {
  const int64_t vecs = (cols + vec - 1) / vec;
  for (int nv : {1, 2, 4})
    if (vecs <= 32 * nv) return {vec, nv, kWarpRowBlock, true};
  for (int nv : {1, 2, 4, 8}) {
    if (vec == 8 && nv == 8) break;
    const int64_t threads = ((vecs + nv - 1) / nv + 31) / 32 * 32;
    if (threads <= row_threads(false, nv)) return {vec, nv, int(threads), false};
  }
  return {vec, 0, kLoopThreads, false};
}

// Whether every pointer and row of the call is 16-byte aligned.
struct AlignCheck {
  bool ok = true;
  void add(const void* p, int64_t stride, int64_t rows, size_t elem) {
    if (p && (!aligned_to(p, 16) || (rows > 1 && (stride * elem) % 16 != 0))) ok = false;
  }
};

template <class T, class R, int V, bool kFp8>
cudaError_t launch_fwd(const NormParams& p, const RowPlan& pl, cudaStream_t st) {
  const size_t smem = kFp8 ? size_t(p.groups) * 4 * (pl.warp_row ? kWarpRowBlock / 32 : 1) : 0;
  if (pl.nv == 0) {
    norm_fwd_loop_kernel<T, R, kFp8><<<unsigned(p.rows), kLoopThreads, smem, st>>>(p);
    return cudaGetLastError();
  }
  const unsigned grid = unsigned(pl.warp_row ? (p.rows + kWarpRowBlock / 32 - 1) / (kWarpRowBlock / 32) : p.rows);
  if (pl.warp_row) {
    if (pl.nv == 1) norm_fwd_kernel<T, R, V, 1, true, kFp8><<<grid, pl.threads, smem, st>>>(p);
    if (pl.nv == 2) norm_fwd_kernel<T, R, V, 2, true, kFp8><<<grid, pl.threads, smem, st>>>(p);
    if (pl.nv == 4) norm_fwd_kernel<T, R, V, 4, true, kFp8><<<grid, pl.threads, smem, st>>>(p);
  } else {
    if (pl.nv == 1) norm_fwd_kernel<T, R, V, 1, false, kFp8><<<grid, pl.threads, smem, st>>>(p);
    if (pl.nv == 2) norm_fwd_kernel<T, R, V, 2, false, kFp8><<<grid, pl.threads, smem, st>>>(p);
    if (pl.nv == 4) norm_fwd_kernel<T, R, V, 4, false, kFp8><<<grid, pl.threads, smem, st>>>(p);
    if constexpr (V < 8) {
      if (pl.nv == 8) norm_fwd_kernel<T, R, V, 8, false, kFp8><<<grid, pl.threads, smem, st>>>(p);
    }
  }
  return cudaGetLastError();
}

template <class T, class R, bool kFp8>
cudaError_t launch_fwd_types(const NormParams& p, bool vec_ok, cudaStream_t st) {
  constexpr int kV = 16 / sizeof(T);
  if (vec_ok && p.cols % kV == 0) return launch_fwd<T, R, kV, kFp8>(p, plan_row(p.cols, kV), st);
  return launch_fwd<T, R, 1, kFp8>(p, plan_row(p.cols, 1), st);
}

template <bool kFp8>
cudaError_t launch_fwd_any(const NormParams& p, int32_t dt, int32_t rdt, bool vec_ok, cudaStream_t st) {
  if (dt == FLCE_F32) return launch_fwd_types<float, float, kFp8>(p, vec_ok, st);
  if (dt == FLCE_BF16)
    return rdt == FLCE_F32 ? launch_fwd_types<__nv_bfloat16, float, kFp8>(p, vec_ok, st)
                           : launch_fwd_types<__nv_bfloat16, __nv_bfloat16, kFp8>(p, vec_ok, st);
  return rdt == FLCE_F32 ? launch_fwd_types<__half, float, kFp8>(p, vec_ok, st)
                         : launch_fwd_types<__half, __half, kFp8>(p, vec_ok, st);
}

// Partial dweight rows, at most; one per block of the backward.
constexpr int kMaxBwdBlocks = 512;
constexpr int kLoopSplits = 64;

int bwd_blocks(const NormBwdParams& p, const RowPlan& pl, int num_sms) {
  const int per_block = pl.warp_row ? kWarpRowBlock / 32 : 1;
  const int64_t want = (p.rows + per_block - 1) / per_block;
  return int(std::min<int64_t>(want, std::min(kMaxBwdBlocks, 2 * num_sms)));
}

template <class T, class R, int V>
cudaError_t launch_bwd(const NormBwdParams& p, const RowPlan& pl, int blocks, cudaStream_t st) {
  if (pl.nv == 0) {
    if (p.part) {
      norm_dweight_kernel<T, R><<<dim3(unsigned((p.cols + 255) / 256), unsigned(blocks)), 256, 0, st>>>(p);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    if (p.dx || p.dr) norm_bwd_loop_kernel<T, R><<<unsigned(p.rows), kLoopThreads, 0, st>>>(p);
    return cudaGetLastError();
  }
  if (pl.warp_row) {
    const size_t smem = p.part ? size_t(p.cols) * 4 : 0;
    if (pl.nv == 1) norm_bwd_kernel<T, R, V, 1, true><<<blocks, pl.threads, smem, st>>>(p);
    if (pl.nv == 2) norm_bwd_kernel<T, R, V, 2, true><<<blocks, pl.threads, smem, st>>>(p);
    if (pl.nv == 4) norm_bwd_kernel<T, R, V, 4, true><<<blocks, pl.threads, smem, st>>>(p);
  } else {
    if (pl.nv == 1) norm_bwd_kernel<T, R, V, 1, false><<<blocks, pl.threads, 0, st>>>(p);
    if (pl.nv == 2) norm_bwd_kernel<T, R, V, 2, false><<<blocks, pl.threads, 0, st>>>(p);
    if (pl.nv == 4) norm_bwd_kernel<T, R, V, 4, false><<<blocks, pl.threads, 0, st>>>(p);
    if constexpr (V < 8) {
      if (pl.nv == 8) norm_bwd_kernel<T, R, V, 8, false><<<blocks, pl.threads, 0, st>>>(p);
    }
  }
  return cudaGetLastError();
}

template <class T, class R>
cudaError_t launch_bwd_types(const NormBwdParams& p, const RowPlan& pl, int blocks, cudaStream_t st) {
  if (pl.vec == 1) return launch_bwd<T, R, 1>(p, pl, blocks, st);
  return launch_bwd<T, R, 16 / sizeof(T)>(p, pl, blocks, st);
}

cudaError_t launch_bwd_any(const NormBwdParams& p, int32_t dt, int32_t rdt, const RowPlan& pl, int blocks,
                           cudaStream_t st) {
  if (dt == FLCE_F32) return launch_bwd_types<float, float>(p, pl, blocks, st);
  if (dt == FLCE_BF16)
    return rdt == FLCE_F32 ? launch_bwd_types<__nv_bfloat16, float>(p, pl, blocks, st)
                           : launch_bwd_types<__nv_bfloat16, __nv_bfloat16>(p, pl, blocks, st);
  return rdt == FLCE_F32 ? launch_bwd_types<__half, float>(p, pl, blocks, st)
                         : launch_bwd_types<__half, __half>(p, pl, blocks, st);
}

int validate(const flce_norm_problem* p) {
  if (!p) return FLCE_ERR_INVALID_ARG;
  if (p->rows < 0 || p->rows > INT32_MAX || p->cols < 1 || p->cols > kMaxCols) return FLCE_ERR_INVALID_ARG;
  if (!known_dtype(p->dtype) || !known_dtype(p->residual_dtype)) return FLCE_ERR_UNSUPPORTED_DTYPE;
  if (p->residual_dtype != p->dtype && p->residual_dtype != FLCE_F32) return FLCE_ERR_DTYPE_MISMATCH;
  if (p->x_stride < 0 || p->residual_stride < 0 || p->h_stride < 0 || p->y_stride < 0 || p->dresidual_stride < 0)
    return FLCE_ERR_INVALID_ARG;
  if (!std::isfinite(p->eps) || p->eps < 0.f || !std::isfinite(p->weight_offset)) return FLCE_ERR_INVALID_ARG;
  return FLCE_OK;
}

// Rows of an output must not overlap.
bool out_rows_ok(const flce_norm_problem* p, const void* out, int64_t stride) {
  return !out || p->rows <= 1 || stride >= p->cols;
}

int forward(const flce_norm_problem* p, const void* x, const void* residual, const void* weight, void* h, void* y,
            float* rstd, float* scale, bool fp8, flce_stream_t stream) {
  FLCE_TRY(validate(p));
  if (weight && !known_dtype(p->weight_dtype)) return FLCE_ERR_UNSUPPORTED_DTYPE;
  if (!residual && p->residual_dtype != p->dtype) return FLCE_ERR_DTYPE_MISMATCH;
  if (fp8 && (p->quant_group < 0 || p->quant_group % 16 != 0)) return FLCE_ERR_INVALID_ARG;
  if (p->rows == 0) return FLCE_OK;
  if (!x || !y || (residual != nullptr) != (h != nullptr) || (fp8 && !scale)) return FLCE_ERR_INVALID_ARG;
  if (!out_rows_ok(p, h, p->h_stride) || !out_rows_ok(p, y, p->y_stride)) return FLCE_ERR_INVALID_ARG;
  const size_t es = elem_size(p->dtype), er = elem_size(p->residual_dtype), ey = fp8 ? 1 : es;
  if (!aligned_to(x, es) || !aligned_to(y, ey) || !aligned_to(residual, er) || !aligned_to(h, er) ||
      (weight && !aligned_to(weight, elem_size(p->weight_dtype))) || !aligned_to(rstd, 4) || !aligned_to(scale, 4))
    return FLCE_ERR_MISALIGNED;
  DeviceInfo dev;
  FLCE_TRY(get_device(&dev));
  FLCE_TRY(check_local(dev, x, residual, weight, h, y, rstd, scale));
  AlignCheck a;
  a.add(x, p->x_stride, p->rows, es);
  a.add(residual, p->residual_stride, p->rows, er);
  a.add(h, p->h_stride, p->rows, er);
  a.add(weight, 0, 1, es);
  a.add(y, p->y_stride, p->rows, ey);
  NormParams n{};
  n.x = x;
  n.r = residual;
  n.w = weight;
  n.h = h;
  n.y = y;
  n.rstd = rstd;
  n.scale = scale;
  n.rows = p->rows;
  n.xs = p->x_stride;
  n.rs = p->residual_stride;
  n.hs = p->h_stride;
  n.ys = p->y_stride;
  n.cols = int32_t(p->cols);
  n.w_dtype = p->weight_dtype;
  n.group = p->quant_group == 0 ? n.cols : int32_t(std::min<int64_t>(p->quant_group, p->cols));
  n.groups = (n.cols + n.group - 1) / n.group;
  n.eps = p->eps;
  n.offset = p->weight_offset;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return logged(FLCE_LAUNCH_OTHER, st, [&] {
    return fp8 ? launch_fwd_any<true>(n, p->dtype, p->residual_dtype, a.ok, st)
               : launch_fwd_any<false>(n, p->dtype, p->residual_dtype, a.ok, st);
  });
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_add_rms_norm(const flce_norm_problem* problem, const void* x, const void* residual, const void* weight,
                      void* h, void* y, float* rstd, flce_stream_t stream) {
  return forward(problem, x, residual, weight, h, y, rstd, nullptr, false, stream);
}

int flce_add_rms_norm_fp8(const flce_norm_problem* problem, const void* x, const void* residual, const void* weight,
                          void* h, void* q, float* scale, flce_stream_t stream) {
  return forward(problem, x, residual, weight, h, q, nullptr, scale, true, stream);
}

int flce_add_rms_norm_workspace_size(const flce_norm_problem* problem, size_t* bytes) {
  if (!bytes) return FLCE_ERR_INVALID_ARG;
  FLCE_TRY(validate(problem));
  *bytes = size_t(std::min<int64_t>(problem->rows, kMaxBwdBlocks)) * size_t(problem->cols) * 4 + 256;
  return FLCE_OK;
}

int flce_add_rms_norm_backward(const flce_norm_problem* problem, const void* dy, const void* h, const void* weight,
                               const float* rstd, const void* dh, void* dx, void* dresidual, void* dweight,
                               void* workspace, size_t workspace_bytes, flce_stream_t stream) {
  const flce_norm_problem* p = problem;
  FLCE_TRY(validate(p));
  if ((weight || dweight) && !known_dtype(p->weight_dtype)) return FLCE_ERR_UNSUPPORTED_DTYPE;
  if (p->rows > 0 && (!dy || !h || !rstd || (!dx && !dresidual && !dweight))) return FLCE_ERR_INVALID_ARG;
  if (dweight && !workspace) return FLCE_ERR_INVALID_ARG;
  if (!out_rows_ok(p, dx, p->y_stride) || !out_rows_ok(p, dresidual, p->dresidual_stride)) return FLCE_ERR_INVALID_ARG;
  const size_t es = elem_size(p->dtype), er = elem_size(p->residual_dtype);
  if (!aligned_to(dy, es) || !aligned_to(dx, es) || !aligned_to(h, er) || !aligned_to(dh, er) ||
      !aligned_to(dresidual, er) || !aligned_to(rstd, 4) || !aligned_to(workspace, 16) ||
      (weight && !aligned_to(weight, elem_size(p->weight_dtype))) ||
      (dweight && !aligned_to(dweight, elem_size(p->weight_dtype))))
    return FLCE_ERR_MISALIGNED;
  size_t need = 0;
  FLCE_TRY(flce_add_rms_norm_workspace_size(p, &need));
  if (dweight && workspace_bytes < need) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  DeviceInfo dev;
  FLCE_TRY(get_device(&dev));
  FLCE_TRY(check_local(dev, dy, h, weight, rstd, dh, dx, dresidual, dweight, workspace));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  NormBwdParams n{};
  n.dy = dy;
  n.h = h;
  n.w = weight;
  n.rstd = rstd;
  n.dh = dh;
  n.dx = dx;
  n.dr = dresidual;
  n.part = dweight ? static_cast<float*>(workspace) : nullptr;
  n.rows = p->rows;
  n.dys = p->x_stride;
  n.hs = p->h_stride;
  n.dhs = p->residual_stride;
  n.dxs = p->y_stride;
  n.drs = p->dresidual_stride;
  n.cols = int32_t(p->cols);
  n.w_dtype = p->weight_dtype;
  n.offset = p->weight_offset;
  int blocks = 0;
  if (p->rows > 0) {
    AlignCheck a;
    a.add(dy, n.dys, n.rows, es);
    a.add(h, n.hs, n.rows, er);
    a.add(weight, 0, 1, es);
    a.add(dh, n.dhs, n.rows, er);
    a.add(dx, n.dxs, n.rows, es);
    a.add(dresidual, n.drs, n.rows, er);
    const int vec = int(16 / es);
    const RowPlan pl = plan_row(n.cols, a.ok && n.cols % vec == 0 ? vec : 1);
    blocks = pl.nv == 0 ? int(std::min<int64_t>(n.rows, kLoopSplits)) : bwd_blocks(n, pl, dev.num_sms);
    FLCE_TRY(logged(FLCE_LAUNCH_OTHER, st,
                    [&] { return launch_bwd_any(n, p->dtype, p->residual_dtype, pl, blocks, st); }));
  }
  if (!dweight) return FLCE_OK;
  return logged(FLCE_LAUNCH_OTHER, st, [&] {
    dweight_reduce_kernel<<<unsigned((n.cols + 31) / 32), kReduceWarps * 32, 0, st>>>(n.part, blocks, n.cols, dweight,
                                                                                    p->weight_dtype);
    return cudaGetLastError();
  });
}

}  // extern "C"
