// flce_norm_bwd.cu — backward kernels of the norm.
#include "flce_norm.cuh"

namespace flce {
namespace {

// Rows go to warps (kWarpRow) or to blocks, in turn; dweight is summed in
// registers over the rows of a warp or block and written as one partial row per
// block, which dweight_reduce_kernel adds up in block order.  With
// a_j = rstd g_j + dh_j the output is a_j - (rstd c) n_j: g itself is not kept.
// 16384 x 4096 bf16 with dh: 93.8 us with the reduction, 5.7 TB/s; without
// dweight nothing but the rows' traffic is left.  What is above the copy rate:
// one wave of blocks (more waves mean more partial rows), the partial rows and
// the reduction's launch.
// Where one block fills an SM nobody hides its waits, so rstd is loaded a row
// ahead too (8192 x 8192: 86 us, not ahead 108; the forms with more blocks lose by
// it, 8 us of 88 at 16384 x 2048 with an fp32 residual).  The widest rows leave
// no registers for the dweight sums: in shared memory, 4096 x 16384 takes 214 us
// in place of 259.
template <class T, class R, int V, int NV, RowForm kForm, bool kRagged>
__global__ void __launch_bounds__(row_threads(kForm), bwd_blocks(kForm, kRagged, V * NV)) norm_bwd_kernel(NormBwdParams p) {
  constexpr bool kWarpRow = kForm == kWarp;
  constexpr bool kCopy = copies(kForm, V);  // rows are copied ahead
  constexpr bool kOne = kForm == kWide || kForm == kBig;  // one block on an SM: nobody hides its waits
  constexpr bool kSumsSmem = kForm == kBig;               // no registers left for them
  extern __shared__ __align__(16) uint8_t smem[];  // weights and slots; later, kWarpRow: [cols] sums
  __shared__ float red[2][32];
  griddep_release();  // the reduction of dweight may be set up
  const int t = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;
  const int width = kWarpRow ? 32 : blockDim.x;
  const int per_block = kWarpRow ? kWarpRowBlock / 32 : 1;
  const int unit = kWarpRow ? threadIdx.x >> 5 : 0;  // the row of the block
  const int64_t step = int64_t(gridDim.x) * per_block;
  int64_t row = int64_t(blockIdx.x) * per_block + unit;
  const T* dy = static_cast<const T*>(p.dy) + row * p.dys;
  const R* h = static_cast<const R*>(p.h) + row * p.hs;
  const R* dh = static_cast<const R*>(p.dh) + row * p.dhs;
  const int shift = kRagged ? int((reinterpret_cast<uintptr_t>(dy) / sizeof(T)) % V) : 0;
  const RowVectors<V, NV, kRagged> at = {t * V - shift, width * V, p.cols, t};
  const int h_at = at.template bytes<T>(), dh_at = h_at + at.template bytes<R>(),
            row_bytes = dh_at + at.template bytes<R>();
  uint8_t* weights = smem + unit * at.template bytes<float>();
  uint8_t* slots = smem + per_block * at.template bytes<float>() + unit * kRowStages * row_bytes;
  Vec<T, V> dye[NV];  // ragged ends of the next row, or a whole row where nothing is copied ahead
  Vec<R, V> he[NV], dhe[NV];
  auto fetch = [&](int64_t n, int stage) {  // row n, if there is one
    if (n < p.rows) {
      uint8_t* to = slots + stage * row_bytes;
      at.fetch(static_cast<const T*>(p.dy) + n * p.dys, to);
      at.fetch(static_cast<const R*>(p.h) + n * p.hs, to + h_at);
      if (p.dh) at.fetch(static_cast<const R*>(p.dh) + n * p.dhs, to + dh_at);
    }
    cp_async_commit();
  };
  auto edges = [&]() {
    at.edges(dy, dye);
    at.edges(h, he);
    if (p.dh) at.edges(dh, dhe);
  };
  if constexpr (kCopy) {
#pragma unroll
    for (int k = 0; k < kRowStages; ++k) fetch(row + k * step, k);
    if (row < p.rows) edges();
  }
  at.keep_weights(p.w, p.w_dtype, p.offset, weights);
  uint8_t* sums = smem + at.template bytes<float>();  // kSumsSmem: behind the weights, laid out alike
  Floats<V> acc[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int j = 0; j < acc[i].kPairs; ++j) acc[i].p[j] = f2_splat(0.f);
    if (kSumsSmem) at.put(sums, i, acc[i]);
  }
  int turn = 0, stage = 0;
  const float inv_cols = 1.0f / float(p.cols);
  float rstd_next = kOne && row < p.rows ? p.rstd[row] : 0.f;  // a row ahead
  for (; row < p.rows; row += step) {
    const float rstd = kOne ? rstd_next : p.rstd[row];
    if (kOne && row + step < p.rows) rstd_next = p.rstd[row + step];
    if constexpr (kCopy) {
      cp_async_wait<kRowStages - 1>();
    } else {
      at.load(dy, dye);
      at.load(h, he);
      if (p.dh) at.load(dh, dhe);
    }
    const uint64_t rstd2 = f2_splat(rstd);
    Floats<V> a[NV], n[NV];
    uint64_t dots = f2_splat(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Vec<T, V> dyv = dye[i];
      Vec<R, V> hv = he[i], dhv = dhe[i];
      if constexpr (kCopy) {
        uint8_t* from = slots + stage * row_bytes;
        dyv = at.read(from, i, dye);
        hv = at.read(from + h_at, i, he);
        if (p.dh) dhv = at.read(from + dh_at, i, dhe);
      }
      const Floats<V> w = at.weight(weights, i), d = widen(dyv), hf = widen(hv);
      if (kSumsSmem) acc[i] = at.weight(sums, i);
#pragma unroll
      for (int j = 0; j < w.kPairs; ++j) {
        n[i].p[j] = f2_mul(hf.p[j], rstd2);
        a[i].p[j] = f2_mul(d.p[j], w.p[j]);
        dots = f2_fma(a[i].p[j], n[i].p[j], dots);
        acc[i].p[j] = f2_fma(d.p[j], n[i].p[j], acc[i].p[j]);
      }
      if (kSumsSmem) at.put(sums, i, acc[i]);
      if (p.dh) {
        const Floats<V> e = widen(dhv);
#pragma unroll
        for (int j = 0; j < w.kPairs; ++j) a[i].p[j] = f2_fma(a[i].p[j], rstd2, e.p[j]);
      } else {
#pragma unroll
        for (int j = 0; j < w.kPairs; ++j) a[i].p[j] = f2_mul(a[i].p[j], rstd2);
      }
    }
    dy += step * p.dys;
    h += step * p.hs;
    dh += step * p.dhs;
    if constexpr (kCopy) {
      fetch(row + kRowStages * step, stage);
      if (kRagged && row + step < p.rows) edges();
      stage = stage + 1 == kRowStages ? 0 : stage + 1;
    }
    const float dot = kWarpRow ? warp_sum(pair_sum(dots)) : block_sum(pair_sum(dots), red[turn]);
    turn ^= 1;
    const uint64_t c2 = f2_splat(-rstd * (dot * inv_cols));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < a[i].kPairs; ++j) a[i].p[j] = f2_fma(n[i].p[j], c2, a[i].p[j]);
      if (p.dx) at.store(static_cast<T*>(p.dx) + row * p.dxs, i, narrow<T>(a[i]));
      if (p.dr) at.store(static_cast<R*>(p.dr) + row * p.drs, i, narrow<R>(a[i]));
    }
  }
  if (!p.part) return;
  float sum[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (kSumsSmem) acc[i] = at.weight(sums, i);
#pragma unroll
    for (int j = 0; j < acc[i].kPairs; ++j) {
      float hi;
      f2_unpack(acc[i].p[j], sum[i][2 * j], V == 1 ? hi : sum[i][V == 1 ? 0 : 2 * j + 1]);
    }
  }
  float* part = p.part + int64_t(blockIdx.x) * p.cols;
  if (kWarpRow) {  // the warps add their sums in warp order
    float* dw_s = reinterpret_cast<float*>(smem);
    __syncthreads();  // every warp is done with its slots
    for (int c = threadIdx.x; c < p.cols; c += kWarpRowBlock) dw_s[c] = 0.f;
    __syncthreads();
    for (int wp = 0; wp < per_block; ++wp) {
      if (unit == wp) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k)
            if (at.has(i, k)) dw_s[at.col(i) + k] += sum[i][k];
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < p.cols; c += kWarpRowBlock) part[c] = dw_s[c];
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (at.has(i, k)) part[at.col(i) + k] = sum[i][k];
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
    dot = fmaf(to_f32(dy[c]) * load_weight(p.w, p.w_dtype, p.offset, c), to_f32(h[c]) * rstd, dot);
  }
  const float c0 = block_sum(dot, red) / float(p.cols);
  for (int c = threadIdx.x; c < p.cols; c += kLoopThreads) {
    const float g = to_f32(dy[c]) * load_weight(p.w, p.w_dtype, p.offset, c);
    float d = rstd * fmaf(-to_f32(h[c]) * rstd, c0, g);
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

template <class T, class R, int V>
cudaError_t launch_bwd(const NormBwdParams& p, const RowPlan& pl, int blocks, cudaStream_t st) {
  if (pl.form == kLoop) {
    if (p.part) {
      norm_dweight_kernel<T, R><<<dim3(unsigned((p.cols + 255) / 256), unsigned(blocks)), 256, 0, st>>>(p);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    if (p.dx || p.dr) norm_bwd_loop_kernel<T, R><<<unsigned(p.rows), kLoopThreads, 0, st>>>(p);
    return cudaGetLastError();
  }
  auto kern = pick_form<V>(pl, [](auto nv, auto form, auto ragged) {
    return &norm_bwd_kernel<T, R, V, decltype(nv)::value, decltype(form)::value, decltype(ragged)::value>;
  });
  const int sums = pl.form == kBig ? pl.threads * pl.nv * pl.vec * 4 : 0;
  const int slots = row_smem(pl, sizeof(T) + 2 * sizeof(R)) + sums;
  const int smem = std::max(slots, pl.form == kWarp ? p.cols * 4 : 0);
  if (smem > 47 * 1024) {  // the kernels also have some of their own
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<blocks, pl.threads, smem, st>>>(p);
  return cudaGetLastError();
}

template <class T, class R>
cudaError_t launch_bwd_types(const NormBwdParams& p, const RowPlan& pl, int blocks, cudaStream_t st) {
  if (pl.vec == 1) return launch_bwd<T, R, 1>(p, pl, blocks, st);
  return launch_bwd<T, R, kVecOf<T, R>>(p, pl, blocks, st);
}

}  // namespace

cudaError_t launch_norm_bwd(const NormBwdParams& p, int32_t dt, int32_t rdt, const RowPlan& pl, int blocks,
                            cudaStream_t st) {
  if (dt == FLCE_F32) return launch_bwd_types<float, float>(p, pl, blocks, st);
  if (dt == FLCE_BF16)
    return rdt == FLCE_F32 ? launch_bwd_types<__nv_bfloat16, float>(p, pl, blocks, st)
                           : launch_bwd_types<__nv_bfloat16, __nv_bfloat16>(p, pl, blocks, st);
  return rdt == FLCE_F32 ? launch_bwd_types<__half, float>(p, pl, blocks, st)
                         : launch_bwd_types<__half, __half>(p, pl, blocks, st);
}

}  // namespace flce
