// flce_elem.cuh — element types, vectors and reductions of the operators on
// either side of the head (norm, gradient clipping, logit processing).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "flce.h"

namespace flce {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// V adjacent elements, loaded and stored as 16-byte words (V * sizeof(T) is 16,
// 32, or one element's size for V = 1).
template <class T, int V>
struct alignas(V * sizeof(T) < 16 ? V * sizeof(T) : 16) Vec {
  T v[V];
};

template <class T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T* p) { return *reinterpret_cast<const Vec<T, V>*>(p); }
template <class T, int V>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, V>& x) { *reinterpret_cast<Vec<T, V>*>(p) = x; }

// One element of a type known at run time.
__device__ __forceinline__ float load_as(const void* p, int dtype, int64_t i) {
  if (dtype == FLCE_F32) return static_cast<const float*>(p)[i];
  if (dtype == FLCE_BF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
  return to_f32(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store_as(void* p, int dtype, int64_t i, float x) {
  if (dtype == FLCE_F32) {
    static_cast<float*>(p)[i] = x;
  } else if (dtype == FLCE_BF16) {
    static_cast<__nv_bfloat16*>(p)[i] = from_f32<__nv_bfloat16>(x);
  } else {
    static_cast<__half*>(p)[i] = from_f32<__half>(x);
  }
}

// Sum over a warp (every lane gets the same value, in a fixed order).
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// Sum over the block (every thread gets it); `buf` holds 32 values, and the
// call after next may reuse it (callers in a loop alternate two buffers).
__device__ __forceinline__ float block_sum(float x, float* buf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = (blockDim.x + 31) >> 5;
  x = warp_sum(x);
  if (lane == 0) buf[warp] = x;
  __syncthreads();
  return warp_sum(lane < warps ? buf[lane] : 0.f);
}

// As a programmatic dependent of the kernel before it on the stream (it
// may start while that one finishes, and waits for it in griddep_wait).
template <class... P, class... A>
inline cudaError_t launch_dependent(void (*kern)(P...), unsigned grid, unsigned block, cudaStream_t st, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

inline size_t elem_size(int32_t dtype) { return dtype == FLCE_F32 ? 4 : 2; }
inline bool known_dtype(int32_t dtype) { return dtype == FLCE_F32 || dtype == FLCE_BF16 || dtype == FLCE_F16; }
inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace flce
