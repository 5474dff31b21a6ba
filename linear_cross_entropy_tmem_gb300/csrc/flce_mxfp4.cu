// flce_mxfp4.cu — matrices to 4 bits with a power of two per 32 columns, and back:
// kernels and C entry points.
//
//   m = max |x| of a block,  k = floor(log2 m) - 2 within [-127, 125],  code = e2m1(x / 2^k)
//
// Bound by memory: x read once, 17/32 byte per element written.  A warp takes 256
// columns of four rows that are 32 apart: the four rows' scales of four blocks
// are 16 adjacent bytes of a scale tile, and eight warps of a block fill a line.

#include <algorithm>

#include "flce_mxfp4.cuh"

namespace flce {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreadsQ = 256;
constexpr int kWarpsQ = kThreadsQ / 32;
constexpr int kSeg = 256;   // columns of a warp: eight blocks, two groups of four

// Scale byte of a block whose largest |x| has these bits: its exponent less 2, plus
// 127; 255 (NaN) for a NaN or an infinity.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  return top >= 0x7f800000u ? 255u : uint32_t(max(int(top >> 23) - 2, 0));
}
// 2^-k of a scale byte, 0 for NaN's: x 2^-k is exact.
__device__ __forceinline__ float inverse_scale(uint32_t s) { return s == 255u ? 0.f : __uint_as_float((254u - s) << 23); }
// 2^k of a scale byte.
__device__ __forceinline__ float scale_value(uint32_t s) {
  return s == 255u ? NAN : __uint_as_float(s == 0u ? 0x00400000u : s << 23);
}

// kVec: rows start on 16-byte boundaries and a lane takes eight adjacent columns, a
// block being four lanes'; else a lane takes one column of each block.
template <class T, bool kVec>
__global__ void __launch_bounds__(kThreadsQ) mx_quantize_kernel(MxQuantParams p) {
  griddep_release();
  if (p.status && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * kWarpsQ + (threadIdx.x >> 5);
  if (item >= p.items) return;
  // r32 fastest: the warps of a block share a scale tile
  const int r32 = int(item & 31);
  const int64_t rest = item >> 5;
  const int seg = int(rest % p.segs);
  const int64_t th = rest / p.segs;
  const int half = int(th % p.halves);
  const int64_t tile = th / p.halves;
  const int col0 = seg * kSeg;
  const int64_t blocks = mx_cdiv(p.cols, kMxBlock), row_bytes = blocks * 16;
  float x[4][8];
  bool there[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int rr = half * 128 + r32 + 32 * i;
    const int64_t r = tile * p.tile_rows + rr;
    there[i] = rr < p.tile_rows && r < p.rows;
    const T* row = static_cast<const T*>(p.x) + r * p.stride;
    if constexpr (kVec) {
      const int c = col0 + lane * 8;
      if (there[i] && c + 8 <= p.cols) {
        const Vec<T, 8> v = load_vec<T, 8>(row + c);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = to_f32(v.v[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = there[i] && c + e < p.cols ? to_f32(row[c + e]) : 0.f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = col0 + e * 32 + lane;
        x[i][e] = there[i] && c < p.cols ? to_f32(row[c]) : 0.f;
      }
    }
  }
  uint32_t word[4][2];  // the scale bytes of the row's two groups of four blocks
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = tile * p.tile_rows + half * 128 + r32 + 32 * i;
    uint8_t* to = p.codes + r * row_bytes + col0 / 2;
    if constexpr (kVec) {
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[i][e]) & 0x7fffffffu);
      top = max(top, __shfl_xor_sync(kFull, top, 1));
      top = max(top, __shfl_xor_sync(kFull, top, 2));
      const uint32_t s = scale_byte(top);
      const float inv = inverse_scale(s);
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = s == 255u ? 0.f : x[i][e] * inv;
      const uint32_t codes = to_e2m1x8(y);
      if (there[i] && col0 + (lane & ~3) * 8 < p.cols) reinterpret_cast<uint32_t*>(to)[lane] = codes;
      uint32_t w = s << (8 * ((lane >> 2) & 3));  // blocks of no column have top = 0 and s = 0
      w |= __shfl_xor_sync(kFull, w, 4);
      w |= __shfl_xor_sync(kFull, w, 8);
      word[i][0] = __shfl_sync(kFull, w, 0);
      word[i][1] = __shfl_sync(kFull, w, 16);
    } else {
      word[i][0] = word[i][1] = 0;
      uint32_t nibbles = 0;  // of block e at bits 4 e
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t top = __reduce_max_sync(kFull, __float_as_uint(x[i][e]) & 0x7fffffffu);
        const uint32_t s = scale_byte(top);
        y[e] = s == 255u ? 0.f : x[i][e] * inverse_scale(s);
        word[i][e >> 2] |= s << (8 * (e & 3));
      }
      nibbles = to_e2m1x8(y);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t v = ((nibbles >> (4 * e)) & 15u) << (4 * (lane & 7));
        v |= __shfl_xor_sync(kFull, v, 1);
        v |= __shfl_xor_sync(kFull, v, 2);
        v |= __shfl_xor_sync(kFull, v, 4);
        if ((lane & 7) == 0 && there[i] && col0 + e * 32 < p.cols)
          *reinterpret_cast<uint32_t*>(to + e * 16 + (lane >> 3) * 4) = v;
      }
    }
  }
  // group g's tile: 16 bytes for r32, four for each of the rows
  if (lane < 2 && seg * 2 + lane < p.groups) {
    uint8_t* t = p.scales + ((tile * p.groups + seg * 2 + lane) * p.halves + half) * kScaleTile + r32 * 16;
    const uint4 v = lane == 0 ? make_uint4(word[0][0], word[1][0], word[2][0], word[3][0])
                              : make_uint4(word[0][1], word[1][1], word[2][1], word[3][1]);
    *reinterpret_cast<uint4*>(t) = v;
  }
}

// Two e2m1 codes as fp32.
__device__ __forceinline__ float2 from_e2m1x2(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 t, u;\n\tmov.b16 {t, u}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
      : "=r"(h)
      : "h"(static_cast<unsigned short>(byte)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

struct MxDequantParams {
  const uint8_t *codes, *scales;
  void* out;
  int64_t stride, rows;
  int32_t cols, groups, octets;  // octets: of eight columns in a row
};

template <class T, bool kVec>
__global__ void __launch_bounds__(kThreadsQ) mx_dequantize_kernel(MxDequantParams p) {
  const int64_t at = int64_t(blockIdx.x) * kThreadsQ + threadIdx.x;
  const int64_t r = at / p.octets;
  if (r >= p.rows) return;
  const int oct = int(at - r * p.octets), c = oct * 8, b = oct >> 2;
  const int64_t row_bytes = mx_cdiv(p.cols, kMxBlock) * 16;
  const uint32_t codes = *reinterpret_cast<const uint32_t*>(p.codes + r * row_bytes + oct * 4);
  const uint32_t s =
      p.scales[((r >> 7) * p.groups + (b >> 2)) * kScaleTile + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (b & 3)];
  const float scale = scale_value(s);
  Vec<T, 8> v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 x = from_e2m1x2((codes >> (8 * e)) & 0xffu);
    v.v[2 * e] = from_f32<T>(x.x * scale);
    v.v[2 * e + 1] = from_f32<T>(x.y * scale);
  }
  T* row = static_cast<T*>(p.out) + r * p.stride;
  if (kVec && c + 8 <= p.cols) {
    store_vec<T, 8>(row + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < p.cols) row[c + e] = v.v[e];
  }
}

bool whole_rows(const void* p, int64_t stride, int64_t rows, size_t es) {
  return aligned_to(p, 16) && (rows <= 1 || stride * int64_t(es) % 16 == 0);
}

template <class T>
cudaError_t launch_quantize(const MxQuantParams& p, cudaStream_t st) {
  const unsigned grid = unsigned(mx_cdiv(p.items, kWarpsQ));
  if (whole_rows(p.x, p.stride, p.rows, sizeof(T))) {
    mx_quantize_kernel<T, true><<<grid, kThreadsQ, 0, st>>>(p);
  } else {
    mx_quantize_kernel<T, false><<<grid, kThreadsQ, 0, st>>>(p);
  }
  return cudaGetLastError();
}
template <class T>
cudaError_t launch_dequantize(const MxDequantParams& p, cudaStream_t st) {
  const unsigned grid = unsigned(mx_cdiv(p.rows * p.octets, kThreadsQ));
  if (whole_rows(p.out, p.stride, p.rows, sizeof(T))) {
    mx_dequantize_kernel<T, true><<<grid, kThreadsQ, 0, st>>>(p);
  } else {
    mx_dequantize_kernel<T, false><<<grid, kThreadsQ, 0, st>>>(p);
  }
  return cudaGetLastError();
}

int validate(const flce_mxfp4_problem* p) {
  if (!p) return FLCE_ERR_INVALID_ARG;
  if (p->rows < 0 || p->rows > INT32_MAX - 256 || p->cols < 1 || p->cols > (1 << 24) || p->stride < 0)
    return FLCE_ERR_INVALID_ARG;
  // one warp for four rows of 256 columns
  if (mx_cdiv(p->rows, 128) * 32 * mx_cdiv(p->cols, kSeg) > int64_t(INT32_MAX) * kWarpsQ ||
      p->rows * mx_cdiv(p->cols, 8) > int64_t(INT32_MAX) * kThreadsQ)
    return FLCE_ERR_INVALID_ARG;
  if (!known_dtype(p->dtype)) return FLCE_ERR_UNSUPPORTED_DTYPE;
  return FLCE_OK;
}

}  // namespace

cudaError_t launch_mx_quantize(MxQuantParams p, int dtype, int64_t rows_padded, cudaStream_t st) {
  p.groups = int32_t(mx_groups(p.cols));
  p.segs = int32_t(mx_cdiv(p.cols, kSeg));
  p.halves = int32_t(mx_cdiv(p.tile_rows, 128));
  p.items = mx_cdiv(rows_padded, p.tile_rows) * p.halves * p.segs * 32;
  if (dtype == FLCE_F32) return launch_quantize<float>(p, st);
  if (dtype == FLCE_BF16) return launch_quantize<__nv_bfloat16>(p, st);
  return launch_quantize<__half>(p, st);
}

}  // namespace flce

using namespace flce;

extern "C" {

int flce_mxfp4_size(const flce_mxfp4_problem* problem, size_t* codes_bytes, size_t* scales_bytes) {
  if (!problem || !codes_bytes || !scales_bytes) return FLCE_ERR_INVALID_ARG;
  flce_mxfp4_problem p = *problem;
  p.stride = 0;
  p.dtype = FLCE_F32;
  FLCE_TRY(validate(&p));
  *codes_bytes = size_t(p.rows) * size_t(mx_row_bytes(p.cols));
  *scales_bytes = size_t(mx_cdiv(p.rows, 128)) * size_t(mx_groups(p.cols)) * kScaleTile;
  return FLCE_OK;
}

int flce_mxfp4_quantize(const flce_mxfp4_problem* problem, const void* x, void* codes, void* scales,
                        flce_stream_t stream) {
  const flce_mxfp4_problem* p = problem;
  FLCE_TRY(validate(p));
  if (p->rows == 0) return FLCE_OK;
  if (!x || !codes || !scales) return FLCE_ERR_INVALID_ARG;
  if (!aligned_to(x, elem_size(p->dtype)) || !aligned_to(codes, 16) || !aligned_to(scales, 16))
    return FLCE_ERR_MISALIGNED;
  DeviceInfo dev;
  FLCE_TRY(get_device(&dev));
  FLCE_TRY(check_local(dev, x, codes, scales));
  MxQuantParams q{};
  q.x = x;
  q.codes = static_cast<uint8_t*>(codes);
  q.scales = static_cast<uint8_t*>(scales);
  q.rows = p->rows;
  q.stride = p->stride;
  q.cols = int32_t(p->cols);
  q.tile_rows = 128;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return logged(FLCE_LAUNCH_OTHER, st, [&] { return launch_mx_quantize(q, p->dtype, p->rows, st); });
}

int flce_mxfp4_dequantize(const flce_mxfp4_problem* problem, const void* codes, const void* scales, void* out,
                          flce_stream_t stream) {
  const flce_mxfp4_problem* p = problem;
  FLCE_TRY(validate(p));
  if (p->rows == 0) return FLCE_OK;
  if (!out || !codes || !scales || (p->rows > 1 && p->stride < p->cols)) return FLCE_ERR_INVALID_ARG;
  if (!aligned_to(out, elem_size(p->dtype)) || !aligned_to(codes, 16) || !aligned_to(scales, 16))
    return FLCE_ERR_MISALIGNED;
  DeviceInfo dev;
  FLCE_TRY(get_device(&dev));
  FLCE_TRY(check_local(dev, out, codes, scales));
  MxDequantParams q{};
  q.codes = static_cast<const uint8_t*>(codes);
  q.scales = static_cast<const uint8_t*>(scales);
  q.out = out;
  q.stride = p->stride;
  q.rows = p->rows;
  q.cols = int32_t(p->cols);
  q.groups = int32_t(mx_groups(p->cols));
  q.octets = int32_t(mx_cdiv(p->cols, 8));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return logged(FLCE_LAUNCH_OTHER, st, [&] {
    if (p->dtype == FLCE_F32) return launch_dequantize<float>(q, st);
    if (p->dtype == FLCE_BF16) return launch_dequantize<__nv_bfloat16>(q, st);
    return launch_dequantize<__half>(q, st);
  });
}

}  // extern "C"
