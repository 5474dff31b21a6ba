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

// A warp's work: rows r32, r32 + 32, ... of a scale tile (128 rows), a stretch of
// columns.  r32 is the fastest index: a block's warps share scale tiles.
struct Item {
  int r32, seg, half;
  int64_t tile;
  __device__ __forceinline__ Item(int64_t i, int segs, int halves) {
    r32 = int(i & 31);
    const uint32_t rest = uint32_t(i >> 5), th = rest / uint32_t(segs);
    seg = int(rest - th * uint32_t(segs));
    const uint32_t t = th / uint32_t(halves);
    half = int(th - t * uint32_t(halves));
    tile = t;
  }
};

// The largest |x| of three (|a| is one already), a NaN if there is one.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return y;
}

// Eight values of a block's row segment as codes, at `to` with its scale's byte in
// place in `word`; a lane has eight adjacent columns, a block is four lanes'.
__device__ __forceinline__ void quantize_adjacent(float (&y)[8], bool write, uint32_t* to, uint32_t& word) {
  const int lane = threadIdx.x & 31;
  float m = max_abs(max_abs(max_abs(fabsf(y[0]), y[1], y[2]), y[3], y[4]), y[5], y[6]);
  m = max_abs(m, y[7], __shfl_xor_sync(kFull, max_abs(m, y[7], y[7]), 1));
  m = max_abs(m, m, __shfl_xor_sync(kFull, m, 2));
  const uint32_t s = scale_byte(__float_as_uint(m));
  const float inv = inverse_scale(s);
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] *= inv;
  const uint32_t codes = s == 255u ? 0u : to_e2m1x8(y);
  if (write) *to = codes;
  uint32_t w = s << (8 * ((lane >> 2) & 3));  // blocks of no column have m = 0 and s = 0
  w |= __shfl_xor_sync(kFull, w, 4);
  word = w | __shfl_xor_sync(kFull, w, 8);
}
__device__ __forceinline__ void copy_async16(void* dst, const void* src, int bytes) {  // the rest of 16 as zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}

// kVec: rows start on 16-byte boundaries.  A warp keeps the rows of kItems - 1 further
// items under way, copied into shared memory of its own (each lane reads what it
// copied).  128256 x 2048 bf16, where the copy rate gives 98 us: 137 us; with loads to
// registers, 80 KB of them under way on an SM, 170.
// Else the warp loads 32 adjacent elements at a time and passes them on through shared
// memory: 1380 x 9469 bf16 9.4 us, the copy rate gives 4.9.  (Asynchronous copies of 4
// or 8 bytes where rows start on such: 20000 x 1027 fp32 36 us in place of 20, 28992 x
// 396 fp16 10.7 in place of 10.1.)
template <class T>
constexpr int kItems = sizeof(T) == 2 ? 4 : 2;
template <class T>
constexpr int kItemBytes = 4 * 32 * 8 * int(sizeof(T));
template <class T, bool kVec>
__global__ void __launch_bounds__(kThreadsQ) mx_quantize_kernel(MxQuantParams p) {
  constexpr int kSlots = kVec ? kItems<T> : 1;
  extern __shared__ __align__(16) uint8_t ring[];
  griddep_release();
  if (p.status && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row_bytes = (p.cols + kMxBlock - 1) / kMxBlock * 16;
  const int64_t step = int64_t(gridDim.x) * kWarpsQ, first = int64_t(blockIdx.x) * kWarpsQ + warp;
  // the item's rows r0, r0 + 32, ...: how many there are
  auto rows_of = [&](const Item& it, int64_t& r0) {
    r0 = it.tile * p.tile_rows + it.half * 128 + it.r32;
    return int(min((min(int64_t(p.tile_rows) * (it.tile + 1), p.rows) - r0 + 31) / 32, int64_t(4)));
  };
  Vec<T, 8>* mine = reinterpret_cast<Vec<T, 8>*>(ring) + warp * kSlots * 128 + lane;  // [item][row][lane]
  auto copy = [&](int64_t item, int slot) {
    if (item < p.items) {
      const Item it(item, p.segs, p.halves);
      int64_t r0;
      const int rows = rows_of(it, r0), c = it.seg * kSeg + lane * 8;
      const int bytes = max(0, min(8, p.cols - c)) * int(sizeof(T));
      const T* row = static_cast<const T*>(p.x) + r0 * p.stride + c;
#pragma unroll
      for (int i = 0; i < 4; ++i, row += 32 * p.stride) {
        const int n = i < rows ? bytes : 0;
        uint8_t* dst = reinterpret_cast<uint8_t*>(mine + slot * 128 + i * 32);
#pragma unroll
        for (int o = 0; o < 8 * int(sizeof(T)); o += 16)
          copy_async16(dst + o, n > o ? reinterpret_cast<const uint8_t*>(row) + o : static_cast<const uint8_t*>(p.x),
                            max(0, min(n - o, 16)));
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if constexpr (kVec) {
#pragma unroll
    for (int k = 0; k < kSlots - 1; ++k) copy(first + k * step, k);
  }
  int slot = 0;
  for (int64_t item = first; item < p.items; item += step) {
    const Item it(item, p.segs, p.halves);
    const int col0 = it.seg * kSeg;
    int64_t r0;
    const int rows = rows_of(it, r0);
    if constexpr (kVec) {
      copy(item + (kSlots - 1) * step, (slot + kSlots - 1) % kSlots);
      asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
    } else {
      T x[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const T* row = static_cast<const T*>(p.x) + (r0 + 32 * i) * p.stride;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = col0 + e * 32 + lane;
          x[i][e] = i < rows && c < p.cols ? row[c] : from_f32<T>(0.f);
        }
      }
      __syncwarp();  // the last item's are read
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) reinterpret_cast<T*>(mine - lane + i * 32)[e * 32 + lane] = x[i][e];
      __syncwarp();
    }
    uint32_t word[4];  // the scale bytes of the row's four blocks of the lane's group
    uint8_t* to = p.codes + r0 * row_bytes + col0 / 2;
#pragma unroll
    for (int i = 0; i < 4; ++i, to += int64_t(32) * row_bytes) {
      float y[8];
      const Vec<T, 8> x = mine[slot * 128 + i * 32];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = to_f32(x.v[e]);
      quantize_adjacent(y, i < rows && col0 + (lane & ~3) * 8 < p.cols, reinterpret_cast<uint32_t*>(to) + lane, word[i]);
    }
    // a group's tile: 16 bytes for r32, four for each of the rows
    const int group = it.seg * 2 + (lane >> 4);
    if ((lane & 15) == 0 && group < p.groups) {
      uint8_t* t = p.scales + ((it.tile * p.groups + group) * p.halves + it.half) * kScaleTile + it.r32 * 16;
      *reinterpret_cast<uint4*>(t) = make_uint4(word[0], word[1], word[2], word[3]);
    }
    slot = (slot + 1) % kSlots;
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
  int64_t stride, rows, items;
  int32_t cols, groups, segs;
};

// The same warps' work as above; a lane has eight adjacent columns.  kVec: the rows
// start on 16-byte boundaries; else the warp passes each row on through shared memory
// and stores 32 adjacent elements at a time (1380 x 9469 bf16: 7.4 us,
// the copy rate gives 4.9; there and back 17, and 62 where lanes stored their own
// elements one by one and a block's maximum was taken over a warp).
template <class T, bool kVec>
__global__ void __launch_bounds__(kThreadsQ) mx_dequantize_kernel(MxDequantParams p) {
  __shared__ __align__(16) T turned[kVec ? 1 : kWarpsQ][kVec ? 8 : kSeg];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = int64_t(blockIdx.x) * kWarpsQ + warp;
  if (item >= p.items) return;
  const Item it(item, p.segs, 1);
  const int c = it.seg * kSeg + lane * 8, group = it.seg * 2 + (lane >> 4);
  const bool in = c < p.cols;
  if (kVec && !in) return;
  const int64_t row_bytes = mx_cdiv(p.cols, kMxBlock) * 16, r0 = it.tile * 128 + it.r32;
  uint4 s4 = make_uint4(0u, 0u, 0u, 0u);
  if (in) s4 = *reinterpret_cast<const uint4*>(p.scales + (it.tile * p.groups + group) * kScaleTile + it.r32 * 16);
  const uint32_t words[4] = {s4.x, s4.y, s4.z, s4.w};
  uint32_t codes[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    codes[i] = in && r0 + 32 * i < p.rows ? *reinterpret_cast<const uint32_t*>(p.codes + (r0 + 32 * i) * row_bytes + c / 2) : 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 32 * i;
    if (r >= p.rows) return;
    const float scale = scale_value((words[i] >> (8 * ((lane >> 2) & 3))) & 0xffu);
    Vec<T, 8> v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = from_e2m1x2((codes[i] >> (8 * e)) & 0xffu);
      v.v[2 * e] = from_f32<T>(x.x * scale);
      v.v[2 * e + 1] = from_f32<T>(x.y * scale);
    }
    T* row = static_cast<T*>(p.out) + r * p.stride;
    if constexpr (kVec) {
      if (c + 8 <= p.cols) {
        store_vec<T, 8>(row + c, v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < p.cols) row[c + e] = v.v[e];
      }
    } else {
      __syncwarp();  // the last row's are read
      store_vec<T, 8>(&turned[warp][lane * 8], v);
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int col = it.seg * kSeg + e * 32 + lane;
        if (col < p.cols) row[col] = turned[warp][e * 32 + lane];
      }
    }
  }
}

bool whole_rows(const void* p, int64_t stride, int64_t rows, size_t es) {
  return aligned_to(p, 16) && (rows <= 1 || stride * int64_t(es) % 16 == 0);
}

template <class T, bool kVec>
cudaError_t launch_quantize(const MxQuantParams& p, int num_sms, cudaStream_t st) {
  auto kern = mx_quantize_kernel<T, kVec>;
  constexpr int smem = kWarpsQ * (kVec ? kItems<T> : 1) * kItemBytes<T>;  // kVec: three blocks on an SM
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t grid = std::min<int64_t>(mx_cdiv(p.items, kWarpsQ), int64_t(num_sms) * (kVec ? 3 : 32));
  kern<<<unsigned(grid), kThreadsQ, smem, st>>>(p);
  return cudaGetLastError();
}
template <class T>
cudaError_t launch_quantize(const MxQuantParams& p, int num_sms, cudaStream_t st) {
  return whole_rows(p.x, p.stride, p.rows, sizeof(T)) ? launch_quantize<T, true>(p, num_sms, st)
                                                      : launch_quantize<T, false>(p, num_sms, st);
}
template <class T>
cudaError_t launch_dequantize(const MxDequantParams& p, cudaStream_t st) {
  const unsigned grid = unsigned(mx_cdiv(p.items, kWarpsQ));
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
  if (mx_cdiv(p->rows, 128) * mx_cdiv(p->cols, kSeg) > (1 << 28)) return FLCE_ERR_INVALID_ARG;  // a grid's blocks
  if (!known_dtype(p->dtype)) return FLCE_ERR_UNSUPPORTED_DTYPE;
  return FLCE_OK;
}

}  // namespace

cudaError_t launch_mx_quantize(MxQuantParams p, int dtype, int64_t rows_padded, int num_sms, cudaStream_t st) {
  p.groups = int32_t(mx_groups(p.cols));
  p.segs = int32_t(mx_cdiv(p.cols, kSeg));
  p.halves = int32_t(mx_cdiv(p.tile_rows, 128));
  p.items = mx_cdiv(rows_padded, p.tile_rows) * p.halves * p.segs * 32;
  if (dtype == FLCE_F32) return launch_quantize<float>(p, num_sms, st);
  if (dtype == FLCE_BF16) return launch_quantize<__nv_bfloat16>(p, num_sms, st);
  return launch_quantize<__half>(p, num_sms, st);
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
  return logged(FLCE_LAUNCH_OTHER, st, [&] { return launch_mx_quantize(q, p->dtype, p->rows, dev.num_sms, st); });
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
  q.segs = int32_t(mx_cdiv(p->cols, kSeg));
  q.items = mx_cdiv(p->rows, 128) * q.segs * 32;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return logged(FLCE_LAUNCH_OTHER, st, [&] {
    if (p->dtype == FLCE_F32) return launch_dequantize<float>(q, st);
    if (p->dtype == FLCE_BF16) return launch_dequantize<__nv_bfloat16>(q, st);
    return launch_dequantize<__half>(q, st);
  });
}

}  // extern "C"
