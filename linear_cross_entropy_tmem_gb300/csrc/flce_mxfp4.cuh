// flce_mxfp4.cuh — the 4-bit block-scaled format: conversions, and how the head's
// product lays out its operands (internal).
#pragma once

#include "flce_device.cuh"
#include "flce_elem.cuh"
#include "flce_host.h"

namespace flce {

constexpr int kMxBlock = 32;        // columns that share a scale
constexpr int kScaleTile = 512;     // bytes of the scales of 128 rows x 4 blocks

__host__ __device__ constexpr int64_t mx_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
constexpr int64_t mx_blocks(int64_t cols) { return mx_cdiv(cols, kMxBlock); }
constexpr int64_t mx_row_bytes(int64_t cols) { return mx_blocks(cols) * (kMxBlock / 2); }
constexpr int64_t mx_groups(int64_t cols) { return mx_cdiv(mx_blocks(cols), 4); }

// Eight values to e2m1 (nearest even, saturating), the first in the lowest four bits.
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// A matrix's rows in tiles of `tile_rows`, whose scales take `halves` scale tiles of
// 128 rows for each four blocks: tile_rows = 128 and one of them for a weight, the
// product's tile of tokens for its hidden states.
struct MxQuantParams {
  const void* x;
  uint8_t *codes, *scales;
  int* status;          // set to 0, or nullptr
  int64_t rows, stride;
  int64_t items;        // warps' worth of work
  int32_t cols, tile_rows, halves, groups, segs;
};

cudaError_t launch_mx_quantize(MxQuantParams p, int dtype, int64_t rows_padded, int num_sms, cudaStream_t st);

}  // namespace flce
