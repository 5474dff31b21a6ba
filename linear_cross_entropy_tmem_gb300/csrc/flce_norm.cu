// flce_norm.cu — the norm's C entry points, and the reduction of its dweight.
#include <algorithm>
#include <cmath>

#include "flce_host.h"
#include "flce_norm.cuh"

namespace flce {
namespace {

// dw[j] = sum over blocks of part[b][j], in a fixed order: 32 columns per
// block, warp k takes the partial rows k, k + 32, ...
constexpr int kReduceWarps = 32;
__global__ void __launch_bounds__(kReduceWarps * 32) dweight_reduce_kernel(const float* part, int blocks, int cols,
                                                                           void* dw, int dtype) {
  __shared__ float s[kReduceWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  griddep_wait();  // the partial rows are there
  float a = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int b = warp; b < blocks; b += kReduceWarps) a += part[int64_t(b) * cols + c];
  }
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
// Partial dweight rows, at most; one per block of the backward.
constexpr int kMaxBwdBlocks = 2048;
constexpr int kLoopSplits = 64;  // partial rows of a row too wide for registers

// Whether each row starts equally far past a 16-byte boundary in all of the
// call's matrices, in elements modulo the vector's width.
struct Phases {
  int vec;
  bool same = true, first = true;
  int64_t phase = 0, stride = 0;
  bool shifted = false;
  void add(const void* p, int64_t row_stride, int64_t rows, size_t elem) {
    if (!p) return;
    const int64_t a = int64_t(reinterpret_cast<uintptr_t>(p) / elem % unsigned(vec)), s = rows > 1 ? row_stride % vec : 0;
    if (first) {
      phase = a;
      stride = s;
      first = false;
      shifted = a != 0 || s != 0;
    }
    same = same && a == phase && s == stride;
  }
  RowPlan plan(int64_t cols) const { return same ? plan_row(cols, vec, shifted) : plan_row(cols, 1, false); }
};

// Blocks of a row kernel: `waves` times what runs at once (`per_sm` blocks of
// the form's most threads, as far as shared memory goes), in a multiple of 8 so
// that a block's rows all have one shift; fewer waves where a block would get
// less than kRowsPerBlock rows, and whole ones (8192 x 2048 fp16 with the 8-bit
// output: 1.7 us of 28 less with one wave than with 1.1).  At 16384 x 4096 bf16 the
// forward takes 96 us with one wave and 82 us with four: SMs do not all see
// memory alike, and later blocks go where earlier ones end.  The backward takes
// 94 us with one and 115 us with four, as each block also writes a partial row.
constexpr int kRowsPerBlock = 6;
int row_blocks(const RowPlan& pl, int64_t rows, int num_sms, int per_sm, int smem, int waves) {
  constexpr int kSmemPerSm = 227 * 1024, kOwn = 1280;  // of a block besides: its static and the system's
  const int per_block = pl.form == kWarp ? kWarpRowBlock / 32 : 1;
  const int64_t want = (rows + per_block - 1) / per_block;
  const int64_t once = int64_t(num_sms) * std::max(1, std::min(per_sm * row_threads(pl.form) / pl.threads, kSmemPerSm / (smem + kOwn)));
  const int64_t most = once * std::max<int64_t>(1, std::min<int64_t>(waves, want / kRowsPerBlock / once));
  return int(std::min(want, std::max<int64_t>(8, most / 8 * 8)));
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
  Phases ph{vec_of(es, er)};
  ph.add(x, p->x_stride, p->rows, es);
  ph.add(residual, p->residual_stride, p->rows, er);
  ph.add(h, p->h_stride, p->rows, er);
  ph.add(y, p->y_stride, p->rows, ey);
  const RowPlan pl = ph.plan(p->cols);
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
  // A group's vectors are neighbouring lanes' where it is a power of two of
  // them, and rows are not shifted; then no group's place depends on the row.
  const int lanes = n.group / pl.vec;
  if (pl.vec > 1 && !pl.ragged && n.group % pl.vec == 0 && lanes <= 32 && (lanes & (lanes - 1)) == 0) n.lanes = lanes;
  n.eps = p->eps;
  n.offset = p->weight_offset;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int grid = row_blocks(pl, p->rows, dev.num_sms, fwd_blocks(pl.form, pl.ragged), row_smem(pl, es + er), 4);
  // 16-bit weights (or none) with no offset: their products with a 16-bit h are exact in fp32
  const bool exact = er == 2 && (!weight || p->weight_dtype != FLCE_F32) && p->weight_offset == 0.f;
  const auto launch = !fp8 ? launch_norm_fwd : exact ? launch_norm_fwd_fp8_exact : launch_norm_fwd_fp8_left;
  return logged(FLCE_LAUNCH_OTHER, st, [&] { return launch(n, p->dtype, p->residual_dtype, pl, grid, st); });
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
  // a partial dweight row per block; rows over 16 elements x 1024 threads take kLoopSplits
  const int64_t blocks = problem->cols > 16 * kMaxThreads ? kLoopSplits : kMaxBwdBlocks;
  *bytes = size_t(std::min<int64_t>(problem->rows, blocks)) * size_t(problem->cols) * 4 + 256;
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
    Phases ph{vec_of(es, er)};
    ph.add(dy, n.dys, n.rows, es);
    ph.add(h, n.hs, n.rows, er);
    ph.add(dh, n.dhs, n.rows, er);
    ph.add(dx, n.dxs, n.rows, es);
    ph.add(dresidual, n.drs, n.rows, er);
    const RowPlan pl = ph.plan(n.cols);
    blocks = pl.form == kLoop
                 ? int(std::min<int64_t>(n.rows, kLoopSplits))
                 : std::min(kMaxBwdBlocks, row_blocks(pl, n.rows, dev.num_sms, bwd_blocks(pl.form, pl.ragged, pl.vec * pl.nv),
                                                      row_smem(pl, es + 2 * er), 1));
    FLCE_TRY(logged(FLCE_LAUNCH_OTHER, st,
                    [&] { return launch_norm_bwd(n, p->dtype, p->residual_dtype, pl, blocks, st); }));
  }
  if (!dweight) return FLCE_OK;
  return logged(FLCE_LAUNCH_OTHER, st, [&] {
    return launch_dependent(dweight_reduce_kernel, unsigned((n.cols + 31) / 32), kReduceWarps * 32, st,
                            static_cast<const float*>(n.part), blocks, n.cols, dweight, p->weight_dtype);
  });
}

}  // extern "C"
