// flce_host.h — host services shared by the C entry points (internal): device
// information, pointer checks, and the launch log and counter.  Defined in
// flce_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "flce.h"
#include "flce_testing.h"

#define FLCE_TRY(expr)               \
  do {                               \
    const int rc_ = (expr);          \
    if (rc_ != FLCE_OK) return rc_;  \
  } while (0)

namespace flce {

struct DeviceInfo {
  bool init = false;
  int index = 0;
  int num_sms = 0;
  int major = 0, minor = 0;
};

// The current device (cached per index); FLCE_ERR_UNSUPPORTED_DEVICE off sm_103.
int get_device(DeviceInfo* out);

// FLCE_OK for nullptr and for memory of the current device (device or managed
// memory), FLCE_ERR_INVALID_ARG for anything else.
int check_local(const DeviceInfo& dev, const void* p);
template <class... P>
int check_local(const DeviceInfo& dev, const void* p, P... rest) {
  FLCE_TRY(check_local(dev, p));
  return check_local(dev, rest...);
}

// The same for many pointers of one call: one inside an allocation that the call
// has already found local needs no query.
struct LocalRanges {
  uintptr_t begin = 0, end = 0;  // the last allocation found local
};
int check_local(const DeviceInfo& dev, const void* p, LocalRanges* known);

// 2-D map of bytes with the 128-byte swizzle (rows `row_bytes` apart, boxes of
// box_inner bytes x box_outer rows); what lies outside reads as 0.
int make_byte_map(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows, uint32_t box_inner,
                  uint32_t box_outer);

int log_begin(cudaStream_t st, flce_launch_record** rec);
int log_end(int kind, cudaStream_t st, flce_launch_record* rec);

// Runs `launch` (returning cudaError_t) on `st`, bracketed by logged events
// when the launch log is on; counts the launch.
template <class F>
int logged(int kind, cudaStream_t st, F&& launch) {
  flce_launch_record* rec = nullptr;
  FLCE_TRY(log_begin(st, &rec));
  if (launch() != cudaSuccess) return FLCE_ERR_CUDA;
  return log_end(kind, st, rec);
}

}  // namespace flce
