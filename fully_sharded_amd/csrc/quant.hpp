// Internal structures of the all-gather in 8 bits: the chosen matrices of a
// unit, the work table of its kernels, and the launchers.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <map>
#include <mutex>
#include <vector>

#include "fsdp_mi355x.h"
#include "kernels.hpp"
#include "plan.hpp"

namespace fsdp {

// One workgroup's part of the unit: n_rows rows of cols elements, one after
// the other from src on in shard space and from flat on in the unit.  Of a
// chosen parameter: the first row's codes are at byte `to`, the next row's
// pitch bytes on, its scale at `scale`.  pitch 0: another parameter's elements
// (one row), which go to element `to` of rest.
struct alignas(16) QuantItem {
  int64_t src, flat, to, scale;
  int32_t n_rows, cols, pitch, unused;
};
static_assert(sizeof(QuantItem) == 48);

// Rows up to this many elements are a wave's each, longer ones a workgroup's.
constexpr int64_t kWaveRow = 2048;
// Elements of rest per item.
constexpr int64_t kRestItem = 2048;
constexpr int64_t kMaxCols = int64_t(1) << 30;

struct QuantParam {
  int64_t to, rows, cols, pitch, scale;  // of a chosen one
};

}  // namespace fsdp

struct fsdp_quant {
  int32_t R = 0;
  int64_t T = 0, S = 0;
  int64_t code_bytes = 0, n_scales = 0, n_rest = 0;
  std::vector<fsdp::QuantParam> params;  // every parameter's; others: to -1, rows = place in
                                         // rest, cols = elements
  std::vector<fsdp::QuantItem> items;

  // The table on the current device, uploaded on first use (synchronous;
  // freed with the object).
  fsdp_status device(const fsdp::QuantItem** out) const;
  ~fsdp_quant();

 private:
  mutable std::mutex mu_;
  mutable std::map<int, void*> dev_;
};

namespace fsdp {

fsdp_status build_quant(const fsdp_plan* plan, int32_t n_params, const int32_t* params,
                        fsdp_quant* qu);

// The receivers of a call, in their order, those that are skipped left out.
struct QuantBuffers {
  PtrArray codes, scales, rest;
  int n = 0;
};

// stream: the codes pass the caches by.
hipError_t launch_gather_quantize(const QuantItem* items, int64_t n, const void* shards, int dt,
                                  const QuantBuffers& to, bool stream, const Sink& sink);
hipError_t launch_dequantize(const QuantItem* items, int64_t n, const QuantBuffers& from,
                             int rest_dt, const PtrArray& full, int out_dt, const Sink& sink);

struct QuantizeRows {
  const void* x;
  const float* channel;    // null: none
  const int32_t* offsets;  // null: one group of all rows
  int8_t* codes;
  float* scales;
  int64_t ldx, ldc, channel_stride;
  int32_t rows, cols, groups;
};
hipError_t launch_quantize_rows(const QuantizeRows& a, int dt, const Sink& sink);

}  // namespace fsdp
