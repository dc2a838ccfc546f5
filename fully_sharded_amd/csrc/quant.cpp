// Host side of the all-gather in 8 bits: the choice of matrices, the work
// table, and the C entry points' checks and launches.
#include "quant.hpp"

#include <algorithm>
#include <new>

#include "checks.hpp"
#include "ops.hpp"

namespace fsdp {
namespace {

// Codes of all receivers that the memory-side cache (256 MiB) still holds.
constexpr int64_t kCached = int64_t(1) << 28;

// Rows per item of a matrix: about 4,096 elements, a multiple of the four
// waves that share it.
int64_t item_rows(int64_t cols) {
  if (cols > kWaveRow) return 1;
  return std::min<int64_t>(64, std::max<int64_t>(4, 4096 / cols / 4 * 4));
}

}  // namespace

fsdp_status build_quant(const fsdp_plan* plan, int32_t n_params, const int32_t* params,
                        fsdp_quant* qu) {
  qu->R = plan->R;
  qu->T = plan->T;
  qu->S = plan->S;
  const int32_t n_all = static_cast<int32_t>(plan->params.size());
  std::vector<char> chosen(n_all, 0);
  for (int32_t k = 0; k < n_params; ++k) {
    const int32_t p = params[k];
    if (p < 0 || p >= n_all || chosen[p] || plan->shapes[p].size() < 2)
      return FSDP_ERR_INVALID_ARG;
    if (plan->shapes[p].back() > kMaxCols) return FSDP_ERR_UNSUPPORTED;
    chosen[p] = 1;
  }
  // the number of items first: a table that is refused is not built
  int64_t n_items = 0;
  for (int32_t p = 0; p < n_all; ++p) {
    const Param& q = plan->params[p];
    const int64_t cols = plan->shapes[p].back();
    const int64_t pieces = plan->layout == FSDP_LAYOUT_FLAT ? 1 : plan->R;
    n_items += (chosen[p] ? q.numel / cols / item_rows(cols) : q.numel / kRestItem) + pieces;
    if (n_items > kMaxItems) return FSDP_ERR_UNSUPPORTED;
  }
  qu->items.reserve(static_cast<size_t>(n_items));
  for (int32_t p = 0; p < n_all; ++p) {
    const Param& q = plan->params[p];
    const int64_t cols = chosen[p] ? plan->shapes[p].back() : 1;
    const int64_t pitch = chosen[p] ? (cols + 15) / 16 * 16 : 0;
    const int64_t per = chosen[p] ? item_rows(cols) : kRestItem;
    const int64_t rows = q.numel / cols;
    const QuantParam at = chosen[p] ? QuantParam{qu->code_bytes, rows, cols, pitch, qu->n_scales}
                                    : QuantParam{-1, qu->n_rest, q.numel, 0, 0};
    qu->params.push_back(at);
    // rows [first, first + count) of the parameter, contiguous from src on
    auto piece = [&](int64_t first, int64_t count, int64_t src) {
      for (int64_t i = 0; i < count; i += per) {
        const int64_t n = std::min(per, count - i), row = first + i;
        QuantItem w{};
        w.src = src + i * cols;
        w.flat = q.flat_off + row * cols;
        if (chosen[p]) {
          w.to = at.to + row * pitch;
          w.scale = at.scale + row;
          w.n_rows = static_cast<int32_t>(n);
          w.cols = static_cast<int32_t>(cols);
          w.pitch = static_cast<int32_t>(pitch);
        } else {
          w.to = at.rows + row;
          w.n_rows = 1;
          w.cols = static_cast<int32_t>(n);
        }
        qu->items.push_back(w);
      }
    };
    if (plan->layout == FSDP_LAYOUT_FLAT) {
      piece(0, rows, q.flat_off);  // the shards are the unit, one after the other
    } else {
      const int64_t each = q.row / cols;  // rows per entry of the first dimension
      for (int64_t r = 0; r < plan->R; ++r) {
        const int64_t lo = std::min(r * q.k, q.d0), hi = std::min((r + 1) * q.k, q.d0);
        piece(lo * each, (hi - lo) * each, r * plan->S + q.shard_off);
      }
    }
    if (chosen[p]) {
      qu->code_bytes += rows * pitch;
      qu->n_scales += rows;
    } else {
      qu->n_rest += q.numel;
    }
  }
  return FSDP_OK;
}

}  // namespace fsdp

using namespace fsdp;

fsdp_status fsdp_quant::device(const QuantItem** out) const {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) {
    (void)hipGetLastError();
    return FSDP_ERR_HIP;
  }
  std::lock_guard<std::mutex> lock(mu_);
  auto it = dev_.find(dev);
  if (it == dev_.end()) {
    void* mem = nullptr;
    const size_t bytes = items.size() * sizeof(QuantItem);
    if (hipMalloc(&mem, bytes) != hipSuccess) {
      (void)hipGetLastError();
      return FSDP_ERR_OUT_OF_MEMORY;
    }
    if (hipMemcpy(mem, items.data(), bytes, hipMemcpyHostToDevice) != hipSuccess) {
      (void)hipGetLastError();
      (void)hipFree(mem);
      return FSDP_ERR_HIP;
    }
    it = dev_.emplace(dev, mem).first;
  }
  *out = static_cast<const QuantItem*>(it->second);
  return FSDP_OK;
}

fsdp_quant::~fsdp_quant() {
  for (auto& kv : dev_) (void)hipFree(kv.second);
}

namespace {

// A list of ranges of any length: three buffers for each of 64 receivers, and
// what they are made from.
struct Many {
  Range r[4 * FSDP_MAX_RANKS + 1];
  size_t n = 0;
  void add(const void* p, int64_t bytes) { r[n++] = range_of(p, bytes); }
};

bool meet(const Many& writes, const Many& reads) {
  for (size_t i = 0; i < writes.n; ++i) {
    for (size_t j = 0; j < reads.n; ++j)
      if (overlap(writes.r[i], reads.r[j])) return true;
    for (size_t j = i + 1; j < writes.n; ++j)
      if (overlap(writes.r[i], writes.r[j])) return true;
  }
  return false;
}

// One receiver's buffers, checked and added to both lists.
fsdp_status take(const fsdp_quant* qu, const void* codes, const void* scales, const void* rest,
                 int64_t es, QuantBuffers* b, Many* ranges) {
  if (!codes || !scales || (qu->n_rest && !rest) || !aligned(codes, 16) || !aligned(scales, 4) ||
      !aligned(rest, es))
    return FSDP_ERR_INVALID_ARG;
  b->codes.p[b->n] = codes;
  b->scales.p[b->n] = scales;
  b->rest.p[b->n] = rest;
  ++b->n;
  ranges->add(codes, qu->code_bytes);
  ranges->add(scales, qu->n_scales * 4);
  ranges->add(rest, qu->n_rest * es);
  return FSDP_OK;
}

}  // namespace

extern "C" {

fsdp_status fsdp_quant_plan(const fsdp_plan* plan, int32_t n_params, const int32_t* params,
                            fsdp_quant** out) {
  if (!out) return FSDP_ERR_INVALID_ARG;
  *out = nullptr;
  if (!plan || n_params < 1 || !params) return FSDP_ERR_INVALID_ARG;
  fsdp_quant* qu = new (std::nothrow) fsdp_quant();
  if (!qu) return FSDP_ERR_OUT_OF_MEMORY;
  const fsdp_status st = guarded([&] { return build_quant(plan, n_params, params, qu); });
  if (st != FSDP_OK) {
    delete qu;
    return st;
  }
  *out = qu;
  return FSDP_OK;
}

void fsdp_quant_destroy(fsdp_quant* qu) { delete qu; }

fsdp_status fsdp_quant_prepare(const fsdp_quant* qu, void* stream) {
  (void)stream;
  return guarded([&]() -> fsdp_status {
    if (!qu) return FSDP_ERR_INVALID_ARG;
    const QuantItem* items = nullptr;
    return qu->device(&items);
  });
}

fsdp_status fsdp_quant_sizes(const fsdp_quant* qu, int64_t* out) {
  if (!qu || !out) return FSDP_ERR_INVALID_ARG;
  out[0] = qu->code_bytes;
  out[1] = qu->n_scales;
  out[2] = qu->n_rest;
  return FSDP_OK;
}

fsdp_status fsdp_quant_param(const fsdp_quant* qu, int32_t p, int64_t* out) {
  if (!qu || !out || p < 0 || p >= static_cast<int32_t>(qu->params.size()))
    return FSDP_ERR_INVALID_ARG;
  const QuantParam& q = qu->params[p];
  out[0] = q.to;
  out[1] = q.rows;
  out[2] = q.cols;
  out[3] = q.pitch;
  out[4] = q.scale;
  return FSDP_OK;
}

fsdp_status fsdp_gather_quantize(const fsdp_quant* qu, const void* shards, int32_t dtype,
                                 int8_t* const* codes, float* const* scales, void* const* rest,
                                 void* stream) {
  return guarded([&]() -> fsdp_status {
    if (!qu || !shards || !valid_dtype(dtype) || !codes || !scales || (qu->n_rest && !rest))
      return FSDP_ERR_INVALID_ARG;
    const int64_t es = dtype_size(dtype);
    if (!aligned(shards, es)) return FSDP_ERR_INVALID_ARG;
    QuantBuffers to;
    Many reads, writes;
    reads.add(shards, qu->R * qu->S * es);
    for (int r = 0; r < qu->R; ++r) {
      if (!codes[r]) continue;
      const fsdp_status st =
          take(qu, codes[r], scales[r], qu->n_rest ? rest[r] : nullptr, es, &to, &writes);
      if (st != FSDP_OK) return st;
    }
    if (meet(writes, reads)) return FSDP_ERR_INVALID_ARG;
    if (!to.n) return FSDP_OK;
    const QuantItem* items = nullptr;
    const fsdp_status st = qu->device(&items);
    if (st != FSDP_OK) return st;
    return status_of(launch_gather_quantize(items, static_cast<int64_t>(qu->items.size()), shards,
                                            dtype, to, to.n * qu->code_bytes > kCached,
                                            StreamSink(stream)));
  });
}

fsdp_status fsdp_dequantize(const fsdp_quant* qu, const int8_t* const* codes,
                            const float* const* scales, const void* const* rest,
                            int32_t rest_dtype, void* const* full_out, int32_t out_dtype,
                            void* stream) {
  return guarded([&]() -> fsdp_status {
    if (!qu || !codes || !scales || (qu->n_rest && !rest) || !full_out ||
        !valid_dtype(rest_dtype) || !valid_dtype(out_dtype))
      return FSDP_ERR_INVALID_ARG;
    const int64_t es = dtype_size(out_dtype);
    QuantBuffers from;
    PtrArray full{};
    Many reads, writes;
    for (int r = 0; r < qu->R; ++r) {
      if (!full_out[r]) continue;
      if (!aligned(full_out[r], es)) return FSDP_ERR_INVALID_ARG;
      full.p[from.n] = full_out[r];
      writes.add(full_out[r], qu->T * es);
      const fsdp_status st = take(qu, codes[r], scales[r], qu->n_rest ? rest[r] : nullptr,
                                  dtype_size(rest_dtype), &from, &reads);
      if (st != FSDP_OK) return st;
    }
    if (meet(writes, reads)) return FSDP_ERR_INVALID_ARG;
    if (!from.n) return FSDP_OK;
    const QuantItem* items = nullptr;
    const fsdp_status st = qu->device(&items);
    if (st != FSDP_OK) return st;
    return status_of(launch_dequantize(items, static_cast<int64_t>(qu->items.size()), from,
                                       rest_dtype, full, out_dtype, StreamSink(stream)));
  });
}

fsdp_status fsdp_quantize_rows(const void* x, int32_t dtype, int64_t rows, int64_t cols,
                               int64_t ldx, const float* channel, int64_t channel_stride,
                               const int32_t* offsets, int32_t groups, int8_t* codes, int64_t ldc,
                               float* scales, void* stream) {
  return guarded([&]() -> fsdp_status {
    if (!valid_dtype(dtype) || rows < 0 || cols < 1 || groups < 1 || ldx < cols ||
        channel_stride < 0 || ldc % 16 || ldc < (cols + 15) / 16 * 16)
      return FSDP_ERR_INVALID_ARG;
    if (!offsets && groups != 1) return FSDP_ERR_INVALID_ARG;
    const int64_t x_len = reach(rows, ldx, cols), c_len = reach(rows, ldc, (cols + 15) / 16 * 16);
    const int64_t channels = channel ? reach(groups, channel_stride, cols) : 0;
    if (rows > kMaxItems || cols > kMaxCols || groups > 65536 || x_len < 0 || c_len < 0 ||
        channels < 0)
      return FSDP_ERR_UNSUPPORTED;
    const int64_t es = dtype_size(dtype);
    if (!aligned(x, es) || !aligned(channel, 4) || !aligned(offsets, 4) || !aligned(codes, 16) ||
        !aligned(scales, 4))
      return FSDP_ERR_INVALID_ARG;
    if (rows == 0) return FSDP_OK;
    if (!x || !codes || !scales) return FSDP_ERR_INVALID_ARG;
    Many reads, writes;
    reads.add(x, x_len * es);
    reads.add(channel, channels * 4);
    reads.add(offsets, offsets ? (int64_t(groups) + 1) * 4 : 0);
    writes.add(codes, c_len);
    writes.add(scales, rows * 4);
    if (meet(writes, reads)) return FSDP_ERR_INVALID_ARG;
    const QuantizeRows a{x,   channel, offsets,        codes,
                         scales, ldx,  ldc,            channel_stride,
                         static_cast<int32_t>(rows),   static_cast<int32_t>(cols), groups};
    return status_of(launch_quantize_rows(a, dtype, StreamSink(stream)));
  });
}

}  // extern "C"
