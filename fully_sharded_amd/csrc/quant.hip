// gfx950 kernels of the 8-bit codes: rows quantised (of a tensor, or of a
// unit's shards for every receiver) and units read back.  All are bound by
// memory; a row is read once, into registers, and its largest magnitude found
// before its codes are made.  Measured: 218M elements gathered for 8 ranks 384 us
// (5.7 TB/s; of fp32 483, 5.4 TB/s), read back by all 865 (6.0 TB/s; units' stores
// that stay in the caches 890; to fp32 1,927, 4.5 TB/s: a lane's 32 bytes in two
// stores); 3.1M for 4 ranks 6.6 and 8.0 us.  8192 rows of 4096 bf16 22.5 us (4.5
// TB/s; from the memory-side cache 19.5), of fp32 31 (5.4 TB/s), of 14336 bf16 64
// (5.5 TB/s; 70 with the row waiting as floats); times a channel's scales, which
// every row reads twice from L2, 31, 37 and 86.
#include <hip/hip_runtime.h>

#include "device.hpp"
#include "quant.hpp"

namespace fsdp {
namespace {

constexpr int kThreads = 256;
constexpr int kLane = 8;                     // adjacent elements of a lane
constexpr int kWavePass = 64 * kLane, kGroupPass = kThreads * kLane;
constexpr int kWavePasses = kWaveRow / kWavePass;
constexpr int kGroupPasses = 8;              // longer rows are read twice

// `have` of eight adjacent elements as they are, zeros behind; they may begin
// anywhere.  A row waits for its largest magnitude in this form: as floats,
// bf16 rows took twice the registers.
struct Raw16 {
  u4 v;
};
struct Raw32 {
  f4 v[2];
};
__device__ __forceinline__ Raw16 load8(const u16* p, int have) {
  typedef u4 any __attribute__((aligned(2)));
  Raw16 r;
  if (have >= 8) {
    r.v = *reinterpret_cast<const any*>(p);
  } else {
    r.v = u4{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k < have) r.v[k / 2] |= static_cast<uint32_t>(p[k]) << (k % 2 * 16);
  }
  return r;
}
__device__ __forceinline__ Raw32 load8(const float* p, int have) {
  typedef f4 any __attribute__((aligned(4)));
  Raw32 r;
  if (have >= 8) {
    r.v[0] = reinterpret_cast<const any*>(p)[0];
    r.v[1] = reinterpret_cast<const any*>(p)[1];
  } else {
    r.v[0] = r.v[1] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k < have) r.v[k / 4][k % 4] = p[k];
  }
  return r;
}
// Their values.
__device__ __forceinline__ void unpack(const Raw16& r, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(r.v[k] << 16);
    x[2 * k + 1] = __uint_as_float(r.v[k] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const Raw32& r, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = r.v[k / 4][k % 4];
}
__device__ __forceinline__ void store8(u16* p, int have, const float (&x)[8]) {
  typedef u4 any __attribute__((aligned(2)));
  u4 v;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = f32_to_bf16(x[2 * k]) | f32_to_bf16(x[2 * k + 1]) << 16;
  if (have >= 8) {
    __builtin_nontemporal_store(v, reinterpret_cast<any*>(p));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < have) p[k] = static_cast<u16>(v[k / 2] >> (k % 2 * 16));
  }
}
__device__ __forceinline__ void store8(float* p, int have, const float (&x)[8]) {
  typedef f4 any __attribute__((aligned(4)));
  if (have >= 8) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      __builtin_nontemporal_store(f4{x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]},
                                  reinterpret_cast<any*>(p) + h);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < have) p[k] = x[k];
  }
}

// Magnitudes compare as their bits do, infinities and NaN above all others.
__device__ __forceinline__ uint32_t largest(uint32_t m, const float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(x[k]) & 0x7fffffffu);
  return m;
}
__device__ __forceinline__ uint32_t wave_largest(uint32_t m) {
#pragma unroll
  for (int d = 32; d; d >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d)));
  return m;
}

// A row's scale, and what its entries are multiplied with.  One multiplication
// per entry in place of a division: of bf16 entries it gives the rounding of the
// exact x 127 / a but at a tie (x = a / 2 and the like), where it gives either
// neighbour.  (Entries are xs 2^e and as 2^f with 8-bit xs and as: x 127 / a is a
// tie or at least 1 / (2 as 2^j) > 2^-(9 + j) from one, j = f - e, while the three
// roundings move it by less than 2^(7 - j) 2^-21: each by 2^-24 of it at most, and
// the reciprocal of an a above 2^126, which is subnormal, by 2^-22.)
struct Scale {
  float scale, factor;
};
__device__ __forceinline__ Scale scale_of(uint32_t m) {
  if (m >= 0x7f800000u) return Scale{__uint_as_float(0x7fc00000u), 0.f};
  const float a = __uint_as_float(m);
  if (a < 0x1p-100f) return Scale{0.f, 0.f};
  return Scale{a * (1.f / 127.f), 1.f / a * 127.f};
}
__device__ __forceinline__ u2 codes_of(const float (&x)[8], float factor) {
  u2 v;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // (a factor of zero stands for codes of zero, whatever the entry is)
      const float c = factor == 0.f ? 0.f : rintf(x[4 * h + k] * factor);
      w |= (static_cast<uint32_t>(static_cast<int>(c)) & 0xffu) << (8 * k);
    }
    v[h] = w;
  }
  return v;
}

// One row by a wave (cols <= kWaveRow) or a workgroup.  get(first, have) loads
// eight entries, val(raw, first, have, x) are their values, put(first, codes)
// stores theirs and done(scale) the scale.
template <typename G, typename V, typename P, typename D>
__device__ __forceinline__ void wave_row(int cols, const G& get, const V& val, const P& put,
                                         const D& done) {
  const int lane = threadIdx.x & 63, padded = (cols + 15) / 16 * 16;
  decltype(get(0, 0)) raw[kWavePasses];
  uint32_t m = 0;
#pragma unroll
  for (int p = 0; p < kWavePasses; ++p) {
    const int at = p * kWavePass + lane * kLane;
    if (p * kWavePass < cols) raw[p] = get(at, cols - at);
  }
  float x[8];
#pragma unroll
  for (int p = 0; p < kWavePasses; ++p) {
    const int at = p * kWavePass + lane * kLane;
    if (p * kWavePass < cols) {
      val(raw[p], at, cols - at, x);
      m = largest(m, x);
    }
  }
  const Scale s = scale_of(wave_largest(m));
#pragma unroll
  for (int p = 0; p < kWavePasses; ++p) {
    const int at = p * kWavePass + lane * kLane;
    if (at < padded) {
      val(raw[p], at, cols - at, x);
      put(at, codes_of(x, s.factor));
    }
  }
  if (lane == 0) done(s.scale);
}

__device__ __forceinline__ uint32_t group_largest(uint32_t m) {
  __shared__ uint32_t part[kThreads / 64];
  m = wave_largest(m);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kThreads / 64; ++k) m = max(m, part[k]);
  return m;
}

template <typename G, typename V, typename P, typename D>
__device__ __forceinline__ void group_row(int cols, const G& get, const V& val, const P& put,
                                          const D& done) {
  const int padded = (cols + 15) / 16 * 16, tid = threadIdx.x;
  uint32_t m = 0;
  float x[8];
  if (cols <= kGroupPasses * kGroupPass) {
    decltype(get(0, 0)) raw[kGroupPasses];
#pragma unroll
    for (int p = 0; p < kGroupPasses; ++p) {
      const int at = p * kGroupPass + tid * kLane;
      if (p * kGroupPass < cols) raw[p] = get(at, cols - at);
    }
#pragma unroll
    for (int p = 0; p < kGroupPasses; ++p) {
      const int at = p * kGroupPass + tid * kLane;
      if (p * kGroupPass < cols) {
        val(raw[p], at, cols - at, x);
        m = largest(m, x);
      }
    }
    const Scale s = scale_of(group_largest(m));
#pragma unroll
    for (int p = 0; p < kGroupPasses; ++p) {
      const int at = p * kGroupPass + tid * kLane;
      if (at < padded) {
        val(raw[p], at, cols - at, x);
        put(at, codes_of(x, s.factor));
      }
    }
    if (tid == 0) done(s.scale);
  } else {
    for (int at = tid * kLane; at < cols; at += kGroupPass) {
      val(get(at, cols - at), at, cols - at, x);
      m = largest(m, x);
    }
    const Scale s = scale_of(group_largest(m));
    for (int at = tid * kLane; at < padded; at += kGroupPass) {
      val(get(at, cols - at), at, cols - at, x);
      put(at, codes_of(x, s.factor));
    }
    if (tid == 0) done(s.scale);
  }
}

// -------------------------------------------------------------- rows of x
template <typename T, bool WAVE>
__global__ __launch_bounds__(kThreads) void k_quantize_rows(QuantizeRows a) {
  const int row = WAVE ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (row >= a.rows) return;
  int g = 0;
  if (a.offsets) {
    // the group whose rows these are: the last that begins at or before it
    int lo = 0, hi = a.groups;
    if (row < a.offsets[0] || row >= a.offsets[hi]) return;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.offsets[mid] <= row)
        lo = mid;
      else
        hi = mid;
    }
    g = lo;
  }
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const float* ch = a.channel ? a.channel + g * a.channel_stride : nullptr;
  int8_t* to = a.codes + row * a.ldc;
  auto get = [&](int at, int have) { return load8(x + at, have); };
  auto val = [&](const auto& raw, int at, int have, float (&v)[8]) {
    unpack(raw, v);
    if (ch) {
      float c[8];
      unpack(load8(ch + at, have), c);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = v[k] * c[k];
    }
  };
  auto put = [&](int at, u2 v) { *reinterpret_cast<u2*>(to + at) = v; };
  auto done = [&](float s) { a.scales[row] = s; };
  if constexpr (WAVE)
    wave_row(a.cols, get, val, put, done);
  else
    group_row(a.cols, get, val, put, done);
}

// ------------------------------------------------------------- the gather
template <int N>
struct GatherArgs {
  const void* codes[N];
  const void* scales[N];
  const void* rest[N];
  int n;
};

// STREAM: codes that the caches cannot hold pass them by (8 receivers of 218M
// codes each 384 us and 396; 4 of 3.1M stay for their reader, 16.6 and 15.3 us
// with it).
template <typename T, int N, bool STREAM>
__global__ __launch_bounds__(kThreads) void k_gather_quantize(const QuantItem* __restrict__ items,
                                                              const T* __restrict__ shards,
                                                              GatherArgs<N> to) {
  const QuantItem w = items[blockIdx.x];
  if (w.pitch == 0) {
    for (int e = threadIdx.x; e < w.cols; e += kThreads) {
      const T x = shards[w.src + e];
      for (int r = 0; r < to.n; ++r)
        static_cast<T*>(const_cast<void*>(to.rest[r]))[w.to + e] = x;
    }
    return;
  }
  auto row = [&](int i, auto body) {
    const T* x = shards + w.src + int64_t(i) * w.cols;
    body(
        w.cols, [&](int at, int have) { return load8(x + at, have); },
        [&](const auto& raw, int, int, float (&v)[8]) { unpack(raw, v); },
        [&](int at, u2 v) {
          for (int r = 0; r < to.n; ++r) {
            u2* p = reinterpret_cast<u2*>(static_cast<char*>(const_cast<void*>(to.codes[r])) +
                                          w.to + int64_t(i) * w.pitch + at);
            if constexpr (STREAM)
              __builtin_nontemporal_store(v, p);
            else
              *p = v;
          }
        },
        [&](float s) {
          for (int r = 0; r < to.n; ++r)
            static_cast<float*>(const_cast<void*>(to.scales[r]))[w.scale + i] = s;
        });
  };
  if (w.cols > kWaveRow)
    row(0, [](auto... x) { group_row(x...); });
  else
    for (int i = threadIdx.x >> 6; i < w.n_rows; i += kThreads / 64)
      row(i, [](auto... x) { wave_row(x...); });
}

// ------------------------------------------------------------ reading back
template <int N>
struct ReadArgs {
  GatherArgs<N> from;
  void* full[N];
};

template <typename T>
__device__ __forceinline__ float value(T x) {
  if constexpr (sizeof(T) == 2)
    return bf16_to_f32(x);
  else
    return x;
}

template <typename T, typename O, int N>
__global__ __launch_bounds__(kThreads) void k_dequantize(const QuantItem* __restrict__ items,
                                                         ReadArgs<N> a) {
  const QuantItem w = items[blockIdx.x];
  const int r = blockIdx.y;
  O* full = static_cast<O*>(a.full[r]) + w.flat;
  if (w.pitch == 0) {
    const T* rest = static_cast<const T*>(a.from.rest[r]) + w.to;
    for (int e = threadIdx.x; e < w.cols; e += kThreads) {
      const T x = rest[e];
      if constexpr (sizeof(T) == sizeof(O))
        full[e] = x;
      else if constexpr (sizeof(O) == 2)
        full[e] = static_cast<u16>(f32_to_bf16(value(x)));
      else
        full[e] = value(x);
    }
    return;
  }
  const char* codes = static_cast<const char*>(a.from.codes[r]) + w.to;
  const float* scales = static_cast<const float*>(a.from.scales[r]) + w.scale;
  const bool wave = w.cols <= kWaveRow;
  const int first = wave ? threadIdx.x & 63 : threadIdx.x, step = wave ? 64 : kThreads;
  for (int i = wave ? threadIdx.x >> 6 : 0; i < w.n_rows; i += wave ? kThreads / 64 : 1) {
    const float s = scales[i];
    for (int at = first * kLane; at < w.cols; at += step * kLane) {
      const u2 v = *reinterpret_cast<const u2*>(codes + int64_t(i) * w.pitch + at);
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        x[k] = static_cast<float>(static_cast<int>(v[k / 4] << (24 - k % 4 * 8)) >> 24) * s;
      store8(full + int64_t(i) * w.cols + at, w.cols - at, x);
    }
  }
}

template <int N>
GatherArgs<N> gather_args(const QuantBuffers& b) {
  GatherArgs<N> a{};
  for (int r = 0; r < b.n; ++r) {
    a.codes[r] = b.codes.p[r];
    a.scales[r] = b.scales.p[r];
    a.rest[r] = b.rest.p[r];
  }
  a.n = b.n;
  return a;
}

template <typename T, int N>
hipError_t gather(const QuantItem* items, int64_t n, const void* shards, const QuantBuffers& b,
                  bool stream, const Sink& sink) {
  GatherArgs<N> a = gather_args<N>(b);
  void* p[] = {&items, &shards, &a};
  return sink.launch(stream ? reinterpret_cast<const void*>(&k_gather_quantize<T, N, true>)
                            : reinterpret_cast<const void*>(&k_gather_quantize<T, N, false>),
                     dim3(static_cast<unsigned>(n)), dim3(kThreads), p, 0);
}

template <typename T, typename O, int N>
hipError_t read_back(const QuantItem* items, int64_t n, const QuantBuffers& b,
                     const PtrArray& full, const Sink& sink) {
  ReadArgs<N> a{};
  a.from = gather_args<N>(b);
  for (int r = 0; r < b.n; ++r) a.full[r] = const_cast<void*>(full.p[r]);
  void* p[] = {&items, &a};
  return sink.launch(reinterpret_cast<const void*>(&k_dequantize<T, O, N>),
                     dim3(static_cast<unsigned>(n), static_cast<unsigned>(b.n)), dim3(kThreads), p,
                     0);
}

template <typename T, typename O>
hipError_t read_back(const QuantItem* items, int64_t n, const QuantBuffers& b,
                     const PtrArray& full, const Sink& sink) {
  return b.n <= kSmallPtrs ? read_back<T, O, kSmallPtrs>(items, n, b, full, sink)
                           : read_back<T, O, FSDP_MAX_RANKS>(items, n, b, full, sink);
}

template <typename T>
hipError_t quantize(const QuantizeRows& args, const Sink& sink) {
  QuantizeRows a = args;
  void* p[] = {&a};
  if (a.cols <= kWaveRow)
    return sink.launch(reinterpret_cast<const void*>(&k_quantize_rows<T, true>),
                       dim3(static_cast<unsigned>((a.rows + 3) / 4)), dim3(kThreads), p, 0);
  return sink.launch(reinterpret_cast<const void*>(&k_quantize_rows<T, false>),
                     dim3(static_cast<unsigned>(a.rows)), dim3(kThreads), p, 0);
}

}  // namespace

hipError_t launch_gather_quantize(const QuantItem* items, int64_t n, const void* shards, int dt,
                                  const QuantBuffers& to, bool stream, const Sink& sink) {
  if (dt == FSDP_BF16)
    return to.n <= kSmallPtrs ? gather<u16, kSmallPtrs>(items, n, shards, to, stream, sink)
                              : gather<u16, FSDP_MAX_RANKS>(items, n, shards, to, stream, sink);
  return to.n <= kSmallPtrs ? gather<float, kSmallPtrs>(items, n, shards, to, stream, sink)
                            : gather<float, FSDP_MAX_RANKS>(items, n, shards, to, stream, sink);
}

hipError_t launch_dequantize(const QuantItem* items, int64_t n, const QuantBuffers& from,
                             int rest_dt, const PtrArray& full, int out_dt, const Sink& sink) {
  if (rest_dt == FSDP_BF16)
    return out_dt == FSDP_BF16 ? read_back<u16, u16>(items, n, from, full, sink)
                               : read_back<u16, float>(items, n, from, full, sink);
  return out_dt == FSDP_BF16 ? read_back<float, u16>(items, n, from, full, sink)
                             : read_back<float, float>(items, n, from, full, sink);
}

hipError_t launch_quantize_rows(const QuantizeRows& a, int dt, const Sink& sink) {
  return dt == FSDP_BF16 ? quantize<u16>(a, sink) : quantize<float>(a, sink);
}

}  // namespace fsdp
