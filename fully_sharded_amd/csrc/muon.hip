// gfx950 kernels of the Muon step.
//
// The per-element kernels (momentum, apply) touch every byte once and are
// bound by HBM.  The Newton-Schulz products of one step are
//   A  = X X^T          lower triangle, mirrored into the upper
//   B  = b A + c A A    the same (A is symmetric)
//   X' = a X + B X
// and share one tile loop.  The rows of A's, B's and the first product's
// operands lie along the sum; X in the last one lies across it and is
// transposed on its way from LDS to registers (the 16-bit transposing LDS
// read), so X is kept, written and read in one orientation only.
//
// Operands are fp16: the matrices are bounded (singular values near 1), so
// a fixed power of two keeps them in range, and fp16 has 3 bits more than
// bf16 at the same rate.  Relative errors of the result against 64 bits,
// before its rounding to bf16 (1.65e-3), for white, low-rank and steep
// spectra of 512 x 512 to 1024 x 4096: bf16 operands 0.8-2.4e-2, fp16
// 1.1-4.7e-3, and fp16 with two things kept finer 2-8e-4: the residual a X
// is read as a high part in fp16 and a low part in bf8 (its small singular
// directions would otherwise carry the rounding of the large ones, amplified
// by a each step; a low part in fp16 is no better and one more byte to read
// and write), and the diagonals of A and B, their largest part once X is near
// orthogonal, are fp32 vectors d and e beside planes with zeros there:
//   A A = (A - d)(A - d) + (d_i + d_j) (A - d)_ij + d^2
//   X'  = (a + e) X + (B - e) X
#include <hip/hip_runtime.h>

#include <type_traits>

#include "muon.hpp"

namespace fsdp {
namespace {

using u16 = uint16_t;
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

// Planes hold X * kSx and A * kSa, B * kSa: |X| < 2 before the first step
// (its norm is in [1, 2)) and about 1.2 after it, |A| < 4, |B| < 12, each
// at least 8 times below fp16's largest value, and an entry 2^-16 of the
// largest still keeps all its bits.  Where X itself is small, as for an
// update far below eps, the planes hold X 2^-q with a q per matrix and step
// (k_convert): the same sizes, and the same bits kept.
constexpr float kSx = 4096.f;
constexpr float kSa = 1024.f;

// ------------------------------------------------------------- conversions
__device__ __forceinline__ float bf16_to_f32(uint32_t h) { return __uint_as_float(h << 16); }
__device__ __forceinline__ uint32_t f32_to_bf16(float x) {
  const uint32_t u = __float_as_uint(x);
  if ((u & 0x7fffffffu) > 0x7f800000u) return (u >> 16) | 0x40u;
  return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}

// Elements of T (float, or bf16 bits) as floats: one, or four adjacent ones
// in one nontemporal access (vec: 16- or 8-byte aligned).
template <typename T>
struct El;
template <>
struct El<float> {
  __device__ __forceinline__ static float load(const float* p) { return *p; }
  __device__ __forceinline__ static void store(float* p, float x) { *p = x; }
  __device__ __forceinline__ static void load4(const float* p, float (&x)[4]) {
    const f4 v = __builtin_nontemporal_load(reinterpret_cast<const f4*>(p));
    for (int k = 0; k < 4; ++k) x[k] = v[k];
  }
  __device__ __forceinline__ static void store4(float* p, const float (&x)[4]) {
    __builtin_nontemporal_store(f4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f4*>(p));
  }
};
template <>
struct El<u16> {
  __device__ __forceinline__ static float load(const u16* p) { return bf16_to_f32(*p); }
  __device__ __forceinline__ static void store(u16* p, float x) {
    *p = static_cast<u16>(f32_to_bf16(x));
  }
  __device__ __forceinline__ static void load4(const u16* p, float (&x)[4]) {
    const u2 v = __builtin_nontemporal_load(reinterpret_cast<const u2*>(p));
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xffff0000u);
  }
  __device__ __forceinline__ static void store4(u16* p, const float (&x)[4]) {
    u2 v;
    v.x = f32_to_bf16(x[0]) | (f32_to_bf16(x[1]) << 16);
    v.y = f32_to_bf16(x[2]) | (f32_to_bf16(x[3]) << 16);
    __builtin_nontemporal_store(v, reinterpret_cast<u2*>(p));
  }
};

// ------------------------------------------------------- per-element passes
// One workgroup per item: 1024 elements, four adjacent ones per lane, the
// lanes on multiples of four of the destination space.  Where the source
// space is not on the same grid (shards that begin at odd places) it is
// read element by element, which the first-level cache turns into the same
// lines.  Bound by HBM; measured: momentum 9.9 us (5.7 TB/s) on 3.1M
// parameters, R = 4, and 0.92 ms (6.2 TB/s) on 218M, R = 8, both bf16; apply
// 6.7 us (5.6 TB/s) and 0.42 ms (6.2 TB/s).  Items of 512 or 2,048 elements
// measured level.
template <int N>
struct MomentumArgs {
  const void* g[N];
  int R;
  float* m;
  void* update;
  MuonScalars sc;
  bool vec;
};

__device__ __forceinline__ void momentum1(float g, float& m, float& u, const MuonScalars& sc) {
  const double gd = sc.one_minus * static_cast<double>(g);
  m = static_cast<float>(sc.momentum * static_cast<double>(m) + gd);
  u = sc.nesterov ? static_cast<float>(gd + sc.momentum * static_cast<double>(m)) : m;
}

// RT > 0: R replicas known at compile time, every load issued before the
// first add; 0: any R; -1: the reduced gradient, in shard space.
template <typename G, typename U, int RT, int N>
__global__ __launch_bounds__(kThreads) void k_momentum(const MuonItem* __restrict__ items,
                                                       MomentumArgs<N> a) {
  const MuonItem w = items[blockIdx.x];
  U* update = static_cast<U*>(a.update);
  const int64_t e0 = (w.dst & ~int64_t(3)) + 4 * threadIdx.x;
  const int64_t end = w.dst + w.len;
  if (e0 >= end) return;
  const int64_t s0 = w.src + (e0 - w.dst);
  const int R = RT > 0 ? RT : a.R;
  if (a.vec && e0 >= w.dst && e0 + 4 <= end) {
    const bool svec = (s0 & 3) == 0;
    float g[4], m[4], u[4];
    if constexpr (RT < 0) {
      const float* p = static_cast<const float*>(a.g[0]) + s0;
      if (svec) {
        El<float>::load4(p, g);
      } else {
        for (int k = 0; k < 4; ++k) g[k] = p[k];
      }
    } else {
      float x[RT > 0 ? RT : 1][4];
      if constexpr (RT > 0) {
#pragma unroll
        for (int q = 0; q < RT; ++q) El<G>::load4(static_cast<const G*>(a.g[q]) + e0, x[q]);
      } else {
        El<G>::load4(static_cast<const G*>(a.g[0]) + e0, x[0]);
      }
      for (int k = 0; k < 4; ++k) g[k] = x[0][k];
      if constexpr (RT > 0) {
#pragma unroll
        for (int q = 1; q < RT; ++q)
          for (int k = 0; k < 4; ++k) g[k] = g[k] + x[q][k];
      } else {
#pragma unroll 4
        for (int q = 1; q < R; ++q) {
          float y[4];
          El<G>::load4(static_cast<const G*>(a.g[q]) + e0, y);
          for (int k = 0; k < 4; ++k) g[k] = g[k] + y[k];
        }
      }
      for (int k = 0; k < 4; ++k) g[k] = g[k] / static_cast<float>(R);
    }
    if (svec) {
      El<float>::load4(a.m + s0, m);
    } else {
      for (int k = 0; k < 4; ++k) m[k] = a.m[s0 + k];
    }
    for (int k = 0; k < 4; ++k) momentum1(g[k], m[k], u[k], a.sc);
    if (svec) {
      El<float>::store4(a.m + s0, m);
    } else {
      for (int k = 0; k < 4; ++k) a.m[s0 + k] = m[k];
    }
    El<U>::store4(update + e0, u);
    return;
  }
  for (int k = 0; k < 4; ++k) {
    const int64_t e = e0 + k, s = s0 + k;
    if (e < w.dst || e >= end) continue;
    float g, u;
    if constexpr (RT < 0) {
      g = static_cast<const float*>(a.g[0])[s];
    } else {
      g = El<G>::load(static_cast<const G*>(a.g[0]) + e);
      for (int q = 1; q < R; ++q) g = g + El<G>::load(static_cast<const G*>(a.g[q]) + e);
      g = g / static_cast<float>(R);
    }
    float m = a.m[s];
    momentum1(g, m, u, a.sc);
    a.m[s] = m;
    El<U>::store(update + e, u);
  }
}

struct ApplyArgs {
  const MuonScale* scales;
  const void* ortho;
  float* master;
  void* param;
  MuonScalars sc;
  bool vec;
};

template <typename O, typename P>
__global__ __launch_bounds__(kThreads) void k_apply(const MuonItem* __restrict__ items,
                                                    ApplyArgs a) {
  const MuonItem w = items[blockIdx.x];
  const int64_t e0 = (w.dst & ~int64_t(3)) + 4 * threadIdx.x;
  const int64_t end = w.dst + w.len;
  if (e0 >= end) return;
  const O* ortho = static_cast<const O*>(a.ortho);
  P* param = static_cast<P*>(a.param);
  const int64_t s0 = w.src + (e0 - w.dst);
  // lr times the matrix's scale
  double rate = a.sc.lr;
  if (a.sc.scale == FSDP_MUON_SCALE_ASPECT) rate *= a.scales[w.mat].aspect;
  if (a.sc.scale == FSDP_MUON_SCALE_RMS) rate *= a.scales[w.mat].rms;
  auto one = [&](float p, float x) {
    return static_cast<float>(static_cast<double>(p) * a.sc.decay -
                              rate * static_cast<double>(x));
  };
  if (a.vec && e0 >= w.dst && e0 + 4 <= end) {
    float x[4], p[4];
    if ((s0 & 3) == 0) {
      El<O>::load4(ortho + s0, x);
    } else {
      for (int k = 0; k < 4; ++k) x[k] = El<O>::load(ortho + s0 + k);
    }
    El<float>::load4(a.master + e0, p);
    for (int k = 0; k < 4; ++k) p[k] = one(p[k], x[k]);
    El<float>::store4(a.master + e0, p);
    El<P>::store4(param + e0, p);
    return;
  }
  for (int k = 0; k < 4; ++k) {
    const int64_t e = e0 + k;
    if (e < w.dst || e >= end) continue;
    const float p = one(a.master[e], El<O>::load(ortho + s0 + k));
    a.master[e] = p;
    El<P>::store(param + e, p);
  }
}

// ----------------------------------------------------- norm and conversion
// The sum of a workgroup's values, in a fixed order, to every lane.
__device__ __forceinline__ double block_sum(double x) {
  __shared__ double part[kThreads / 64];
  for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = 0;
  for (int k = 0; k < kThreads / 64; ++k) s += part[k];
  return s;
}

// Partial sums of squares, in 64 bits: a square of any finite fp32 value is
// neither infinite nor lost.  One workgroup per chunk (4,096 elements or more,
// at most 1,024 of them per matrix, which every conversion tile adds up again
// in the same order).  89 us for 218M bf16 elements (4.9 TB/s).
template <typename T>
__global__ __launch_bounds__(kThreads) void k_norm(const MuonChunk* __restrict__ chunks,
                                                   const T* __restrict__ u,
                                                   double* __restrict__ partial) {
  const MuonChunk t = chunks[blockIdx.x];
  const int64_t lo = t.lo, hi = t.hi;
  double s = 0;
  if ((reinterpret_cast<uintptr_t>(u + lo) & (4 * sizeof(T) - 1)) == 0) {
    int64_t e = lo + 4 * threadIdx.x;
    for (; e + 4 <= hi; e += 4 * kThreads) {
      float x[4];
      El<T>::load4(u + e, x);
      for (int k = 0; k < 4; ++k) s += static_cast<double>(x[k]) * x[k];
    }
    for (; e < hi; ++e) {  // the chunk's last, cut group: one lane has it
      const double x = El<T>::load(u + e);
      s += x * x;
    }
  } else {
    for (int64_t e = lo + threadIdx.x; e < hi; e += kThreads) {
      const double x = El<T>::load(u + e);
      s += x * x;
    }
  }
  s = block_sum(s);
  if (threadIdx.x == 0) partial[t.to] = s;
}

// Four values in bf8 (5 bits of exponent, 2 of mantissa), and back.  The low
// part of a plane's entry is below 2^-11 of it; entries small enough for it
// to leave bf8's range are below 2^-16 of the largest.
__device__ __forceinline__ uint32_t pack_bf8(const float (&x)[4]) {
  int v = __builtin_amdgcn_cvt_pk_bf8_f32(x[0], x[1], 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_bf8_f32(x[2], x[3], v, true));
}
__device__ __forceinline__ f4 unpack_bf8(uint32_t v) {
  const auto a = __builtin_amdgcn_cvt_pk_f32_bf8(static_cast<int>(v), false);
  const auto b = __builtin_amdgcn_cvt_pk_f32_bf8(static_cast<int>(v), true);
  return f4{a[0], a[1], b[0], b[1]};
}

struct ConvertArgs {
  const MuonConvertTile* tiles;
  const double* partial;
  MuonCoef* coef;  // per matrix and step
  int steps;
  _Float16* xh;
  void* xl;    // null: the low parts are not wanted
  bool bytes;  // they are wanted in bf8
  double eps, a, b, c;
};

// Eight adjacent elements (aligned to 16 bytes) as floats.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    const u4 v = __builtin_nontemporal_load(reinterpret_cast<const u4*>(p));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(v[k] << 16);
      x[2 * k + 1] = __uint_as_float(v[k] & 0xffff0000u);
    }
  } else {
    float y[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      El<float>::load4(p + 4 * h, y);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[4 * h + k] = y[k];
    }
  }
}

// 64 x 64 tiles of the update into X, transposed where the parameter has
// more rows than columns.  The planes get U 2^-e with 2^e <= |U| < 2^(e+1):
// exact for bf16 updates, but for entries below 2^-29 of |U|.  What is left,
// f = 2^e / N with N = |U| + eps, goes into the first step's coefficients: A
// is then A f^-2 and X is X f^-1.  Where eps is not small beside |U|, X is:
// at fixed scales an |X| of 1e-8 was 13-51% off for want of bits in fp16.  So
// the planes hold X 2^-q after a step, 2^q the power of two below what X's
// singular values can be, 1 at most: s = |U| / N before the first step, and
// |a| s + |b| s^3 + |c| s^5 after each.  P = X 2^-q steps by
//   P' = a 2^(q-q') P + b 2^(3q-q') P^3 + c 2^(5q-q') P^5
// where no coefficient is above 2 for q' < 0; at q = q' = 0, as everywhere
// that eps does not matter, these are a, b and c.  q stops at -400: X is then
// 0 in fp32, and no 16 steps of coefficients up to 16 make it anything else.
// A lane has 8 adjacent entries of each of two rows.  198 us for 218M bf16
// elements (4.4 TB/s read and written).
template <typename T>
__global__ __launch_bounds__(kThreads) void k_convert(const T* __restrict__ update,
                                                      ConvertArgs a) {
  constexpr int Ld = 72;
  __shared__ __align__(16) _Float16 tile[64 * Ld];
  const MuonConvertTile t = a.tiles[blockIdx.x];
  const int64_t r0 = int64_t(t.i) * 64, c0 = int64_t(t.j) * 64;
  const int lr = threadIdx.x >> 3, lc = (threadIdx.x & 7) * 8;
  float x[2][8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t r = r0 + lr + 32 * h, c = c0 + lc;
    const T* u = update + t.flat_off + r * t.cols + c;
    if (r < t.rows && c + 8 <= t.cols && (reinterpret_cast<uintptr_t>(u) & 15) == 0) {
      load8(u, x[h]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        x[h][k] = r < t.rows && c + k < t.cols ? El<T>::load(u + k) : 0.f;
    }
  }
  double s = 0;
  for (int k = threadIdx.x; k < t.norm_count; k += kThreads) s += a.partial[t.norm_first + k];
  const double mass = sqrt(block_sum(s)), norm = mass + a.eps;
  const bool bad = !(norm < INFINITY), some = !bad && mass > 0;
  const int e = some ? ilogb(mass) : 0;
  const double scale = ldexp(static_cast<double>(kSx), -e);
  if (t.i == 0 && t.j == 0 && threadIdx.x < a.steps) {
    // lane n: of step n, which goes from q to `to`
    const bool grows = fabs(a.a) + fabs(a.b) + fabs(a.c) >= 1;
    double most = some ? mass / norm : 0;  // of X's singular values
    int q = 0, to = 0;
    for (int n = 0; n <= static_cast<int>(threadIdx.x) && !bad; ++n) {
      q = to;
      if (grows && most >= 1) {  // and so from here on
        to = 0;
        break;
      }
      const double most2 = most * most;
      most *= fabs(a.a) + most2 * (fabs(a.b) + most2 * fabs(a.c));
      to = most > 0 ? max(min(ilogb(most), 0), -400) : -400;
      most = min(most, 16.0);
    }
    MuonCoef k{1.f, 1.f, 1.f, q - to, 3 * q - to, 5 * q - to, to, 0};
    if (threadIdx.x == 0) {
      k.ea = k.eb = k.ec = 0;
      const double f = some ? ldexp(1.0, e) / norm : 0;
      k.a = bad ? NAN : static_cast<float>(ldexp(a.a * f, -to));
      k.b = bad ? NAN : static_cast<float>(ldexp(a.b * f * f * f, -to));
      k.c = bad ? NAN : static_cast<float>(ldexp(a.c * f * f * f * f * f, -to));
    }
    a.coef[t.mat * kMuonSteps + threadIdx.x] = k;
  }
  // where a lane's entries go: rows of X, across them in a tall parameter
  const int64_t to0 = t.tall ? (c0 + lr) * t.ldx + r0 + lc : (r0 + lr) * t.ldx + c0 + lc;
  const int64_t to[2] = {t.off_x + to0, t.off_x + to0 + 32 * int64_t(t.ldx)};
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int k = 0; k < 8; ++k)
      x[h][k] = static_cast<float>(static_cast<double>(x[h][k]) * scale);
  union {
    _Float16 h[8];
    u4 v;
  } part[2];
  for (int low = 0; low < (a.xl && !a.bytes ? 2 : 1); ++low) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        part[h].h[k] = static_cast<_Float16>(x[h][k]);
        x[h][k] -= static_cast<float>(part[h].h[k]);
      }
    if (t.tall) {
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<u4*>(tile + (lr + 32 * h) * Ld + lc) = part[h].v;
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 8; ++k) part[h].h[k] = tile[(lc + k) * Ld + lr + 32 * h];
    }
    _Float16* out = low ? static_cast<_Float16*>(a.xl) : a.xh;
#pragma unroll
    for (int h = 0; h < 2; ++h) *reinterpret_cast<u4*>(out + to[h]) = part[h].v;
  }
  if (!a.xl || !a.bytes) return;
  union {
    char b[8];
    u2 v;
  } low[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    low[h].v = u2{pack_bf8({x[h][0], x[h][1], x[h][2], x[h][3]}),
                  pack_bf8({x[h][4], x[h][5], x[h][6], x[h][7]})};
  if (t.tall) {
    char* bytes = reinterpret_cast<char*>(tile);
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) *reinterpret_cast<u2*>(bytes + (lr + 32 * h) * Ld + lc) = low[h].v;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 8; ++k) low[h].b[k] = bytes[(lc + k) * Ld + lr + 32 * h];
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    *reinterpret_cast<u2*>(static_cast<char*>(a.xl) + to[h]) = low[h].v;
}

// ---------------------------------------------------------------- products
struct GemmArgs {
  const MuonCoef* coef;  // per matrix and step, from this step's first on
  float a, b, c;         // the step's; the first's are in coef, these 1
  float *adiag, *bdiag;  // the diagonals of A and B
  // X of this step and of the next; the low parts in bf8 or, where they are
  // operands, in fp16 (xl null in the first step of a bf16 update: zeros)
  const _Float16* xh;
  const void* xl;
  _Float16* yh;
  void* yl;
  _Float16 *ah, *al, *bh, *bl;
  void* ortho;
  float* sums;  // A's partial sums
};

enum Stage { kGram, kPoly, kStep, kLast };

// A BM x BN tile by WM x WN waves, BK of the sum per round, NS rounds in LDS,
// registers for WPS waves per SIMD.
template <int BM_, int BN_, int WM_, int WN_, int BK_, int NS_, int WPS_>
struct Shape {
  static constexpr int Waves = WPS_;  // per SIMD
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = BK_, NS = NS_;
  static constexpr int NW = WM * WN, Threads = 64 * NW;
  static constexpr int TM = BM / WM, TN = BN / WN;  // a wave's tile
  static constexpr int FM = TM / 16, FN = TN / 16;  // its 16 x 16 parts
  static constexpr int RB = BK * 2;                 // bytes of a row of one round
  static constexpr int RowsPerLoad = 1024 / RB;     // rows that one wave's load fills
  static constexpr int LP = BM / RowsPerLoad / NW, LQ = BN / RowsPerLoad / NW;
  static constexpr int RoundBytes = (BM + BN) * RB;
};

// The place of 16-byte chunk c of row r in LDS: the 16 rows that a wave reads
// at one chunk, 128 or 64 bytes apart, spread over all banks.
template <int BK>
__device__ __forceinline__ int place(int r, int c) {
  return BK == 64 ? c ^ (r & 7) : c ^ ((r >> 1) & 3);
}
// The same for rows across the sum (BN entries): a transposing read takes 32
// bytes of rows 0-3, 8-11, 16-19 and 24-27 (or 4-7, ...) of 32 at a time, so
// the pairs of chunks move by bits 0, 1 and 3 of the row; rows of 128 bytes
// alternate by themselves with bit 0, rows of 64 bytes with bits 0 and 1.
template <int BN>
__device__ __forceinline__ int place_across(int r, int c) {
  const int b = (r & 3) | ((r >> 1) & 4);
  return c ^ (BN == 32 ? (b & 4) >> 1 : BN == 64 ? b & 6 : b << 1);
}

// 16 bytes per lane from global memory to LDS at a wave-uniform address, lane
// after lane.  An asm statement (its only register is M0): of the builtin the
// compiler waits for all loads under way before every transposing LDS read,
// which it cannot tell from a read of the bytes being loaded.  M0 as an
// operand that the compiler sets, apart from the load, took 0.4-0.6% longer.
// Waited for by wait_and_meet.
__device__ __forceinline__ void load_to_lds(const void* from, uint32_t to) {
  uint32_t m0;
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               : "=&{m0}"(m0)
               : "v"(from), "s"(__builtin_amdgcn_readfirstlane(to))
               : "memory");
}

// Wait until all of this wave's LDS reads are done (the builtin, not an asm
// statement: the compiler counts on from it).
__device__ __forceinline__ void wait_lds() {
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));
}
// Wait until at most N of this wave's global accesses are under way.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64);
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
// The same and for all its LDS reads, then for the other waves.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  static_assert(N < 64);
  // products stay on their side: those before it hide the loads waited for
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// 4 x 4 half-words over 4 adjacent lanes, transposed: lane s holds (x, y) =
// entries 0..3 of row s and gets entry s of rows 0..3.
__device__ __forceinline__ u2 transpose4(u2 v, uint32_t odd_sel, bool high) {
  // with the neighbour: even lanes entries 0 and 2 of rows (s, s+1), odd
  // lanes entries 1 and 3 of rows (s-1, s)
  const uint32_t px = __builtin_amdgcn_mov_dpp(v.x, 0xB1, 0xf, 0xf, true);
  const uint32_t py = __builtin_amdgcn_mov_dpp(v.y, 0xB1, 0xf, 0xf, true);
  const uint32_t x = __builtin_amdgcn_perm(px, v.x, odd_sel);
  const uint32_t y = __builtin_amdgcn_perm(py, v.y, odd_sel);
  // with the lane two away
  const uint32_t qx = __builtin_amdgcn_mov_dpp(x, 0x4E, 0xf, 0xf, true);
  const uint32_t qy = __builtin_amdgcn_mov_dpp(y, 0x4E, 0xf, 0xf, true);
  return high ? u2{qy, y} : u2{x, qx};
}

__device__ __forceinline__ u2 pack4(const float (&x)[4]) {
  union {
    h4 h;
    u2 u;
  } v;
#pragma unroll
  for (int r = 0; r < 4; ++r) v.h[r] = static_cast<_Float16>(x[r]);
  return v.u;
}

// 16 of a wave's rows to global memory, 16 bytes per lane, through LDS of the
// wave's own: v[j] is row lane % 16, columns 16 j + 4 (lane / 16) + 0..3.
// store(row, col, eight adjacent entries).
template <int FN, typename F>
__device__ __forceinline__ void store_rows(char* lds, const u2 (&v)[FN], F store) {
  constexpr int Ld = (FN * 16 + 8) * 2;  // bytes: rows spread over the banks
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int j = 0; j < FN; ++j)
    *reinterpret_cast<u2*>(lds + (lane & 15) * Ld + (j * 16 + (lane >> 4) * 4) * 2) = v[j];
  constexpr int PerRow = FN * 2, Rows = 64 / PerRow, N = 16 / Rows;
  const int r = lane / PerRow, c = lane % PerRow * 8;
  u4 out[N];
#pragma unroll
  for (int k = 0; k < N; ++k)
    out[k] = *reinterpret_cast<const u4*>(lds + (k * Rows + r) * Ld + c * 2);
#pragma unroll
  for (int k = 0; k < N; ++k) store(k * Rows + r, c, out[k]);
}

// The same for rows of bytes, 8 per lane: v[j] has the four of row lane % 16.
template <int FN, typename F>
__device__ __forceinline__ void store_byte_rows(char* lds, const uint32_t (&v)[FN], F store) {
  constexpr int Ld = FN * 16 + 8;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int j = 0; j < FN; ++j)
    *reinterpret_cast<uint32_t*>(lds + (lane & 15) * Ld + j * 16 + (lane >> 4) * 4) = v[j];
  constexpr int PerRow = FN * 2, Rows = 64 / PerRow, N = 16 / Rows;
  const int r = lane / PerRow, c = lane % PerRow * 8;
#pragma unroll
  for (int k = 0; k < N; ++k)
    store(k * Rows + r, c, *reinterpret_cast<const u2*>(lds + (k * Rows + r) * Ld + c));
}

// The same values into a transposed image (columns as rows, ld bytes each).
template <int FN>
__device__ __forceinline__ void keep_transposed(char* lds, int ld, int i, const u2 (&v)[FN]) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lk = lane >> 4;
  const uint32_t sel = lane & 1 ? 0x03020706u : 0x05040100u;
#pragma unroll
  for (int j = 0; j < FN; ++j)
    *reinterpret_cast<u2*>(lds + (j * 16 + lk * 4 + (lr & 3)) * ld + (i * 16 + (lr & 12)) * 2) =
        transpose4(v[j], sel, lane & 2);
}

// A transposed image of R rows of C to global memory.
template <int R, int C, typename F>
__device__ __forceinline__ void store_image(const char* lds, F store) {
  constexpr int Ld = (C + 8) * 2, PerRow = C / 8, Rows = 64 / PerRow, N = R / Rows;
  constexpr int Batch = N < 8 ? N : 8;
  const int lane = threadIdx.x & 63;
  const int r = lane / PerRow, c = lane % PerRow * 8;
#pragma unroll
  for (int b = 0; b < N; b += Batch) {
    u4 out[Batch];
#pragma unroll
    for (int k = 0; k < Batch; ++k)
      out[k] = *reinterpret_cast<const u4*>(lds + ((b + k) * Rows + r) * Ld + c * 2);
#pragma unroll
    for (int k = 0; k < Batch; ++k) store((b + k) * Rows + r, c, out[k]);
  }
}

// The operands of one product: D (rows of P x rows or columns of Q).
template <Stage ST, bool SPLIT>
struct Operands {
  static constexpr bool kAcross = ST == kStep || ST == kLast;  // Q lies across the sum
  const _Float16 *ph, *pl = nullptr, *qh, *ql = nullptr;
  int prows, qrows, depth;
  int ld, lp, lq;  // row pitch of the result and of the operands

  __device__ __forceinline__ Operands(const GemmArgs& g, const MuonGemmTile& t) {
    if constexpr (ST == kGram) {
      ph = qh = g.xh + t.off_x;
      if (SPLIT) pl = ql = static_cast<const _Float16*>(g.xl) + t.off_x;
      prows = qrows = t.mp;
      ld = t.lda;
      lp = lq = t.ldx;
      depth = t.np;
    } else if constexpr (ST == kPoly) {
      ph = qh = g.ah + t.off_a;
      if (SPLIT) pl = ql = g.al + t.off_a;
      prows = qrows = t.mp;
      ld = lp = lq = t.lda;
      depth = t.mp;
    } else {
      ph = g.bh + t.off_a;
      qh = g.xh + t.off_x;
      if (SPLIT) {
        pl = g.bl + t.off_a;
        ql = static_cast<const _Float16*>(g.xl) + t.off_x;
      }
      prows = t.mp;
      qrows = t.np;
      lp = t.lda;
      ld = lq = t.ldx;
      depth = t.mp;
    }
  }
};

// Where a round begins in P and Q.
struct From {
  const _Float16 *p, *q;
};

// A workgroup's tile in one scalar load (its table's address is preloaded), and
// the arguments asked for with it:
// read where each is used they made a chain of round trips to memory, some
// 10,000 cycles before the first operand was asked for.
__device__ __forceinline__ MuonGemmTile tile_of(const MuonGemmTile* tiles, const GemmArgs& g) {
  typedef int i16 __attribute__((ext_vector_type(16)));
  union {
    i16 v;
    MuonGemmTile t;
  } u;
  u.v = *reinterpret_cast<const i16*>(tiles + blockIdx.x);
  asm volatile("" ::"s"(u.v), "s"(g.coef), "s"(g.adiag), "s"(g.bdiag), "s"(g.xh), "s"(g.xl),
               "s"(g.yh), "s"(g.yl), "s"(g.ah), "s"(g.bh), "s"(g.ortho));
  return u.t;
}
template <int BK, Stage ST, bool SPLIT>
__device__ __forceinline__ From from_round(const Operands<ST, SPLIT>& o, int it, int rounds) {
  From f{o.ph, o.qh};
  int k = it;
  if constexpr (SPLIT) {  // the small products first: high low, low high, high high
    const int part = it / rounds;
    k = it - part * rounds;
    if (part == 0) f.q = o.ql;
    if (part == 1) f.p = o.pl;
  }
  f.p += int64_t(k) * BK;
  f.q += Operands<ST, SPLIT>::kAcross ? int64_t(k) * BK * o.lq : int64_t(k) * BK;
  return f;
}

// One lane's part of a round's loads, by wave `wave` of S::NW: LP pieces of
// P, then LQ of Q, each 1024 bytes of the round's image in LDS.  Rows and
// columns past the plane's last are read from the last ones; their results
// are not stored.
template <typename S, bool ACROSS>
struct Loader {
  int64_t po[S::LP], qo[S::LQ];
  int wave;

  __device__ __forceinline__ Loader(int wave_, int i0, int j0, int prows, int qrows, int lp,
                                    int lq)
      : wave(wave_) {
    const int lane = threadIdx.x & 63;
    constexpr int PerRow = S::BK / 8;
    const int r = lane / PerRow, c = place<S::BK>(r, lane % PerRow);
#pragma unroll
    for (int k = 0; k < S::LP; ++k) {
      const int row = i0 + (wave * S::LP + k) * S::RowsPerLoad + r;
      po[k] = int64_t(row < prows ? row : prows - 1) * lp + c * 8;
    }
    if constexpr (ACROSS) {
      constexpr int Chunks = S::BN / 8, Rows = 64 / Chunks;
#pragma unroll
      for (int k = 0; k < S::LQ; ++k) {
        const int row = (wave * S::LQ + k) * Rows + lane / Chunks;
        const int col = j0 + place_across<S::BN>(row, lane % Chunks) * 8;
        qo[k] = int64_t(row) * lq + (col < qrows ? col : qrows - 8);
      }
    } else {
#pragma unroll
      for (int k = 0; k < S::LQ; ++k) {
        const int row = j0 + (wave * S::LQ + k) * S::RowsPerLoad + r;
        qo[k] = int64_t(row < qrows ? row : qrows - 1) * lq + c * 8;
      }
    }
  }
  // piece x of the round at f into the image at `image`
  __device__ __forceinline__ void load(const From& f, uint32_t image, int x) const {
    if (x < S::LP)
      load_to_lds(f.p + po[x < S::LP ? x : 0], image + (wave * S::LP + x) * 1024);
    else
      load_to_lds(f.q + qo[x < S::LP ? 0 : x - S::LP],
                  image + S::BM * S::RB + (wave * S::LQ + x - S::LP) * 1024);
  }
};

// LDS to registers: the 16 x 32 operands of wave (wm, wn).
template <typename S, bool ACROSS>
struct Fetcher {
  int pat, qat[ACROSS ? S::FN : 1];

  __device__ __forceinline__ Fetcher(int wm, int wn) {
    const int lane = threadIdx.x & 63, lr = lane & 15, lk = lane >> 4;
    pat = (wm * S::TM + lr) * S::RB;
    if constexpr (ACROSS) {
      const int row = lk * 8 + (lr >> 2);  // and 4 more for the second half
#pragma unroll
      for (int j = 0; j < S::FN; ++j)
        qat[j] = S::BM * S::RB + row * S::BN * 2 +
                 place_across<S::BN>(row, wn * (S::TN / 8) + j * 2 + ((lr & 3) >> 1)) * 16 +
                 (lr & 1) * 8;
    } else {
      qat[0] = S::BM * S::RB + (wn * S::TN + lr) * S::RB;
    }
  }
  __device__ __forceinline__ h8 p(const char* image, int kk, int i) const {
    const int lane = threadIdx.x & 63;
    return *reinterpret_cast<const h8*>(
        image + place<S::BK>(lane & 15, kk * 4 + (lane >> 4)) * 16 + pat + i * 16 * S::RB);
  }
  __device__ __forceinline__ h8 q(const char* image, int kk, int j) const {
    if constexpr (ACROSS) {
      typedef short s4 __attribute__((ext_vector_type(4)));
      union {
        s4 s[2];
        h8 h;
      } v;
#pragma unroll
      for (int half = 0; half < 2; ++half)
        v.s[half] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s4*)(image + qat[j] +
                                                    (kk * 32 + half * 4) * S::BN * 2));
      return v.h;
    } else {
      const int lane = threadIdx.x & 63;
      return *reinterpret_cast<const h8*>(
          image + place<S::BK>(lane & 15, kk * 4 + (lane >> 4)) * 16 + qat[0] + j * 16 * S::RB);
    }
  }
};

// A wave's results, FM x FN parts of 16 x 16: acc[i][j][r] is row rb + 16 i +
// lane % 16 of P, row or column cb + 16 j + 4 (lane / 16) + r of Q.  Planes
// are padded to multiples of 64: whole parts are inside or outside.  AHEAD:
// how many sets of 16 rows of what the results are added to (A's or X's own
// entries) are in registers at once.  Loads and stores are waited for in
// order: with one set ahead each set waited for the stores of the one before.
// The sets come in whole rows, 16 bytes per lane, and reach the lanes of the
// results through LDS: read as the results lie, 8 bytes of each of 16 rows
// at a time, they took 20,000 of a 128 x 128 tile's 47,000 cycles (depth
// 512).
template <int FM, int FN, int AHEAD, Stage ST, bool SPLIT, typename O>
struct Result {
  static constexpr int TM = FM * 16, TN = FN * 16;
  static constexpr bool kAcross = ST == kStep || ST == kLast;
  static constexpr bool kMirror = ST == kGram || ST == kPoly;
  // One part of 16 x 16 goes to memory from the registers; more by way of a
  // wave's part of LDS: 16 rows, and a transposed image (fp32 results: one of
  // fp32, either way round).
  static constexpr bool kDirect = FM * FN == 1;
  static constexpr int kRows = 16 * (TN + 8) * 2;
  static constexpr int kImage = ST == kStep ? 0 : TN * (TM + 8) * 2;
  static constexpr int kOut =
      kRows + (ST == kLast && sizeof(O) == 4 ? ((TM + 1) * (TN + 1) * 4 + 15) / 16 * 16 : kImage);

  static constexpr bool kOwnLow = kAcross || SPLIT;
  static constexpr bool kBytes = kAcross && !SPLIT;  // low parts in bf8
  static constexpr int kOwnLd = (TN + 8) * 2;  // of 16 rows in LDS
  static constexpr int kPerRow = TN / 8, kStepRows = kDirect ? 16 : 64 / kPerRow;
  static constexpr int kSets = kDirect ? 1 : 16 / kStepRows;
  static_assert(64 % TN == 0);

  int rb, cb, lr, lk;
  u4 own_h[AHEAD][kSets], own_l[AHEAD][kSets];  // kDirect: in the first two words
  float di[FM];
  MuonCoef coef;
  f4 dj[FN];

  __device__ __forceinline__ void own_rows(const GemmArgs& g, const MuonGemmTile& t,
                                           const Operands<ST, SPLIT>& o, int i) {
    const _Float16* oh = ST == kPoly ? o.ph : o.qh;
    const char* ol = ST == kPoly ? reinterpret_cast<const char*>(o.pl)
                                 : static_cast<const char*>(g.xl);
    if (ST != kPoly && ol) ol += t.off_x * (kBytes ? 1 : 2);
    if constexpr (ST != kGram) {
      const int lane = threadIdx.x & 63;
      const int64_t at =
          kDirect ? int64_t(rb + lr) * o.ld + cb + lk * 4
                  : int64_t(rb + i * 16 + lane / kPerRow) * o.ld + cb + lane % kPerRow * 8;
      const bool in = rb + i * 16 < o.prows && cb < o.qrows;  // uniform: TN divides 64
#pragma unroll
      for (int k = 0; k < kSets; ++k) {
        u4 &h = own_h[i % AHEAD][k], &l = own_l[i % AHEAD][k];
        h = l = u4{0, 0, 0, 0};
        if (in) {
          const int64_t e = at + int64_t(k) * kStepRows * o.ld;
          if constexpr (kDirect) {
            const u2 v = *reinterpret_cast<const u2*>(oh + e);
            h.x = v.x;
            h.y = v.y;
            if (kOwnLow && ol) {
              if constexpr (kBytes) {
                l.x = *reinterpret_cast<const uint32_t*>(ol + e);
              } else {
                const u2 w = *reinterpret_cast<const u2*>(ol + e * 2);
                l.x = w.x;
                l.y = w.y;
              }
            }
          } else {
            h = *reinterpret_cast<const u4*>(oh + e);
            if (kOwnLow && ol) {
              if constexpr (kBytes) {
                const u2 w = *reinterpret_cast<const u2*>(ol + e);
                l.x = w.x;
                l.y = w.y;
              } else {
                l = *reinterpret_cast<const u4*>(ol + e * 2);
              }
            }
          }
        }
      }
    }
  }

  // One plane of set i, as the results lie.
  __device__ __forceinline__ void spread(char* rows16, const u4 (&from)[kSets],
                                         h4 (&to)[FN]) const {
    union {
      u2 u;
      h4 h;
    } v;
    if constexpr (kDirect) {
      v.u = u2{from[0].x, from[0].y};
      to[0] = v.h;
    } else {
      const int lane = threadIdx.x & 63;
#pragma unroll
      for (int k = 0; k < kSets; ++k)
        *reinterpret_cast<u4*>(rows16 + (k * kStepRows + lane / kPerRow) * kOwnLd +
                               lane % kPerRow * 16) = from[k];
#pragma unroll
      for (int j = 0; j < FN; ++j)
        to[j] = *reinterpret_cast<const h4*>(rows16 + lr * kOwnLd + (j * 16 + lk * 4) * 2);
    }
  }

  // The low parts of set i, likewise.
  __device__ __forceinline__ void spread_low(char* rows16, const u4 (&from)[kSets],
                                             f4 (&to)[FN]) const {
    if constexpr (kBytes) {
      if constexpr (kDirect) {
        to[0] = unpack_bf8(from[0].x);
      } else {
        constexpr int Ld = TN + 8;
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int k = 0; k < kSets; ++k)
          *reinterpret_cast<u2*>(rows16 + (k * kStepRows + lane / kPerRow) * Ld +
                                 lane % kPerRow * 8) = u2{from[k].x, from[k].y};
#pragma unroll
        for (int j = 0; j < FN; ++j)
          to[j] = unpack_bf8(
              *reinterpret_cast<const uint32_t*>(rows16 + lr * Ld + j * 16 + lk * 4));
      }
    } else {
      h4 l[FN];
      spread(rows16, from, l);
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) to[j][r] = static_cast<float>(l[j][r]);
    }
  }

  // Ask for everything that is not a sum.
  __device__ __forceinline__ void ask(const GemmArgs& g, const MuonGemmTile& t,
                                      const Operands<ST, SPLIT>& o, int rb_, int cb_) {
    const int lane = threadIdx.x & 63;
    lr = lane & 15;
    lk = lane >> 4;
    rb = rb_;
    cb = cb_;
    // (used in finish: a product here would be waited for before the sums)
    if constexpr (ST != kGram) coef = g.coef[(t.mat & ~kMuonTall) * kMuonSteps];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      dj[j] = f4{0.f, 0.f, 0.f, 0.f};
      if (ST == kPoly && cb + j * 16 < o.qrows)
        dj[j] = *reinterpret_cast<const f4*>(g.adiag + t.off_d + cb + j * 16 + lk * 4);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      di[i] = 0.f;
      if (ST != kGram && rb + i * 16 < o.prows)
        di[i] = (ST == kPoly ? g.adiag : g.bdiag)[t.off_d + rb + i * 16 + lr];
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) own_rows(g, t, o, i);
  }

  // Four results of a lane, columns col to col + 3 of a row.
  __device__ __forceinline__ void direct(const GemmArgs& g, const MuonGemmTile& t,
                                         const Operands<ST, SPLIT>& o, int row, int col,
                                         float (&x)[4]) const {
    if constexpr (ST == kLast) {
      O* out = static_cast<O*>(g.ortho) + t.flat_off;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (row < t.m && col + r < t.n)
          El<O>::store(out + (t.mat & kMuonTall ? int64_t(col + r) * t.m + row : int64_t(row) * t.n + col + r),
                       x[r]);
    } else {
      _Float16* d[2] = {ST == kStep ? g.yh + t.off_x : (ST == kGram ? g.ah : g.bh) + t.off_a,
                        ST == kStep ? static_cast<_Float16*>(g.yl) + t.off_x
                               : (ST == kGram ? g.al : g.bl) + t.off_a};
      const int lane = threadIdx.x & 63;
      const uint32_t sel = lane & 1 ? 0x03020706u : 0x05040100u;
#pragma unroll
      for (int low = 0; low < (ST == kStep || SPLIT ? 2 : 1); ++low) {
        union {
          u2 u;
          h4 h;
        } v;
        v.u = pack4(x);
        if (kBytes && low) {
          *reinterpret_cast<uint32_t*>(static_cast<char*>(g.yl) + t.off_x +
                                       int64_t(row) * o.ld + col) = pack_bf8(x);
          continue;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] -= static_cast<float>(v.h[r]);
        *reinterpret_cast<u2*>(d[low] + int64_t(row) * o.ld + col) = v.u;
        if (kMirror && t.i != t.j)
          *reinterpret_cast<u2*>(d[low] + int64_t(col + (lr & 3)) * o.ld + row - (lr & 3)) =
              transpose4(v.u, sel, lane & 2);
      }
    }
  }

  // The results to where they belong, through `lds` (kOut bytes of the
  // wave's own).  acc is used up.
  __device__ __forceinline__ void finish(const GemmArgs& g, const MuonGemmTile& t,
                                         const Operands<ST, SPLIT>& o, f4 (&acc)[FM][FN],
                                         char* lds) {
    if (rb >= o.prows || cb >= o.qrows) return;
    const int lane = threadIdx.x & 63;
    float ca = 0.f, cb1 = 0.f, cc = 0.f;
    if constexpr (ST != kGram) {
      ca = __builtin_amdgcn_ldexpf(g.a * coef.a, coef.ea);
      cb1 = __builtin_amdgcn_ldexpf(g.b * coef.b, coef.eb);
      cc = __builtin_amdgcn_ldexpf(g.c * coef.c, coef.ec);
    }
    char* rows16 = lds;
    char* image = rows16 + kRows;
    constexpr int kImageLd = (TM + 8) * 2;
    const bool mirror = ST == kLast ? (t.mat & kMuonTall) != 0 : t.i != t.j;
    O* out = static_cast<O*>(g.ortho) + t.flat_off;  // kLast
    const bool tall = t.mat & kMuonTall;
    const int64_t cols = tall ? t.m : t.n;
    // 16 bytes of the result where the rows' and the base's alignment allow it
    const bool vec = ((reinterpret_cast<uintptr_t>(out) | (cols * 2)) & 15) == 0;
    auto put = [&](int64_t r, int64_t c, int64_t n_rows, u4 v) {
      if (r >= n_rows || c >= cols) return;
      u16* d = reinterpret_cast<u16*>(out) + r * cols + c;
      if (vec && c + 8 <= cols) {
        *reinterpret_cast<u4*>(d) = v;
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k < cols) d[k] = static_cast<u16>(v[k / 2] >> (16 * (k & 1)));
      }
    };
    // eight adjacent entries of a plane; it is padded to multiples of 64
    const int ld = o.ld;
    auto to = [&](_Float16* plane, int64_t first, int64_t second, int n_cols) {
      return [=](int r, int c, u4 v) {
        if (second + c < n_cols)
          *reinterpret_cast<u4*>(plane + (first + r) * ld + second + c) = v;
      };
    };
    _Float16* dh = ST == kStep ? g.yh + t.off_x : (ST == kGram ? g.ah : g.bh) + t.off_a;
    _Float16* dl = ST == kStep ? static_cast<_Float16*>(g.yl) + t.off_x
                               : (ST == kGram ? g.al : g.bl) + t.off_a;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if (rb + i * 16 >= o.prows) break;
      const int row = rb + i * 16 + lr;
      u2 hi[FN], lo[FN];
      uint32_t low8[FN];
      h4 h[FN];
      f4 l[FN];
      if constexpr (ST != kGram) spread(rows16, own_h[i % AHEAD], h);
      if constexpr (ST != kGram && kOwnLow) spread_low(rows16, own_l[i % AHEAD], l);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int col = cb + j * 16 + lk * 4;
        float x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float sum = acc[i][j][r];
          float own = 0.f;
          if constexpr (ST != kGram) own = static_cast<float>(h[j][r]);
          if constexpr (ST != kGram && kOwnLow) own += l[j][r];
          if constexpr (ST == kGram) {
            x[r] = sum * (kSa / (kSx * kSx));
          } else if constexpr (ST == kPoly) {
            x[r] = fmaf(fmaf(cc, di[i] + dj[j][r], cb1), own, cc * (sum * (1.f / kSa)));
          } else {
            x[r] = fmaf(ca + di[i], own, sum * (1.f / kSa));
            static_assert(kSx == 4096.f);
            if (ST == kLast) x[r] = __builtin_amdgcn_ldexpf(x[r], coef.q - 12);
          }
          if (kMirror && row == col + r) {
            if (ST == kGram)
              g.adiag[t.off_d + row] = x[r] * (1.f / kSa);
            else
              g.bdiag[t.off_d + row] = fmaf(di[i], fmaf(cc, di[i], cb1), x[r] * (1.f / kSa));
            x[r] = 0.f;
          }
        }
        if constexpr (kDirect) {
          direct(g, t, o, row, col, x);
        } else if constexpr (ST == kLast && sizeof(O) == 4) {
          // in the parameter's orientation, one element at a time
          float* f = reinterpret_cast<float*>(image);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int y = i * 16 + lr, z = j * 16 + lk * 4 + r;
            f[tall ? z * (TM + 1) + y : y * (TN + 1) + z] = x[r];
          }
        } else if constexpr (ST == kLast) {
          hi[j] = u2{f32_to_bf16(x[0]) | (f32_to_bf16(x[1]) << 16),
                     f32_to_bf16(x[2]) | (f32_to_bf16(x[3]) << 16)};
        } else {
          union {
            u2 u;
            h4 h;
          } v;
          v.u = hi[j] = pack4(x);
          if (ST == kStep || SPLIT) {
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] -= static_cast<float>(v.h[r]);
            if (kBytes)
              low8[j] = pack_bf8(x);
            else
              lo[j] = pack4(x);
          }
        }
      }
      if (i + AHEAD < FM) own_rows(g, t, o, i + AHEAD);
      if constexpr (!kDirect && !(ST == kLast && sizeof(O) == 4)) {
        const int r0 = rb + i * 16;
        if constexpr (ST == kLast) {
          if (!tall)
            store_rows<FN>(rows16, hi, [&](int r, int c, u4 v) { put(r0 + r, cb + c, t.m, v); });
        } else {
          store_rows<FN>(rows16, hi, to(dh, r0, cb, o.qrows));
          if constexpr (kBytes) {
            char* plane = static_cast<char*>(g.yl) + t.off_x;
            store_byte_rows<FN>(rows16, low8, [&](int r, int c, u2 v) {
              *reinterpret_cast<u2*>(plane + int64_t(r0 + r) * ld + cb + c) = v;
            });
          } else if constexpr (ST == kStep || SPLIT) {
            store_rows<FN>(rows16, lo, to(dl, r0, cb, o.qrows));
          }
        }
        if (ST != kStep && mirror) keep_transposed<FN>(image, kImageLd, i, hi);
        if constexpr (SPLIT && kMirror) {
#pragma unroll
          for (int j = 0; j < FN; ++j) {  // for a second image: over the sums
            acc[i][j][0] = __uint_as_float(lo[j].x);
            acc[i][j][1] = __uint_as_float(lo[j].y);
          }
        }
      }
    }
    if constexpr (kDirect) {
      return;
    } else if constexpr (ST == kLast && sizeof(O) == 4) {
      const float* f = reinterpret_cast<const float*>(image);
      const int n_rows = tall ? TN : TM, width = tall ? TM : TN;
      const int64_t r0 = tall ? cb : rb, c0 = tall ? rb : cb, last = tall ? t.n : t.m;
      for (int e = lane; e < n_rows * width; e += 64) {
        const int r = e / width, c = e % width;
        if (r0 + r < last && c0 + c < cols)
          out[(r0 + r) * cols + c0 + c] = f[r * (width + 1) + c];
      }
    } else if constexpr (ST == kLast) {
      if (mirror)
        store_image<TN, TM>(image, [&](int r, int c, u4 v) { put(cb + r, rb + c, t.n, v); });
    } else if constexpr (kMirror) {
      if (mirror) {
        // the image's rows are inside the plane: a tile below the diagonal
        // has its columns before its rows
        store_image<TN, TM>(image, to(dh, cb, rb, o.prows));
        if constexpr (SPLIT) {
#pragma unroll
          for (int i = 0; i < FM; ++i) {
            u2 lo[FN];
#pragma unroll
            for (int j = 0; j < FN; ++j)
              lo[j] = u2{__float_as_uint(acc[i][j][0]), __float_as_uint(acc[i][j][1])};
            keep_transposed<FN>(image, kImageLd, i, lo);
          }
          store_image<TN, TM>(image, to(dl, cb, rb, o.prows));
        }
      }
    }
  }
};

// Split operands: the matrix cores' sums go to a second set of accumulators
// every 128 of the depth.  One chain over a long positive sum (A's diagonal)
// loses 2^-24 of it at every link: 40 x 1025 measured 4.3e-6 off that way,
// three times what blocked fp32 sums are.
template <int FM, int FN>
__device__ __forceinline__ void zero(f4 (&x)[FM][FN]) {
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) x[i][j] = f4{0.f, 0.f, 0.f, 0.f};
}
template <int FM, int FN>
__device__ __forceinline__ void flush(f4 (&sum)[FM][FN], f4 (&acc)[FM][FN]) {
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) sum[i][j] += acc[i][j];
  zero(acc);
}

// One tile of a product, all waves on the same rounds.  A round's loads go
// straight to LDS, NS - 1 rounds ahead.  The products of one part of a round
// (32 of the sum) are issued row by row with the LDS reads of the next part
// and the loads of a later round between them: issued in one go, those loads
// keep a wave from its products for a thousand cycles.
//
// Measured on the hidden-4096 block (7 matrices, 256 x 256 tiles): A 736 us
// (1,260 TFLOP/s, diagonal tiles whole), B 325 (1,155), the step 1,527
// (1,125); alone, so without the clock's fall under load, the matrix cores are
// 73, 67 and 63% busy.  The rest is a tile's start and end (12% of 64 rounds)
// and the rounds' loads.
template <typename S, Stage ST, bool SPLIT, typename O>
__global__ __launch_bounds__(S::Threads, S::Waves - (SPLIT && S::BM > 64 ? 1 : 0)) void k_gemm(
    const MuonGemmTile* __restrict__ tiles, GemmArgs g) {
  constexpr int FM = S::FM, FN = S::FN, TM = S::TM, TN = S::TN, BK = S::BK, NS = S::NS;
  constexpr int LP = S::LP, LQ = S::LQ;
  constexpr bool kAcross = ST == kStep || ST == kLast;
  // what the results are added to is asked for before the sums, or, where
  // there is no room in registers, after them
  constexpr bool kEarly = S::BM <= 128;
  using Res = Result<FM, FN, kEarly ? FM : FM / 2, ST, SPLIT, O>;
  constexpr int kLds =
      S::RoundBytes * NS > Res::kOut * S::NW ? S::RoundBytes * NS : Res::kOut * S::NW;
  __shared__ __align__(128) char lds[kLds];

  const MuonGemmTile t = tile_of(tiles, g);
  if (t.mat < 0) return;  // filled up
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  const Operands<ST, SPLIT> o(g, t);
  const int i0 = t.i * S::BM, j0 = t.j * S::BN;
  const Loader<S, kAcross> loader(wave, i0, j0, o.prows, o.qrows, o.lp, o.lq);
  const Fetcher<S, kAcross> fetcher(wm, wn);
  static_assert(BK == kMuonRound);
  const int rounds = o.depth / BK;
  constexpr bool kParts = ST == kGram && S::BM == 64;
  const int first = kParts ? t.m : 0;
  const int total = kParts ? t.n : SPLIT ? 3 * rounds : rounds;
  const uint32_t lds0 = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)lds));

  f4 acc[FM][FN], sum[SPLIT ? FM : 1][SPLIT ? FN : 1];
  zero(acc);
  zero(sum);
  Res res;

  constexpr int KK = BK / 32;
  h8 p[2][FM], q[2][FN];
  // The products of operand set `set`, with the next operands (other set)
  // read from `buf`, part kk, and with LOADS the loads of round f into
  // buffer `into` between their rows.
  auto products = [&](int set, int buf, int kk, auto loads, const From& f, int into) {
    constexpr int kFetch = FM + FN, kLoad = LP + LQ;
    const char* image = lds + buf * S::RoundBytes;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
      for (int x = i * kFetch / FM; x < (i + 1) * kFetch / FM; ++x) {
        if (x < FN)
          q[set ^ 1][x] = fetcher.q(image, kk, x);
        else
          p[set ^ 1][x - FN] = fetcher.p(image, kk, x - FN);
      }
      if constexpr (decltype(loads)::value) {
#pragma unroll
        for (int x = i * kLoad / FM; x < (i + 1) * kLoad / FM; ++x)
          loader.load(f, lds0 + into * S::RoundBytes, x);
      }
#pragma unroll
      for (int j = 0; j < FN; ++j)
        acc[i][j] =
            __builtin_amdgcn_mfma_f32_16x16x32_f16(q[set][j], p[set][i], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

#pragma unroll
  for (int s = 0; s < NS; ++s)
    if (s < total) {
      const From f = from_round<BK>(o, first + s, rounds);
#pragma unroll
      for (int x = 0; x < LP + LQ; ++x) loader.load(f, lds0 + s * S::RoundBytes, x);
    }
  if constexpr (kEarly) res.ask(g, t, o, i0 + wm * TM, j0 + wn * TN);
  if (total >= NS)
    wait_and_meet<(NS - 1) * (LP + LQ)>();
  else
    wait_and_meet<0>();
#pragma unroll
  for (int j = 0; j < FN; ++j) q[0][j] = fetcher.q(lds, 0, j);
#pragma unroll
  for (int i = 0; i < FM; ++i) p[0][i] = fetcher.p(lds, 0, i);
  // Before a round's last part: the next round has landed for every wave, and
  // every wave is done reading this one, whose buffer is loaded again.  The
  // last round reads operands that nothing uses: with a tail of its own the
  // accumulators were copied around in every round.
  int buf = 0;
  auto one = [&](int it, auto loads) {
    const int next = buf + 1 == NS ? 0 : buf + 1;
    constexpr int kWait = decltype(loads)::value ? (NS - 2) * (LP + LQ) : 0;
    From f{};
    static_assert(KK == 2);
    wait_lds();  // set 0: asked for half a round ago
    products(0, buf, 1, std::false_type{}, f, 0);
    wait_and_meet<kWait>();
    if (decltype(loads)::value) f = from_round<BK>(o, first + it + NS, rounds);
    products(1, next, 0, loads, f, buf);
    if constexpr (SPLIT) {
      if (it & 1) flush(sum, acc);
    }
    buf = next;
  };
  int it = 0;
  for (; it + NS < total; ++it) one(it, std::true_type{});
  for (; it < total; ++it) one(it, std::false_type{});
  if constexpr (SPLIT) {
    flush(sum, acc);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = sum[i][j];
  }

  if constexpr (kParts) {
    if (t.flat_off >= 0) {  // a part
      f4* to = reinterpret_cast<f4*>(g.sums) + t.flat_off * (FM * FN * S::Threads) + threadIdx.x;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) to[(i * FN + j) * S::Threads] = acc[i][j];
      return;
    }
  }
  if constexpr (!kEarly) res.ask(g, t, o, i0 + wm * TM, j0 + wn * TN);
  __syncthreads();  // every wave is done with the operands in LDS
  res.finish(g, t, o, acc, lds + wave * Res::kOut);
}

// A 32 x 32 tile with the sum dealt over 4 waves: wave w takes rounds w, w +
// 4, ... with loads, LDS and accumulators of its own, so nothing is waited
// for but its own loads until the four are added up, each wave one 16 x 16
// part.  For few tiles: a compute unit takes in 46 bytes a cycle, so with 64
// x 64 tiles the operands of a sum of 512 alone are 2,800 cycles (1.3 us of
// a launch's 6), and most compute units have no tile.  A's may be parts of a
// sum (k_join).
template <typename S, Stage ST, bool SPLIT, typename O>
__global__ __launch_bounds__(256, S::Waves) void k_thin(
    const MuonGemmTile* __restrict__ tiles, GemmArgs g) {
  constexpr int BK = S::BK, NS = S::NS, kLoads = S::LP + S::LQ, KK = BK / 32;
  constexpr int FM = S::FM, FN = S::FN;
  static_assert(S::NW == 1 && FM * FN == 4);
  constexpr bool kAcross = ST == kStep || ST == kLast;
  constexpr int kOwn = S::RoundBytes * NS;
  static_assert(kOwn >= FM * FN * 1024);
  __shared__ __align__(128) char lds[4 * kOwn];

  const MuonGemmTile t = tile_of(tiles, g);
  if (t.mat < 0) return;  // filled up
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Operands<ST, SPLIT> o(g, t);
  const int i0 = t.i * S::BM, j0 = t.j * S::BN;
  static_assert(BK == kMuonRound);
  const int rounds = o.depth / BK;
  const int first = ST == kGram ? t.m : 0;
  const int total = ST == kGram ? t.n : SPLIT ? 3 * rounds : rounds;
  const int mine = (total - wave + 3) / 4;  // total > 0; none for wave >= total
  char* own = lds + wave * kOwn;
  const uint32_t own0 =
      static_cast<uint32_t>(
          reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)lds)) +
      wave * kOwn;
  Result<1, 1, 1, ST, SPLIT, O> res;
  const Loader<S, kAcross> loader(0, i0, j0, o.prows, o.qrows, o.lp, o.lq);
  const Fetcher<S, kAcross> fetcher(0, 0);
  auto issue = [&](int r, int buf) {
    const From f = from_round<BK>(o, first + wave + 4 * r, rounds);
#pragma unroll
    for (int x = 0; x < kLoads; ++x) loader.load(f, own0 + buf * S::RoundBytes, x);
  };
#pragma unroll
  for (int s = 0; s < NS; ++s)
    if (s < mine) issue(s, s);
  res.ask(g, t, o, i0 + wave / FN * 16, j0 + wave % FN * 16);

  f4 acc[FM][FN], sum[SPLIT ? FM : 1][SPLIT ? FN : 1];
  zero(acc);
  zero(sum);
  int buf = 0;
  for (int r = 0; r < mine; ++r) {
    if (r + NS <= mine)
      wait_loads<(NS - 1) * kLoads>();
    else
      wait_loads<0>();
    h8 p[KK][FM], q[KK][FN];
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
#pragma unroll
      for (int j = 0; j < FN; ++j) q[kk][j] = fetcher.q(own + buf * S::RoundBytes, kk, j);
#pragma unroll
      for (int i = 0; i < FM; ++i) p[kk][i] = fetcher.p(own + buf * S::RoundBytes, kk, i);
    }
    if (r + NS < mine) {
      wait_lds();  // the buffer is read: load it again
      asm volatile("" ::: "memory");
      issue(r + NS, buf);
    }
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] =
              __builtin_amdgcn_mfma_f32_16x16x32_f16(q[kk][j], p[kk][i], acc[i][j], 0, 0, 0);
    if constexpr (SPLIT) flush(sum, acc);
    buf = buf + 1 == NS ? 0 : buf + 1;
  }
  // the four waves' sums, in their order
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      if constexpr (SPLIT) acc[i][j] = sum[i][j];
      *reinterpret_cast<f4*>(own + ((i * FN + j) * 64 + lane) * 16) = acc[i][j];
    }
  __syncthreads();
  f4 all[1][1];
  all[0][0] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < 4; ++w)
    all[0][0] += *reinterpret_cast<const f4*>(lds + w * kOwn + (wave * 64 + lane) * 16);
  if (ST == kGram && t.flat_off >= 0)  // a part
    reinterpret_cast<f4*>(g.sums)[t.flat_off * 256 + threadIdx.x] = all[0][0];
  else
    res.finish(g, t, o, all, nullptr);
}

// A's tiles whose sums came in parts: the parts in their order, four chains
// of them, and to where k_thin's (F = 1) or k_gemm's (F = 2) own go.  A lane
// has F x F f4's of each part.  8.4 us for 36 tiles of 15 parts (512 x 32000,
// the parts 17.7), 23 us for 3 of 171 (32 x 1M, the parts 32: a workgroup
// reads 700 KB alone).
template <int F, bool SPLIT>
__global__ __launch_bounds__(256) void k_join(const MuonGemmTile* __restrict__ tiles, GemmArgs g) {
  const MuonGemmTile t = tile_of(tiles, g);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Operands<kGram, SPLIT> o(g, t);
  using Res = Result<F, F, F, kGram, SPLIT, u16>;
  __shared__ __align__(16) char lds[F == 1 ? 16 : 4 * Res::kOut];
  Res res;
  res.ask(g, t, o, (t.i * 2 + wave / 2) * 16 * F, (t.j * 2 + wave % 2) * 16 * F);
  constexpr int N = F * F;
  const f4* from = reinterpret_cast<const f4*>(g.sums) + t.flat_off * (N * 256) + threadIdx.x;
  f4 chain[4][N];
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int x = 0; x < N; ++x) chain[k][x] = f4{0.f, 0.f, 0.f, 0.f};
  int p = 0;
#pragma unroll 2
  for (; p + 4 <= t.n; p += 4)
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int x = 0; x < N; ++x) chain[k][x] += from[((p + k) * N + x) * 256];
  for (; p < t.n; ++p)
#pragma unroll
    for (int x = 0; x < N; ++x) chain[0][x] += from[(p * N + x) * 256];
  f4 all[F][F];
#pragma unroll
  for (int x = 0; x < N; ++x)
    all[x / F][x % F] = (chain[0][x] + chain[1][x]) + (chain[2][x] + chain[3][x]);
  res.finish(g, t, o, all, F == 1 ? nullptr : lds + wave * Res::kOut);
}

// `from`: which plane holds X.  Its low parts are replaced in place, by the
// workgroup that reads them, unless they are an operand too.
GemmArgs gemm_args(const MuonArgs& a, int from) {
  auto half = [&](int64_t off) { return reinterpret_cast<_Float16*>(a.ws + off); };
  GemmArgs g{};
  g.coef = reinterpret_cast<const MuonCoef*>(a.ws + a.w.coef) + a.step;
  g.adiag = reinterpret_cast<float*>(a.ws + a.w.adiag);
  g.bdiag = reinterpret_cast<float*>(a.ws + a.w.bdiag);
  g.xh = half(a.w.xh[from]);
  g.xl = a.ws + a.w.xl[from];
  g.yh = half(a.w.xh[1 - from]);
  g.yl = a.ws + a.w.xl[1 - from];
  g.ah = half(a.w.ah);
  g.al = half(a.w.al);
  g.bh = half(a.w.bh);
  g.bl = half(a.w.bl);
  g.sums = reinterpret_cast<float*>(a.ws + a.w.sums);
  return g;
}

using Thin = Shape<32, 32, 1, 1, 64, 2, 2>;  // per wave
using Small = Shape<64, 64, 2, 2, 64, 3, 2>;
using Mid = Shape<128, 128, 2, 2, 64, 2, 2>;
using Big = Shape<256, 256, 2, 4, 64, 2, 2>;
static_assert(Thin::BM == kMuonTiles[0] && Small::BM == kMuonTiles[1] &&
              Mid::BM == kMuonTiles[2] && Big::BM == kMuonTiles[3]);

template <typename S, Stage ST, bool SPLIT, typename O>
hipError_t launch_shape(const MuonTiles& t, GemmArgs& g, const Sink& sink) {
  const int64_t n = t.n;
  const MuonGemmTile* tiles = t.tiles;
  void* p[] = {&tiles, &g};
  if constexpr (S::NW == 1)
    return sink.launch(reinterpret_cast<const void*>(&k_thin<S, ST, SPLIT, O>),
                       dim3(static_cast<unsigned>(n)), dim3(256), p, 0);
  else
    return sink.launch(reinterpret_cast<const void*>(&k_gemm<S, ST, SPLIT, O>),
                       dim3(static_cast<unsigned>(n)), dim3(S::Threads), p, 0);
}

template <Stage ST, typename O>
hipError_t launch_gemm(bool split, const MuonTiles& t, GemmArgs& g, const Sink& sink) {
  if (t.n <= 0) return hipErrorInvalidValue;
  if constexpr (!(ST == kLast && sizeof(O) == 2)) {
    if (split) {
      switch (t.shape) {
        case 0: return launch_shape<Thin, ST, true, O>(t, g, sink);
        case 1: return launch_shape<Small, ST, true, O>(t, g, sink);
        default: return launch_shape<Mid, ST, true, O>(t, g, sink);
      }
    }
  }
  if constexpr (ST == kLast && sizeof(O) == 4) {
    return hipErrorInvalidValue;  // fp32 results take split operands
  } else {
    switch (t.shape) {
      case 0: return launch_shape<Thin, ST, false, O>(t, g, sink);
      case 1: return launch_shape<Small, ST, false, O>(t, g, sink);
      case 2: return launch_shape<Mid, ST, false, O>(t, g, sink);
      default: return launch_shape<Big, ST, false, O>(t, g, sink);
    }
  }
}

template <typename G, typename U, int RT, int N>
hipError_t momentum_n(const MuonItem* items, int64_t n, const PtrArray& grads, int R, float* m,
                      void* update, const MuonScalars& sc, bool vec, const Sink& sink) {
  MomentumArgs<N> a{};
  for (int q = 0; q < N && q < R; ++q) a.g[q] = grads.p[q];
  a.R = R;
  a.m = m;
  a.update = update;
  a.sc = sc;
  a.vec = vec;
  void* p[] = {&items, &a};
  return sink.launch(reinterpret_cast<const void*>(&k_momentum<G, U, RT, N>),
                     dim3(static_cast<unsigned>(n)), dim3(kThreads), p, 0);
}

template <typename G, typename U>
hipError_t momentum_r(const MuonItem* items, int64_t n, const PtrArray& grads, int R,
                      bool replicas, float* m, void* update, const MuonScalars& sc, bool vec,
                      const Sink& sink) {
  if (!replicas)
    return momentum_n<float, U, -1, 1>(items, n, grads, 1, m, update, sc, vec, sink);
  switch (R) {
    case 1: return momentum_n<G, U, 1, 8>(items, n, grads, R, m, update, sc, vec, sink);
    case 2: return momentum_n<G, U, 2, 8>(items, n, grads, R, m, update, sc, vec, sink);
    case 3: return momentum_n<G, U, 3, 8>(items, n, grads, R, m, update, sc, vec, sink);
    case 4: return momentum_n<G, U, 4, 8>(items, n, grads, R, m, update, sc, vec, sink);
    case 8: return momentum_n<G, U, 8, 8>(items, n, grads, R, m, update, sc, vec, sink);
    default:
      return momentum_n<G, U, 0, FSDP_MAX_RANKS>(items, n, grads, R, m, update, sc, vec, sink);
  }
}

}  // namespace

hipError_t launch_muon_momentum(const MuonItem* items, int64_t n, const PtrArray& grads, int R,
                                int grad_dt, bool replicas, float* m, void* update, int update_dt,
                                const MuonScalars& sc, bool vec, const Sink& sink) {
  if (n <= 0) return hipErrorInvalidValue;
  const bool gb = grad_dt == FSDP_BF16, ub = update_dt == FSDP_BF16;
  if (gb && ub) return momentum_r<u16, u16>(items, n, grads, R, replicas, m, update, sc, vec, sink);
  if (gb) return momentum_r<u16, float>(items, n, grads, R, replicas, m, update, sc, vec, sink);
  if (ub) return momentum_r<float, u16>(items, n, grads, R, replicas, m, update, sc, vec, sink);
  return momentum_r<float, float>(items, n, grads, R, replicas, m, update, sc, vec, sink);
}

hipError_t launch_muon_apply(const MuonItem* items, int64_t n, const MuonScale* scales,
                             const void* ortho, int ortho_dt, float* master, void* param,
                             int param_dt, const MuonScalars& sc, bool vec, const Sink& sink) {
  if (n <= 0) return hipErrorInvalidValue;
  ApplyArgs a{scales, ortho, master, param, sc, vec};
  const bool ob = ortho_dt == FSDP_BF16, pb = param_dt == FSDP_BF16;
  const void* fn = ob ? (pb ? reinterpret_cast<const void*>(&k_apply<u16, u16>)
                            : reinterpret_cast<const void*>(&k_apply<u16, float>))
                      : (pb ? reinterpret_cast<const void*>(&k_apply<float, u16>)
                            : reinterpret_cast<const void*>(&k_apply<float, float>));
  void* p[] = {&items, &a};
  return sink.launch(fn, dim3(static_cast<unsigned>(n)), dim3(kThreads), p, 0);
}

hipError_t launch_muon_norm(const MuonArgs& a, const MuonChunk* tiles, int64_t n,
                            const void* update, int dt, const Sink& sink) {
  if (n <= 0) return hipErrorInvalidValue;
  double* partial = reinterpret_cast<double*>(a.ws + a.w.partial);
  void* p[] = {&tiles, &update, &partial};
  const void* fn = dt == FSDP_BF16 ? reinterpret_cast<const void*>(&k_norm<u16>)
                                   : reinterpret_cast<const void*>(&k_norm<float>);
  return sink.launch(fn, dim3(static_cast<unsigned>(n)), dim3(kThreads), p, 0);
}

hipError_t launch_muon_convert(const MuonArgs& a, const MuonConvertTile* tiles, int64_t n,
                               const void* update, int dt, double eps, const double (&poly)[3],
                               const Sink& sink) {
  if (n <= 0) return hipErrorInvalidValue;
  auto half = [&](int64_t off) { return reinterpret_cast<_Float16*>(a.ws + off); };
  ConvertArgs c{};
  c.tiles = tiles;
  c.partial = reinterpret_cast<const double*>(a.ws + a.w.partial);
  c.coef = reinterpret_cast<MuonCoef*>(a.ws + a.w.coef);
  c.steps = a.steps;
  c.xh = half(a.w.xh[0]);
  c.xl = a.low ? a.ws + a.w.xl[0] : nullptr;
  c.bytes = !a.split;
  c.eps = eps;
  c.a = poly[0];
  c.b = poly[1];
  c.c = poly[2];
  void* p[] = {&update, &c};
  const void* fn = dt == FSDP_BF16 ? reinterpret_cast<const void*>(&k_convert<u16>)
                                   : reinterpret_cast<const void*>(&k_convert<float>);
  return sink.launch(fn, dim3(static_cast<unsigned>(n)), dim3(kThreads), p, 0);
}

hipError_t launch_muon_gram(const MuonArgs& a, const MuonTiles& t, const MuonTiles& join, int from,
                            const Sink& sink) {
  GemmArgs g = gemm_args(a, from);
  const hipError_t e = launch_gemm<kGram, u16>(a.split, t, g, sink);
  if (e != hipSuccess || join.n == 0) return e;
  const MuonGemmTile* tiles = join.tiles;
  void* p[] = {&tiles, &g};
  const void* fn = t.shape == 0 ? (a.split ? reinterpret_cast<const void*>(&k_join<1, true>)
                                           : reinterpret_cast<const void*>(&k_join<1, false>))
                                : (a.split ? reinterpret_cast<const void*>(&k_join<2, true>)
                                           : reinterpret_cast<const void*>(&k_join<2, false>));
  return sink.launch(fn, dim3(static_cast<unsigned>(join.n)), dim3(256), p, 0);
}

hipError_t launch_muon_poly(const MuonArgs& a, const MuonTiles& t, bool first,
                            const double (&poly)[3], const Sink& sink) {
  GemmArgs g = gemm_args(a, 0);
  g.b = first ? 1.f : static_cast<float>(poly[1]);
  g.c = first ? 1.f : static_cast<float>(poly[2]);
  return launch_gemm<kPoly, u16>(a.split, t, g, sink);
}

hipError_t launch_muon_step(const MuonArgs& a, const MuonTiles& t, int from, bool first,
                            bool last, const double (&poly)[3], void* ortho, int ortho_dt,
                            const Sink& sink) {
  GemmArgs g = gemm_args(a, from);
  g.a = first ? 1.f : static_cast<float>(poly[0]);
  if (first && !a.low) g.xl = nullptr;
  g.ortho = ortho;
  if (!last) return launch_gemm<kStep, u16>(a.split, t, g, sink);
  return ortho_dt == FSDP_BF16 ? launch_gemm<kLast, u16>(a.split, t, g, sink)
                               : launch_gemm<kLast, float>(a.split, t, g, sink);
}

}  // namespace fsdp
