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
// 1.1-4.7e-3, and fp16 with two things kept finer 0.5-7e-4: the residual a X
// is read as fp16 high and low parts (its small singular directions would
// otherwise carry the rounding of the large ones, amplified by a each
// step), and the diagonals of A and B, their largest part once X is near
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
// largest still keeps all its bits.
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
// lines.
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
  const MuonMat* mats;
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
  const double rows = static_cast<double>(a.mats[w.mat].rows);
  const double cols = static_cast<double>(a.mats[w.mat].cols);
  double rate = a.sc.lr;
  if (a.sc.scale == FSDP_MUON_SCALE_ASPECT)
    rate *= sqrt(fmax(1.0, rows / cols));
  else if (a.sc.scale == FSDP_MUON_SCALE_RMS)
    rate *= 0.2 * sqrt(fmax(rows, cols));
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
// neither infinite nor lost.  One workgroup per chunk.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_norm(const MuonMat* __restrict__ mats,
                                                   const MuonTile* __restrict__ tiles,
                                                   const T* __restrict__ update,
                                                   double* __restrict__ partial) {
  const MuonTile t = tiles[blockIdx.x];
  const MuonMat& mat = mats[t.mat];
  const int64_t lo = int64_t(t.i) * mat.norm_chunk;
  const int64_t n = mat.rows * mat.cols;
  const int64_t hi = lo + mat.norm_chunk < n ? lo + mat.norm_chunk : n;
  const T* u = update + mat.flat_off;
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
  if (threadIdx.x == 0) partial[mat.norm_first + t.i] = s;
}

struct ConvertArgs {
  const MuonMat* mats;
  const MuonTile* tiles;
  const double* partial;
  float* coef;  // per matrix: a f, b f^3, c f^5
  _Float16 *xh, *xl;  // xl null: the low parts are not wanted
  double eps, a, b, c;
};

// 64 x 64 tiles of the update into X, transposed where the parameter has
// more rows than columns.  With |U| + eps = N, the planes get U 2^-e with
// 2^e <= N < 2^(e+1): exact for bf16 updates.  What is left, f = 2^e / N,
// goes into the first step's coefficients: A is then A f^-2 and X is X f^-1.
// A lane has 16 adjacent entries of a row.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_convert(const T* __restrict__ update,
                                                      ConvertArgs a) {
  constexpr int Ld = 72;
  __shared__ __align__(16) _Float16 tile[64 * Ld];
  const MuonTile t = a.tiles[blockIdx.x];
  const MuonMat& mat = a.mats[t.mat];
  const int64_t r0 = int64_t(t.i) * 64, c0 = int64_t(t.j) * 64;
  const int lr = threadIdx.x >> 2, lc = (threadIdx.x & 3) * 16;
  const int64_t r = r0 + lr, c = c0 + lc;
  const T* u = update + mat.flat_off + r * mat.cols + c;
  float x[16];
  if (r < mat.rows && c + 16 <= mat.cols &&
      (reinterpret_cast<uintptr_t>(u) & (4 * sizeof(T) - 1)) == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float y[4];
      El<T>::load4(u + 4 * k, y);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[4 * k + q] = y[q];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k)
      x[k] = r < mat.rows && c + k < mat.cols ? El<T>::load(u + k) : 0.f;
  }
  double s = 0;
  for (int k = threadIdx.x; k < mat.norm_count; k += kThreads)
    s += a.partial[mat.norm_first + k];
  const double norm = sqrt(block_sum(s)) + a.eps;
  const int e = ilogb(norm);
  const double scale = ldexp(static_cast<double>(kSx), -e);
  if (t.i == 0 && t.j == 0 && threadIdx.x == 0) {
    const double f = ldexp(1.0, e) / norm;
    const bool bad = !(norm < INFINITY);
    float* k = a.coef + 4 * t.mat;
    k[0] = bad ? NAN : static_cast<float>(a.a * f);
    k[1] = bad ? NAN : static_cast<float>(a.b * f * f * f);
    k[2] = bad ? NAN : static_cast<float>(a.c * f * f * f * f * f);
  }
  union {
    _Float16 h[16];
    u4 v[2];
  } part;
#pragma unroll
  for (int k = 0; k < 16; ++k) x[k] = static_cast<float>(static_cast<double>(x[k]) * scale);
  for (int low = 0; low < (a.xl ? 2 : 1); ++low) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      part.h[k] = static_cast<_Float16>(x[k]);
      x[k] -= static_cast<float>(part.h[k]);
    }
    _Float16* out = (low ? a.xl : a.xh) + mat.off_x;
    if (!mat.tall) {
      u4* d = reinterpret_cast<u4*>(out + r * mat.ldx + c);
      d[0] = part.v[0];
      d[1] = part.v[1];
    } else {
      __syncthreads();
      u4* d = reinterpret_cast<u4*>(tile + lr * Ld + lc);
      d[0] = part.v[0];
      d[1] = part.v[1];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 16; ++k) part.h[k] = tile[(lc + k) * Ld + lr];
      d = reinterpret_cast<u4*>(out + (c0 + lr) * mat.ldx + r0 + lc);
      d[0] = part.v[0];
      d[1] = part.v[1];
    }
  }
}

// ---------------------------------------------------------------- products
struct GemmArgs {
  const MuonGemmTile* tiles;
  const float* coef;  // non-null: the first step's coefficients, per matrix
  float a, b, c;      // the other steps'
  float *adiag, *bdiag;  // the diagonals of A and B
  const _Float16 *xh, *xl;  // X of this step (xl null in the first one: zeros)
  _Float16 *yh, *yl;        // X of the next
  _Float16 *ah, *al, *bh, *bl;
  void* ortho;
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
// alternate by themselves with bit 0.
template <int BN>
__device__ __forceinline__ int place_across(int r, int c) {
  const int b = (r & 3) | ((r >> 1) & 4);
  return c ^ (BN == 64 ? b & 6 : b << 1);
}

// 16 bytes per lane from global memory to LDS at a wave-uniform address, lane
// after lane.  An asm statement (it writes no register): of the builtin the
// compiler waits for all loads under way before every transposing LDS read,
// which it cannot tell from a read of the bytes being loaded.  Waited for by
// wait_and_meet.
__device__ __forceinline__ void load_to_lds(const void* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from),
               "s"(__builtin_amdgcn_readfirstlane(to))
               : "memory");
}

// Wait until at most N of this wave's global accesses are under way and all
// its LDS reads are done (the builtin, not an asm statement: the compiler
// counts on from it), then for the other waves.
__device__ __forceinline__ void wait_lds() {
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));
}
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

// One tile of a product.  A round's loads go straight to LDS, NS - 1 rounds
// ahead.  The products of one part of a round (32 of the sum) are issued row
// by row with the LDS reads of the next part and the loads of a later round
// between them: issued in one go, those loads keep a wave from its products
// for a thousand cycles.  Operand rows and columns past the plane's last are
// read from the last ones; their results are not stored.
template <typename S, Stage ST, bool SPLIT, typename O>
__global__ __launch_bounds__(S::Threads, S::Waves - (SPLIT && S::BM > 64 ? 1 : 0)) void k_gemm(
    GemmArgs g) {
  constexpr int FM = S::FM, FN = S::FN, TM = S::TM, TN = S::TN, BK = S::BK, NS = S::NS;
  constexpr int BM = S::BM, BN = S::BN, RB = S::RB, LP = S::LP, LQ = S::LQ;
  constexpr bool kAcross = ST == kStep || ST == kLast;  // Q lies across the sum
  constexpr bool kMirror = ST == kGram || ST == kPoly;
  // a wave's part of LDS after the sums: 16 rows, and a transposed image
  // (fp32 results: one of fp32, either way round)
  constexpr int kRows = 16 * (TN + 8) * 2;
  constexpr int kImage = ST == kStep ? 0 : TN * (TM + 8) * 2;
  constexpr int kOut = ST == kLast && sizeof(O) == 4 ? (TM + 1) * (TN + 1) * 4 : kImage + kRows;
  constexpr int kLds = S::RoundBytes * NS > kOut * S::NW ? S::RoundBytes * NS : kOut * S::NW;
  __shared__ __align__(128) char lds[kLds];

  const MuonGemmTile t = g.tiles[blockIdx.x];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int lr = lane & 15, lk = lane >> 4;

  const int mp = t.mp, np = t.np;
  const _Float16 *ph, *pl = nullptr, *qh, *ql = nullptr;
  int prows, qrows, depth;
  int ld, lp, lq;  // of the result and of the operands
  if constexpr (ST == kGram) {
    ph = qh = g.xh + t.off_x;
    if (SPLIT) pl = ql = g.xl + t.off_x;
    prows = qrows = mp;
    ld = t.lda;
    lp = lq = t.ldx;
    depth = np;
  } else if constexpr (ST == kPoly) {
    ph = qh = g.ah + t.off_a;
    if (SPLIT) pl = ql = g.al + t.off_a;
    prows = qrows = mp;
    ld = lp = lq = t.lda;
    depth = mp;
  } else {
    ph = g.bh + t.off_a;
    qh = g.xh + t.off_x;
    if (SPLIT) {
      pl = g.bl + t.off_a;
      ql = g.xl + t.off_x;
    }
    prows = mp;
    qrows = np;
    lp = t.lda;
    ld = lq = t.ldx;
    depth = mp;
  }
  const int i0 = t.i * BM, j0 = t.j * BN;

  // this lane's part of a round's loads, from the round's first element
  int64_t po[LP], qo[LQ];
  {
    constexpr int PerRow = BK / 8;
    const int r = lane / PerRow, c = place<BK>(r, lane % PerRow);
#pragma unroll
    for (int k = 0; k < LP; ++k) {
      const int row = i0 + (wave * LP + k) * S::RowsPerLoad + r;
      po[k] = int64_t(row < prows ? row : prows - 1) * lp + c * 8;
    }
    if constexpr (kAcross) {
      constexpr int Chunks = BN / 8, Rows = 64 / Chunks;
#pragma unroll
      for (int k = 0; k < LQ; ++k) {
        const int row = (wave * LQ + k) * Rows + lane / Chunks;
        const int col = j0 + place_across<BN>(row, lane % Chunks) * 8;
        qo[k] = int64_t(row) * lq + (col < np ? col : np - 8);
      }
    } else {
#pragma unroll
      for (int k = 0; k < LQ; ++k) {
        const int row = j0 + (wave * LQ + k) * S::RowsPerLoad + r;
        qo[k] = int64_t(row < qrows ? row : qrows - 1) * lq + c * 8;
      }
    }
  }
  const int64_t qstep = kAcross ? int64_t(BK) * lq : BK;
  const int rounds = depth / BK;
  const int total = SPLIT ? 3 * rounds : rounds;
  // where round `it` begins in P and Q
  struct From {
    const _Float16 *p, *q;
  };
  auto from = [&](int it) {
    From f{ph, qh};
    int k = it;
    if constexpr (SPLIT) {  // the small products first: high low, low high, high high
      const int part = it / rounds;
      k = it - part * rounds;
      if (part == 0) f.q = ql;
      if (part == 1) f.p = pl;
    }
    f.p += int64_t(k) * BK;
    f.q += k * qstep;
    return f;
  };
  // load x of a round's LP + LQ
  const uint32_t lds0 = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)lds));
  auto load = [&](const From& f, int buf, int x) {
    const uint32_t base = lds0 + buf * S::RoundBytes + (x < LP ? 0 : BM * RB);
    const _Float16* from1 = x < LP ? f.p + po[x < LP ? x : 0] : f.q + qo[x < LP ? 0 : x - LP];
    const int at = x < LP ? wave * LP + x : wave * LQ + x - LP;
    load_to_lds(from1, base + at * 1024);
  };

  f4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};

  // Split operands: the matrix cores' sums go to a second set of
  // accumulators every 128 of the depth.  One chain over a long positive sum
  // (A's diagonal) loses 2^-24 of it at every link: 40 x 1025 measured
  // 4.3e-6 off that way, three times what blocked fp32 sums are.
  f4 sum[SPLIT ? FM : 1][SPLIT ? FN : 1];
  auto flush = [&] {
    if constexpr (SPLIT) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          sum[i][j] += acc[i][j];
          acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};
        }
    }
  };
  if constexpr (SPLIT) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) sum[i][j] = f4{0.f, 0.f, 0.f, 0.f};
  }

  // ---- LDS to registers
  constexpr int KK = BK / 32;
  h8 p[2][FM], q[2][FN];
  const int pat = (wm * TM + lr) * RB;
  int qat[kAcross ? FN : 1];
  if constexpr (kAcross) {
    const int row = lk * 8 + (lr >> 2);  // and 4 more for the second half
#pragma unroll
    for (int j = 0; j < FN; ++j)
      qat[j] = BM * RB + row * BN * 2 +
               place_across<BN>(row, wn * (TN / 8) + j * 2 + ((lr & 3) >> 1)) * 16 +
               (lr & 1) * 8;
  } else {
    qat[0] = BM * RB + (wn * TN + lr) * RB;
  }
  auto fetch_p = [&](int buf, int kk, int set, int i) {
    p[set][i] = *reinterpret_cast<const h8*>(lds + buf * S::RoundBytes +
                                             place<BK>(lr, kk * 4 + lk) * 16 + pat +
                                             i * 16 * RB);
  };
  auto fetch_q = [&](int buf, int kk, int set, int j) {
    if constexpr (kAcross) {
      typedef short s4 __attribute__((ext_vector_type(4)));
      union {
        s4 s[2];
        h8 h;
      } v;
#pragma unroll
      for (int half = 0; half < 2; ++half)
        v.s[half] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s4*)(lds + buf * S::RoundBytes + qat[j] +
                                                    (kk * 32 + half * 4) * BN * 2));
      q[set][j] = v.h;
    } else {
      q[set][j] = *reinterpret_cast<const h8*>(lds + buf * S::RoundBytes +
                                               place<BK>(lr, kk * 4 + lk) * 16 + qat[0] +
                                               j * 16 * RB);
    }
  };
  // The products of operand set `set`, with the next operands (other set)
  // read from `buf`, part kk, and with LOADS the loads of round f into
  // buffer `into` between their rows.
  auto products = [&](int set, int buf, int kk, auto loads, const From& f, int into) {
    constexpr int kFetch = FM + FN, kLoad = LP + LQ;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
      for (int x = i * kFetch / FM; x < (i + 1) * kFetch / FM; ++x) {
        if (x < FN)
          fetch_q(buf, kk, set ^ 1, x);
        else
          fetch_p(buf, kk, set ^ 1, x - FN);
      }
      if constexpr (decltype(loads)::value) {
#pragma unroll
        for (int x = i * kLoad / FM; x < (i + 1) * kLoad / FM; ++x) load(f, into, x);
      }
#pragma unroll
      for (int j = 0; j < FN; ++j)
        acc[i][j] =
            __builtin_amdgcn_mfma_f32_16x16x32_f16(q[set][j], p[set][i], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // What the results are added to: A's or X's own entries, 16 rows at a time,
  // Ahead sets of them in registers: all, asked for before the sums begin, or
  // as many as fit after them.  Loads and stores are waited for in order, so
  // with one set ahead each set waited for the stores of the one before.
  const int rb = i0 + wm * TM, cb = j0 + wn * TN;
  constexpr bool kEarly = S::BM <= 128;
  constexpr int Ahead = kEarly ? FM : FM / 2;
  const _Float16* oh = ST == kPoly ? ph : qh;
  const _Float16* ol = ST == kPoly ? pl : (g.xl ? g.xl + t.off_x : nullptr);
  h4 h[Ahead][FN], l[Ahead][FN];
  auto own_rows = [&](int i) {
    const int64_t at = int64_t(rb + i * 16 + lr) * ld + cb + lk * 4;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      h[i % Ahead][j] = l[i % Ahead][j] = h4{0, 0, 0, 0};
      if (ST != kGram && rb + i * 16 < prows && cb + j * 16 < qrows) {
        h[i % Ahead][j] = *reinterpret_cast<const h4*>(oh + at + j * 16);
        if ((kAcross || SPLIT) && ol)
          l[i % Ahead][j] = *reinterpret_cast<const h4*>(ol + at + j * 16);
      }
    }
  };
  float ca = g.a, cb1 = g.b, cc = g.c, di[FM];
  f4 dj[FN];
  auto others = [&] {
    if (g.coef) {
      ca = g.coef[4 * t.mat];
      cb1 = g.coef[4 * t.mat + 1];
      cc = g.coef[4 * t.mat + 2];
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      dj[j] = f4{0.f, 0.f, 0.f, 0.f};
      if (ST == kPoly && cb + j * 16 < qrows)
        dj[j] = *reinterpret_cast<const f4*>(g.adiag + t.off_d + cb + j * 16 + lk * 4);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      di[i] = 0.f;
      if (ST != kGram && rb + i * 16 < prows)
        di[i] = (ST == kPoly ? g.adiag : g.bdiag)[t.off_d + rb + i * 16 + lr];
    }
#pragma unroll
    for (int i = 0; i < Ahead; ++i) own_rows(i);
  };
  if constexpr (kEarly) others();

#pragma unroll
  for (int s = 0; s < NS; ++s)
    if (s < total) {
      const From f = from(s);
#pragma unroll
      for (int x = 0; x < LP + LQ; ++x) load(f, s, x);
    }
  if (total >= NS)
    wait_and_meet<(NS - 1) * (LP + LQ)>();
  else
    wait_and_meet<0>();
#pragma unroll
  for (int j = 0; j < FN; ++j) fetch_q(0, 0, 0, j);
#pragma unroll
  for (int i = 0; i < FM; ++i) fetch_p(0, 0, 0, i);
  // Before a round's last part: the next round has landed for every wave, and
  // every wave is done reading this one, whose buffer is loaded again.  The
  // last round reads operands that nothing uses: with a tail of its own the
  // accumulators were copied around in every round.
  int buf = 0;
  // round `it`, its last part's operands in set `set`
  auto one = [&](int it, auto set, auto loads) {
    const int next = buf + 1 == NS ? 0 : buf + 1;
    constexpr int kWait = decltype(loads)::value ? (NS - 2) * (LP + LQ) : 0;
    From f{};
    if constexpr (KK == 2) {
      wait_lds();  // set 0: asked for half a round ago
      products(0, buf, 1, std::false_type{}, f, 0);
    }
    wait_and_meet<kWait>();
    if (decltype(loads)::value) f = from(it + NS);
    products(set, next, 0, loads, f, buf);
    buf = next;
  };
  int it = 0;
  if constexpr (KK == 2) {
    for (; it + NS < total; ++it) {
      one(it, 1, std::true_type{});
      if (SPLIT && (it & 1)) flush();
    }
    for (; it < total; ++it) {
      one(it, 1, std::false_type{});
      if (SPLIT && (it & 1)) flush();
    }
  } else {
    // total is even: the depth is a multiple of 64
    auto two = [&](auto first, auto second) {
      one(it, 0, first);
      one(it + 1, 1, second);
      if (SPLIT && (it & 2)) flush();
    };
    for (; it + 1 + NS < total; it += 2) two(std::true_type{}, std::true_type{});
    if (it + NS < total) {
      two(std::true_type{}, std::false_type{});
      it += 2;
    }
    for (; it < total; it += 2) two(std::false_type{}, std::false_type{});
  }
  if constexpr (SPLIT) {
    flush();
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = sum[i][j];
  }

  // ---- the results: acc[i][j][r] is row rb + 16 i + lane % 16 of P, row or
  // column cb + 16 j + 4 (lane / 16) + r of Q.  Planes are padded to
  // multiples of 64: whole 16 x 16 parts are inside or outside.
  char* rows16 = lds + wave * kOut;
  char* image = rows16 + kRows;
  constexpr int kImageLd = (TM + 8) * 2;
  const bool mirror = ST == kLast ? t.tall : t.i != t.j;
  O* out = static_cast<O*>(g.ortho) + t.flat_off;  // kLast
  const int64_t cols = t.tall ? t.m : t.n;
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
  auto to = [&](_Float16* plane, int64_t first, int64_t second, int n_cols) {
    return [=](int r, int c, u4 v) {
      if (second + c < n_cols)
        *reinterpret_cast<u4*>(plane + (first + r) * ld + second + c) = v;
    };
  };
  _Float16* dh = ST == kStep ? g.yh + t.off_x : (ST == kGram ? g.ah : g.bh) + t.off_a;
  _Float16* dl = ST == kStep ? g.yl + t.off_x : (ST == kGram ? g.al : g.bl) + t.off_a;

  if constexpr (!kEarly) others();
  __syncthreads();  // every wave is done with the operands in LDS
  if (rb >= prows || cb >= qrows) return;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    if (rb + i * 16 >= prows) break;
    const int row = rb + i * 16 + lr;
    u2 hi[FN], lo[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int col = cb + j * 16 + lk * 4;
      float x[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float sum1 = acc[i][j][r];
        const float own =
            static_cast<float>(h[i % Ahead][j][r]) + static_cast<float>(l[i % Ahead][j][r]);
        if constexpr (ST == kGram) {
          x[r] = sum1 * (kSa / (kSx * kSx));
        } else if constexpr (ST == kPoly) {
          x[r] = fmaf(fmaf(cc, di[i] + dj[j][r], cb1), own, cc * (sum1 * (1.f / kSa)));
        } else {
          x[r] = fmaf(ca + di[i], own, sum1 * (1.f / kSa));
          if (ST == kLast) x[r] *= 1.f / kSx;
        }
        if (kMirror && row == col + r) {
          if (ST == kGram)
            g.adiag[t.off_d + row] = x[r] * (1.f / kSa);
          else
            g.bdiag[t.off_d + row] = fmaf(di[i], fmaf(cc, di[i], cb1), x[r] * (1.f / kSa));
          x[r] = 0.f;
        }
      }
      if constexpr (ST == kLast && sizeof(O) == 4) {
        // in the parameter's orientation, one element at a time
        float* f = reinterpret_cast<float*>(rows16);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int y = i * 16 + lr, z = j * 16 + lk * 4 + r;
          f[t.tall ? z * (TM + 1) + y : y * (TN + 1) + z] = x[r];
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
          lo[j] = pack4(x);
        }
      }
    }
    if (i + Ahead < FM) own_rows(i + Ahead);
    if constexpr (ST == kLast && sizeof(O) == 4) continue;
    const int r0 = rb + i * 16;
    if constexpr (ST == kLast) {
      if (!t.tall)
        store_rows<FN>(rows16, hi, [&](int r, int c, u4 v) { put(r0 + r, cb + c, t.m, v); });
    } else {
      store_rows<FN>(rows16, hi, to(dh, r0, cb, qrows));
      if constexpr (ST == kStep || SPLIT) store_rows<FN>(rows16, lo, to(dl, r0, cb, qrows));
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
  if constexpr (ST == kLast && sizeof(O) == 4) {
    const float* f = reinterpret_cast<const float*>(rows16);
    const int n_rows = t.tall ? TN : TM, width = t.tall ? TM : TN;
    const int64_t r0 = t.tall ? cb : rb, c0 = t.tall ? rb : cb, last = t.tall ? t.n : t.m;
    for (int e = lane; e < n_rows * width; e += 64) {
      const int r = e / width, c = e % width;
      if (r0 + r < last && c0 + c < cols) out[(r0 + r) * cols + c0 + c] = f[r * (width + 1) + c];
    }
  } else if constexpr (ST == kLast) {
    if (mirror)
      store_image<TN, TM>(image, [&](int r, int c, u4 v) { put(cb + r, rb + c, t.n, v); });
  } else if constexpr (kMirror) {
    if (mirror) {
      // rows of the image past the plane: tiles of the lower triangle have
      // their columns inside wherever their rows are
      store_image<TN, TM>(image, to(dh, cb, rb, prows));
      if constexpr (SPLIT) {
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          u2 lo[FN];
#pragma unroll
          for (int j = 0; j < FN; ++j)
            lo[j] = u2{__float_as_uint(acc[i][j][0]), __float_as_uint(acc[i][j][1])};
          keep_transposed<FN>(image, kImageLd, i, lo);
        }
        store_image<TN, TM>(image, to(dl, cb, rb, prows));
      }
    }
  }
}

// `from`: which plane holds X.  Its low parts are replaced in place, by the
// workgroup that reads them, unless they are an operand too.
GemmArgs gemm_args(const MuonArgs& a, const MuonGemmTile* tiles, int from) {
  auto half = [&](int64_t off) { return reinterpret_cast<_Float16*>(a.ws + off); };
  GemmArgs g{};
  g.tiles = tiles;
  g.adiag = reinterpret_cast<float*>(a.ws + a.w.adiag);
  g.bdiag = reinterpret_cast<float*>(a.ws + a.w.bdiag);
  g.xh = half(a.w.xh[from]);
  g.xl = half(a.w.xl[from]);
  g.yh = half(a.w.xh[1 - from]);
  g.yl = half(a.w.xl[1 - from]);
  g.ah = half(a.w.ah);
  g.al = half(a.w.al);
  g.bh = half(a.w.bh);
  g.bl = half(a.w.bl);
  return g;
}

using Small = Shape<64, 64, 2, 2, 64, 3, 2>;
using Mid = Shape<128, 128, 2, 2, 64, 2, 2>;
using Big = Shape<256, 256, 2, 4, 64, 2, 2>;
static_assert(Small::BM == kMuonTiles[0] && Mid::BM == kMuonTiles[1] && Big::BM == kMuonTiles[2]);

template <typename S, Stage ST, bool SPLIT, typename O>
hipError_t launch_shape(GemmArgs& g, int64_t n, const Sink& sink) {
  void* p[] = {&g};
  return sink.launch(reinterpret_cast<const void*>(&k_gemm<S, ST, SPLIT, O>),
                     dim3(static_cast<unsigned>(n)), dim3(S::Threads), p, 0);
}

template <Stage ST, typename O>
hipError_t launch_gemm(bool split, const MuonTiles& t, GemmArgs& g, const Sink& sink) {
  if (t.n <= 0) return hipErrorInvalidValue;
  if constexpr (!(ST == kLast && sizeof(O) == 2)) {
    if (split)
      return t.shape == 0 ? launch_shape<Small, ST, true, O>(g, t.n, sink)
                          : launch_shape<Mid, ST, true, O>(g, t.n, sink);
  }
  if constexpr (ST == kLast && sizeof(O) == 4) {
    return hipErrorInvalidValue;  // fp32 results take split operands
  } else {
    switch (t.shape) {
      case 0: return launch_shape<Small, ST, false, O>(g, t.n, sink);
      case 1: return launch_shape<Mid, ST, false, O>(g, t.n, sink);
      default: return launch_shape<Big, ST, false, O>(g, t.n, sink);
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

hipError_t launch_muon_apply(const MuonItem* items, int64_t n, const MuonMat* mats,
                             const void* ortho, int ortho_dt, float* master, void* param,
                             int param_dt, const MuonScalars& sc, bool vec, const Sink& sink) {
  if (n <= 0) return hipErrorInvalidValue;
  ApplyArgs a{mats, ortho, master, param, sc, vec};
  const bool ob = ortho_dt == FSDP_BF16, pb = param_dt == FSDP_BF16;
  const void* fn = ob ? (pb ? reinterpret_cast<const void*>(&k_apply<u16, u16>)
                            : reinterpret_cast<const void*>(&k_apply<u16, float>))
                      : (pb ? reinterpret_cast<const void*>(&k_apply<float, u16>)
                            : reinterpret_cast<const void*>(&k_apply<float, float>));
  void* p[] = {&items, &a};
  return sink.launch(fn, dim3(static_cast<unsigned>(n)), dim3(kThreads), p, 0);
}

hipError_t launch_muon_norm(const MuonArgs& a, const MuonTile* tiles, int64_t n,
                            const void* update, int dt, const Sink& sink) {
  if (n <= 0) return hipErrorInvalidValue;
  const MuonMat* mats = a.mats;
  double* partial = reinterpret_cast<double*>(a.ws + a.w.partial);
  void* p[] = {&mats, &tiles, &update, &partial};
  const void* fn = dt == FSDP_BF16 ? reinterpret_cast<const void*>(&k_norm<u16>)
                                   : reinterpret_cast<const void*>(&k_norm<float>);
  return sink.launch(fn, dim3(static_cast<unsigned>(n)), dim3(kThreads), p, 0);
}

hipError_t launch_muon_convert(const MuonArgs& a, const MuonTile* tiles, int64_t n,
                               const void* update, int dt, double eps, const double (&poly)[3],
                               const Sink& sink) {
  if (n <= 0) return hipErrorInvalidValue;
  auto half = [&](int64_t off) { return reinterpret_cast<_Float16*>(a.ws + off); };
  ConvertArgs c{};
  c.mats = a.mats;
  c.tiles = tiles;
  c.partial = reinterpret_cast<const double*>(a.ws + a.w.partial);
  c.coef = reinterpret_cast<float*>(a.ws + a.w.coef);
  c.xh = half(a.w.xh[0]);
  c.xl = a.low ? half(a.w.xl[0]) : nullptr;
  c.eps = eps;
  c.a = poly[0];
  c.b = poly[1];
  c.c = poly[2];
  void* p[] = {&update, &c};
  const void* fn = dt == FSDP_BF16 ? reinterpret_cast<const void*>(&k_convert<u16>)
                                   : reinterpret_cast<const void*>(&k_convert<float>);
  return sink.launch(fn, dim3(static_cast<unsigned>(n)), dim3(kThreads), p, 0);
}

hipError_t launch_muon_gram(const MuonArgs& a, const MuonTiles& t, int from, const Sink& sink) {
  GemmArgs g = gemm_args(a, t.tiles, from);
  return launch_gemm<kGram, u16>(a.split, t, g, sink);
}

hipError_t launch_muon_poly(const MuonArgs& a, const MuonTiles& t, bool first,
                            const double (&poly)[3], const Sink& sink) {
  GemmArgs g = gemm_args(a, t.tiles, 0);
  g.coef = first ? reinterpret_cast<const float*>(a.ws + a.w.coef) : nullptr;
  g.b = static_cast<float>(poly[1]);
  g.c = static_cast<float>(poly[2]);
  return launch_gemm<kPoly, u16>(a.split, t, g, sink);
}

hipError_t launch_muon_step(const MuonArgs& a, const MuonTiles& t, int from, bool first,
                            bool last, const double (&poly)[3], void* ortho, int ortho_dt,
                            const Sink& sink) {
  GemmArgs g = gemm_args(a, t.tiles, from);
  g.coef = first ? reinterpret_cast<const float*>(a.ws + a.w.coef) : nullptr;
  g.a = static_cast<float>(poly[0]);
  if (first && !a.low) g.xl = nullptr;
  g.ortho = ortho;
  if (!last) return launch_gemm<kStep, u16>(a.split, t, g, sink);
  return ortho_dt == FSDP_BF16 ? launch_gemm<kLast, u16>(a.split, t, g, sink)
                               : launch_gemm<kLast, float>(a.split, t, g, sink);
}

}  // namespace fsdp
