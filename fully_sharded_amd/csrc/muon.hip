// gfx950 kernels of the Muon step.
//
// The per-element kernels (momentum, apply) touch every byte once and are
// bound by HBM.  The Newton-Schulz products are matrix products of the
// form D = P Q^T with both operands' rows contiguous along the sum, so one
// tile loop serves all three of a step:
//   A  = X X^T          P = Q = X  (m x n)       lower triangle, mirrored
//   B  = b A + c A A    P = Q = A  (symmetric)   lower triangle, mirrored
//   X' = a X + B X, as its transpose X'^T = a X^T + X^T B:
//                       P = X^T (n x m), Q = B (symmetric)
// The last one writes both X'^T (the next step's P and residual) and X'
// (the next A's operand), so no product ever needs a transposed read.
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
  _Float16 *xh, *xl, *th, *tl;
  double eps, a, b, c;
};

__device__ __forceinline__ void split_half(float x, _Float16& hi, _Float16& lo) {
  hi = static_cast<_Float16>(x);
  lo = static_cast<_Float16>(x - static_cast<float>(hi));
}

// 64 x 64 tiles of the update into X and its transpose.  With |U| + eps =
// N, the planes get U 2^-e with 2^e <= N < 2^(e+1): exact for bf16
// updates.  What is left, f = 2^e / N, goes into the first step's
// coefficients: A is then A f^-2 and X is X f^-1.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_convert(const T* __restrict__ update,
                                                      ConvertArgs a) {
  __shared__ float tile[64][65];
  const MuonTile t = a.tiles[blockIdx.x];
  const MuonMat& mat = a.mats[t.mat];
  double s = 0;
  for (int k = threadIdx.x; k < mat.norm_count; k += kThreads)
    s += a.partial[mat.norm_first + k];
  const double norm = sqrt(block_sum(s)) + a.eps;
  const int e = ilogb(norm);
  const double scale = ldexp(static_cast<double>(kSx), -e);
  if (t.i == 0 && t.j == 0 && threadIdx.x == 0) {
    const double f = ldexp(1.0, e) / norm;
    const bool bad = !(norm < INFINITY);
    float* c = a.coef + 4 * t.mat;
    c[0] = bad ? NAN : static_cast<float>(a.a * f);
    c[1] = bad ? NAN : static_cast<float>(a.b * f * f * f);
    c[2] = bad ? NAN : static_cast<float>(a.c * f * f * f * f * f);
  }
  const int64_t r0 = int64_t(t.i) * 64, c0 = int64_t(t.j) * 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const T* u = update + mat.flat_off;
  // the parameter's own orientation, and the other
  const int64_t ld = mat.tall ? mat.mp : mat.np, ldt = mat.tall ? mat.np : mat.mp;
  _Float16* oh = (mat.tall ? a.th : a.xh) + mat.off_x;
  _Float16* ol = mat.tall ? a.tl : a.xl;
  _Float16* ph = (mat.tall ? a.xh : a.th) + mat.off_x;
  _Float16* pl = mat.tall ? a.xl : a.tl;
  for (int k = wave; k < 64; k += kThreads / 64) {
    const int64_t r = r0 + k, c = c0 + lane;
    float x = 0.f;
    if (r < mat.rows && c < mat.cols)
      x = static_cast<float>(static_cast<double>(El<T>::load(u + r * mat.cols + c)) * scale);
    tile[k][lane] = x;
    _Float16 hi, lo;
    split_half(x, hi, lo);
    oh[r * ld + c] = hi;
    if (ol) ol[mat.off_x + r * ld + c] = lo;
  }
  __syncthreads();
  for (int k = wave; k < 64; k += kThreads / 64) {
    const int64_t c = c0 + k, r = r0 + lane;
    _Float16 hi, lo;
    split_half(tile[lane][k], hi, lo);
    ph[c * ldt + r] = hi;
    if (pl) pl[mat.off_x + c * ldt + r] = lo;
  }
}

// ---------------------------------------------------------------- products
struct GemmArgs {
  const MuonMat* mats;
  const MuonTile* tiles;
  const float* coef;  // non-null: the first step's coefficients, per matrix
  float a, b, c;      // the other steps'
  float *adiag, *bdiag;  // the diagonals of A and B
  _Float16 *xh, *xl;
  const _Float16 *th, *tl;  // X^T of this step
  _Float16 *uh, *ul;        // X^T of the next
  _Float16 *ah, *al, *bh, *bl;
  void* ortho;
};

enum Stage { kGram, kPoly, kStep, kLast };

// BM x BN tile of P Q^T, 64 of the sum per round, double-buffered in LDS:
// a round's loads go straight to LDS and are waited for a round later.
// Rows of 64 halves are 128 bytes, 8 chunks of 16; chunk c of row r sits at
// place c ^ (r & 7), so that the 16 rows a wave reads at one place of the
// sum spread over all banks.  Operand rows past the plane's last are read
// from the last one; their results are not stored.
template <int BM, int BN, int WM, int WN, Stage ST, bool SPLIT, typename O>
__global__ __launch_bounds__(64 * WM * WN) void k_gemm(GemmArgs g) {
  constexpr int NW = WM * WN;
  constexpr int TM = BM / WM, TN = BN / WN;    // a wave's tile
  constexpr int FM = TM / 16, FN = TN / 16;    // its 16 x 16 parts
  constexpr int BK = 64;
  __shared__ __align__(128) char lds[2][(BM + BN) * BK * 2];

  const MuonTile t = g.tiles[blockIdx.x];
  const MuonMat& mat = g.mats[t.mat];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;

  const int mp = mat.mp, np = mat.np;
  const _Float16 *ph, *pl = nullptr, *qh, *ql = nullptr;
  int prows, qrows, depth;
  if constexpr (ST == kGram) {
    ph = qh = g.xh + mat.off_x;
    if (SPLIT) pl = ql = g.xl + mat.off_x;
    prows = qrows = mp;
    depth = np;
  } else if constexpr (ST == kPoly) {
    ph = qh = g.ah + mat.off_a;
    if (SPLIT) pl = ql = g.al + mat.off_a;
    prows = qrows = mp;
    depth = mp;
  } else {
    ph = g.th + mat.off_x;
    qh = g.bh + mat.off_a;
    if (SPLIT) {
      pl = g.tl + mat.off_x;
      ql = g.bl + mat.off_a;
    }
    prows = np;
    qrows = mp;
    depth = mp;
  }
  const int i0 = t.i * BM, j0 = t.j * BN;

  // this lane's part of a round's loads: rows 8 apart per wave, one chunk
  constexpr int LP = BM / 8 / NW, LQ = BN / 8 / NW;
  int64_t po[LP], qo[LQ];
  {
    const int r = lane >> 3, c = (lane & 7) ^ r;
#pragma unroll
    for (int k = 0; k < LP; ++k) {
      const int row = i0 + (wave * LP + k) * 8 + r;
      po[k] = int64_t(row < prows ? row : prows - 1) * depth + c * 8;
    }
#pragma unroll
    for (int k = 0; k < LQ; ++k) {
      const int row = j0 + (wave * LQ + k) * 8 + r;
      qo[k] = int64_t(row < qrows ? row : qrows - 1) * depth + c * 8;
    }
  }
  const int rounds = depth / BK;
  const int total = SPLIT ? 3 * rounds : rounds;
  auto issue = [&](int it, int buf) {
    const _Float16 *p = ph, *q = qh;
    int k = it;
    if constexpr (SPLIT) {  // the small products first: high low, low high, high high
      const int part = it / rounds;
      k = it - part * rounds;
      if (part == 0) q = ql;
      if (part == 1) p = pl;
    }
    p += k * BK;
    q += k * BK;
    char* base = lds[buf];
#pragma unroll
    for (int x = 0; x < LP; ++x)
      __builtin_amdgcn_global_load_lds(
          reinterpret_cast<const __attribute__((address_space(1))) void*>(
              reinterpret_cast<uintptr_t>(p + po[x])),
          (__attribute__((address_space(3))) void*)(base + (wave * LP + x) * 1024), 16, 0, 0);
#pragma unroll
    for (int x = 0; x < LQ; ++x)
      __builtin_amdgcn_global_load_lds(
          reinterpret_cast<const __attribute__((address_space(1))) void*>(
              reinterpret_cast<uintptr_t>(q + qo[x])),
          (__attribute__((address_space(3))) void*)(base + BM * 128 + (wave * LQ + x) * 1024), 16,
          0, 0);
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

  const int lr = lane & 15, lk = lane >> 4;
  issue(0, 0);
  for (int it = 0; it < total; ++it) {
    // every wave's loads of this round have landed, and every wave has
    // read the last round's buffer
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (it + 1 < total) issue(it + 1, (it + 1) & 1);
    const char* base = lds[it & 1];
#pragma unroll
    for (int kk = 0; kk < BK / 32; ++kk) {
      h8 p[FM], q[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int row = wm * TM + i * 16 + lr;
        p[i] = *reinterpret_cast<const h8*>(base + row * 128 + (((kk * 4 + lk) ^ (row & 7)) * 16));
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int row = wn * TN + j * 16 + lr;
        q[j] = *reinterpret_cast<const h8*>(base + BM * 128 + row * 128 +
                                            (((kk * 4 + lk) ^ (row & 7)) * 16));
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(q[j], p[i], acc[i][j], 0, 0, 0);
    }
    if (SPLIT && (it & 1)) flush();
  }
  if constexpr (SPLIT) {
    flush();
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = sum[i][j];
  }

  // acc[i][j][r]: row i0 + wm TM + 16 i + lane % 16 of P, row
  // j0 + wn TN + 16 j + 4 (lane / 16) + r of Q
  float ca = g.a, cb = g.b, cc = g.c;
  if (g.coef) {
    ca = g.coef[4 * t.mat];
    cb = g.coef[4 * t.mat + 1];
    cc = g.coef[4 * t.mat + 2];
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int row = i0 + wm * TM + i * 16 + lr;
    if (row >= prows) continue;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int col = j0 + wn * TN + j * 16 + lk * 4;
      if (col >= qrows) continue;
      float x[4];
      const int64_t at = int64_t(row) * mp + col;  // in A, B or X^T
      if constexpr (ST == kGram) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[r] = acc[i][j][r] * (kSa / (kSx * kSx));
          if (row == col + r) {
            g.adiag[mat.off_d + row] = x[r] * (1.f / kSa);
            x[r] = 0.f;
          }
        }
      } else if constexpr (ST == kPoly) {
        const h4 hi = *reinterpret_cast<const h4*>(ph + at);
        h4 lo = {0, 0, 0, 0};
        if (SPLIT) lo = *reinterpret_cast<const h4*>(pl + at);
        const float di = g.adiag[mat.off_d + row];
        const f4 dj = *reinterpret_cast<const f4*>(g.adiag + mat.off_d + col);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float own = static_cast<float>(hi[r]) + static_cast<float>(lo[r]);
          x[r] = fmaf(fmaf(cc, di + dj[r], cb), own, cc * (acc[i][j][r] * (1.f / kSa)));
          if (row == col + r) {
            g.bdiag[mat.off_d + row] = fmaf(di, fmaf(cc, di, cb), x[r] * (1.f / kSa));
            x[r] = 0.f;
          }
        }
      } else {
        const h4 hi = *reinterpret_cast<const h4*>(ph + at);
        const h4 lo = *reinterpret_cast<const h4*>(g.tl + mat.off_x + at);
        const f4 d = *reinterpret_cast<const f4*>(g.bdiag + mat.off_d + col);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float own = static_cast<float>(hi[r]) + static_cast<float>(lo[r]);
          x[r] = fmaf(ca + d[r], own, acc[i][j][r] * (1.f / kSa));
        }
      }
      if constexpr (ST == kLast) {
        O* out = static_cast<O*>(g.ortho) + mat.flat_off;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (row < mat.n && col + r < mat.m)
            El<O>::store(out + (mat.tall ? int64_t(row) * mat.cols + col + r
                                         : int64_t(col + r) * mat.cols + row),
                         x[r] * (1.f / kSx));
      } else {
        h4 hi, lo;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          _Float16 a, b;
          split_half(x[r], a, b);
          hi[r] = a;
          lo[r] = b;
        }
        if constexpr (ST == kStep) {
          *reinterpret_cast<h4*>(g.uh + mat.off_x + at) = hi;
          *reinterpret_cast<h4*>(g.ul + mat.off_x + at) = lo;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int64_t x_at = mat.off_x + int64_t(col + r) * np + row;
            g.xh[x_at] = hi[r];
            if (SPLIT) g.xl[x_at] = lo[r];
          }
        } else {
          _Float16* dh = (ST == kGram ? g.ah : g.bh) + mat.off_a;
          _Float16* dl = (ST == kGram ? g.al : g.bl) + mat.off_a;
          *reinterpret_cast<h4*>(dh + at) = hi;
          if (SPLIT) *reinterpret_cast<h4*>(dl + at) = lo;
          if (t.i != t.j) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              dh[int64_t(col + r) * mp + row] = hi[r];
              if (SPLIT) dl[int64_t(col + r) * mp + row] = lo[r];
            }
          }
        }
      }
    }
  }
}

GemmArgs gemm_args(const MuonArgs& a) {
  auto half = [&](int64_t off) { return reinterpret_cast<_Float16*>(a.ws + off); };
  GemmArgs g{};
  g.mats = a.mats;
  g.tiles = a.tiles;
  g.adiag = reinterpret_cast<float*>(a.ws + a.w.adiag);
  g.bdiag = reinterpret_cast<float*>(a.ws + a.w.bdiag);
  g.xh = half(a.w.xh);
  g.xl = half(a.w.xl);
  g.ah = half(a.w.ah);
  g.al = half(a.w.al);
  g.bh = half(a.w.bh);
  g.bl = half(a.w.bl);
  return g;
}

template <typename A>
hipError_t launch_one(const void* fn, int64_t blocks, int threads, A& args, const Sink& sink) {
  void* p[] = {&args};
  return sink.launch(fn, dim3(static_cast<unsigned>(blocks)), dim3(threads), p, 0);
}

template <Stage ST, typename O>
hipError_t launch_gemm(const MuonArgs& a, GemmArgs& g, const Sink& sink) {
  const void* fn = a.split
                       ? reinterpret_cast<const void*>(&k_gemm<128, 128, 2, 2, ST, true, O>)
                       : reinterpret_cast<const void*>(&k_gemm<128, 128, 2, 2, ST, false, O>);
  return launch_one(fn, a.n_tiles, 256, g, sink);
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

hipError_t launch_muon_norm(const MuonArgs& a, const void* update, int dt, const Sink& sink) {
  if (a.n_tiles <= 0) return hipErrorInvalidValue;
  const MuonMat* mats = a.mats;
  const MuonTile* tiles = a.tiles;
  double* partial = reinterpret_cast<double*>(a.ws + a.w.partial);
  void* p[] = {&mats, &tiles, &update, &partial};
  const void* fn = dt == FSDP_BF16 ? reinterpret_cast<const void*>(&k_norm<u16>)
                                   : reinterpret_cast<const void*>(&k_norm<float>);
  return sink.launch(fn, dim3(static_cast<unsigned>(a.n_tiles)), dim3(kThreads), p, 0);
}

hipError_t launch_muon_convert(const MuonArgs& a, const void* update, int dt, double eps,
                               const double (&poly)[3], const Sink& sink) {
  if (a.n_tiles <= 0) return hipErrorInvalidValue;
  auto half = [&](int64_t off) { return reinterpret_cast<_Float16*>(a.ws + off); };
  ConvertArgs c{};
  c.mats = a.mats;
  c.tiles = a.tiles;
  c.partial = reinterpret_cast<const double*>(a.ws + a.w.partial);
  c.coef = reinterpret_cast<float*>(a.ws + a.w.coef);
  c.xh = half(a.w.xh);
  c.xl = a.split ? half(a.w.xl) : nullptr;
  c.th = half(a.w.th[0]);
  c.tl = half(a.w.tl[0]);
  c.eps = eps;
  c.a = poly[0];
  c.b = poly[1];
  c.c = poly[2];
  void* p[] = {&update, &c};
  const void* fn = dt == FSDP_BF16 ? reinterpret_cast<const void*>(&k_convert<u16>)
                                   : reinterpret_cast<const void*>(&k_convert<float>);
  return sink.launch(fn, dim3(static_cast<unsigned>(a.n_tiles)), dim3(kThreads), p, 0);
}

hipError_t launch_muon_gram(const MuonArgs& a, const Sink& sink) {
  if (a.n_tiles <= 0) return hipErrorInvalidValue;
  GemmArgs g = gemm_args(a);
  return launch_gemm<kGram, float>(a, g, sink);
}

hipError_t launch_muon_poly(const MuonArgs& a, bool first, const double (&poly)[3],
                            const Sink& sink) {
  if (a.n_tiles <= 0) return hipErrorInvalidValue;
  GemmArgs g = gemm_args(a);
  g.coef = first ? reinterpret_cast<const float*>(a.ws + a.w.coef) : nullptr;
  g.b = static_cast<float>(poly[1]);
  g.c = static_cast<float>(poly[2]);
  return launch_gemm<kPoly, float>(a, g, sink);
}

hipError_t launch_muon_step(const MuonArgs& a, int from, bool first, bool last,
                            const double (&poly)[3], void* ortho, int ortho_dt, const Sink& sink) {
  if (a.n_tiles <= 0) return hipErrorInvalidValue;
  auto half = [&](int64_t off) { return reinterpret_cast<_Float16*>(a.ws + off); };
  GemmArgs g = gemm_args(a);
  g.coef = first ? reinterpret_cast<const float*>(a.ws + a.w.coef) : nullptr;
  g.a = static_cast<float>(poly[0]);
  g.th = half(a.w.th[from]);
  g.tl = half(a.w.tl[from]);
  g.uh = half(a.w.th[1 - from]);
  g.ul = half(a.w.tl[1 - from]);
  g.ortho = ortho;
  if (!last) return launch_gemm<kStep, float>(a, g, sink);
  return ortho_dt == FSDP_BF16 ? launch_gemm<kLast, u16>(a, g, sink)
                               : launch_gemm<kLast, float>(a, g, sink);
}

}  // namespace fsdp
