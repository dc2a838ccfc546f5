// gfx950 kernels of the unit's matrix products: the linear layers of a gathered
// unit, grouped by expert, and their gradients.
//
//   NT  C[t, n] = sum_k A[t, k] B_g[n, k]     forward, weights [out, in]
//   NN  C[t, n] = sum_k A[t, k] B_g[k, n]     input gradient
//   TN  C_g[n, k] = sum_t A[t, n] B[t, k]     weight gradient, t over g's rows
//
// with g the group of row t.  Operands are bf16, 8-bit codes with a scale per
// row (NT and NN), or fp32, and sums fp32 (codes: 32-bit integers, exact).
//
// One tile loop serves bf16 and codes: both take 16 bytes per lane and matrix
// instruction, which are 8 or 16 entries of the sum.  An operand whose rows lie
// along the sum is kept in LDS as rows of 128 bytes and read as it is; one
// whose rows lie across it as its rows are, and transposed by the LDS read (of
// 16- or 8-bit entries).  So no operand is ever written transposed.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "device.hpp"
#include "products.hpp"

namespace fsdp {
namespace {

typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef int i2 __attribute__((ext_vector_type(2)));
typedef int i4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));

struct Bf16 {
  static constexpr int kBytes = 2;
  using Acc = f4;
  __device__ __forceinline__ static Acc mma(u4 q, u4 p, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, q),
                                                   __builtin_bit_cast(b8, p), c, 0, 0, 0);
  }
};
struct I8 {
  static constexpr int kBytes = 1;
  using Acc = i4;
  __device__ __forceinline__ static Acc mma(u4 q, u4 p, Acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i4, q),
                                                 __builtin_bit_cast(i4, p), c, 0, 0, 0);
  }
};

constexpr int kRow = 128;  // bytes of the sum per round, of a row along it

// A BM x BN tile by WM x WN waves, NS rounds in LDS, registers for WPS waves
// per SIMD.
template <int BM_, int BN_, int WM_, int WN_, int NS_, int WPS_>
struct Tile {
  static constexpr int Waves = WPS_;
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr int NW = WM * WN, Threads = 64 * NW;
  static constexpr int TM = BM / WM, TN = BN / WN;  // a wave's tile
  static constexpr int FM = TM / 16, FN = TN / 16;  // its 16 x 16 parts
  static constexpr int LP = BM * kRow / 1024 / NW, LQ = BN * kRow / 1024 / NW;
  static constexpr int RoundBytes = (BM + BN) * kRow;
  // LDS of a wave that has rounds, and at the end results, of its own
  static constexpr int Pitch = BN + 4;
  static constexpr int Own =
      RoundBytes * NS > BM * Pitch * 4 ? RoundBytes * NS : BM * Pitch * 4;
};

using Small = Tile<64, 64, 2, 2, 3, 2>;
// TN: a wave's results are 64 columns wide, so 16 rows of fp32 ones are 256
// bytes each (50 and 57 us for 16 groups of 2048 x 512 that are added to).
template <int OP>
using Mid = std::conditional_t<OP == FSDP_MATMUL_TN, Tile<128, 128, 4, 2, 2, 4>,
                               Tile<128, 128, 2, 4, 2, 4>>;
template <int OP>
using Deep = std::conditional_t<OP == FSDP_MATMUL_TN, Tile<128, 128, 4, 2, 4, 2>,
                                Tile<128, 128, 2, 4, 4, 2>>;
using Big = Tile<256, 256, 2, 4, 2, 2>;
using Half = Tile<128, 256, 2, 4, 2, 2>;
using Quarter = Tile<128, 128, 2, 4, 4, 2>;
// Operands that pass through registers.
using SmallStaged = Tile<64, 64, 2, 2, 2, 2>;
using MidStaged = Tile<128, 128, 2, 4, 2, 4>;
// Tiles whose waves share the sum.
template <int OP>
using Thin = Tile<16, OP == FSDP_MATMUL_NT ? 32 : 64, 1, 1, 2, 2>;
using Apart = Tile<64, 64, 1, 1, 2, 1>;

// The place of 16-byte piece c of row r along the sum: the 16 rows that a wave
// reads at one piece spread over all banks.
__device__ __forceinline__ int place(int r, int c) { return c ^ (r & 7); }
// The same for rows across the sum, BM entries of BYTES each: a transposing
// read takes 32 bytes of rows 0-3, 8-11, 16-19 and 24-27 (or 4-7, ...) of 32 at
// a time of 16-bit entries, and 16 bytes of rows 0-7 and 16-23 (or 8-15, ...)
// of 64 of 8-bit ones.  The row's bits that tell those apart move the piece,
// but for the ones that the length of a row moves by itself (256 bytes are all
// banks once).
template <int BM, int BYTES>
__device__ __forceinline__ int place_across(int r, int c) {
  if constexpr (BYTES == 2) {
    const int b = (r & 3) | ((r >> 1) & 4);
    return c ^ (BM == 64 ? b & 6 : b << 1);
  } else {
    return c ^ (BM == 256  ? (r & 7) | ((r >> 1) & 8)
                : BM == 128 ? ((r >> 1) & 3) | ((r >> 2) & 4)
                            : ((r >> 2) & 1) | ((r >> 3) & 2));
  }
}

// 16 bytes per lane from a buffer to LDS at a wave-uniform address, lane after
// lane; zeros for offsets from kOutside on.  An asm statement for the reason
// given at load_to_lds, and waited for as those are.
constexpr uint32_t kOutside = 0x80000000u;
__device__ __forceinline__ void buffer_to_lds(u4 buffer, uint32_t offset, uint32_t to) {
  uint32_t m0;
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               : "=&{m0}"(m0)
               : "v"(offset), "s"(buffer), "s"(to)
               : "memory");
}
// A raw buffer of kOutside bytes.
__device__ __forceinline__ u4 buffer_at(const char* p) {
  const uint64_t x = reinterpret_cast<uint64_t>(p);
  return u4{static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x))),
            static_cast<uint32_t>(
                __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x >> 32) & 0xffffu)),
            kOutside, 0x00020000u};
}

// An operand of a tile: where its first entry is, and how much of it there is.
struct Operand {
  const char* p;   // entry (first row or column of the tile, first of the sum)
  int64_t ld;      // bytes from one row to the next
  int side;        // rows (along) or columns (across) from there on that exist
  int sum;         // entries of the sum
};

// This wave's pieces of an operand's round, L of 1024 bytes each.
template <typename T, int SIDE, int L, bool ACROSS>
struct Pieces {
  static constexpr int kEach = 16 / T::kBytes;     // entries of a piece
  static constexpr int kSum = kRow / T::kBytes;    // of the sum per round
  static constexpr int kPerRow = ACROSS ? SIDE / kEach : kRow / 16;
  static constexpr int kRows = 64 / kPerRow;       // rows that a wave's load fills
  static_assert(kPerRow <= 64);

  // Row and first entry (in the row) of this lane's piece x.
  __device__ __forceinline__ static int row(int wave, int x) {
    return (wave * L + x) * kRows + (static_cast<int>(threadIdx.x) & 63) / kPerRow;
  }
  __device__ __forceinline__ static int col(int wave, int x) {
    const int r = row(wave, x), c = (threadIdx.x & 63) % kPerRow;
    return (ACROSS ? place_across<SIDE, T::kBytes>(r, c) : place(r, c)) * kEach;
  }
};

// Pieces that go straight to LDS.  Rows and columns that do not exist, and the
// sum's entries behind its end, are zeros.  (Codes along the sum: a piece that
// the end cuts is read whole; its row is padded with zeros.)
template <typename T, int SIDE, int L, bool ACROSS>
struct Direct {
  using P = Pieces<T, SIDE, L, ACROSS>;
  uint32_t off[L];
  const char* p;
  int64_t step;
  int sum, wave;

  __device__ __forceinline__ void begin(const Operand& o, int wave_) {
    wave = wave_;
    p = o.p;
    sum = o.sum;
    step = ACROSS ? P::kSum * o.ld : kRow;
#pragma unroll
    for (int x = 0; x < L; ++x) {
      const int r = P::row(wave, x), c = P::col(wave, x);
      off[x] = static_cast<uint32_t>(r) * static_cast<uint32_t>(o.ld) + c * T::kBytes;
      if ((ACROSS ? c : r) >= o.side) off[x] = kOutside;
    }
  }
  __device__ __forceinline__ void load(int round, uint32_t image, int x) const {
    const int left = sum - round * P::kSum;
    const int at = ACROSS ? P::row(wave, x) : P::col(wave, x);
    buffer_to_lds(buffer_at(p + round * step), at < left ? off[x] : kOutside,
                  __builtin_amdgcn_readfirstlane(image + (wave * L + x) * 1024));
  }
};

// Pieces that pass through registers, AHEAD rounds ahead: for rows that begin
// anywhere.  Every piece is the five words around its entries, of a buffer that
// ends where the operand does, shifted by half a word where it begins at an odd
// entry, and what is behind the row's or the sum's end set to 0 when it is
// written to LDS: loads that branched at the ends were waited for one by one (38
// us of 777 x 1025 x 2049 in two groups, 24 so).
template <typename T, int SIDE, int L, bool ACROSS, int AHEAD>
struct Staged {
  static_assert(T::kBytes == 2);
  using P = Pieces<T, SIDE, L, ACROSS>;
  u4 v[AHEAD][L];
  uint32_t more[AHEAD][L];  // the fifth words
  uint32_t off[L];
  const char* p;
  int64_t step, bytes;  // to the operand's end
  int side, sum, wave;

  __device__ __forceinline__ void begin(const Operand& o, int wave_) {
    wave = wave_;
    const uint32_t half = reinterpret_cast<uintptr_t>(o.p) & 2;
    p = o.p - half;
    side = o.side;
    sum = o.sum;
    step = ACROSS ? P::kSum * o.ld : kRow;
    bytes = half + (ACROSS ? (o.sum - 1) * o.ld + int64_t(o.side) * T::kBytes
                           : (o.side - 1) * o.ld + int64_t(o.sum) * T::kBytes);
#pragma unroll
    for (int x = 0; x < L; ++x) {
      const int r = P::row(wave, x), c = P::col(wave, x);
      off[x] = half + static_cast<uint32_t>(r) * static_cast<uint32_t>(o.ld) + c * T::kBytes;
      if ((ACROSS ? c : r) >= o.side) off[x] = kOutside;
    }
  }
  __device__ __forceinline__ void fetch(int round, int set) {
    int64_t left = (bytes - round * step + 3) & ~int64_t(3);
    if (left < 0) left = 0;
    if (left > kOutside - 4) left = kOutside - 4;
    const auto buffer = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(p + round * step), 0, static_cast<int>(left), 0x00020000);
#pragma unroll
    for (int x = 0; x < L; ++x) {
      const uint32_t at = off[x] & ~3u;
      v[set][x] = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(buffer, at, 0, 0));
      more[set][x] = __builtin_amdgcn_raw_buffer_load_b32(buffer, at + 16, 0, 0);
    }
  }
  __device__ __forceinline__ void put(char* image, int round, int set) const {
    const int left = sum - round * P::kSum;
#pragma unroll
    for (int x = 0; x < L; ++x) {
      const int r = P::row(wave, x), c = P::col(wave, x);
      const int have = ACROSS ? (r < left ? side - c : 0) : left - c;
      u4 w = v[set][x];
      if (off[x] & 2)
        w = u4{w[0] >> 16 | w[1] << 16, w[1] >> 16 | w[2] << 16, w[2] >> 16 | w[3] << 16,
               w[3] >> 16 | more[set][x] << 16};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] &= have >= 2 * e + 2 ? 0xffffffffu : have == 2 * e + 1 ? 0xffffu : 0u;
      *reinterpret_cast<u4*>(image + (wave * L + x) * 1024 + (threadIdx.x & 63) * 16) = w;
    }
  }
};

// LDS to registers: the matrix instruction's operands, 16 rows (columns of an
// across operand) by 64 bytes of the sum, COUNT of them from row `from` on.
template <typename T, int SIDE, int COUNT, bool ACROSS>
struct Fetch {
  int at[ACROSS ? COUNT : 1];

  __device__ __forceinline__ explicit Fetch(int from) {
    const int lane = threadIdx.x & 63, lr = lane & 15, lk = lane >> 4;
    if constexpr (!ACROSS) {
      at[0] = (from + lr) * kRow;
    } else {
      const int row = T::kBytes == 2 ? lk * 8 + (lr >> 2) : lk * 16 + (lr >> 1);
#pragma unroll
      for (int i = 0; i < COUNT; ++i) {
        const int c = T::kBytes == 2 ? (from + i * 16) / 8 + ((lr & 3) >> 1) : (from + i * 16) / 16;
        at[i] = row * SIDE * T::kBytes + place_across<SIDE, T::kBytes>(row, c) * 16 + (lr & 1) * 8;
      }
    }
  }
  __device__ __forceinline__ u4 get(const char* image, int kk, int i) const {
    if constexpr (!ACROSS) {
      const int lane = threadIdx.x & 63;
      return *reinterpret_cast<const u4*>(image + place(lane & 15, kk * 4 + (lane >> 4)) * 16 +
                                          at[0] + i * 16 * kRow);
    } else if constexpr (T::kBytes == 2) {
      union {
        s4 s[2];
        u4 u;
      } v;
#pragma unroll
      for (int half = 0; half < 2; ++half)
        v.s[half] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s4*)(image + at[i] +
                                                    (kk * 32 + half * 4) * SIDE * 2));
      return v.u;
    } else {
      union {
        i2 s[2];
        u4 u;
      } v;
#pragma unroll
      for (int half = 0; half < 2; ++half)
        v.s[half] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) i2*)(image + at[i] + (kk * 64 + half * 8) * SIDE));
      return v.u;
    }
  }
};

// ------------------------------------------------------- which tile is whose
struct Place {
  int group;       // < 0: none
  int lo, hi;      // its rows
  int i, j;        // the tile
  int part, parts; // of it
};

__device__ __forceinline__ int clamp_to(int x, int lo, int hi) {
  return x < lo ? lo : x > hi ? hi : x;
}
// Rows of group g.  Offsets that do not ascend or leave [0, rows] give wrong
// results, but no row outside.
__device__ __forceinline__ void rows_of(const ProductArgs& a, int g, int* lo, int* hi) {
  if (!a.offsets) {
    *lo = 0;
    *hi = a.rows;
    return;
  }
  *lo = clamp_to(a.offsets[g], 0, a.rows);
  *hi = clamp_to(a.offsets[g + 1], *lo, a.rows);
}

// Tiles are numbered along bands of 8 tiles down, column by column, and each of
// the 8 dies, to which workgroups go in turn, takes a contiguous range: the 32
// tiles that a die has in flight share 8 panels of A and 4 of B in its L2.
constexpr int kBand = 8, kXcds = 8, kCus = 256;
__device__ __forceinline__ bool in_band(int id, int ni, int nj, int* i, int* j) {
  const int band = id / (kBand * nj), first = band * kBand;
  const int high = ni - first < kBand ? ni - first : kBand;
  const int in = id - first * nj;
  *i = first + in % high;
  *j = in / high;
  return *i < ni && *j < nj;
}

// Tiles of NT and NN: every group's rows in tiles of BM, which a wave counts
// with one group per lane.
//   SPLIT: the tiles behind the last that fill all compute units are cut in two
// or four, t.part being which, where the parts still find a compute unit each:
// 1,100 tiles (4.3 per compute unit) of depth 14336 take 1,660 us, and 1,795
// without; 3,860 of depth 4096 (15.1) 1,644 and 1,670.  (Tiles with at most 128
// rows left in their group as halves, whole launches over: level or 1% longer.)
template <int BM, bool SPLIT>
__device__ __forceinline__ Place ragged_tile(const ProductArgs& a, int nj) {
  const int lane = threadIdx.x & 63;
  Place t{-1, 0, 0, 0, 0, 0, 1};
  int ni = 0, lo = 0, hi = 0, incl = 0;
  auto scan = [&](int base) {  // inclusive count over 64 groups from base on
    lo = hi = 0;
    if (base + lane < a.groups) rows_of(a, base + lane, &lo, &hi);
    incl = (hi - lo + BM - 1) / BM;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int x = __shfl_up(incl, d);
      if (lane >= d) incl += x;
    }
    return __builtin_amdgcn_readlane(incl, 63);
  };
  for (int base = 0; base < a.groups; base += 64) ni += scan(base);
  const int total = ni * nj;
  int whole = total;
  if constexpr (SPLIT) {
    const int rest = total % kCus;
    if (total > kCus && rest > 0 && rest <= kCus / 2) {
      whole = total - rest;
      t.parts = rest <= kCus / 4 ? 4 : 2;
    }
  }
  const int b = blockIdx.x;
  int id;
  if (b < whole || t.parts == 1) {
    const int per = (whole + kXcds - 1) / kXcds;
    id = (b % kXcds) * per + b / kXcds;
    if (b / kXcds >= per || id >= whole) return t;
    t.parts = 1;
  } else {
    const int rest = total - whole;
    id = whole + (b - whole) % rest;
    t.part = (b - whole) / rest;
    if (t.part >= t.parts) return t;
  }
  int i, j;
  if (!in_band(id, ni, nj, &i, &j)) return t;
  for (int base = 0, before = 0; base < a.groups; base += 64) {
    const int here = a.groups > 64 ? scan(base) : ni;
    const uint64_t past = __ballot(before + incl > i);
    if (past) {
      const int l = __builtin_ctzll(past);
      t.lo = __builtin_amdgcn_readlane(lo, l);
      t.hi = __builtin_amdgcn_readlane(hi, l);
      const int tiles = (t.hi - t.lo + BM - 1) / BM;
      t.i = i - before - (__builtin_amdgcn_readlane(incl, l) - tiles);
      t.j = j;
      if (t.i >= 0 && t.i < tiles) t.group = base + l;
      return t;
    }
    before += here;
  }
  return t;
}

// Tiles of TN: ni x nj of every group, each in a.n_parts parts.  The dies share
// every group, as groups differ in length.  (The longest groups first measured
// level.)
__device__ __forceinline__ Place weight_tile(const ProductArgs& a, int ni, int nj) {
  Place t{-1, 0, 0, 0, 0, 0, 1};
  const int tiles = ni * nj, all = tiles * a.n_parts, per = (all + kXcds - 1) / kXcds;
  const int q = blockIdx.x / kXcds, g = q / per;
  if (g >= a.groups) return t;
  const int die = (blockIdx.x + static_cast<uint32_t>(g) * static_cast<uint32_t>(all)) % kXcds;
  const int id = die * per + q % per;
  if (id >= all) return t;
  t.part = id / tiles;
  if (!in_band(id % tiles, ni, nj, &t.i, &t.j)) return t;
  rows_of(a, g, &t.lo, &t.hi);
  t.group = g;
  return t;
}

// ------------------------------------------------------------------ results
// N adjacent results of a row (4 in fp32, 8 in bf16: 16 bytes), `have` of them;
// they may begin anywhere.
template <bool F32>
__device__ __forceinline__ u4 load_row(const void* c, int64_t at, int have) {
  u4 v = {0, 0, 0, 0};
  if constexpr (F32) {
    typedef u4 any __attribute__((aligned(4)));
    const uint32_t* p = static_cast<const uint32_t*>(c) + at;
    if (have >= 4) return *reinterpret_cast<const any*>(p);
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < have) v[e] = p[e];
  } else {
    typedef u4 any __attribute__((aligned(2)));
    const u16* p = static_cast<const u16*>(c) + at;
    if (have >= 8) return *reinterpret_cast<const any*>(p);
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < have) v[e / 2] |= static_cast<uint32_t>(p[e]) << (e % 2 * 16);
  }
  return v;
}
template <bool F32>
__device__ __forceinline__ void store_row(void* c, int64_t at, u4 v, int have) {
  if constexpr (F32) {
    typedef u4 any __attribute__((aligned(4)));
    uint32_t* p = static_cast<uint32_t*>(c) + at;
    if (have >= 4) {
      *reinterpret_cast<any*>(p) = v;
      return;
    }
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < have) p[e] = v[e];
  } else {
    typedef u4 any __attribute__((aligned(2)));
    u16* p = static_cast<u16*>(c) + at;
    if (have >= 8) {
      *reinterpret_cast<any*>(p) = v;
      return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < have) p[e] = static_cast<u16>(v[e / 2] >> (e % 2 * 16));
  }
}
// Their values in fp32, and back.
template <bool F32, int N>
__device__ __forceinline__ void add_row(float (&x)[N], u4 v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (F32) {
      x[e] += __uint_as_float(v[e]);
    } else {
      x[2 * e] += __uint_as_float(v[e] << 16);
      x[2 * e + 1] += __uint_as_float(v[e] & 0xffff0000u);
    }
  }
}
template <bool F32, int N>
__device__ __forceinline__ u4 pack_row(const float (&x)[N]) {
  if constexpr (F32) {
    return u4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
              __float_as_uint(x[3])};
  } else {
    typedef float f8 __attribute__((ext_vector_type(8)));
    const f8 v = {x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]};
    return __builtin_bit_cast(u4, __builtin_convertvector(v, b8));
  }
}

// A wave's results: entry e of acc[i][j] is row r0 + 16 i + lane % 16, column c0 +
// 16 j + 4 (lane / 16) + e of what begins at `to`; rows x cols of it exist.  16
// rows at a time pass through LDS (kStage floats of this wave's own), so that
// memory gets whole lines (stored as the lanes hold them, 32 bytes of 16 rows
// at a time, 256 tiles of 256 x 256 took 3 us longer; their end in a loop over
// the rows, in place of straight code, level).
template <int FN>
constexpr int kStage = 16 * (FN * 16 + 4);

template <typename T, bool F32, int FM, int FN>
__device__ __forceinline__ void finish_as(const ProductArgs& a,
                                          const typename T::Acc (&acc)[FM][FN], float* stage,
                                          int64_t to, int r0, int c0, int rows, int cols,
                                          const float* sa, const float* sb) {
  constexpr int kCols = FN * 16, kPitch = kCols + 4, kN = F32 ? 4 : 8;
  constexpr int kPerRow = kCols / kN;  // lanes of a store's rows, and how many rows
  constexpr int kAtOnce = 64 / kPerRow < 16 ? 64 / kPerRow : 16;
  const int lane = threadIdx.x & 63;
  const int r = lane / kPerRow, c = lane % kPerRow * kN;
  const int have = r < kAtOnce ? cols - (c0 + c) : 0;
  float scale[kN];
  if constexpr (T::kBytes == 1) {
#pragma unroll
    for (int e = 0; e < kN; ++e) scale[e] = sb && e < have ? sb[c0 + c + e] : 1.f;
  }
  // what the results are added to is asked for 16 rows ahead
  constexpr int kStores = 16 / kAtOnce;
  u4 old[2][kStores];
  auto ask = [&](int i) {
#pragma unroll
    for (int h = 0; h < kStores; ++h) {
      const int row = r0 + i * 16 + h * kAtOnce + r;
      if (row < rows && have > 0)
        old[i & 1][h] = load_row<F32>(a.c, to + row * a.ldc + c0 + c, have);
    }
  };
  if (a.accumulate) ask(0);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    if (a.accumulate && i + 1 < FM) ask(i + 1);
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      f4 x;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = static_cast<float>(acc[i][j][e]);
      *reinterpret_cast<f4*>(stage + (lane & 15) * kPitch + j * 16 + (lane >> 4) * 4) = x;
    }
#pragma unroll
    for (int h = 0; h < kStores; ++h) {
      const int row = r0 + i * 16 + h * kAtOnce + r;
      float x[kN];
#pragma unroll
      for (int e = 0; e < kN; e += 4) {
        const f4 v = *reinterpret_cast<const f4*>(stage + (h * kAtOnce + r % kAtOnce) * kPitch +
                                                  c + e);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[e + k] = v[k];
      }
      if (row >= rows || have <= 0) continue;
      if constexpr (T::kBytes == 1) {
        const float s = sa[row];
#pragma unroll
        for (int e = 0; e < kN; ++e) x[e] = x[e] * s * scale[e];
      }
      if (a.accumulate) add_row<F32>(x, old[i & 1][h]);
      store_row<F32>(a.c, to + row * a.ldc + c0 + c, pack_row<F32>(x), have);
    }
  }
}
template <typename T, int FM, int FN>
__device__ __forceinline__ void finish(const ProductArgs& a, const typename T::Acc (&acc)[FM][FN],
                                       float* stage, int64_t to, int r0, int c0, int rows,
                                       int cols, const float* sa, const float* sb) {
  if (a.out_f32)
    finish_as<T, true>(a, acc, stage, to, r0, c0, rows, cols, sa, sb);
  else
    finish_as<T, false>(a, acc, stage, to, r0, c0, rows, cols, sa, sb);
}

// Where a tile's operands begin, and its results: those from row i0 and column
// j0 on of t's group (of TN's gradient).
struct Site {
  Operand p, q;
  int64_t to;
};
template <typename T, int OP>
__device__ __forceinline__ Site site_of(const ProductArgs& a, const Place& t, int i0, int j0) {
  constexpr int B = T::kBytes, kSum = kRow / B;
  const char* ab = static_cast<const char*>(a.a);
  const char* bb = static_cast<const char*>(a.b);
  Site s;
  if constexpr (OP == FSDP_MATMUL_TN) {
    // this part's rows of the group, whole rounds but for the last
    const int rounds = (t.hi - t.lo + kSum - 1) / kSum;
    const int from = static_cast<int>(int64_t(rounds) * t.part / a.n_parts) * kSum;
    int end = static_cast<int>(int64_t(rounds) * (t.part + 1) / a.n_parts) * kSum;
    if (end > t.hi - t.lo) end = t.hi - t.lo;
    const int64_t row = t.lo + from;
    s.p = Operand{ab + (row * a.lda + i0) * B, a.lda * B, a.n - i0, end - from};
    s.q = Operand{bb + (row * a.ldb + j0) * B, a.ldb * B, a.k - j0, end - from};
    s.to = t.group * a.group_stride + i0 * a.ldc + j0;
  } else {
    const int64_t row = t.lo + i0;
    const char* b = bb + t.group * a.group_stride * B;
    s.p = Operand{ab + row * a.lda * B, a.lda * B, t.hi - t.lo - i0, a.k};
    s.q = Operand{b + (OP == FSDP_MATMUL_NT ? j0 * a.ldb : int64_t(j0)) * B, a.ldb * B, a.n - j0,
                  a.k};
    s.to = row * a.ldc + j0;
  }
  return s;
}

__device__ __forceinline__ uint32_t lds_address(const char* lds) {
  return static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)lds));
}

// ------------------------------------------------------------- the tile loop
// One tile, all waves on the same rounds of 128 bytes of the sum.  The products
// of one half of a round are issued row by row with the LDS reads of the next
// half and the loads of a later round between them.
//
// Measured, 256 x 256 tiles: bf16 8192 cubed 757 us (1,450 TFLOP/s; a library's
// 1,380-1,600 by order of the operands), 8192 x 14336 x 4096 700 us (1,375) in
// each of the three products; codes 387 us (2,490 TOP/s), 8192 x 4096 x 14336 337
// (2,860).  A round of 64 KB takes 1.45 us: its products alone 0.83 (2,048 cycles),
// with the LDS reads 1.15, and the rest is the loads' way from L2 (11-12 TB/s over
// all dies) and the clock under load (zeros for operands: 1,700 TFLOP/s).  Rounds
// of 64 bytes four or five deep, all LDS reads at a half's beginning, four waves
// of 128 x 128 and 32 x 32 matrix instructions measured level to 10% longer.  A
// tile's beginning and end take 10 us, which nothing hides: one workgroup has a
// compute unit's LDS.
template <typename T, typename S, int OP, bool DIRECT>
__device__ __forceinline__ void tile(const ProductArgs& a, const Place& t, int i0, int j0,
                                     char* lds) {
  constexpr int FM = S::FM, FN = S::FN, NS = S::NS, LP = S::LP, LQ = S::LQ;
  constexpr bool PA = OP == FSDP_MATMUL_TN, QA = OP != FSDP_MATMUL_NT;
  constexpr int B = T::kBytes, kSum = kRow / B;
  // (a second round in registers leaves room for one workgroup of 128 tiles)
  constexpr int kAhead = S::BM == 64 ? 2 : 1;
  using Acc = typename T::Acc;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  const Site site = site_of<T, OP>(a, t, i0, j0);
  const Operand &po = site.p, &qo = site.q;
  const int64_t to = site.to;
  const int total = (po.sum + kSum - 1) / kSum;
  if (OP == FSDP_MATMUL_TN && total == 0 && a.accumulate && a.n_parts == 1) return;

  std::conditional_t<DIRECT, Direct<T, S::BM, LP, PA>, Staged<T, S::BM, LP, PA, kAhead>> pl;
  std::conditional_t<DIRECT, Direct<T, S::BN, LQ, QA>, Staged<T, S::BN, LQ, QA, kAhead>> ql;
  pl.begin(po, wave);
  ql.begin(qo, wave);
  const Fetch<T, S::BM, FM, PA> pf(wm * S::TM);
  const Fetch<T, S::BN, FN, QA> qf(wn * S::TN);
  const uint32_t lds0 = lds_address(lds);

  Acc acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = Acc{0, 0, 0, 0};

  auto load = [&](int round, int buf, int x) {
    if constexpr (DIRECT) {
      if (x < LP)
        pl.load(round, lds0 + buf * S::RoundBytes, x < LP ? x : 0);
      else
        ql.load(round, lds0 + buf * S::RoundBytes + S::BM * kRow, x < LP ? 0 : x - LP);
    }
  };
  u4 p[2][FM], q[2][FN];
  auto products = [&](int set, int buf, int kk, auto loads, int round, int into) {
    constexpr int kFetch = FM + FN, kLoad = LP + LQ;
    const char* image = lds + buf * S::RoundBytes;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
      for (int x = i * kFetch / FM; x < (i + 1) * kFetch / FM; ++x) {
        if (x < FN)
          q[set ^ 1][x] = qf.get(image + S::BM * kRow, kk, x);
        else
          p[set ^ 1][x - FN] = pf.get(image, kk, x - FN);
      }
      if constexpr (decltype(loads)::value) {
#pragma unroll
        for (int x = i * kLoad / FM; x < (i + 1) * kLoad / FM; ++x) load(round, into, x);
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = T::mma(q[set][j], p[set][i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  if (total > 0) {
    if constexpr (DIRECT) {
#pragma unroll
      for (int s = 0; s < NS; ++s)
        if (s < total) {
#pragma unroll
          for (int x = 0; x < LP + LQ; ++x) load(s, s, x);
        }
      if (total >= NS)
        wait_and_meet<(NS - 1) * (LP + LQ)>();
      else
        wait_and_meet<0>();
    } else {
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        pl.fetch(s, s);
        ql.fetch(s, s);
      }
      pl.put(lds, 0, 0);
      ql.put(lds + S::BM * kRow, 0, 0);
      pl.fetch(kAhead, 0);
      ql.fetch(kAhead, 0);
      meet();
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) q[0][j] = qf.get(lds + S::BM * kRow, 0, j);
#pragma unroll
    for (int i = 0; i < FM; ++i) p[0][i] = pf.get(lds, 0, i);
    int buf = 0;
    if constexpr (DIRECT) {
      // Before a round's last half: the next round has landed for every wave,
      // and every wave is done reading this one, whose buffer is loaded again.
      // The last round reads operands that nothing uses.
      auto one = [&](int it, auto loads) {
        const int next = buf + 1 == NS ? 0 : buf + 1;
        wait_lds();  // set 0: asked for half a round ago
        products(0, buf, 1, std::false_type{}, 0, 0);
        wait_and_meet<decltype(loads)::value ? (NS - 2) * (LP + LQ) : 0>();
        products(1, next, 0, loads, it + NS, buf);
        buf = next;
      };
      int it = 0;
      for (; it + NS < total; ++it) one(it, std::true_type{});
      for (; it < total; ++it) one(it, std::false_type{});
    } else {
      // Two buffers: the next round's is written while this one's is read.
      // Rounds behind the last are zeros.
      for (int it = 0; it < total; it += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int set = (u + 1) % kAhead;  // round it + u + 1
          char* next = lds + (buf ^ 1) * S::RoundBytes;
          pl.put(next, it + u + 1, set);
          ql.put(next + S::BM * kRow, it + u + 1, set);
          pl.fetch(it + u + 1 + kAhead, set);
          ql.fetch(it + u + 1 + kAhead, set);
          products(0, buf, 1, std::false_type{}, 0, 0);
          meet();
          products(1, buf ^ 1, 0, std::false_type{}, 0, 0);
          buf ^= 1;
        }
      }
    }
  }

  if constexpr (OP == FSDP_MATMUL_TN) {
    // Of 64 x 64 tiles alone.  The others have the branch, never taken, for what it
    // does to the code behind it: without it the compiler puts more waits between
    // the stores there (16 experts' gradients into fp32, with their input gradients,
    // 80.6 us and 83.7).
    if (a.n_parts > 1) {
      const int ni = (a.n + S::BM - 1) / S::BM, nj = (a.k + S::BN - 1) / S::BN;
      const int64_t at = ((int64_t(t.group) * ni * nj + t.i * nj + t.j) * a.n_parts + t.part) *
                         (FM * FN * S::Threads);
      f4* part = reinterpret_cast<f4*>(a.parts) + at + threadIdx.x;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) part[(i * FN + j) * S::Threads] = acc[i][j];
      return;
    }
  }
  static_assert(S::NW * kStage<FN> * 4 <= S::RoundBytes * NS);
  __syncthreads();  // every wave is done with the operands in LDS
  float* stage = reinterpret_cast<float*>(lds) + wave * kStage<FN>;
  if constexpr (T::kBytes == 1) {
    finish<T>(a, acc, stage, to, wm * S::TM, wn * S::TN, po.side, qo.side, a.sa + t.lo + i0,
              a.sb ? a.sb + t.group * a.sb_stride + j0 : nullptr);
  } else {
    finish<T>(a, acc, stage, to, wm * S::TM, wn * S::TN, po.side, qo.side, nullptr, nullptr);
  }
}

// A workgroup's tile; of the largest, where few are left, a half or a quarter.
template <typename T, typename S, int OP, bool DIRECT>
__global__ __launch_bounds__(S::Threads, S::Waves) void k_product(ProductArgs a) {
  __shared__ __align__(1024) char lds[S::RoundBytes * S::NS];
  if constexpr (OP == FSDP_MATMUL_TN) {
    const Place t = weight_tile(a, (a.n + S::BM - 1) / S::BM, (a.k + S::BN - 1) / S::BN);
    if (t.group >= 0) tile<T, S, OP, DIRECT>(a, t, t.i * S::BM, t.j * S::BN, lds);
  } else {
    constexpr bool kSplit = S::BM == 256;
    const Place t = ragged_tile<S::BM, kSplit>(a, (a.n + S::BN - 1) / S::BN);
    if (t.group < 0) return;
    int i0 = t.i * S::BM, j0 = t.j * S::BN;
    if constexpr (kSplit) {
      static_assert(Half::Threads == S::Threads && Quarter::Threads == S::Threads);
      static_assert(Half::RoundBytes * Half::NS <= sizeof(lds) &&
                    Quarter::RoundBytes * Quarter::NS <= sizeof(lds));
      const int rows = t.hi - t.lo;
      if (t.parts == 4) {
        i0 += t.part / 2 * Quarter::BM;
        j0 += t.part % 2 * Quarter::BN;
        if (i0 < rows && j0 < a.n) tile<T, Quarter, OP, DIRECT>(a, t, i0, j0, lds);
        return;
      }
      if (t.parts == 2) {
        i0 += t.part * Half::BM;
        if (i0 < rows) tile<T, Half, OP, DIRECT>(a, t, i0, j0, lds);
        return;
      }
    }
    tile<T, S, OP, DIRECT>(a, t, i0, j0, lds);
  }
}

// A tile with the sum dealt over 4 waves: wave w takes rounds w, w + 4, ... with
// loads, LDS and accumulators of its own, so it waits for nothing but its own
// loads, until the four are added up.
//   Thin, for few rows, is bound by the weights' way from memory: one row of
// 14336 x 4096 codes 11.7 us (5.0 TB/s), in bf16 22.6 (5.2 TB/s); three or four
// rounds ahead measured level or longer, as did 32 columns where the weights lie
// across the sum (36 us and 26).
//   Apart, for no more tiles than compute units: alone on its unit, a workgroup has
// nothing else that covers a wait, and four waves that each wait alone wait less
// than four that meet every round (128 x 4096 x 14336 in bf16 64 us, 41 where the
// memory-side cache has the weights; waves that share the tile's rounds 84).  The
// joining costs 1 us, so short sums stay there.
template <typename T, typename S, int OP>
__global__ __launch_bounds__(256, S::Waves) void k_apart(ProductArgs a) {
  constexpr int FM = S::FM, FN = S::FN, BN = S::BN, NS = S::NS, LP = S::LP, LQ = S::LQ;
  constexpr bool QA = OP != FSDP_MATMUL_NT;
  constexpr int B = T::kBytes, kSum = kRow / B;
  using Acc = typename T::Acc;
  __shared__ __align__(1024) char lds[4 * S::Own];
  const Place t = ragged_tile<S::BM, false>(a, (a.n + BN - 1) / BN);
  if (t.group < 0) return;
  const int i0 = t.i * S::BM, j0 = t.j * BN, lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Site site = site_of<T, OP>(a, t, i0, j0);
  const int total = (a.k + kSum - 1) / kSum, mine = (total - wave + 3) / 4;
  char* own = lds + wave * S::Own;
  const uint32_t own0 = __builtin_amdgcn_readfirstlane(lds_address(lds) + wave * S::Own);
  Direct<T, S::BM, LP, false> pl;
  Direct<T, BN, LQ, QA> ql;
  pl.begin(site.p, 0);
  ql.begin(site.q, 0);
  const Fetch<T, S::BM, FM, false> pf(0);
  const Fetch<T, BN, FN, QA> qf(0);
  auto load = [&](int r, int buf) {  // behind the last: zeros, not read
#pragma unroll
    for (int x = 0; x < LP; ++x) pl.load(wave + 4 * r, own0 + buf * S::RoundBytes, x);
#pragma unroll
    for (int x = 0; x < LQ; ++x)
      ql.load(wave + 4 * r, own0 + buf * S::RoundBytes + S::BM * kRow, x);
  };
  Acc acc[FM][FN] = {};
#pragma unroll
  for (int s = 0; s < NS; ++s) load(s, s);
  int buf = 0;
  for (int r = 0; r < mine; ++r) {
    wait_loads<(NS - 1) * (LP + LQ)>();
    const char* image = own + buf * S::RoundBytes;
    u4 p[2][FM], q[2][FN];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
      for (int i = 0; i < FM; ++i) p[kk][i] = pf.get(image, kk, i);
#pragma unroll
      for (int j = 0; j < FN; ++j) q[kk][j] = qf.get(image + S::BM * kRow, kk, j);
    }
    wait_lds();  // the buffer is read: load it again
    asm volatile("" ::: "memory");
    load(r + NS, buf);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = T::mma(q[kk][j], p[kk][i], acc[i][j]);
    buf = buf + 1 == NS ? 0 : buf + 1;
  }
  wait_loads<0>();
  // the four waves' sums, in their order: adjacent results of a row per lane
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
      *reinterpret_cast<Acc*>(own + ((i * 16 + (lane & 15)) * S::Pitch + j * 16 +
                                     (lane >> 4) * 4) * 4) = acc[i][j];
  __syncthreads();
  constexpr int kEach = S::BM * BN / 256, kPerRow = BN / kEach;
  const int r = threadIdx.x / kPerRow, c = threadIdx.x % kPerRow * kEach;
  const int have = a.n - (j0 + c);
  if (i0 + r >= t.hi - t.lo || have <= 0) return;
  using E = std::conditional_t<B == 1, int, float>;
  E sum[kEach] = {};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const E* from = reinterpret_cast<const E*>(lds + w * S::Own) + r * S::Pitch + c;
#pragma unroll
    for (int e = 0; e < kEach; ++e) sum[e] += from[e];
  }
  const int64_t at = site.to + r * a.ldc + c;
  float x[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    x[e] = static_cast<float>(sum[e]);
    if constexpr (B == 1) {
      x[e] *= a.sa[t.lo + i0 + r];
      if (a.sb && e < have) x[e] *= a.sb[t.group * a.sb_stride + j0 + c + e];
    }
  }
  if constexpr (kEach % 8 == 0) {
    auto rows = [&](auto f32) {
      constexpr bool F32 = decltype(f32)::value;
      constexpr int kN = F32 ? 4 : 8;
#pragma unroll
      for (int e = 0; e < kEach; e += kN) {
        if (e >= have) break;
        float y[kN];
#pragma unroll
        for (int k = 0; k < kN; ++k) y[k] = x[e + k];
        if (a.accumulate) add_row<F32>(y, load_row<F32>(a.c, at + e, have - e));
        store_row<F32>(a.c, at + e, pack_row<F32>(y), have - e);
      }
    };
    if (a.out_f32)
      rows(std::true_type{});
    else
      rows(std::false_type{});
  } else {
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      if (e >= have) break;
      if (a.out_f32) {
        float* to = static_cast<float*>(a.c) + at + e;
        *to = a.accumulate ? *to + x[e] : x[e];
      } else {
        u16* to = static_cast<u16*>(a.c) + at + e;
        *to = static_cast<u16>(f32_to_bf16(a.accumulate ? bf16_to_f32(*to) + x[e] : x[e]));
      }
    }
  }
}

// A weight gradient's tiles that came in parts, added up in their order.  Parts
// are of 64 x 64 tiles: there are few results.
__global__ __launch_bounds__(Small::Threads) void k_join_parts(ProductArgs a) {
  using S = Small;
  static_assert(S::WM == SmallStaged::WM && S::WN == SmallStaged::WN);
  constexpr int FM = S::FM, FN = S::FN;
  const int ni = (a.n + S::BM - 1) / S::BM, nj = (a.k + S::BN - 1) / S::BN;
  const int g = blockIdx.x / (ni * nj), id = blockIdx.x % (ni * nj);
  const int i0 = id / nj * S::BM, j0 = id % nj * S::BN;
  const int wave = threadIdx.x >> 6;
  int lo, hi;
  rows_of(a, g, &lo, &hi);
  // nothing to add: C stays as it is (a -0 too)
  const int rows = a.accumulate && lo == hi ? 0 : a.n - i0;
  __shared__ __align__(16) float stage[S::NW * kStage<FN>];
  const f4* part = reinterpret_cast<const f4*>(a.parts) +
                   int64_t(blockIdx.x) * a.n_parts * (FM * FN * S::Threads) + threadIdx.x;
  f4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = part[(i * FN + j) * S::Threads];
  for (int p = 1; p < a.n_parts; ++p) {
    part += FM * FN * S::Threads;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] += part[(i * FN + j) * S::Threads];
  }
  finish<Bf16>(a, acc, stage + wave * kStage<FN>,
               g * a.group_stride + int64_t(i0) * a.ldc + j0, wave / S::WN * S::TM,
               wave % S::WN * S::TN, rows, a.k - j0, nullptr, nullptr);
}

// ---------------------------------------------------------------------- fp32
// fp32 operands (4096 cubed 1,150 us, 119 TFLOP/s of the matrix cores' 157; a
// library's 142): BM x BM results by four or eight waves, 32 of the sum per round, which
// pass through registers (rows may begin anywhere).  Both operands are kept in
// LDS as rows across the sum, which is how the matrix instruction reads single
// entries: entry k of row r at place r ^ 8 (k / 4) ^ 16 (k % 4) of row k, so that
// neither the reads (16 rows of 4 k) nor the writes of rows along the sum (8 rows
// of 8 times 4 k) meet on a bank.
template <int BM>
struct F32Tile {
  static constexpr int BK = 32, Threads = BM == 32 ? 256 : 512;
  static constexpr int WM = BM == 64 ? 4 : 2, WN = Threads / 64 / WM;
  static constexpr int FM = BM / WM / 16, FN = BM / WN / 16;
  static constexpr int L = BM * BK / 4 / Threads;  // four entries each, of a lane
  // Rounds in registers: 4096 cubed 1,114-1,166 us, with one 1,198-1,441; 1000 x
  // 333 x 510 in five groups 12.7, and 15.4 with one, 14.0 with three.
  static constexpr int Ahead = 2;
};
template <int BM>
__device__ __forceinline__ int place_f32(int k, int r) {
  if constexpr (BM == 32)  // two rows are all banks once
    return r ^ ((k >> 2 & 3) << 3) ^ ((k >> 1 & 1) << 4);
  else
    return r ^ ((k >> 2 & 7) << 3) ^ ((k & 3) << 4);
}

template <int BM, bool ACROSS>
struct F32Operand {
  using S = F32Tile<BM>;
  const char* p;
  int64_t step, bytes;  // to the operand's end
  int side, sum;
  uint32_t off[S::L];
  f4 v[S::Ahead][S::L];

  // row (or column) and entry of the sum of this lane's x-th four
  __device__ __forceinline__ static int row(int x) {
    return ACROSS ? static_cast<int>(threadIdx.x) % (BM / 4) * 4
                  : static_cast<int>(threadIdx.x) / 8 + S::Threads / 8 * x;
  }
  __device__ __forceinline__ static int entry(int x) {
    return ACROSS ? static_cast<int>(threadIdx.x) / (BM / 4) + S::Threads * 4 / BM * x
                  : static_cast<int>(threadIdx.x) % 8 * 4;
  }
  __device__ __forceinline__ void begin(const float* from, int64_t ld, int side_, int sum_) {
    p = reinterpret_cast<const char*>(from);
    side = side_;
    sum = sum_;
    step = ACROSS ? S::BK * ld * 4 : S::BK * 4;
    bytes = 4 * (ACROSS ? (sum - 1) * ld + side : (side - 1) * ld + sum);
#pragma unroll
    for (int x = 0; x < S::L; ++x) {
      const int r = row(x), k = entry(x);
      off[x] = 4 * (ACROSS ? static_cast<uint32_t>(k) * static_cast<uint32_t>(ld) + r
                           : static_cast<uint32_t>(r) * static_cast<uint32_t>(ld) + k);
      if (r >= side) off[x] = kOutside;
    }
  }
  __device__ __forceinline__ void fetch(int round, int set) {
    int64_t left = bytes - round * step;
    if (left < 0) left = 0;
    if (left > kOutside - 4) left = kOutside - 4;
    const auto buffer = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(p + round * step), 0, static_cast<int>(left), 0x00020000);
#pragma unroll
    for (int x = 0; x < S::L; ++x)
      v[set][x] = __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(buffer, off[x], 0, 0));
  }
  // what is behind the row's or the sum's end becomes 0
  __device__ __forceinline__ void put(float* image, int round, int set) const {
#pragma unroll
    for (int x = 0; x < S::L; ++x) {
      const int r = row(x), k = entry(x), left = sum - round * S::BK;
      const int have = ACROSS ? (k < left ? side - r : 0) : left - k;
      f4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = e < have ? v[set][x][e] : 0.f;
      if constexpr (ACROSS) {
        *reinterpret_cast<f4*>(image + k * BM + place_f32<BM>(k, r)) = w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) image[(k + e) * BM + place_f32<BM>(k + e, r)] = w[e];
      }
    }
  }
};

template <int OP, int BM>
__global__ __launch_bounds__(F32Tile<BM>::Threads) void k_product_f32(ProductArgs a) {
  using S = F32Tile<BM>;
  constexpr int BK = S::BK, FM = S::FM, FN = S::FN, kImage = BK * BM;
  __shared__ __align__(16) float lds[4 * kImage];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int qrows = OP == FSDP_MATMUL_TN ? a.k : a.n;
  const int nj = (qrows + BM - 1) / BM;
  Place t;
  if constexpr (OP == FSDP_MATMUL_TN)
    t = weight_tile(a, (a.n + BM - 1) / BM, nj);
  else
    t = ragged_tile<BM, false>(a, nj);
  if (t.group < 0) return;
  const int i0 = t.i * BM, j0 = t.j * BM;
  F32Operand<BM, OP == FSDP_MATMUL_TN> p;
  F32Operand<BM, OP != FSDP_MATMUL_NT> q;
  const float* pa = static_cast<const float*>(a.a);
  const float* qb = static_cast<const float*>(a.b);
  int64_t to;
  int side, sum;
  if constexpr (OP == FSDP_MATMUL_TN) {
    pa += t.lo * a.lda + i0;
    qb += t.lo * a.ldb + j0;
    side = a.n - i0;
    sum = t.hi - t.lo;
    to = t.group * a.group_stride + i0 * a.ldc + j0;
    if (sum == 0 && a.accumulate) return;
  } else {
    pa += (t.lo + i0) * a.lda;
    qb += t.group * a.group_stride + (OP == FSDP_MATMUL_NT ? j0 * a.ldb : int64_t(j0));
    side = t.hi - t.lo - i0;
    sum = a.k;
    to = (t.lo + i0) * a.ldc + j0;
  }
  p.begin(pa, a.lda, side, sum);
  q.begin(qb, a.ldb, qrows - j0, sum);
  const int wm = wave / S::WN * (BM / S::WM), wn = wave % S::WN * (BM / S::WN);
  // sums of 128 entries are added up apart: of 8192 entries they are off by 2.5e-7
  // of the result (rms; a library's in one go by 1.6e-6), for 3% of the time
  constexpr int kFlush = 4;
  static_assert(kFlush % S::Ahead == 0);  // the loop's steps meet it
  f4 acc[FM][FN] = {}, all[FM][FN] = {};
  auto flush = [&] {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        all[i][j] += acc[i][j];
        acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};
      }
  };
#pragma unroll
  for (int u = 0; u < S::Ahead; ++u) {
    p.fetch(u, u);
    q.fetch(u, u);
  }
  int buf = 0;
  // (rounds behind the last are zeros)
  for (int it = 0; it * BK < sum; it += S::Ahead) {
#pragma unroll
    for (int u = 0; u < S::Ahead; ++u, buf ^= 1) {
      float* ps = lds + buf * 2 * kImage;
      float* qs = ps + kImage;
      p.put(ps, it + u, u);
      q.put(qs, it + u, u);
      meet();  // and the other buffer, written next, is read
      p.fetch(it + u + S::Ahead, u);
      q.fetch(it + u + S::Ahead, u);
#pragma unroll
      for (int kk = 0; kk < BK; kk += 4) {
        const int k = kk + (lane >> 4);
        float x[FM], y[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i)
          x[i] = ps[k * BM + place_f32<BM>(k, wm + i * 16 + (lane & 15))];
#pragma unroll
        for (int j = 0; j < FN; ++j)
          y[j] = qs[k * BM + place_f32<BM>(k, wn + j * 16 + (lane & 15))];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(y[j], x[i], acc[i][j], 0, 0, 0);
      }
    }
    if (it % kFlush == kFlush - S::Ahead) flush();
  }
  flush();
  __syncthreads();
  static_assert(S::Threads / 64 * kStage<FN> <= 4 * kImage);
  finish<Bf16>(a, all, lds + wave * kStage<FN>, to, wm, wn, p.side, q.side, nullptr, nullptr);
}

// ---------------------------------------------------------------- launchers
template <typename T, typename S, int OP, bool DIRECT>
hipError_t launch_tile(const ProductArgs& args, const ProductRule& rule, const Sink& sink) {
  ProductArgs a = args;
  void* p[] = {&a};
  hipError_t e = sink.launch(reinterpret_cast<const void*>(&k_product<T, S, OP, DIRECT>),
                             dim3(static_cast<unsigned>(rule.grid)), dim3(S::Threads), p, 0);
  if constexpr (OP == FSDP_MATMUL_TN && S::BM == Small::BM) {
    if (e == hipSuccess && rule.n_parts > 1)
      e = sink.launch(reinterpret_cast<const void*>(&k_join_parts),
                      dim3(static_cast<unsigned>(rule.join)), dim3(S::Threads), p, 0);
  }
  return e;
}

template <typename T, int OP>
hipError_t launch_op(const ProductArgs& args, const ProductRule& rule, const Sink& sink) {
  if constexpr (T::kBytes == 2) {
    if (!rule.direct) {
      if (rule.tile == kSmall) return launch_tile<T, SmallStaged, OP, false>(args, rule, sink);
      return launch_tile<T, MidStaged, OP, false>(args, rule, sink);
    }
    if (rule.tile == kDeep) return launch_tile<T, Deep<OP>, OP, true>(args, rule, sink);
  }
  if constexpr (OP != FSDP_MATMUL_TN) {
    if (rule.tile == kThin || rule.tile == kApart) {
      ProductArgs a = args;
      void* p[] = {&a};
      return sink.launch(rule.tile == kThin
                             ? reinterpret_cast<const void*>(&k_apart<T, Thin<OP>, OP>)
                             : reinterpret_cast<const void*>(&k_apart<T, Apart, OP>),
                         dim3(static_cast<unsigned>(rule.grid)), dim3(256), p, 0);
    }
  }
  switch (rule.tile) {
    case kSmall: return launch_tile<T, Small, OP, true>(args, rule, sink);
    case kMid: return launch_tile<T, Mid<OP>, OP, true>(args, rule, sink);
    default: return launch_tile<T, Big, OP, true>(args, rule, sink);
  }
}

template <int OP>
hipError_t launch_f32(const ProductArgs& args, const ProductRule& rule, const Sink& sink) {
  ProductArgs a = args;
  void* p[] = {&a};
  auto launch = [&](auto kernel, int threads) {
    return sink.launch(reinterpret_cast<const void*>(kernel),
                       dim3(static_cast<unsigned>(rule.grid)), dim3(threads), p, 0);
  };
  switch (rule.tile) {
    case kTiny: return launch(&k_product_f32<OP, 32>, F32Tile<32>::Threads);
    case kSmall: return launch(&k_product_f32<OP, 64>, F32Tile<64>::Threads);
    default: return launch(&k_product_f32<OP, 128>, F32Tile<128>::Threads);
  }
}

}  // namespace

hipError_t launch_product(const ProductArgs& a, ProductType type, int32_t op,
                          const ProductRule& rule, const Sink& sink) {
  switch (type) {
    case kProductF32:
      switch (op) {
        case FSDP_MATMUL_NT: return launch_f32<FSDP_MATMUL_NT>(a, rule, sink);
        case FSDP_MATMUL_NN: return launch_f32<FSDP_MATMUL_NN>(a, rule, sink);
        default: return launch_f32<FSDP_MATMUL_TN>(a, rule, sink);
      }
    case kProductBf16:
      switch (op) {
        case FSDP_MATMUL_NT: return launch_op<Bf16, FSDP_MATMUL_NT>(a, rule, sink);
        case FSDP_MATMUL_NN: return launch_op<Bf16, FSDP_MATMUL_NN>(a, rule, sink);
        default: return launch_op<Bf16, FSDP_MATMUL_TN>(a, rule, sink);
      }
    default:
      if (op == FSDP_MATMUL_NT) return launch_op<I8, FSDP_MATMUL_NT>(a, rule, sink);
      return launch_op<I8, FSDP_MATMUL_NN>(a, rule, sink);
  }
}

}  // namespace fsdp
