// Internal structures of the Muon step: the chosen matrices of a unit, the
// work tables of its kernels, the workspace's layout and the launchers.
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

// One chosen matrix.  It is worked on with its shorter side first: X is
// m x n with m <= n, the matrix itself or (tall) its transpose.  Planes
// hold it with both sides padded to multiples of kMuonPad, zeros there.
struct MuonMat {
  int64_t flat_off;    // in the unit's buffers [T]
  int64_t rows, cols;  // as the parameter has them
  int64_t off_x;       // first element in a plane of X (mp rows of ldx)
  int64_t off_a;       // first element in a plane of A or B (mp rows of lda)
  int64_t off_d;       // first entry of the diagonals of A and B
  int64_t norm_chunk;  // elements per partial sum of the norm
  int32_t norm_first, norm_count;  // its partial sums
  int32_t m, n, mp, np;
  int32_t ldx, lda;
  int32_t tall;  // rows > cols
};

constexpr int kMuonPad = 64;

// Rows of the planes are an odd number of 256-byte blocks apart.  A tile's
// loads take the same 128 to 512 bytes of many rows, and addresses are
// spread over the caches' channels by 256 bytes: rows a multiple of 4 KiB
// apart (sides that are powers of two) all met on one channel.
inline int64_t muon_pitch(int64_t cols) { return (cols + 127) / 128 * 128 + (((cols + 127) / 128) % 2 ? 0 : 128); }

// The kernels' tiles hold all that a workgroup needs to know of its matrix:
// one load at its start, where a tile naming a matrix took a chain of them.

// A chunk of the update, [lo, hi) of the unit, for one partial sum.
struct MuonChunk {
  int64_t lo, hi;
  int64_t to, unused;
};

// A 64 x 64 tile of the update, row and column i and j of those.
struct alignas(64) MuonConvertTile {
  int64_t flat_off, off_x;
  int32_t rows, cols, ldx, i, j, mat;
  int32_t norm_first, norm_count;
  int32_t tall, unused[3];
};

// A product's tile.  mat < 0: none.  Bit 30 of mat: more rows than columns.
// A's tiles of up to kMuonPartTile, which write nothing to the unit, may be a
// part of the sum: n rounds from round m on, into partial sum flat_off (-1:
// the whole sum, straight into A); in `join`, n partial sums from flat_off on.
struct alignas(64) MuonGemmTile {
  int64_t off_x, off_a, flat_off;
  int32_t off_d, i, j, mat;
  int32_t mp, np, m, n;
  int32_t ldx, lda;
};
constexpr int32_t kMuonTall = 1 << 30;
constexpr int kMuonRound = 64;  // of the sum, loaded at once
constexpr int kMuonPartTile = 64;
static_assert(sizeof(MuonConvertTile) == 64 && sizeof(MuonGemmTile) == 64);

// Sides of the products' tiles.
constexpr int kMuonTiles[4] = {32, 64, 128, 256};

// One kind of product's tiles on the device.
struct MuonTiles {
  const MuonGemmTile* tiles;
  int64_t n;
  int shape;  // index into kMuonTiles
};

// Work items of the per-element kernels: `len` elements at `dst` (a
// multiple-of-1024 window of the destination space) from `src` on.
struct MuonItem {
  int64_t dst, src;
  int32_t len, mat;
};

// One step's numbers for one matrix, made with the planes of its update.  Its
// coefficients are a 2^ea, b 2^eb and c 2^ec, with a, b and c from here in the
// first step and the optimiser's in the others (from here: 1); q: the planes
// hold X 2^-q after it.
struct alignas(32) MuonCoef {
  float a, b, c;
  int32_t ea, eb, ec, q, unused;
};
constexpr int kMuonSteps = 16;  // the most; a matrix has that many MuonCoef

// A matrix's scales.
struct MuonScale {
  double aspect, rms;
};

// Device copies of the tables, one per device, in one allocation.
struct MuonDevice {
  const MuonChunk* norm;
  const MuonConvertTile* convert;
  MuonTiles gram, poly, step;  // the lower triangles of A and of B, X
  MuonTiles join;              // those of A's tiles that come in parts
  const MuonItem* momentum;   // flat space
  const MuonItem* apply;      // shard space
  const MuonScale* scales;    // per matrix
};

// Where each part of fsdp_orthogonalize's workspace begins, in bytes.
// split: every operand in two fp16 parts (FSDP_F32 results).
struct MuonWorkspace {
  int64_t partial, coef, adiag, bdiag;
  int64_t xh[2], xl[2], ah, al, bh, bl;
  int64_t sums;  // A's partial sums
  int64_t bytes;
};

// Everything the launchers of the products need.
struct MuonArgs {
  char* ws;
  MuonWorkspace w;
  bool split;
  bool low;  // the update has low parts: fp32, or split operands
  int32_t steps, step;  // how many, and the one that is launched
};

}  // namespace fsdp

struct fsdp_muon {
  int32_t R = 0;
  int64_t T = 0, S = 0;
  std::vector<fsdp::MuonMat> mats;
  std::vector<fsdp::MuonChunk> norm;
  std::vector<fsdp::MuonConvertTile> convert;
  // the products' tiles for results in bf16, and for split operands
  struct Tiles {
    std::vector<fsdp::MuonGemmTile> gram, poly, step, join;
    int gram_shape = 0, poly_shape = 0, step_shape = 0;
    int64_t n_sums = 0;  // A's partial sums, a tile of fp32 each
  } tiles[2];
  std::vector<fsdp::MuonItem> momentum, apply;
  std::vector<fsdp::MuonScale> scales;
  fsdp::WorkTable rest;  // shard space: all that is not chosen, padding too
  int64_t nx = 0, na = 0, nd = 0, n_partial = 0;  // plane, diagonal and partial-sum sizes

  // Device tables on the current device, uploaded on first use
  // (synchronous; freed with the object).
  fsdp_status device(bool split, fsdp::MuonDevice* out) const;
  ~fsdp_muon();

 private:
  mutable std::mutex mu_;
  mutable std::map<int, void*> dev_;
};

namespace fsdp {

fsdp_status build_muon(const fsdp_plan* plan, int32_t n_params, const int32_t* params,
                       fsdp_muon* mu);

MuonWorkspace muon_workspace(const fsdp_muon* mu, bool split);

// Scalars of the per-element kernels.
struct MuonScalars {
  double momentum, one_minus;  // mu, 1 - mu
  double decay, lr;            // 1 - lr wd, lr
  int32_t nesterov, scale;
};

hipError_t launch_muon_momentum(const MuonItem* items, int64_t n, const PtrArray& grads, int R,
                                int grad_dt, bool replicas, float* m, void* update, int update_dt,
                                const MuonScalars& sc, bool vec, const Sink& sink);

hipError_t launch_muon_apply(const MuonItem* items, int64_t n, const MuonScale* scales,
                             const void* ortho, int ortho_dt, float* master, void* param,
                             int param_dt, const MuonScalars& sc, bool vec, const Sink& sink);

hipError_t launch_muon_norm(const MuonArgs& a, const MuonChunk* tiles, int64_t n,
                            const void* update, int dt, const Sink& sink);
// The update into the planes of X, scaled by a power of two, the first step's
// coefficients with what is left of the norm, and all steps' exponents.
hipError_t launch_muon_convert(const MuonArgs& a, const MuonConvertTile* tiles, int64_t n,
                               const void* update, int dt, double eps, const double (&poly)[3],
                               const Sink& sink);
// A = X X^T; join: the tiles of it that t has in parts (none: no launch).
hipError_t launch_muon_gram(const MuonArgs& a, const MuonTiles& t, const MuonTiles& join, int from,
                            const Sink& sink);
// B = b A + c A A.
hipError_t launch_muon_poly(const MuonArgs& a, const MuonTiles& t, bool first,
                            const double (&poly)[3], const Sink& sink);
// X <- a X + B X, from plane `from` into the other; the last step writes
// ortho instead.
hipError_t launch_muon_step(const MuonArgs& a, const MuonTiles& t, int from, bool first,
                            bool last, const double (&poly)[3], void* ortho, int ortho_dt,
                            const Sink& sink);

}  // namespace fsdp
