// Internal structures of the unit's matrix products: what the C entry points
// hand to the launchers, and the rules both sides share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "fsdp_mi355x.h"
#include "kernels.hpp"

namespace fsdp {

// The operand types of a product.
enum ProductType { kProductF32 = FSDP_F32, kProductBf16 = FSDP_BF16, kProductI8 = 2 };

// One call, checked.  The inner sizes are n and k of fsdp_matmul; `rows` are
// the ragged ones.
struct ProductArgs {
  const void *a, *b;
  void* c;
  const float *sa, *sb;    // scales of the codes; sb null: none
  const int32_t* offsets;  // null: one group of all rows
  float* parts;            // partial sums (n_parts > 1)
  int64_t lda, ldb, ldc;   // elements
  int64_t group_stride;    // of b, or with FSDP_MATMUL_TN of c
  int64_t sb_stride;
  int32_t rows, groups, n, k;
  int32_t accumulate, out_f32;
  int32_t n_parts;
};

// The tiles: rows and columns of results that a workgroup makes.
// (kTiny: of fp32 operands only, which have kSmall and kMid besides; kThin and
// kApart: their waves share the sum).
enum ProductTile { kThin, kTiny, kApart, kSmall, kMid, kDeep, kBig };
constexpr int kProductRows[7] = {16, 32, 64, 64, 128, 128, 256};
inline int product_cols(int tile, int32_t op) {
  return tile == kThin ? (op == FSDP_MATMUL_NT ? 32 : 64) : kProductRows[tile];
}

// How a call is carried out, a function of its sizes, types and alignment.
struct ProductRule {
  int tile;      // ProductTile
  bool direct;   // operands go straight to LDS, in 16-byte pieces
  int n_parts;   // of a weight gradient's sums
  int64_t grid;  // workgroups
  int64_t join;  // workgroups that join the parts
  int64_t workspace;
};

// direct: the operands' rows begin and end at multiples of 16 bytes.
ProductRule product_rule(const fsdp_matmul& m, ProductType type, bool direct);

hipError_t launch_product(const ProductArgs& a, ProductType type, int32_t op,
                          const ProductRule& rule, const Sink& sink);

}  // namespace fsdp
