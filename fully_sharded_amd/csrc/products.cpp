// Host side of the unit's matrix products: the C entry points' checks, the
// rule that chooses a tile, and the launches.
#include "products.hpp"

#include <algorithm>

#include "checks.hpp"
#include "ops.hpp"

namespace fsdp {
namespace {

constexpr int64_t kCus = 256;      // compute units
constexpr int64_t kXcds = 8;
constexpr int64_t kMaxSum = 131072;  // of codes: 127 * 127 * this fits 31 bits (128 * 128
                                     // * this does not: such codes are for shorter sums)
constexpr int64_t kMaxGroups = 65536;
constexpr int64_t kMaxRows = int64_t(1) << 30, kMaxSide = int64_t(1) << 26;
// Bytes from one row of an operand to the next: 256 rows within 2^31.  (Of one
// row, nothing is reached by it.)
constexpr int64_t kMaxPitch = (int64_t(1) << 23) - 1;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// The tile: the largest that gives every compute unit one (the weight gradients
// of several groups, which differ in length: two).  Measured, us a call:
//   kBig and kMid: one weight's gradient 4096 x 4096, sum 2048 (256 tiles of 256)
//     59 and 74; 16 groups' of 2048 x 512 (256, groups of 0 to 1,400 rows) 67, 56
//   kDeep, kMid and kSmall (bf16, up to one tile of 128 per compute unit: a workgroup
//   has all of its LDS, and four rounds in it):
//     n = 2048, sum 2048: 128 tiles of 128 17, 24 and 15, 144 to 192 17, 24 and 20,
//     208 to 240 18, 25 and 26, 256 19, 25 and 26, 272 33, 26 and 30; sum 4096: 128
//     28, 42 and 26, 144 28, 43 and 35, 256 33, 44 and 49; sum 512: 128 7.6, 8.0 and
//     6.4, 144 8.0, 9.1 and 8.0, 256 8.6, 9.7 and 11.1; the other two products within
//     a tenth of these.  200 tiles that hold 400 of 64 (25600 x 64), which all run at
//     once: along the sum 2048 30, 37 and 29, 4096 47, 65 and 49; across it 1024
//     12.3, 14.3 and 12.9, 2048 25, 32 and 32.
//     Several groups, kDeep and kSmall: 12 of 80 rows each (208 tiles), sum 512 9.2
//     and 9.0, 768 11.9 and 12.5; 6 of 100 (224), sum 512 9.9 and 9.0; four of 400
//     (224), sum 512 8.7 and 11.3, 256 6.7 and 8.5, of 250 (144) 6.3 and 6.1; 128 of
//     136 (200, every second one nearly empty), sum 824 16.0 and 13.8.  Where they
//     fill little of a tile: 80 of 64 rows x 192, sum 4096 43 and 36; 12 of 16 rows x
//     2048, sum 2048 25.4 and 25.3; weights across the sum, 64 of 12 rows x 408 (256),
//     sum 2256 27 and 33, 128 of 31 x 168 (256), sum 3208 38 and 46, 80 of 64 x 192
//     (160), sum 4096 42 and 36.
//     Weight gradients of several: four of 512 rows, unlike in length, 160 tiles
//     10.6 and 9.5, 224 11.9 and 12.9; eight of 312 x 128 x 3288 (208) 11.2 and 9.9;
//     fifteen of 512 x 512 (240), 1,024 rows each 18 and 26; sixty of 256 x 256 (240)
//     26 and 31, 256 rows 13.3 and 11.5; 200 of 128 x 128, 1,024 rows 56 and 40 (a
//     group's tiles are dealt to eight dies); 150 of 64 x 64, 2,048 rows 49 and, in
//     parts, 20.  Where kDeep does not pay at 256 tiles, kMid and kSmall: 32 of 960 x
//     120, 19 rows 5.5 and 7.5; forward, 128 of 2 rows x 176, sum 3752 70 and 47.
//   Codes: kDeep and kMid level.
//   kMid and kSmall: 288 tiles (8192 x 512 x 2048 in 16 groups) 30 and 34, 8 groups
//     of 1024 x 1024 over 4,096 rows 17.1 and 18.6
//   kThin and kSmall, codes and weights read along the sum: 16 x 4096 x 14336 11.7
//     and 28.2, 32 x 4096 x 4096 6.2 and 10.9, 64 x 4096 x 4096 8.2 and 11.1; 64 x
//     14336 x 4096, where 64 tiles are 224 and thin ones read the weights four
//     times, 21.0 and 12.6; 32 x 14336 x 4096 (448 thin tiles) 13.3 and 11.8, in
//     bf16 across the sum 40 and 30; eight groups of 2048 x 512 with two rows each
//     (256 tiles) 5.0 and 4.8
//   kApart and kSmall, 64-row tiles that are full for the most: 512 x 2048 x 2048
//     in bf16 10.3 and 11.1, 128 x 4096 x 14336 64 and 84, codes 23 and 30; 400 x
//     1024 x 4096 in four groups 16.3 and 18.7, codes across the sum 15.5 and 14.1;
//     sums under 4 KiB: 512 cubed in bf16 5.8 and 4.8; eight groups of 12 rows,
//     which wait for the weights, 14.3 and 12.9
//   fp32, kSmall and kTiny: 512 x 512 x 2048 61 and 27, 1024 cubed (256) 33 and 32
// A weight gradient's sums in parts, where there are fewer tiles than compute
// units: 2,001 rows of 1001 x 1003 in 28 us.
ProductRule product_rule(const fsdp_matmul& m, ProductType type, bool direct) {
  ProductRule r{};
  const bool weight = m.op == FSDP_MATMUL_TN;
  const int64_t met = std::max<int64_t>(1, std::min<int64_t>(m.groups, m.rows));
  // tiles about as many as there will be: every group's last row of tiles is
  // half empty
  auto tiles = [&](ProductTile t) {
    const int64_t down = kProductRows[t], across = product_cols(t, m.op);
    if (weight) return m.groups * ceil_div(m.n, down) * ceil_div(m.k, across);
    return (met == 1 ? ceil_div(m.rows, down) : std::max(met, m.rows / down + (met + 1) / 2)) *
           ceil_div(m.n, across);
  };
  // of up to one tile of 128 per compute unit
  auto deep = [&] {
    const int64_t t = tiles(kMid), small = tiles(kSmall), sum = weight ? m.rows / met : m.k;
    if (t <= kCus / 2) return false;
    // 64 x 64 tiles that do not all run at once, and fill the larger ones for the most
    const bool full = small > 2 * kCus && 5 * t <= 2 * small;
    const bool most = t > 3 * kCus / 4;
    if (weight ? m.groups == 1 : met == 1)
      return full ? most || sum >= 192 : sum >= (m.op == FSDP_MATMUL_NT ? 4096 : 2048);
    if (!full)
      return m.op == FSDP_MATMUL_NN && most && sum >= 2048 && 4 * t <= 3 * small;
    if (weight) return most && sum >= 512 && t >= m.groups * (sum >= 1024 ? 4 : 8);
    if (m.rows < 128 * met) return sum >= 768;
    // (groups a little longer than a tile fill two by half, and groups' lengths may
    // give a row of tiles more)
    return m.rows >= 192 * met && t + ceil_div(m.n, 128) <= kCus &&
           (sum >= 768 || (most && sum >= 384));
  };
  r.direct = direct && type != kProductF32;
  r.tile = kSmall;
  if (type == kProductF32) {
    r.tile = tiles(kMid) >= kCus ? kMid : tiles(kSmall) >= 2 * kCus ? kSmall : kTiny;
  } else if (r.direct && !weight && tiles(kSmall) < kCus &&
             tiles(kSmall) * ceil_div(m.rows, 16 * met) <= kCus) {
    r.tile = kThin;
  } else if (r.direct && !weight && tiles(kSmall) <= kCus && m.rows > 64 * met &&
             m.k * (type == kProductI8 ? 1 : 2) >= 4096) {
    r.tile = kApart;
  } else if (r.direct && tiles(kBig) >= (weight && m.groups > 1 ? 2 * kCus : kCus)) {
    r.tile = kBig;
  } else if (r.direct && type == kProductBf16 && tiles(kMid) <= kCus && deep()) {
    r.tile = kDeep;
  } else if (tiles(kMid) > kCus ||
             (tiles(kMid) == kCus && (weight || !r.direct || type != kProductBf16))) {
    r.tile = kMid;
  }
  const int64_t down = kProductRows[r.tile], across = product_cols(r.tile, m.op);
  r.n_parts = 1;
  if (weight) {
    const int64_t per_group = ceil_div(m.n, down) * ceil_div(m.k, across);
    const int64_t all = per_group * m.groups;
    // long sums of few tiles in parts, eight rounds of 64 rows or more each
    if (type == kProductBf16 && r.tile == kSmall && all < kCus)
      r.n_parts = static_cast<int>(std::max<int64_t>(
          1, std::min<int64_t>({2 * kCus / all, m.rows / met / 512, 64})));
    r.grid = kXcds * ceil_div(per_group * r.n_parts, kXcds) * m.groups;
    r.join = all;
    if (r.n_parts > 1) r.workspace = all * r.n_parts * down * across * 4;
  } else {
    const int64_t most = m.groups == 1 ? ceil_div(m.rows, down) : m.rows / down + met;
    r.grid = kXcds * ceil_div(most * ceil_div(m.n, across), kXcds);
    // up to half as many tiles as compute units may be cut, in four at most
    if (r.tile == kBig) r.grid += 3 * kCus / 4;
  }
  return r;
}

namespace {

struct Extents {
  int64_t a, b, c;  // elements from the first to behind the last
};

// (-1: no length that an array can have)
Extents extents(const fsdp_matmul& m) {
  const bool nt = m.op == FSDP_MATMUL_NT;
  // a group's matrix, then all groups' ones
  auto stack = [&](int64_t rows, int64_t ld, int64_t cols) {
    const int64_t one = reach(rows, ld, cols);
    return one < 0 ? one : reach(m.groups, m.group_stride, one);
  };
  if (m.op == FSDP_MATMUL_TN)
    return Extents{reach(m.rows, m.lda, m.n), reach(m.rows, m.ldb, m.k),
                   stack(m.n, m.ldc, m.k)};
  return Extents{reach(m.rows, m.lda, m.k), stack(nt ? m.n : m.k, m.ldb, nt ? m.k : m.n),
                 reach(m.rows, m.ldc, m.n)};
}

// Sizes and strides, without the pointers.
fsdp_status check_sizes(const fsdp_matmul* m, bool codes) {
  if (!m) return FSDP_ERR_INVALID_ARG;
  if (m->op < FSDP_MATMUL_NT || m->op > FSDP_MATMUL_TN || (codes && m->op == FSDP_MATMUL_TN) ||
      m->groups < 1 || m->rows < 0 || m->n < 1 || m->k < 1 ||
      (m->accumulate != 0 && m->accumulate != 1))
    return FSDP_ERR_INVALID_ARG;
  if (m->groups > kMaxGroups || m->rows >= kMaxRows || m->n >= kMaxSide || m->k >= kMaxSide)
    return FSDP_ERR_UNSUPPORTED;
  const int64_t a_cols = m->op == FSDP_MATMUL_TN ? m->n : m->k;
  const int64_t b_cols = m->op == FSDP_MATMUL_NN ? m->n : m->k;
  const int64_t c_cols = m->op == FSDP_MATMUL_TN ? m->k : m->n;
  if (m->lda < a_cols || m->ldb < b_cols || m->ldc < c_cols || m->group_stride < 0)
    return FSDP_ERR_INVALID_ARG;
  const Extents e = extents(*m);
  if (e.a < 0 || e.b < 0 || e.c < 0) return FSDP_ERR_UNSUPPORTED;
  // a group's gradient must not meet the next one's
  if (m->op == FSDP_MATMUL_TN && m->groups > 1 &&
      m->group_stride < (m->n - 1) * m->ldc + m->k)
    return FSDP_ERR_INVALID_ARG;
  if (codes && m->k > kMaxSum) return FSDP_ERR_UNSUPPORTED;
  return FSDP_OK;
}

// The product with the pitches of operands of one row, which nothing is apart
// by, set to the row's length.
fsdp_matmul with_pitches(const fsdp_matmul& given) {
  fsdp_matmul m = given;
  const bool tn = m.op == FSDP_MATMUL_TN, nt = m.op == FSDP_MATMUL_NT;
  if (m.rows <= 1) m.lda = tn ? m.n : m.k;
  if ((tn ? m.rows : nt ? m.n : m.k) <= 1) m.ldb = nt || tn ? m.k : m.n;
  return m;
}
// Whether rows of either operand, of es bytes per entry, lie too far apart.
bool too_far(const fsdp_matmul& m, int64_t es) {
  const int64_t b_rows =
      m.op == FSDP_MATMUL_TN ? m.rows : m.op == FSDP_MATMUL_NT ? m.n : m.k;
  return (m.rows > 1 && m.lda > kMaxPitch / es) || (b_rows > 1 && m.ldb > kMaxPitch / es);
}

// Whether bf16 operands can go straight to LDS: every 16-byte piece of a row
// is aligned and inside the row.
bool pieces(const fsdp_matmul& m, const void* a, const void* b) {
  const int64_t a_cols = m.op == FSDP_MATMUL_TN ? m.n : m.k;
  const int64_t b_cols = m.op == FSDP_MATMUL_NN ? m.n : m.k;
  return aligned(a, 16) && aligned(b, 16) && a_cols % 8 == 0 && b_cols % 8 == 0 &&
         m.lda % 8 == 0 && m.ldb % 8 == 0 &&
         (m.op == FSDP_MATMUL_TN || m.groups == 1 || m.group_stride % 8 == 0);
}

ProductArgs product_args(const fsdp_matmul& m, const int32_t* offsets, const void* a,
                         const void* b, void* c, int32_t out_dtype) {
  ProductArgs p{};
  p.a = a;
  p.b = b;
  p.c = c;
  p.offsets = offsets;
  p.lda = m.lda;
  p.ldb = m.ldb;
  p.ldc = m.ldc;
  p.group_stride = m.group_stride;
  p.rows = static_cast<int32_t>(m.rows);
  p.groups = m.groups;
  p.n = static_cast<int32_t>(m.n);
  p.k = static_cast<int32_t>(m.k);
  p.accumulate = m.accumulate;
  p.out_f32 = out_dtype == FSDP_F32;
  p.n_parts = 1;
  return p;
}

bool fits(const ProductRule& r) {
  // workgroups of up to 512 lanes
  return r.grid <= kMaxItems / 2 && r.join <= kMaxItems / 2;
}

}  // namespace
}  // namespace fsdp

using namespace fsdp;

extern "C" {

fsdp_status fsdp_grouped_matmul_workspace(const fsdp_matmul* m, int32_t dtype, int64_t* bytes) {
  if (!bytes || !valid_dtype(dtype)) return FSDP_ERR_INVALID_ARG;
  const fsdp_status st = check_sizes(m, false);
  if (st != FSDP_OK) return st;
  // whichever way the operands turn out to be aligned
  const ProductType type = static_cast<ProductType>(dtype);
  *bytes = std::max(product_rule(*m, type, true).workspace,
                    product_rule(*m, type, false).workspace);
  return FSDP_OK;
}

fsdp_status fsdp_grouped_matmul(const fsdp_matmul* given, const int32_t* offsets, const void* a,
                                const void* b, int32_t dtype, void* c, int32_t out_dtype,
                                void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> fsdp_status {
    if (!valid_dtype(dtype) || !valid_dtype(out_dtype)) return FSDP_ERR_INVALID_ARG;
    fsdp_status st = check_sizes(given, false);
    if (st != FSDP_OK) return st;
    const fsdp_matmul one = with_pitches(*given), *m = &one;
    if (!offsets && m->groups != 1) return FSDP_ERR_INVALID_ARG;
    const bool reads_b = m->op != FSDP_MATMUL_TN || m->rows > 0;
    // (an array of nothing may be at NULL)
    if ((m->rows > 0 && !a) || (reads_b && !b) || ((m->op == FSDP_MATMUL_TN || m->rows > 0) && !c))
      return FSDP_ERR_INVALID_ARG;
    const int64_t es = dtype_size(dtype), ces = dtype_size(out_dtype);
    if (!aligned(a, es) || !aligned(b, es) || !aligned(c, ces) || !aligned(offsets, 4))
      return FSDP_ERR_INVALID_ARG;
    const ProductType type = static_cast<ProductType>(dtype);
    if (too_far(*m, es)) return FSDP_ERR_UNSUPPORTED;
    const ProductRule rule = product_rule(*m, type, pieces(*m, a, b));
    if (!fits(rule)) return FSDP_ERR_UNSUPPORTED;
    const Extents e = extents(*m);
    Ranges reads, writes;
    reads.push_back(range_of(a, e.a * es));
    reads.push_back(range_of(b, reads_b ? e.b * es : 0));
    reads.push_back(range_of(offsets, offsets ? (int64_t(m->groups) + 1) * 4 : 0));
    writes.push_back(range_of(c, e.c * ces));
    if (rule.workspace) {
      if (!workspace || workspace_bytes < rule.workspace || !aligned(workspace, 256))
        return FSDP_ERR_INVALID_ARG;
      writes.push_back(range_of(workspace, rule.workspace));
    }
    for (const Range& w : writes)
      for (const Range& r : reads)
        if (overlap(w, r)) return FSDP_ERR_INVALID_ARG;
    if (any_overlap(writes)) return FSDP_ERR_INVALID_ARG;
    if (m->op != FSDP_MATMUL_TN && m->rows == 0) return FSDP_OK;
    ProductArgs p = product_args(*m, offsets, a, b, c, out_dtype);
    p.parts = static_cast<float*>(workspace);
    p.n_parts = rule.n_parts;
    return status_of(launch_product(p, type, m->op, rule, StreamSink(stream)));
  });
}

fsdp_status fsdp_grouped_matmul_i8(const fsdp_matmul* given, const int32_t* offsets,
                                   const int8_t* a, const float* a_scale, const int8_t* b,
                                   const float* b_scale, int64_t b_scale_stride, void* c,
                                   int32_t out_dtype, void* stream) {
  return guarded([&]() -> fsdp_status {
    if (!valid_dtype(out_dtype) || !b) return FSDP_ERR_INVALID_ARG;
    fsdp_status st = check_sizes(given, true);
    if (st != FSDP_OK) return st;
    if (given->lda % 16 || given->ldb % 16) return FSDP_ERR_INVALID_ARG;
    const fsdp_matmul one = with_pitches(*given), *m = &one;
    if (!offsets && m->groups != 1) return FSDP_ERR_INVALID_ARG;
    if (m->rows > 0 && (!a || !a_scale || !c)) return FSDP_ERR_INVALID_ARG;
    const int64_t ces = dtype_size(out_dtype);
    if (!aligned(a, 16) || !aligned(b, 16) || (m->groups > 1 && m->group_stride % 16) ||
        !aligned(a_scale, 4) || !aligned(b_scale, 4) || !aligned(c, ces) || !aligned(offsets, 4) ||
        b_scale_stride < 0)
      return FSDP_ERR_INVALID_ARG;
    const int64_t scales = b_scale ? reach(m->groups, b_scale_stride, m->n) : 0;
    if (too_far(*m, 1) || scales < 0) return FSDP_ERR_UNSUPPORTED;
    const ProductRule rule = product_rule(*m, kProductI8, true);
    if (!fits(rule)) return FSDP_ERR_UNSUPPORTED;
    Extents e = extents(*m);
    // rows of codes are read to the next multiple of 16
    e.a = (e.a + 15) / 16 * 16;
    e.b = (e.b + 15) / 16 * 16;
    const Range w = range_of(c, e.c * ces);
    const Range reads[] = {
        range_of(a, e.a), range_of(b, e.b), range_of(a_scale, m->rows * 4),
        range_of(b_scale, scales * 4),
        range_of(offsets, offsets ? (int64_t(m->groups) + 1) * 4 : 0)};
    for (const Range& r : reads)
      if (overlap(w, r)) return FSDP_ERR_INVALID_ARG;
    if (m->rows == 0) return FSDP_OK;
    ProductArgs p = product_args(*m, offsets, a, b, c, out_dtype);
    p.sa = a_scale;
    p.sb = b_scale;
    p.sb_stride = b_scale_stride;
    return status_of(launch_product(p, kProductI8, m->op, rule, StreamSink(stream)));
  });
}

}  // extern "C"
