// Host side of the Muon step: the choice of matrices, its work tables, and
// the C entry points' checks and launches.
#include "muon.hpp"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "checks.hpp"
#include "ops.hpp"

namespace fsdp {
namespace {

constexpr int64_t kItem = 1024;           // elements per work item of the per-element kernels
constexpr int64_t kMaxSide = int64_t(1) << 30;
constexpr int64_t kNormChunk = 4096;      // least elements per partial sum
constexpr int64_t kNormParts = 1024;      // most partial sums per matrix
constexpr int64_t kCus = 256;             // compute units
constexpr int kConvert = 64;              // side of a conversion's tile
constexpr int kXcds = 8;

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Cut [dst, dst + len) <- src at multiples of kItem in the destination.
void emit(int64_t dst, int64_t src, int64_t len, int32_t mat, std::vector<MuonItem>& out) {
  while (len > 0) {
    const int64_t n = std::min(len, (dst / kItem + 1) * kItem - dst);
    out.push_back(MuonItem{dst, src, static_cast<int32_t>(n), mat});
    dst += n;
    src += n;
    len -= n;
  }
}

// Workgroups go to the 8 accelerator dies in turn, each with its own L2.  A
// matrix that is a small part of the work goes to one die as a whole, the one
// with the least so far: its operands are then read into one L2 (72 matrices
// of hidden 512, their tiles spread over all dies, read 265 MB for A where X
// has 75, at the fabric's 6 TB/s).  Larger ones are cut in 8 contiguous parts
// (of an order that keeps neighbours together).  Queues are filled up with
// empty tiles, so that every die gets its own.
class Deal {
 public:
  explicit Deal(int64_t all) : all_(all) {}
  void add(const std::vector<MuonGemmTile>& tiles, int64_t depth) {
    const int64_t n = static_cast<int64_t>(tiles.size());
    int order[kXcds];
    for (int k = 0; k < kXcds; ++k) order[k] = k;
    std::stable_sort(order, order + kXcds, [&](int a, int b) { return load_[a] < load_[b]; });
    const int parts = n * depth * kXcds * 3 <= all_ ? 1 : kXcds;
    int64_t at = 0;
    for (int k = 0; k < parts; ++k) {
      const int64_t take = n / parts + (k < n % parts ? 1 : 0);
      auto& q = queue_[order[k]];
      q.insert(q.end(), tiles.begin() + at, tiles.begin() + at + take);
      load_[order[k]] += take * depth;
      at += take;
    }
  }
  std::vector<MuonGemmTile> dealt() const {
    std::vector<MuonGemmTile> out;
    MuonGemmTile none{};
    none.mat = -1;
    size_t longest = 0;
    for (const auto& q : queue_) longest = std::max(longest, q.size());
    for (size_t r = 0; r < longest; ++r)
      for (int x = 0; x < kXcds; ++x) out.push_back(r < queue_[x].size() ? queue_[x][r] : none);
    while (out.back().mat < 0) out.pop_back();
    return out;
  }

 private:
  std::vector<MuonGemmTile> queue_[kXcds];
  int64_t load_[kXcds] = {};  // tiles times depth
  int64_t all_;
};

// Tiles of a grid of ni x nj, in bands of 8 rows, column by column: any 32
// consecutive ones (a die's compute units) share 8 row panels and 4 column
// panels.  lower: those of the lower triangle.
std::vector<MuonGemmTile> grid(const MuonMat& t, int32_t mat, int64_t ni, int64_t nj,
                               bool lower) {
  std::vector<MuonGemmTile> out;
  for (int64_t b = 0; b < ni; b += 8)
    for (int64_t j = 0; j < nj; ++j)
      for (int64_t i = b; i < std::min(ni, b + 8); ++i)
        if (!lower || i >= j)
          out.push_back(MuonGemmTile{t.off_x, t.off_a, t.flat_off, static_cast<int32_t>(t.off_d),
                                     static_cast<int32_t>(i), static_cast<int32_t>(j),
                                     mat | (t.tall ? kMuonTall : 0), t.mp,
                                     t.np, t.m, t.n, t.ldx, t.lda});
  return out;
}

int64_t count(const std::vector<MuonMat>& mats, int64_t tile, bool square) {
  int64_t n = 0;
  for (const MuonMat& t : mats) {
    const int64_t si = (t.mp + tile - 1) / tile, sj = (t.np + tile - 1) / tile;
    n += square ? si * (si + 1) / 2 : si * sj;
  }
  return n;
}

// The tile of one kind of product (index into kMuonTiles): the largest that
// still gives every compute unit two.  256 x 256 tiles also need deep sums to
// pay for their long ends: the step of 72 matrices of hidden 512 (576 such
// tiles, depth 512) took 93 us with them and 83 with 128 x 128, a pass over
// the hidden-4096 block (depth 4096) 13.6 ms and 15.7.  The 32 x 32 tiles,
// whose four waves share a sum, are for launches that would leave compute
// units without a tile: one 512 x 512 matrix (36 and 64 tiles of 64 x 64)
// takes 62 us a pass with them and 90 without; of one block of hidden 512,
// A (216 tiles, depth up to 2048) gains 6 us a pass, B (216) loses 5 and the
// step (768) 45.  (build_muon takes 64 x 64 tiles for A all the same where
// their sums, in parts, fill the compute units.)
int shape_of(const std::vector<MuonMat>& mats, bool square, bool gram, bool split) {
  int64_t tiles = 0, rounds = 0;
  for (const MuonMat& t : mats) {
    const int64_t n = count({t}, 256, square);
    tiles += n;
    rounds += n * (gram ? t.np : t.mp);
  }
  if (!split && tiles >= 2 * kCus && rounds >= tiles * 1024) return 3;
  if (count(mats, 128, square) >= 2 * kCus) return 2;
  return count(mats, 64, square) <= (gram ? kCus : kCus / 2) ? 0 : 1;
}

// A's smaller tiles, where a few of them have long sums: these are cut into
// parts, each a workgroup's, and joined by a second launch.  Parts are as
// long as gives every compute unit two, kPart rounds at least, and are made
// only where the longest sum gets kJoin rounds and a fifth shorter, so that
// the second launch and the partial sums' way through memory pay.  Of one 32 x n matrix,
// five steps, whole sums and parts: n = 4,096 77 us and 88 (so they stay
// whole), 6,144 90 and 90, 16,384 152 and 91, 1M 7,020 and 860; fp32 results,
// with three products 124 and 95 at 4,096; 1440 x 16384 (276 tiles of 64 x 64)
// 1,013 and 935, 1800 x 32000 (435) 2,290 and 2,360.  Parts of 16 rounds
// measured 5-10% longer, four per compute unit level.
constexpr int64_t kPart = 32, kJoin = 64;

int64_t rounds_of(const std::vector<MuonMat>& mats, int64_t side, int products) {
  int64_t work = 0;
  for (const MuonMat& t : mats)
    work += count({t}, side, true) * products * (t.np / kMuonRound);
  return work;
}

int64_t part_rounds(const std::vector<MuonMat>& mats, int64_t side, int products) {
  const int64_t work = rounds_of(mats, side, products);
  int64_t longest = 0;
  for (const MuonMat& t : mats)
    longest = std::max(longest, int64_t(products) * t.np / kMuonRound);
  const int64_t len = std::max(kPart, (work + 2 * kCus - 1) / (2 * kCus));
  return longest >= len + std::max(kJoin, len / 4) ? len : longest;
}

// Whether A in 64 x 64 tiles gains more by reading half as much than it loses
// by joining: one workgroup adds up a tile's parts, 0.4 us each.  To 32 parts
// it does; beyond, where the reading saved is 12 MB a part or more.  Measured
// by MB a part, us a step against 32 x 32 tiles: 0.4 (64 x 1M beside 1024 x
// 1024, 443 parts) 185 more, 1.5 (100 x 400000, 900 x 900) 67, 5.6 (192 x
// 400000, 600 x 600) 19, 8.4 (256 x 200000, 600 x 600) 9; 12 (64 x 1M, 320 x
// 300000) 7 less, 14 (320 x 150000, 300 x 300) 12, 20 (256 x 500000, 600 x 600)
// 47, 40 (256 x 1M, 600 x 600) 217; fp32 results 6.6 21 more, 14 4 more, 13 3
// less, 17 36 less.
bool larger_pay(const std::vector<MuonMat>& mats, int products) {
  const int64_t len = part_rounds(mats, kMuonTiles[1], products);
  int64_t most = 1, saved = 0;
  for (const MuonMat& t : mats) {
    most = std::max(most, (int64_t(products) * t.np / kMuonRound + len - 1) / len);
    // two operands of `side` rows a tile, in fp16
    saved += (count({t}, kMuonTiles[0], true) * kMuonTiles[0] -
              count({t}, kMuonTiles[1], true) * kMuonTiles[1]) * 4 * products * t.np;
  }
  return most <= 32 || saved >= most * 12000000;
}

// `all`: rounds of the matrix's sums.  The same part of all tiles lies
// together: they read the same columns.
std::vector<MuonGemmTile> in_parts(const std::vector<MuonGemmTile>& tiles, int64_t all,
                                   int64_t len, fsdp_muon::Tiles* to) {
  std::vector<MuonGemmTile> out;
  const int64_t parts = (all + len - 1) / len, n = static_cast<int64_t>(tiles.size());
  for (int64_t p = 0; p < parts; ++p)
    for (int64_t k = 0; k < n; ++k) {
      MuonGemmTile t = tiles[k];
      t.m = static_cast<int32_t>(all * p / parts);
      t.n = static_cast<int32_t>(all * (p + 1) / parts) - t.m;
      t.flat_off = parts > 1 ? to->n_sums + k * parts + p : -1;
      out.push_back(t);
    }
  if (parts == 1) return out;
  for (MuonGemmTile t : tiles) {
    t.m = 0;
    t.n = static_cast<int32_t>(parts);
    t.flat_off = to->n_sums;
    to->n_sums += parts;
    to->join.push_back(t);
  }
  return out;
}

}  // namespace

fsdp_status build_muon(const fsdp_plan* plan, int32_t n_params, const int32_t* params,
                       fsdp_muon* mu) {
  mu->R = plan->R;
  mu->T = plan->T;
  mu->S = plan->S;
  const int32_t n_all = static_cast<int32_t>(plan->params.size());
  std::vector<int32_t> chosen(n_all, -1);  // matrix number of a parameter
  for (int32_t k = 0; k < n_params; ++k) {
    const int32_t p = params[k];
    if (p < 0 || p >= n_all || chosen[p] >= 0 || plan->shapes[p].size() < 2)
      return FSDP_ERR_INVALID_ARG;
    const Param& q = plan->params[p];
    if (q.d0 > kMaxSide || q.row > kMaxSide) return FSDP_ERR_UNSUPPORTED;
    chosen[p] = k;
    MuonMat t{};
    t.flat_off = q.flat_off;
    t.rows = q.d0;
    t.cols = q.row;
    t.tall = t.rows > t.cols;
    t.m = static_cast<int32_t>(std::min(t.rows, t.cols));
    t.n = static_cast<int32_t>(std::max(t.rows, t.cols));
    t.mp = static_cast<int32_t>(round_up(t.m, kMuonPad));
    t.np = static_cast<int32_t>(round_up(t.n, kMuonPad));
    t.ldx = static_cast<int32_t>(muon_pitch(t.np));
    t.lda = static_cast<int32_t>(muon_pitch(t.mp));
    t.off_x = mu->nx;
    t.off_a = mu->na;
    t.off_d = mu->nd;
    mu->nx += int64_t(t.mp) * t.ldx;
    mu->na += int64_t(t.mp) * t.lda;
    mu->nd += t.mp;
    const int64_t numel = t.rows * t.cols;
    t.norm_chunk =
        std::max(kNormChunk, round_up((numel + kNormParts - 1) / kNormParts, kNormChunk));
    t.norm_first = static_cast<int32_t>(mu->n_partial);
    t.norm_count = static_cast<int32_t>((numel + t.norm_chunk - 1) / t.norm_chunk);
    mu->n_partial += t.norm_count;
    if (k >= kMuonTall - 1) return FSDP_ERR_UNSUPPORTED;
    mu->mats.push_back(t);
    const double rows = static_cast<double>(t.rows), cols = static_cast<double>(t.cols);
    mu->scales.push_back(MuonScale{std::sqrt(std::max(1.0, rows / cols)),
                                   0.2 * std::sqrt(std::max(rows, cols))});
  }
  // grids first: a table that is refused is not built
  int64_t n_convert = 0, n_wide = 0, n_square = 0;
  for (const MuonMat& t : mu->mats) {
    n_convert += int64_t(t.mp / kConvert) * (t.np / kConvert);
    const int64_t si = t.mp / kMuonTiles[0], sj = t.np / kMuonTiles[0];
    n_wide += si * sj;
    n_square += si * (si + 1) / 2;
    // products have workgroups of up to 512 lanes
    if (n_convert > kMaxItems || n_wide > kMaxItems / 2 || n_square > kMaxItems / 2)
      return FSDP_ERR_UNSUPPORTED;
  }
  if (mu->n_partial > kMaxItems || mu->nd > INT32_MAX) return FSDP_ERR_UNSUPPORTED;

  // the per-element work: the plan's runs, cut where parameters end
  int64_t elements = 0;
  for (const MuonMat& t : mu->mats) elements += t.rows * t.cols;
  mu->apply.reserve(static_cast<size_t>(elements / kItem + 1));
  mu->momentum.reserve(static_cast<size_t>(elements / kItem + 1));
  mu->convert.reserve(static_cast<size_t>(n_convert));
  std::vector<Work> rest;
  auto split = [&](int64_t shard, int64_t flat, int64_t len) {
    // first parameter that ends after `flat`
    size_t p = std::upper_bound(plan->params.begin(), plan->params.end(), flat,
                                [](int64_t x, const Param& q) { return x < q.flat_off + q.numel; }) -
               plan->params.begin();
    for (; len > 0; ++p) {
      const Param& q = plan->params[p];
      const int64_t n = std::min(len, q.flat_off + q.numel - flat);
      if (chosen[p] < 0) {
        push_run(rest, shard, flat, n);
      } else {
        emit(shard, flat, n, chosen[p], mu->apply);
        emit(flat, shard, n, chosen[p], mu->momentum);
      }
      shard += n;
      flat += n;
      len -= n;
    }
  };
  for (const Work& w : plan->shard_runs) {
    if (w.src < 0)
      push_run(rest, w.dst, -1, w.len);
    else
      split(w.dst, w.src, w.len);
  }
  if (static_cast<int64_t>(mu->apply.size()) > kMaxItems ||
      static_cast<int64_t>(mu->momentum.size()) > kMaxItems ||
      count_items(rest, kShardChunk) > kMaxItems)
    return FSDP_ERR_UNSUPPORTED;
  emit_items(rest, kShardChunk, mu->rest.host);
  // in the order of the flat space (the flat layout has them so already)
  const auto before = [](const MuonItem& a, const MuonItem& b) { return a.dst < b.dst; };
  if (!std::is_sorted(mu->momentum.begin(), mu->momentum.end(), before))
    std::sort(mu->momentum.begin(), mu->momentum.end(), before);

  for (int32_t k = 0; k < n_params; ++k) {
    const MuonMat& t = mu->mats[k];
    for (int64_t i = 0; i < t.norm_count; ++i)
      mu->norm.push_back(MuonChunk{t.flat_off + i * t.norm_chunk,
                                   t.flat_off + std::min((i + 1) * t.norm_chunk, t.rows * t.cols),
                                   t.norm_first + i, 0});
    const int64_t ri = (t.tall ? t.np : t.mp) / kConvert, cj = (t.tall ? t.mp : t.np) / kConvert;
    for (int64_t i = 0; i < ri; ++i)
      for (int64_t j = 0; j < cj; ++j)
        mu->convert.push_back(MuonConvertTile{
            t.flat_off, t.off_x, static_cast<int32_t>(t.rows), static_cast<int32_t>(t.cols),
            t.ldx, static_cast<int32_t>(i), static_cast<int32_t>(j), k, t.norm_first,
            t.norm_count, t.tall, {}});
  }
  // products: the longest sums first, so that the short ones fill the end
  for (int split = 0; split < 2; ++split) {
    fsdp_muon::Tiles& to = mu->tiles[split];
    auto fill = [&](std::vector<MuonGemmTile>& out, int* shape, bool square, bool gram) {
      *shape = shape_of(mu->mats, square, gram, split != 0);
      const int products = split ? 3 : 1;
      // 64 x 64 tiles read half as much, where their parts are as many and not
      // too many of one tile: 1024 x 32000 takes 882 us with them and 1,133 in
      // parts of 32 x 32 (whole sums: 1,154), 512 x 32000 337 and 367 (426);
      // one tile of 32 x 1M in 512 parts took 1,920
      if (gram && *shape == 0 && count(mu->mats, kMuonTiles[1], true) >= kCus / 16 &&
          rounds_of(mu->mats, kMuonTiles[1], products) >= 2 * kCus * kPart &&
          larger_pay(mu->mats, products))
        *shape = 1;
      auto depth = [gram](const MuonMat& t) { return int64_t(gram ? t.np : t.mp); };
      const int64_t side = kMuonTiles[*shape];
      std::vector<int32_t> order(n_params);
      for (int32_t k = 0; k < n_params; ++k) order[k] = k;
      std::stable_sort(order.begin(), order.end(), [&](int32_t a, int32_t b) {
        return depth(mu->mats[a]) > depth(mu->mats[b]);
      });
      int64_t all = 0;
      for (const MuonMat& t : mu->mats) all += count({t}, side, square) * depth(t);
      Deal deal(all);
      const int64_t len = part_rounds(mu->mats, side, products);
      for (int32_t k : order) {
        const MuonMat& t = mu->mats[k];
        const int64_t si = (t.mp + side - 1) / side, sj = (t.np + side - 1) / side;
        const std::vector<MuonGemmTile> tiles =
            square ? grid(t, k, si, si, true) : grid(t, k, si, sj, false);
        if (gram && side <= kMuonPartTile) {
          const int64_t rounds = int64_t(products) * t.np / kMuonRound;
          const std::vector<MuonGemmTile> parts = in_parts(tiles, rounds, len, &to);
          deal.add(parts, depth(t) * static_cast<int64_t>(tiles.size()) /
                              static_cast<int64_t>(parts.size()));
        } else {
          deal.add(tiles, depth(t));
        }
      }
      out = deal.dealt();
    };
    fill(to.gram, &to.gram_shape, true, true);
    fill(to.poly, &to.poly_shape, true, false);
    fill(to.step, &to.step_shape, false, false);
    // (filling up may have made a table longer than its tiles)
    for (const auto* t : {&to.gram, &to.poly, &to.step})
      if (static_cast<int64_t>(t->size()) > kMaxItems / 2) return FSDP_ERR_UNSUPPORTED;
  }
  return FSDP_OK;
}

MuonWorkspace muon_workspace(const fsdp_muon* mu, bool split) {
  MuonWorkspace w{};
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += round_up(bytes, 256);
    return here;
  };
  const int64_t x = mu->nx * 2, a = mu->na * 2;
  w.partial = take(mu->n_partial * 8);
  w.coef = take(static_cast<int64_t>(mu->mats.size() * kMuonSteps * sizeof(MuonCoef)));
  w.adiag = take(mu->nd * 4);
  w.bdiag = take(mu->nd * 4);
  w.xh[0] = take(x);
  w.xh[1] = take(x);
  // the low parts, in bf8, are only read by the workgroup that replaces them,
  // unless they are an operand too, in fp16
  w.xl[0] = take(split ? x : mu->nx);
  w.xl[1] = split ? take(x) : w.xl[0];
  w.ah = take(a);
  w.bh = take(a);
  w.al = split ? take(a) : 0;
  w.bl = split ? take(a) : 0;
  const fsdp_muon::Tiles& t = mu->tiles[split ? 1 : 0];
  w.sums = take(t.n_sums * kMuonTiles[t.gram_shape] * kMuonTiles[t.gram_shape] * 4);
  w.bytes = at;
  return w;
}

}  // namespace fsdp

using fsdp::Range;
using fsdp::Ranges;
using fsdp::aligned;
using fsdp::any_overlap;
using fsdp::dtype_size;
using fsdp::overlap;
using fsdp::range_of;
using fsdp::valid_dtype;

fsdp_status fsdp_muon::device(bool split, fsdp::MuonDevice* out) const {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) {
    (void)hipGetLastError();
    return FSDP_ERR_HIP;
  }
  constexpr int kParts = 13;
  const void* from[kParts];
  int64_t size[kParts], at[kParts], bytes = 0;
  int n = 0;
  auto part = [&](const auto& v) {
    from[n] = v.data();
    size[n] = static_cast<int64_t>(v.size() * sizeof(v[0]));
    at[n] = bytes;
    bytes += (size[n] + 255) / 256 * 256;
    ++n;
  };
  part(norm);
  part(convert);
  part(momentum);
  part(apply);
  part(scales);
  for (const Tiles& t : tiles) {
    part(t.gram);
    part(t.poly);
    part(t.step);
    part(t.join);
  }
  static_assert(kParts == 5 + 2 * 4);
  std::lock_guard<std::mutex> lock(mu_);
  auto it = dev_.find(dev);
  if (it == dev_.end()) {
    // one copy: a small unit's tables are 13 of a few KB
    std::vector<char> all(static_cast<size_t>(bytes));
    for (int k = 0; k < kParts; ++k)
      if (size[k]) std::memcpy(all.data() + at[k], from[k], static_cast<size_t>(size[k]));
    void* mem = nullptr;
    if (hipMalloc(&mem, static_cast<size_t>(bytes)) != hipSuccess) {
      (void)hipGetLastError();
      return FSDP_ERR_OUT_OF_MEMORY;
    }
    if (hipMemcpy(mem, all.data(), all.size(), hipMemcpyHostToDevice) != hipSuccess) {
      (void)hipGetLastError();
      (void)hipFree(mem);
      return FSDP_ERR_HIP;
    }
    it = dev_.emplace(dev, mem).first;
  }
  const char* b = static_cast<const char*>(it->second);
  out->norm = reinterpret_cast<const fsdp::MuonChunk*>(b + at[0]);
  out->convert = reinterpret_cast<const fsdp::MuonConvertTile*>(b + at[1]);
  out->momentum = reinterpret_cast<const fsdp::MuonItem*>(b + at[2]);
  out->apply = reinterpret_cast<const fsdp::MuonItem*>(b + at[3]);
  const Tiles& t = tiles[split ? 1 : 0];
  out->scales = reinterpret_cast<const fsdp::MuonScale*>(b + at[4]);
  const int k = split ? 9 : 5;
  auto gemm = [&](int i, const std::vector<fsdp::MuonGemmTile>& v, int shape) {
    return fsdp::MuonTiles{reinterpret_cast<const fsdp::MuonGemmTile*>(b + at[i]),
                           static_cast<int64_t>(v.size()), shape};
  };
  out->gram = gemm(k, t.gram, t.gram_shape);
  out->poly = gemm(k + 1, t.poly, t.poly_shape);
  out->step = gemm(k + 2, t.step, t.step_shape);
  out->join = gemm(k + 3, t.join, t.gram_shape);
  return FSDP_OK;
}

fsdp_muon::~fsdp_muon() {
  for (auto& kv : dev_) (void)hipFree(kv.second);
}

namespace {

fsdp_status check(const fsdp_muon_hparams* hp) {
  if (!hp) return FSDP_ERR_INVALID_ARG;
  const double all[] = {hp->lr, hp->momentum, hp->weight_decay, hp->eps,
                        hp->ns_a, hp->ns_b, hp->ns_c};
  for (double x : all)
    if (!std::isfinite(x)) return FSDP_ERR_INVALID_ARG;
  if (hp->lr < 0 || !(hp->momentum >= 0 && hp->momentum < 1) || hp->weight_decay < 0 ||
      !(hp->eps >= 1e-300) || std::fabs(hp->ns_a) > 16 || std::fabs(hp->ns_b) > 16 ||
      std::fabs(hp->ns_c) > 16 || hp->ns_steps < 1 || hp->ns_steps > fsdp::kMuonSteps ||
      (hp->nesterov != 0 && hp->nesterov != 1) || hp->scale < FSDP_MUON_SCALE_NONE ||
      hp->scale > FSDP_MUON_SCALE_RMS)
    return FSDP_ERR_INVALID_ARG;
  return FSDP_OK;
}

fsdp::MuonScalars scalars(const fsdp_muon_hparams* hp) {
  return fsdp::MuonScalars{hp->momentum, 1.0 - hp->momentum, 1.0 - hp->lr * hp->weight_decay,
                           hp->lr,       hp->nesterov,       hp->scale};
}

// The gradients of a call, checked: R replicas [T], or the reduced [R][S].
fsdp_status take_grads(const fsdp_muon* mu, const void* const* grads, int32_t grad_dtype,
                       int32_t replicas, fsdp::PtrArray* g, Ranges* reads, bool* vec) {
  if (!grads || !valid_dtype(grad_dtype) || (replicas != 0 && replicas != 1))
    return FSDP_ERR_INVALID_ARG;
  if (!replicas && grad_dtype != FSDP_F32) return FSDP_ERR_INVALID_ARG;
  const int64_t es = dtype_size(grad_dtype);
  for (int q = 0; q < (replicas ? mu->R : 1); ++q) {
    if (!grads[q] || !aligned(grads[q], es)) return FSDP_ERR_INVALID_ARG;
    g->p[q] = grads[q];
    reads->push_back(range_of(grads[q], (replicas ? mu->T : mu->R * mu->S) * es));
    *vec = *vec && aligned(grads[q], 16);
  }
  return FSDP_OK;
}

bool meet(const Ranges& writes, const Ranges& reads) {
  for (const Range& w : writes)
    for (const Range& r : reads)
      if (overlap(w, r)) return true;
  return any_overlap(writes);
}

// The products of one fsdp_orthogonalize, arguments checked.
fsdp_status orthogonalize(const fsdp_muon* mu, const fsdp::MuonDevice& d,
                          const fsdp_muon_hparams* hp, const void* update, int32_t update_dt,
                          void* ortho, int32_t ortho_dt, char* ws, const fsdp::Sink& sink) {
  fsdp::MuonArgs a{};
  a.ws = ws;
  a.split = ortho_dt == FSDP_F32;
  a.low = a.split || update_dt == FSDP_F32;
  a.w = fsdp::muon_workspace(mu, a.split);
  a.steps = hp->ns_steps;
  const double poly[3] = {hp->ns_a, hp->ns_b, hp->ns_c};
  hipError_t e = fsdp::launch_muon_norm(a, d.norm, static_cast<int64_t>(mu->norm.size()), update,
                                        update_dt, sink);
  if (e == hipSuccess)
    e = fsdp::launch_muon_convert(a, d.convert, static_cast<int64_t>(mu->convert.size()), update,
                                  update_dt, hp->eps, poly, sink);
  for (int s = 0; s < hp->ns_steps && e == hipSuccess; ++s) {
    a.step = s;
    e = fsdp::launch_muon_gram(a, d.gram, d.join, s & 1, sink);
    if (e == hipSuccess) e = fsdp::launch_muon_poly(a, d.poly, s == 0, poly, sink);
    if (e == hipSuccess)
      e = fsdp::launch_muon_step(a, d.step, s & 1, s == 0, s == hp->ns_steps - 1, poly, ortho,
                                 ortho_dt, sink);
  }
  return fsdp::status_of(e);
}

}  // namespace

extern "C" {

fsdp_status fsdp_muon_plan(const fsdp_plan* plan, int32_t n_params, const int32_t* params,
                           fsdp_muon** out) {
  if (!out) return FSDP_ERR_INVALID_ARG;
  *out = nullptr;
  if (!plan || n_params < 1 || !params) return FSDP_ERR_INVALID_ARG;
  fsdp_muon* mu = new (std::nothrow) fsdp_muon();
  if (!mu) return FSDP_ERR_OUT_OF_MEMORY;
  const fsdp_status st =
      fsdp::guarded([&] { return fsdp::build_muon(plan, n_params, params, mu); });
  if (st != FSDP_OK) {
    delete mu;
    return st;
  }
  *out = mu;
  return FSDP_OK;
}

void fsdp_muon_destroy(fsdp_muon* mu) { delete mu; }

fsdp_status fsdp_muon_prepare(const fsdp_muon* mu, void* stream) {
  (void)stream;
  return fsdp::guarded([&]() -> fsdp_status {
    if (!mu) return FSDP_ERR_INVALID_ARG;
    fsdp::MuonDevice d;
    const fsdp::Work* w = nullptr;
    const fsdp_status st = mu->device(false, &d);
    return st != FSDP_OK ? st : mu->rest.device(&w);
  });
}

fsdp_status fsdp_muon_workspace(const fsdp_muon* mu, int32_t update_dtype, int32_t ortho_dtype,
                                int64_t* ortho_bytes, int64_t* step_bytes) {
  if (!mu || !valid_dtype(update_dtype) || !valid_dtype(ortho_dtype)) return FSDP_ERR_INVALID_ARG;
  if (ortho_bytes) *ortho_bytes = fsdp::muon_workspace(mu, ortho_dtype == FSDP_F32).bytes;
  if (step_bytes)
    *step_bytes = fsdp::muon_workspace(mu, false).bytes + (mu->T * 2 + 255) / 256 * 256;
  return FSDP_OK;
}

fsdp_status fsdp_muon_work_items(const fsdp_muon* mu, int32_t space, int64_t* out,
                                 int64_t capacity, int64_t* n) {
  if (!mu || !n || (space != 0 && space != 1)) return FSDP_ERR_INVALID_ARG;
  const std::vector<fsdp::MuonItem>& items = space == 0 ? mu->apply : mu->momentum;
  *n = static_cast<int64_t>(items.size());
  if (!out) return FSDP_OK;
  if (capacity < *n) return FSDP_ERR_INVALID_ARG;
  for (size_t i = 0; i < items.size(); ++i) {
    out[3 * i + 0] = items[i].dst;
    out[3 * i + 1] = items[i].src;
    out[3 * i + 2] = items[i].len;
  }
  return FSDP_OK;
}

fsdp_status fsdp_muon_momentum(const fsdp_muon* mu, const fsdp_muon_hparams* hp,
                               const void* const* grads, int32_t grad_dtype,
                               int32_t grads_are_replicas, float* m, void* update,
                               int32_t update_dtype, void* stream) {
  return fsdp::guarded([&]() -> fsdp_status {
    if (!mu || !m || !update || !valid_dtype(update_dtype)) return FSDP_ERR_INVALID_ARG;
    fsdp_status st = check(hp);
    if (st != FSDP_OK) return st;
    const int64_t ues = dtype_size(update_dtype);
    if (!aligned(m, 4) || !aligned(update, ues)) return FSDP_ERR_INVALID_ARG;
    fsdp::PtrArray g{};
    Ranges reads, writes;
    bool vec = aligned(m, 16) && aligned(update, 16);
    st = take_grads(mu, grads, grad_dtype, grads_are_replicas, &g, &reads, &vec);
    if (st != FSDP_OK) return st;
    writes.push_back(range_of(m, mu->R * mu->S * 4));
    writes.push_back(range_of(update, mu->T * ues));
    if (meet(writes, reads)) return FSDP_ERR_INVALID_ARG;
    fsdp::MuonDevice d;
    if ((st = mu->device(false, &d)) != FSDP_OK) return st;
    return fsdp::status_of(fsdp::launch_muon_momentum(
        d.momentum, static_cast<int64_t>(mu->momentum.size()), g, mu->R, grad_dtype,
        grads_are_replicas != 0, m, update, update_dtype, scalars(hp), vec,
        fsdp::StreamSink(stream)));
  });
}

fsdp_status fsdp_orthogonalize(const fsdp_muon* mu, const fsdp_muon_hparams* hp,
                               const void* update, int32_t update_dtype, void* ortho,
                               int32_t ortho_dtype, void* workspace, int64_t workspace_bytes,
                               void* stream) {
  return fsdp::guarded([&]() -> fsdp_status {
    if (!mu || !update || !ortho || !workspace || !valid_dtype(update_dtype) ||
        !valid_dtype(ortho_dtype))
      return FSDP_ERR_INVALID_ARG;
    fsdp_status st = check(hp);
    if (st != FSDP_OK) return st;
    const int64_t need = fsdp::muon_workspace(mu, ortho_dtype == FSDP_F32).bytes;
    if (workspace_bytes < need || !aligned(workspace, 256) ||
        !aligned(update, dtype_size(update_dtype)) || !aligned(ortho, dtype_size(ortho_dtype)))
      return FSDP_ERR_INVALID_ARG;
    const Range u = range_of(update, mu->T * dtype_size(update_dtype));
    const Range o = range_of(ortho, mu->T * dtype_size(ortho_dtype));
    const Range w = range_of(workspace, need);
    const bool in_place = update == ortho && update_dtype == ortho_dtype;
    if (overlap(w, u) || overlap(w, o) || (!in_place && overlap(u, o)))
      return FSDP_ERR_INVALID_ARG;
    fsdp::MuonDevice d;
    if ((st = mu->device(ortho_dtype == FSDP_F32, &d)) != FSDP_OK) return st;
    return orthogonalize(mu, d, hp, update, update_dtype, ortho, ortho_dtype,
                         static_cast<char*>(workspace), fsdp::StreamSink(stream));
  });
}

fsdp_status fsdp_muon_apply(const fsdp_muon* mu, const fsdp_muon_hparams* hp, const void* ortho,
                            int32_t ortho_dtype, float* master, void* param_out,
                            int32_t param_dtype, void* stream) {
  return fsdp::guarded([&]() -> fsdp_status {
    if (!mu || !ortho || !master || !param_out || !valid_dtype(ortho_dtype) ||
        !valid_dtype(param_dtype))
      return FSDP_ERR_INVALID_ARG;
    fsdp_status st = check(hp);
    if (st != FSDP_OK) return st;
    const int64_t oes = dtype_size(ortho_dtype), pes = dtype_size(param_dtype);
    if (!aligned(ortho, oes) || !aligned(master, 4) || !aligned(param_out, pes))
      return FSDP_ERR_INVALID_ARG;
    Ranges reads, writes;
    reads.push_back(range_of(ortho, mu->T * oes));
    writes.push_back(range_of(master, mu->R * mu->S * 4));
    writes.push_back(range_of(param_out, mu->R * mu->S * pes));
    if (meet(writes, reads)) return FSDP_ERR_INVALID_ARG;
    fsdp::MuonDevice d;
    if ((st = mu->device(false, &d)) != FSDP_OK) return st;
    return fsdp::status_of(fsdp::launch_muon_apply(
        d.apply, static_cast<int64_t>(mu->apply.size()), d.scales, ortho, ortho_dtype, master,
        param_out, param_dtype, scalars(hp),
        aligned(ortho, 16) && aligned(master, 16) && aligned(param_out, 16),
        fsdp::StreamSink(stream)));
  });
}

fsdp_status fsdp_muon_shard_step(const fsdp_muon* mu, const fsdp_muon_hparams* hp,
                                 const fsdp_adamw_hparams* adamw, int64_t step,
                                 const void* const* grads, int32_t grad_dtype, float* master,
                                 float* m, float* v, void* param_out, int32_t param_dtype,
                                 void* workspace, int64_t workspace_bytes, void* stream) {
  return fsdp::guarded([&]() -> fsdp_status {
    if (!mu || !master || !m || (adamw && !v) || !param_out || !workspace ||
        !valid_dtype(param_dtype))
      return FSDP_ERR_INVALID_ARG;
    fsdp_status st = check(hp);
    if (st != FSDP_OK) return st;
    fsdp::AdamScalars sc{};
    if (adamw && (st = fsdp::adam_scalars(adamw, step, &sc)) != FSDP_OK) return st;
    const int64_t n = mu->R * mu->S, pes = dtype_size(param_dtype);
    const int64_t update_bytes = (mu->T * 2 + 255) / 256 * 256;
    const int64_t need = fsdp::muon_workspace(mu, false).bytes + update_bytes;
    if (workspace_bytes < need || !aligned(workspace, 256) || !aligned(master, 4) ||
        !aligned(m, 4) || (adamw && !aligned(v, 4)) || !aligned(param_out, pes))
      return FSDP_ERR_INVALID_ARG;
    fsdp::PtrArray g{};
    Ranges reads, writes;
    bool vec = aligned(master, 16) && aligned(m, 16) && aligned(param_out, 16) &&
               (!adamw || aligned(v, 16));
    st = take_grads(mu, grads, grad_dtype, 1, &g, &reads, &vec);
    if (st != FSDP_OK) return st;
    writes.push_back(range_of(master, n * 4));
    writes.push_back(range_of(m, n * 4));
    if (adamw) writes.push_back(range_of(v, n * 4));
    writes.push_back(range_of(param_out, n * pes));
    writes.push_back(range_of(workspace, need));
    if (meet(writes, reads)) return FSDP_ERR_INVALID_ARG;
    fsdp::MuonDevice d;
    const fsdp::Work* rest = nullptr;
    if ((st = mu->device(false, &d)) != FSDP_OK) return st;
    if (adamw && (st = mu->rest.device(&rest)) != FSDP_OK) return st;
    const fsdp::StreamSink sink(stream);
    void* update = workspace;
    const fsdp::MuonScalars ms = scalars(hp);
    st = fsdp::status_of(fsdp::launch_muon_momentum(
        d.momentum, static_cast<int64_t>(mu->momentum.size()), g, mu->R, grad_dtype, true, m,
        update, FSDP_BF16, ms, vec, sink));
    if (st == FSDP_OK)
      st = orthogonalize(mu, d, hp, update, FSDP_BF16, update, FSDP_BF16,
                         static_cast<char*>(workspace) + update_bytes, sink);
    if (st == FSDP_OK)
      st = fsdp::status_of(fsdp::launch_muon_apply(
          d.apply, static_cast<int64_t>(mu->apply.size()), d.scales, update, FSDP_BF16, master,
          param_out, param_dtype, ms, vec, sink));
    if (st == FSDP_OK && adamw && !mu->rest.host.empty())
      st = fsdp::status_of(fsdp::launch_fused(rest, static_cast<int64_t>(mu->rest.host.size()), g,
                                              mu->R, grad_dtype, master, m, v, param_out,
                                              param_dtype, sc, nullptr, vec, sink));
    return st;
  });
}

}  // extern "C"
