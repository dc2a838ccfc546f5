// Random units and products through the host side, under the sanitizers: the
// gather's table covers every element, code, scale and element of rest once, a
// product's grid has a workgroup for every tile that there can be, and the entry
// points refuse or reach the launch.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "products.hpp"
#include "quant.hpp"

static int failures = 0;
#define CHECK(c)                                          \
  do {                                                    \
    if (!(c)) {                                           \
      ++failures;                                         \
      std::printf("%s:%d: %s\n", __FILE__, __LINE__, #c); \
    }                                                     \
  } while (0)

static void check_unit(std::mt19937& rng) {
  auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  const int n = pick(1, 6), R = pick(1, 9), layout = pick(0, 1);
  std::vector<int32_t> ndims, params;
  std::vector<int64_t> dims;
  for (int p = 0; p < n; ++p) {
    const int d = pick(1, 3);
    ndims.push_back(d);
    for (int k = 0; k < d; ++k)
      dims.push_back(pick(0, 9) ? pick(1, 40) : k == d - 1 ? pick(1900, 5000) : pick(1, 90));
    if (d > 1 && pick(0, 3)) params.push_back(p);
  }
  fsdp_plan* plan = nullptr;
  CHECK(fsdp_plan_layout(n, ndims.data(), dims.data(), R, layout, &plan) == FSDP_OK);
  fsdp_quant* qu = nullptr;
  const fsdp_status st =
      fsdp_quant_plan(plan, static_cast<int32_t>(params.size()), params.data(), &qu);
  CHECK((st == FSDP_OK) == !params.empty());
  if (st != FSDP_OK) {
    fsdp_plan_destroy(plan);
    return;
  }
  std::vector<int64_t> shard_of(plan->T, -1);
  for (const fsdp::Segment& s : plan->segments)
    for (int64_t i = 0; i < s.len; ++i)
      shard_of[s.flat_off + i] = s.rank * plan->S + s.shard_off + i;
  std::vector<int> unit(plan->T), codes(qu->code_bytes), scales(qu->n_scales), rest(qu->n_rest);
  for (const fsdp::QuantItem& w : qu->items) {
    CHECK(w.n_rows >= 1 && w.cols >= 1);
    CHECK(w.pitch == 0 || (w.pitch % 16 == 0 && w.to % 16 == 0 && w.pitch >= w.cols));
    CHECK(w.cols <= fsdp::kWaveRow || w.n_rows == 1);
    for (int64_t r = 0; r < w.n_rows; ++r) {
      for (int64_t e = 0; e < w.cols; ++e) {
        const int64_t flat = w.flat + r * w.cols + e;
        CHECK(shard_of.at(flat) == w.src + r * w.cols + e);
        ++unit.at(flat);
        if (w.pitch == 0) ++rest.at(w.to + e);
      }
      if (w.pitch == 0) continue;
      ++scales.at(w.scale + r);
      for (int64_t e = 0; e < w.pitch; ++e) ++codes.at(w.to + r * w.pitch + e);
    }
  }
  for (const auto& all : {unit, codes, scales, rest})
    for (int x : all) CHECK(x == 1);
  std::vector<char> shards(plan->R * plan->S * 2 + 16);
  const size_t nc = qu->code_bytes + 16, ns = qu->n_scales + 1, nr = qu->n_rest + 1;
  std::vector<std::vector<char>> buf;
  std::vector<int8_t*> pc;
  std::vector<float*> ps;
  std::vector<void*> pr, pf;
  for (int r = 0; r < R; ++r) {
    for (size_t bytes : {nc, ns * 4, nr * 2, static_cast<size_t>(plan->T) * 4 + 16})
      buf.emplace_back(bytes + 16);
    auto up = [&](size_t back) {
      return reinterpret_cast<char*>(
          (reinterpret_cast<uintptr_t>(buf[buf.size() - back].data()) + 15) / 16 * 16);
    };
    pc.push_back(reinterpret_cast<int8_t*>(up(4)));
    ps.push_back(reinterpret_cast<float*>(up(3)));
    pr.push_back(up(2));
    pf.push_back(up(1));
  }
  CHECK(fsdp_gather_quantize(qu, shards.data(), FSDP_BF16, pc.data(), ps.data(), pr.data(),
                             nullptr) == FSDP_ERR_HIP);
  CHECK(fsdp_dequantize(qu, pc.data(), ps.data(), pr.data(), FSDP_BF16, pf.data(), FSDP_F32,
                        nullptr) == FSDP_ERR_HIP);
  if (R > 1) {
    std::swap(pc[0], pc[1]);
    pc[1] = pc[0];
    CHECK(fsdp_gather_quantize(qu, shards.data(), FSDP_BF16, pc.data(), ps.data(), pr.data(),
                               nullptr) == FSDP_ERR_INVALID_ARG);
  }
  fsdp_quant_destroy(qu);
  fsdp_plan_destroy(plan);
}

static void check_product(std::mt19937& rng) {
  auto pick = [&](int64_t lo, int64_t hi) {
    return std::uniform_int_distribution<int64_t>(lo, hi)(rng);
  };
  fsdp_matmul m{};
  m.op = static_cast<int32_t>(pick(0, 2));
  m.groups = static_cast<int32_t>(pick(0, 2) ? pick(1, 8) : pick(1, 300));
  m.rows = pick(0, 3) ? pick(0, 300) : pick(0, 20000);
  m.n = pick(0, 2) ? pick(1, 300) : pick(1, 9000);
  m.k = pick(0, 2) ? pick(1, 300) : pick(1, 9000);
  m.lda = std::max(m.n, m.k) + pick(0, 9);
  m.ldb = std::max(m.n, m.k) + pick(0, 9);
  m.ldc = std::max(m.n, m.k) + pick(0, 9);
  m.group_stride = std::max(m.n, m.k) * (std::max(m.n, m.k) + 9);
  const bool direct = pick(0, 1);
  const auto type = static_cast<fsdp::ProductType>(pick(0, m.op == FSDP_MATMUL_TN ? 1 : 2));
  const fsdp::ProductRule r = fsdp::product_rule(m, type, direct || type == fsdp::kProductI8);
  CHECK(r.tile >= 0 && r.tile < 7);
  const int64_t rows = fsdp::kProductRows[r.tile], cols = fsdp::product_cols(r.tile, m.op);
  CHECK(r.n_parts >= 1 && r.n_parts <= 64 && r.grid >= 0);
  CHECK(type != fsdp::kProductF32 || ((r.tile == fsdp::kTiny || r.tile == fsdp::kSmall || r.tile == fsdp::kMid) &&
                                       r.n_parts == 1));
  CHECK(r.direct || r.tile == fsdp::kSmall || r.tile == fsdp::kMid || type == fsdp::kProductF32);
  CHECK((r.tile == fsdp::kTiny) <= (type == fsdp::kProductF32));
  auto down = [&](int64_t x) { return (x + rows - 1) / rows; };
  auto across = [&](int64_t x) { return (x + cols - 1) / cols; };
  if (m.op == FSDP_MATMUL_TN) {
    CHECK(r.tile != fsdp::kThin && r.tile != fsdp::kApart);
    const int64_t all = down(m.n) * across(m.k) * r.n_parts;
    CHECK(r.grid >= (all + 7) / 8 * 8 * m.groups);
    CHECK(r.join == down(m.n) * across(m.k) * m.groups);
    CHECK(r.workspace == (r.n_parts > 1 ? all * m.groups * rows * cols * 4 : 0));
  } else {
    CHECK(r.workspace == 0 && r.n_parts == 1);
    // random sizes that add up to rows, and the worst ones: single rows
    // behind whole tiles
    std::vector<int64_t> cut(m.groups + 1, 0);
    cut[m.groups] = m.rows;
    for (int64_t g = 1; g < m.groups; ++g) cut[g] = pick(0, m.rows);
    std::sort(cut.begin(), cut.end());
    // the last tiles of the largest may be cut in two or four
    auto wanted = [&](int64_t tiles) {
      const int64_t rest = tiles % 256;
      if (r.tile == fsdp::kBig && tiles > 256 && rest <= 128)
        tiles += rest * (rest <= 64 ? 3 : 1);
      return (tiles + 7) / 8 * 8;
    };
    int64_t sum = 0;
    for (int64_t g = 0; g < m.groups; ++g) sum += down(cut[g + 1] - cut[g]);
    CHECK(r.grid >= wanted(sum * across(m.n)) && r.grid % 8 == 0);
    if (m.groups > 1) {
      const int64_t ones = std::min<int64_t>(m.groups - 1, m.rows);
      CHECK(r.grid >= wanted((ones + down(m.rows - ones)) * across(m.n)));
    }
  }
  int64_t bytes = -1;
  if (type == fsdp::kProductI8) return;
  CHECK(fsdp_grouped_matmul_workspace(&m, type, &bytes) == FSDP_OK && bytes >= r.workspace);
  // far-apart addresses that nothing reads
  const uintptr_t base = uintptr_t(1) << 45, far = uintptr_t(1) << 42;
  auto at = [&](int i) { return reinterpret_cast<void*>(base + i * far); };
  const fsdp_status st =
      fsdp_grouped_matmul(&m, static_cast<const int32_t*>(at(0)), at(1), at(2), type, at(3),
                          FSDP_F32, at(4), bytes, nullptr);
  CHECK(st == (m.rows == 0 && m.op != FSDP_MATMUL_TN ? FSDP_OK : FSDP_ERR_HIP));
}

int main(int argc, char** argv) {
  const int n = argc > 1 ? std::atoi(argv[1]) : 100;
  std::mt19937 rng(5);
  for (int i = 0; i < n; ++i) check_unit(rng);
  for (int i = 0; i < 20 * n; ++i) check_product(rng);
  std::printf("checked %d random units, failures %d\n", n, failures);
  return failures ? 1 : 0;
}
