// Random units through the host side of the Muon step, under the sanitizers:
// the tables of every kernel cover what they have to, once, inside the
// workspace, and the entry points refuse or reach the first launch.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <tuple>
#include <vector>

#include "muon.hpp"

static int failures = 0;
#define CHECK(c)                                                   \
  do {                                                             \
    if (!(c)) {                                                    \
      ++failures;                                                  \
      std::printf("%s:%d: %s\n", __FILE__, __LINE__, #c);          \
    }                                                              \
  } while (0)

// Every tile of every matrix once, each with its matrix's own numbers; tables
// that mix empty tiles in keep them behind a die's own.
static void check_tiles(const fsdp_muon& mu, const std::vector<fsdp::MuonGemmTile>& tiles,
                        int shape, bool square, bool parts = false) {
  const int64_t side = fsdp::kMuonTiles[shape];
  std::set<std::tuple<int, int, int, int>> seen;
  size_t whole = 0;
  bool ended[8] = {};
  for (size_t p = 0; p < tiles.size(); ++p) {
    const fsdp::MuonGemmTile& t = tiles[p];
    if (t.mat < 0) {
      ended[p % 8] = true;
      continue;
    }
    CHECK(!ended[p % 8]);
    const int k = t.mat & ~fsdp::kMuonTall;
    CHECK(k < static_cast<int>(mu.mats.size()));
    const fsdp::MuonMat& m = mu.mats[k];
    CHECK(((t.mat & fsdp::kMuonTall) != 0) == (m.rows > m.cols));
    CHECK(t.off_x == m.off_x && t.off_a == m.off_a && t.off_d == m.off_d);
    CHECK(t.mp == m.mp && t.np == m.np);
    CHECK(parts || (t.flat_off == m.flat_off && t.m == m.m && t.n == m.n));
    CHECK(t.ldx == m.ldx && t.lda == m.lda);
    CHECK(t.i >= 0 && t.j >= 0 && t.i * side < m.mp && t.j * side < (square ? m.mp : m.np));
    CHECK(!square || t.i >= t.j);
    CHECK(seen.insert({k, t.i, t.j, parts ? t.m : 0}).second);
    whole += !parts || t.m == 0;  // first parts stand for their tiles
  }
  CHECK(tiles.empty() || tiles.back().mat >= 0);
  size_t want = 0;
  for (const fsdp::MuonMat& m : mu.mats) {
    const int64_t si = (m.mp + side - 1) / side, sj = (m.np + side - 1) / side;
    want += square ? si * (si + 1) / 2 : si * sj;
  }
  CHECK(whole == want);
}

// A's smaller tiles: the parts of a tile's sum follow each other from its
// first round to its last, each with a partial sum of its own, which the
// tile's join reads in that order; a sum in one piece has neither.  A join is
// worth 64 rounds at least, and parts give every compute unit two at most.
static int check_parts(const fsdp_muon& mu, const fsdp_muon::Tiles& t, int products) {
  if (t.gram_shape > 1) {
    CHECK(t.join.empty() && t.n_sums == 0);
    check_tiles(mu, t.gram, t.gram_shape, true);
    return 0;
  }
  std::map<std::tuple<int, int, int>, std::map<int, const fsdp::MuonGemmTile*>> tiles;
  std::map<std::tuple<int, int, int>, const fsdp::MuonGemmTile*> joins;
  for (const fsdp::MuonGemmTile& g : t.gram)
    if (g.mat >= 0) CHECK((tiles[{g.mat, g.i, g.j}].insert({g.m, &g}).second));
  for (const fsdp::MuonGemmTile& g : t.join) CHECK((joins.insert({{g.mat, g.i, g.j}, &g}).second));
  std::set<int64_t> used;
  int longest = 0, whole = 0, in_parts = 0;
  for (const auto& [key, list] : tiles) {
    const int all = products * (list.begin()->second->np / 64);
    int at = 0, k = 0;
    const auto join = joins.find(key);
    CHECK((join != joins.end()) == (list.size() > 1));
    for (const auto& [first, g] : list) {
      CHECK(first == at && g->n > 0);
      at += g->n;
      longest = std::max<int>(longest, g->n);
      if (join == joins.end()) {
        CHECK(g->flat_off == -1);
      } else {
        CHECK(g->flat_off == join->second->flat_off + k && used.insert(g->flat_off).second);
        CHECK(g->flat_off >= 0 && g->flat_off < t.n_sums);
      }
      ++k;
    }
    CHECK(at == all);
    whole = std::max(whole, all);
    if (join != joins.end()) {
      CHECK(join->second->n == k);
      in_parts += k;
    }
  }
  CHECK(static_cast<int64_t>(used.size()) == t.n_sums && in_parts == t.n_sums);
  CHECK(t.n_sums == 0 || whole >= longest + 64);
  CHECK(in_parts <= 512 + static_cast<int>(tiles.size()));
  check_tiles(mu, t.gram, t.gram_shape, true, true);
  return t.n_sums > 0;
}

static int parted = 0;

static void check_unit(const fsdp_muon& mu) {
  int64_t x = 0, a = 0, d = 0;
  for (const fsdp::MuonMat& m : mu.mats) {
    CHECK(m.m == std::min(m.rows, m.cols) && m.n == std::max(m.rows, m.cols));
    CHECK(m.mp % 64 == 0 && m.np % 64 == 0 && m.mp >= m.m && m.np >= m.n);
    CHECK(m.mp - m.m < 64 && m.np - m.n < 64);
    CHECK(m.ldx >= m.np && m.lda >= m.mp && m.ldx / 128 % 2 == 1 && m.lda / 128 % 2 == 1);
    CHECK(m.ldx % 128 == 0 && m.lda % 128 == 0);
    CHECK(m.off_x == x && m.off_a == a && m.off_d == d);
    x += int64_t(m.mp) * m.ldx;
    a += int64_t(m.mp) * m.lda;
    d += m.mp;
  }
  CHECK(mu.nx == x && mu.na == a && mu.nd == d);
  for (const auto& t : mu.tiles) {
    parted += check_parts(mu, t, &t == mu.tiles ? 1 : 3);
    check_tiles(mu, t.poly, t.poly_shape, true);
    check_tiles(mu, t.step, t.step_shape, false);
  }
  CHECK(mu.tiles[1].gram_shape < 3 && mu.tiles[1].poly_shape < 3 && mu.tiles[1].step_shape < 3);
  // norm: chunks tile every matrix; conversion: 64 x 64 tiles of its planes
  std::map<int64_t, int64_t> next;
  for (const fsdp::MuonMat& m : mu.mats) next[m.flat_off] = m.flat_off;
  int64_t to = 0;
  for (const fsdp::MuonChunk& c : mu.norm) {
    CHECK(c.to == to++ && c.lo < c.hi);
    auto it = next.upper_bound(c.lo);
    --it;
    CHECK(it->second == c.lo);
    it->second = c.hi;
  }
  CHECK(to == mu.n_partial);
  for (const fsdp::MuonMat& m : mu.mats) CHECK(next[m.flat_off] == m.flat_off + m.rows * m.cols);
  std::set<std::tuple<int, int, int>> seen;
  size_t want = 0;
  for (const fsdp::MuonMat& m : mu.mats) want += size_t(m.mp / 64) * (m.np / 64);
  for (const fsdp::MuonConvertTile& t : mu.convert) {
    const fsdp::MuonMat& m = mu.mats[t.mat];
    CHECK(t.i * 64 < (m.tall ? m.np : m.mp) && t.j * 64 < (m.tall ? m.mp : m.np));
    CHECK(t.rows == m.rows && t.cols == m.cols && t.off_x == m.off_x && t.ldx == m.ldx);
    CHECK(t.norm_first == m.norm_first && t.norm_count == m.norm_count && t.norm_count <= 1024);
    CHECK(seen.insert({t.mat, t.i, t.j}).second);
  }
  CHECK(seen.size() == want);
  for (bool split : {false, true}) {
    const fsdp::MuonWorkspace w = fsdp::muon_workspace(&mu, split);
    const int64_t lo = split ? 2 * x : x;
    std::vector<std::pair<int64_t, int64_t>> parts = {
        {w.partial, mu.n_partial * 8}, {w.coef, int64_t(mu.mats.size()) * 16},
        {w.adiag, d * 4},              {w.bdiag, d * 4},
        {w.xh[0], 2 * x},              {w.xh[1], 2 * x},
        {w.xl[0], lo},                 {w.ah, 2 * a},
        {w.bh, 2 * a},                 {w.sums, mu.tiles[split].n_sums * (mu.tiles[split].gram_shape ? 16384 : 4096)}};
    if (split) {
      parts.push_back({w.xl[1], lo});
      parts.push_back({w.al, 2 * a});
      parts.push_back({w.bl, 2 * a});
    }
    for (size_t i = 0; i < parts.size(); ++i) {
      CHECK(parts[i].first % 256 == 0 && parts[i].first + parts[i].second <= w.bytes);
      for (size_t j = 0; j < i; ++j)
        CHECK(parts[i].first + parts[i].second <= parts[j].first ||
              parts[j].first + parts[j].second <= parts[i].first);
    }
  }
}

int main(int argc, char** argv) {
  const int n = argc > 1 ? std::atoi(argv[1]) : 100;
  std::mt19937 rng(7);
  auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  for (int u = 0; u < n; ++u) {
    const int k = pick(1, u % 10 == 0 ? 60 : 8);
    const int most = u % 7 == 0 ? 2500 : 300;
    const int wide = u % 11 == 0 ? 100 : 1;  // second dimensions
    std::vector<int32_t> nd;
    std::vector<int64_t> dims;
    for (int p = 0; p < k; ++p) {
      const int dd = pick(1, 3);
      nd.push_back(dd);
      for (int q = 0; q < dd; ++q) dims.push_back(q < 2 ? pick(1, most) * (q ? wide : 1) : pick(1, 4));
    }
    fsdp_plan* plan = nullptr;
    CHECK(fsdp_plan_layout(k, nd.data(), dims.data(), pick(1, 9), pick(0, 1), &plan) == FSDP_OK);
    std::vector<int32_t> chosen;
    for (int p = 0; p < k; ++p)
      if (nd[p] >= 2 && pick(0, 3)) chosen.push_back(p);
    std::shuffle(chosen.begin(), chosen.end(), rng);
    fsdp_muon* mu = nullptr;
    const fsdp_status st =
        fsdp_muon_plan(plan, static_cast<int32_t>(chosen.size()), chosen.data(), &mu);
    CHECK(st == (chosen.empty() ? FSDP_ERR_INVALID_ARG : FSDP_OK) && (mu != nullptr) == (st == 0));
    const fsdp_plan_info info = [&] {
      fsdp_plan_info i;
      fsdp_plan_get_info(plan, &i);
      return i;
    }();
    fsdp_plan_destroy(plan);
    if (!mu) continue;
    check_unit(*mu);
    // the items of both spaces, through the entry point
    for (int space = 0; space < 2; ++space) {
      int64_t count = 0;
      CHECK(fsdp_muon_work_items(mu, space, nullptr, 0, &count) == FSDP_OK);
      std::vector<int64_t> out(3 * count);
      CHECK(fsdp_muon_work_items(mu, space, out.data(), count - 1, &count) ==
            (count ? FSDP_ERR_INVALID_ARG : FSDP_OK));
      CHECK(fsdp_muon_work_items(mu, space, out.data(), count, &count) == FSDP_OK);
      int64_t all = 0;
      for (int64_t i = 0; i < count; ++i) all += out[3 * i + 2];
      int64_t elements = 0;
      for (const fsdp::MuonMat& m : mu->mats) elements += m.rows * m.cols;
      CHECK(all == elements);
    }
    // arguments that pass every check get as far as the device; others do not
    fsdp_muon_hparams hp{1e-3, 0.95, 0.01, 1e-7, 3.4445, -4.775, 2.0315, 5, 1, 2};
    fsdp_adamw_hparams ad{1e-3, 0.9, 0.999, 1e-8, 0.01};
    auto at = [](int i) { return reinterpret_cast<void*>(uintptr_t(1) << 40 | uintptr_t(i) << 32); };
    const void* grads[64];
    for (int q = 0; q < info.world; ++q) grads[q] = at(20 + q);
    int64_t ortho = 0, step = 0;
    CHECK(fsdp_muon_workspace(mu, FSDP_F32, FSDP_F32, &ortho, &step) == FSDP_OK);
    float* f = static_cast<float*>(at(1));
    float* m = static_cast<float*>(at(2));
    float* v = static_cast<float*>(at(3));
    CHECK(fsdp_muon_momentum(mu, &hp, grads, FSDP_BF16, 1, m, at(4), FSDP_BF16, nullptr) < 0);
    CHECK(fsdp_orthogonalize(mu, &hp, at(4), FSDP_F32, at(5), FSDP_F32, at(6), ortho, nullptr) < 0);
    CHECK(fsdp_orthogonalize(mu, &hp, at(4), FSDP_F32, at(5), FSDP_F32, at(6), ortho - 1,
                             nullptr) == FSDP_ERR_INVALID_ARG);
    CHECK(fsdp_muon_apply(mu, &hp, at(5), FSDP_BF16, f, at(7), FSDP_F32, nullptr) < 0);
    CHECK(fsdp_muon_shard_step(mu, &hp, &ad, 1, grads, FSDP_BF16, f, m, v, at(7), FSDP_BF16, at(6),
                               step, nullptr) < 0);
    CHECK(fsdp_muon_shard_step(mu, &hp, &ad, 0, grads, FSDP_BF16, f, m, v, at(7), FSDP_BF16, at(6),
                               step, nullptr) == FSDP_ERR_INVALID_ARG);
    fsdp_muon_destroy(mu);
  }
  CHECK(n < 100 || parted >= 10);
  std::printf("checked %d random units, failures %d\n", n, failures);
  return failures != 0;
}
