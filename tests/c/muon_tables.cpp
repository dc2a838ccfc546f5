// Which tiles a unit's products get (no GPU).  Every line of the input is one
// unit, "rows columns rows columns ..."; every line of the output its choice
// for bf16 results and then for fp32 ones: the tiles' sides of A, B and X',
// the longest sum of a launch of A in rounds, and the most parts that one of
// A's tiles is joined from (1: none).
#include <algorithm>
#include <cstdio>
#include <iostream>
#include <sstream>
#include <string>
#include <vector>

#include "muon.hpp"

int main() {
  std::string line;
  while (std::getline(std::cin, line)) {
    std::istringstream in(line);
    std::vector<int64_t> dims;
    for (int64_t d; in >> d;) dims.push_back(d);
    const int32_t n = static_cast<int32_t>(dims.size() / 2);
    std::vector<int32_t> nd(n, 2), all(n);
    for (int32_t k = 0; k < n; ++k) all[k] = k;
    fsdp_plan* plan = nullptr;
    fsdp_muon* mu = nullptr;
    if (fsdp_plan_layout(n, nd.data(), dims.data(), 1, 0, &plan) != FSDP_OK ||
        fsdp_muon_plan(plan, n, all.data(), &mu) != FSDP_OK)
      return 1;
    for (const auto& t : mu->tiles) {
      int longest = 0, parts = 1;
      if (t.gram_shape <= 1) {
        for (const fsdp::MuonGemmTile& g : t.gram)
          if (g.mat >= 0) longest = std::max(longest, g.n);
        for (const fsdp::MuonGemmTile& g : t.join) parts = std::max(parts, g.n);
      }
      std::printf("%d %d %d %d %d ", fsdp::kMuonTiles[t.gram_shape],
                  fsdp::kMuonTiles[t.poly_shape], fsdp::kMuonTiles[t.step_shape], longest, parts);
    }
    std::printf("\n");
    fsdp_muon_destroy(mu);
    fsdp_plan_destroy(plan);
  }
  return 0;
}
