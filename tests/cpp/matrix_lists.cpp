// The work lists that rs_plan_load makes for the matrix products, on the host,
// for operands of one or two parts: what each launch is worth, and that its
// jobs are sound.
//
// Reads "parts n" and n lines "rows cols" (WHOLE tensors) on stdin. Prints per
// list "[tiles of side, cut, jobs, share, behind, ahead]": the end of the launch
// over the mean share of the places that run at once, how many steps it is
// behind the mean, and how many ahead of the same launch with its cut tiles
// whole, longest first; then the workspace's bytes and those of the cut tiles'
// parts. Or "violation" where a step of a tile is missing or run twice, a part
// has no slab of its own or a cut tile is not joined once. Includes plan.cpp for
// lower_muon(); link with planner.cpp.
#include "plan.cpp"

#include <array>
#include <cstdio>
#include <map>
#include <set>

using namespace rs;

// When a launch ends whose jobs, in order, go to the place that is free first.
static double run(std::vector<double> places, const std::vector<double>& costs) {
  for (double c : costs) *std::min_element(places.begin(), places.end()) += c;
  return *std::max_element(places.begin(), places.end());
}

static bool sound(const ProductList& l, const std::vector<MuonMat>& mats, bool over_n) {
  std::map<std::array<int, 3>, std::map<int, ProductJob>> tiles;   // by tile, by first step
  for (const ProductJob& p : l.jobs)
    if (!tiles[{p.mat, p.i, p.j}].insert({p.k0, p}).second) return false;
  std::map<std::array<int, 3>, int> joined;   // first slab of each cut tile
  for (const ProductJob& p : l.joins)
    if (!joined.insert({{p.mat, p.i, p.j}, p.slab}).second) return false;
  std::set<int> slabs;
  for (const auto& [tile, parts] : tiles) {
    const MuonMat& q = mats[tile[0]];
    int step = 0, number = 0;
    for (const auto& [k0, p] : parts) {
      if (k0 != step || p.k1 <= k0 || p.parts != parts.size()) return false;
      step = p.k1;
      if (parts.size() == 1) continue;
      if (!joined.count(tile) || p.slab != joined[tile] + number++ || p.slab >= l.slabs || !slabs.insert(p.slab).second) return false;
    }
    if (step != (over_n ? q.np : q.mp) / kMatK || (parts.size() > 1) != (joined.count(tile) > 0)) return false;
  }
  for (const auto& join : joined)
    if (!tiles.count(join.first)) return false;
  return true;
}

int main() {
  int n = 0, parts = 1;
  if (std::scanf("%d %d", &parts, &n) != 2) return 1;
  std::vector<Tensor> t;
  for (int64_t i = 0, at = 0; i < n; ++i) {
    Tensor x{};
    if (std::scanf("%ld %ld", &x.rows, &x.cols) != 2) return 1;
    x.n = x.g = x.rows * x.cols;
    x.start = at;
    x.kind = RS_WHOLE;
    at += (x.n + 15) / 16 * 16;
    t.push_back(x);
  }
  MuonTables mt;
  lower_muon(t, &mt, parts);
  auto weight = [&](const ProductJob& p) { return mt.mats[p.mat].two_part ? 3.0 : 1.0; };
  int64_t slabs = 0;
  for (int w = 0; w < kMatLists; ++w) {
    const ProductList& l = mt.list[w];
    const bool apply = w == kApply || w == kApplySingle;
    size_t tiles = 0;
    for (const MuonMat& q : mt.mats) {
      if (parts == 2 && (!q.two_part || q.paired)) {
        std::printf("violation: one-part operands\n");
        return 0;
      }
      if (w == kSquarePaired ? !q.paired : (w == kGramSingle || w == kApplySingle) && q.paired) continue;
      const int64_t ti = ceil_div(q.m, l.side);
      tiles += apply ? ti * ceil_div(q.n, l.side) : ti * (ti + 1) / 2;
    }
    std::set<std::array<int, 3>> seen;
    std::vector<double> costs, uncut, whole;
    double total = 0;
    for (const ProductJob& p : l.jobs) {
      seen.insert({p.mat, p.i, p.j});
      costs.push_back((p.k1 - p.k0) * weight(p));
      total += costs.back();
      if (p.parts == 1) uncut.push_back(costs.back());
    }
    if (seen.size() != tiles || !sound(l, mt.mats, w == kGram || w == kGramSingle)) {
      std::printf("violation: list %d\n", w);
      return 0;
    }
    for (const ProductJob& p : l.joins) whole.push_back(p.k1 * weight(p));
    std::sort(whole.begin(), whole.end(), std::greater<double>());
    uncut.insert(uncut.end(), whole.begin(), whole.end());
    const std::vector<double> places(mat_places(l.side), 0.0);
    const double end = run(places, costs), mean = total / places.size();
    std::printf("[%zu tiles of %d, %zu cut, %zu jobs, share %.2f, behind %.1f, ahead %.1f] ", tiles, l.side, l.joins.size(),
                l.jobs.size(), total ? end / mean : 1.0, end - mean, run(places, uncut) - end);
    slabs = std::max(slabs, int64_t(4) * l.side * l.side * l.slabs);
  }
  std::printf("work %lld parts %lld\n", static_cast<long long>(mt.work_bytes), static_cast<long long>(slabs));
  return 0;
}
