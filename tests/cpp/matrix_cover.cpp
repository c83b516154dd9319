// Host check of the work lists that rs_plan_load makes for the matrix
// products (rs_orthogonalize, rs_muon_step): every step of every output tile
// is run exactly once, the parts of a cut tile have slabs of their own in
// order and are joined once, chunks and spread tiles cover each matrix once,
// operands do not overlap in the workspace, and the launch's jobs, taken in
// order by the places that run at once, end together.
//
// Reads "n" and n lines "rows cols" (WHOLE tensors) on stdin; prints "ok" and
// per product the tile side, tiles, cut tiles, jobs, the end over the mean
// share and how many steps it is behind it, or the first violation. With an argument 1-4 it
// first plants a mistake (a job dropped, a step doubled, a slab shared, two
// operands overlapping), which must be reported. Includes plan.cpp for
// lower_muon(); link with planner.cpp.
#include "plan.cpp"

#include <cstdio>
#include <map>
#include <set>
#include <tuple>

using namespace rs;

static int bad(const char* what) {
  std::printf("violation: %s\n", what);
  return 0;
}

int main(int argc, char** argv) {
  const int plant = argc > 1 ? std::atoi(argv[1]) : 0;
  int n = 0;
  if (std::scanf("%d", &n) != 1) return 1;
  std::vector<Tensor> t;
  int64_t at = 0;
  for (int i = 0; i < n; ++i) {
    Tensor x{};
    if (std::scanf("%ld %ld", &x.rows, &x.cols) != 2) return 1;
    x.n = x.g = x.rows * x.cols;
    x.start = at;
    x.kind = RS_WHOLE;
    at += (x.n + 15) / 16 * 16;
    t.push_back(x);
  }
  MuonTables mt;
  lower_muon(t, &mt);
  if (plant == 1) mt.list[0].jobs.pop_back();
  if (plant == 2) mt.list[2].jobs[0].k1 += 1;
  if (plant == 3)
    for (auto& l : mt.list)
      for (auto& j : l.jobs)
        if (j.parts > 1) j.slab = l.joins[0].slab;
  if (plant == 4) mt.mats[0].xl = mt.mats[0].xh;

  std::map<int32_t, int64_t> chunks;
  for (const auto& c : mt.chunks) {
    if (c.chunk != chunks[c.mat]++) return bad("chunks");
  }
  for (size_t k = 0; k < mt.mats.size(); ++k)
    if (chunks[k] * kMatChunk < int64_t(mt.mats[k].rows) * mt.mats[k].cols ||
        (chunks[k] - 1) * kMatChunk >= int64_t(mt.mats[k].rows) * mt.mats[k].cols || chunks[k] != mt.mats[k].n_part)
      return bad("chunk count");
  std::set<std::tuple<int, int, int>> spread;
  for (const auto& j : mt.spread) spread.insert({j.mat, j.i, j.j});
  size_t want = 0;
  for (const auto& q : mt.mats) want += size_t(q.mp / kMatSpread) * (q.np / kMatSpread);
  if (spread.size() != want || mt.spread.size() != want) return bad("spread tiles");

  // byte ranges of the workspace
  std::vector<std::pair<int64_t, int64_t>> use;
  for (const auto& q : mt.mats) {
    const int64_t x = int64_t(2) * q.m * q.np, xt = int64_t(2) * q.n * q.mp, a = int64_t(2) * q.m * q.mp;
    for (auto r : {std::make_pair(q.xh, x), {q.xl, x}, {q.xt[0], xt}, {q.xt[1], xt}, {q.a, a}, {q.b, a},
                   {q.da, int64_t(4) * q.m}, {q.db, int64_t(4) * q.m}, {q.part, int64_t(8) * q.n_part}, {q.inv, int64_t(8)}})
      use.push_back({r.first, r.first + r.second});
    if (q.paired)
      for (auto r : {std::make_pair(q.c, a), {q.t, a}, {q.dc, int64_t(4) * q.m}, {q.dt, int64_t(4) * q.m}, {q.da2, int64_t(4) * q.m}})
        use.push_back({r.first, r.first + r.second});
    if (q.two_part)
      for (auto r : {std::make_pair(q.xtl[0], xt), {q.xtl[1], xt}, {q.al, a}, {q.bl, a}}) use.push_back({r.first, r.first + r.second});
  }
  int64_t slabs = 0;
  for (const auto& l : mt.list) slabs = std::max(slabs, int64_t(4) * l.side * l.side * l.slabs);
  use.push_back({mt.slabs, mt.slabs + slabs});
  std::sort(use.begin(), use.end());
  int64_t end = 0;
  for (auto& r : use) {
    if (r.first < end || r.first % 256) return bad("workspace overlap");
    end = std::max(end, r.second);
  }
  if (end > mt.work_bytes) return bad("workspace size");

  std::string text;
  for (int w = 0; w < kMatLists; ++w) {
    const ProductList& l = mt.list[w];
    const bool apply = w == kApply || w == kApplySingle;
    std::map<std::tuple<int, int, int>, std::vector<ProductJob>> tiles;
    std::vector<double> share(mat_places(l.side), 0.0);
    double total = 0;
    for (const ProductJob& p : l.jobs) {
      tiles[{p.mat, p.i, p.j}].push_back(p);
      const double s = (p.k1 - p.k0) * (mt.mats[p.mat].two_part ? 3 : 1);
      *std::min_element(share.begin(), share.end()) += s;
      total += s;
    }
    size_t need = 0, cut = 0;
    for (size_t k = 0; k < mt.mats.size(); ++k) {
      const MuonMat& q = mt.mats[k];
      if (w == kSquarePaired ? !q.paired : (w == kGramSingle || w == kApplySingle) && q.paired) continue;
      const int64_t ti = ceil_div(q.m, l.side), tj = apply ? ceil_div(q.n, l.side) : ti;
      need += apply ? ti * tj : ti * (ti + 1) / 2;
    }
    if (tiles.size() != need) return bad("tiles missing");
    std::map<std::tuple<int, int, int>, ProductJob> joins;
    for (const ProductJob& p : l.joins)
      if (!joins.insert({{p.mat, p.i, p.j}, p}).second) return bad("joined twice");
    std::vector<char> slab(l.slabs, 0);
    for (auto& [key, js] : tiles) {
      const MuonMat& q = mt.mats[std::get<0>(key)];
      const int i = std::get<1>(key), j = std::get<2>(key), steps = (w == kGram || w == kGramSingle ? q.np : q.mp) / kMatK;
      if (int64_t(i) * l.side >= q.m || int64_t(j) * l.side >= (apply ? q.n : q.m) || (!apply && j > i)) return bad("tile outside");
      std::sort(js.begin(), js.end(), [](const ProductJob& a, const ProductJob& b) { return a.k0 < b.k0; });
      int k = 0, number = 0;
      for (const ProductJob& p : js) {
        if (p.k0 != k || p.k1 <= p.k0 || p.parts != js.size()) return bad("steps");
        k = p.k1;
        if (p.parts > 1) {
          if (!joins.count(key) || joins[key].parts != js.size() || p.slab != joins[key].slab + number || p.slab < 0 ||
              p.slab >= l.slabs || slab[p.slab]++)
            return bad("slabs");
        }
        ++number;
      }
      if (k != steps) return bad("steps end");
      if (js.size() > 1) ++cut;
    }
    if (joins.size() != cut) return bad("joins");
    char line[200];
    std::snprintf(line, sizeof line, " [%d tiles of %d, %zu cut, %zu jobs, share %.2f, behind %.1f]", static_cast<int>(need), l.side, cut,
                  l.jobs.size(), total ? *std::max_element(share.begin(), share.end()) / (total / share.size()) : 1.0,
                  *std::max_element(share.begin(), share.end()) - total / share.size());
    text += line;
  }
  std::printf("ok%s\n", text.c_str());
  return 0;
}
