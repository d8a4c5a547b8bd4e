// The arithmetic by which attention work is shared out (attend_plan.cuh), on the CPU:
// closed forms against sums, and every unit's K/V tiles taken once by the CTAs' runs.
// Prints what does not hold; the exit status is 0 if all does.
#include <algorithm>
#include <cstdio>
#include <map>
#include <random>
#include <tuple>
#include <vector>

#include "attend_plan.cuh"

using namespace specv;

static long long failures = 0;
static void expect(bool ok, const char* what, long long a = 0, long long b = 0, long long c = 0) {
  if (!ok && ++failures <= 20) std::printf("%s: %lld %lld %lld\n", what, a, b, c);
}

static std::mt19937_64 rng(1);
static long long pick(long long lo, long long hi) {
  return lo + (long long)(rng() % (unsigned long long)(hi - lo + 1));
}

static void divisions() {
  std::vector<long long> ds = {1, 2, 3, 7, 24, 127, 128, 129, 65535, 65536, (1 << 30) - 1, 1 << 30};
  for (int i = 0; i < 300; ++i) ds.push_back(pick(1, 1LL << pick(1, 30)));
  for (long long d : ds) {
    const FastDiv f = fast_div((uint32_t)d);
    const long long top = 0x7fffffffLL, most = top / d;
    std::vector<long long> ks = {0, 1, 2, most - 1, most};
    for (int i = 0; i < 40; ++i) ks.push_back(pick(0, most));
    for (long long k : ks)
      for (long long n : {k * d - 1, k * d, k * d + 1, top})
        if (n >= 0 && n <= top) expect(f((uint32_t)n) == n / d, "quotient", n, d);
  }
  for (int i = 0; i < 3000; ++i) {
    const long long n = pick(0, 60), m = pick(1, 200), a = pick(0, 400), b = pick(0, 400);
    long long want = 0;
    for (long long j = 0; j < n; ++j) want += (a * j + b) / m;
    expect(floor_sum(n, m, a, b) == want, "floor_sum", n, m, a);
  }
}

static AttendSeq sequence(int row0) {
  const int n = (int)(pick(0, 2) == 0 ? pick(0, 4) : pick(0, 1) ? pick(0, 700) : pick(0, 5000));
  const int kind = (int)pick(0, 8);
  const int len = (int)(kind == 0 ? 0 : kind < 3 ? pick(0, n) : n + pick(0, 3000));
  return AttendSeq{row0, n, len};
}

static void costs() {
  for (int group = 1; group <= kTileRows; ++group) {
    const AttendShape sh = attend_shape(group);
    expect(sh.tpt == kTileRows / group && sh.w == 2 * sh.tpt, "shape", group);
    for (int i = 0; i < 12; ++i) {
      const AttendSeq s = sequence(0);
      long long sum = 0;
      for (int u = 0; u < sh.units(s); ++u) {
        expect(sh.cost_before(s, u) == sum, "cost_before", group, s.n, s.len);
        const int last = std::min((u + 1) * sh.w, s.n) - 1, key = s.len - s.n + last;
        expect(sh.unit_tiles(s, u) == (key < 0 ? 0 : key / kTileKeys + 1), "unit_tiles", group, u);
        sum += sh.unit_tiles(s, u) + kUnitCost;
      }
      expect(sh.head_cost(s) == sum, "head_cost", group, s.n, s.len);
    }
    // As many rows and positions as a call may have: steps of the same sum.
    for (int i = 0; i < 40; ++i) {
      const int n = (int)pick(1, 1 << 30);
      const AttendSeq s{0, n, (int)pick(0, 1) ? (int)pick(n, 1 << 30) : (int)pick(0, 1 << 30)};
      const int u = (int)pick(0, sh.units(s) - 1);
      expect(sh.cost_before(s, u + 1) - sh.cost_before(s, u) == sh.unit_tiles(s, u) + kUnitCost,
             "step", group, s.n, s.len);
    }
  }
}

// The runs of all CTAs, as the kernel finds and walks them.
static void runs() {
  for (int trial = 0; trial < 1500; ++trial) {
    const int group = (int)(trial % 7 ? pick(1, 16) : pick(1, kTileRows));
    const int heads = (int)pick(1, 4), B = (int)pick(1, 6);
    const AttendShape sh = attend_shape(group);
    std::vector<AttendSeq> seqs;
    std::vector<long long> cost;
    long long total = 0;
    for (int b = 0, row = 0; b < B; ++b) {
      seqs.push_back(sequence(row));
      if (pick(0, 4) == 0) seqs[b].n = 0;
      row += seqs[b].n;
      cost.push_back(sh.head_cost(seqs[b]) * heads);
      total += cost[b];
    }
    const int ctas = (int)(trial % 3 ? 148 : pick(1, 150));
    const long long share = (total + ctas - 1) / ctas;
    auto seq = [&](int b) { return seqs[b]; };
    struct Part {
      int cta, t0, t1, head, parts;
    };
    std::map<std::tuple<int, int, int>, std::vector<Part>> units;
    for (int cta = 0; cta < ctas; ++cta) {
      const long long from = share * cta, to = std::min(total, from + share);
      if (from >= to) continue;
      int b = 0;
      long long at = 0;
      while (at + cost[b] <= from) at += cost[b++];
      const long long head = sh.head_cost(seqs[b]);
      const int h = (int)((from - at) / head);
      const long long y = (from - at) % head;
      int u = 0;
      while (u + 1 < sh.units(seqs[b]) && sh.cost_before(seqs[b], u + 1) <= y) ++u;
      AttendCursor<decltype(seq)> cur(sh, seq, B, heads, b, h, u,
                                      (int)(y - sh.cost_before(seqs[b], u)), to - from, seqs[b]);
      std::vector<AttendPiece> pieces;
      for (AttendPiece x; cur.next(&x);) pieces.push_back(x);
      for (size_t i = 0; i < pieces.size(); ++i) {
        const AttendPiece& x = pieces[i];
        Part p{cta, x.t0, x.t1, cta, 1};
        if (x.t0 > 0 || x.t1 < x.nt) {
          expect(x.t0 == 0 || i == 0, "a later part begins a run", cta);
          expect(x.t1 == x.nt || i + 1 == pieces.size(), "a first part ends a run", cta);
          const long long unit = x.t0 > 0 ? from - x.t0 : to - x.t1;
          p.head = (int)(unit / share);
          p.parts = (int)((unit + x.nt - 1) / share) - p.head + 1;
        }
        expect(x.nt == sh.unit_tiles(x.s, x.u) && x.tok0 == x.u * sh.w &&
                   x.ntok == std::min(sh.w, x.s.n - x.tok0) && x.ntok > 0,
               "piece", x.b, x.u, x.nt);
        units[{x.b, x.h, x.u}].push_back(p);
      }
    }
    for (int b = 0; b < B; ++b)
      for (int h = 0; h < heads; ++h)
        for (int u = 0; u < sh.units(seqs[b]); ++u) {
          const auto it = units.find({b, h, u});
          expect(it != units.end(), "a unit is taken", b, h, u);
          if (it == units.end()) continue;
          int t = 0;
          const auto& parts = it->second;
          for (size_t i = 0; i < parts.size(); ++i) {
            expect(parts[i].t0 == t, "tiles in order", b, u, t);
            expect(parts[i].head == parts[0].cta && parts[i].cta == parts[0].cta + (int)i &&
                       parts[i].parts == (int)parts.size(),
                   "head and count of parts", b, u, (long long)i);
            t = parts[i].t1;
          }
          expect(t == sh.unit_tiles(seqs[b], u), "all tiles", b, u, t);
          units.erase(it);
        }
    expect(units.empty(), "units that are there", trial);
  }
}

int main() {
  divisions();
  costs();
  runs();
  if (failures) std::printf("%lld failures\n", failures);
  return failures != 0;
}
