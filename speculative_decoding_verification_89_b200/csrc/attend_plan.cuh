// How attention work is cut up and shared out: host and device code without
// any launch, so the arithmetic can be checked on a CPU.
//
// A unit is a run of consecutive query rows (tokens) of one sequence under one
// K/V head. The group of G query heads that share the head are packed into
// the 128-row tiles of the matrix instructions: row r of a tile is token
// r / G, query head h*G + r % G, so a tile holds TPT = 128 / G whole tokens and
// a K/V tile is read once for all G heads. A sequence's units hold 2*TPT
// tokens (two tiles that share each K/V tile); a unit of at most TPT tokens
// has one tile, and its K/V tiles go to the two accumulators in turn.
//
// Row i of a sequence with n new rows and `len` keys sees keys 0 .. len-n+i, so
// a unit needs the K/V tiles (128 keys) up to its last row's. Its cost is
// their number plus one (prologue and epilogue). The costs of all units in
// (sequence, head, unit) order form one line, cut into equal runs, one per
// CTA: a unit that a cut divides leaves partial results to be combined.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define SPECV_HD __host__ __device__ __forceinline__
#else
#define SPECV_HD inline
#endif

namespace specv {

constexpr int kTileRows = 128;  // query rows of a tile
constexpr int kTileKeys = 128;  // keys of a K/V tile
constexpr int kUnitCost = 1;    // a unit's fixed cost, in K/V tiles

// sum_{i=0}^{n-1} floor((a*i + b) / m) for n, a, b >= 0, m > 0: the lattice
// points under a line, by Euclid's algorithm on (a, m).
SPECV_HD long long floor_sum(long long n, long long m, long long a, long long b) {
  long long ans = 0;
  while (n > 0) {
    ans += (n - 1) * n / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const long long top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top % m;
    const long long t = m;
    m = a;
    a = t;
  }
  return ans;
}

// One sequence: its n new rows start at packed row row0 and see up to len keys.
struct AttendSeq {
  int row0, n, len;
};

struct AttendShape {
  int tpt;  // tokens of a tile
  SPECV_HD int units(const AttendSeq& s) const { return (s.n + 2 * tpt - 1) / (2 * tpt); }
  // K/V tiles that rows up to token `last` need.
  SPECV_HD int tiles_upto(const AttendSeq& s, int last) const {
    const int key = s.len - s.n + last;
    return key < 0 ? 0 : key / kTileKeys + 1;
  }
  SPECV_HD int unit_tiles(const AttendSeq& s, int u) const {
    const int end = (u + 1) * 2 * tpt;
    return tiles_upto(s, (end < s.n ? end : s.n) - 1);
  }
  // Cost of units 0 .. u-1.
  SPECV_HD long long cost_before(const AttendSeq& s, int u) const {
    const int all = units(s);
    long long c = (long long)u * kUnitCost;
    int full = u;  // units whose last token is (i + 1) * 2 * tpt - 1
    if (u == all && u > 0) {
      c += unit_tiles(s, u - 1);
      --full;
    }
    // sum_{i=1}^{full} of floor((base + i*w - 1) / 128) + 1 where that is >= 0
    const int w = 2 * tpt, base = s.len - s.n;
    int skip = 0;  // units whose rows see nothing
    if (base < 0) {
      skip = (-base) / w;  // base + i*w - 1 < 0 for i <= skip
      if (skip > full) skip = full;
    }
    const long long m = full - skip;
    if (m > 0)
      c += m + floor_sum(m, kTileKeys, w, (long long)base + (long long)(skip + 1) * w - 1);
    return c;
  }
  SPECV_HD long long head_cost(const AttendSeq& s) const { return cost_before(s, units(s)); }
};

// A CTA's share of one unit: K/V tiles [t0, t1) of the unit's nt.
struct AttendPiece {
  AttendSeq s;
  int b, h, u;
  int t0, t1, nt;
  int tok0, ntok;  // the unit's tokens within the sequence
};

// Walks a CTA's run of the cost line. `seq(b)` gives sequence b.
template <typename SeqFn>
struct AttendCursor {
  AttendShape sh;
  SeqFn seq;
  int B, heads;
  int b, h, u;
  int x;           // cost already taken of unit u
  long long left;  // cost left in the run
  AttendSeq s;

  SPECV_HD AttendCursor(AttendShape shape, SeqFn fn, int nseq, int nheads, int b_, int h_, int u_,
                        int x_, long long left_)
      : sh(shape), seq(fn), B(nseq), heads(nheads), b(b_), h(h_), u(u_), x(x_), left(left_) {
    if (left > 0) s = seq(b);
  }
  SPECV_HD bool next(AttendPiece* p) {
    while (left > 0) {
      const int nt = sh.unit_tiles(s, u), cost = nt + kUnitCost;
      const int x0 = x;
      const int take = left < (long long)(cost - x) ? (int)left : cost - x;
      x += take;
      left -= take;
      p->s = s;
      p->b = b;
      p->h = h;
      p->u = u;
      p->nt = nt;
      p->t0 = x0 < nt ? x0 : nt;
      p->t1 = x < nt ? x : nt;
      p->tok0 = u * 2 * sh.tpt;
      const int rest = s.n - p->tok0;
      p->ntok = rest < 2 * sh.tpt ? rest : 2 * sh.tpt;
      if (x == cost) {
        x = 0;
        if (++u == sh.units(s)) {
          u = 0;
          if (++h == heads) {
            h = 0;
            do {
              ++b;
              if (b < B) s = seq(b);
            } while (b < B && s.n == 0);
            if (b >= B) left = 0;
          }
        }
      }
      if (p->t0 < p->t1 || nt == 0) return true;
    }
    return false;
  }
};

}  // namespace specv
