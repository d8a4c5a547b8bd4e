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
// their number plus kUnitCost (prologue and epilogue). The costs of all units in
// (sequence, head, unit) order form one line, cut into equal runs, one per
// CTA: a unit that a cut divides leaves partial results to be combined. So
// few rows over many keys are split over the GPU by the same rule that shares
// out many ragged prompts, without a choice between kernels.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define SPECV_HD __host__ __device__ __forceinline__
#define SPECV_HD_CALL __host__ __device__ __noinline__
#else
#define SPECV_HD inline
#define SPECV_HD_CALL inline
#endif

namespace specv {

constexpr int kTileRows = 128;  // query rows of a tile
constexpr int kTileKeys = 128;  // keys of a K/V tile
// A unit's fixed cost, in K/V tiles: what its first loads, the filling of the
// pipeline and its output take. Measured with 2, 3, 4: 8192 rows 462, 466, 471 us;
// 16 ragged prompts 345, 348, 358; four chunks 175 each; one row over 65000 keys 56, 54,
// 53. So long prompts would gain 1 % with 2, and a step of decoding over a long cache
// lose 4 %.
constexpr int kUnitCost = 3;

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

// Division by a fixed d >= 1 of n < 2^31: n / d = (n * mul) >> (31 + bits), bits =
// ceil(log2 d), mul = floor(2^(31+bits) / d) + 1 < 2^32 (Granlund and Montgomery,
// "Division by invariant integers using multiplication", PLDI 1994).
struct FastDiv {
  uint32_t d, mul;
  int bits;
  SPECV_HD uint32_t operator()(uint32_t n) const {
    return (uint32_t)(((unsigned long long)n * mul) >> (31 + bits));
  }
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  while ((1u << f.bits) < d) ++f.bits;
  f.mul = (uint32_t)((1ull << (31 + f.bits)) / d + 1);
  return f;
}

struct AttendShape {
  int tpt;     // tokens of a tile
  int w;       // tokens of a unit, 2 * tpt
  int log_w;   // log2 of w, -1 where it is no power of two
  FastDiv by_w;

  SPECV_HD int units(const AttendSeq& s) const { return (int)by_w((uint32_t)(s.n + w - 1)); }
  // K/V tiles that rows up to token `last` need.
  SPECV_HD int tiles_upto(const AttendSeq& s, int last) const {
    const int key = s.len - s.n + last;
    return key < 0 ? 0 : key / kTileKeys + 1;
  }
  SPECV_HD int unit_tiles(const AttendSeq& s, int u) const {
    const int end = (u + 1) * w;
    return tiles_upto(s, (end < s.n ? end : s.n) - 1);
  }
  // sum_{j<x} floor(j / 2^r)
  SPECV_HD static long long step_sum(long long x, int r) {
    const long long t = x >> r;
    return ((t * (t - 1) / 2) << r) + t * (x - (t << r));
  }
  // sum_{i<m} floor((b + i*w) / 128), b >= 0: closed where w is a power of two.
  SPECV_HD long long tile_sum(long long m, int b) const {
    if (log_w < 0) return floor_sum(m, kTileKeys, w, b);
    if (log_w >= 7) return m * (b >> 7) + (m * (m - 1) / 2 << (log_w - 7));
    const int s = (b & 127) >> log_w;  // floor((b + i*w) / 128) = b>>7 + floor((s + i) / (128/w))
    return m * (b >> 7) + step_sum(m + s, 7 - log_w) - step_sum(s, 7 - log_w);
  }
  // Cost of units 0 .. u-1.
  SPECV_HD_CALL long long cost_before(const AttendSeq& s, int u) const {
    const int all = units(s);
    long long c = (long long)u * kUnitCost;
    int full = u;  // units whose last token is (i + 1) * w - 1
    if (u == all && u > 0) {
      c += unit_tiles(s, u - 1);
      --full;
    }
    // sum_{i=1}^{full} of floor((base + i*w - 1) / 128) + 1 where that is >= 0
    const int base = s.len - s.n;
    int skip = 0;  // units whose rows see nothing
    if (base < 0) {
      skip = (-base) / w;  // base + i*w - 1 < 0 for i <= skip
      if (skip > full) skip = full;
    }
    const long long m = full - skip;
    if (m > 0) c += m + tile_sum(m, base + (skip + 1) * w - 1);
    return c;
  }
  SPECV_HD long long head_cost(const AttendSeq& s) const { return cost_before(s, units(s)); }
};
inline AttendShape attend_shape(int group) {
  AttendShape s;
  s.tpt = kTileRows / group;
  s.w = 2 * s.tpt;
  s.log_w = -1;
  for (int i = 1; i <= 8; ++i)
    if (s.w == 1 << i) s.log_w = i;
  s.by_w = fast_div((uint32_t)s.w);
  return s;
}

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
  const AttendShape& sh;
  SeqFn seq;
  int B, heads;
  int b, h, u;
  int x;           // cost already taken of unit u
  long long left;  // cost left in the run
  AttendSeq s;

  SPECV_HD AttendCursor(const AttendShape& shape, SeqFn fn, int nseq, int nheads, int b_, int h_,
                        int u_, int x_, long long left_, const AttendSeq& s_)
      : sh(shape), seq(fn), B(nseq), heads(nheads), b(b_), h(h_), u(u_), x(x_), left(left_), s(s_) {
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
      p->tok0 = u * sh.w;
      const int rest = s.n - p->tok0;
      p->ntok = rest < sh.w ? rest : sh.w;
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
      if (p->t0 < p->t1 || (nt == 0 && x0 == 0)) return true;
    }
    return false;
  }
};

}  // namespace specv
