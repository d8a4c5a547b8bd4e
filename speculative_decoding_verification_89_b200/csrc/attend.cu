// Attention of packed query rows over packed or paged keys and values:
//   o_i = sum_{j <= len-n+i} p_ij v_j,  p_ij = softmax_j(scale * q_i . k_j)
// in one pass over the keys: with a running reference m and sum l,
//   p~ = 2^(c s - m),  l += sum p~,  O += P~ V,  o = O / l,
// c = scale * log2(e). The reference need not be the running maximum: it is
// raised (and l, O scaled down) only when a maximum passes it by more than
// kSlack, to kHead below that maximum, so p~ stays within 2^kSlack and the scaling
// of O is rare. Scores, m, l, O and parts of divided units are float32. p~ is
// rounded to the inputs' type for the second product, as the matrix instruction
// takes one type for both operands: half a step of a weight, and for fp16 no
// more than 2^-25 of a p~ (2^-32 of the row's largest) where it is subnormal,
// which is why the reference lies kHead below the maximum; l sums the
// unrounded p~. Outputs are rounded once more, to the type of out.
//
// HiSpec (gist.science summary of arXiv 2510.01336), section 2
// "Unterstuetzung fuer Batch-Inferenz" (paged attention with block tables) and
// "Wiederverwendung von KV-Cache und versteckten Zustaenden" (K/V rows staged
// while drafting, kept or dropped by the check).
//
// One persistent CTA per SM takes a run of K/V tiles (attend_plan.cuh). Of its
// three warpgroups the first two are softmax warps, one thread per row of a
// 128-row tile; in the third, one thread issues the matrix instructions
// (tcgen05, accumulators in tensor memory) and three warps load. Scores S =
// Q K^T of a tile land in tensor memory; its warpgroup turns them into P~ in
// place (two-byte elements over the same columns), which the next instruction
// reads as its left operand for O += P~ V. While one warpgroup works on its
// scores, the tensor cores form the other's.
//
// Times on the device, 32 query and 8 K/V heads of 128, bf16, of calls a few at a time; in
// brackets in a loop of calls for seconds, where power holds the clock down. 8192 rows:
// 472 us (555), 1165 TFLOP/s (332 us at the measured 1656): a K/V tile with two query tiles takes
// about 3500 cycles where the products alone need 2048 and the exponentials, 16 a
// cycle, 2048; maximum, scaling, rounding and the hand-over between the two make
// up the rest. 64 sequences of 9 staged rows over 512 to 4096 keys 114 to 129 us by the
// card (137), one row over 65000 keys 53 to 57 (57): 4.5 to 5.1 TB/s both (89 and 41 us
// at the measured 6.55 TB/s), bound by HBM and the gaps between units. 8192 rows of
// heads of 64: 415 us, bound by exponentials alone. One row over 700 keys 13 us:
// launch, plan, first instruction fetches and join, one after the other.
#include <cuda_fp16.h>

#include <type_traits>

#include "attend.cuh"
#include "kernels.cuh"
#include "tc05.cuh"

namespace specv {

namespace {

constexpr int kThreads = 384;
constexpr int kLoaders = 96;      // warps 9-11
constexpr int kTmemCols = 512;    // S0 S1 O0 O1
constexpr float kSlack = 15.0f;   // log2 of the largest p~ (fp16 ends at 65504)
constexpr float kHead = 7.0f;     // log2 of the largest p~ under a new reference

// Buffers of one 128-row tile (Q, K or V) each; all of them serve all three.
template <int DP>
struct Tile {
  static constexpr int kBytes = 128 * DP * 2;
  static constexpr int kCount = DP == 128 ? 7 : 8;
  static constexpr int kSmemTiles = kCount * kBytes;
};

// A piece as the scheduling warp (the third loading warp) passes it to the others.
struct Msg {
  AttendSeq s;
  int b, h;
  int t0, m;         // first K/V tile and number of tiles
  int tok0, ntok;    // the unit's tokens within the sequence
  int c0, c1;        // tiles of each accumulator
  int two;           // two query tiles
  int part;          // 0 whole, 1 a later part of its unit, 2 the first of several
  int head, parts;   // (parts) the CTA that has the first one, how many there are
  int end;           // no piece: the run is over
};
constexpr int kMsgs = 4;

struct Shared {
  uint64_t msg_full[kMsgs], msg_empty[kMsgs];
  uint64_t full[8], empty[8], landed[8];
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];
  uint64_t swap, drain;
  uint64_t parted, ticketed;
  uint32_t tmem;
  long long warp_sum[kThreads / 32];
  AttendSeq seq;      // the first unit's sequence
  int start[4];       // sequence, head, unit, cost taken of it
  long long from, run, share;  // start and cost of this CTA's run, cost of a full one
  int last;           // this CTA wrote the last part of a unit
  int counted;        // divided pieces of this CTA's run that are counted
  int failed;         // a wait ran out
  int odd;            // an output is NaN
  int joined;         // divided units joined here: 1 that of the first piece, 2 of the last
  Msg msg[kMsgs];
  float2 ml[2][kTileRows];
};
static_assert(Tile<128>::kSmemTiles + sizeof(Shared) <= 227 * 1024, "shared memory");

// A wait on a barrier phase, bounded by kWaitCycles of the SM's clock (2 s at
// 1.9 GHz; cheaper to read than the global timer). In assembly to stay a few
// instructions long: it is in many places. A role whose wait runs out ends; the
// others' waits then run out too.
constexpr long long kWaitCycles = 3800000000ll;
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t"
      ".reg .pred p, q;\n\t"
      ".reg .b64 t, u;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "mov.u64 t, %%clock64;\n\t"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "mov.u64 u, %%clock64;\n\t"
      "sub.s64 u, u, t;\n\t"
      "setp.lt.s64 q, u, %3;\n\t"
      "@q bra AGAIN;\n\t"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "l"(kWaitCycles)
      : "memory");
  return ok != 0;
}

// Sequence b, with what is invalid made empty.
struct SeqOf {
  const AttendArgs* a;
  __device__ AttendSeq operator()(int b) const { return get(b, nullptr); }
  __device__ AttendSeq get(int b, int* bad) const {
    AttendSeq s;
    if (a->row_off) {
      const int lo = a->row_off[b], hi = a->row_off[b + 1];
      s.row0 = lo;
      s.n = hi - lo;
      if (lo < 0 || hi < lo || hi > a->T) {
        s.row0 = s.n = 0;
        if (bad) *bad = 1;
      }
    } else {
      s.row0 = b * a->rows_per_seq;
      s.n = a->rows_per_seq;
    }
    if (!a->tables) {
      s.len = s.n;
      return s;
    }
    s.len = a->seq_lens[b];
    if (s.len < 0 || s.len > a->max_blocks * a->block_size || (a->stage_k && s.n > a->stage_rows)) {
      s.len = 0;
      if (bad) *bad = 1;
    } else if (a->stage_k) {
      s.len += s.n;
    }
    return s;
  }
};

using Cursor = AttendCursor<SeqOf>;

// a / b where it mostly fits 32 bits
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// The cost of a sequence under one head; of one unit without the general sum.
__device__ __forceinline__ long long cost_of_head(const AttendShape& shape, const AttendSeq& s) {
  if (s.n <= 0) return 0;
  return s.n <= shape.w ? shape.tiles_upto(s, s.n - 1) + kUnitCost : shape.head_cost(s);
}

// Where this CTA's run of the cost line starts, into sh; all threads.
__device__ __forceinline__ void find_run(const AttendArgs& a, Shared* sh) {
  const SeqOf seq{&a};
  const AttendShape& shape = a.shape;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  long long sum = 0;
  int bad = 0;
  for (int b = b0; b < b1; ++b) {
    const AttendSeq s = seq.get(b, &bad);
    sum += cost_of_head(shape, s) * a.kv_heads;
  }
  if (bad && blockIdx.x == 0) set_status(a.status, SPEC_EDEVICE);
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sh->warp_sum[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sh->warp_sum[w];
    total += sh->warp_sum[w];
  }
  const long long share = quotient(total + gridDim.x - 1, gridDim.x);
  const long long from = share * blockIdx.x;
  const long long to = min(total, from + share);
  long long at = before + incl - sum;
  if (from < to && from >= at && from < at + sum) {
    for (int b = b0; b < b1; ++b) {
      const AttendSeq s = seq(b);
      const long long head = cost_of_head(shape, s);
      if (from < at + head * a.kv_heads) {
        const int h = (int)quotient(from - at, head);
        const long long y = from - at - h * head;
        int lo = 0, hi = shape.units(s) - 1;  // the unit u with cost_before(u) <= y
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (shape.cost_before(s, mid) <= y) lo = mid; else hi = mid - 1;
        }
        sh->seq = s;
        sh->start[0] = b;
        sh->start[1] = h;
        sh->start[2] = lo;
        sh->start[3] = (int)(lo ? y - shape.cost_before(s, lo) : y);
        sh->run = to - from;
        sh->from = from;
        sh->share = share;
        break;
      }
      at += head * a.kv_heads;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ Cursor cursor(const AttendArgs& a, const Shared* sh) {
  return Cursor(a.shape, SeqOf{&a}, a.B, a.kv_heads, sh->start[0], sh->start[1], sh->start[2],
                sh->start[3], sh->run, sh->seq);
}

// Of a divided piece's unit: the CTA that has its first part, and how many parts.
// The unit's place on the cost line: a later part begins with the run, a first one
// ends with it.
__device__ __forceinline__ long long unit_from(const Shared* sh, const AttendPiece& x) {
  return x.t0 > 0 ? sh->from - x.t0 : sh->from + sh->run - x.t1;
}
__device__ __forceinline__ int unit_head(const Shared* sh, const AttendPiece& x) {
  return (int)quotient(unit_from(sh, x), sh->share);
}
__device__ __forceinline__ int unit_parts(const Shared* sh, const AttendPiece& x, int head) {
  return (int)quotient(unit_from(sh, x) + x.nt - 1, sh->share) - head + 1;
}
// Counts a part of the unit that CTA `head` begins; whether it was the last one, which
// leaves the count at zero for the next call.
__device__ __forceinline__ bool count_part(const AttendArgs& a, int head, int parts) {
  int n;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
               : "=r"(n)
               : "l"(a.counts + head)
               : "memory");
  const bool last = n == parts - 1;
  if (last) a.counts[head] = 0;
  return last;
}
// Counts the divided pieces that a CTA did not get to, so that the counts return to
// zero also in a call whose waits ran out. One thread, after all roles.
__device__ __forceinline__ void count_rest(const AttendArgs& a, Shared* sh) {
  Cursor cur = cursor(a, sh);
  AttendPiece x;
  for (int i = 0; cur.next(&x);) {
    if (x.t0 == 0 && x.t1 == x.nt) continue;
    const int head = unit_head(sh, x);
    if (i++ >= sh->counted) count_part(a, head, unit_parts(sh, x, head));
  }
}

// The free buffers, in the order in which they will be given back: a queue of
// 4-bit numbers, the next one lowest. The loading and the issuing warps step
// through one program of takes and gives, so each n-th take gets the same
// buffer on both sides; the barriers' phases follow from each buffer's uses.
template <int N>
struct Buffers {
  uint32_t queue, end;  // end: bit position behind the last one
  uint32_t phases;      // bit b: parity of buffer b's next use
  __device__ Buffers() : queue(0), end(4 * N), phases(0) {
#pragma unroll
    for (int i = 0; i < N; ++i) queue |= (uint32_t)i << (4 * i);
  }
  __device__ __forceinline__ int take(uint32_t* parity) {
    const int b = (int)(queue & 15);
    queue >>= 4;
    end -= 4;
    *parity = (phases >> b) & 1;
    phases ^= 1u << b;
    return b;
  }
  __device__ __forceinline__ void give(int b) {
    queue |= (uint32_t)b << end;
    end += 4;
  }
};

// One lane of a warp, the same for every call by the whole warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// A role's place in the ring of messages. `read` copies the next one; the caller
// then gives its slot back (one arrival per softmax warp, issuer and copying warp).
struct MsgRing {
  int i = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void step() {
    if (++i == kMsgs) {
      i = 0;
      ph ^= 1;
    }
  }
};

// Tiles of a unit that its first 128-row tile needs (two-tile units).
__device__ __forceinline__ int first_tile_count(const AttendShape& shape, const AttendPiece& p) {
  const int nt0 = shape.tiles_upto(p.s, p.tok0 + shape.tpt - 1);
  return max(0, min(p.t1, nt0) - p.t0);
}

// The program of a piece. Two query tiles: both use each K
// and V tile, the first may need fewer of them; K tiles are one ahead of the V
// tiles. One query tile: the K/V tiles go to the two accumulators in turn, K
// two ahead. Side:
//   take_q(w), take_k(t), take_v(t): the next buffer, for query tile w, K or V
//     tile t; give_q(w), give_k(), give_v(): it is free once what was issued is done;
//   qk(w, x): scores of accumulator w with query tile x; pv(w, first, last):
//     weights times V.
// Every step is written once: the code of both sides has to stay small enough
// for the instruction cache beside the softmax warps' (unrolled by case all kernels
// were 376 KB: 64 x 9 rows took 170 us, at 100 KB 138, before later steps).
// (The loading warps' side is Loader::fill: the same takes and gives in the
// same order, with one place that loads.)
template <typename Side>
__device__ __forceinline__ bool piece_program(int m, bool two, int c0, Side& side) {
  if (m == 0) return true;  // rows that see nothing
  if (!side.take_q(0)) return false;
  if (two) {
    if (!side.take_q(1)) return false;
#pragma unroll 1
    for (int i = -1; i < m; ++i) {
      const bool more = i + 1 < m;
      if (i >= 0) {
        if (!side.take_v(i)) return false;
        if (i < c0 && !side.pv(0, i == 0, i + 1 == c0)) return false;
      }
      if (more) {
        if (!side.take_k(i + 1)) return false;
        if (i + 1 < c0) side.qk(0, 0);
        if (i + 1 == max(c0 - 1, 0)) side.give_q(0);
      }
      if (i >= 0) {
        if (!side.pv(1, i == 0, !more)) return false;
        side.give_v();
      }
      if (more) {
        side.qk(1, 1);
        if (i + 2 == m) side.give_q(1);
        side.give_k();
      }
    }
  } else {
#pragma unroll 1
    for (int i = -2; i < m; ++i) {
      const int w = i & 1;
      if (i >= 0) {
        if (!side.take_v(i) || !side.pv(w, i < 2, i + 2 >= m)) return false;
        side.give_v();
      }
      if (i + 2 < m) {
        if (!side.take_k(i + 2)) return false;
        side.qk(w, 0);
        if (i + 3 == m) side.give_q(0);
        side.give_k();
      }
    }
  }
  return true;
}

// ---------------------------------------------------------------------------
// Loading: query rows, then K and V tiles in the order they are used
// ---------------------------------------------------------------------------
// Warp 9 copies columns 0-63 and warp 10 columns 64-127 of each tile with tiled
// (TMA) copies: one for a query tile or 128 packed rows, one per page or part of a
// page for the pool (row by row, as it was first, 8192 rows took 1266 us, with tiled
// copies 796, before later steps). Warp 11 puts right what the copies of a sequence's last tiles cannot:
// V rows past the keys are set to zero (what lies there must not reach a
// product: a weight of 0 times a NaN) and staged rows are put in their place.
// A tile is full when all three warps have arrived. Pages whose rows are no
// multiple of 8 are copied row by row by all three.
template <int DP, bool kMends>
struct Loader {
  static constexpr int kChunks = DP / 8;   // 16-byte chunks of a row
  const AttendArgs& a;
  Shared* sh;
  uint32_t tiles;     // shared address of the tiles
  int role, lane;     // 0-2: columns 0-63, columns 64-127, mending
  Buffers<Tile<DP>::kCount> buf;
  Msg p;
  int pooled;         // keys of the sequence in the pool (or packed rows)
  int q_buf[2];
  uint32_t issued;    // buffers filled at least once, by bit
  uint32_t land_ph;   // parity of each buffer's next use of `landed`
  // Table entries of 32 consecutive pages, one per lane: the group that the K
  // tiles have reached, the one before (V tiles follow) and the next one.
  int group, cur, prev, next;
  uint64_t policy;

  __device__ Loader(const AttendArgs& a_, Shared* s, uint32_t t, int thread)
      : a(a_), sh(s), tiles(t), role(thread >> 5), lane(thread & 31), issued(0), land_ph(0) {}
  __device__ bool wait(uint64_t* bar, uint32_t ph) {
    return __all_sync(0xffffffffu, wait_bar(bar, ph));
  }
  // The copies in flight land before the CTA ends, also after a wait that ran out.
  __device__ void drain() {
#pragma unroll 1
    for (int b = 0; b < Tile<DP>::kCount; ++b)
      if (issued >> b & 1) wait_bar(&sh->full[b], ((buf.phases >> b) & 1) ^ 1);
  }
  __device__ bool take(int* b) {
    uint32_t ph;
    *b = buf.take(&ph);
    if (!wait(&sh->empty[*b], ph ^ 1)) {
      buf.phases ^= 1u << *b;  // not filled
      return false;
    }
    issued |= 1u << *b;
    return true;
  }
  __device__ uint32_t tile(int b) const { return tiles + b * Tile<DP>::kBytes; }
  __device__ int entry(int page) const {
    return page < a.max_blocks ? a.tables[(long long)p.b * a.max_blocks + page] : 0;
  }
  __device__ int page_of(int key) const { return (int)a.by_bs((uint32_t)key); }
  __device__ bool copies() const { return role == 0 || (role == 1 && a.dim > 64); }
  __device__ void begin() {
    pooled = a.stage_k ? p.s.len - p.s.n : p.s.len;
    if (kMends || !a.tables || !a.box_rows || p.m == 0) return;
    // K/V that one unit reads go first when the L2 needs room: streamed through it,
    // they would push out the instructions (64 x 9 rows: 117 us, 128 without).
    policy = p.two ? l2_evict_normal() : l2_evict_first();
    group = page_of(p.t0 * kTileKeys) >> 5;
    cur = entry(group * 32 + lane);
    next = entry(group * 32 + 32 + lane);
    prev = 0;
  }
  // This warp's columns of query tile w: rows (token, head of the group).
  __device__ bool take_q(int w) {
    int b;
    if (!take(&b)) return false;
    if (w) q_buf[1] = b; else q_buf[0] = b;
    uint64_t* bar = &sh->full[b];
    const int tok0 = p.s.row0 + p.tok0 + w * a.shape.tpt;
    const uint32_t bytes = a.shape.tpt * a.group * 128;
    const uint32_t dst = tile(b) + role * (128 * 128);
    if (elect_one()) {
      if (!kMends && copies()) {
        mbar_arrive_expect_tx(bar, bytes);
        tma_box4_hint(dst, &a.map_q, role * 64, 0, p.h, tok0, bar, l2_evict_first());  // read once
      } else {
        mbar_arrive(bar);
      }
    }
    return true;
  }
  // K (v = 0) or V (v = 1) rows of tile t of the piece's sequence.
  __device__ bool load_kv(int t, int v, int b) {
    if (!a.box_rows) {
      load_rows(t, v, tile(b));
      if (elect_one()) mbar_arrive(&sh->full[b]);
      return true;
    }
    const bool mend = (t + 1) * kTileKeys > pooled && (v || a.stage_k);
    uint64_t* bar = mend ? &sh->landed[b] : &sh->full[b];
    if constexpr (kMends) {
      if (mend) {
        if (!mend_tile(t, v, b)) return false;
      } else if (elect_one()) {
        mbar_arrive(&sh->full[b]);
      }
    } else if (copies()) {
      if (elect_one()) {
        mbar_arrive_expect_tx(bar, 128 * 128);
        if (mend) mbar_arrive(&sh->full[b]);
      }
      load_boxes(t, v, tile(b) + role * (128 * 128), bar);
    } else if (elect_one()) {
      if (mend) mbar_arrive(&sh->landed[b]);
      mbar_arrive(&sh->full[b]);
    }
    if (mend) land_ph ^= 1u << b;
    return true;
  }
  // Boxes [i0, i0 + kBoxes) of a tile; lane at + i has the block of box i and, unless
  // boxes are whole pages, its first row there. The numbers first, then all
  // copies in a row: one at a time, each behind its own election, pages of 32
  // rows cost 133 us where pages of 16 took 119 (64 x 9 rows).
  template <int kBoxes, bool kWhole>
  __device__ void page_boxes(const void* map, uint32_t dst, int i0, int at, int block, int row,
                             uint64_t* bar) {
    int blocks[kBoxes], rows[kBoxes];
#pragma unroll
    for (int i = 0; i < kBoxes; ++i) {
      blocks[i] = __shfl_sync(0xffffffffu, block, at + i);
      rows[i] = kWhole ? 0 : __shfl_sync(0xffffffffu, row, at + i);
    }
    if (elect_one()) {
#pragma unroll
      for (int i = 0; i < kBoxes; ++i)
        tma_box4_hint(dst + (i0 + i) * a.box_rows * 128, map, role * 64, p.h, rows[i], blocks[i],
                      bar, policy);
    }
  }
  __device__ void load_boxes(int t, int v, uint32_t dst, uint64_t* bar) {
    const void* map = v ? &a.map_v : &a.map_k;
    if (!a.tables) {
      if (elect_one()) tma_box3(dst, map, role * 64, p.h, p.s.row0 + t * kTileKeys, bar);
      return;
    }
    const int page = page_of(t * kTileKeys), g = page >> 5;  // a group holds whole tiles
    if (!v && g != group) {
      prev = cur;
      cur = next;
      group = g;
      next = entry(g * 32 + 32 + lane);
    }
    int id = g == group ? cur : prev;
    const bool held = (g * 32 + lane) * (long long)a.block_size < pooled;
    if (!held || id < 0 || id >= a.num_blocks) {
      const int pages = page_of(t * kTileKeys + kTileKeys - 1) - page + 1;
      if (held && (unsigned)(lane - (page & 31)) < (unsigned)pages)
        set_status(a.status, SPEC_EDEVICE);
      id = a.num_blocks;  // outside the tensor: zeros
    }
    const int boxes = kTileKeys / a.box_rows;
    if (a.block_size == kTileKeys / 8) {  // pages of 16 rows, without the general form's
      page_boxes<8, true>(map, dst, 0, page & 31, id, 0, bar);  // shuffles (119 us; 124 with)
      return;
    }
    const int key = t * kTileKeys + min(lane, boxes - 1) * a.box_rows, mine = page_of(key);
    id = __shfl_sync(0xffffffffu, id, mine & 31);
    const int row = key - mine * a.block_size;
    if (boxes >= 8) {
#pragma unroll 1
      for (int i = 0; i < boxes; i += 8) page_boxes<8, false>(map, dst, i, i, id, row, bar);
    } else if (boxes == 4) {
      page_boxes<4, false>(map, dst, 0, 0, id, row, bar);
    } else {
#pragma unroll 1
      for (int i = 0; i < boxes; ++i) page_boxes<1, false>(map, dst, i, i, id, row, bar);
    }
  }
  __device__ uint32_t chunk_addr(uint32_t tile, int row, int c) const {
    return tile + (c >> 3) * (128 * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
  }
  // Warp 11, once the copies have landed: staged rows to their places, zeros
  // in the V rows past the keys that the copies may have filled.
  __device__ bool mend_tile(int t, int v, int b) {
    constexpr int kRows = 32 / kChunks;  // rows of a step
    // Steps read at once: a turn takes about a microsecond (64 x 32 staged rows 136 us,
    // 141 with 4, 132 with 8, with which 8192 rows took 479 instead of 472; 202 where
    // rows behind the first turn were read one step at a time).
    constexpr int kAhead = 6;
    const int c = lane % kChunks, key0 = t * kTileKeys;
    const int first = max(0, pooled - key0);             // first row not from the pool
    const int end = min(kTileKeys, p.s.len - key0);      // first row past the keys
    const int staged = a.stage_k ? max(0, end - first) : 0;
    const unsigned char* src = nullptr;
    if (staged)
      src = (v ? a.stage_v : a.stage_k) + p.b * a.stage_seq +
            (long long)(key0 + first - pooled) * a.stage_row + ((long long)p.h * a.dim + c * 8) * 2;
    const uint32_t dst = tile(b);
    const int r0 = lane / kChunks;
#pragma unroll 1
    for (int at = r0; at == r0 || at < staged; at += kAhead * kRows) {
      uint4 x[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int r = at + i * kRows;
        x[i] = r < staged && c * 8 < a.dim
                   ? __ldg(reinterpret_cast<const uint4*>(src + r * a.stage_row))
                   : make_uint4(0, 0, 0, 0);
      }
      // All lanes come here at least once; their first batch waits for the copies.
      if (at == r0 && !wait(&sh->landed[b], (land_ph >> b) & 1)) return false;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int r = at + i * kRows;
        if (r < staged) st_shared16(chunk_addr(dst, first + r, c), x[i]);
      }
    }
    if (v) {
      int stop = kTileKeys;  // pages past the last are zeros already
      if (a.tables) {
        const int last = pooled > 0 ? page_of(pooled - 1) + 1 : 0;
        stop = (int)min((long long)kTileKeys, (long long)last * a.block_size - key0);
      }
#pragma unroll 1
      for (int r = first + staged + r0; r < stop; r += kRows)
        st_shared16(chunk_addr(dst, r, c), make_uint4(0, 0, 0, 0));
    }
    fence_proxy_async_smem();
    if (elect_one_after_sync()) mbar_arrive(&sh->full[b]);
    return true;
  }
  __device__ void load_rows(int t, int v, uint32_t dst) {
    constexpr int kStep = kLoaders / kChunks;
    const int thread = role * 32 + lane, c = thread % kChunks;
    const long long col = ((long long)p.h * a.dim + c * 8) * 2;
    const unsigned char* base = v ? a.v : a.k;
    const long long ld = v ? a.ld_v : a.ld_k;
    const int32_t* table = a.tables + (long long)p.b * a.max_blocks;
    bool bad = false;
#pragma unroll 2
    for (int r = thread / kChunks; r < kTileKeys; r += kStep) {
      const int key = t * kTileKeys + r;
      bool ok = key < p.s.len && c * 8 < a.dim;
      const unsigned char* src = base;
      if (key < pooled) {
        const int blk = page_of(key);
        int id = ok ? table[blk] : 0;
        if (id < 0 || id >= a.num_blocks) {
          bad = true;
          ok = false;
          id = 0;
        }
        src = base + id * a.page_bytes + (key - blk * a.block_size) * ld + col;
      } else if (ok) {
        src = (v ? a.stage_v : a.stage_k) + p.b * a.stage_seq + (key - pooled) * a.stage_row + col;
      }
      cp_async16(chunk_addr(dst, r, c), src, ok ? 16u : 0u);
    }
    if (bad) set_status(a.status, SPEC_EDEVICE);
    cp_async_wait_all();
    fence_proxy_async_smem();
    __syncwarp();
  }
  __device__ bool elect_one_after_sync() {
    __syncwarp();
    return elect_one();
  }
  // The loads of a piece, in piece_program's order of takes and gives.
  __device__ bool fill() {
    const int m = p.m;
    if (m == 0) return true;
    const bool two = p.two;
    const int ahead = two ? 1 : 2, c0 = two ? p.c0 : m;
#pragma unroll 1
    for (int w = 0; w < (two ? 2 : 1); ++w)
      if (!take_q(w)) return false;
#pragma unroll 1
    for (int i = -ahead; i < m; ++i) {
      const bool more = i + ahead < m;
      int v_buf = 0, k_buf = 0;
#pragma unroll 1
      for (int v = i >= 0; v >= (more ? 0 : 1); --v) {
        int b;
        if (!take(&b) || !load_kv(p.t0 + (v ? i : i + ahead), v, b)) return false;
        if (v) v_buf = b; else k_buf = b;
        if (v && !two) buf.give(b);
      }
      if (more && i + ahead == max(c0 - 1, 0)) buf.give(q_buf[0]);
      if (two && i >= 0) buf.give(v_buf);
      if (two && more && i + ahead == m - 1) buf.give(q_buf[1]);
      if (more) buf.give(k_buf);
    }
    return true;
  }
  // The copying warps.
  __device__ bool run() {
    MsgRing ring;
    for (;;) {
      if (!wait(&sh->msg_full[ring.i], ring.ph)) return false;
      p = sh->msg[ring.i];
      __syncwarp();
      if (p.end) return true;
      if (lane == 0) mbar_arrive(&sh->msg_empty[ring.i]);
      ring.step();
      begin();
      if (!fill()) return false;
    }
  }
  // The third warp walks the CTA's run, two pieces ahead of the one that it mends:
  // a message's slot is free once all have read the one four before it, for which
  // every piece before that has to be mended.
  __device__ bool schedule() {
    Cursor cur_ = cursor(a, sh);
    MsgRing out, in;
    int ahead = 0;
    bool over = false;
    for (;;) {
      while (!over && ahead < 3) {
        AttendPiece x;
        over = !cur_.next(&x);
        if (!wait(&sh->msg_empty[out.i], out.ph ^ 1)) return false;
        if (lane == 0) {
          Msg* q = &sh->msg[out.i];
          q->end = over;
          if (!over) {
            const int m = x.t1 - x.t0;
            const bool two = x.ntok > a.shape.tpt;
            q->s = x.s;
            q->b = x.b;
            q->h = x.h;
            q->t0 = x.t0;
            q->m = m;
            q->tok0 = x.tok0;
            q->ntok = x.ntok;
            q->two = two;
            q->c0 = two ? first_tile_count(a.shape, x) : (m + 1) / 2;
            q->c1 = two ? m : m / 2;
            q->part = x.t0 > 0 ? 1 : x.t1 < x.nt ? 2 : 0;
            if (q->part) {
              q->head = unit_head(sh, x);
              q->parts = unit_parts(sh, x, q->head);
            }
          }
          mbar_arrive(&sh->msg_full[out.i]);
        }
        out.step();
        ++ahead;
      }
      __syncwarp();
      p = sh->msg[in.i];
      in.step();
      --ahead;
      if (p.end) break;
      begin();
      if (!fill()) return false;
    }
    return true;
  }
};

// ---------------------------------------------------------------------------
// Matrix instructions, issued by one thread
// ---------------------------------------------------------------------------
// Between two products it is what the tensor cores wait for, so it makes no
// votes and no elections (a whole warp with elections: 8192 rows 557 us, so 519).
template <typename T, int DP>
struct Issuer {
  static constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
  static constexpr uint32_t kIdescQK = mma_idesc(kBf, 128, 128, false);
  static constexpr uint32_t kIdescPV = mma_idesc(kBf, 128, DP, true);
  const AttendArgs& a;
  Shared* sh;
  uint32_t tiles, tmem;
  Buffers<Tile<DP>::kCount> buf;
  int q0_buf, q1_buf, k_buf, v_buf;
  uint32_t p_ph;     // bit w: parity of p_full[w]
  uint32_t o_ph;     // bit w: parity of o_empty[w], 1 before its first use

  __device__ Issuer(const AttendArgs& a_, Shared* s, uint32_t t, uint32_t m)
      : a(a_), sh(s), tiles(t), tmem(m), p_ph(0), o_ph(3) {}
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t ph) {
    return wait_bar(bar, ph);
  }
  __device__ __forceinline__ bool take(int* b) {
    uint32_t ph;
    *b = buf.take(&ph);
    return wait(&sh->full[*b], ph);
  }
  __device__ __forceinline__ bool take_q(int w) { return take(w ? &q1_buf : &q0_buf); }
  __device__ __forceinline__ bool take_k(int) { return take(&k_buf); }
  __device__ __forceinline__ bool take_v(int) { return take(&v_buf); }
  __device__ __forceinline__ void give(int b) {
    tc_commit(&sh->empty[b]);
    buf.give(b);
  }
  __device__ __forceinline__ void give_q(int w) { give(w ? q1_buf : q0_buf); }
  __device__ __forceinline__ void give_k() { give(k_buf); }
  __device__ __forceinline__ void give_v() { give(v_buf); }
  // Low words of the descriptors; the high word is the same for all.
  __device__ __forceinline__ uint32_t desc(int b, uint32_t lead_bytes) const {
    return ((tiles + b * Tile<DP>::kBytes) >> 4) | ((lead_bytes >> 4) << 16);
  }
  // S_w = Q K^T
  __device__ __forceinline__ void qk(int w, int x) {
    const uint32_t qd = desc(x ? q1_buf : q0_buf, 16), kd = desc(k_buf, 16);
    const uint32_t s = tmem + w * 128;
#pragma unroll
    for (int k = 0; k < DP / 16; ++k) {
      const uint32_t off = (k >> 2) * (128 * 128 / 16) + (k & 3) * 2;
      mma_ss(s, mma_sdesc(qd + off), mma_sdesc(kd + off), kIdescQK, k > 0);
    }
    tc_commit(&sh->s_full[w]);
  }
  // O_w (+)= P_w V, the first once the softmax warps have read the last piece's.
  __device__ __forceinline__ bool pv(int w, bool first, bool last) {
    const uint32_t vd = desc(v_buf, 128 * 128);
    const uint32_t s = tmem + w * 128, o = tmem + 256 + w * DP;
    if (!wait(&sh->p_full[w], (p_ph >> w) & 1)) return false;
    p_ph ^= 1u << w;
    if (first) {
      if (!wait(&sh->o_empty[w], (o_ph >> w) & 1)) return false;
      o_ph ^= 1u << w;
    }
    tc_fence_after();
#pragma unroll
    for (int k = 0; k < kTileKeys / 16; ++k)
      mma_ts(o, s + k * 8, mma_sdesc(vd + k * (16 * 128 / 16)), kIdescPV, k > 0 || !first);
    if (last) tc_commit(&sh->o_full[w]);
    return true;
  }
  __device__ __forceinline__ bool run() {
    MsgRing ring;
    bool ok = false;
    while ((int)blockIdx.x != a.stop_cta) {
      if (!wait(&sh->msg_full[ring.i], ring.ph)) break;
      const Msg* q = &sh->msg[ring.i];
      const int m = q->m, two = q->two, c0 = q->c0, end = q->end;
      ok = end;
      if (end) break;
      mbar_arrive(&sh->msg_empty[ring.i]);
      ring.step();
      if (!piece_program(m, two, c0, *this)) break;
    }
    // Instructions in flight and their arrivals on barriers end before tensor memory
    // is given back and the CTA ends.
    tc_commit(&sh->drain);
    return wait_bar(&sh->drain, 0) && ok;
  }
};

// ---------------------------------------------------------------------------
// Softmax and output, one thread per row
// ---------------------------------------------------------------------------
// A row's 128 scores are loaded at once and stay in registers through maximum,
// exponentials and rounding; a thread needs no other's maximum or sum.
template <typename T> struct Pack;
template <> struct Pack<__nv_bfloat16> {
  static __device__ __forceinline__ float2 both(uint32_t x) {
    return make_float2(bf_lo(x), bf_hi(x));
  }
  static __device__ __forceinline__ uint32_t two(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};
template <> struct Pack<__half> {
  static __device__ __forceinline__ float2 both(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
  }
  static __device__ __forceinline__ uint32_t two(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};

// The largest of each half as a signed number, of top and two more words of outputs:
// 0x7fff, as which the conversions above write NaN, is larger than any other value.
__device__ __forceinline__ uint32_t top_halves(uint32_t x, uint32_t y, uint32_t top) {
  return __vimax3_s16x2(x, y, top);
}
// Sets *flag where a half of `top` (0 to 0x7fff) is NaN; without a branch, as every
// instruction at a unit's end is fetched anew (16 ragged prompts 355 us with one).
__device__ __forceinline__ void flag_nan(int* flag, uint32_t top) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 t;\n\t"
      "add.u32 t, %1, 0x00010001;\n\t"
      "and.b32 t, t, 0x80008000;\n\t"
      "setp.ne.u32 p, t, 0;\n\t"
      "@p st.shared.b32 [%0], 1;\n\t}" ::"r"(smem_u32(flag)),
      "r"(top)
      : "memory");
}

// Two fp32 operations per instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float weight(float m, float ref) {
  return m == -INFINITY ? 0.0f : ex2(m - ref);
}

// The products give a row 0 times each V value that it does not see, which is NaN where
// the value is not finite. So where an output is NaN, the CTA looks at its end for
// such values, and a row with one behind its last key in its unit's tiles gets those
// columns again, from the keys that it sees: what is not finite among their values,
// as no weight changes that, else the sum of the weighted values, which only rows of
// the last tiles before the first such value need. All 256 threads look, a warp
// forms four rows at once, a key per lane: 8192 rows with one NaN near their end take
// 40 ms (350 with a thread per row), with all values infinite 2.5 (122).
// (Values taken out of the tiles that not all rows of a unit see, before their
// products, cost 16 ragged prompts 30 us; looking at the outputs costs 10 to 14.)
template <typename T, int DP>
struct Redo {
  static constexpr int kCols = DP / 32;  // columns of a lane
  static constexpr int kRows = 4;        // rows of a warp at once
  static constexpr int kStride = DP * 2 + 16;  // of rows in shared memory: eight lanes'
                                               // 16 bytes lie in different banks
  static_assert(8 * (kRows + 32) * kStride <= Tile<DP>::kSmemTiles, "scratch");
  const AttendArgs& a;
  Shared* sh;
  AttendPiece x;
  // Of each column, in place of the softmax warps' exchange: the first key with NaN, an
  // infinity, a negative one; the last with any of them that not all rows see.
  __device__ int* first(int kind) const { return reinterpret_cast<int*>(sh->ml) + kind * 128; }
  __device__ int* last() const { return first(3); }
  __device__ void barrier() const {
    __syncwarp();  // the barrier takes whole warps
    asm volatile("bar.sync 1, 256;" ::: "memory");
  }
  // K (v = 0) or V row of a key; null: a bad table entry, which stands for zeros
  __device__ const unsigned char* row(int v, int key) const {
    const int pooled = a.stage_k ? x.s.len - x.s.n : x.s.len;
    const unsigned char* p = v ? a.v : a.k;
    const long long ld = v ? a.ld_v : a.ld_k;
    if (key >= pooled) {
      p = (v ? a.stage_v : a.stage_k) + x.b * a.stage_seq + (key - pooled) * a.stage_row;
    } else if (a.tables) {
      const int page = (int)a.by_bs((uint32_t)key);
      const int id = a.tables[(long long)x.b * a.max_blocks + page];
      if (id < 0 || id >= a.num_blocks) return nullptr;
      p += id * a.page_bytes + (key - page * a.block_size) * ld;
    } else {
      p += (x.s.row0 + (long long)key) * ld;
    }
    return p + (long long)x.h * a.dim * 2;
  }
  // Notes what is not finite in V rows [from, to); early: all rows see them.
  __device__ void look(int from, int to, bool early) {
    constexpr int kChunks = DP / 8, kStep = 256 / kChunks, kAhead = 4;
    const int c = threadIdx.x % kChunks;
    uint32_t seen[3] = {0, 0, 0};  // columns of the chunk with NaN, ...
#pragma unroll 1
    for (int at = from + threadIdx.x / kChunks; at < to; at += kAhead * kStep) {
      uint4 z[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int key = at + k * kStep;
        const unsigned char* v = key < to && c * 8 < a.dim ? row(1, key) : nullptr;
        z[k] = load(reinterpret_cast<const uint4*>(v) + c, v);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const uint32_t w[4] = {z[k].x, z[k].y, z[k].z, z[k].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = Pack<T>::both(w[i / 2]);
          const float y = i % 2 ? f.y : f.x;
          if (isfinite(y)) continue;
          const int kind = y != y ? 0 : y > 0 ? 1 : 2, key = early ? 0 : at + k * kStep;
          if (early) {
            if (seen[kind] >> i & 1) continue;
            seen[0] |= (uint32_t)(kind == 0) << i;
            seen[1] |= (uint32_t)(kind == 1) << i;
            seen[2] |= (uint32_t)(kind == 2) << i;
          } else {
            atomicMax(last() + c * 8 + i, key);
          }
          atomicMin(first(kind) + c * 8 + i, key);
        }
      }
    }
  }
  // 16 bytes, or zeros: without a branch, so that several are in flight.
  __device__ uint4 load(const uint4* p, bool there) const {
    const uint4 z = *(there ? p : reinterpret_cast<const uint4*>(a.v));
    return there ? z : make_uint4(0, 0, 0, 0);
  }
  // `n` rows at the addresses that lanes 0 .. n-1 hold (0: zeros) to dst, zeros behind
  // the last column.
  template <int n>
  __device__ void copy(unsigned long long src, unsigned char* dst) {
    constexpr int kChunks = DP / 8;
    const int lane = threadIdx.x & 31;
#pragma unroll 8
    for (int i = lane; i < n * kChunks; i += 32) {
      const int r = i / kChunks, c = i % kChunks;
      const uint4* p = reinterpret_cast<const uint4*>(__shfl_sync(0xffffffffu, src, r));
      *reinterpret_cast<uint4*>(dst + r * kStride + c * 16) = load(p + c, p && c * 8 < a.dim);
    }
  }
  // kRows rows of the unit, from row r0 on (token, head of the group), by a warp.
  __device__ void rows_again(int r0) {
    const int lane = threadIdx.x & 31, col = lane * kCols;
    // This warp's place in what held the tiles: the rows' queries, then 32 K rows.
    unsigned char* scratch = reinterpret_cast<unsigned char*>(sh) - Tile<DP>::kSmemTiles +
                             (threadIdx.x >> 5) * ((kRows + 32) * kStride);
    int seen[kRows], most = 0;
    long long out[kRows];  // bytes into out
    unsigned long long q = 0;
    float o[kRows][kCols];
    uint32_t bad = 0, sums = 0;  // by bit: this lane's columns of all rows
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int r = min(r0 + k, x.ntok * a.group - 1), t = (int)a.by_group((uint32_t)r);
      const long long at = x.s.row0 + x.tok0 + t;
      const long long head = (long long)(x.h * a.group + r - t * a.group) * a.dim * 2;
      seen[k] = max(0, x.s.len - x.s.n + x.tok0 + t + 1);
      if (lane == k) q = (unsigned long long)(a.q + at * a.ld_q + head);
      out[k] = at * a.ld_out + head;
      uint32_t formed = 0;
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const bool behind = last()[col + i] >= seen[k], nan = first(0)[col + i] < seen[k],
                   pos = first(1)[col + i] < seen[k], neg = first(2)[col + i] < seen[k];
        const bool sum = behind && !(nan || pos || neg);
        bad |= (uint32_t)(behind && r0 + k == r) << (k * kCols + i);
        formed |= (uint32_t)sum << (k * kCols + i);
        o[k][i] = nan || (pos && neg) ? NAN : pos ? INFINITY : neg ? -INFINITY : 0.0f;
      }
      sums |= formed;
      if (!__any_sync(0xffffffffu, formed)) seen[k] = 0;
      most = max(most, seen[k]);
    }
    if (!__any_sync(0xffffffffu, bad)) return;
    __syncwarp();
    copy<kRows>(q, scratch);
    float top[kRows], l[kRows], acc[kRows][kCols];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      top[k] = -INFINITY;
      l[k] = 0.0f;
#pragma unroll
      for (int i = 0; i < kCols; ++i) acc[k][i] = 0.0f;
    }
#pragma unroll 1
    for (int key0 = 0; key0 < most; key0 += 32) {
      const int key = key0 + lane;
      unsigned long long kp = 0, vp = 0;
      if (key < most) {
        kp = (unsigned long long)row(0, key);
        vp = (unsigned long long)row(1, key);
      }
      const bool there = vp != 0;
      if (!there) vp = (unsigned long long)a.v;  // any rows, with weights of 0
      __syncwarp();
      copy<32>(kp, scratch + kRows * kStride);
      __syncwarp();
      float w[kRows];
#pragma unroll
      for (int k = 0; k < kRows; ++k) w[k] = 0.0f;
#pragma unroll 2
      for (int c = 0; c < DP / 8; ++c) {
        const uint4 z =
            *reinterpret_cast<const uint4*>(scratch + (kRows + lane) * kStride + c * 16);
        const uint32_t zw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
          const uint4 u = *reinterpret_cast<const uint4*>(scratch + k * kStride + c * 16);
          const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = Pack<T>::both(uw[i]), g = Pack<T>::both(zw[i]);
            w[k] = fmaf(f.x, g.x, fmaf(f.y, g.y, w[k]));
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const float s = key < seen[k] ? w[k] * a.scale_log2 : -INFINITY;
        float m = s;
#pragma unroll
        for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        m = fmaxf(m, top[k]);
        const float f = weight(top[k], m);
        top[k] = m;
        w[k] = key < seen[k] ? ex2(s - (m == -INFINITY ? 0.0f : m)) : 0.0f;
        l[k] = l[k] * f + w[k];
        if (!there) w[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < kCols; ++i) acc[k][i] *= f;
      }
#pragma unroll 8
      for (int j = 0; j < 32; ++j) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(__shfl_sync(0xffffffffu, vp, j));
        float y[kCols];
#pragma unroll
        for (int i = 0; i < kCols; i += 2) {
          const float2 f = Pack<T>::both(p[(min(col, a.dim - kCols) + i) / 2]);
          y[i] = f.x;
          y[i + 1] = f.y;
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
          const float wj = __shfl_sync(0xffffffffu, w[k], j);
#pragma unroll
          for (int i = 0; i < kCols; ++i)  // what it does not see may not be finite
            acc[k][i] = wj == 0.0f ? acc[k][i] : fmaf(wj, y[i], acc[k][i]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
#pragma unroll
      for (int d = 16; d; d >>= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], d);
      const float inv = l[k] > 0.0f || l[k] != l[k] ? 1.0f / l[k] : 0.0f;
      T* d = reinterpret_cast<T*>(a.out + out[k]) + col;
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (bad >> (k * kCols + i) & 1)
          d[i] = T(sums >> (k * kCols + i) & 1 ? acc[k][i] * inv : o[k][i]);
    }
  }
  // The rows of one unit, by 256 threads.
  __device__ void unit() {
    const int common = max(0, x.s.len - x.s.n + x.tok0 + 1);  // keys that all rows see
    barrier();
    for (int i = threadIdx.x; i < 512; i += 256) first(0)[i] = i < 384 ? INT32_MAX : -1;
    barrier();
    look(common, min(x.s.len, x.nt * kTileKeys), false);
    barrier();
    int most = -1;
    for (int i = 0; i < DP; ++i) most = max(most, last()[i]);
    if (most < 0) return;
    look(0, common, true);
    barrier();
#pragma unroll 1
    for (int r = (threadIdx.x >> 5) * kRows; r < x.ntok * a.group; r += 8 * kRows) rows_again(r);
  }
};
// What may be left at a CTA's end, by its softmax warps: the counts of a call whose waits
// ran out, else the rows to be formed again, of the units whose output the CTA wrote.
template <typename T, int DP>
__device__ __noinline__ void finish(const AttendArgs& a, Shared* sh) {
  if (sh->failed) {
    if (threadIdx.x == 0) count_rest(a, sh);
    return;
  }
  Cursor cur = cursor(a, sh);
  Redo<T, DP> r{a, sh};
  while (cur.next(&r.x)) {
    const bool whole = r.x.t0 == 0 && r.x.t1 == r.x.nt;
    if (r.x.nt && (whole || (sh->joined & (r.x.t0 > 0 ? 1 : 2)))) r.unit();
  }
}

template <typename T, int DP>
struct Softmax {
  const AttendArgs& a;
  Shared* sh;
  uint32_t tmem;    // with this warp's lanes
  int w, row;       // warpgroup, row of the tile
  int tok, head;    // row's token within a tile and query head within the group
  uint32_t s_ph, o_ph[2], x_ph, part_ph;

  __device__ bool wait(uint64_t* bar, uint32_t ph) {
    return __all_sync(0xffffffffu, wait_bar(bar, ph));
  }
  __device__ void arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
  }
  // Scores of one tile to p~; m is the reference and l the sum, both of this row.
  __device__ bool tile(int key0, int limit, int warp_limit, bool live, bool valid, bool first,
                       float& m, float& l) {
    if (!wait(&sh->s_full[w], s_ph)) return false;
    s_ph ^= 1;
    if (live) {
      tc_fence_after();
      uint32_t s[128];
      const uint32_t col = tmem + w * 128;
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32(col + 32 * i, s, 32 * i);
      tmem_wait_ld(s);
      if (key0 + kTileKeys - 1 > warp_limit) {
        const int lim = limit - key0;
#pragma unroll
        for (int i = 0; i < 128; ++i)
          if (i > lim) s[i] = 0xff800000u;
      }
      float mx[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) mx[i] = __uint_as_float(s[i]);
#pragma unroll
      for (int i = 4; i < 124; i += 8)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mx[j] = fmaxf(fmaxf(mx[j], __uint_as_float(s[i + j])), __uint_as_float(s[i + 4 + j]));
#pragma unroll
      for (int j = 0; j < 4; ++j) mx[j] = fmaxf(mx[j], __uint_as_float(s[124 + j]));
      const float top =
          fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
      const bool raise = valid && (top > m + kSlack || (m == -INFINITY && top > m));
      if (__any_sync(0xffffffffu, raise)) {
        const float ref = fmaxf(m, top - kHead), f = weight(m, ref);
        m = ref;
        l *= f;
        if (!first) {  // the products up to the last tile's are in O
#pragma unroll 1
          for (int c = 0; c < DP; c += 32) {
            uint32_t o[32];
            tmem_ld32(tmem + 256 + w * DP + c, o, 0);
            tmem_wait_ld(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st32(tmem + 256 + w * DP + c, o, 0);
          }
        }
      }
      const float ref = m == -INFINITY ? 0.0f : m;
      const uint64_t c2 = pair(a.scale_log2, a.scale_log2), r2 = pair(-ref, -ref);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 128; i += 64) {
        uint32_t p[32];
#pragma unroll
        for (int j = 0; j < 64; j += 2) {
          float e0, e1;
          unpair(fma2(pair(__uint_as_float(s[i + j]), __uint_as_float(s[i + j + 1])), c2, r2), e0,
                 e1);
          e0 = ex2(e0);
          e1 = ex2(e1);
          sum[(j >> 1) & 1] = add2(sum[(j >> 1) & 1], pair(e0, e1));
          p[j / 2] = Pack<T>::two(e0, e1);
        }
        tmem_st32(col + i / 2, p, 0);
      }
      float l0, l1;
      unpair(add2(sum[0], sum[1]), l0, l1);
      l += l0 + l1;
      tmem_wait_st();
      tc_fence_before();
    }
    arrive(&sh->p_full[w]);
    return true;
  }
  // Columns [c0, c0 + 32) of f0 * O0 + f1 * O1; all lanes. A factor of 0 drops its
  // part whatever it holds (rows that saw no key there, beside values not finite).
  __device__ void read_o(int c0, bool has0, float f0, bool has1, float f1, float (&o)[32]) {
    uint32_t x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = 0.0f;
    if (has0) {
      tmem_ld32(tmem + 256 + c0, x, 0);
      tmem_wait_ld(x);
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = f0 == 0.0f ? 0.0f : f0 * __uint_as_float(x[i]);
    }
    if (has1) {
      tmem_ld32(tmem + 256 + DP + c0, x, 0);
      tmem_wait_ld(x);
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = f1 == 0.0f ? o[i] : fmaf(f1, __uint_as_float(x[i]), o[i]);
    }
  }
  // 16 columns of a row from col on, packed; 32-byte sectors where the rows begin on them.
  __device__ __forceinline__ void write16(unsigned char* row, int col, const uint32_t (&x)[8]) {
    unsigned char* d = row + col * 2;
    if (a.out_sectors) {
      if (col < a.dim)
        asm volatile("st.global.L1::no_allocate.v8.b32 "
                     "[%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d),
                     "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]),
                     "r"(x[7])
                     : "memory");
    } else {
      if (col < a.dim) *reinterpret_cast<uint4*>(d) = make_uint4(x[0], x[1], x[2], x[3]);
      if (col + 8 < a.dim) *reinterpret_cast<uint4*>(d + 16) = make_uint4(x[4], x[5], x[6], x[7]);
    }
  }
  // The row's address in out; null for a row without a token.
  __device__ __forceinline__ unsigned char* out_row(const Msg& p, int base, int r) const {
    const int tk = (int)a.by_group((uint32_t)r);
    if (tk >= min(a.shape.tpt, p.ntok - base)) return nullptr;
    return a.out + (long long)(p.s.row0 + p.tok0 + base + tk) * a.ld_out +
           (long long)(p.h * a.group + r - tk * a.group) * a.dim * 2;
  }
  // Columns [from, to) of f0 * O0 + f1 * O1 to out, all lanes. A thread holds a
  // row, and rows lie far apart: a store would cover 32 bytes of each of 32 rows. So
  // 64 packed columns go back to tensor memory (over columns already read) and
  // are read as 16 rows of which 4 lanes share each: with the columns in the order
  // of their places, a lane has 16 of the 64, and a store covers 128 bytes of 8
  // rows (chunks of 300 to 512 rows 187 us, 196 without). Nothing reads them here,
  // so they are not kept in the L1 (8192 rows 488 us, so 482).
  // A valid row's NaN is flagged, for finish().
  __device__ void write_rows(const Msg& p, int base, int from, int to, uint32_t stage, bool has0,
                             float f0, bool has1, float f1, bool valid) {
    const int lane = threadIdx.x & 31;
    uint32_t top = 0;  // halves of outputs, the largest
    // Half of a head of 64: a row's 64 bytes by its thread. So are the zeros of a tile
    // without keys, as the next piece's products may be in tensor memory already.
    if (to - from < 64 || !(has0 || has1)) {
      unsigned char* dst = out_row(p, base, row);
#pragma unroll 1
      for (int c = from; c < to; c += 32) {
        float o[32];
        read_o(c, has0, f0, has1, f1, o);
#pragma unroll
        for (int i = 0; i < 32; i += 16) {
          uint32_t x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = Pack<T>::two(o[i + 2 * k], o[i + 2 * k + 1]);
          if constexpr (DP == 64) {
#pragma unroll
            for (int k = 0; k < 8; k += 2) top = top_halves(x[k], x[k + 1], top);
          }
          if (dst) write16(dst, c + i, x);
        }
      }
      flag_nan(&sh->odd, valid ? top : 0);
      return;
    }
#pragma unroll 1
    for (int c = from; c < to; c += 64) {
      uint32_t x[32];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float o[32];
        read_o(c + 32 * half, has0, f0, has1, f1, o);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int at = 16 * half + i;  // packed column 8 l + 2 k + e to place 8 k + 2 l + e
          x[8 * ((at >> 1) & 3) + 2 * (at >> 3) + (at & 1)] = Pack<T>::two(o[2 * i], o[2 * i + 1]);
        }
      }
      tmem_st32(stage, x, 0);
#pragma unroll
      for (int i = 0; i < 32; i += 2) top = top_halves(x[i], x[i + 1], top);
      tmem_wait_st();
      tmem_ld_rows16(stage, x, 0);
      tmem_ld_rows16(stage + (16u << 16), x, 16);
      tmem_wait_ld(x);
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // rows lane / 4 + 8 j
        unsigned char* dst = out_row(p, base, (row & ~31) + (lane >> 2) + 8 * j);
        uint32_t y[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          y[2 * k] = x[16 * (j >> 1) + 4 * k + 2 * (j & 1)];
          y[2 * k + 1] = x[16 * (j >> 1) + 4 * k + 2 * (j & 1) + 1];
        }
        if (dst) write16(dst, c + 16 * (lane & 3), y);
      }
      stage += 32;
    }
    flag_nan(&sh->odd, valid ? top : 0);
  }
  __device__ bool run() {
    MsgRing ring;
    for (;;) {
      if (!wait(&sh->msg_full[ring.i], ring.ph)) return false;
      const Msg p = sh->msg[ring.i];
      if (p.end) return true;
      arrive(&sh->msg_empty[ring.i]);
      ring.step();
      const bool two = p.two;
      const int tpt = a.shape.tpt;
      const int base = two ? w * tpt : 0;  // the tile's first token in the unit
      const bool valid = tok < min(tpt, p.ntok - base);
      const bool live = __any_sync(0xffffffffu, valid);
      const int limit = valid ? p.s.len - p.s.n + p.tok0 + base + tok : INT32_MAX;
      const int warp_limit = __reduce_min_sync(0xffffffffu, limit);
      const int c0 = p.c0, c1 = p.c1, mine = w ? c1 : c0;
      float m = -INFINITY, l = 0.0f;
#pragma unroll 1
      for (int i = 0; i < mine; ++i) {
        const int t = p.t0 + (two ? i : 2 * i + w);
        if (!tile(t * kTileKeys, limit, warp_limit, live, valid, i == 0, m, l)) return false;
      }
      const bool whole = p.part == 0;
      const long long slot = 2 * blockIdx.x + (p.part == 1 ? 0 : 1);
      const long long prow = (slot * 2 + (two ? w : 0)) * kTileRows + row;
      const int r = p.s.row0 + p.tok0 + base + tok;
      const int qh = p.h * a.group + head;
      float f0 = w == 0 ? 1.0f : 0.0f, f1 = 1.0f - f0;
      int from = 0, to = DP;
      bool has0 = w == 0 && c0 > 0, has1 = w == 1 && c1 > 0;
      if (!two) {  // both warpgroups hold part of every row: join, half the columns each
        sh->ml[w][row] = make_float2(m, l);
        arrive(&sh->swap);
        if (!wait(&sh->swap, x_ph)) return false;
        x_ph ^= 1;
        const float2 u = sh->ml[w ^ 1][row];
        arrive(&sh->swap);
        if (!wait(&sh->swap, x_ph)) return false;
        x_ph ^= 1;
        const float top = fmaxf(m, u.x);
        const float fm = weight(m, top), fu = weight(u.x, top);
        f0 = w ? fu : fm;
        f1 = w ? fm : fu;
        l = fm * l + fu * u.y;
        m = top;
        has0 = c0 > 0;
        has1 = c1 > 0;
        from = w * (DP / 2);
        to = from + DP / 2;
      }
      // With two query tiles a warpgroup waits for its own accumulator's barrier only:
      // waiting for both put them in step, where one should work on scores while
      // the other waits for products (8192 rows 482 us, so 468; 16 ragged prompts 390,
      // 345). With one it waits for both, behind the exchange: the other warpgroup
      // has then seen all earlier phases of its barrier, so none is taken for the
      // one before it.
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if ((x ? c1 : c0) > 0) {
          if ((!two || x == w) && !wait(&sh->o_full[x], o_ph[x])) return false;
          o_ph[x] ^= 1;
        }
      if (live) {
        tc_fence_after();
        if (whole) {
          const float inv = l > 0.0f || l != l ? __fdividef(1.0f, l) : 0.0f;
          f0 *= inv;
          f1 *= inv;
        }
        if (whole) {
          write_rows(p, base, from, to, tmem + 256 + (two ? w * DP : from), has0, f0, has1, f1,
                     valid);
        } else {
#pragma unroll 1
          for (int c = from; c < to; c += 32) {
            float o[32];
            read_o(c, has0, f0, has1, f1, o);
            float4* po = part_o(slot, two ? w : 0, c / 4);
            if (valid) {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                po[(i / 4) * kTileRows + row] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            }
          }
        }
        if (valid && (two || w == 0)) {
          if (!whole) a.part_ml[prow] = make_float2(m, l);
          else if (a.lse)
            a.lse[(long long)r * a.q_heads + qh] =
                l > 0.0f || l != l ? (m + __log2f(l)) * (float)kLn2 : -INFINITY;
        }
        tc_fence_before();
      }
      __syncwarp();
      if ((threadIdx.x & 31) == 0) {  // eight arrivals on each accumulator's barrier
        if (c0 > 0 && !(two && w)) mbar_arrive(&sh->o_empty[0], two ? 2 : 1);
        if (c1 > 0 && !(two && !w)) mbar_arrive(&sh->o_empty[1], two ? 2 : 1);
      }
      if (!whole && !join_parts(p)) return false;
    }
  }
  // Columns [4 * c4, ...) of a part's tile: four columns of all rows, then the next four.
  __device__ __forceinline__ float4* part_o(long long slot, int tile, int c4) const {
    return reinterpret_cast<float4*>(a.part_o) +
           ((slot * 2 + tile) * (DP / 4) + c4) * kTileRows;
  }
  // A part of a divided unit is written: the CTA that counts the unit's last one
  // joins them, in their order, and leaves the count at zero.
  __device__ bool join_parts(const Msg& p) {
    __threadfence();
    arrive(&sh->parted);
    if (threadIdx.x < 32) {
      if (!wait(&sh->parted, part_ph)) return false;
      if (threadIdx.x == 0) {
        sh->last = count_part(a, p.head, p.parts);
        if (sh->last) sh->joined |= p.part;
        ++sh->counted;
        mbar_arrive(&sh->ticketed);
      }
      __syncwarp();
    }
    if (!wait(&sh->ticketed, part_ph)) return false;
    part_ph ^= 1;
    if (!sh->last) return true;
    fence_acq_rel();
    const int tpt = a.shape.tpt;
#pragma unroll 1
    for (int t = 0; t <= p.two; ++t) {
      const int rows = min(tpt, p.ntok - t * tpt) * a.group;
      // What counts is how much is in flight: a read takes about a microsecond, and
      // one SM reads all parts. Few rows (a step of decoding) need several parts at
      // once, 16 rows over 65536 keys in 18 parts 58.5 us where the second form
      // took 61; many fill the reads with their columns, 256 rows over them 118 us
      // where four columns a thread, a part at a time, took 142.
      if (rows <= 16) join_rows<2, 8>(p, t, rows, 4);
      else join_rows<8, 2>(p, t, rows, rows <= 64 ? 6 : 7);
    }
    return true;
  }
  // A thread has one row (of 2^log_slots), kCols groups of four columns, and reads
  // kParts parts at once.
  template <int kCols, int kParts>
  __device__ __forceinline__ void join_rows(const Msg& p, int t, int rows, int log_slots) {
    int tid;  // read here: what depends on it is not held through the tiles' loop
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
    const int r = tid & ((1 << log_slots) - 1);
    if (r >= rows) return;
    const int tk = (int)a.by_group((uint32_t)r), qh = p.h * a.group + r - tk * a.group;
    const long long token = p.s.row0 + p.tok0 + t * a.shape.tpt + tk;
    unsigned char* dst = a.out + token * a.ld_out + (long long)qh * a.dim * 2;
#pragma unroll 1
    for (int c = (tid >> log_slots) * kCols; c < DP / 4; c += (256 >> log_slots) * kCols) {
      float m = -INFINITY, l = 0.0f, o[kCols][4];
#pragma unroll
      for (int j = 0; j < kCols; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
#pragma unroll 1
      for (int k0 = 0; k0 < p.parts; k0 += kParts) {
        float2 ml[kParts];
        float4 v[kParts][kCols];
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
          const int part = min(k0 + k, p.parts - 1);
          const long long slot = 2 * (p.head + part) + (part == 0 ? 1 : 0);
          ml[k] = __ldcg(a.part_ml + (slot * 2 + t) * kTileRows + r);
#pragma unroll
          for (int j = 0; j < kCols; ++j) v[k][j] = __ldcg(part_o(slot, t, c + j) + r);
        }
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
          if (k0 + k >= p.parts) continue;
          const float top = fmaxf(m, ml[k].x);
          const float f = weight(m, top), g = weight(ml[k].x, top);
          l = f * l + g * ml[k].y;
          m = top;
#pragma unroll
          for (int j = 0; j < kCols; ++j) {
            o[j][0] = f * o[j][0] + (g == 0.0f ? 0.0f : g * v[k][j].x);
            o[j][1] = f * o[j][1] + (g == 0.0f ? 0.0f : g * v[k][j].y);
            o[j][2] = f * o[j][2] + (g == 0.0f ? 0.0f : g * v[k][j].z);
            o[j][3] = f * o[j][3] + (g == 0.0f ? 0.0f : g * v[k][j].w);
          }
        }
      }
      const bool some = l > 0.0f || l != l;
      const float inv = some ? __fdividef(1.0f, l) : 0.0f;
      uint32_t x[2 * kCols];
#pragma unroll
      for (int j = 0; j < 2 * kCols; ++j)
        x[j] = Pack<T>::two(o[j / 2][2 * (j & 1)] * inv, o[j / 2][2 * (j & 1) + 1] * inv);
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 2 * kCols; j += 2) top = top_halves(x[j], x[j + 1], top);
      flag_nan(&sh->odd, top);
      if constexpr (kCols >= 4) {
#pragma unroll
        for (int j = 0; j < 2 * kCols; j += 8) {
          const uint32_t y[8] = {x[j],     x[j + 1], x[j + 2], x[j + 3],
                                 x[j + 4], x[j + 5], x[j + 6], x[j + 7]};
          write16(dst, c * 4 + 2 * j, y);
        }
      } else {
        static_assert(kCols >= 4 || kCols == 2, "16 bytes");
        if (c * 4 < a.dim)
          *reinterpret_cast<uint4*>(dst + c * 8) = make_uint4(x[0], x[1], x[2], x[3]);
      }
      if (c == 0 && a.lse)
        a.lse[token * a.q_heads + qh] = some ? (m + __log2f(l)) * (float)kLn2 : -INFINITY;
    }
  }
};

// One CTA per SM: 7 tiles of 32 KB (8 of 16 KB for heads of up to 64) fill its
// shared memory, S0 S1 O0 O1 its tensor memory. Two accumulators, as one alone would leave
// the tensor cores idle while its scores are worked on; a third has no room.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const __grid_constant__ AttendArgs a) {
  extern __shared__ __align__(1024) unsigned char smem[];
  Shared* sh = reinterpret_cast<Shared*>(smem + Tile<DP>::kSmemTiles);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < Tile<DP>::kCount; ++i) {
      mbar_init(&sh->full[i], 3);
      mbar_init(&sh->empty[i], 1);
      mbar_init(&sh->landed[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->s_full[i], 1);
      mbar_init(&sh->p_full[i], 4);
      mbar_init(&sh->o_full[i], 1);
      mbar_init(&sh->o_empty[i], 8);
    }
    mbar_init(&sh->swap, 8);
    mbar_init(&sh->drain, 1);
    mbar_init(&sh->parted, 8);
    mbar_init(&sh->ticketed, 1);
    for (int i = 0; i < kMsgs; ++i) {
      mbar_init(&sh->msg_full[i], 1);
      mbar_init(&sh->msg_empty[i], 8 + 1 + 2);
    }
    sh->run = 0;
    sh->counted = sh->failed = sh->odd = sh->joined = 0;
    fence_barrier_init();
  }
  if (warp == 8) tmem_alloc(&sh->tmem, kTmemCols);
  pdl_begin();
  tc_fence_before();
  find_run(a, sh);  // its barriers publish the above
  tc_fence_after();
  const uint32_t tiles = smem_u32(smem), tmem = sh->tmem;
  // Of the 384 * 168 registers of the launch, 208 to each of the 256 softmax threads, for a
  // row's 128 scores and their weights, 88 to the 128 others. (80 to 88 bytes a thread
  // are spilled, as the compiler reports.)
  bool ok = true;
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int row = tid & 127, t = (int)a.by_group((uint32_t)row);
    Softmax<T, DP> s{a, sh, tmem + ((uint32_t)(warp & 3) << 21), warp >> 2, row, t,
                     row - t * a.group, 0, {0, 0}, 0, 0};
    ok = s.run();
  } else if (warp == 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (elect_one()) {
      Issuer<T, DP> s(a, sh, tiles, tmem);
      ok = s.run();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp < 11) {
      Loader<DP, false> s(a, sh, tiles, tid - 9 * 32);
      ok = s.run();
      s.drain();
    } else {
      Loader<DP, true> s(a, sh, tiles, tid - 9 * 32);
      ok = s.schedule();
    }
  }
  if (!ok) {
    set_status(a.status, SPEC_ETIMEOUT);
    sh->failed = 1;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  // By softmax warps, whose registers suffice for any call.
  if (warp < 8 && (sh->failed | sh->odd)) finish<T, DP>(a, sh);
}

template <typename T, int DP>
cudaError_t launch(const AttendArgs& a, cudaStream_t st) {
  const size_t smem = Tile<DP>::kSmemTiles + sizeof(Shared);
  cudaError_t e = reserve_dyn_smem(attend_kernel<T, DP>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attend_kernel<T, DP>, dim3(a.ctas), dim3(kThreads), smem, st, a);
}

}  // namespace

namespace {
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}
}  // namespace

// Query rows: (column, head of the group, K/V head, row), a box holds the
// whole tokens of a tile in the order of the tile's rows. Packed K/V rows: (column,
// head, row), boxes of 128 rows. Pages: (column, head, row, block), boxes of the
// largest power of two of rows that divides both a page and a tile, so none
// crosses either; a box begins on a whole 1024-byte swizzle atom, so pages
// whose rows are no multiple of 8 are left to the row copies (64 x 9 rows on pages
// of 24: 608 us by row copies). Boxes have 64 columns; those past the head's end
// are filled with zeros.
cudaError_t attend_maps(AttendArgs* a) {
  const EncodeFn encode = encode_fn();
  if (!encode) return cudaErrorNotSupported;
  auto form = [&](CUtensorMap* map, const void* p, cuuint32_t rank, const cuuint64_t* dims,
                  const cuuint64_t* strides, const cuuint32_t* box) {
    const cuuint32_t step[4] = {1, 1, 1, 1};
    return encode(map,
                  a->dtype == SPEC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  rank, const_cast<void*>(p), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const cuuint64_t head = (cuuint64_t)a->dim * 2;
  {
    const cuuint64_t dims[4] = {(cuuint64_t)a->dim, (cuuint64_t)a->group, (cuuint64_t)a->kv_heads,
                                (cuuint64_t)a->T};
    const cuuint64_t strides[3] = {head, head * a->group, (cuuint64_t)a->ld_q};
    const cuuint32_t box[4] = {64, (cuuint32_t)a->group, 1, (cuuint32_t)a->shape.tpt};
    if (!form(&a->map_q, a->q, 4, dims, strides, box)) return cudaErrorInvalidValue;
  }
  const int bs = a->block_size;
  a->box_rows = kTileKeys;
  if (a->tables) a->box_rows = (bs & -bs) < kTileKeys ? (bs & -bs) : kTileKeys;
  if (a->box_rows < 8) a->box_rows = 0;
  if (!a->box_rows) return cudaSuccess;
  for (int v = 0; v < 2; ++v) {
    const cuuint64_t dims[4] = {(cuuint64_t)a->dim, (cuuint64_t)a->kv_heads,
                                (cuuint64_t)(a->tables ? bs : a->T), (cuuint64_t)a->num_blocks};
    const cuuint64_t strides[3] = {head, (cuuint64_t)(v ? a->ld_v : a->ld_k),
                                   (cuuint64_t)a->page_bytes};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)a->box_rows, 1};
    if (!form(v ? &a->map_v : &a->map_k, v ? a->v : a->k, a->tables ? 4 : 3, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t st) {
  if (a.dtype == SPEC_BF16)
    return a.dim <= 64 ? launch<__nv_bfloat16, 64>(a, st) : launch<__nv_bfloat16, 128>(a, st);
  return a.dim <= 64 ? launch<__half, 64>(a, st) : launch<__half, 128>(a, st);
}

}  // namespace specv
