// Growing block tables with the slot map of the new rows, and storing K/V
// rows in the paged pool.
//
// HiSpec (gist.science summary of arXiv 2510.01336), section 2
// "Unterstuetzung fuer Batch-Inferenz": paged attention with block tables lets
// every sequence hold its own number of tokens without padding. The pages
// give no layout; the one here is spec_commit_paged's.
#include "paged.cuh"

namespace specv {

namespace {

constexpr int kExtendThreads = 1024;
constexpr int kFillThreads = 256;

// Blocks of n <= 2^30 rows (64-bit divisions bound the one-launch form when it used
// them: 28 us for 64 prompts of up to 4096 rows).
__device__ __forceinline__ int blocks_for(const ExtendArgs& a, int n) {
  return (int)a.by_bs((uint32_t)(n + a.block_size - 1));
}
__device__ __forceinline__ int block_of(const ExtendArgs& a, int pos) {
  return (int)a.by_bs((uint32_t)pos);
}

// Block-wide exclusive scan of two counts per thread; totals in tot.
__device__ longlong2 block_excl_scan2(longlong2 v, longlong2* tot) {
  __shared__ longlong2 warp_sums[32];
  __shared__ longlong2 s_tot;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  longlong2 incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl.x, o);
    const long long y = __shfl_up_sync(0xffffffffu, incl.y, o);
    if (lane >= o) { incl.x += x; incl.y += y; }
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const longlong2 w = lane < (int)(blockDim.x >> 5) ? warp_sums[lane] : make_longlong2(0, 0);
    longlong2 wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, wi.x, o);
      const long long y = __shfl_up_sync(0xffffffffu, wi.y, o);
      if (lane >= o) { wi.x += x; wi.y += y; }
    }
    warp_sums[lane] = make_longlong2(wi.x - w.x, wi.y - w.y);
    if (lane == 31) s_tot = wi;
  }
  __syncthreads();
  const longlong2 base = warp_sums[warp];
  *tot = s_tot;
  return make_longlong2(base.x + incl.x - v.x, base.y + incl.y - v.y);
}

// What both forms of the call check, by the whole block: lengths and counts,
// the entry of a part-filled last block, the stack. Sequences are dealt to threads
// in runs of consecutive ones (their order is that of the pops); on return
// cnt holds the thread's missing blocks and new rows, pre those of the sequences
// before, tot all. SPEC_OK, or the code of the failure, the same in all threads.
__device__ int extend_check(const ExtendArgs& a, int b0, int b1, int ft, longlong2* pre,
                            longlong2* tot) {
  const int bs = a.block_size;
  longlong2 cnt = make_longlong2(0, 0);
  int bad = 0;
  for (int b = b0; b < b1; ++b) {
    const int len = a.seq_lens[b], add = a.add_len[b];
    if (len < 0 || add < 0 || (long long)len + add > (long long)a.max_blocks * bs) {
      bad = 1;
      continue;
    }
    const int held = blocks_for(a, len);
    if (add > 0 && held * (long long)bs > len) {  // rows go into the held last block
      const int id = a.tables[(size_t)b * a.max_blocks + held - 1];
      if (id < 0 || id >= a.num_blocks) bad = 1;
    }
    cnt.x += blocks_for(a, len + add) - held;
    cnt.y += add;
  }
  *pre = block_excl_scan2(cnt, tot);
  if (__syncthreads_or(bad) || ft < 0 || ft > a.num_blocks || tot->y > INT32_MAX ||
      (a.slot_map && tot->y > a.cap))
    return SPEC_EINVAL;
  if (tot->x > ft) return SPEC_ENOBLOCKS;
  bad = 0;  // popped ids must be valid
  for (int p = ft - (int)tot->x + threadIdx.x; p < ft; p += blockDim.x) {
    const int id = a.free_stack[p];
    if (id < 0 || id >= a.num_blocks) bad = 1;
  }
  return __syncthreads_or(bad) ? SPEC_EINVAL : SPEC_OK;
}

// One launch, a cluster of CTAs. Every CTA checks everything for itself and keeps
// in shared memory, per sequence, its length and the rows, blocks to be popped and
// blocks with new rows before it; once all have read the state (cluster
// barrier), the blocks that hold new rows are dealt out, 16 lanes each: a
// block's number comes from the table (a part-filled last block) or directly
// from the stack, so nothing waits for a table entry.
__global__ void __launch_bounds__(kExtendThreads) extend_kernel(ExtendArgs a) {
  pdl_begin();
  extern __shared__ int s_seq[];  // [4][B + 1]
  int* s_len = s_seq;
  int* s_row = s_len + a.B + 1;
  int* s_pop = s_row + a.B + 1;
  int* s_blk = s_pop + a.B + 1;
  __shared__ int s_st0;
  if (threadIdx.x == 0) s_st0 = *(volatile int32_t*)a.status;
  const int bs = a.block_size, ft = *a.free_top;
  const int per = (a.B + blockDim.x - 1) / blockDim.x;
  const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
  longlong2 pre, tot;
  const int code = extend_check(a, b0, b1, ft, &pre, &tot);  // its barriers publish s_st0
  const bool run = s_st0 == SPEC_OK && code == SPEC_OK;      // the same in every CTA
  long long nblk = 0;
  if (run) {
    longlong2 cnt = make_longlong2(0, 0), all;
    for (int b = b0; b < b1; ++b) {
      const int len = a.seq_lens[b], add = a.add_len[b];
      if (add > 0) cnt.x += block_of(a, len + add - 1) - block_of(a, len) + 1;
    }
    const longlong2 before = block_excl_scan2(cnt, &all);
    nblk = all.x;
    int row = (int)pre.y, pop = (int)pre.x, blk = (int)before.x;
    for (int b = b0; b < b1; ++b) {
      const int len = a.seq_lens[b], add = a.add_len[b];
      s_len[b] = len;
      s_row[b] = row;
      s_pop[b] = pop;
      s_blk[b] = blk;
      row += add;
      pop += blocks_for(a, len + add) - blocks_for(a, len);
      if (add > 0) blk += block_of(a, len + add - 1) - block_of(a, len) + 1;
    }
    if (threadIdx.x == 0) s_row[a.B] = (int)tot.y;
  }
  // Every CTA has read lengths and stack height: new_lens and new_top may be theirs.
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (!run) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && s_st0 == SPEC_OK) set_status(a.status, code);
    return;
  }
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
      a.row_off[b] = s_row[b];
      a.new_lens[b] = s_len[b] + s_row[b + 1] - s_row[b];
    }
    if (threadIdx.x == 0) {
      a.row_off[a.B] = (int)tot.y;
      *a.new_top = ft - (int)tot.x;
    }
  }
  const int lane = threadIdx.x & 15;
  const int groups = gridDim.x * (blockDim.x / 16);
  constexpr int kAtOnce = 4;  // blocks of a group in flight: each waits for its number
  for (long long u0 = blockIdx.x * (blockDim.x / 16) + (threadIdx.x >> 4); u0 < nblk;
       u0 += (long long)groups * kAtOnce) {
    int seq[kAtOnce], i[kAtOnce], id[kAtOnce];
    bool fresh[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const long long u = u0 + (long long)k * groups;
      if (u >= nblk) continue;
      int lo = 0, hi = a.B - 1;  // the last sequence b with s_blk[b] <= u
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_blk[mid] <= u) lo = mid; else hi = mid - 1;
      }
      const int held = blocks_for(a, s_len[lo]);
      seq[k] = lo;
      i[k] = block_of(a, s_len[lo]) + (int)(u - s_blk[lo]);
      fresh[k] = i[k] >= held;
      id[k] = __ldcg(fresh[k] ? a.free_stack + (ft - 1 - (s_pop[lo] + i[k] - held))
                              : a.tables + (size_t)lo * a.max_blocks + i[k]);
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (u0 + (long long)k * groups >= nblk) continue;
      if (fresh[k] && lane == 0) a.tables[(size_t)seq[k] * a.max_blocks + i[k]] = id[k];
      if (!a.slot_map) continue;
      const int len = s_len[seq[k]], row = s_row[seq[k]], add = s_row[seq[k] + 1] - row;
      const int first = max(len, i[k] * bs);
      const int end = (int)min((long long)len + add, (i[k] + 1LL) * bs);
      for (int pos = first + lane; pos < end; pos += 16)
        a.slot_map[row + pos - len] = (long long)id[k] * bs + pos - i[k] * bs;
    }
  }
  if (a.slot_map)
    for (long long r = tot.y + (long long)blockIdx.x * blockDim.x + threadIdx.x; r < a.cap;
         r += (long long)gridDim.x * blockDim.x)
      a.slot_map[r] = -1;
}

// The plan of many rows or sequences: one CTA checks everything, then takes the
// missing blocks off the stack (sequences ascending, entries ascending), a warp per
// sequence, and writes lengths and offsets.
__global__ void __launch_bounds__(kExtendThreads) extend_plan_kernel(ExtendArgs a) {
  pdl_begin();
  extern __shared__ int s_seq[];  // [B] blocks popped for the sequences before
  __shared__ int s_st0;
  if (threadIdx.x == 0) s_st0 = *(volatile int32_t*)a.status;
  __syncthreads();
  if (s_st0 != SPEC_OK) return;
  const int per = (a.B + blockDim.x - 1) / blockDim.x;
  const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
  const int ft = *a.free_top;
  longlong2 pre, tot;
  const int code = extend_check(a, b0, b1, ft, &pre, &tot);
  if (code != SPEC_OK) {
    if (threadIdx.x == 0) set_status(a.status, code);
    return;
  }
  int pop = (int)pre.x, off = (int)pre.y;
  for (int b = b0; b < b1; ++b) {
    const int len = a.seq_lens[b], add = a.add_len[b];
    s_seq[b] = pop;
    pop += blocks_for(a, len + add) - blocks_for(a, len);
    a.row_off[b] = off;
    off += add;
  }
  __syncthreads();
  for (int b = threadIdx.x >> 5; b < a.B; b += blockDim.x >> 5) {
    const int len = a.seq_lens[b], held = blocks_for(a, len);
    const int n = blocks_for(a, len + a.add_len[b]) - held;
    int32_t* tab = a.tables + (size_t)b * a.max_blocks + held;
    for (int i = threadIdx.x & 31; i < n; i += 32)
      tab[i] = __ldcg(a.free_stack + (ft - 1 - (s_seq[b] + i)));
  }
  __syncthreads();  // new_lens may be seq_lens
  for (int b = b0; b < b1; ++b) a.new_lens[b] = a.seq_lens[b] + a.add_len[b];
  if (threadIdx.x == 0) {
    a.row_off[a.B] = (int)tot.y;
    *a.new_top = ft - (int)tot.x;
  }
}

// Slots of the new rows, -1 behind the last; after the plan.
__global__ void __launch_bounds__(kFillThreads) extend_fill_kernel(ExtendArgs a) {
  pdl_begin();
  if (*(volatile int32_t*)a.status != SPEC_OK) return;
  const int total = a.row_off[a.B];
  for (long long r = (long long)blockIdx.x * blockDim.x + threadIdx.x; r < a.cap;
       r += (long long)gridDim.x * blockDim.x) {
    long long slot = -1;
    if (r < total) {
      int lo = 0, hi = a.B - 1;  // the sequence b with row_off[b] <= r < row_off[b + 1]
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.row_off[mid] <= r) lo = mid; else hi = mid - 1;
      }
      const int pos = a.new_lens[lo] - (a.row_off[lo + 1] - (int)r);
      const int i = block_of(a, pos);
      slot = (long long)a.tables[(size_t)lo * a.max_blocks + i] * a.block_size + pos -
             i * a.block_size;
    }
    a.slot_map[r] = slot;
  }
}

// K and V rows to their slots: a warp per token, up to four 16-byte vectors of
// each row per lane in flight before the first is stored, loaded while the slot
// is looked up. Bound by HBM (each byte read and written once): 20000 rows of 8
// heads of 128 take 28.5 us, 5.8 TB/s (25.0 us at the measured copy rate); 64 rows
// 2.3 us, one warp's chain of two loads and a store, then the cluster's barrier.
constexpr int kStoreThreads = 256;
constexpr int kStoreRows = kStoreThreads / 32;  // rows of a CTA
constexpr int kStoreClusterRows = 8 * kStoreRows;

__device__ __forceinline__ bool bad_slot(const StoreArgs& a, long long slot) {
  return slot < -1 || slot >= (long long)a.num_blocks * a.block_size;
}

// Row t by one warp; returns whether its slot is bad.
__device__ __forceinline__ bool store_row(const StoreArgs& a, int t) {
  const int lane = threadIdx.x & 31;
  const int st0 = a.status ? *(volatile int32_t*)a.status : SPEC_OK;
  const long long slot = a.slot_map[t];
  const uint4* k = reinterpret_cast<const uint4*>(a.k + t * a.ld_k);
  const uint4* v = reinterpret_cast<const uint4*>(a.v + t * a.ld_v);
  const int n = a.row_bytes / 16;
  uint4 x[4], y[4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (lane + 32 * u < n) {
      x[u] = __ldcs(k + lane + 32 * u);
      y[u] = __ldcs(v + lane + 32 * u);
    }
  if (st0 != SPEC_OK || slot == -1) return false;
  if (bad_slot(a, slot)) return true;
  const long long slots = (long long)a.num_blocks * a.block_size;
  const long long block =
      slots <= INT32_MAX ? (uint32_t)slot / (uint32_t)a.block_size : slot / a.block_size;
  uint4* dst = reinterpret_cast<uint4*>(a.pool + block * a.page_bytes +
                                        (slot - block * a.block_size) * a.row_bytes);
  const long long to_v = (long long)a.block_size * n;  // V rows follow a block's K rows
  for (int i = lane;;) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + 32 * u < n) {
        dst[i + 32 * u] = x[u];
        dst[to_v + i + 32 * u] = y[u];
      }
    i += 128;
    if (i - lane >= n) break;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + 32 * u < n) {
        x[u] = __ldcs(k + i + 32 * u);
        y[u] = __ldcs(v + i + 32 * u);
      }
  }
  return false;
}

// A row is stored unless the status word held an error before the call, so the
// call's own error, of a bad slot, may appear there only once every row has read
// the word: after the barrier of the cluster that is the whole grid (up to
// kStoreClusterRows rows), else in a launch of its own (store_flag_kernel). 64 rows
// take 2.3 us with the barrier, 3.0 with the launch, and from Python, where the
// host is the limit, 7.1 and 8.9.
template <bool kCluster>
__global__ void __launch_bounds__(kStoreThreads) store_kv_kernel(StoreArgs a) {
  pdl_begin();
  const int t = blockIdx.x * kStoreRows + (threadIdx.x >> 5);
  const bool bad = t < a.T && store_row(a, t);
  if constexpr (kCluster) {
    __syncwarp();  // the barrier takes whole warps
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (bad && (threadIdx.x & 31) == 0) set_status(a.status, SPEC_EINVAL);
  }
}

// Flags bad slots after store_kv_kernel.
__global__ void __launch_bounds__(kStoreThreads) store_flag_kernel(StoreArgs a) {
  pdl_begin();  // every row has read the status word
  bool bad = false;
  for (long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x; t < a.T;
       t += (long long)gridDim.x * blockDim.x)
    bad |= bad_slot(a, a.slot_map[t]);
  if (bad) set_status(a.status, SPEC_EINVAL);
}

}  // namespace

// One launch for up to kClusterRows rows of slot map (a cluster of 8 CTAs, one CTA
// for up to kOneCtaRows), else a plan and a second launch that fills the map. 64
// sequences growing to rows in all, one launch against two: 1024 5.8 and 6.9 us, 4096
// 5.9 and 6.9, 8192 6.9 and 6.7, 16384 7.9 and 7.0, 147200 25.5 and 10.3, as a cluster
// has few SMs; 4096 sequences growing by a row 19.8 and 31.4. One CTA against eight:
// 512 rows 5.7 and 5.5, 1024 7.0 and 5.8.
constexpr long long kClusterRows = 8192, kOneCtaRows = 512;
constexpr int kClusterSeqs = 4096;  // whose records fit the cluster's shared memory

cudaError_t launch_extend(const ExtendArgs& a, cudaStream_t st) {
  if (a.B <= kClusterSeqs && a.cap <= kClusterRows) {
    const size_t smem = 4 * ((size_t)a.B + 1) * sizeof(int);
    const cudaError_t e = reserve_dyn_smem(extend_kernel, smem);
    if (e != cudaSuccess) return e;
    const unsigned ctas = a.cap <= kOneCtaRows ? 1 : 8;
    return launch_pdl_cluster(extend_kernel, dim3(ctas), dim3(kExtendThreads), smem, st, ctas, a);
  }
  const size_t smem = (size_t)a.B * sizeof(int);
  cudaError_t e = reserve_dyn_smem(extend_plan_kernel, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(extend_plan_kernel, dim3(1), dim3(kExtendThreads), smem, st, a);
  if (e != cudaSuccess || !a.slot_map || a.cap == 0) return e;
  const long long want = (a.cap + kFillThreads - 1) / kFillThreads;
  const unsigned grid = (unsigned)(want < sm_count() * 8 ? want : sm_count() * 8);
  return launch_pdl(extend_fill_kernel, dim3(grid), dim3(kFillThreads), 0, st, a);
}

cudaError_t launch_store_kv(const StoreArgs& a, cudaStream_t st) {
  if (a.status && a.T <= kStoreClusterRows) {
    const unsigned ctas = a.T <= kStoreRows ? 1 : kStoreClusterRows / kStoreRows;
    return launch_pdl_cluster(store_kv_kernel<true>, dim3(ctas), dim3(kStoreThreads), 0, st, ctas,
                              a);
  }
  const unsigned grid = (unsigned)((a.T + (long long)kStoreRows - 1) / kStoreRows);
  const cudaError_t e =
      launch_pdl(store_kv_kernel<false>, dim3(grid), dim3(kStoreThreads), 0, st, a);
  if (e != cudaSuccess || !a.status) return e;
  const long long want = (a.T + (long long)kStoreThreads - 1) / kStoreThreads;
  const unsigned flags = (unsigned)(want < sm_count() ? want : sm_count());
  return launch_pdl(store_flag_kernel, dim3(flags), dim3(kStoreThreads), 0, st, a);
}

}  // namespace specv
