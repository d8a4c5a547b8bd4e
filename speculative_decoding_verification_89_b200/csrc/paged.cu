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

__device__ __forceinline__ long long blocks_for(long long n, int bs) { return (n + bs - 1) / bs; }

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

// One CTA checks everything, then takes the missing blocks off the stack
// (sequences ascending, entries ascending) and writes lengths and offsets. The
// order of the pops couples all sequences, hence the single CTA.
__global__ void __launch_bounds__(kExtendThreads) extend_plan_kernel(ExtendArgs a) {
  pdl_begin();
  __shared__ int s_code, s_bad, s_st0;
  if (threadIdx.x == 0) {
    s_st0 = *(volatile int32_t*)a.status;
    s_bad = 0;
    s_code = SPEC_OK;
  }
  __syncthreads();
  if (s_st0 != SPEC_OK) return;
  const int bs = a.block_size;
  const int per = (a.B + blockDim.x - 1) / blockDim.x;
  const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
  const int ft = *a.free_top;
  longlong2 cnt = make_longlong2(0, 0);  // missing blocks, new rows
  int bad = 0;
  for (int b = b0; b < b1; ++b) {
    const int len = a.seq_lens[b], add = a.add_len[b];
    if (len < 0 || add < 0 || blocks_for((long long)len + add, bs) > a.max_blocks ||
        (long long)len + add > INT32_MAX) {
      bad = 1;
      continue;
    }
    const int held = (int)blocks_for(len, bs);
    if (add > 0 && held * (long long)bs > len) {  // rows go into the held last block
      const int id = a.tables[(size_t)b * a.max_blocks + held - 1];
      if (id < 0 || id >= a.num_blocks) bad = 1;
    }
    cnt.x += blocks_for((long long)len + add, bs) - held;
    cnt.y += add;
  }
  if (bad) s_bad = 1;
  longlong2 tot;
  const longlong2 pre = block_excl_scan2(cnt, &tot);  // its barriers publish s_bad
  if (threadIdx.x == 0) {
    if (s_bad || ft < 0 || ft > a.num_blocks || tot.y > INT32_MAX ||
        (a.slot_map && tot.y > a.cap))
      s_code = SPEC_EINVAL;
    else if (tot.x > ft)
      s_code = SPEC_ENOBLOCKS;
  }
  __syncthreads();
  if (s_code == SPEC_OK) {  // popped ids must be valid
    bad = 0;
    for (int p = ft - (int)tot.x + threadIdx.x; p < ft; p += blockDim.x) {
      const int id = a.free_stack[p];
      if (id < 0 || id >= a.num_blocks) bad = 1;
    }
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0) s_code = SPEC_EINVAL;
  }
  __syncthreads();
  if (s_code != SPEC_OK) {
    if (threadIdx.x == 0) set_status(a.status, s_code);
    return;
  }
  int k = (int)pre.x, off = (int)pre.y;
  for (int b = b0; b < b1; ++b) {
    const int len = a.seq_lens[b], add = a.add_len[b];
    int32_t* tab = a.tables + (size_t)b * a.max_blocks;
    const int held = (int)blocks_for(len, bs), need = (int)blocks_for((long long)len + add, bs);
    for (int i = held; i < need; ++i) tab[i] = a.free_stack[ft - 1 - k++];
    a.row_off[b] = off;
    off += add;
    a.new_lens[b] = len + add;
  }
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
      slot = (long long)a.tables[(size_t)lo * a.max_blocks + pos / a.block_size] * a.block_size +
             pos % a.block_size;
    }
    a.slot_map[r] = slot;
  }
}

// K and V rows to their slots: a warp per row, 16 bytes per lane and access.
constexpr int kStoreThreads = 256;
__global__ void __launch_bounds__(kStoreThreads) store_kv_kernel(StoreArgs a) {
  pdl_begin();
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * (kStoreThreads / 32) + (threadIdx.x >> 5);
  if (item >= 2LL * a.T) return;
  if (a.status && *(volatile int32_t*)a.status != SPEC_OK) return;
  const int t = (int)(item >> 1), part = (int)(item & 1);
  const long long slot = a.slot_map[t];
  if (slot == -1) return;
  if (slot < -1 || slot >= (long long)a.num_blocks * a.block_size) {
    if (lane == 0) set_status(a.status, SPEC_EINVAL);
    return;
  }
  const long long block = slot / a.block_size;
  const int row = (int)(slot - block * a.block_size);
  const uint4* src = reinterpret_cast<const uint4*>(part ? a.v + t * a.ld_v : a.k + t * a.ld_k);
  uint4* dst = reinterpret_cast<uint4*>(a.pool + block * a.page_bytes +
                                        ((long long)part * a.block_size + row) * a.row_bytes);
  for (int i = lane; i < a.row_bytes / 16; i += 32) dst[i] = __ldcs(src + i);
}

}  // namespace

cudaError_t launch_extend(const ExtendArgs& a, cudaStream_t st) {
  cudaError_t e = launch_pdl(extend_plan_kernel, dim3(1), dim3(kExtendThreads), 0, st, a);
  if (e != cudaSuccess || !a.slot_map || a.cap == 0) return e;
  const long long want = (a.cap + kFillThreads - 1) / kFillThreads;
  const unsigned grid = (unsigned)(want < sm_count() * 8 ? want : sm_count() * 8);
  return launch_pdl(extend_fill_kernel, dim3(grid), dim3(kFillThreads), 0, st, a);
}

cudaError_t launch_store_kv(const StoreArgs& a, cudaStream_t st) {
  const long long items = 2LL * a.T;
  const unsigned grid = (unsigned)((items + kStoreThreads / 32 - 1) / (kStoreThreads / 32));
  return launch_pdl(store_kv_kernel, dim3(grid), dim3(kStoreThreads), 0, st, a);
}

}  // namespace specv
