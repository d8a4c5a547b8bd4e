// Arguments and launchers of the paged-cache operators: growing block tables
// with their slot map, and storing K/V rows in the pool.
#pragma once
#include "attend_plan.cuh"
#include "common.cuh"

namespace specv {

struct ExtendArgs {
  int B, block_size, max_blocks, num_blocks;
  FastDiv by_bs;      // division by block_size
  int32_t* tables;
  const int32_t* seq_lens;
  const int32_t* add_len;
  const int32_t* free_stack;
  const int32_t* free_top;
  int32_t* new_lens;  // may be seq_lens
  int32_t* new_top;   // may be free_top
  int32_t* row_off;
  int64_t* slot_map;
  long long cap;
  int32_t* status;
};
cudaError_t launch_extend(const ExtendArgs& a, cudaStream_t st);

struct StoreArgs {
  const unsigned char* k;
  const unsigned char* v;
  long long ld_k, ld_v;  // bytes between token rows
  int T;
  const int64_t* slot_map;
  unsigned char* pool;   // at (block 0, layer, K)
  long long page_bytes;  // one block: layers * 2 * block_size * row_bytes
  int row_bytes;         // kv_heads * head_dim * 2
  int block_size, num_blocks;
  int32_t* status;
};
cudaError_t launch_store_kv(const StoreArgs& a, cudaStream_t st);

}  // namespace specv
