// Arguments and launchers of the attention operators.
#pragma once
#include <cuda.h>

#include "attend_plan.cuh"
#include "common.cuh"

namespace specv {

constexpr int kAttendMaxCtas = 148;
constexpr int kAttendMaxGroup = kTileRows;  // query heads that share a K/V head

struct AttendArgs {
  int B, T, q_heads, kv_heads, group, dim;
  int dtype;          // SPEC_BF16 or SPEC_F16
  AttendShape shape;
  FastDiv by_group, by_bs;  // division by group, block_size
  int rows_per_seq;   // rows of each sequence where row_off is NULL
  const int32_t* row_off;
  float scale_log2;   // scale * log2(e)
  const unsigned char* q;
  long long ld_q;     // bytes between token rows
  unsigned char* out;
  long long ld_out;
  float* lse;
  // keys and values: packed rows (tables NULL), or the pool at (block 0, layer)
  const unsigned char* k;
  const unsigned char* v;
  long long ld_k, ld_v;   // bytes between token rows (packed), or between a block's rows
  long long page_bytes;   // bytes between blocks
  const int32_t* tables;
  const int32_t* seq_lens;
  int max_blocks, num_blocks, block_size;
  // the new rows' own keys and values, staged (NULL: they are in the pool)
  const unsigned char* stage_k;
  const unsigned char* stage_v;
  long long stage_seq, stage_row;  // bytes between sequences, rows
  int stage_rows;
  int32_t* status;
  float* part_o;     // [2 * ctas][2][DP / 4][kTileRows][4] unnormalised
  float2* part_ml;   // [2 * ctas][2 * kTileRows] (maximum in log2 units, sum)
  int32_t* counts;   // [ctas] parts written of the unit that CTA begins; 0 between calls
  int ctas;
  int stop_cta;       // test: the CTA that issues nothing, -1 for none
  bool out_sectors;   // rows of heads in out begin on 32-byte boundaries
  // Tensors for tiled copies of 64 columns; those of K and V have box_rows rows,
  // 0: the pages fit no box and rows are copied one by one.
  int box_rows;
  CUtensorMap map_q, map_k, map_v;
};
// Forms the maps.
cudaError_t attend_maps(AttendArgs* a);
// Workspace: the counts first, in the same place for all head sizes (one
// workspace may serve calls of several), then the parts, rows padded to DP columns.
struct AttendWs {
  size_t ml, o, total;
};
inline int attend_padded_dim(int dim) { return dim <= 64 ? 64 : 128; }
inline AttendWs attend_ws(int dim) {
  const size_t rows = (size_t)2 * kAttendMaxCtas * 2 * kTileRows;
  AttendWs w;
  w.ml = (kAttendMaxCtas * sizeof(int32_t) + 255) & ~(size_t)255;
  w.o = w.ml + rows * sizeof(float2);
  w.total = w.o + rows * attend_padded_dim(dim) * sizeof(float);
  return w;
}
cudaError_t launch_attend(const AttendArgs& a, cudaStream_t st);

}  // namespace specv
