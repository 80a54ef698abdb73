// Internal interface between the differential-attention entry points (diff_api.cu) and
// their kernels (attn_diff.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace xs {

// What a unit costs beside its KV tiles (its first loads and its epilogue), in tiles: 2 at d = 64, 3
// to 4 at 128 and 256. In the split schedule a unit takes so many places more than it has tiles.
constexpr int kUnitCost = 3;
// Rows of a tile up to which a merge is spread over columns and pieces.
constexpr int kFewRows = 8;

struct DiffParams {
  // q [B][H][Nq][d], k and v [B][Hk][Nk][d], any strides: 4-D maps {d, rows, heads, batch},
  // box {64, 128, 1, 1}, 128-byte swizzle.
  CUtensorMap tm_q, tm_k, tm_v;
  void *shards[kMaxShards];           // shard_mode 1: [B][Nq/P][H][d] each
  void *o;                            // shard_mode 0: strides in elements
  long long o_b, o_h, o_n;
  const float *lambda;                // [H]
  const float *weight;                // [d] or null: no norm
  const int *kv_len;                  // [B] or null: Nk keys everywhere
  int B, H, group, Nq, Nk;            // group: query heads per k/v head
  int shard_mode, rows_per_shard;
  int n_qtiles, v_parts;              // 128-row query tiles; halves of v's columns (2 at d = 256)
  int units_b, n_units;               // units of a batch entry (H * n_qtiles * v_parts), of all
  // Work list of a CTA (G = gridDim.x): units blockIdx.x + k*G, all of them (split = 0) or the
  // first `waves` (split = 1); then the KV tiles of the remaining units, unit-major, in contiguous
  // ranges of equal cost.
  int split, waves;
  int min_places;                     // shortest range worth a CTA
  float scale_log2, eps, out_scale;
  float *parts;                       // split: [G][2 slots] partial results
  int *count;                         // split: pieces done of the unit that begins in CTA c's range
  // The d = 256 kernel: rows of a tile's partial results (Nq up to 128), and where map 1 of a whole
  // unit waits for map 2: [G][256 columns][part_rows] fp32.
  int part_rows;
  float *stash;
  int *status;
  unsigned long long wait_limit_ns;
};

int diff_part_floats(int d);          // fp32 values of one piece's partial result
cudaError_t launch_attn_diff(const DiffParams &p, int d, int grid, cudaStream_t s);
cudaError_t launch_diff_zero(const DiffParams &p, int d, int grid, cudaStream_t s);   // no keys at all
// d = 256 with a workspace.
int diff_wide_part_floats(int rows);
cudaError_t launch_attn_diff_wide(const DiffParams &p, int grid, cudaStream_t s);

}  // namespace xs
