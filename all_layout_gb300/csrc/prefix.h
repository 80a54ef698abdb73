// Internal interface between the shared-prefix attention entry points (prefix_api.cu) and
// their kernels (attn_prefix.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "cache.h"
#include "internal.h"

namespace xs {

// Batch entries of one launch: their places among the packed own keys lie in shared memory.
constexpr int kPrefixEntries = 256;
// Division of n in [0, 2^31) by a fixed d: with l the least l for which d <= 2^l, n m >> (31 + l) for
// m = ceil(2^(31 + l) / d). (A plain division is some forty instructions, and a launch's first ones wait
// for instructions more than for anything else.)
struct Divisor {
  unsigned m, shift;   // m = 0: d = 1
  void set(unsigned d) {
    unsigned l = 0;
    while ((1ull << l) < d) ++l;
    m = d > 1 ? static_cast<unsigned>(((1ull << (31 + l)) + d - 1) / d) : 0;
    shift = l > 0 ? l - 1 : 0;
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int of(int n) const {
    return m ? static_cast<int>(__umulhi(static_cast<unsigned>(n), m) >> shift) : n;
  }
#endif
};

// What the schedule goes by; the kernels keep a copy in shared memory for the calls that walk it.
struct PrefixGeo {
  int rows, entry_rows;                  // rows of a k/v head: (entry, head of the group, query padded to nq_rows)
  int row_tile, n_tiles, n_units;        // rows of a unit; units of a head, of all
  int n_prefix;                          // 128-key tiles of the prefix
  int split, waves, min_places;          // see PrefixWalk
  int unit_cost, own_cost;               // see place_of; own_cost <= min_places
  Divisor by_entry, by_tiles;            // entry_rows, n_tiles
};

struct PrefixParams : PrefixGeo {
  // Keys and values that lie in tensors: the prefix [Hk][Np][d], the own ones [B][Hk][Nk][d], any
  // strides: maps {d, rows, heads, batch} with boxes of 64 columns and 128 rows, 128-byte swizzle; the flat
  // kernel's own ones also with boxes of 16 rows. The tall kernel's queries: boxes of 8 rows.
  CUtensorMap tm_q, tm_pk, tm_pv, tm_k, tm_v, tm_k16, tm_v16;
  // The flat kernel's cached keys, two codes as one element: map {d / 2, rows of a page, heads, pages}, boxes of a page's
  // rows, 128 at most, and of 16; the swizzle is as wide as a row.
  CUtensorMap tm_c, tm_c16;
  // Those that lie in the cache.
  PageLists prefix_pages, own_pages;
  const uint8_t *codes[2], *scales[2];   // of k and v
  int prefix_cached, own_cached;
  const uint16_t *q;                     // [B][H][Nq][d], strides in elements
  long long q_b, q_h, q_n;
  void *shards[kMaxShards];              // shard_mode 1: [all batches][Nq/P][H][d] each
  uint16_t *o;                           // shard_mode 0: strides in elements
  long long o_b, o_h, o_n;
  int shard_mode, rows_per_shard;
  const int *kv_len;                     // [B] or null: Nk keys everywhere
  int b0, B;                             // the launch's batch entries; q, o, kv_len and the own pages begin at b0
  int H, Hk, group, Nq, Np, Nk;          // group: query heads per k/v head
  int nq_rows;                           // entry_rows >= group * nq_rows, rows = B * entry_rows
  Divisor by_nq, by_shard;               // nq_rows, rows_per_shard
  int copies;                            // flat kernel: copies of a unit's rows in its 128 lanes
  int grain;                             // own keys of an entry begin at multiples of this among the packed ones
  float scale_log2;
  float *parts;                          // split: [grid][2 slots] partial results
  int4 *cuts;                            // split: what the join is to do (cut_place)
  int grid;                              // CTAs of the launch
  int *status;
  unsigned long long wait_limit_ns;
};

int prefix_part_floats(int d, int rows);   // fp32 values of one piece's partial result
// Few rows for each k/v head: one 128-lane tile of rows at a time, two KV tiles in turn.
cudaError_t launch_prefix_flat(const PrefixParams &p, int d, int grid, cudaStream_t s);
// Many rows: pairs of 128-row tiles; keys and values in tensors.
cudaError_t launch_prefix_tall(const PrefixParams &p, int d, int grid, cudaStream_t s);
// Joins the pieces of cut units, after a launch of `grid` CTAs that had split set; sms: of the device.
cudaError_t launch_prefix_join(const PrefixParams &p, int d, int grid, int sms, cudaStream_t s);

}  // namespace xs
