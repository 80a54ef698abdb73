// Attention of a batch of requests that share a prefix, for sm_103a (tcgen05 tensor cores,
// Tensor Memory, TMA).
//
// Per request b and query head h, whose k/v head is hk:
//     o = softmax(q [K_p | K_b]^T s) [V_p | V_b],   s the caller's scale,
// K_p, V_p [Np][d] the same for every request, K_b, V_b [kv_len[b]][d] its own; both in bf16
// tensors or in pages of an e4m3 cache (cache.cu). A row without any key gives zeros.
//
// Rows. The queries of all requests and of all heads that share a k/v head are the rows of one
// matrix, [entry][head of the group][query], cut into tiles: each key of the prefix is read
// once for a whole tile of them, whatever requests they belong to.
// Keys. The own keys of all requests are packed one after the other, each request's beginning
// at a multiple of `grain`; 128 of them are a KV tile, which may hold several short requests'.
// A unit (k/v head, tile of rows) goes over the prefix's tiles and then those that hold its
// requests' own keys; a row sees the range [lo, hi) of the packed keys, and what lies outside
// gets the score -inf.
//
// Schedule: persistent CTAs take whole units, strided; with a workspace the units past the last
// full wave but one are cut into contiguous ranges of KV tiles of equal cost. A cut unit's
// pieces leave (m, l, O) in the workspace, and a second launch joins them in piece order.
// Lengths are on the device, so each CTA works out its range itself.
//
// Waits are bounded: a role that gives up records a timeout; the softmax warps then run their
// control flow to its end without waiting, the others drain what they issued.
#include <cfloat>
#include <climits>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "../../include/xs.h"
#include "internal.h"
#include "prefix.h"
#include "ptx.cuh"

namespace xs {
namespace {

constexpr int BM = kTileRows, BN = kTileRows;
constexpr int kHalf = BM * 128;   // one 64-column half of a 128-row tile
constexpr uint32_t kSleepNs = 100000;
constexpr float kGrowth = 8.0f;   // log2 units: rescale O only when the maximum grows by more than 2^8

// ------------------------------------------------------------------ schedule
__device__ __forceinline__ int keys_of(const PrefixParams &p, int b) {
  return p.kv_len ? min(max(__ldg(p.kv_len + b), 0), p.Nk) : p.Nk;
}

// Table in shared memory: where each entry's own keys begin among the packed ones ([B]: their end), and
// from kLens on how many each has.
constexpr int kLens = kPrefixEntries + 4, kTable = 2 * kLens;
__device__ __forceinline__ int len_of(const int *table, int b) { return table[kLens + b]; }

// Fills the table, by one warp.
__device__ void pack_keys(const PrefixParams &p, int *start) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  for (int b = lane; b - lane < p.B; b += 32) {
    const int len = b < p.B ? keys_of(p, b) : 0, mine = (len + p.grain - 1) / p.grain * p.grain;
    int incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (b < p.B) {
      start[b] = base + incl - mine;
      start[kLens + b] = len;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) start[p.B] = base;
}

struct PrefixUnit {
  int unit, hk, row0;   // first row of the k/v head's rows
  int b_lo, b_hi;       // entries of its rows
  int t0, n;            // first own tile; tiles, the prefix's first
};
__device__ __forceinline__ PrefixUnit unit_of(const PrefixGeo &p, const int *start, int unit) {
  PrefixUnit u;
  u.unit = unit;
  u.hk = p.by_tiles.of(unit);
  u.row0 = (unit - u.hk * p.n_tiles) * p.row_tile;
  u.b_lo = p.by_entry.of(u.row0);
  u.b_hi = p.by_entry.of(min(u.row0 + p.row_tile, p.rows) - 1);
  const int s = start[u.b_lo], e = start[u.b_hi + 1];
  u.t0 = s / BN;
  // (Rows without any key keep a tile, fully masked, that gives their zeros.)
  u.n = max(1, p.n_prefix + (e > s ? (e + BN - 1) / BN - u.t0 : 0));
  return u;
}

// The split region: its places (unit_cost for a unit, then one for each of the prefix's tiles and own_cost for
// each own one, which begins at the first of them), the CTAs that share it, and the unit where this CTA begins
// in it.
__device__ __forceinline__ unsigned place_of(const PrefixGeo &p, int tile) {
  return tile <= p.n_prefix ? tile : p.n_prefix + (tile - p.n_prefix) * static_cast<unsigned>(p.own_cost);
}
// The first tile that begins at a place or behind it.
__device__ __forceinline__ int tile_at(const PrefixGeo &p, unsigned place) {
  const unsigned np = p.n_prefix, each = p.own_cost;
  return static_cast<int>(place <= np ? place : np + (place - np + each - 1) / each);
}
__device__ __forceinline__ unsigned places_of(const PrefixGeo &p, int n) { return p.unit_cost + place_of(p, n); }
struct PrefixPlan {
  unsigned total, per;   // places; of a CTA
  unsigned begin;        // first place of `unit`
  int unit;
};

struct PrefixItem : PrefixUnit {
  int kv0, kv1;     // KV tiles to do
  unsigned u0;      // a cut unit: its first tile's place in the split region
  bool piece;
};

// Walks a CTA's work list; every role walks its own copy.
struct PrefixWalk {
  int k, unit;
  unsigned pos, end, begin;

  __device__ __forceinline__ void start(const PrefixGeo &p, const PrefixPlan &plan) {
    k = 0;
    pos = end = 0;
    if (p.split) {
      pos = min(blockIdx.x * plan.per, plan.total);
      end = min(pos + plan.per, plan.total);
    }
    unit = plan.unit;
    begin = plan.begin;
  }
  __device__ __forceinline__ bool next(const PrefixGeo &p, const int *table, PrefixItem &it) {
    if (!p.split || k < p.waves) {
      const int u = static_cast<int>(blockIdx.x) + k * static_cast<int>(gridDim.x);
      ++k;
      if (u >= p.n_units) return false;
      static_cast<PrefixUnit &>(it) = unit_of(p, table, u);
      it.kv0 = 0;
      it.kv1 = it.n;
      it.u0 = 0;
      it.piece = false;
      return true;
    }
    while (pos < end) {
      static_cast<PrefixUnit &>(it) = unit_of(p, table, unit);
      const unsigned past = begin + places_of(p, it.n);
      if (pos < past) {
        it.u0 = begin + p.unit_cost;
        if (end <= it.u0) break;   // the range ends before the unit's first tile
        it.kv0 = pos > it.u0 ? tile_at(p, pos - it.u0) : 0;
        it.kv1 = min(tile_at(p, end - it.u0), it.n);
        it.piece = it.kv0 > 0 || it.kv1 < it.n;
        pos = min(end, past);
        if (it.kv0 < it.kv1) return true;
        continue;   // behind the beginning of the unit's last tile
      }
      begin = past;
      ++unit;
    }
    pos = end;
    return false;
  }
};

// The schedule in shared memory: its geometry, and where a CTA begins, which one warp works out for all.
struct PrefixStart {
  PrefixGeo geo;
  PrefixPlan plan;
  PrefixWalk walk;    // past `item`
  PrefixItem item;
  int any;            // whether there is an item
};
static_assert(sizeof(PrefixStart) <= 192, "room in shared memory");
// A call with memory of its own, so that neither walk nor item takes registers between items.
__device__ __noinline__ bool next_item(const PrefixStart *start, const int *table, PrefixWalk *walk, PrefixItem *item) {
  return walk->next(start->geo, table, *item);
}

// The split region's size and this CTA's place in it, by one warp.
__device__ PrefixPlan plan_split(const PrefixParams &p, const int *table) {
  const int lane = threadIdx.x & 31, first = p.waves * static_cast<int>(gridDim.x);
  auto size_of = [&](int u) -> unsigned { return u < p.n_units ? places_of(p, unit_of(p, table, u).n) : 0; };
  unsigned total = 0;
  for (int u = first + lane; u < p.n_units; u += 32) total += size_of(u);
  total = __reduce_add_sync(0xffffffffu, total);
  // (Lengths up to 2^29 are 2^22 tiles, own ones two places each, and there are fewer than two units for each CTA here:
  // with 152 of them no place, and no multiple of `per`, reaches 2^32.)
  PrefixPlan plan{total, max((total + gridDim.x - 1) / gridDim.x, static_cast<unsigned>(p.min_places)), 0, first};
  const unsigned pos = blockIdx.x * plan.per;
  if (pos >= total) return plan;
  unsigned base = 0;
  for (int u = first;; u += 32) {   // the unit that holds pos; ends, as pos < total
    const unsigned mine = size_of(u + lane);
    unsigned incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned past = __ballot_sync(0xffffffffu, pos < base + incl);
    if (past) {
      const int at = __ffs(past) - 1;
      plan.begin = base + __shfl_sync(0xffffffffu, incl - mine, at);
      plan.unit = u + at;
      return plan;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// Fills the table and the start, by one warp.
__device__ __forceinline__ void begin_schedule(const PrefixParams &p, int *table, PrefixStart *start) {
  pack_keys(p, table);
  __syncwarp();
  PrefixPlan plan{0, 1, 0, 0};
  if (p.split) plan = plan_split(p, table);
  if ((threadIdx.x & 31) == 0) {
    start->geo = p;
    start->plan = plan;
    PrefixWalk walk;
    PrefixItem item = {};
    walk.start(p, plan);
    start->any = walk.next(p, table, item);
    start->walk = walk;
    start->item = item;
  }
}

// Where the join finds the unit that begins in this CTA's range: with no more units than CTAs in the split
// region a place for each unit (the join is then launched for so many), else one for each CTA.
__device__ __forceinline__ bool cut_by_unit(const PrefixGeo &p) {
  return p.n_units - p.waves * static_cast<int>(gridDim.x) <= static_cast<int>(gridDim.x);
}
__device__ __forceinline__ int4 *cut_place(const PrefixParams &p, int unit) {
  return p.cuts + (cut_by_unit(p) ? unit - p.waves * static_cast<int>(gridDim.x) : static_cast<int>(blockIdx.x));
}
// How many consecutive CTAs, from the one that begins the unit, its pieces run on.
// (No range between is without a tile, as none is shorter than own_cost.)
__device__ __forceinline__ int pieces_of(const PrefixGeo &p, const PrefixPlan &plan, unsigned u0, int n) {
  return static_cast<int>((u0 + place_of(p, n - 1)) / plan.per - u0 / plan.per) + 1;
}

// One row of a k/v head's rows; n >= Nq or h past the k/v head's: padding.
struct PrefixRow {
  int b, h, n;
};
__device__ __forceinline__ PrefixRow row_of(const PrefixParams &p, int hk, int row) {
  PrefixRow r;
  r.b = p.by_entry.of(row);
  const int in = row - r.b * p.entry_rows, g = p.by_nq.of(in);
  r.h = hk * p.group + g;
  r.n = in - g * p.nq_rows;
  return r;
}
// Where a row's output begins; null for padding.
__device__ __forceinline__ uint16_t *out_row(const PrefixParams &p, int hk, int row, int d) {
  if (row >= p.rows) return nullptr;
  const PrefixRow r = row_of(p, hk, row);
  if (r.n >= p.Nq || r.h >= (hk + 1) * p.group) return nullptr;
  if (p.shard_mode) {
    const int sh = p.by_shard.of(r.n), i = r.n - sh * p.rows_per_shard;
    return static_cast<uint16_t *>(p.shards[sh]) +
           ((static_cast<long long>(p.b0 + r.b) * p.rows_per_shard + i) * p.H + r.h) * d;
  }
  return p.o + r.b * p.o_b + r.h * p.o_h + r.n * p.o_n;
}
// The range of keys that a row sees: of the prefix [0, Np), of the packed own ones [lo, hi).
struct PrefixRange {
  int lo, hi;
};
__device__ __forceinline__ PrefixRange range_of(const PrefixParams &p, const int *table, int row) {
  if (row >= p.rows) return PrefixRange{0, 0};
  const int b = p.by_entry.of(row), s = table[b];
  return PrefixRange{s, s + len_of(table, b)};
}

// Partial result of a piece: O as float4 groups [column / 4][lane], then the lanes' maxima and sums. (A lane is
// a row, or one copy of it.)
template <int D>
__device__ __forceinline__ float *part_of(const PrefixParams &p, int cta, int slot, int rows) {
  return p.parts + (static_cast<size_t>(cta) * 2 + slot) * ((D + 2) * rows);
}

// ------------------------------------------------------------------ waits
// Bounded wait on a barrier phase; false after a timeout here or elsewhere in the CTA.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *status,
                                       uint64_t limit, bool sleepy) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (sleepy ? mbar_try_wait_sleep(bar, parity, kSleepNs) : mbar_try_wait(bar, parity)) return true;
    if ((it & 15u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > limit) {
        *abort_flag = 1;
        atomicExch(status, kDevTimeout);
        return false;
      }
    }
  }
}
template <bool SLEEPY>
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                         const PrefixParams &p) {
  const bool ok = mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort_flag, p.status, p.wait_limit_ns, SLEEPY);
  return __all_sync(0xffffffffu, ok);
}
// Tear-down: waits for this thread's own copies or MMAs in flight, whatever the abort flag, still bounded.
__device__ __noinline__ void drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > 2000000000ull) return;
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
// `bytes` (a multiple of 16) of memory into shared memory, both 16-byte aligned.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// The wait for tmem_ld16, naming its registers so that no use of them moves before it.
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// ------------------------------------------------------------------ MMAs
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t dcol, uint64_t qdesc, uint64_t kdesc) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, 0);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint64_t off = static_cast<uint64_t>(((kk / 4) * kHalf + (kk % 4) * 32) >> 4);
    tc_mma_ss(dcol, qdesc + off, kdesc + off, idesc, kk > 0 ? 1u : 0u);
  }
}
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t dcol, uint32_t pcol, uint64_t vdesc, uint32_t accumulate) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, D, 1);
#pragma unroll
  for (int kk = 0; kk < BN / 16; ++kk)
    tc_mma_ts(dcol, pcol + kk * 8, vdesc + static_cast<uint64_t>((kk * 2048) >> 4), idesc,
              (kk > 0 || accumulate) ? 1u : 0u);
}

#include "attn_prefix_flat.cuh"
#include "attn_prefix_tall.cuh"

// ------------------------------------------------------------------ joining pieces
// The pieces of the unit that begins in CTA blockIdx.x's range: 32 rows (blockIdx.y) and a slice of the columns
// (blockIdx.z of gridDim.z) a block, a lane per row. The eight warps share the parts and the groups of eight
// columns between them: with few parts a warp takes all of them, with many each takes every eighth. Six parts
// are under way at a time and joined with a running maximum, the warps' sums in order, so the result does not
// depend on the order in which the pieces ended. Bound by the latency of its loads: from cold
// memory 8.5 us for the pieces of 24 units of 16 rows (11 MB), 21 us for 38 MB of pieces of 256 rows.
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ PrefixParams p) {
  constexpr int U = 6;   // parts under way
  __shared__ float sums[kJoinWarps][10][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int row = blockIdx.y * 32 + lane;
  const int R = p.row_tile > BM ? p.row_tile : BM;
  const int groups = D / 8 / gridDim.z;   // of columns
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 cut = __ldcg(p.cuts + blockIdx.x);   // first CTA, pieces (0: not cut), k/v head, first row
  // (The places are of the launch before, but for a CTA that gave up: nothing is taken on trust.)
  if (cut.y <= 0 || cut.x < 0 || cut.y > p.grid - cut.x || cut.z < 0 || cut.z >= p.Hk || cut.w < 0 ||
      cut.w + static_cast<int>(blockIdx.y) * 32 >= p.rows)
    return;
  // Part k: copy k mod copies of piece k / copies.
  const int step = p.copies == 4 ? 2 : p.copies - 1, parts = cut.y << step;
  int shared = parts <= 4 ? 1 : parts <= 8 ? 2 : parts <= 16 ? 4 : 8;   // warps that share the parts of a group
  if (shared * groups < kJoinWarps) shared = kJoinWarps / groups;
  const int pw = warp & (shared - 1), others = kJoinWarps / shared;
  uint16_t *dst = row < p.row_tile ? out_row(p, cut.z, cut.w + row, D) : nullptr;
#pragma unroll 1
  for (int g = warp / shared; g < groups; g += others) {   // (as many turns for each warp)
    const int c8 = blockIdx.z * groups + g;
    float m = -INFINITY, x[9];
#pragma unroll
    for (int i = 0; i < 9; ++i) x[i] = 0.f;
#pragma unroll 1
    for (int k0 = pw; k0 < parts; k0 += U * shared) {
      float mk[U], l[U];
      float4 a[U], b[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int k = min(k0 + i * shared, parts - 1);
        const float *q = part_of<D>(p, cut.x + (k >> step), k >> step == 0 ? 1 : 0, R);
        const int at = (k & (p.copies - 1)) * p.row_tile + row;
        mk[i] = __ldcg(q + D * R + at);
        l[i] = __ldcg(q + (D + 1) * R + at);
        a[i] = __ldcg(reinterpret_cast<const float4 *>(q) + (2 * c8) * R + at);
        b[i] = __ldcg(reinterpret_cast<const float4 *>(q) + (2 * c8 + 1) * R + at);
      }
      const float before = m;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (k0 + i * shared >= parts) mk[i] = -INFINITY;
        m = fmaxf(m, mk[i]);
      }
      const float keep = shrink(before, m);
#pragma unroll
      for (int i = 0; i < 9; ++i) x[i] *= keep;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (k0 + i * shared >= parts) break;
        const float f = shrink(mk[i], m);
        x[0] = fmaf(f, a[i].x, x[0]);
        x[1] = fmaf(f, a[i].y, x[1]);
        x[2] = fmaf(f, a[i].z, x[2]);
        x[3] = fmaf(f, a[i].w, x[3]);
        x[4] = fmaf(f, b[i].x, x[4]);
        x[5] = fmaf(f, b[i].y, x[5]);
        x[6] = fmaf(f, b[i].z, x[6]);
        x[7] = fmaf(f, b[i].w, x[7]);
        x[8] = fmaf(f, l[i], x[8]);
      }
    }
    if (shared > 1) {
#pragma unroll
      for (int i = 0; i < 9; ++i) sums[warp][i][lane] = x[i];
      sums[warp][9][lane] = m;
      __syncthreads();
      if (pw == 0) {
        for (int w = warp; w < warp + shared; ++w) m = fmaxf(m, sums[w][9][lane]);
#pragma unroll
        for (int i = 0; i < 9; ++i) x[i] = 0.f;
        for (int w = warp; w < warp + shared; ++w) {
          const float f = shrink(sums[w][9][lane], m);
#pragma unroll
          for (int i = 0; i < 9; ++i) x[i] = fmaf(f, sums[w][i][lane], x[i]);
        }
      }
      __syncthreads();
    }
    if (pw == 0 && dst) {
      const float f = x[8] == 0.f ? 0.f : 1.f / x[8];
      reinterpret_cast<uint4 *>(dst)[c8] =
          make_uint4(pack_bf16x2(x[0] * f, x[1] * f), pack_bf16x2(x[2] * f, x[3] * f), pack_bf16x2(x[4] * f, x[5] * f),
                     pack_bf16x2(x[6] * f, x[7] * f));
    }
  }
}

template <int D>
cudaError_t launch_flat(const PrefixParams &p, int grid, cudaStream_t s) {
  using C = FlatCfg<D>;
  const cudaError_t e = cudaFuncSetAttribute(prefix_flat_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  prefix_flat_kernel<D><<<grid, C::THREADS, C::SMEM, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_tall(const PrefixParams &p, int grid, cudaStream_t s) {
  using C = TallCfg<D>;
  const cudaError_t e = cudaFuncSetAttribute(prefix_tall_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  prefix_tall_kernel<D><<<grid, C::THREADS, C::SMEM, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_join(const PrefixParams &p, int grid, int sms, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  // Slices of the columns: about eight blocks an SM at most, of the units that may be cut.
  const int rows = ((p.row_tile < p.rows ? p.row_tile : p.rows) + 31) / 32;
  const long long cut = static_cast<long long>(p.n_units) - static_cast<long long>(p.waves) * grid;
  int slices = D / 8;
  while (slices > 1 && (cut < grid ? cut : grid) * rows * slices > 8 * sms) slices /= 2;
  cfg.gridDim = dim3(static_cast<unsigned>(cut < grid ? cut : grid), rows, slices);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D>, p);
}

}  // namespace

int prefix_part_floats(int d, int rows) { return (d + 2) * (rows > BM ? rows : BM); }

cudaError_t launch_prefix_flat(const PrefixParams &p, int d, int grid, cudaStream_t s) {
  return d == 64 ? launch_flat<64>(p, grid, s) : launch_flat<128>(p, grid, s);
}

cudaError_t launch_prefix_tall(const PrefixParams &p, int d, int grid, cudaStream_t s) {
  return d == 64 ? launch_tall<64>(p, grid, s) : launch_tall<128>(p, grid, s);
}

cudaError_t launch_prefix_join(const PrefixParams &p, int d, int grid, int sms, cudaStream_t s) {
  return d == 64 ? launch_join<64>(p, grid, sms, s) : launch_join<128>(p, grid, sms, s);
}

}  // namespace xs
