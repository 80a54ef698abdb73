// Differential attention for sm_103a (tcgen05 tensor cores, Tensor Memory, TMA).
//
// Per batch b and head h, q = [q1 | q2] and k = [k1 | k2] in the d columns of a head:
//     x = (softmax(q1 k1^T * s) - lambda_h softmax(q2 k2^T * s)) v,   s = 1/sqrt(d/2),
//     o = x / sqrt(mean(x^2) + eps) * w * out_scale      (the norm where w is given),
// over the first kv_len[b] of Nk keys; a batch entry without keys gives zeros.
//
// One pass over the keys: each map keeps its own running maximum, sum and unnormalised
// output (x cannot be accumulated at once, as the two sums are known only at the end), and
//     x = O1 / l1 - lambda O2 / l2.
// Flops per query/key pair and head: 2d for the two score maps (d/2 columns each) and 4d
// for the two products with v.
//
// Work unit: one (batch, head) and one 128-row query tile (at d = 256 also one half of
// v's columns, the scores being computed in both). The two maps of a unit ping-pong
// through one MMA issuer exactly as two query tiles would: while the tensor pipe works on
// one map, the other map's softmax runs.
//
// Roles (320 threads, one CTA per SM):
//   warps 0-3  softmax warp group 0: map 1 (S1, P1, O1), row r of the tile = TMEM lane r
//   warps 4-7  softmax warp group 1: map 2
//   warp 8     MMA issuer and Tensor Memory allocation
//   warp 9     TMA loader
// In the epilogue each group takes half of the columns and reads both maps' O for them.
// Tensor Memory: S1 [0,128) S2 [128,256) O1 [256,256+DV) O2 [256+DV,256+2DV); P_t (bf16
// pairs) overwrites the first 64 columns of S_t.
// Shared memory: Q | ring of K and V tiles (64-column halves of 128 rows x 128 bytes,
// 128-byte swizzle) | barriers | 128 rows x 2 exchange words (twice for the norm).
//
// Order per KV step j, t = 1, 2: O_t += P_t(j-1) V(j-1); S_t = Q_t K_t(j)^T. One thread's
// tcgen05 operations execute in order, so S_t(j) cannot overwrite P_t(j-1) before it is
// read, and the commit that signals S_t(j) also covers PV_t(j-1).
//
// Schedule: persistent CTAs take whole units, strided; with a workspace the units past the
// last full wave but one are cut into equal contiguous ranges of KV tiles, and so are all
// units when there are fewer than SMs (few queries, long keys). A cut unit's pieces leave
// (m, l, O) of both maps in the workspace; the CTA that counts the last piece in merges
// them in piece order, so the result does not depend on who was last.
//
// Waits are bounded: a role that gives up records a timeout; the softmax warps then run
// their control flow to its end without waiting (so that they meet at the same named
// barriers), the issuer and the loader drain what they issued.
#include <cstdint>
#include <cstring>

#include "../../include/xs.h"
#include "diff.h"
#include "internal.h"
#include "ptx.cuh"

namespace xs {
namespace {

constexpr int BM = kTileRows, BN = kTileRows;
constexpr int kDiffThreads = 320;
constexpr int kDiffMmaWarp = 8, kDiffLoadWarp = 9;
constexpr int kDiffHalf = BM * 128;                 // one 64-column half of a 128-row tile
constexpr uint32_t kDiffSleepNs = 100000;
constexpr float kDiffRescale = 8.0f;                // log2 units: rescale O only past a growth of 2^8
constexpr int kFewRows = 8;                         // rows of a tile up to which a merge is spread over columns and pieces

// DH: columns of one map's q and k; DV: columns of v that a unit takes.
template <int DH_, int DV_>
struct DCfg {
  static constexpr int DH = DH_, DV = DV_, DQ = 2 * DH;
  static constexpr int SLOT = BN * DV * 2;          // a ring slot: the V tile, or DV columns of the K tile
  static constexpr int KSL = DQ / DV;               // slots of a K tile (2 at d = 256: one per map)
  static constexpr int USES = KSL + 1;              // ring uses per KV step
  static constexpr int QB = BM * DQ * 2;
  static constexpr int STAGES = DV == 64 ? 10 : 5;
  static constexpr bool NORM = DQ == DV;            // the whole row is in one unit: the norm is fused
  static constexpr int OFF_RING = QB;
  static constexpr int OFF_BAR = OFF_RING + STAGES * SLOT;
  static constexpr int OFF_EXCH = OFF_BAR + 1024;
  static constexpr int SMEM = OFF_EXCH + (NORM ? 2 : 1) * 1024 + 1024;   // + slack to align the base
  static constexpr uint32_t COL_O = 256;
  static constexpr int PART = 2 * DV * 128 + 4 * 128;   // floats of one piece's partial result
  static_assert(SMEM <= 232448, "shared memory per CTA");
  static_assert(COL_O + 2 * DV <= 512, "Tensor Memory columns");
};

// ------------------------------------------------------------------ schedule
__device__ __forceinline__ int keys_of(const DiffParams &p, int b) {
  if (!p.kv_len) return p.Nk;
  return min(max(__ldg(p.kv_len + b), 0), p.Nk);
}
// KV tiles of a batch entry; one without keys keeps a tile, fully masked, that gives its zeros.
__device__ __forceinline__ int tiles_of(int keys) { return max(1, (keys + BN - 1) / BN); }

// The split region: its KV tiles, the CTAs that share it, and where this CTA begins in it.
struct DPlan {
  long long total, bstart;   // bstart: first tile of batch entry b
  int grid, b;
};

struct DItem {
  int unit, b, keys;       // unit, its batch entry and that entry's keys
  int kv0, kv1, nk;        // KV tiles to do, and the unit's
  long long u0;            // a cut unit: its first tile in the split region
  bool piece;
};

// Walks a CTA's work list; every role walks its own copy.
struct DWalk {
  int k, b;
  long long pos, end, bstart;

  __device__ __forceinline__ void start(const DiffParams &p, const DPlan &plan) {
    k = 0;
    pos = end = 0;
    if (p.split && static_cast<int>(blockIdx.x) < plan.grid) {
      const long long T = plan.total, c = blockIdx.x;
      pos = c * T / plan.grid;
      end = (c + 1) * T / plan.grid;
    }
    b = plan.b;
    bstart = plan.bstart;
  }
  __device__ __forceinline__ bool next(const DiffParams &p, DItem &it) {
    const int G = gridDim.x;
    if (!p.split || k < p.waves) {
      it.unit = static_cast<int>(blockIdx.x) + k * G;
      ++k;
      if (it.unit >= p.n_units) return false;
      it.b = it.unit / p.units_b;
      it.keys = keys_of(p, it.b);
      it.nk = tiles_of(it.keys);
      it.kv0 = 0;
      it.kv1 = it.nk;
      it.u0 = 0;
      it.piece = false;
      return true;
    }
    if (pos >= end) return false;
    const int first = p.waves * G;                   // the region's first unit
    const int b0 = first / p.units_b;
    for (;;) {
      it.keys = keys_of(p, b);
      it.nk = tiles_of(it.keys);
      const int skip = b == b0 ? first - b0 * p.units_b : 0;
      const long long size = static_cast<long long>(p.units_b - skip) * it.nk;
      if (pos < bstart + size) {
        const int ul = static_cast<int>((pos - bstart) / it.nk);
        it.u0 = bstart + static_cast<long long>(ul) * it.nk;
        it.kv0 = static_cast<int>(pos - it.u0);
        it.kv1 = end - pos < it.nk - it.kv0 ? it.kv0 + static_cast<int>(end - pos) : it.nk;
        it.unit = b * p.units_b + skip + ul;
        it.b = b;
        it.piece = it.kv0 > 0 || it.kv1 < it.nk;
        pos += it.kv1 - it.kv0;
        return true;
      }
      bstart += size;
      ++b;
    }
  }
};

struct DBars {
  uint64_t q_full, q_empty;
  uint64_t kv_full[10], kv_empty[10];
  uint64_t s_full[2], p_full[2];
  uint64_t o_full, drain;
  DPlan plan;
  DWalk walk[8];      // the softmax warps' places in the work list and their items: kept here, as
  DItem item[8];      // registers are short while a row of scores is held
  uint32_t tmem_base;
  int abort, last;
  float red[8];
};
static_assert(sizeof(DBars) <= 1024, "barrier block too large");

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x,
                                            int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
// Meeting of the eight softmax warps.
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Bounded wait on a barrier phase; false after a timeout here or elsewhere in the CTA.
__device__ __noinline__ bool diff_wait_slow(uint32_t bar, uint32_t parity, DBars *bars, int *status,
                                            uint64_t limit) {
  volatile int *abort_flag = &bars->abort;
  const bool sleepy = threadIdx.x / 32 != kDiffMmaWarp;   // the issuer polls
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (sleepy ? mbar_try_wait_sleep(bar, parity, kDiffSleepNs) : mbar_try_wait(bar, parity))
      return true;
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
__device__ __forceinline__ bool diff_wait(uint32_t bar, uint32_t parity, DBars *bars,
                                          const DiffParams &p) {
  const bool ok = mbar_try_wait(bar, parity) ||
                  diff_wait_slow(bar, parity, bars, p.status, p.wait_limit_ns);
  return __all_sync(0xffffffffu, ok);
}
// Tear-down: waits for this thread's own copies or MMAs in flight, whatever the abort flag and
// however short the limit of the other waits, still bounded.
__device__ __noinline__ void diff_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > 2000000000ull) return;
}

// The split region's size and this CTA's place in it, by one warp.
__device__ void plan_split(const DiffParams &p, DBars *bars) {
  const int lane = threadIdx.x & 31;
  const int first = p.waves * static_cast<int>(gridDim.x), b0 = first / p.units_b;
  auto size_of = [&](int b) -> long long {
    if (b >= p.B) return 0;
    const int skip = b == b0 ? first - b0 * p.units_b : 0;
    return static_cast<long long>(p.units_b - skip) * tiles_of(keys_of(p, b));
  };
  long long total = 0;
  for (int b = b0 + lane; b < p.B; b += 32) total += size_of(b);
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int grid = static_cast<int>(total < gridDim.x ? total : gridDim.x);
  const long long pos = static_cast<int>(blockIdx.x) < grid
                            ? static_cast<long long>(blockIdx.x) * total / grid
                            : 0;
  long long base = 0;
  int b = b0;
  for (;; b += 32) {   // the batch entry that holds pos; ends, as pos < total
    const long long mine = size_of(b + lane);
    long long incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned past = __ballot_sync(0xffffffffu, pos < base + incl);
    if (past) {
      const int at = __ffs(past) - 1;
      const long long begin = __shfl_sync(0xffffffffu, base + incl - mine, at);
      if (lane == 0) {
        bars->plan = DPlan{total, begin, grid, b + at};
      }
      return;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
    if (b + 32 >= p.B) break;
  }
  if (lane == 0) bars->plan = DPlan{0, 0, 0, b0};
}

struct DPlace {
  int h, q0, vp;
};
__device__ __forceinline__ DPlace place_of(const DiffParams &p, const DItem &it) {
  int u = it.unit - it.b * p.units_b;
  DPlace r;
  r.vp = u % p.v_parts;
  u /= p.v_parts;
  r.h = u / p.n_qtiles;
  r.q0 = (u - r.h * p.n_qtiles) * BM;
  return r;
}

// ------------------------------------------------------------------ TMA loader
template <class C>
__device__ void diff_loader(const DiffParams &p, uint8_t *smem, DBars *bars) {
  uint32_t it = 0, items = 0;   // ring uses, items
  const uint32_t q_full = smem_u32(&bars->q_full), q_empty = smem_u32(&bars->q_empty);
  DWalk walk;
  walk.start(p, bars->plan);
  DItem item;
  bool ok = true;
  // One ring use: DV columns from x of rows [j*128, +128) of a K or V head.
  auto load = [&](const CUtensorMap *m, int x, int j, int h, int b) {
    const uint32_t slot = it % C::STAGES, ph = (it / C::STAGES) & 1;
    if (!diff_wait(smem_u32(&bars->kv_empty[slot]), ph ^ 1, bars, p)) return false;
    const uint32_t full = smem_u32(&bars->kv_full[slot]);
    if (elect_one()) {
      mbar_arrive_expect_tx(full, C::SLOT);
      for (int hf = 0; hf < C::DV / 64; ++hf)
        tma_load_4d(smem_u32(smem + C::OFF_RING + slot * C::SLOT + hf * kDiffHalf), m, full,
                    x + hf * 64, j * BN, h, b);
    }
    __syncwarp();
    ++it;
    return true;
  };
  for (; ok && walk.next(p, item); ++items) {
    const DPlace at = place_of(p, item);
    const int hk = at.h / p.group;
    if (items > 0 && !diff_wait(q_empty, (items - 1) & 1, bars, p)) break;
    if (elect_one()) {
      mbar_arrive_expect_tx(q_full, C::QB);
      for (int hf = 0; hf < C::DQ / 64; ++hf)
        tma_load_4d(smem_u32(smem + hf * kDiffHalf), &p.tm_q, q_full, hf * 64, at.q0, at.h, item.b);
    }
    __syncwarp();
    for (int j = item.kv0; ok && j < item.kv1; ++j) {
      for (int ks = 0; ok && ks < C::KSL; ++ks) ok = load(&p.tm_k, ks * C::DV, j, hk, item.b);
      ok = ok && load(&p.tm_v, at.vp * C::DV, j, hk, item.b);
    }
  }
  // Every load issued must land before the CTA releases its shared memory.
  for (uint32_t s = 0; s < C::STAGES && s < it; ++s) {
    const uint32_t last = s + ((it - 1 - s) / C::STAGES) * C::STAGES;
    diff_drain(smem_u32(&bars->kv_full[s]), (last / C::STAGES) & 1);
  }
  if (items > 0) diff_drain(q_full, (items - 1) & 1);
}

// ------------------------------------------------------------------ MMA issuer
// S_t = Q_t K_t^T: DH columns from t * DH of the Q tile and of the K tile.
template <class C>
__device__ __forceinline__ void diff_qk(uint32_t dcol, uint64_t qdesc, uint64_t kdesc, int t) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, 0);
#pragma unroll
  for (int kk = 0; kk < C::DH / 16; ++kk) {
    const int qc = t * C::DH + kk * 16;                            // column within the Q tile
    const int kc = C::KSL == 2 ? kk * 16 : qc;                     // within the K slot
    const uint64_t qo = static_cast<uint64_t>(((qc / 64) * kDiffHalf + (qc % 64) * 2) >> 4);
    const uint64_t ko = static_cast<uint64_t>(((kc / 64) * kDiffHalf + (kc % 64) * 2) >> 4);
    tc_mma_ss(dcol, qdesc + qo, kdesc + ko, idesc, kk > 0 ? 1u : 0u);
  }
}
template <class C>
__device__ __forceinline__ void diff_pv(uint32_t dcol, uint32_t pcol, uint64_t vdesc,
                                        uint32_t accumulate) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, C::DV, 1);
#pragma unroll
  for (int kk = 0; kk < BN / 16; ++kk)
    tc_mma_ts(dcol, pcol + kk * 8, vdesc + static_cast<uint64_t>((kk * 2048) >> 4), idesc,
              (kk > 0 || accumulate) ? 1u : 0u);
}

template <class C>
__device__ void diff_issuer(const DiffParams &p, uint8_t *smem, DBars *bars, uint32_t tmem_in) {
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_in, 0);
  const int lane = threadIdx.x & 31;
  uint32_t it = 0, items = 0;
  uint32_t pc = 0;                                    // P phases, the same for both maps
  const uint32_t q_full = smem_u32(&bars->q_full), q_empty = smem_u32(&bars->q_empty);
  const uint64_t qdesc = smem_desc_sw128(smem_u32(smem), 16, 1024);
  const uint64_t kdesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_RING), 16, 1024);
  const uint64_t vdesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_RING), kDiffHalf, 1024);
  auto slot_of = [&](uint32_t use) { return use % C::STAGES; };
  auto full = [&](uint32_t use) {
    return diff_wait(smem_u32(&bars->kv_full[slot_of(use)]), (use / C::STAGES) & 1, bars, p);
  };
  auto empty = [&](uint32_t use) { return smem_u32(&bars->kv_empty[slot_of(use)]); };
  auto at = [&](uint64_t d, uint32_t use) {
    return d + static_cast<uint64_t>(slot_of(use) * (C::SLOT >> 4));
  };
  // S_t of the step whose K uses start at `use`; its slots are released after their last reader.
  auto issue_qk = [&](int t, uint32_t use, bool last) {
    const uint32_t ku = use + (C::KSL == 2 ? t : 0);
    if (C::KSL == 2 || t == 0) {
      if (!full(ku)) return false;
      tc_fence_after();
    }
    if (elect_one()) {
      diff_qk<C>(tmem + t * 128, qdesc, at(kdesc0, ku), t);
      tc_commit(smem_u32(&bars->s_full[t]));
      if (C::KSL == 2 || t == 1) tc_commit(empty(ku));
      if (last && t == 1) tc_commit(q_empty);
    }
    __syncwarp();
    return true;
  };
  // A key past the batch entry's length has weight 0, but what lies in its row of V may not
  // be a number: the rows behind the last key are cleared before the products read them.
  // (Rows past Nk were filled with zeros by the load.)
  auto clear_tail = [&](uint32_t use, int keys, int j) {
    const int valid = keys - j * BN;
    if (valid >= BN || keys >= p.Nk) return;
    uint8_t *tile = smem + C::OFF_RING + slot_of(use) * C::SLOT;
    for (int hf = 0; hf < C::DV / 64; ++hf)
      for (int o = valid * 128 + lane * 16; o < kDiffHalf; o += 512)
        *reinterpret_cast<uint4 *>(tile + hf * kDiffHalf + o) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
  };
  DWalk walk;
  walk.start(p, bars->plan);
  DItem item;
  for (; walk.next(p, item); ++items) {
    const int nk = item.kv1 - item.kv0;
    if (!diff_wait(q_full, items & 1, bars, p)) goto drain;
    for (int t = 0; t < 2; ++t)
      if (!issue_qk(t, it, nk == 1)) goto drain;
    for (int j = 0; j < nk; ++j) {
      const uint32_t vu = it + C::KSL, next = it + C::USES;
      const bool more = j + 1 < nk;
      if (!full(vu)) goto drain;
      clear_tail(vu, item.keys, item.kv0 + j);
      for (int t = 0; t < 2; ++t) {
        if (!diff_wait(smem_u32(&bars->p_full[t]), pc & 1, bars, p)) goto drain;
        tc_fence_after();
        if (elect_one()) {
          diff_pv<C>(tmem + C::COL_O + t * C::DV, tmem + t * 128, at(vdesc0, vu), j > 0 ? 1u : 0u);
          if (t == 1) tc_commit(empty(vu));
          if (t == 1 && !more) tc_commit(smem_u32(&bars->o_full));
        }
        __syncwarp();
        if (more && !issue_qk(t, next, j + 2 == nk)) goto drain;
      }
      ++pc;
      it += C::USES;
    }
  }
drain:
  // All MMAs issued must finish before Tensor Memory is released.
  if (elect_one()) tc_commit(smem_u32(&bars->drain));
  __syncwarp();
  diff_drain(smem_u32(&bars->drain), 0);
}

// ------------------------------------------------------------------ softmax / epilogue
// Where output row n of (b, h) begins (bf16), and where its fp32 form for a norm over both
// column halves.
__device__ __forceinline__ uint16_t *out_row(const DiffParams &p, int b, int h, int n, int d) {
  if (p.shard_mode) {
    const int sh = n / p.rows_per_shard, i = n - sh * p.rows_per_shard;
    return static_cast<uint16_t *>(p.shards[sh]) +
           ((static_cast<long long>(b) * p.rows_per_shard + i) * p.H + h) * d;
  }
  return static_cast<uint16_t *>(p.o) + b * p.o_b + h * p.o_h + n * p.o_n;
}
__device__ __forceinline__ float *stage_row(const DiffParams &p, int b, int h, int n, int d) {
  return p.stage + ((static_cast<long long>(b) * p.H + h) * p.Nq + n) * d;
}

// Maximum over 64 raw scores in 8 chains of 3-input max; `first` starts the chains.
__device__ __forceinline__ void diff_max(const uint32_t (&a)[32], const uint32_t (&b)[32],
                                         float (&mp)[8], bool first) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = __uint_as_float(a[i]), y = __uint_as_float(a[i + 8]);
    mp[i] = first ? fmaxf(x, y) : max3(mp[i], x, y);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    mp[i] = max3(mp[i], __uint_as_float(a[i + 16]), __uint_as_float(a[i + 24]));
#pragma unroll
  for (int i = 0; i < 8; ++i)
    mp[i] = max3(mp[i], __uint_as_float(b[i]), __uint_as_float(b[i + 8]));
#pragma unroll
  for (int i = 0; i < 8; ++i)
    mp[i] = max3(mp[i], __uint_as_float(b[i + 16]), __uint_as_float(b[i + 24]));
}

// This thread's NX columns (from col0 of the unit's) of one finished row: norm, scale, store.
// `ss` is the whole row's sum of squares.
template <class C, int NX>
__device__ __forceinline__ void finish_row(const DiffParams &p, const DItem &item, const DPlace &at,
                                           int n, int col0, float (&x)[NX], float ss) {
  constexpr int D = C::DQ;
  if (!C::NORM && p.weight) {   // d = 256: the norm follows in a kernel of its own
    float4 *dst = reinterpret_cast<float4 *>(stage_row(p, item.b, at.h, n, D) + at.vp * C::DV + col0);
#pragma unroll
    for (int i = 0; i < NX / 4; ++i)
      dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    return;
  }
  uint16_t *dst = out_row(p, item.b, at.h, n, D) + at.vp * C::DV + col0;
  if (C::NORM && p.weight) {
    const float r = rsqrtf(ss * (1.f / D) + p.eps) * p.out_scale;
#pragma unroll
    for (int i = 0; i < NX / 4; ++i) {
      const float4 w = __ldg(reinterpret_cast<const float4 *>(p.weight + col0) + i);
      x[4 * i] *= r * w.x;
      x[4 * i + 1] *= r * w.y;
      x[4 * i + 2] *= r * w.z;
      x[4 * i + 3] *= r * w.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NX; ++i) x[i] *= p.out_scale;
  }
  if constexpr (NX >= 8) {
#pragma unroll
    for (int i = 0; i < NX / 8; ++i)
      reinterpret_cast<uint4 *>(dst)[i] =
          make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                     pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
  } else {
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  }
}

// What a map's sum stands for in x = f1 O1 + f2 O2; a row without keys gives 0.
__device__ __forceinline__ float map_factor(int t, float lambda, float l) {
  return l == 0.f ? 0.f : (t == 0 ? 1.f : -lambda) / l;
}

// One piece of a cut unit: leaves its partial result in the workspace; the CTA that counts the
// last piece merges all of them. All eight softmax warps take part.
template <class C>
__device__ void diff_piece(const DiffParams &p, DBars *bars, float *exch, const DItem &item,
                           const DPlace &at, uint32_t tmem, float m, float l, float lambda, bool dead) {
  const int tid = threadIdx.x, t = tid / 128, row = tid & 127, lane = tid & 31;
  const int rows = min(BM, p.Nq - at.q0);
  const long long T = bars->plan.total;
  const int G = bars->plan.grid;
  auto start = [&](int c) { return static_cast<long long>(c) * T / G; };
  auto owner = [&](long long pos) {
    int c = static_cast<int>(pos * G / T);
    while (c + 1 < G && start(c + 1) <= pos) ++c;
    while (c > 0 && start(c) > pos) --c;
    return c;
  };
  const int c0 = owner(item.u0);
  const int S = owner(item.u0 + item.nk - 1) - c0 + 1;
  // Piece k ran on CTA c0 + k, as its first item (slot 0), but for the unit's first piece, which
  // is the last item of its CTA (slot 1).
  auto part = [&](int k) {
    return p.parts + (static_cast<size_t>(c0 + k) * 2 + (k == 0 ? 1 : 0)) * C::PART;
  };
  auto stat_of = [&](int k) { return reinterpret_cast<float4 *>(part(k) + 2 * C::DV * 128); };
  const int own = static_cast<int>(blockIdx.x) - c0;
  if (row < rows && !dead) reinterpret_cast<float2 *>(stat_of(own) + row)[t] = make_float2(m, l);
  {
    // Columns as float4 groups, [col/4][row][4]: a warp instruction moves 512 bytes.
    const uint32_t tO = tmem + (static_cast<uint32_t>((row & ~31)) << 16) + C::COL_O + t * C::DV;
    float4 *o4 = reinterpret_cast<float4 *>(part(own) + t * C::DV * 128);
    if ((row & ~31) < rows) {
#pragma unroll 1
      for (int c = 0; c < C::DV / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * c, o);
        tmem_wait_ld_regs(o);
        if (row < rows && !dead) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            __stcg(o4 + (8 * c + i) * 128 + row,
                   make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                               __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3])));
        }
      }
    }
  }
  tc_fence_before();
  __threadfence();
  softmax_sync();
  if (tid == 0) {
    int last = 0;
    if (!dead) last = atomicAdd(p.count + c0, 1) == S - 1;
    if (last) p.count[c0] = 0;   // every piece has arrived: ready for the next launch
    bars->last = last;
  }
  softmax_sync();
  const int last = bars->last;
  if (!last) return;   // the next write of `last` follows another meeting
  __threadfence();
  if (rows > kFewRows) {
    // A thread takes one row and half of the columns.
    constexpr int NX = C::DV / 2;
    float x[NX];
#pragma unroll
    for (int i = 0; i < NX; ++i) x[i] = 0.f;
    float ss = 0.f;
    if (row < rows) {
      float m1 = -INFINITY, m2 = -INFINITY, l1 = 0.f, l2 = 0.f;
#pragma unroll 4
      for (int k = 0; k < S; ++k) {
        const float4 s = __ldcg(stat_of(k) + row);
        m1 = fmaxf(m1, s.x);
        m2 = fmaxf(m2, s.z);
      }
#pragma unroll 4
      for (int k = 0; k < S; ++k) {
        const float4 s = __ldcg(stat_of(k) + row);
        l1 = fmaf(ex2_approx(s.x - m1), s.y, l1);
        l2 = fmaf(ex2_approx(s.z - m2), s.w, l2);
      }
      const float f1 = map_factor(0, lambda, l1), f2 = map_factor(1, lambda, l2);
#pragma unroll 1
      for (int k = 0; k < S; ++k) {
        const float4 s = __ldcg(stat_of(k) + row);
        const float g1 = f1 * ex2_approx(s.x - m1), g2 = f2 * ex2_approx(s.z - m2);
        const float4 *a = reinterpret_cast<const float4 *>(part(k)) + (t * (NX / 4)) * 128 + row;
        const float4 *b = a + C::DV / 4 * 128;
#pragma unroll
        for (int i = 0; i < NX / 4; ++i) {
          const float4 u = __ldcg(a + i * 128), v = __ldcg(b + i * 128);
          x[4 * i] = fmaf(g1, u.x, fmaf(g2, v.x, x[4 * i]));
          x[4 * i + 1] = fmaf(g1, u.y, fmaf(g2, v.y, x[4 * i + 1]));
          x[4 * i + 2] = fmaf(g1, u.z, fmaf(g2, v.z, x[4 * i + 2]));
          x[4 * i + 3] = fmaf(g1, u.w, fmaf(g2, v.w, x[4 * i + 3]));
        }
      }
#pragma unroll
      for (int i = 0; i < NX; ++i) ss = fmaf(x[i], x[i], ss);
    }
    if constexpr (C::NORM) {
      exch[256 + tid] = ss;
      softmax_sync();
      ss += exch[256 + (tid ^ 128)];
    }
    if (row < rows) finish_row<C, NX>(p, item, at, at.q0 + row, t * NX, x, ss);
    return;
  }
  // Few rows: row by row, a warp takes CW groups of four columns, and its lanes share the pieces.
  constexpr int CW = C::DV / 4 / 8, PG = 32 / CW;
  const int c4 = (tid / 32) * CW + lane % CW, pg = lane / CW;
  for (int r = 0; r < rows; ++r) {
    float m1 = -INFINITY, m2 = -INFINITY, l1 = 0.f, l2 = 0.f;
    for (int k = lane; k < S; k += 32) {
      const float4 s = __ldcg(stat_of(k) + r);
      m1 = fmaxf(m1, s.x);
      m2 = fmaxf(m2, s.z);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
      m2 = fmaxf(m2, __shfl_xor_sync(0xffffffffu, m2, o));
    }
    for (int k = lane; k < S; k += 32) {
      const float4 s = __ldcg(stat_of(k) + r);
      l1 = fmaf(ex2_approx(s.x - m1), s.y, l1);
      l2 = fmaf(ex2_approx(s.z - m2), s.w, l2);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
      l2 += __shfl_xor_sync(0xffffffffu, l2, o);
    }
    const float f1 = map_factor(0, lambda, l1), f2 = map_factor(1, lambda, l2);
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k = pg; k < S; k += PG) {
      const float4 s = __ldcg(stat_of(k) + r);
      const float4 u = __ldcg(reinterpret_cast<const float4 *>(part(k)) + c4 * 128 + r);
      const float4 v = __ldcg(reinterpret_cast<const float4 *>(part(k)) + (C::DV / 4 + c4) * 128 + r);
      const float g1 = f1 * ex2_approx(s.x - m1), g2 = f2 * ex2_approx(s.z - m2);
      x[0] = fmaf(g1, u.x, fmaf(g2, v.x, x[0]));
      x[1] = fmaf(g1, u.y, fmaf(g2, v.y, x[1]));
      x[2] = fmaf(g1, u.z, fmaf(g2, v.z, x[2]));
      x[3] = fmaf(g1, u.w, fmaf(g2, v.w, x[3]));
    }
#pragma unroll
    for (int o = CW; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
    float ss = 0.f;
    if constexpr (C::NORM) {
      ss = x[0] * x[0] + x[1] * x[1] + x[2] * x[2] + x[3] * x[3];
#pragma unroll
      for (int o = 1; o < CW; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      softmax_sync();   // the previous row's sums have been read
      if (lane == 0) bars->red[tid / 32] = ss;
      softmax_sync();
      ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += bars->red[i];
    }
    if (pg == 0) finish_row<C, 4>(p, item, at, at.q0 + r, c4 * 4, x, ss);
  }
}

template <class C>
__device__ void diff_softmax(const DiffParams &p, uint8_t *smem, DBars *bars, uint32_t tmem) {
  const int t = threadIdx.x / 128, row = threadIdx.x & 127, wq = (threadIdx.x / 32) & 3;
  const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
  const uint32_t tS = tmem + lane_base + t * 128;
  const uint32_t tO = tmem + lane_base + C::COL_O + t * C::DV;
  const uint32_t s_full = smem_u32(&bars->s_full[t]), p_full = smem_u32(&bars->p_full[t]);
  const uint32_t o_full = smem_u32(&bars->o_full);
  float *exch = reinterpret_cast<float *>(smem + C::OFF_EXCH);
  const float scale = p.scale_log2;
  uint32_t sc = 0, items = 0;
  bool dead = false;   // a wait gave up: go on without waiting, store nothing
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (!dead && !diff_wait(bar, parity, bars, p)) dead = true;
  };
  DWalk &walk = bars->walk[threadIdx.x / 32];
  DItem &item = bars->item[threadIdx.x / 32];
  const int lane = threadIdx.x & 31;
  if (lane == 0) walk.start(p, bars->plan);
  for (;; ++items) {
    int more = 0;
    if (lane == 0) more = walk.next(p, item);
    if (!__shfl_sync(0xffffffffu, more, 0)) break;
    __syncwarp();
    // No query in this warp's rows: nothing to compute or store.
    const bool idle = place_of(p, item).q0 + wq * 32 >= p.Nq;
    const int nk = item.kv1 - item.kv0;
    int valid = item.keys - item.kv0 * BN;   // keys from this tile on that count
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < nk; ++j, ++sc, valid -= BN) {
      wait(s_full, sc & 1);
      if (idle) {
        mbar_arrive(p_full);
        continue;
      }
      tc_fence_after();
      uint32_t s[4][32];
      tmem_ld32(tS, s[0]);
      tmem_ld32(tS + 32, s[1]);
      tmem_wait_ld_regs(s[0]);
      tmem_wait_ld_regs(s[1]);
      tmem_ld32(tS + 64, s[2]);
      tmem_ld32(tS + 96, s[3]);
      float mp[8];
      if (valid < BN) {
        tmem_wait_ld_regs(s[2]);
        tmem_wait_ld_regs(s[3]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * c + i >= valid) s[c][i] = 0xff800000u;   // -inf, whatever the score was
        diff_max(s[0], s[1], mp, true);
      } else {
        diff_max(s[0], s[1], mp, true);
        tmem_wait_ld_regs(s[2]);
        tmem_wait_ld_regs(s[3]);
      }
      diff_max(s[2], s[3], mp, false);
      const float mx = max3(max3(mp[0], mp[1], mp[2]), max3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7]));
      const float m_new = fmaxf(m, mx * scale);
      float alpha = 1.f;
      bool rescale = false;
      if (j == 0) {
        m = m_new;
      } else {
        const bool need = m_new > m + kDiffRescale;
        if (__any_sync(0xffffffffu, need)) {
          rescale = true;
          if (need) {
            alpha = ex2_approx(m - m_new);
            m = m_new;
          }
        }
      }
      // A tile without any key has m = -inf; its weights are 2^(-inf - 0) = 0.
      const float neg_m = m == -INFINITY ? 0.f : -m;
      const uint64_t scale2 = f2_pack(scale, scale), negm2 = f2_pack(neg_m, neg_m);
      float lsum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint64_t x2 = f2_fma(
              f2_pack(__uint_as_float(s[c][2 * i]), __uint_as_float(s[c][2 * i + 1])), scale2, negm2);
          float x0, x1;
          f2_unpack(x2, x0, x1);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          lsum[i & 3] += p0 + p1;
          pk[i] = pack_bf16x2(p0, p1);   // P goes to the tensor cores in bf16, as V does; l sums it in fp32
        }
        tmem_st16(tS + 16 * c, pk);
      }
      l = fmaf(l, alpha, (lsum[0] + lsum[1]) + (lsum[2] + lsum[3]));
      if (rescale) {
#pragma unroll 1
        for (int c = 0; c < C::DV / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + 32 * c, o);
          tmem_wait_ld_regs(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st32(tO + 32 * c, o);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(p_full);
    }
    // Both maps' O are final once the unit's last product completes.
    wait(o_full, items & 1);
    tc_fence_after();
    const DPlace at = place_of(p, item);
    const float lambda = __ldg(p.lambda + at.h);
    if (item.piece) {
      diff_piece<C>(p, bars, exch, item, at, tmem, m, l, lambda, dead);
      __syncwarp();
      continue;
    }
    exch[threadIdx.x] = map_factor(t, lambda, l);
    softmax_sync();
    constexpr int NX = C::DV / 2;
    float x[NX], ss = 0.f;
    if (!idle) {
      const float f1 = exch[row], f2 = exch[128 + row];
      const uint32_t o1 = tmem + lane_base + C::COL_O + t * NX;
#pragma unroll
      for (int c = 0; c < NX / 32; ++c) {
        uint32_t a[32], b[32];
        tmem_ld32(o1 + 32 * c, a);
        tmem_ld32(o1 + C::DV + 32 * c, b);
        tmem_wait_ld_regs(a);
        tmem_wait_ld_regs(b);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float v = fmaf(f1, __uint_as_float(a[i]), f2 * __uint_as_float(b[i]));
          x[32 * c + i] = v;
          ss = fmaf(v, v, ss);
        }
      }
    }
    tc_fence_before();
    if constexpr (C::NORM) exch[256 + threadIdx.x] = ss;
    // Both groups have read O: a group's next P may let the next unit's products overwrite it.
    softmax_sync();
    if constexpr (C::NORM) ss += exch[256 + (threadIdx.x ^ 128)];
    if (at.q0 + row < p.Nq && !dead) finish_row<C, NX>(p, item, at, at.q0 + row, t * NX, x, ss);
    __syncwarp();   // `item` has been read
  }
}

template <class C>
__global__ void __launch_bounds__(kDiffThreads, 1) attn_diff_kernel(const __grid_constant__ DiffParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  DBars *bars = reinterpret_cast<DBars *>(smem + C::OFF_BAR);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars->q_full), 1);
    mbar_init(smem_u32(&bars->q_empty), 1);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(smem_u32(&bars->kv_full[s]), 1);
      mbar_init(smem_u32(&bars->kv_empty[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&bars->s_full[t]), 1);
      mbar_init(smem_u32(&bars->p_full[t]), 128);
    }
    mbar_init(smem_u32(&bars->o_full), 1);
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1 && p.split) plan_split(p, bars);
  if (warp == kDiffMmaWarp) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  if (warp == kDiffLoadWarp && lane == 0) {
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  if (warp == kDiffLoadWarp) {
    diff_loader<C>(p, smem, bars);
    __syncwarp();
  } else if (warp == kDiffMmaWarp) {
    diff_issuer<C>(p, smem, bars, tmem);
    __syncwarp();
  } else {
    diff_softmax<C>(p, smem, bars, tmem);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kDiffMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// d = 256: the norm of the staged fp32 rows (their columns come from two units), a warp per row.
__global__ void __launch_bounds__(256) diff_norm_kernel(const __grid_constant__ DiffParams p) {
  const int lane = threadIdx.x & 31;
  const long long rows = static_cast<long long>(p.B) * p.H * p.Nq;
  const float4 w0 = __ldg(reinterpret_cast<const float4 *>(p.weight) + 2 * lane);
  const float4 w1 = __ldg(reinterpret_cast<const float4 *>(p.weight) + 2 * lane + 1);
  for (long long r = static_cast<long long>(blockIdx.x) * 8 + threadIdx.x / 32; r < rows;
       r += static_cast<long long>(gridDim.x) * 8) {
    const float4 *src = reinterpret_cast<const float4 *>(p.stage + r * 256) + 2 * lane;
    const float4 a = __ldcs(src), b = __ldcs(src + 1);
    float ss = a.x * a.x + a.y * a.y + a.z * a.z + a.w * a.w + b.x * b.x + b.y * b.y + b.z * b.z +
               b.w * b.w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float f = rsqrtf(ss * (1.f / 256) + p.eps) * p.out_scale;
    const long long bh = r / p.Nq;
    const int n = static_cast<int>(r - bh * p.Nq), bb = static_cast<int>(bh / p.H);
    uint16_t *dst = out_row(p, bb, static_cast<int>(bh - static_cast<long long>(bb) * p.H), n, 256);
    reinterpret_cast<uint4 *>(dst)[lane] =
        make_uint4(pack_bf16x2(a.x * f * w0.x, a.y * f * w0.y), pack_bf16x2(a.z * f * w0.z, a.w * f * w0.w),
                   pack_bf16x2(b.x * f * w1.x, b.y * f * w1.y), pack_bf16x2(b.z * f * w1.z, b.w * f * w1.w));
  }
}

// Every output row to zero, 16 bytes a thread.
__global__ void __launch_bounds__(256) diff_zero_kernel(const __grid_constant__ DiffParams p, int d) {
  const int vecs = d / 8;
  const long long total = static_cast<long long>(p.B) * p.H * p.Nq * vecs;
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * 256) {
    const long long r = i / vecs, bh = r / p.Nq;
    const int bb = static_cast<int>(bh / p.H), h = static_cast<int>(bh - static_cast<long long>(bb) * p.H);
    reinterpret_cast<uint4 *>(out_row(p, bb, h, static_cast<int>(r - bh * p.Nq), d))[i - r * vecs] =
        make_uint4(0, 0, 0, 0);
  }
}

template <class C>
cudaError_t launch_cfg(const DiffParams &p, int grid, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(attn_diff_kernel<C>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  attn_diff_kernel<C><<<grid, kDiffThreads, C::SMEM, s>>>(p);
  return cudaGetLastError();
}

using D64 = DCfg<32, 64>;
using D128 = DCfg<64, 128>;
using D256 = DCfg<128, 128>;

}  // namespace

int diff_part_floats(int d) { return d == 64 ? D64::PART : D128::PART; }

cudaError_t launch_attn_diff(const DiffParams &p, int d, int grid, cudaStream_t s) {
  if (d == 64) return launch_cfg<D64>(p, grid, s);
  if (d == 128) return launch_cfg<D128>(p, grid, s);
  return launch_cfg<D256>(p, grid, s);
}

cudaError_t launch_diff_zero(const DiffParams &p, int d, int grid, cudaStream_t s) {
  diff_zero_kernel<<<grid, 256, 0, s>>>(p, d);
  return cudaGetLastError();
}

cudaError_t launch_diff_norm(const DiffParams &p, int grid, cudaStream_t s) {
  diff_norm_kernel<<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace xs
