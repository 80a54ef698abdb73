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
// Work unit: one (batch, head) and one 128-row query tile. This file has the schedule and
// the kernel for d = 64 and 128, whose two maps of a unit run beside each other: 2 x 128
// score columns and 2 x d of O fill Tensor Memory. d = 256 has a kernel of its own
// (attn_diff_wide.cuh); without a norm, where the workspace is missing or small or the call
// short, it runs here, on halves of v's columns (a unit is then a half, and the scores are
// computed in both).
//
// Roles (352 or 384 threads, one CTA per SM):
//   warps 0-3  softmax of map 1, row r of the tile = TMEM lane r
//   warps 4-7  softmax of map 2
//   warp 8     issues the scores; Tensor Memory allocation
//   warp 9     issues the products with v
//   warp 10    TMA loader; publishes the items of the list to the softmax warps
// In the epilogue each group takes half of the columns and reads both maps' O for them.
// Tensor Memory: S1 [0,128) S2 [128,256) O1 [256,256+DV) O2 [256+DV,256+2DV); P_t (bf16
// pairs) overwrites the first 64 columns of S_t.
// Shared memory: Q | ring of K tiles | ring of V tiles (64-column halves of 128 rows x 128
// bytes, 128-byte swizzle) | barriers | staged output rows | sums and the norm's weights.
//
// A tile of 128 keys goes in halves of 64. The early half's scores lie in columns 64-127 of
// S_t, which P never covers: they are computed as soon as the softmax holds the tile
// before's in registers, so its exponentials run while the tensor cores do the products of
// the tile before. The late half's, in P's columns, follow those products. Each half's
// weights go to the products as they are written.
//
// Bound: at d = 128 the tensor pipe has 1536 cycles of work a tile and both maps (512
// scores, 1024 products), the softmax 2 x 128 x 128 exponentials, 1024 cycles of the
// four special-function units and about as many issue slots again. A tile takes 1.17 us
// (2420 cycles): the chain late scores - late softmax - products - late scores of a map is
// what the other map's work does not hide, and the softmax warps' own instructions (without
// the row sums a tile would take 7% less, with half of the exponentials no less).
// At d = 64 (1.1 us a tile, 768 cycles of tensor work) it is the softmax itself, with two warps
// a scheduler: 6 heads of 16384 725 us (853 TFLOP/s, 46%). Measured (GB300, 2070 MHz): d = 128,
// 24 heads of 4096 queries and keys 232 us (1331 TFLOP/s, 71% of the cuBLAS rate), of 16384
// 3.34 ms (1482, 79%); one query of 4 x 24 heads against 16384 keys 129 us (6.2 TB/s of K and V,
// 92% of the copy rate). A unit costs 3.8 us beside its tiles (first loads, epilogue). Few
// queries: a 128-row tile holds those of one query head, also where heads share k and v, so
// 24 heads on 8 k/v heads take as long as on 24.
// Tried at d = 128, time of a tile: an issuer per map 1.37; scores in the order early 1, late 1,
// early 2, late 2 1.76; registers moved from the issuers to the softmax 1.34 (all three
// against 1.23); sixteen softmax warps on column halves no gain; tiles of 64 keys with S
// doubled 3.8 to 5.3 ms at 16384 (several arrangements); late weights
// without their maximum too, the early ones stored after them, 273 us at 4096. At d = 64, P in
// columns of its own, so that late scores need not wait for the products: 1.30.
//
// Schedule: persistent CTAs take whole units, strided; with a workspace the units past the
// last full wave but one are cut into contiguous ranges of KV tiles of equal cost, and so are
// all units when there are fewer than SMs (few queries, long keys), where that is quicker. A cut
// unit's pieces leave (m, l, O) of both maps in the workspace; the CTA that counts the last
// piece in merges them in piece order, so the result does not depend on who was last.
//
// Waits are bounded: a role that gives up records a timeout; the softmax warps then run
// their control flow to its end without waiting (so that they meet at the same named
// barriers), the issuers and the loader drain what they issued.
#include <cstdint>
#include <cstring>

#include "../../include/xs.h"
#include "diff.h"
#include "internal.h"
#include "ptx.cuh"

namespace xs {
namespace {

constexpr int BM = kTileRows, BN = kTileRows;
constexpr int BC = 64;                              // keys of half a KV tile
constexpr int kSoftWarps = 8, kSoftThreads = 32 * kSoftWarps;
constexpr int kScoreWarp = kSoftWarps, kProductWarp = kSoftWarps + 1, kDiffLoadWarp = kSoftWarps + 2;
constexpr int kDiffHalf = BM * 128;                 // one 64-column half of a 128-row tile
constexpr uint32_t kDiffSleepNs = 100000;
constexpr float kDiffRescale = 8.0f;                // d = 256, log2 units: rescale O only past a growth of 2^8

// DH: columns of one map's q and k; DV: columns of v that a unit takes.
template <int DH_, int DV_>
struct DCfg {
  static constexpr int DH = DH_, DV = DV_, DQ = 2 * DH;
  // With a twelfth warp, which does nothing, the compiler's schedule of the softmax comes out faster
  // at DV = 128 (a KV tile 1.20 -> 1.17 us) and slower at 64 (1.10 -> 1.20).
  static constexpr int THREADS = kSoftThreads + (DV == 64 ? 96 : 128);
  static constexpr int SLOT = BN * DV * 2;          // a ring slot: the V tile, or DV columns of the K tile
  static constexpr int KSL = DQ / DV;               // slots of a K tile (2 at d = 256: one per map)
  static constexpr int QB = BM * DQ * 2;
  static constexpr int KS = 3, VS = DV == 64 ? 3 : 2;   // slots of the K ring, of the V ring behind it
  static constexpr bool NORM = DQ == DV;            // the whole row is in one unit: the norm is fused
  static constexpr int OFF_RING = QB;
  static constexpr int OFF_BAR = OFF_RING + (KS + VS) * SLOT;
  static constexpr int OFF_STG = OFF_BAR + 512;   // a warp's 32 rows of half the columns, bf16
  static constexpr int OFF_EXCH = OFF_STG + (NORM ? BM * DV * 2 : 0);    // sums; squares and the norm's weights
  static constexpr int SMEM = OFF_EXCH + (NORM ? 8 * kSoftThreads + 4 * DV : 4 * kSoftThreads);
  static constexpr uint32_t COL_O = 256;
  static_assert(SMEM <= 232448, "shared memory per CTA");
  static_assert(COL_O + 2 * DV <= 512, "Tensor Memory columns");
};

// Floats of one piece's partial result: O and (m, l) of both maps.
template <int DV>
constexpr int kPart = 2 * DV * 128 + 4 * 128;

// ------------------------------------------------------------------ schedule
__device__ __forceinline__ int keys_of(const DiffParams &p, int b) {
  if (!p.kv_len) return p.Nk;
  return min(max(__ldg(p.kv_len + b), 0), p.Nk);
}
// KV tiles of a batch entry; one without keys keeps a tile, fully masked, that gives its zeros.
__device__ __forceinline__ int tiles_of(int keys) { return max(1, (keys + BN - 1) / BN); }

// The split region: its places (kUnitCost for a unit and then one for each of its KV tiles), the
// CTAs that share it, and where this CTA begins in it.
struct DPlan {
  long long total, bstart;   // bstart: first place of batch entry b
  int grid, b;
};

struct DItem {
  int unit, b, keys;       // unit, its batch entry and that entry's keys
  int kv0, kv1, nk;        // KV tiles to do, and the unit's
  long long u0;            // a cut unit: its first tile's place in the split region
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
      const int places = it.nk + kUnitCost;
      const long long size = static_cast<long long>(p.units_b - skip) * places;
      if (pos < bstart + size) {
        const int ul = static_cast<int>((pos - bstart) / places);
        it.u0 = bstart + static_cast<long long>(ul) * places + kUnitCost;
        if (end <= it.u0) {   // the range ends before the unit's first tile
          pos = end;
          return false;
        }
        it.kv0 = pos > it.u0 ? static_cast<int>(pos - it.u0) : 0;
        it.kv1 = end - it.u0 < it.nk ? static_cast<int>(end - it.u0) : it.nk;
        it.unit = b * p.units_b + skip + ul;
        it.b = b;
        it.piece = it.kv0 > 0 || it.kv1 < it.nk;
        pos = it.u0 + it.kv1;
        return true;
      }
      bstart += size;
      ++b;
    }
  }
};

struct DPlace {
  int h, q0, vp;
};
// What the softmax warps know of an item.
struct DTask {
  long long u0;
  int b, keys, kv0, kv1, nk;
  int h, q0;
  short vp, kind;   // kind: 0 none (the list's end), 1 a whole unit, 2 a piece
};

struct DBars {
  static constexpr int kScore = kScoreWarp, kProduct = kProductWarp;   // warps
  uint64_t q_full, q_empty;
  uint64_t kv_full[6], kv_empty[6];
  uint64_t e_full[2], e_free[2];   // [map]: the early half's scores written; read into registers
  uint64_t l_full[2];              // the late half's scores written
  uint64_t p_full[2][2];           // [map][half]: the weights written
  uint64_t pv_done[2];             // the tile's products done
  uint64_t o_full, drain[2];
  uint64_t item_full[4];
  DPlan plan;
  DTask task[4];           // the softmax warps' items, published by the loader (task i mod 4)
  uint32_t tmem_base;
  int abort, last;
  float red[kSoftWarps];
};
static_assert(sizeof(DBars) <= 512, "barrier block too large");

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x,
                                            int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
// Meeting of all softmax warps.
__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 9, %0;" ::"n"(kSoftThreads) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// The wait for tmem_ld16, naming its registers so that no use of them moves before it.
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// Bounded wait on a barrier phase; false after a timeout here or elsewhere in the CTA.
template <class B>
__device__ __noinline__ bool diff_wait_slow(uint32_t bar, uint32_t parity, B *bars, int *status,
                                            uint64_t limit) {
  volatile int *abort_flag = &bars->abort;
  const int warp = threadIdx.x / 32;
  const bool sleepy = warp != B::kScore && warp != B::kProduct;   // the issuers poll
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
template <class B>
__device__ __forceinline__ bool diff_wait(uint32_t bar, uint32_t parity, B *bars,
                                          const DiffParams &p) {
  const bool ok = mbar_try_wait(bar, parity) ||
                  diff_wait_slow(bar, parity, bars, p.status, p.wait_limit_ns);
  return __all_sync(0xffffffffu, ok);
}
// The same with no call, for waits made while most registers are live.
template <class B>
__device__ __forceinline__ bool diff_wait_inline(uint32_t bar, uint32_t parity, B *bars,
                                                 const DiffParams &p) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    volatile int *abort_flag = &bars->abort;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
      ok = mbar_try_wait_sleep(bar, parity, kDiffSleepNs);
      if (ok) break;
      if ((it & 15u) == 0) {
        if (*abort_flag) break;
        if (globaltimer_ns() - t0 > p.wait_limit_ns) {
          *abort_flag = 1;
          atomicExch(p.status, kDevTimeout);
          break;
        }
      }
    }
  }
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
template <class B>
__device__ void plan_split(const DiffParams &p, B *bars) {
  const int lane = threadIdx.x & 31;
  const int first = p.waves * static_cast<int>(gridDim.x), b0 = first / p.units_b;
  auto size_of = [&](int b) -> long long {
    if (b >= p.B) return 0;
    const int skip = b == b0 ? first - b0 * p.units_b : 0;
    return static_cast<long long>(p.units_b - skip) * (tiles_of(keys_of(p, b)) + kUnitCost);
  };
  long long total = 0;
  for (int b = b0 + lane; b < p.B; b += 32) total += size_of(b);
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const long long most = max(1ll, total / p.min_places);
  const int grid = static_cast<int>(most < gridDim.x ? most : gridDim.x);
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

// The consecutive CTAs that a cut unit's pieces run on.
struct DSpan {
  int first, pieces;
};
__device__ __forceinline__ DSpan span_of(const DPlan &plan, const DTask &item) {
  const long long T = plan.total;
  const int G = plan.grid;
  auto start = [&](int c) { return static_cast<long long>(c) * T / G; };
  auto owner = [&](long long pos) {
    int c = static_cast<int>(pos * G / T);
    while (c + 1 < G && start(c + 1) <= pos) ++c;
    while (c > 0 && start(c) > pos) --c;
    return c;
  };
  const int first = owner(item.u0);
  return DSpan{first, owner(item.u0 + item.nk - 1) - first + 1};
}

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
  uint32_t k_use = 0, v_use = 0, items = 0;   // uses of the two rings, items
  const uint32_t q_full = smem_u32(&bars->q_full), q_empty = smem_u32(&bars->q_empty);
  DWalk walk;
  walk.start(p, bars->plan);
  DItem item;
  bool ok = true;
  // The next use of a ring (`first` slot, `n` slots): DV columns from x of rows [j*128, +128) of a
  // K or V head.
  auto load = [&](uint32_t &use, int first, int n, const CUtensorMap *m, int x, int j, int h, int b) {
    const uint32_t slot = first + use % n, ph = (use / n) & 1;
    if (!diff_wait(smem_u32(&bars->kv_empty[slot]), ph ^ 1, bars, p)) return false;
    const uint32_t full = smem_u32(&bars->kv_full[slot]);
    if (elect_one()) {
      mbar_arrive_expect_tx(full, C::SLOT);
      for (int hf = 0; hf < C::DV / 64; ++hf)
        tma_load_4d(smem_u32(smem + C::OFF_RING + slot * C::SLOT + hf * kDiffHalf), m, full,
                    x + hf * 64, j * BN, h, b);
    }
    __syncwarp();
    ++use;
    return true;
  };
  // Item i's record is written once the scores of item i - 1 are done: the softmax has then
  // begun the last tile of item i - 2 at least, and four records are enough (the end's included).
  auto publish = [&](const DTask &task) {
    if (elect_one()) {
      bars->task[items & 3] = task;
      mbar_arrive(smem_u32(&bars->item_full[items & 3]));
    }
    __syncwarp();
  };
  for (; ok && walk.next(p, item); ++items) {
    const DPlace at = place_of(p, item);
    const int hk = at.h / p.group;
    if (items > 0 && !diff_wait(q_empty, (items - 1) & 1, bars, p)) break;
    publish(DTask{item.u0, item.b, item.keys, item.kv0, item.kv1, item.nk, at.h, at.q0,
                  static_cast<short>(at.vp), static_cast<short>(item.piece ? 2 : 1)});
    if (elect_one()) {
      mbar_arrive_expect_tx(q_full, C::QB);
      for (int hf = 0; hf < C::DQ / 64; ++hf)
        tma_load_4d(smem_u32(smem + hf * kDiffHalf), &p.tm_q, q_full, hf * 64, at.q0, at.h, item.b);
    }
    __syncwarp();
    for (int j = item.kv0; ok && j < item.kv1; ++j) {
      for (int ks = 0; ok && ks < C::KSL; ++ks) ok = load(k_use, 0, C::KS, &p.tm_k, ks * C::DV, j, hk, item.b);
      ok = ok && load(v_use, C::KS, C::VS, &p.tm_v, at.vp * C::DV, j, hk, item.b);
    }
  }
  publish(DTask{0, 0, 0, 0, 0, 0, 0, 0, 0, 0});   // the end, also after a wait that gave up
  // Every load issued must land before the CTA releases its shared memory.
  for (uint32_t s = 0; s < C::KS + C::VS; ++s) {
    const uint32_t n = s < C::KS ? C::KS : C::VS, first = s < C::KS ? s : s - C::KS;
    const uint32_t uses = s < C::KS ? k_use : v_use;
    if (uses > first) diff_drain(smem_u32(&bars->kv_full[s]), ((uses - 1 - first) / n) & 1);
  }
  if (items > 0) diff_drain(q_full, (items - 1) & 1);
}

// ------------------------------------------------------------------ MMA issuers
// S = Q_t K_t^T for 64 keys: DH columns from t * DH of the Q tile and of the K tile.
template <class C>
__device__ __forceinline__ void diff_qk(uint32_t dcol, uint64_t qdesc, uint64_t kdesc, int t) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, BC, 0);
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
  for (int kk = 0; kk < BC / 16; ++kk)
    tc_mma_ts(dcol, pcol + kk * 8, vdesc + static_cast<uint64_t>((kk * 2048) >> 4), idesc,
              (kk > 0 || accumulate) ? 1u : 0u);
}
// A ring's place as a consumer sees it: the slot (and its descriptor offset) and the parity of the
// slot's use. K and V have a ring each, so that a consumer sees every phase of the barriers it
// waits on: a parity wait that skips one could pass too early.
template <int FIRST, int N, int BYTES>
struct DRing {
  uint32_t slot = 0, parity = 0;
  __device__ __forceinline__ void advance() {
    if (++slot == N) {
      slot = 0;
      parity ^= 1;
    }
  }
  __device__ __forceinline__ bool full(DBars *bars, const DiffParams &p) const {
    return diff_wait(smem_u32(&bars->kv_full[FIRST]) + slot * 8, parity, bars, p);
  }
  __device__ __forceinline__ uint32_t empty(DBars *bars) const {
    return smem_u32(&bars->kv_empty[FIRST]) + slot * 8;
  }
  __device__ __forceinline__ uint64_t offset() const {
    return static_cast<uint64_t>((FIRST + slot) * (BYTES >> 4));
  }
};
// An item's tiles, as a value that the compiler knows to be the same in every lane: the issuers'
// loops, and the addresses and descriptors they step, then stay in uniform registers. (An issuer
// stands between every two halves of the softmax: with these in vector registers a tile took 5%
// longer, with the loops below rolled up as well 35%.)
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
constexpr uint64_t kChunkRows = (BC * 128) >> 4;   // descriptor step to a tile's second 64 keys

// The score issuer. The first 64 keys of a tile (the early half) go out as soon as the softmax
// holds those of the tile before in registers; the others (the late half), which share their
// columns with P, once the products of the tile before have read it (pv_done: a wait, as the
// order of two threads' tcgen05 operations, or of two shapes, is not given).
template <class C>
__device__ void diff_score_issuer(const DiffParams &p, uint8_t *smem, DBars *bars, uint32_t tmem_in) {
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_in, 0);
  uint32_t q_parity = 0, parity = 0;   // of the item, of the tile
  DRing<0, C::KS, C::SLOT> ring;
  const uint64_t qdesc = smem_desc_sw128(smem_u32(smem), 16, 1024);
  const uint64_t kdesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_RING), 16, 1024);
  const uint32_t q_full = smem_u32(&bars->q_full), q_empty = smem_u32(&bars->q_empty);
  const uint32_t e_free = smem_u32(&bars->e_free[0]), e_full = smem_u32(&bars->e_full[0]);
  const uint32_t l_full = smem_u32(&bars->l_full[0]), pv_done = smem_u32(&bars->pv_done[0]);
  DWalk walk;
  walk.start(p, bars->plan);
  DItem item;
  for (; walk.next(p, item); q_parity ^= 1) {
    const int nk = uniform(item.kv1 - item.kv0);
    if (!diff_wait(q_full, q_parity, bars, p)) goto drain;
    for (int j = 0; j < nk; ++j, parity ^= 1) {
      // K of one map per slot at d = 256: its second slot is the next one.
      DRing<0, C::KS, C::SLOT> kr[2] = {ring, ring};
      if (C::KSL == 2) kr[1].advance();
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (half == 0 && (C::KSL == 2 || t == 0) && !kr[t].full(bars, p)) goto drain;
          // The phase before this tile's (none before the first tile: such a wait passes).
          if (!diff_wait((half == 0 ? e_free : pv_done) + 8 * t, parity ^ 1, bars, p)) goto drain;
          tc_fence_after();
          if (elect_one()) {
            diff_qk<C>(tmem + t * 128 + (half == 0 ? BC : 0), qdesc,
                       kdesc0 + kr[t].offset() + (half == 0 ? 0 : kChunkRows), t);
            tc_commit((half == 0 ? e_full : l_full) + 8 * t);
            if (half == 1 && (C::KSL == 2 || t == 1)) tc_commit(kr[t].empty(bars));
            if (half == 1 && t == 1 && j == nk - 1) tc_commit(q_empty);
          }
          __syncwarp();
        }
      ring = kr[1];
      ring.advance();
    }
  }
drain:
  // All MMAs issued must finish before Tensor Memory is released.
  if (elect_one()) tc_commit(smem_u32(&bars->drain[0]));
  __syncwarp();
  diff_drain(smem_u32(&bars->drain[0]), 0);
}

template <class C>
__device__ void diff_product_issuer(const DiffParams &p, uint8_t *smem, DBars *bars, uint32_t tmem_in) {
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_in, 0);
  const int lane = threadIdx.x & 31;
  uint32_t parity = 0;
  DRing<C::KS, C::VS, C::SLOT> ring;
  const uint64_t vdesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_RING), kDiffHalf, 1024);
  const uint32_t p_full = smem_u32(&bars->p_full[0][0]), pv_done = smem_u32(&bars->pv_done[0]);
  const uint32_t o_full = smem_u32(&bars->o_full);
  // A key past the batch entry's length has weight 0, but what lies in its row of V may not
  // be a number: the rows behind the last key are cleared before the products read them.
  // (Rows past Nk were filled with zeros by the load.)
  auto clear_tail = [&](int valid) {
    uint8_t *tile = smem + C::OFF_RING + (C::KS + ring.slot) * C::SLOT;
    for (int hf = 0; hf < C::DV / 64; ++hf)
      for (int o = valid * 128 + lane * 16; o < kDiffHalf; o += 512)
        *reinterpret_cast<uint4 *>(tile + hf * kDiffHalf + o) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
  };
  DWalk walk;
  walk.start(p, bars->plan);
  DItem item;
  while (walk.next(p, item)) {
    const int nk = uniform(item.kv1 - item.kv0);
    // Of the item's tiles only its batch entry's last one can hold such keys.
    const int last_valid = uniform(item.keys >= p.Nk || item.kv1 < item.nk ? BN : item.keys - (item.nk - 1) * BN);
    for (int j = 0; j < nk; ++j, parity ^= 1) {
      if (!ring.full(bars, p)) goto drain;
      if (j == nk - 1 && last_valid < BN) clear_tail(last_valid);
      // Each half's products as soon as its weights are written: the early half's run beside the
      // late half's exponentials.
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int t = u >> 1, half = u & 1;
        if (!diff_wait(p_full + 8 * u, parity, bars, p)) goto drain;
        tc_fence_after();
        if (elect_one()) {
          diff_pv<C>(tmem + C::COL_O + t * C::DV, tmem + t * 128 + half * 32,
                     vdesc0 + ring.offset() + (half == 0 ? 0 : kChunkRows), j > 0 || half == 1 ? 1u : 0u);
          if (half == 1) tc_commit(pv_done + 8 * t);
          if (u == 3) {
            tc_commit(ring.empty(bars));
            if (j == nk - 1) tc_commit(o_full);
          }
        }
        __syncwarp();
      }
      ring.advance();
    }
  }
drain:
  if (elect_one()) tc_commit(smem_u32(&bars->drain[1]));
  __syncwarp();
  diff_drain(smem_u32(&bars->drain[1]), 0);
}

// ------------------------------------------------------------------ softmax / epilogue
// Where output row n of (b, h) begins.
__device__ __forceinline__ uint16_t *out_row(const DiffParams &p, int b, int h, int n, int d) {
  if (p.shard_mode) {
    const int sh = n / p.rows_per_shard, i = n - sh * p.rows_per_shard;
    return static_cast<uint16_t *>(p.shards[sh]) +
           ((static_cast<long long>(b) * p.rows_per_shard + i) * p.H + h) * d;
  }
  return static_cast<uint16_t *>(p.o) + b * p.o_b + h * p.o_h + n * p.o_n;
}
// Maximum over 64 raw scores, in 8 chains of 3-input max.
__device__ __forceinline__ float max64(const uint32_t (&a)[32], const uint32_t (&b)[32]) {
  float mp[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    mp[i] = max3(__uint_as_float(a[i]), __uint_as_float(a[i + 8]), __uint_as_float(a[i + 16]));
#pragma unroll
  for (int i = 0; i < 8; ++i)
    mp[i] = max3(mp[i], __uint_as_float(a[i + 24]), __uint_as_float(b[i]));
#pragma unroll
  for (int i = 0; i < 8; ++i)
    mp[i] = max3(mp[i], __uint_as_float(b[i + 8]), __uint_as_float(b[i + 16]));
#pragma unroll
  for (int i = 0; i < 8; ++i) mp[i] = fmaxf(mp[i], __uint_as_float(b[i + 24]));
  return max3(max3(mp[0], mp[1], mp[2]), max3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7]));
}

// The sum of squares of a row, or of a part of one, as the norm passes it on: the sum, or, where squares
// that count may have left fp32's range, minus its root. Rows with an infinity or NaN keep the sum.
// (Below: scaled_squares and its like. Their code costs 24 heads of 4096 at d = 128 0.9%, at d = 64 nothing;
// inlined, or with an eps in this test, which would spare rows that are small beside it, 1.3 to 1.6%.)
__device__ __forceinline__ bool squares_fit(float ss) {   // in [2^-80, 2^120]
  return __float_as_uint(ss) - __float_as_uint(0x1p-80f) <= __float_as_uint(0x1p120f) - __float_as_uint(0x1p-80f);
}
// The power of two that brings x near 1 (x > 0 and finite).
__device__ __forceinline__ float near_one(float x) {
  return __int_as_float((254 - min(max(__float_as_int(x) >> 23, 1), 253)) << 23);
}
// From the largest magnitude `big` and the sum `sum` of the squares times near_one(big)^2.
__device__ __forceinline__ float minus_root(float sum, float big) { return -(sqrtf(sum) * near_one(near_one(big))); }
__device__ __forceinline__ bool has_root(float big, float ss) { return big > 0.f && big < INFINITY && ss == ss; }
template <int NX>
__device__ __forceinline__ float scaled_squares(const float (&x)[NX], float ss) {
  float big = 0.f, sum = 0.f;
#pragma unroll
  for (int i = 0; i < NX; ++i) big = fmaxf(big, fabsf(x[i]));
  if (!has_root(big, ss)) return ss;
  const float s = near_one(big);
#pragma unroll
  for (int i = 0; i < NX; ++i) sum = fmaf(x[i] * s, x[i] * s, sum);
  return minus_root(sum, big);
}
// Of two parts of a row (join_roots: one of them minus its root).
__device__ __noinline__ float join_roots(float a, float b) {
  const float ra = a < 0.f ? -a : sqrtf(a), rb = b < 0.f ? -b : sqrtf(b);
  const float most = ra > rb ? ra : rb, q = (ra > rb ? rb : ra) / most;
  return -(most * sqrtf(fmaf(q, q, 1.f)));
}
__device__ __forceinline__ float join_squares(float a, float b) {
  return fminf(a, b) < 0.f ? join_roots(a, b) : a + b;
}
// The same of a row whose parts lie in N values of each of the first `lanes` lanes (a power of two),
// repeated over the warp; `ss` is its sum.
template <int N>
__device__ __forceinline__ float lanes_squares(const float (&x)[N], float ss, int lanes) {
  if (!__any_sync(0xffffffffu, !squares_fit(ss))) return ss;
  float big = 0.f, sum = 0.f;
  for (int i = 0; i < N; ++i) big = fmaxf(big, fabsf(x[i]));
  for (int o = 1; o < lanes; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
  const bool root = !squares_fit(ss) && has_root(big, ss);
  const float s = root ? near_one(big) : 1.f;
  for (int i = 0; i < N; ++i) sum = fmaf(x[i] * s, x[i] * s, sum);
  for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return root ? minus_root(sum, big) : ss;
}

// norm_factor of a sum passed on as minus its root.
__device__ __noinline__ float root_factor(float root, int d, float eps) {
  const float s = near_one(fmaxf(fabsf(root), sqrtf(eps))), y = root * s;
  return fminf(rsqrtf(y * y / d + eps * s * s) * s, 0x1p127f);
}
// 1 / sqrt(mean + eps) of a row of d columns. A row of zeros (no keys) stays one, also with eps = 0.
__device__ __forceinline__ float norm_factor(float ss, int d, float eps) {
  if (ss < 0.f) return root_factor(ss, d, eps);
  return ss == 0.f ? 0.f : rsqrtf(ss * (1.f / d) + eps);
}

// The norm, from the whole row's sum of squares `ss`, and the output's factor on NX columns.
template <class C, int NX>
__device__ __forceinline__ void scale_row(const DiffParams &p, const float *weight, int col0, float (&x)[NX], float ss) {
  if (C::NORM && p.weight) {
    const float r = norm_factor(ss, C::DQ, p.eps) * p.out_scale;
#pragma unroll
    for (int i = 0; i < NX / 4; ++i) {
      const float4 w = reinterpret_cast<const float4 *>(weight + col0)[i];
      x[4 * i] *= r * w.x;
      x[4 * i + 1] *= r * w.y;
      x[4 * i + 2] *= r * w.z;
      x[4 * i + 3] *= r * w.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NX; ++i) x[i] *= p.out_scale;
  }
}

// This thread's NX columns (from col0 of the unit's) of one finished row: norm, scale, store.
// `ss` is the whole row's sum of squares.
template <class C, int NX>
__device__ __forceinline__ void finish_row(const DiffParams &p, const float *weight, int b, const DPlace &at, int n, int col0, float (&x)[NX], float ss) {
  constexpr int D = C::DQ;
  uint16_t *dst = out_row(p, b, at.h, n, D) + at.vp * C::DV + col0;
  scale_row<C, NX>(p, weight, col0, x, ss);
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

// Four columns of a merged row: x += g1 O1 + g2 O2 of one piece.
__device__ __forceinline__ void add_piece(float *x, float g1, const float4 &u, float g2, const float4 &v) {
  x[0] = fmaf(g1, u.x, fmaf(g2, v.x, x[0]));
  x[1] = fmaf(g1, u.y, fmaf(g2, v.y, x[1]));
  x[2] = fmaf(g1, u.z, fmaf(g2, v.z, x[2]));
  x[3] = fmaf(g1, u.w, fmaf(g2, v.w, x[3]));
}

// One piece of a cut unit: leaves its partial result in the workspace; the CTA that counts the
// last piece merges all of them. All softmax warps take part; `l` is this thread's map's sum.
template <class C>
__device__ __noinline__ void diff_piece(const DiffParams &p, DBars *bars, float *exch, const DTask item,
                                        uint32_t tmem, float m, float l, bool dead) {
  const int tid = threadIdx.x, t = tid >> 7, row = tid & 127, lane = tid & 31;
  const DPlace at{item.h, item.q0, item.vp};
  const float lambda = __ldg(p.lambda + at.h);
  const int rows = min(BM, p.Nq - at.q0);
  const DSpan span = span_of(bars->plan, item);
  const int c0 = span.first, S = span.pieces;
  // Piece k ran on CTA c0 + k, as its first item (slot 0), but for the unit's first piece, which
  // is the last item of its CTA (slot 1).
  auto part = [&](int k) {
    return p.parts + (static_cast<size_t>(c0 + k) * 2 + (k == 0 ? 1 : 0)) * kPart<C::DV>;
  };
  auto stat_of = [&](int k) { return reinterpret_cast<float4 *>(part(k) + 2 * C::DV * 128); };
  const int own = static_cast<int>(blockIdx.x) - c0;
  if (row < rows && !dead)
    __stcg(reinterpret_cast<float2 *>(stat_of(own) + row) + t, make_float2(m, l));
  if ((row & ~31) < rows) {
    // The columns as float4 groups [col/4][row][4]: a warp instruction moves 512 bytes.
    const uint32_t tO = tmem + (static_cast<uint32_t>(row & ~31) << 16) + C::COL_O + t * C::DV;
    float4 *o4 = reinterpret_cast<float4 *>(part(own)) + t * (C::DV / 4) * 128 + row;
#pragma unroll 1
    for (int c = 0; c < C::DV / 32; ++c) {
      uint32_t o[32];
      tmem_ld32(tO + 32 * c, o);
      tmem_wait_ld_regs(o);
      if (row < rows && !dead) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          __stcg(o4 + (8 * c + i) * 128,
                 make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                             __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3])));
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
  if (!bars->last) return;   // its next write follows another meeting
  __threadfence();
  if (rows > 64) {
    // A thread takes one row and half of the columns.
    constexpr int NX = C::DV / 2;
    const int col0 = (tid >> 7) * NX;
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
        const float4 *a = reinterpret_cast<const float4 *>(part(k)) + (col0 / 4) * 128 + row;
        const float4 *b = a + C::DV / 4 * 128;
#pragma unroll
        for (int i = 0; i < NX / 4; ++i) {
          const float4 u = __ldcg(a + i * 128), v = __ldcg(b + i * 128);
          add_piece(x + 4 * i, g1, u, g2, v);
        }
      }
#pragma unroll
      for (int i = 0; i < NX; ++i) ss = fmaf(x[i], x[i], ss);
      if (p.weight && !squares_fit(ss)) ss = scaled_squares(x, ss);
    }
    float *sums = exch + kSoftThreads;
    sums[tid] = ss;
    softmax_sync();
    ss = join_squares(sums[row], sums[row + 128]);
    if (row < rows) finish_row<C, NX>(p, exch + 2 * kSoftThreads, item.b, at, at.q0 + row, col0, x, ss);
    return;
  }
  if (rows > kFewRows) {
    // Up to 64 rows: a thread takes one row and every CG-th chunk of eight columns (with the mapping
    // above 16 queries against 65536 keys took 92 us instead of 47). Four pieces' loads are in
    // flight at a time, the sum runs in piece order. A row that is still to be normed waits in the
    // first piece's place, each value for the thread that wrote it.
    const int R = rows > 32 ? 64 : rows > 16 ? 32 : 16;
    const int r = min(tid & (R - 1), rows - 1), cg = tid / R, CG = kSoftThreads / R;
    const bool live = (tid & (R - 1)) < rows;
    float m1 = -INFINITY, m2 = -INFINITY, l1 = 0.f, l2 = 0.f;
#pragma unroll 4
    for (int k = 0; k < S; ++k) {
      const float4 s = __ldcg(stat_of(k) + r);
      m1 = fmaxf(m1, s.x);
      m2 = fmaxf(m2, s.z);
    }
#pragma unroll 4
    for (int k = 0; k < S; ++k) {
      const float4 s = __ldcg(stat_of(k) + r);
      l1 = fmaf(ex2_approx(s.x - m1), s.y, l1);
      l2 = fmaf(ex2_approx(s.z - m2), s.w, l2);
    }
    const float f1 = map_factor(0, lambda, l1), f2 = map_factor(1, lambda, l2);
    const bool normed = p.weight != nullptr;
    float4 *hold = reinterpret_cast<float4 *>(part(0)) + r;
    float ss = 0.f;
#pragma unroll 1
    for (int c = cg; c < C::DV / 8; c += CG) {
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int k = 0; k < S; k += 4) {
        float4 s[4], u[4][2], v[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int kk = min(k + i, S - 1);
          s[i] = __ldcg(stat_of(kk) + r);
          const float4 *a = reinterpret_cast<const float4 *>(part(kk)) + 2 * c * 128 + r;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            u[i][h] = __ldcg(a + h * 128);
            v[i][h] = __ldcg(a + (C::DV / 4 + h) * 128);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (k + i >= S) break;
          const float g1 = f1 * ex2_approx(s[i].x - m1), g2 = f2 * ex2_approx(s[i].z - m2);
          add_piece(x, g1, u[i][0], g2, v[i][0]);
          add_piece(x + 4, g1, u[i][1], g2, v[i][1]);
        }
      }
      if (!live) continue;
      if (normed) {
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
        __stcg(hold + 2 * c * 128, make_float4(x[0], x[1], x[2], x[3]));
        __stcg(hold + (2 * c + 1) * 128, make_float4(x[4], x[5], x[6], x[7]));
      } else {
        finish_row<C, 8>(p, nullptr, item.b, at, at.q0 + r, 8 * c, x, 0.f);
      }
    }
    if (!normed) return;
    if (live && !squares_fit(ss)) {
      float big = 0.f, sum = 0.f;
      for (int c = cg; c < C::DV / 8; c += CG)
        for (int i = 0; i < 2; ++i) {
          const float4 a = __ldcg(hold + (2 * c + i) * 128);
          big = fmaxf(big, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))));
        }
      if (has_root(big, ss)) {
        const float s = near_one(big);
        for (int c = cg; c < C::DV / 8; c += CG)
          for (int i = 0; i < 2; ++i) {
            const float4 a = __ldcg(hold + (2 * c + i) * 128);
            sum = fmaf(a.x * s, a.x * s, sum);
            sum = fmaf(a.y * s, a.y * s, sum);
            sum = fmaf(a.z * s, a.z * s, sum);
            sum = fmaf(a.w * s, a.w * s, sum);
          }
        ss = minus_root(sum, big);
      }
    }
    float *sums = exch + kSoftThreads;
    sums[tid] = ss;
    softmax_sync();
    if (!live) return;
    ss = sums[r];
    for (int g = 1; g < CG; ++g) ss = join_squares(ss, sums[g * R + r]);
#pragma unroll 1
    for (int c = cg; c < C::DV / 8; c += CG) {
      const float4 a = __ldcg(hold + 2 * c * 128), b = __ldcg(hold + (2 * c + 1) * 128);
      float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      finish_row<C, 8>(p, exch + 2 * kSoftThreads, item.b, at, at.q0 + r, 8 * c, x, ss);
    }
    return;
  }
  // Few rows: row by row, a warp takes CW groups of four columns, and its lanes share the pieces.
  constexpr int CW = C::DV / 4 / kSoftWarps, PG = 32 / CW;
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
    float ss = x[0] * x[0] + x[1] * x[1] + x[2] * x[2] + x[3] * x[3];
#pragma unroll
    for (int o = 1; o < CW; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (p.weight) ss = lanes_squares(x, ss, CW);
    softmax_sync();   // the previous row's sums have been read
    if (lane == 0) bars->red[tid / 32] = ss;
    softmax_sync();
    ss = 0.f;
    float least = 0.f;
#pragma unroll
    for (int i = 0; i < kSoftWarps; ++i) {
      ss += bars->red[i];
      least = fminf(least, bars->red[i]);
    }
    if (least < 0.f) {
      ss = bars->red[0];
      for (int i = 1; i < kSoftWarps; ++i) ss = join_squares(ss, bars->red[i]);
    }
    if (pg == 0) finish_row<C, 4>(p, exch + 2 * kSoftThreads, item.b, at, at.q0 + r, c4 * 4, x, ss);
  }
}

// scaled_squares of half a row's columns f1 O1 + f2 O2, read from Tensor Memory again; all lanes take part.
template <int DV>
__device__ __noinline__ float unit_squares(uint32_t o1, float f1, float f2, float ss) {
  if (!__any_sync(0xffffffffu, f1 != 0.f || f2 != 0.f)) return ss;   // no keys: zeros
  float big = 0.f, sum = 0.f;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    const float s = near_one(big);   // (2^126 in the first pass, which does not use the sum)
    sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < DV / 32; ++c) {
      uint32_t a[16], v[16];
      tmem_ld16(o1 + 16 * c, a);
      tmem_ld16(o1 + DV + 16 * c, v);
      tmem_wait_ld16(a);
      tmem_wait_ld16(v);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float y = fmaf(f1, __uint_as_float(a[i]), f2 * __uint_as_float(v[i]));
        big = fmaxf(big, fabsf(y));
        sum = fmaf(y * s, y * s, sum);
      }
    }
  }
  return !squares_fit(ss) && has_root(big, ss) ? minus_root(sum, big) : ss;
}

// 32 scores of a row to weights 2^(s * scale - m), rounded to bf16 pairs: P goes to the tensor
// cores in bf16, as V does.
__device__ __forceinline__ void weights32(const uint32_t (&s)[32], uint64_t scale2, uint64_t negm2,
                                          uint32_t (&pk)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint64_t x2 =
        f2_fma(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), scale2, negm2);
    float x0, x1;
    f2_unpack(x2, x0, x1);
    pk[i] = pack_bf16x2(ex2_approx(x0), ex2_approx(x1));
  }
}
// Their sum in fp32 (four chains), of the rounded weights: the output is then a true mean of V's
// rows, and a weight's rounding counts only as far as its row of V lies from that mean. (With the
// sum of the weights before their rounding the error of results without a norm against 64 bits was
// up to a tenth larger, and the launch 4% faster at d = 128.) Taken when the weights are on their
// way to the tensor cores.
__device__ __forceinline__ void add_weights(const uint32_t (&pk)[16], float (&sum)[4]) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tadd.rn.f32.bf16 %0, a, %0;\n\tadd.rn.f32.bf16 %1, b, %1;}"
        : "+f"(sum[2 * (i & 1)]), "+f"(sum[2 * (i & 1) + 1])
        : "r"(pk[i]));
}
__device__ __forceinline__ float sum_of(const uint32_t (&pk)[2][16]) {
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  add_weights(pk[0], sum);
  add_weights(pk[1], sum);
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}
// Without any key the maximum is -inf, and the weights are 2^(-inf - 0) = 0.
__device__ __forceinline__ uint64_t neg2(float m) {
  const float n = m == -INFINITY ? 0.f : -m;
  return f2_pack(n, n);
}
// Whether a barrier's phase is complete, without waiting; asked early, so that a phase that is
// complete costs no wait (about 100 cycles) when it is needed.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// The scores of keys from `valid` on, of 64 in Tensor Memory, become -inf, whatever they were. (In
// place, one column at a time: selects on the registers would double the inner loop's code.)
__device__ __noinline__ void mask64(uint32_t taddr, int valid) {
  for (int c = max(valid, 0); c < BC; ++c)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr + c), "r"(0xff800000u)
                 : "memory");
  tmem_wait_st();
}

// The reference m of a row's weights 2^(s - m): kHead above the maximum of its first keys, kNone while
// all scores were -inf. A larger maximum mx moves it by a whole number.
constexpr float kHead = 7.f, kMove = 1.f, kMany = 512.f, kNone = -1e30f;
__device__ __forceinline__ float first_ref(float mx) { return mx == -INFINITY ? kNone : mx + kHead; }
// (Two forms of the same: from kNone the first step of the second ends at 0, and from anywhere else
// its second step is 0. In the inner loop the compiler does better with the first at DV = 64, 722
// against 753 us for 6 heads of 16384, and with the second at 128, 231 against 233 for 24 of 4096.)
template <int DV>
__device__ __forceinline__ float moved_ref(float m, float mx) {
  if (DV == 64) return m == kNone ? mx + kHead : m + ceilf(mx + kHead - m);
  m += ceilf(mx + kHead - m);
  return m + ceilf(mx + kHead - m);
}

// The factor 2^(a - b) of a maximum that moved from a to b; 1 where it did not (-inf included).
__device__ __forceinline__ float shrink(float a, float b) { return a == b ? 1.f : ex2_approx(a - b); }

// Softmax of one map, a thread per row, in halves of 64 keys: the early half's exponentials run
// while the tensor cores finish the last tile's products and compute the late half's scores.
// The weights' reference begins kHead above the first keys' own maximum: where that is the row's, the
// largest weight is a power of two, which bf16 holds exactly, and rows with few keys, or one among the
// first that stands out, keep the formula's precision (with it rounded up to a whole number, two keys'
// error against 64 bits was 0.0026 of the result instead of 0.0018). It moves only when it has to, and by
// whole numbers (log2 units), so that every rescaling is by a power of two, exact for weights already
// rounded (until scores of 2^16, where fp32 no longer holds the reference's fraction: one more rounding
// then). For the late half it moves when a score is kMove above it; for the early half, which does not
// look for its maximum, when its sum is kMany and more (a weight is 8 then at least). Nothing can overflow
// before that shows: a weight that is infinite makes the sum so too, and the scores are still there. (With
// the early half's maximum too 24 heads of 4096 took 244 us instead of 230.)
template <class C>
__device__ void diff_softmax(const DiffParams &p, uint8_t *smem, DBars *bars, uint32_t tmem) {
  const int tid = threadIdx.x, t = tid >> 7, row = tid & 127, wq = row >> 5;
  const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
  const uint32_t tS = tmem + lane_base + t * 128;   // late half and P [0, 64), early half [64, 128)
  const uint32_t tO = tmem + lane_base + C::COL_O + t * C::DV;
  const uint32_t e_full = smem_u32(&bars->e_full[t]), e_free = smem_u32(&bars->e_free[t]);
  const uint32_t l_full = smem_u32(&bars->l_full[t]), p_full = smem_u32(&bars->p_full[t][0]);
  const uint32_t o_full = smem_u32(&bars->o_full);
  float *exch = reinterpret_cast<float *>(smem + C::OFF_EXCH);
  const float scale = p.scale_log2;
  uint32_t step = 0, items = 0;
  bool dead = false;   // a wait gave up: go on without waiting, store nothing
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (!dead && !diff_wait_inline(bar, parity, bars, p)) dead = true;
  };
  for (;; ++items) {
    const uint32_t item_full = smem_u32(&bars->item_full[items & 3]);
    wait(item_full, (items >> 2) & 1);
    if (dead) diff_drain(item_full, (items >> 2) & 1);   // every warp sees the same list to its end
    const DTask &item = bars->task[items & 3];
    if (item.kind == 0) break;
    // No query in this warp's rows: nothing to compute or store, but the barriers' arrivals.
    const bool idle = item.q0 + wq * 32 >= p.Nq;
    const float lambda = __ldg(p.lambda + item.h);
    const int nk = item.kv1 - item.kv0;
    int valid = item.keys - item.kv0 * BN;   // keys from this tile on that count
    float m = -INFINITY, l = 0.f;
    const uint64_t scale2 = f2_pack(scale, scale);
    bool ready = false;   // this tile's early scores were seen complete
    for (int j = 0; j < nk; ++j, ++step, valid -= BN) {
      if (!__all_sync(0xffffffffu, ready)) wait(e_full, step & 1);
      if (idle) {
        mbar_arrive(e_free);
        wait(l_full, step & 1);
        mbar_arrive(p_full);
        mbar_arrive(p_full + 8);
        continue;
      }
      uint32_t pe[2][16], pl[2][16];
      float alpha = 1.f, early;   // early: the sum of the early half's weights
      bool rescale;               // of O, by alpha, in some lane
      tc_fence_after();
      {
        if (valid < BC) mask64(tS + BC, valid);
        uint32_t s[2][32];
        tmem_ld32(tS + 64, s[0]);
        tmem_ld32(tS + 96, s[1]);
        tmem_wait_ld_regs(s[0]);
        tmem_wait_ld_regs(s[1]);
        rescale = false;
        if (j == 0) m = first_ref(max64(s[0], s[1]) * scale);
        const uint64_t negm2 = f2_pack(-m, -m);
        weights32(s[0], scale2, negm2, pe[0]);
        ready = mbar_test(l_full, step & 1);
        weights32(s[1], scale2, negm2, pe[1]);
        early = sum_of(pe);
        // (Not a number asks too.)
        if (__any_sync(0xffffffffu, !(early < kMany))) {
          tmem_ld32(tS + 64, s[0]);
          tmem_ld32(tS + 96, s[1]);
          tmem_wait_ld_regs(s[0]);
          tmem_wait_ld_regs(s[1]);
          const float mx = max64(s[0], s[1]) * scale, before = m;
          if (mx > m + kMove) m = moved_ref<C::DV>(m, mx);
          alpha = shrink(before, m);
          rescale = j > 0;
          const uint64_t neg = f2_pack(-m, -m);
          weights32(s[0], scale2, neg, pe[0]);
          weights32(s[1], scale2, neg, pe[1]);
          early = sum_of(pe);
        }
        tc_fence_before();
        mbar_arrive(e_free);
      }
      if (!__all_sync(0xffffffffu, ready)) wait(l_full, step & 1);
      tc_fence_after();
      if (valid < BN) mask64(tS, valid - BC);
      uint32_t s[2][32];
      tmem_ld32(tS, s[0]);
      tmem_ld32(tS + 32, s[1]);
      tmem_wait_ld_regs(s[0]);
      tmem_wait_ld_regs(s[1]);
      const float mx = max64(s[0], s[1]) * scale, before = m;
      if (__any_sync(0xffffffffu, mx > m + kMove)) {
        if (mx > m + kMove) m = moved_ref<C::DV>(m, mx);
        const float a = shrink(before, m);   // in bf16 a power of two: exact on the rounded weights
        const uint32_t a2 = pack_bf16x2(a, a);
        alpha *= a;
        early *= a;
        rescale = j > 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 16; ++i) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(pe[h][i]) : "r"(a2));
      }
      // The late half's scores came after the products of the last tile: P and O are free.
      if (rescale) {
#pragma unroll 1
        for (int h = 0; h < C::DV / 16; ++h) {
          uint32_t o[16];
          tmem_ld16(tO + 16 * h, o);
          tmem_wait_ld16(o);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st16(tO + 16 * h, o);
        }
      }
      tmem_st16(tS, pe[0]);
      tmem_st16(tS + 16, pe[1]);
      // Some exponentials hide the store's latency.
      const uint64_t negm2 = f2_pack(-m, -m);
      weights32(s[0], scale2, negm2, pl[0]);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(p_full);
      weights32(s[1], scale2, negm2, pl[1]);
      tmem_st16(tS + 32, pl[0]);
      tmem_st16(tS + 48, pl[1]);
      ready = j + 1 < nk && mbar_test(e_full, (step + 1) & 1);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(p_full + 8);
      l = fmaf(l, alpha, early + sum_of(pl));
    }
    // Both maps' O are final once the unit's last product completes.
    wait(o_full, items & 1);
    tc_fence_after();
    if constexpr (C::NORM) {   // (the halves of v at d = 256 have no pieces)
      if (item.kind == 2) {
        diff_piece<C>(p, bars, exch, item, tmem, m, l, dead);
        continue;
      }
    }
    exch[tid] = l;
    softmax_sync();
    constexpr int NX = C::DV / 2;
    const DPlace at{item.h, item.q0, item.vp};
    const int b = item.b;
    const int col0 = t * NX;
    float x[NX], ss = 0.f;
    if (!idle) {
      const float f1 = map_factor(0, lambda, exch[row]);
      const float f2 = map_factor(1, lambda, exch[row + 128]);
      const uint32_t o1 = tmem + lane_base + C::COL_O + col0;
#pragma unroll
      for (int c = 0; c < NX / 32; ++c) {
        uint32_t a[32], v[32];
        tmem_ld32(o1 + 32 * c, a);
        tmem_ld32(o1 + C::DV + 32 * c, v);
        tmem_wait_ld_regs(a);
        tmem_wait_ld_regs(v);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float y = fmaf(f1, __uint_as_float(a[i]), f2 * __uint_as_float(v[i]));
          x[32 * c + i] = y;
          ss = fmaf(y, y, ss);
        }
      }
      if (C::NORM && p.weight && __any_sync(0xffffffffu, !squares_fit(ss)))
        ss = unit_squares<C::DV>(o1, f1, f2, ss);
    }
    tc_fence_before();
    float *sums = exch + kSoftThreads;
    if constexpr (C::NORM) sums[tid] = ss;
    // All have read O (and l): a map's next P may let the next unit's products overwrite it.
    softmax_sync();
    if constexpr (C::NORM) ss = join_squares(sums[row], sums[row + 128]);
    if (idle || dead) continue;
    if constexpr (!C::NORM) {   // no room to stage the rows
      if (at.q0 + row < p.Nq) finish_row<C, NX>(p, exch + 2 * kSoftThreads, b, at, at.q0 + row, col0, x, ss);
      continue;
    }
    // Rows lie across the lanes: through shared memory (16-byte chunks, each row's permuted by
    // its number against bank conflicts), so that NX / 8 lanes store one row's part together.
    constexpr int CH = NX / 8, RPS = 32 / CH;   // chunks of a row's part; rows a warp stores at once
    uint4 *stg = reinterpret_cast<uint4 *>(smem + C::OFF_STG) + (tid / 32) * 32 * CH;
    const int lane = tid & 31;
    scale_row<C, NX>(p, exch + 2 * kSoftThreads, col0, x, ss);
#pragma unroll
    for (int i = 0; i < CH; ++i)
      stg[lane * CH + (i ^ (lane & (CH - 1)))] =
          make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                     pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
    unsigned long long dst = 0;
    if (at.q0 + row < p.Nq)
      dst = reinterpret_cast<unsigned long long>(out_row(p, b, at.h, at.q0 + row, C::DQ) + at.vp * C::DV + col0);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int r = k * RPS + lane / CH, ch = lane % CH;
      const unsigned long long to = __shfl_sync(0xffffffffu, dst, r);
      const uint4 v = stg[r * CH + (ch ^ (r & (CH - 1)))];
      if (to) reinterpret_cast<uint4 *>(to)[ch] = v;
    }
    __syncwarp();   // the staged rows have been read
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) attn_diff_kernel(const __grid_constant__ DiffParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];   // the swizzle pattern repeats every 1024 bytes
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicExch(p.status, kDevBadPlan);
    return;
  }
  DBars *bars = reinterpret_cast<DBars *>(smem + C::OFF_BAR);
  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars->q_full), 1);
    mbar_init(smem_u32(&bars->q_empty), 1);
    for (int s = 0; s < (C::KS + C::VS); ++s) {
      mbar_init(smem_u32(&bars->kv_full[s]), 1);
      mbar_init(smem_u32(&bars->kv_empty[s]), 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&bars->item_full[i]), 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&bars->e_full[t]), 1);
      mbar_init(smem_u32(&bars->e_free[t]), 128);
      mbar_init(smem_u32(&bars->l_full[t]), 1);
      mbar_init(smem_u32(&bars->p_full[t][0]), 128);
      mbar_init(smem_u32(&bars->p_full[t][1]), 128);
      mbar_init(smem_u32(&bars->pv_done[t]), 1);
    }
    mbar_init(smem_u32(&bars->o_full), 1);
    mbar_init(smem_u32(&bars->drain[0]), 1);
    mbar_init(smem_u32(&bars->drain[1]), 1);
    bars->abort = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1 && p.split) plan_split(p, bars);
  if (C::NORM && p.weight && warp >= 4 && warp < 4 + C::DV / 32) {   // the norm's weights
    const int i = threadIdx.x - 128;
    reinterpret_cast<float *>(smem + C::OFF_EXCH)[2 * kSoftThreads + i] = __ldg(p.weight + i);
  }
  if (warp == kScoreWarp) {
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
  } else if (warp == kScoreWarp) {
    diff_score_issuer<C>(p, smem, bars, tmem);
    __syncwarp();
  } else if (warp == kProductWarp) {
    diff_product_issuer<C>(p, smem, bars, tmem);
    __syncwarp();
  } else if (warp < kSoftWarps) {
    diff_softmax<C>(p, smem, bars, tmem);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kScoreWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

#include "attn_diff_wide.cuh"

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
  attn_diff_kernel<C><<<grid, C::THREADS, C::SMEM, s>>>(p);
  return cudaGetLastError();
}

using D64 = DCfg<32, 64>;
using D128 = DCfg<64, 128>;
using D256 = DCfg<128, 128>;

}  // namespace

int diff_part_floats(int d) { return d == 64 ? kPart<64> : kPart<128>; }

cudaError_t launch_attn_diff(const DiffParams &p, int d, int grid, cudaStream_t s) {
  if (d == 64) return launch_cfg<D64>(p, grid, s);
  if (d == 128) return launch_cfg<D128>(p, grid, s);
  return launch_cfg<D256>(p, grid, s);
}

cudaError_t launch_diff_zero(const DiffParams &p, int d, int grid, cudaStream_t s) {
  diff_zero_kernel<<<grid, 256, 0, s>>>(p, d);
  return cudaGetLastError();
}

int diff_wide_part_floats(int rows) { return wide_part_floats(rows); }

cudaError_t launch_attn_diff_wide(const DiffParams &p, int grid, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(attn_diff_wide_kernel,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, WideCfg::SMEM);
  if (e != cudaSuccess) return e;
  attn_diff_wide_kernel<<<grid, WideCfg::THREADS, WideCfg::SMEM, s>>>(p);
  return cudaGetLastError();
}

}  // namespace xs
