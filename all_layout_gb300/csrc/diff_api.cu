// C-ABI entry points of differential attention (declared in include/xs.h): argument
// validation, tensor maps, the schedule's plan and the launches. Host code only.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/xs.h"
#include "diff.h"

#define XS_API extern "C" __attribute__((visibility("default")))

namespace {

using namespace xs;

bool aligned(const void *p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

unsigned long long parts_bytes(int grid, int d) {
  return static_cast<unsigned long long>(grid) * 2 * diff_part_floats(d) * 4;
}

// The d = 256 kernel's workspace: rows of a tile's partial results, a CTA's place for map 1 of a
// whole unit, and its two partial results.
int wide_rows(int Nq) { return Nq < kTileRows ? (Nq + 7) / 8 * 8 : kTileRows; }
unsigned long long wide_stash_bytes(int rows) { return 256ull * rows * 4; }
unsigned long long wide_parts_bytes(int rows) { return 2ull * diff_wide_part_floats(rows) * 4; }

// Whole units on min(units, sms) CTAs, or with `room` bytes for partial results the split
// schedule, whichever should end earlier. Times in KV tiles: a unit costs kUnitCost beside its own;
// `merge` is what each of a CTA's two cut units costs more (partial results written and merged).
// It follows from both schedules' measured times (GB300; heads x queries and keys, split / whole):
//   d = 64   12 x 4096 112 / 116 us, 12 x 2048 44 / 44, 20 x 2048 58 / 63, 3 x 8192 108 / 147
//   d = 128  12 x 4096 130 / 129 us, 12 x 2048 55 / 50, 20 x 2048 70 / 71, 3 x 8192 124 / 162
//   d = 256  12 x 4096 220 / 214 us, 12 x 2048 94 / 82, 3 x 8192 227 / 287
// Lengths that are on the device are taken as three quarters of Nk on average (8 entries of 8 heads,
// 777 queries, up to 1101 keys at d = 64, lengths falling to none: split 45 us, whole 34).
struct Plan {
  int split, waves, grid;
  long long cost, rounds;   // expected time in KV tiles; whole units a CTA takes
};
// The shortest range worth a CTA. Merging a piece of more than a few rows takes the last CTA f KV
// tiles' time, so n tiles in s pieces take n / s + f s, least at n / s = sqrt(f n). Measured f at 128
// rows: 0.75, 2 and 1.6 at d = 64, 128 and 256. (With ranges of 4 at least, 128 queries of one head
// against 65536 keys took 120, 353 and 425 us; so 55, 100 and 126.)
int min_places(int d, int nk, int rows) {
  int least = 4;
  const int f4 = d == 64 || (d == 128 && rows <= 64) ? 3 : d == 128 ? 8 : 6;
  if (rows > kFewRows)
    while (4 * least * least < f4 * nk) ++least;
  return least;
}
long merge_cost(int d, int rows) { return d == 64 ? 7 : d == 128 ? 8 : 6 + 4 * rows / kTileRows; }

// `per_cta`: bytes of workspace that a CTA's partial results take.
Plan plan(long long units, int sms, int nk, bool ragged, int least, long merge, unsigned long long per_cta,
          unsigned long long room) {
  const int grid0 = units < sms ? static_cast<int>(units) : sms;
  const long long mean = (ragged ? nk - nk / 4 : nk) + kUnitCost, rounds = (units + grid0 - 1) / grid0;
  const Plan whole{0, 0, grid0, (rounds - 1) * mean + nk + kUnitCost, rounds};
  if (nk < 2) return whole;
  const int waves = units >= sms ? static_cast<int>(units / sms) - 1 : 0;
  const long long left = units - static_cast<long long>(waves) * sms;
  long long per = (left * (nk + kUnitCost) + sms - 1) / sms;
  int grid = sms;
  if (waves == 0) {
    if (per < least) per = least;
    grid = static_cast<int>((left * (nk + kUnitCost) + per - 1) / per);
  }
  if (per_cta * grid > room || grid * 4 > static_cast<int>(XS_WORKSPACE_HEADER_BYTES / sizeof(int)))
    return whole;
  const long long cost = waves * mean + per * mean / (nk + kUnitCost) + 2 * merge;
  return cost < whole.cost ? Plan{1, waves, grid, cost, waves} : whole;
}

// Expected times at d = 256, of both maps one after the other and of both at once on half of v's columns
// (two units then): a KV tile takes 1.95 or 1.55 us, a whole unit 9 or 4 us beside its own, of which the plan's
// cost has kUnitCost tiles. Without a norm either will do, and the one that should end first is taken, so that a
// workspace with places for a few SMs does not keep the others idle. Measured (GB300, no norm, us; one after the
// other with places for 48 and for 80 SMs and with the whole workspace / halves; the first two lose to them):
//   12 heads x 4096 queries and keys 550, 346, 215 / 315    12 x 1024 52, 52, 28 / 36
//   8 heads x 256 queries, 16384 keys 254, 254, 116 / 201   24 x 4096, 1024 keys 381, 241, 148 / 174
//   30 heads x 681 queries, 41 keys (whole) 27 / 21         20 x 3 queries, 685 keys (whole) 21 / 16
// Over 200 random shapes and workspaces the choice was at most 12% from the better one.
long long wide_ns(const Plan &p) { return 1950 * p.cost + 3000 * p.rounds; }
long long halves_ns(const Plan &p) { return 1550 * p.cost - 600 * p.rounds; }

// One operand as a 4-D map {d, rows, heads, batch}; strides of single extents do not matter.
bool encode_operand(CUtensorMap *m, const void *base, int B, int H, int N, int d,
                    const long long *stride) {
  const unsigned long long dims[4] = {static_cast<unsigned long long>(d), static_cast<unsigned long long>(N),
                                      static_cast<unsigned long long>(H), static_cast<unsigned long long>(B)};
  unsigned long long st[3] = {static_cast<unsigned long long>(stride[2]) * 2,
                              static_cast<unsigned long long>(stride[1]) * 2,
                              static_cast<unsigned long long>(stride[0]) * 2};
  for (int i = 0; i < 3; ++i)
    if (dims[i + 1] == 1) st[i] = static_cast<unsigned long long>(d) * 2;
  const unsigned box[4] = {64, kTileRows, 1, 1};
  return encode_map(m, base, 4, dims, st, box);
}

xs_status check_operand(const long long *stride, int B, int H, int N, int d) {
  const long long extent[3] = {B, H, N};
  for (int i = 0; i < 3; ++i)
    if (extent[i] > 1 && stride[i] < d) return XS_ERR_INVALID;
  return XS_OK;
}
bool strides_aligned(const long long *stride, int B, int H, int N) {
  const long long extent[3] = {B, H, N};
  for (int i = 0; i < 3; ++i)
    if (extent[i] > 1 && (stride[i] % 8 != 0 || stride[i] >= (1LL << 38))) return false;
  return true;
}

xs_status diff_call(const xs_diff_args *a, void *o, const long long *o_stride, void *const *shards,
                    int P, void *ws, unsigned long long ws_bytes, void *stream) {
  if (!a || !a->q || !a->lambda) return XS_ERR_INVALID;
  const int B = a->B, H = a->H, Hk = a->H_kv, Nq = a->Nq, Nk = a->Nk, d = a->d;
  if (B < 0 || H < 0 || Hk < 0 || Nq < 0 || Nk < 0) return XS_ERR_INVALID;
  if (Nk > 0 && (!a->k || !a->v)) return XS_ERR_INVALID;
  if (H > 0 && (Hk < 1 || H % Hk != 0)) return XS_ERR_INVALID;
  if (!(a->scale > 0.f) || std::isinf(a->scale) || !(a->eps >= 0.f) || std::isinf(a->eps) ||
      !std::isfinite(a->out_scale))
    return XS_ERR_INVALID;
  if (shards) {
    if (P < 1 || P > kMaxShards || Nq % P != 0) return XS_ERR_INVALID;
    for (int p = 0; p < P; ++p)
      if (!shards[p]) return XS_ERR_INVALID;
  } else if (!o || !o_stride) {
    return XS_ERR_INVALID;
  }
  if (!ws && ws_bytes != 0) return XS_ERR_INVALID;
  const bool empty = B == 0 || H == 0 || Nq == 0;
  xs_status st = XS_OK;
  if (!empty) {
    st = check_operand(a->q_stride, B, H, Nq, d);
    if (st == XS_OK && Nk > 0) st = check_operand(a->k_stride, B, Hk, Nk, d);
    if (st == XS_OK && Nk > 0) st = check_operand(a->v_stride, B, Hk, Nk, d);
    if (st == XS_OK && !shards) st = check_operand(o_stride, B, H, Nq, d);
    if (st != XS_OK) return st;
  }
  if (d != 64 && d != 128 && d != 256) return XS_ERR_UNSUPPORTED;
  const long long qtiles = (static_cast<long long>(Nq) + kTileRows - 1) / kTileRows;
  const int most_parts = d == 256 ? 2 : 1;   // units of a query tile at most
  if (static_cast<double>(B) * H * static_cast<double>(qtiles) * most_parts > 2147483647.0 ||
      Nk > 0x7fffff00 || Nq > 0x7fffff00)
    return XS_ERR_UNSUPPORTED;
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(o, 16) ||
      !aligned(a->norm_weight, 16) || !aligned(a->lambda, 4) || !aligned(a->kv_len, 4) ||
      !aligned(ws, 256))
    return XS_ERR_ALIGN;
  if (shards)
    for (int p = 0; p < P; ++p)
      if (!aligned(shards[p], 16)) return XS_ERR_ALIGN;
  if (empty) return XS_OK;
  if (!strides_aligned(a->q_stride, B, H, Nq) ||
      (Nk > 0 && (!strides_aligned(a->k_stride, B, Hk, Nk) || !strides_aligned(a->v_stride, B, Hk, Nk))) ||
      (!shards && !strides_aligned(o_stride, B, H, Nq)))
    return XS_ERR_ALIGN;
  // d = 256: one map after the other with a workspace (the norm needs the whole row in one CTA),
  // both at once on halves of v's columns without. A small workspace has places for fewer CTAs.
  const unsigned long long room = ws && ws_bytes > XS_WORKSPACE_HEADER_BYTES ? ws_bytes - XS_WORKSPACE_HEADER_BYTES : 0;
  const int rows = wide_rows(Nq);
  const bool fits = d == 256 && room >= wide_stash_bytes(rows);
  if (d == 256 && a->norm_weight && Nk > 0 && !fits) return XS_ERR_INVALID;

  DiffParams p;
  std::memset(&p, 0, sizeof(p));
  p.B = B;
  p.H = H;
  p.group = H / Hk;
  p.Nq = Nq;
  p.Nk = Nk;
  if (shards) {
    for (int i = 0; i < P; ++i) p.shards[i] = shards[i];
    p.shard_mode = 1;
    p.rows_per_shard = Nq / P;
  } else {
    p.o = o;
    p.o_b = o_stride[0];
    p.o_h = o_stride[1];
    p.o_n = o_stride[2];
  }
  const int sms = sm_count();
  if (sms <= 0) return XS_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (Nk == 0) return launch_diff_zero(p, d, sms * 8, s) == cudaSuccess ? XS_OK : XS_ERR_CUDA;
  if (!encode_operand(&p.tm_q, a->q, B, H, Nq, d, a->q_stride) ||
      !encode_operand(&p.tm_k, a->k, B, Hk, Nk, d, a->k_stride) ||
      !encode_operand(&p.tm_v, a->v, B, Hk, Nk, d, a->v_stride))
    return XS_ERR_CUDA;
  p.lambda = a->lambda;
  p.weight = a->norm_weight;
  p.kv_len = a->kv_len;
  p.n_qtiles = static_cast<int>(qtiles);
  const int nk = (Nk + kTileRows - 1) / kTileRows;
  p.min_places = min_places(d, nk, Nq < kTileRows ? Nq : kTileRows);
  const bool ragged = a->kv_len != nullptr;
  const long long tiles = static_cast<long long>(B) * H * p.n_qtiles;
  // Workspace of the d = 256 kernel: counters | a CTA's place for map 1 each | partial results.
  const unsigned long long places = room / wide_stash_bytes(rows);
  const int ctas = places < static_cast<unsigned long long>(sms) ? static_cast<int>(places) : sms;
  Plan pl{0, 0, 0, 0, 0};
  bool wide = fits;
  if (fits)
    pl = plan(tiles, ctas, nk, ragged, p.min_places, merge_cost(d, rows), wide_parts_bytes(rows),
              room - ctas * wide_stash_bytes(rows));
  if (!fits || !a->norm_weight) {
    // Workspace of the others: counters | partial results (none on halves of v's columns).
    const Plan other = plan(d == 256 ? 2 * tiles : tiles, sms, nk, ragged, p.min_places, merge_cost(d, kTileRows),
                            parts_bytes(1, d), d == 256 ? 0 : room);
    wide = fits && wide_ns(pl) <= halves_ns(other);
    if (!wide) pl = other;
  }
  p.v_parts = d == 256 && !wide ? 2 : 1;
  p.units_b = H * p.n_qtiles * p.v_parts;
  p.n_units = B * p.units_b;
  p.split = pl.split;
  p.waves = pl.waves;
  p.scale_log2 = static_cast<float>(1.4426950408889634 * static_cast<double>(a->scale));
  p.eps = a->eps;
  p.out_scale = a->out_scale;
  if (device_status_word(&p.status) != cudaSuccess) return XS_ERR_CUDA;
  p.wait_limit_ns = wait_limit_ns();
  p.count = static_cast<int *>(ws);
  float *area = ws ? reinterpret_cast<float *>(static_cast<char *>(ws) + XS_WORKSPACE_HEADER_BYTES) : nullptr;
  p.parts = area;
  if (!wide) return launch_attn_diff(p, d, pl.grid, s) == cudaSuccess ? XS_OK : XS_ERR_CUDA;
  p.part_rows = rows;
  p.stash = area;
  p.parts = area + ctas * wide_stash_bytes(rows) / 4;
  return launch_attn_diff_wide(p, pl.grid, s) == cudaSuccess ? XS_OK : XS_ERR_CUDA;
}

}  // namespace

XS_API xs_status xs_diff_attn(const xs_diff_args *args, void *o, const long long *o_stride, void *ws,
                              unsigned long long ws_bytes, void *stream) {
  return diff_call(args, o, o_stride, nullptr, 0, ws, ws_bytes, stream);
}

XS_API xs_status xs_diff_attn_fused(const xs_diff_args *args, void *const *out_shards, int P,
                                    void *ws, unsigned long long ws_bytes, void *stream) {
  if (!out_shards) return XS_ERR_INVALID;
  return diff_call(args, nullptr, nullptr, out_shards, P, ws, ws_bytes, stream);
}

XS_API xs_status xs_diff_workspace_bytes(int B, int H, int Nq, int Nk, int d, int norm,
                                         unsigned long long *bytes) {
  (void)norm;   // no schedule depends on it so far
  if (!bytes || B < 0 || H < 0 || Nq < 0 || Nk < 0) return XS_ERR_INVALID;
  if (d != 64 && d != 128 && d != 256) return XS_ERR_UNSUPPORTED;
  *bytes = 0;
  if (B == 0 || H == 0 || Nq == 0 || Nk == 0) return XS_OK;
  const int sms = sm_count();
  if (sms <= 0) return XS_ERR_CUDA;
  const int rows = wide_rows(Nq);
  *bytes = XS_WORKSPACE_HEADER_BYTES +
           (d == 256 ? sms * (wide_stash_bytes(rows) + wide_parts_bytes(rows)) : parts_bytes(sms, d));
  return XS_OK;
}
