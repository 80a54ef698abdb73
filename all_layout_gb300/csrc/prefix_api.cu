// C-ABI entry points of shared-prefix attention (declared in include/xs.h): argument
// validation, tensor maps, the schedule's plan and the launches. Host code only.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/xs.h"
#include "prefix.h"

#define XS_API extern "C" __attribute__((visibility("default")))

namespace {

using namespace xs;

constexpr int kMostLength = 1 << 29;   // (places of a split region then fit 32 bits)
constexpr unsigned long long kCutsBytes = 4096;   // one int4 for each CTA, at most 256 of them

bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// A tensor's strides over more than one row: at least d, and aligned.
bool strides_apart(const long long *stride, const long long *extent, int n, int d) {
  for (int i = 0; i < n; ++i)
    if (extent[i] > 1 && stride[i] < d) return false;
  return true;
}
bool strides_aligned(const long long *stride, const long long *extent, int n) {
  for (int i = 0; i < n; ++i)
    if (extent[i] > 1 && (stride[i] % 8 != 0 || stride[i] >= (1LL << 38))) return false;
  return true;
}

// [batch][heads][rows][d] with strides (batch, head, row) as a map {d, rows, heads, batch}.
bool encode_operand(CUtensorMap *m, const void *base, long long B, int H, int N, int d, long long sb, long long sh,
                    long long sn, unsigned box_rows) {
  const unsigned long long dims[4] = {static_cast<unsigned long long>(d), static_cast<unsigned long long>(N),
                                      static_cast<unsigned long long>(H), static_cast<unsigned long long>(B)};
  unsigned long long st[3] = {static_cast<unsigned long long>(sn) * 2, static_cast<unsigned long long>(sh) * 2,
                              static_cast<unsigned long long>(sb) * 2};
  for (int i = 0; i < 3; ++i)
    if (dims[i + 1] == 1) st[i] = static_cast<unsigned long long>(d) * 2;
  const unsigned box[4] = {64, box_rows, 1, 1};
  return encode_map(m, base, 4, dims, st, box);
}

// Codes of a cache's keys, two as one element: a map {d / 2, rows of a page, heads, pages}.
bool encode_codes(CUtensorMap *m, const xs_cache &c, unsigned box_rows) {
  const unsigned long long page = c.page_size, d = c.d;
  const unsigned long long dims[4] = {d / 2, page, static_cast<unsigned long long>(c.H_kv), static_cast<unsigned long long>(c.n_pages)};
  const unsigned long long st[3] = {d, page * d, c.H_kv * page * d};
  const unsigned box[4] = {static_cast<unsigned>(c.d / 2), box_rows, 1, 1};
  return encode_map(m, c.k, 4, dims, st, box, c.d);
}

// Whole units on min(units, sms) CTAs, or with `room` bytes for partial results the split schedule,
// whichever should end earlier; costs in KV tiles. `mean`, `most`: tiles of a unit; `join`: what pieces and
// the launch that joins them cost.
struct Plan {
  int split, waves, grid;
  double cost;
};
Plan plan(long long units, int sms, double cost_each, double mean, double most, int least, double join, unsigned long long per_cta,
          unsigned long long room) {
  const int grid0 = units < sms ? static_cast<int>(units) : sms;
  const long long rounds = (units + grid0 - 1) / grid0;
  const double unit = mean + cost_each;
  const Plan whole{0, 0, grid0, (rounds - 1) * unit + most};   // (every CTA pays for the start of one unit)
  if (most < 2 || static_cast<unsigned long long>(sms) * sizeof(int4) > kCutsBytes) return whole;
  const int waves = units >= sms ? static_cast<int>(units / sms) - 1 : 0;
  const long long left = units - static_cast<long long>(waves) * sms;
  double per = left * unit / sms;
  int grid = sms;
  if (per < least) {
    per = least;
    grid = static_cast<int>(left * unit / per) + 1;
    if (grid > sms) grid = sms;
  }
  if (per_cta * grid > room) return whole;
  const double cost = waves * unit + per + join;
  return cost < whole.cost ? Plan{1, waves, grid, cost} : whole;
}

// What a launch is to do, of the batch entries of one launch.
struct Shape {
  int B, group, Hk, Nq, Np, Nk, d;
  bool ragged, cached;   // lengths on the device; keys in the cache
};
struct Choice {
  bool tall;
  int grain, nq_rows, entry_rows, copies, row_tile, n_tiles, unit_cost, own_cost;
  long long rows;
  Plan plan;
  double us;
};
constexpr int kLeast = 4;   // the shortest range worth a CTA

Choice choose(const Shape &s, bool tall, int sms, unsigned long long room) {
  Choice c;
  c.tall = tall;
  c.grain = tall ? kTileRows : 16;
  c.nq_rows = tall ? (s.Nq + 7) / 8 * 8 : s.Nq;
  // (In the tall kernel a tile of 128 rows belongs to one request.)
  long long entry = static_cast<long long>(s.group) * c.nq_rows;
  if (tall) entry = (entry + kTileRows - 1) / kTileRows * kTileRows;
  c.entry_rows = static_cast<int>(entry);
  c.rows = s.B * entry;
  c.copies = tall ? 1 : c.rows <= 32 ? 4 : c.rows <= 64 ? 2 : 1;
  c.row_tile = tall ? 2 * kTileRows : kTileRows / c.copies;
  c.n_tiles = static_cast<int>((c.rows + c.row_tile - 1) / c.row_tile);
  // Own tiles of a unit: those of the entries that its rows belong to, two entries' where a unit's rows cross
  // from one to the next (lengths on the device are three quarters of Nk on average).
  const double own = (static_cast<double>((static_cast<long long>(s.Nk) + c.grain - 1) / c.grain * c.grain)) / kTileRows;
  const long long met = c.n_tiles + (entry % c.row_tile == 0 || c.row_tile % entry == 0 ? 0 : s.B - 1);
  const double here = entry >= c.row_tile ? static_cast<double>(met) / c.n_tiles : static_cast<double>(s.B) / c.n_tiles;
  const double top = entry >= c.row_tile ? (met > c.n_tiles ? 2 : 1)
                                         : std::fmin(s.B, (c.row_tile + entry - 1) / entry + (c.row_tile % entry == 0 ? 0 : 1));
  const double prefix = (s.Np + kTileRows - 1) / kTileRows;
  // Times of a KV tile (GB300, us; 64 tiles a CTA, 128, 64 and 32 rows): the flat kernel at d = 128 1.76, 1.64
  // and 1.60 with keys in tensors, 1.79, 1.23 and 1.06 with cached ones; at d = 64 1.22, 0.95 and 0.93, 1.53, 1.03
  // and 0.87. The tall kernel's, for a pair of row tiles: 1.4 and 1.05. The join: 6 us, in the tall kernel 10.
  const bool half = s.d == 64, one = c.copies == 1;
  const double us = tall ? (half ? 1.05 : 1.4)
                         : s.cached ? (half ? (one ? 1.59 : 0.93) : one ? 1.82 : 1.1) : half ? (one ? 1.26 : 0.94) : one ? 1.74 : 1.6;
  // What a unit costs beside its tiles (its queries, its epilogue, the pipeline's start and end), and an own tile
  // whose rows are of several requests, in tiles (see place_of): one token for 8 requests takes 28 us so and 33
  // with 2 and 1, for 16 behind 64K keys 93 and 105; the tall kernel's costs are 2 and 1.
  c.unit_cost = tall ? 2 : 8;
  c.own_cost = !tall && top > 1 ? 2 : 1;
  const double own_places = own * c.own_cost;
  c.plan = plan(static_cast<long long>(s.Hk) * c.n_tiles, sms, c.unit_cost, prefix + own_places * here * (s.ragged ? 0.75 : 1.0),
                prefix + own_places * top, kLeast, (tall ? 10 : 6) / us, 2ull * prefix_part_floats(s.d, c.row_tile) * 4, room);
  c.us = c.plan.cost * us + (tall ? 6.5 : 7.5);   // to the first tile's scores and from the last product to the end
  return c;
}

// Bytes of the workspace that hold cached keys and values read back to bf16, K and V.
unsigned long long unpacked(long long rows, int d) { return (4ull * rows * d + 511) / 512 * 512; }
// Their time: half as much is read as is written.
double unpack_us(unsigned long long bytes) { return bytes == 0 ? 0.0 : 3.0 + bytes * 1.5 / 6.3e6; }

xs_status prefix_call(const xs_prefix_args *a, void *o, const long long *o_stride, void *const *shards, int P,
                      void *ws, unsigned long long ws_bytes, void *stream) {
  if (!a || !a->q) return XS_ERR_INVALID;
  const int B = a->B, H = a->H, Hk = a->H_kv, Nq = a->Nq, Np = a->Np, Nk = a->Nk, d = a->d;
  if (B < 0 || H < 0 || Hk < 0 || Nq < 0 || Np < 0 || Nk < 0) return XS_ERR_INVALID;
  if (H > 0 && (Hk < 1 || H % Hk != 0)) return XS_ERR_INVALID;
  if (!(a->scale > 0.f) || std::isinf(a->scale)) return XS_ERR_INVALID;
  const bool prefix_cached = Np > 0 && !a->prefix_k, own_cached = Nk > 0 && !a->k;
  if (Np > 0 && a->prefix_k && !a->prefix_v) return XS_ERR_INVALID;
  if (Nk > 0 && a->k && !a->v) return XS_ERR_INVALID;
  xs_status st = XS_OK;
  if (prefix_cached || own_cached) {
    st = check_cache(&a->cache);
    if (st == XS_ERR_INVALID) return st;
    if (a->cache.H_kv != Hk || a->cache.d != d) return XS_ERR_INVALID;
    if ((prefix_cached && check_pages(&a->prefix_pages, 1) == XS_ERR_INVALID) ||
        (own_cached && check_pages(&a->pages, B) == XS_ERR_INVALID))
      return XS_ERR_INVALID;
  }
  if (shards) {
    if (P < 1 || P > kMaxShards || Nq % P != 0) return XS_ERR_INVALID;
    for (int p = 0; p < P; ++p)
      if (!shards[p]) return XS_ERR_INVALID;
  } else if (!o || !o_stride) {
    return XS_ERR_INVALID;
  }
  if (!ws && ws_bytes != 0) return XS_ERR_INVALID;
  const bool empty = B == 0 || H == 0 || Nq == 0;
  const long long q_extent[3] = {B, H, Nq}, k_extent[3] = {B, Hk, Nk}, p_extent[2] = {Hk, Np};
  const bool dense_prefix = Np > 0 && !prefix_cached, dense_own = Nk > 0 && !own_cached;
  if (!empty) {
    if (!strides_apart(a->q_stride, q_extent, 3, d) || (!shards && !strides_apart(o_stride, q_extent, 3, d)) ||
        (dense_prefix && (!strides_apart(a->prefix_k_stride, p_extent, 2, d) ||
                          !strides_apart(a->prefix_v_stride, p_extent, 2, d))) ||
        (dense_own && (!strides_apart(a->k_stride, k_extent, 3, d) || !strides_apart(a->v_stride, k_extent, 3, d))))
      return XS_ERR_INVALID;
  }
  if (st == XS_ERR_UNSUPPORTED || (d != 64 && d != 128)) return XS_ERR_UNSUPPORTED;
  if (Np > kMostLength || Nk > kMostLength || Nq > kMostLength) return XS_ERR_UNSUPPORTED;
  // Entries of a launch: as many as the kernels' table holds, and as their packed keys stay within 2^29 for.
  const long long padded = (static_cast<long long>(Nk) + kTileRows - 1) / kTileRows * kTileRows;
  int chunk = kPrefixEntries;
  if (padded > 0 && kMostLength / padded < chunk) chunk = static_cast<int>(kMostLength / padded);
  if (chunk < 1) chunk = 1;
  if (chunk > B) chunk = B;
  const int group = H > 0 ? H / Hk : 1;
  if (!empty && (static_cast<double>(chunk) * group * (Nq + 135.0) > 2147483647.0 - 256 ||
                 (static_cast<double>(chunk) * group * (Nq + 135.0) / 32 + 1) * Hk > 2147483647.0))
    return XS_ERR_UNSUPPORTED;
  if (st != XS_OK || !aligned(a->q, 16) || !aligned(a->prefix_k, 16) || !aligned(a->prefix_v, 16) ||
      !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(o, 16) || !aligned(a->kv_len, 4) || !aligned(ws, 256) ||
      (prefix_cached && !aligned(a->prefix_pages.pages, 4)) || (own_cached && !aligned(a->pages.pages, 4)))
    return XS_ERR_ALIGN;
  if (shards)
    for (int p = 0; p < P; ++p)
      if (!aligned(shards[p], 16)) return XS_ERR_ALIGN;
  if (empty) return XS_OK;
  if (!strides_aligned(a->q_stride, q_extent, 3) || (!shards && !strides_aligned(o_stride, q_extent, 3)) ||
      (dense_prefix && (!strides_aligned(a->prefix_k_stride, p_extent, 2) ||
                        !strides_aligned(a->prefix_v_stride, p_extent, 2))) ||
      (dense_own && (!strides_aligned(a->k_stride, k_extent, 3) || !strides_aligned(a->v_stride, k_extent, 3))))
    return XS_ERR_ALIGN;
  PrefixParams p;
  std::memset(&p, 0, sizeof(p));
  if (shards) {
    for (int i = 0; i < P; ++i) p.shards[i] = shards[i];
    p.shard_mode = 1;
    p.rows_per_shard = Nq / P;
  } else {
    p.o_b = o_stride[0];
    p.o_h = o_stride[1];
    p.o_n = o_stride[2];
  }
  const int sms = sm_count();
  if (sms <= 0) return XS_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  p.H = H;
  p.Hk = Hk;
  p.group = group;
  p.Nq = Nq;
  p.Np = Np;
  p.Nk = Nk;
  p.q_b = a->q_stride[0];
  p.q_h = a->q_stride[1];
  p.q_n = a->q_stride[2];
  const unsigned long long room = ws && ws_bytes > kCutsBytes ? ws_bytes - kCutsBytes : 0;
  char *area = room > 0 ? static_cast<char *>(ws) + kCutsBytes : nullptr;
  p.cuts = static_cast<int4 *>(ws);
  // The kernel: with many rows the tall one, which wants cached keys and values in the workspace first.
  Shape shape{chunk, group, Hk, Nq, Np, Nk, d, a->kv_len != nullptr, Np >= Nk ? prefix_cached : own_cached};
  const unsigned long long prefix_bytes = prefix_cached ? unpacked(static_cast<long long>(Hk) * Np, d) : 0;
  const unsigned long long own_bytes = own_cached ? unpacked(static_cast<long long>(B) * Hk * Nk, d) : 0;
  bool tall = false;
  if (prefix_bytes + own_bytes <= room) {
    const Choice x = choose(shape, true, sms, room - prefix_bytes - own_bytes), y = choose(shape, false, sms, room);
    tall = static_cast<long long>(chunk) * group * Nq > kTileRows &&
           x.us + unpack_us(prefix_bytes + own_bytes) / ((B + chunk - 1) / chunk) < y.us;
  }
  const void *prefix_k = a->prefix_k, *prefix_v = a->prefix_v, *own_k = a->k, *own_v = a->v;
  long long pk_stride[2] = {a->prefix_k_stride[0], a->prefix_k_stride[1]};
  long long pv_stride[2] = {a->prefix_v_stride[0], a->prefix_v_stride[1]};
  long long k_stride[3], v_stride[3];
  std::memcpy(k_stride, a->k_stride, sizeof(k_stride));
  std::memcpy(v_stride, a->v_stride, sizeof(v_stride));
  unsigned long long parts_room = room;
  if (tall) {
    if (prefix_cached) {
      const long long st[3] = {0, static_cast<long long>(Np) * d, d};
      char *v = area + prefix_bytes / 2;
      if (xs_cache_read(&a->cache, area, v, st, st, &a->prefix_pages, nullptr, nullptr, 1, Np, XS_BF16, stream) != XS_OK)
        return XS_ERR_CUDA;
      prefix_k = area;
      prefix_v = v;
      pk_stride[0] = pv_stride[0] = st[1];
      pk_stride[1] = pv_stride[1] = d;
      area += prefix_bytes;
    }
    if (own_cached) {
      const long long st[3] = {static_cast<long long>(Hk) * Nk * d, static_cast<long long>(Nk) * d, d};
      char *v = area + own_bytes / 2;
      if (xs_cache_read(&a->cache, area, v, st, st, &a->pages, nullptr, a->kv_len, B, Nk, XS_BF16, stream) != XS_OK)
        return XS_ERR_CUDA;
      own_k = area;
      own_v = v;
      std::memcpy(k_stride, st, sizeof(st));
      std::memcpy(v_stride, st, sizeof(st));
      area += own_bytes;
    }
    parts_room -= prefix_bytes + own_bytes;
  } else {
    p.prefix_cached = prefix_cached;
    p.own_cached = own_cached;
    if (prefix_cached || own_cached) {
      p.prefix_pages = lists_of(a->cache, &a->prefix_pages);
      p.own_pages = lists_of(a->cache, &a->pages);
      p.codes[0] = static_cast<const uint8_t *>(a->cache.k);
      p.codes[1] = static_cast<const uint8_t *>(a->cache.v);
      p.scales[0] = a->cache.k_scale;
      p.scales[1] = a->cache.v_scale;
      // (A cache without a page has nothing to load.)
      const unsigned most = a->cache.page_size < kTileRows ? a->cache.page_size : kTileRows;
      if (a->cache.n_pages > 0 && (!encode_codes(&p.tm_c, a->cache, most) || !encode_codes(&p.tm_c16, a->cache, 16)))
        return XS_ERR_CUDA;
    }
  }
  p.parts = reinterpret_cast<float *>(area);
  if (Np > 0 && !p.prefix_cached &&
      (!encode_operand(&p.tm_pk, prefix_k, 1, Hk, Np, d, 0, pk_stride[0], pk_stride[1], kTileRows) ||
       !encode_operand(&p.tm_pv, prefix_v, 1, Hk, Np, d, 0, pv_stride[0], pv_stride[1], kTileRows)))
    return XS_ERR_CUDA;
  if (Nk > 0 && !p.own_cached &&
      (!encode_operand(&p.tm_k, own_k, B, Hk, Nk, d, k_stride[0], k_stride[1], k_stride[2], kTileRows) ||
       !encode_operand(&p.tm_v, own_v, B, Hk, Nk, d, v_stride[0], v_stride[1], v_stride[2], kTileRows) ||
       (!tall && (!encode_operand(&p.tm_k16, own_k, B, Hk, Nk, d, k_stride[0], k_stride[1], k_stride[2], 16) ||
                  !encode_operand(&p.tm_v16, own_v, B, Hk, Nk, d, v_stride[0], v_stride[1], v_stride[2], 16)))))
    return XS_ERR_CUDA;
  if (tall && !encode_operand(&p.tm_q, a->q, B, H, Nq, d, p.q_b, p.q_h, p.q_n, 8)) return XS_ERR_CUDA;
  p.n_prefix = (Np + kTileRows - 1) / kTileRows;
  p.min_places = kLeast;
  p.scale_log2 = static_cast<float>(1.4426950408889634 * static_cast<double>(a->scale));
  if (device_status_word(&p.status) != cudaSuccess) return XS_ERR_CUDA;
  p.wait_limit_ns = wait_limit_ns();
  for (int b0 = 0; b0 < B; b0 += chunk) {
    shape.B = B - b0 < chunk ? B - b0 : chunk;
    const Choice c = choose(shape, tall, sms, parts_room);
    p.b0 = b0;
    p.B = shape.B;
    p.q = static_cast<const uint16_t *>(a->q) + b0 * p.q_b;
    if (!shards) p.o = static_cast<uint16_t *>(o) + b0 * p.o_b;
    p.kv_len = a->kv_len ? a->kv_len + b0 : nullptr;
    if (p.own_cached) p.own_pages.pages = a->pages.pages + b0 * a->pages.stride;
    p.grain = c.grain;
    p.nq_rows = c.nq_rows;
    p.entry_rows = c.entry_rows;
    p.rows = static_cast<int>(c.rows);
    p.copies = c.copies;
    p.row_tile = c.row_tile;
    p.n_tiles = c.n_tiles;
    p.n_units = Hk * c.n_tiles;
    p.by_nq.set(p.nq_rows);
    p.by_entry.set(p.entry_rows);
    p.by_tiles.set(p.n_tiles);
    p.by_shard.set(p.rows_per_shard > 0 ? p.rows_per_shard : 1);
    p.unit_cost = c.unit_cost;
    p.own_cost = c.own_cost;
    p.split = c.plan.split;
    p.waves = c.plan.waves;
    p.grid = c.plan.grid;
    if ((tall ? launch_prefix_tall : launch_prefix_flat)(p, d, c.plan.grid, s) != cudaSuccess) return XS_ERR_CUDA;
    if (p.split && launch_prefix_join(p, d, c.plan.grid, sms, s) != cudaSuccess) return XS_ERR_CUDA;
  }
  return XS_OK;
}

}  // namespace

XS_API xs_status xs_prefix_attn(const xs_prefix_args *args, void *o, const long long *o_stride, void *ws,
                                unsigned long long ws_bytes, void *stream) {
  return prefix_call(args, o, o_stride, nullptr, 0, ws, ws_bytes, stream);
}

XS_API xs_status xs_prefix_attn_fused(const xs_prefix_args *args, void *const *out_shards, int P, void *ws,
                                      unsigned long long ws_bytes, void *stream) {
  if (!out_shards) return XS_ERR_INVALID;
  return prefix_call(args, nullptr, nullptr, out_shards, P, ws, ws_bytes, stream);
}

XS_API xs_status xs_prefix_workspace_bytes(int B, int H, int H_kv, int Nq, int Np, int Nk, int d, int cached,
                                           unsigned long long *bytes) {
  if (!bytes || B < 0 || H < 0 || H_kv < 0 || Nq < 0 || Np < 0 || Nk < 0 ||
      (cached & ~(XS_PREFIX_CACHED | XS_OWN_CACHED)) != 0)
    return XS_ERR_INVALID;
  if (H > 0 && (H_kv < 1 || H % H_kv != 0)) return XS_ERR_INVALID;
  if (d != 64 && d != 128) return XS_ERR_UNSUPPORTED;
  *bytes = 0;
  if (B == 0 || H == 0 || Nq == 0) return XS_OK;
  const int sms = sm_count();
  if (sms <= 0) return XS_ERR_CUDA;
  *bytes = kCutsBytes + 2ull * sms * prefix_part_floats(d, 2 * kTileRows) * 4;
  // Rows that one tile of the flat kernel holds never go to the tall one.
  if (static_cast<double>(B) * (H / H_kv) * Nq > kTileRows) {
    if (cached & XS_PREFIX_CACHED) *bytes += unpacked(static_cast<long long>(H_kv) * Np, d);
    if (cached & XS_OWN_CACHED) *bytes += unpacked(static_cast<long long>(B) * H_kv * Nk, d);
  }
  return XS_OK;
}
