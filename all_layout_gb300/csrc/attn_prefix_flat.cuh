// The flat kernel of shared-prefix attention (included by attn_prefix.cu): one tile of up to 128
// rows at a time, for calls with few rows for each k/v head, where reading the keys is the bound.
//
// Copies. The tensor cores always work on 128 rows. With 64 rows or fewer (or 32) the tile holds
// the rows twice (four times), and each copy's softmax takes its half (quarter) of a KV tile's
// keys, the weights of the others being zero: a tile's exponentials are then halved (quartered),
// and the epilogue adds the copies' results, each with its own maximum and sum.
//
// Cached keys. Their codes are operands as they are: TMA brings them from the cache's pages in the layout that the
// MMAs read, and the scores are multiplied by the keys' scales. The queries that meet them are two 8-bit matrices, each
// row times a power of two: of a bf16 value's 8 significant bits e5m2 takes the first 3, and what that rounding
// leaves, an integer of at most 16 in units of the last one, fits e4m3's 4. An MMA in 8 bits takes half as long, so
// the two cost what one in bf16 would; its sums are as exact (a term 2^-26 of the others' came through).
// Scores come out below 2^28 in magnitude (queries below 2^12, codes 448, 128 columns), and scales reach 2^119. So a key's
// factor is its scale times kKeyDown, and a row's factor has the rest: the product of a score and a key's factor is finite, and
// exact or off by 2^-150, times 2^128 at most. A row whose factor would not be finite (queries of 2^119 and more) has kKeyDown
// taken back as its scores are masked.
// Cached values. Their codes and scales go to raw slots, and two groups of four warps turn every second tile of them
// into a bf16 operand (what it is multiplied with, the weights, needs bf16's range): a code's bits moved to bf16's
// place stand for code * 2^-120, so one product with 2^(120 + e) is exact (e > 7 takes two).
//
// Roles (512 threads, one CTA per SM):
//   warps 0-3   softmax, row r of the tile = TMEM lane r
//   warps 4-11  V: codes to bf16, TMA loads of tiles that are not cached, and the queries to Tensor Memory
//   warp 12     issues the scores; scales of the keys; Tensor Memory allocation
//   warp 13     issues the products with V
//   warp 14     loads K; warp 15 loads V's codes and scales
// Tensor Memory: S0 [0,128) S1 [128,256) O [256,256+d) the queries in 8 bits [384,384+d/2), in bf16 [448,448+d/2);
// P_t over S_t's first 64 columns. Scores are double-buffered: QK(i+1) runs beside tile i's softmax.
// Queries are read from Tensor Memory because shared memory is what the SM has least of here. Measured at one token
// for 16 requests of 24 heads behind 64K keys (420 MB of codes): 93 us; with K's codes turned to fp16 operands by four
// warps and V's by four others 120 us, the warps of V setting the pace. A KV tile takes 0.81 us (the same behind 128K
// keys: 159 us), 1570 cycles, of which HBM asks 1450 at this SM's share; start, own tiles and join are the other 28 us.

constexpr int kFlatValues = 4, kFlatGroupWarps = 4, kFlatScores = 12, kFlatProducts = 13, kFlatLoadKeys = 14;   // warps
// Requests whose values are not numbers, a bit each and one (kPrefixEntries) for the prefix: by item modulo two
// and warp of V. A row of V that is not a number must not meet the zero weights of other requests' rows, so its
// place in the operand is cleared, and the rows that see it become NaN at the end. Each warp clears its words before
// it arrives for the item's queries: that arrival alone orders them before the softmax's reading, as a group may
// have no tile of the item to arrive for.
constexpr int kBadWords = kPrefixEntries / 32 + 1;

constexpr float kKeyDown = 1.f / (1 << 20);

template <int D>
struct FlatCfg {
  static constexpr int THREADS = 512;
  static constexpr int TILE = BN * D * 2, RAW = BN * D + BN;   // a bf16 tile; V's codes and scale bytes
  // K's slots hold a tile of codes or 64 columns of a bf16 one; V's operands a slot a group, its raw ring FV a group.
  static constexpr int KN = D == 128 ? 5 : 7, VS = 2, FV = D == 128 ? 2 : 4;
  static constexpr int OFF_K = 0, OFF_V = OFF_K + KN * kHalf, OFF_F = OFF_V + VS * TILE;
  static constexpr int OFF_KS = OFF_F + 2 * FV * RAW;          // scale bytes of K's slots
  static constexpr int OFF_STG = OFF_KS + KN * BN;
  static constexpr int OFF_FIN = OFF_STG + BM * 16 * 4;
  static constexpr int OFF_FAC = OFF_FIN + BM * 4;             // scales of cached keys, of four tiles
  static constexpr int OFF_QF = OFF_FAC + 4 * BN * 4;          // factors of the rows
  static constexpr int OFF_BAD = OFF_QF + BM * 4;              // see kBadWords
  static constexpr int OFF_TAB = OFF_BAD + 2 * 2 * kFlatGroupWarps * kBadWords * 4;
  static constexpr int OFF_BAR = OFF_TAB + kTable * 4;
  static constexpr int SMEM = OFF_BAR + 768;
  static constexpr uint32_t COL_O = 256, COL_Q8 = 384, COL_Q = 448;
  static_assert(SMEM <= 232448, "shared memory per CTA");
  static_assert(OFF_BAR % 16 == 0 && RAW % 16 == 0, "alignment");
};

struct FlatBars {
  uint64_t q_full, q_empty;
  uint64_t k_full[7], k_empty[7], v_full[2], v_empty[2];
  uint64_t raw[2];                   // V tiles whose rows behind a request's last key are still to be cleared
  uint64_t f_full[8], f_empty[8];    // V's raw slots, the second group's behind the first one's
  uint64_t s_full[2], p_full[2], pv_done[2], o_full;
  uint64_t drain, q_seen;
  PrefixStart start;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(FlatBars) <= 768, "barrier block too large");

// The scale bytes of a place that no page holds.
__device__ __align__(16) const unsigned g_nan_scales[32] = {
    ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u,
    ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u, ~0u};

// Sixteen packed own keys from `pos` on (the flat kernel's grain): whose they are, where they begin
// among that entry's, and how many of them count (0: none of the item's entries).
struct Grain {
  int b, off, valid;
};
// `b`: the entry of an earlier place of the item, or first_entry's.
__device__ __forceinline__ Grain grain_at(const int *table, const PrefixUnit &u, int pos, int &b) {
  if (pos < table[u.b_lo] || pos >= table[u.b_hi + 1]) return Grain{u.b_lo, 0, 0};
  while (pos >= table[b + 1]) ++b;   // (those without keys end where they begin)
  const int off = pos - table[b];
  return Grain{b, off, min(max(len_of(table, b) - off, 0), 16)};
}
// An entry at or before that of `pos`, or the item's first one.
__device__ __noinline__ int first_entry(const int *table, int lo, int hi, int pos) {
  if (pos < table[lo]) return lo;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (table[mid] <= pos) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Whether tile j of a unit lies in the cache, and the first packed own key of an own tile.
__device__ __forceinline__ bool is_cached(const PrefixParams &p, int j) {
  return j < p.n_prefix ? p.prefix_cached : p.own_cached;
}
__device__ __forceinline__ int own_pos(const PrefixParams &p, const PrefixUnit &u, int j) {
  return (u.t0 + j - p.n_prefix) * BN;
}
// Of this lane's sixteen keys, lanes 0 to 7, in the first own tile from j on.
__device__ __forceinline__ int entry_of(const PrefixParams &p, const int *table, const PrefixUnit &u, int j) {
  return first_entry(table, u.b_lo, u.b_hi, own_pos(p, u, max(j, p.n_prefix)) + (threadIdx.x & 7) * 16);
}

// Whether a tile's keys (a Grain each in lanes 0 to 7) are of one request, one after the other from lane 0 on.
__device__ __forceinline__ bool one_request(const Grain &g) {
  const int lane = threadIdx.x & 31;
  const int first_b = __shfl_sync(0xffffffffu, g.b, 0), first_off = __shfl_sync(0xffffffffu, g.off, 0);
  return __shfl_sync(0xffffffffu, g.valid, 0) > 0 &&
         __all_sync(0xffffffffu, g.valid == 0 || (g.b == first_b && g.off == first_off + 16 * lane));
}

// ------------------------------------------------------------------ loaders
// Sixteen bytes to shared memory, and an arrival when this thread's copies so far have landed.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// A lane's sixteen rows of a cached tile: page number `page` (as it was read: nothing looks at it before the
// tile's turn, so that the load has a tile's time), from row `at` on; none: at < 0.
struct Part {
  int page, at;
};
__device__ __forceinline__ Part part_at(const PrefixParams &p, const int *table, const PrefixItem &item, int j, int &entry) {
  const int lane = threadIdx.x & 31;
  Part r{0, -1};
  if (j >= item.kv1 || !is_cached(p, j) || lane >= BN / 16) return r;
  const bool prefix = j < p.n_prefix;
  const PageLists &list = prefix ? p.prefix_pages : p.own_pages;
  int b = 0, place = j * BN + lane * 16;
  bool live = place < p.Np;
  if (!prefix) {
    const Grain g = grain_at(table, item, own_pos(p, item, j) + lane * 16, entry);
    b = g.b;
    place = g.off;
    live = g.valid > 0;
  }
  if (!live) return r;
  r.at = place & (list.page - 1);
  r.page = -1;
  if ((place >> list.shift) < list.count) r.page = __ldg(list.pages + b * list.stride + (place >> list.shift));
  return r;
}
// Rows that follow each other in a page: whether this lane's are there, and the lanes of its run.
struct Run {
  bool held;
  int first, end;
  unsigned lanes;   // those that hold rows
};
__device__ __forceinline__ Run run_of(const PrefixParams &p, const Part &r) {
  const int lane = threadIdx.x & 31;
  Run x;
  x.held = r.at >= 0 && static_cast<unsigned>(r.page) < static_cast<unsigned>(p.prefix_pages.n_pages);
  const int last_page = __shfl_up_sync(0xffffffffu, x.held ? r.page : -1, 1);
  const int last_at = __shfl_up_sync(0xffffffffu, r.at, 1);
  // (Lanes 8 to 31 hold nothing.)
  const unsigned heads = __ballot_sync(0xffffffffu, !x.held || lane == 0 || last_page != r.page || last_at + 16 != r.at);
  x.lanes = __ballot_sync(0xffffffffu, x.held);
  x.first = 31 - __clz(heads & (0xffffffffu >> (31 - lane)));
  x.end = lane + (lane < 31 ? __ffs(heads >> (lane + 1)) : 1);
  return x;
}

// K's warp loads every tile of K, a slot of its ring for a tile of codes or for 64 columns of a bf16 one.
template <int D>
__device__ void flat_load_keys(const PrefixParams &p, uint8_t *smem, FlatBars *bars, const int *table) {
  using C = FlatCfg<D>;
  volatile int *abort_flag = &bars->abort;
  const int lane = threadIdx.x & 31;
  uint32_t slot = 0, parity = 1, used = 0;   // the ring's next; slots filled so far
  PrefixWalk walk = bars->start.walk;
  PrefixItem item = bars->start.item;
  bool more = bars->start.any != 0;
  bool ok = true;
  const int psize = p.prefix_pages.page;   // one cache: all its pages have one size
  const int big = min(p.prefix_pages.shift, 7) - 4;   // log2 of the lanes whose rows a large box has
  auto next_slot = [&] {
    ++used;
    if (++slot == C::KN) slot = 0, parity ^= 1;
  };
  for (; ok && more; more = next_item(&bars->start, table, &walk, &item)) {
    int j = item.kv0;
    if (p.prefix_cached && psize >= BN) {
      // The prefix's whole tiles, each in one page: a loop of few instructions.
      const int whole = min(item.kv1, p.Np / BN);
      const uint8_t *scales = p.scales[0] + lane * 16;
      const int shift = p.prefix_pages.shift, n_pages = p.prefix_pages.n_pages, count = p.prefix_pages.count;
      auto page_at = [&](int t) {
        const int i = t * BN >> shift;
        return t < whole && i < count ? __ldg(p.prefix_pages.pages + i) : -1;
      };
      int next = page_at(j);
#pragma unroll 1
      for (; j < whole; ++j) {
        const int page = next, at = j * BN & (psize - 1);
        next = page_at(j + 1);   // (not looked at before its turn)
        const bool held = static_cast<unsigned>(page) < static_cast<unsigned>(n_pages);
        const long long row = (static_cast<long long>(page) * p.Hk + item.hk) * psize + at;
        const uint32_t full = smem_u32(&bars->k_full[slot]);
        if (!(ok = wait_for<true>(smem_u32(&bars->k_empty[slot]), parity, abort_flag, p))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(full, held ? BN * D : 0);
          if (held) tma_load_4d(smem_u32(smem + C::OFF_K + slot * kHalf), &p.tm_c, full, 0, at, item.hk, page);
        }
        if (lane < BN / 16) {
          copy16(smem_u32(smem + C::OFF_KS + slot * BN + lane * 16), held ? static_cast<const void *>(scales + row) : g_nan_scales);
          copies_arrive(full);
        }
        __syncwarp();
        next_slot();
      }
    }
    int entry = entry_of(p, table, item, j), beside = entry;   // of part_at and of bf16 tiles
    Part ahead = part_at(p, table, item, j, entry);
    for (; ok && j < item.kv1; ++j) {
      const Part r = ahead;
      ahead = part_at(p, table, item, j + 1, entry);
      if (is_cached(p, j)) {
        // A run's rows in large boxes as far as they go, the rest in boxes of sixteen rows.
        const Run x = run_of(p, r);
        const int in = lane - x.first, whole = (x.end - x.first) >> big << big;
        if (!(ok = wait_for<true>(smem_u32(&bars->k_empty[slot]), parity, abort_flag, p))) break;
        const uint32_t full = smem_u32(&bars->k_full[slot]), dst = smem_u32(smem + C::OFF_K + slot * kHalf);
        if (lane == 0) mbar_arrive_expect_tx(full, __popc(x.lanes) * 16u * D);
        __syncwarp();
        if (x.held && (in >= whole || (in & ((1 << big) - 1)) == 0))
          tma_load_4d(dst + lane * 16 * D, in < whole ? &p.tm_c : &p.tm_c16, full, 0, r.at, item.hk, r.page);
        if (lane < BN / 16) {
          const long long row = (static_cast<long long>(r.page) * p.Hk + item.hk) * psize + r.at;
          if (r.at >= 0)
            copy16(smem_u32(smem + C::OFF_KS + slot * BN + lane * 16),
                   x.held ? static_cast<const void *>(p.scales[0] + row) : g_nan_scales);
          copies_arrive(full);
        }
        __syncwarp();
        next_slot();
        continue;
      }
      // A bf16 tile, 64 columns at a time.
      Grain g{0, 0, 0};
      bool one = true;   // a box of 128 rows: the prefix's (rows past Np come as zeros) and one request's, past its last key too
      if (j >= p.n_prefix) {
        if (lane < BN / 16) g = grain_at(table, item, own_pos(p, item, j) + lane * 16, beside);
        one = one_request(g);
      }
      const uint32_t bytes = one ? kHalf : __popc(__ballot_sync(0xffffffffu, g.valid > 0)) * 16u * 128;
      for (int hf = 0; hf < D / 64; ++hf) {
        if (!(ok = wait_for<true>(smem_u32(&bars->k_empty[slot]), parity, abort_flag, p))) break;
        const uint32_t full = smem_u32(&bars->k_full[slot]), dst = smem_u32(smem + C::OFF_K + slot * kHalf);
        if (lane == 0) mbar_arrive_expect_tx(full, bytes);
        __syncwarp();
        if (lane < BN / 16) mbar_arrive(full);
        if (j < p.n_prefix) {
          if (lane == 0) tma_load_4d(dst, &p.tm_pk, full, hf * 64, j * BN, item.hk, 0);
        } else if (one ? lane == 0 : g.valid > 0) {
          tma_load_4d(dst + lane * 2048, one ? &p.tm_k : &p.tm_k16, full, hf * 64, g.off, item.hk, p.b0 + g.b);
        }
        __syncwarp();
        next_slot();
      }
    }
  }
  // Every load issued must land before the CTA releases its shared memory.
  for (uint32_t s = 0; s < C::KN && s < used; ++s)
    drain(smem_u32(&bars->k_full[(used - 1 - s) % C::KN]), (used - 1 - s) / C::KN & 1);
}

// V's warp loads the codes and scales of cached tiles; tile t is of group t mod 2.
template <int D>
__device__ void flat_load_values(const PrefixParams &p, uint8_t *smem, FlatBars *bars, const int *table) {
  using C = FlatCfg<D>;
  volatile int *abort_flag = &bars->abort;
  const int lane = threadIdx.x & 31;
  uint32_t tile = 0, use[2] = {0, 0};   // tiles so far; cached ones of each group
  PrefixWalk walk = bars->start.walk;
  PrefixItem item = bars->start.item;
  bool more = bars->start.any != 0;
  bool ok = true;
  const int psize = p.prefix_pages.page;
  for (; ok && more; more = next_item(&bars->start, table, &walk, &item)) {
    int j = item.kv0;
    if (p.prefix_cached && psize >= BN) {
      // The prefix's whole tiles, each in one page: a loop of few instructions.
      const int whole = min(item.kv1, p.Np / BN);
      const uint8_t *codes = p.codes[1], *scales = p.scales[1] + lane * 16;
      const int shift = p.prefix_pages.shift, n_pages = p.prefix_pages.n_pages, count = p.prefix_pages.count;
      auto page_at = [&](int t) {
        const int i = t * BN >> shift;
        return t < whole && i < count ? __ldg(p.prefix_pages.pages + i) : -1;
      };
      int next = page_at(j);
#pragma unroll 1
      for (; j < whole; ++j, ++tile) {
        const int page = next;
        next = page_at(j + 1);   // (not looked at before its turn)
        const bool held = static_cast<unsigned>(page) < static_cast<unsigned>(n_pages);
        const long long row = (static_cast<long long>(page) * p.Hk + item.hk) * psize + (j * BN & (psize - 1));
        const uint32_t u = tile & 1 ? use[1] : use[0], slot = (tile & 1) * C::FV + u % C::FV;
        const uint32_t full = smem_u32(&bars->f_full[slot]), dst = smem_u32(smem + C::OFF_F + slot * C::RAW);
        if (!(ok = wait_for<true>(smem_u32(&bars->f_empty[slot]), (u / C::FV & 1) ^ 1, abort_flag, p))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(full, held ? BN * D : 0);
          if (held) bulk_load(dst, codes + row * D, BN * D, full);
        }
        if (lane < BN / 16) {
          copy16(dst + BN * D + lane * 16, held ? static_cast<const void *>(scales + row) : g_nan_scales);
          copies_arrive(full);
        }
        __syncwarp();
        if (tile & 1) ++use[1]; else ++use[0];
      }
    }
    int entry = entry_of(p, table, item, j);
    Part ahead = part_at(p, table, item, j, entry);
    for (; ok && j < item.kv1; ++j, ++tile) {
      const Part r = ahead;
      ahead = part_at(p, table, item, j + 1, entry);
      if (!is_cached(p, j)) continue;
      const Run x = run_of(p, r);
      const long long row = (static_cast<long long>(r.page) * p.Hk + item.hk) * psize + r.at;
      const uint32_t u = tile & 1 ? use[1] : use[0], slot = (tile & 1) * C::FV + u % C::FV;
      if (!(ok = wait_for<true>(smem_u32(&bars->f_empty[slot]), (u / C::FV & 1) ^ 1, abort_flag, p))) break;
      const uint32_t full = smem_u32(&bars->f_full[slot]), dst = smem_u32(smem + C::OFF_F + slot * C::RAW);
      if (lane == 0) mbar_arrive_expect_tx(full, __popc(x.lanes) * 16u * D);
      __syncwarp();
      if (x.held && lane == x.first) bulk_load(dst + lane * 16 * D, p.codes[1] + row * D, (x.end - lane) * 16 * D, full);
      // The scales by the load/store unit, sixteen a lane: a bulk copy takes the copy engine about 300 cycles,
      // however small.
      if (lane < BN / 16) {
        if (r.at >= 0)
          copy16(dst + BN * D + lane * 16, x.held ? static_cast<const void *>(p.scales[1] + row) : g_nan_scales);
        copies_arrive(full);
      }
      __syncwarp();
      if (tile & 1) ++use[1]; else ++use[0];
    }
  }
  // Every load issued must land before the CTA releases its shared memory.
  for (uint32_t g = 0; g < 2; ++g)
    for (uint32_t s = 0; s < C::FV && s < use[g]; ++s)
      drain(smem_u32(&bars->f_full[g * C::FV + (use[g] - 1 - s) % C::FV]), (use[g] - 1 - s) / C::FV & 1);
}

// ------------------------------------------------------------------ operands
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Bytes of x by selector; 8 to 11 are the sign bits of bytes 0 to 3, eight times each.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t prmt(uint32_t x) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(x), "n"(SEL));
  return r;
}
// Two e4m3 codes as 16-bit integers with their signs extended: the bf16 pair of their values times 2^-120.
__device__ __forceinline__ uint32_t spread(uint32_t z) { return z << 4 & 0x87f087f0u; }
// Eight codes of a row with scale byte `byte` to bf16. PLAIN: the byte is at most 134.
template <bool PLAIN>
__device__ __forceinline__ uint4 to_bf16(uint32_t c0, uint32_t c1, uint32_t byte) {
  // 2^(120 + e) in bf16, twice, for e = byte - 127 <= 7.
  uint32_t f = (PLAIN ? byte : min(byte, 134u)) * 0x00800080u + 0x3c003c00u;
  if (!PLAIN && byte == kNanScale) f = 0x7fff7fffu;
  uint32_t r[4] = {spread(prmt<0x9180>(c0)), spread(prmt<0xb3a2>(c0)), spread(prmt<0x9180>(c1)), spread(prmt<0xb3a2>(c1))};
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = mul_bf16x2(r[i], f);
  if (!PLAIN && byte > 134 && byte != kNanScale) {
    const uint32_t g = (byte - 134 + 127) * 0x00800080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = mul_bf16x2(r[i], g);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// This warp has read a raw slot: its arrival at the slot's barrier.
__device__ __forceinline__ void slot_read(uint32_t empty) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(empty);
}

// The top bit of each byte of `codes` that is a NaN (0x7f or 0xff); in the others nothing below it counts.
__device__ __forceinline__ uint32_t nan_bits(uint32_t codes) { return (codes & 0x7f7f7f7fu) + 0x01010101u; }
__device__ __forceinline__ uint32_t nan_bits(const uint4 &c) {
  return nan_bits(c.x) | nan_bits(c.y) | nan_bits(c.z) | nan_bits(c.w);
}
// Whether any of two bf16 values is an infinity or NaN, for each of the halves.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return __vcmpeq2(w & 0x7f807f80u, 0x7f807f80u); }

// Codes and scale bytes of V's raw slot to a bf16 tile; `valid`, `entry`: of the sixteen rows of lanes 0-7
// (valid_of); `bad`: this warp's words for requests whose values are not numbers. A thread has one 16-byte group of
// every STEP-th row, so its place in the swizzle stays. Short loops: with all groups unrolled the warps waited for
// instructions. A tile whose rows all count, with scales of 2^7 at most and no code of a NaN, goes through the first
// loop; another one (the codes show it at that loop's end, before anyone reads the operand) through the second, which
// looks at each row. Looking for NaN's codes takes long history 92.5 us instead of 90; in a pass of its own, while the
// operand's slot is still in use, 94.
template <int D>
__device__ __forceinline__ void convert_values(const uint8_t *src, uint8_t *dst, int valid, int entry, uint32_t *bad, uint32_t tid,
                                           uint32_t empty) {
  constexpr uint32_t CPR = D / 16, STEP = 32 * kFlatGroupWarps / CPR, U = BN / STEP;   // groups of a row's codes
  const uint32_t lane = tid & 31;
  // (Of eight lanes that store together four are in a row's second half: of the neighbouring row, whose swizzle
  // gives them the other banks.)
  const uint32_t cc = tid % CPR, row0 = tid / CPR ^ cc / 4, first = cc % 4 * 2;
  const uint32_t bytes = *reinterpret_cast<const uint32_t *>(src + BN * D + lane * 4);
  const uint8_t *scales = src + BN * D + row0;
  src += row0 * D + cc * 16;
  dst += (cc / 4) * kHalf + row0 * 128;
  const uint32_t first0 = (first ^ (row0 & 7)) * 16, second0 = ((first + 1) ^ (row0 & 7)) * 16;
  const bool clear = __any_sync(0xffffffffu, valid < 16);
  if (!clear && !__any_sync(0xffffffffu, __vcmpgtu4(bytes, 0x86868686u) != 0)) {
    uint4 c[2], next[2];
    uint32_t byte[2], next_byte[2], nan = 0;
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k) {
      c[k] = *reinterpret_cast<const uint4 *>(src + k * STEP * D);
      byte[k] = scales[k * STEP];
    }
#pragma unroll 1
    for (uint32_t i = 0; i < U; i += 2, dst += 2 * STEP * 128) {
      src += 2 * STEP * D;
      scales += 2 * STEP;
      if (i + 2 < U)
#pragma unroll
        for (uint32_t k = 0; k < 2; ++k) {
          next[k] = *reinterpret_cast<const uint4 *>(src + k * STEP * D);
          next_byte[k] = scales[k * STEP];
        }
#pragma unroll
      for (uint32_t k = 0; k < 2; ++k) {
        uint8_t *to = dst + k * STEP * 128;
        *reinterpret_cast<uint4 *>(to + first0) = to_bf16<true>(c[k].x, c[k].y, byte[k]);
        *reinterpret_cast<uint4 *>(to + second0) = to_bf16<true>(c[k].z, c[k].w, byte[k]);
        nan |= nan_bits(c[k]);
        c[k] = next[k];
        byte[k] = next_byte[k];
      }
    }
    if (!__any_sync(0xffffffffu, (nan & 0x80808080u) != 0)) {
      slot_read(empty);
      return;
    }
    src -= U * STEP * D;
    scales -= U * STEP;
    dst -= U * STEP * 128;
  }
#pragma unroll 1
  for (uint32_t i = 0; i < BN / STEP; ++i) {
    const uint4 c = *reinterpret_cast<const uint4 *>(src + i * STEP * D);
    const uint32_t byte = scales[i * STEP], row = row0 + i * STEP;
    uint4 x = to_bf16<false>(c.x, c.y, byte), y = to_bf16<false>(c.z, c.w, byte);
    const bool counts = static_cast<int>(row & 15) < __shfl_sync(0xffffffffu, valid, row >> 4);
    const int b = __shfl_sync(0xffffffffu, entry, row >> 4);
    // (A scale byte of 255 makes NaN of every value, one past 246 infinities of large ones.)
    const bool odd_row = (nan_bits(c) & 0x80808080u) != 0 || (not_finite(x.x) | not_finite(x.y) | not_finite(x.z) | not_finite(x.w) |
                                                              not_finite(y.x) | not_finite(y.y) | not_finite(y.z) | not_finite(y.w)) != 0;
    if (!counts || odd_row) x = y = make_uint4(0, 0, 0, 0);
    if (counts && odd_row) atomicOr(bad + (b >> 5), 1u << (b & 31));
    uint8_t *to = dst + i * STEP * 128;
    *reinterpret_cast<uint4 *>(to + first0) = x;
    *reinterpret_cast<uint4 *>(to + second0) = y;
  }
  slot_read(empty);
}

// Rows of a bf16 tile of V that do not count to zeros, as well as what is not a finite number in those that do,
// which is noted. By four warps; lanes 0-7 know of sixteen rows each whose they are and how many count.
template <int D>
__device__ __noinline__ void clear_rows(uint8_t *tile, int valid, int entry, uint32_t *bad, int tid) {
#pragma unroll 1
  for (int i = 0; i < BN * D / 8 / 128; ++i) {
    const int at = i * 128 + tid, row = at / 8 % BN;   // 16-byte chunks of the halves, one after the other
    uint4 *chunk = reinterpret_cast<uint4 *>(tile) + at;
    const bool counts = (row & 15) < __shfl_sync(0xffffffffu, valid, row >> 4);
    const int b = __shfl_sync(0xffffffffu, entry, row >> 4);
    uint4 v = *chunk;
    const uint32_t x = not_finite(v.x), y = not_finite(v.y), z = not_finite(v.z), w = not_finite(v.w);
    if (counts && (x | y | z | w) == 0) continue;
    if (counts) atomicOr(bad + (b >> 5), 1u << (b & 31));
    v = counts ? make_uint4(v.x & ~x, v.y & ~y, v.z & ~z, v.w & ~w) : make_uint4(0, 0, 0, 0);
    *chunk = v;
  }
}

// Two bf16 pairs, times s, to a word of four e5m2 codes and one of four e4m3 codes of what they leave.
__device__ __forceinline__ void two_codes(uint32_t u, uint32_t v, float s, uint32_t &first, uint32_t &rest) {
  auto pair = [](float x, float y, uint16_t &hi, uint16_t &lo) {
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y), "f"(x));
    uint32_t back;
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(back) : "h"(hi));
    float bx, by;
    asm("{.reg .b16 t, u;\n\tmov.b32 {t, u}, %2;\n\tcvt.f32.f16 %0, t;\n\tcvt.f32.f16 %1, u;}" : "=f"(bx), "=f"(by) : "r"(back));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y - by), "f"(x - bx));
  };
  uint16_t h0, l0, h1, l1;
  pair(__uint_as_float(u << 16) * s, __uint_as_float(u & 0xffff0000u) * s, h0, l0);
  pair(__uint_as_float(v << 16) * s, __uint_as_float(v & 0xffff0000u) * s, h1, l1);
  first = h0 | static_cast<uint32_t>(h1) << 16;
  rest = l0 | static_cast<uint32_t>(l1) << 16;
}
__device__ __forceinline__ void tmem_st2(uint32_t taddr, uint32_t a, uint32_t b) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// An item's queries to Tensor Memory by the warps of V, every second eight columns of a row a thread and group (the
// copies begin at multiples of row_tile). `bad`: this warp's words of the item (kBadWords), cleared here.
template <int D>
__device__ __forceinline__ bool flat_queries(const PrefixParams &p, uint8_t *smem, FlatBars *bars, const PrefixItem &item,
                                          uint32_t items, uint32_t tmem, int group, uint32_t *bad) {
  using C = FlatCfg<D>;
  volatile int *abort_flag = &bars->abort;
  const int tid = threadIdx.x & 127;
  const int row = item.row0 + tid % p.row_tile;
  const uint16_t *src = nullptr;
  if (row < p.rows) {
    const PrefixRow r = row_of(p, item.hk, row);
    if (r.n < p.Nq) src = p.q + r.b * p.q_b + r.h * p.q_h + r.n * p.q_n;
  }
  const uint32_t to = tmem + (static_cast<uint32_t>(tid & ~31) << 16);
  // (The row is read twice, the second time out of L1: held in registers, its conversion would be long code.)
  auto part = [&](int i) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (src)
      asm volatile("ld.global.ca.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(src + 8 * i));
    return v;
  };
  const bool cached = p.prefix_cached || p.own_cached;
  float s = 1.f, back = 1.f;
  if (cached) {
    // For cached keys: times the power of two that brings the row's largest magnitude to [2^11, 2^12) (e4m3 then
    // holds what is left of it), in two parts. Their sum is exact for values down to 2^-13 of that, and off by 2^-10,
    // 2^-21 of it, at most below. A row with an infinity or NaN becomes NaN by its factor.
    uint32_t big = 0;   // largest magnitudes, as bits, of the even and of the odd columns
    uint4 x[D / 8];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) x[i] = part(i);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const uint4 v = x[i];
      big = __vmaxu2(__vmaxu2(big, v.x & 0x7fff7fffu), __vmaxu2(v.y & 0x7fff7fffu, __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
    }
    const int e = static_cast<int>(max(big & 0xffffu, big >> 16) >> 7);
    const int up = min(265 - e, 253);   // 2^(up - 127), 2^(138 - e) mostly
    s = __int_as_float(up << 23);
    back = e == 255 ? NAN : __int_as_float((254 - up) << 23);
  }
  if (items > 0 && (!wait_for<true>(smem_u32(&bars->q_empty), (items - 1) & 1, abort_flag, p) ||
                    !wait_for<true>(smem_u32(&bars->q_seen), (items - 1) & 1, abort_flag, p)))
    return false;
  // (The softmax is done with the item before last, as it has begun the last one.)
  if ((tid & 31) < kBadWords) bad[tid & 31] = 0;
  __syncwarp();
  if (group == 0) reinterpret_cast<float *>(smem + C::OFF_QF)[tid] = back;
  tc_fence_after();   // (the last item's scores, read from here, are done)
#pragma unroll 1
  for (int c = group; c < D / 8; c += 2) {
    const uint4 v = part(c);
    if (!p.prefix_cached || !p.own_cached) tmem_st4(to + C::COL_Q + 4 * c, v.x, v.y, v.z, v.w);
    if (cached) {
      uint32_t first[2], rest[2];
      two_codes(v.x, v.y, s, first[0], rest[0]);
      two_codes(v.z, v.w, s, first[1], rest[1]);
      tmem_st2(to + C::COL_Q8 + 2 * c, first[0], first[1]);
      tmem_st2(to + C::COL_Q8 + D / 4 + 2 * c, rest[0], rest[1]);
    }
  }
  tmem_wait_st();
  tc_fence_before();
  mbar_arrive(smem_u32(&bars->q_full));
  return true;
}

// The warps of V, two groups of four: every second tile's operand each, in a slot of its own.
template <int D>
__device__ void flat_values(const PrefixParams &p, uint8_t *smem, FlatBars *bars, const int *table, uint32_t tmem, int group) {
  using C = FlatCfg<D>;
  volatile int *abort_flag = &bars->abort;
  const int tid = threadIdx.x & 127, lane = tid & 31;
  const bool issuer = tid < 32;
  uint8_t *dst = smem + C::OFF_V + group * C::TILE;
  const uint32_t full = smem_u32(&bars->v_full[group]), empty = smem_u32(&bars->v_empty[group]);
  const uint32_t raw_full = smem_u32(&bars->raw[group]);
  auto wait = [&](uint32_t bar, uint32_t parity) { return wait_for<true>(bar, parity, abort_flag, p); };
  uint32_t tile = 0, items = 0;            // tiles of all items before this one
  uint32_t use = 0, f_use = 0, r_use = 0;  // uses of the slot, of the group's raw ring, of raw_full
  bool loading = false, raw_loading = false;   // the slot's last use, raw_full's last, are loads of this warp's
  PrefixWalk walk = bars->start.walk;
  PrefixItem item = bars->start.item;
  bool more = bars->start.any != 0;

  uint32_t *bad = nullptr;   // the item's words
  int entry = 0;             // see grain_at
  // Lanes 0-7: of sixteen keys each, whose they are and how many count. (Rows of V behind a request's last key
  // have the weight 0, but what lies there may not be a number.)
  auto valid_of = [&](int j) {
    if (lane >= BN / 16) return Grain{0, 0, 16};
    if (j < p.n_prefix) return Grain{kPrefixEntries, 0, min(max(p.Np - j * BN - lane * 16, 0), 16)};
    return grain_at(table, item, own_pos(p, item, j) + lane * 16, entry);
  };
  // A cached tile; `valid`, `entry` as convert_values takes them.
  auto convert = [&](int valid, int entry) {
    const uint32_t f = group * C::FV + f_use % C::FV;
    if (!wait(smem_u32(&bars->f_full[f]), f_use / C::FV & 1) || !wait(empty, (use & 1) ^ 1)) return false;
    convert_values<D>(smem + C::OFF_F + f * C::RAW, dst, valid, entry, bad, tid, smem_u32(&bars->f_empty[f]));
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(full);
    ++f_use;
    ++use;
    loading = false;
    return true;
  };
  // A tile that is not cached, by TMA. All warps wait for the slot and arrive at its barrier, though one of them
  // issues: a phase then cannot end before each has seen the one before it. (One that fell two phases behind
  // would take the next for its own.)
  auto load = [&](int j) {
    if (!wait(empty, (use & 1) ^ 1)) return false;
    ++use;
    loading = true;
    if (j < p.n_prefix) {   // (rows past Np come as zeros)
      if (issuer && lane == 0) {
        mbar_arrive_expect_tx(full, C::TILE);
        for (int hf = 0; hf < D / 64; ++hf) tma_load_4d(smem_u32(dst) + hf * kHalf, &p.tm_pv, full, hf * 64, j * BN, item.hk, 0);
      } else if (lane == 0) {
        mbar_arrive(full);
      }
      __syncwarp();
      return true;
    }
    Grain g{0, 0, 0};
    if (lane < BN / 16) g = grain_at(table, item, own_pos(p, item, j) + lane * 16, entry);
    // Keys of one request lie one after the other: a box of 128 rows, which may reach past its last.
    const bool one = one_request(g);
    const uint32_t bytes = one ? C::TILE : __popc(__ballot_sync(0xffffffffu, g.valid > 0)) * 16u * D * 2;
    // Rows behind a request's last key are still to be cleared then, and those of an item of several requests to
    // be looked through.
    const bool whole = item.b_lo == item.b_hi && __popc(__ballot_sync(0xffffffffu, g.valid == 16)) == BN / 16;
    const uint32_t bar = whole ? full : raw_full;
    if (issuer) {
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
      __syncwarp();
      if (one ? lane == 0 : g.valid > 0)
        for (int hf = 0; hf < D / 64; ++hf)
          tma_load_4d(smem_u32(dst) + hf * kHalf + lane * 2048, one ? &p.tm_v : &p.tm_v16, bar, hf * 64, g.off, item.hk, p.b0 + g.b);
    } else if (whole && lane == 0) {
      mbar_arrive(full);
    }
    __syncwarp();
    if (whole) return true;
    loading = false;
    raw_loading = true;
    if (!wait(raw_full, r_use & 1)) return false;
    ++r_use;
    raw_loading = false;
    const Grain v = valid_of(j);
    clear_rows<D>(dst, v.valid, v.b, bad, tid);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(full);
    return true;
  };

  bool ok = true;
  for (; ok && more; ++items, more = next_item(&bars->start, table, &walk, &item)) {
    bad = reinterpret_cast<uint32_t *>(smem + C::OFF_BAD) + ((items & 1) * 2 * kFlatGroupWarps + group * kFlatGroupWarps + tid / 32) * kBadWords;
    ok = flat_queries<D>(p, smem, bars, item, items, tmem, group, bad);
    if (!ok) break;
    int j = item.kv0 + ((tile ^ group) & 1);
    tile += item.kv1 - item.kv0;
    const int whole = p.Np / BN;   // of the prefix's tiles
    entry = entry_of(p, table, item, j);
#pragma unroll 1
    for (; ok && j < item.kv1; j += 2) {
      if (is_cached(p, j)) {
        Grain g{kPrefixEntries, 0, 16};
        if (j >= whole) g = valid_of(j);
        ok = convert(g.valid, g.b);
      } else {
        ok = load(j);
      }
    }
  }
  // Every load issued must land before the CTA releases its shared memory.
  if (issuer && loading) drain(full, (use - 1) & 1);
  if (issuer && raw_loading) drain(raw_full, r_use & 1);
}

// ------------------------------------------------------------------ MMA issuer
// Scores of a tile of codes: the queries' two parts one after the other. (Formats: 0 e4m3, 1 e5m2.)
template <int D>
__device__ __forceinline__ void issue_qk_codes(uint32_t dcol, uint32_t qcol, uint64_t kdesc) {
  constexpr uint32_t rest = idesc_bf16_f32(128, 128, 0) & ~(9u << 7), first = rest | 1u << 7;
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(dcol),
        "r"(qcol + kk * 8), "l"(kdesc + static_cast<uint64_t>((kk % (D / 32) * 32) >> 4)), "r"(kk < D / 32 ? first : rest), "r"(kk > 0 ? 1u : 0u)
        : "memory");
}
// 64 columns of a bf16 tile.
__device__ __forceinline__ void issue_qk_half(uint32_t dcol, uint32_t qcol, uint64_t kdesc, uint32_t accumulate) {
#pragma unroll
  for (int kk = 0; kk < 4; ++kk)
    tc_mma_ts(dcol, qcol + kk * 8, kdesc + kk * 2, idesc_bf16_f32(128, 128, 0), kk > 0 || accumulate ? 1u : 0u);
}
// Scores and products have a warp each: a thread is held for about as long as the MMAs run that it issues.
// QK(i) overwrites P(i-2), so it waits until that product is done. The warp of the scores also turns the scale
// bytes of cached keys to factors.
template <int D>
__device__ void flat_scores(const PrefixParams &p, uint8_t *smem, FlatBars *bars, const int *table, uint32_t tmem_in) {
  using C = FlatCfg<D>;
  volatile int *abort_flag = &bars->abort;
  const uint32_t tmem = uniform(tmem_in), lane = threadIdx.x & 31;
  uint32_t g = 0, items = 0;   // tiles, items so far
  uint32_t slot = 0, parity = 0;
  // Slots of codes have rows of D bytes, of bf16 64 columns: 128 bytes; the swizzle is as wide.
  const uint64_t kdesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
  const uint64_t cdesc0 = D == 128 ? kdesc0
                                   : (smem_desc_sw128(smem_u32(smem + C::OFF_K), 16, 512) & ~(7ull << 61)) | 4ull << 61;
  auto wait = [&](uint64_t &bar, uint32_t parity) { return wait_for<false>(smem_u32(&bar), parity, abort_flag, p); };
  auto next_slot = [&] {
    if (++slot == C::KN) slot = 0, parity ^= 1;
  };
  PrefixWalk walk = bars->start.walk;
  PrefixItem item = bars->start.item;
  bool more = bars->start.any != 0;
  for (; more; ++items, more = next_item(&bars->start, table, &walk, &item)) {
    const int kv0 = uniform(item.kv0), kv1 = uniform(item.kv1);
    if (!wait(bars->q_full, items & 1)) goto done;
    for (int j = kv0; j < kv1; ++j, ++g) {
      const uint32_t t = g & 1, dcol = tmem + t * 128;
      if (!wait(bars->k_full[slot], parity)) goto done;
      if (uniform(is_cached(p, j))) {
        // (The softmax is done with tile g - 4, as the scores of g - 1 followed the product of g - 3.)
        const uint32_t bytes = *reinterpret_cast<const uint32_t *>(smem + C::OFF_KS + slot * BN + lane * 4);
        reinterpret_cast<float4 *>(smem + C::OFF_FAC)[(g & 3) * (BN / 4) + lane] =
            make_float4(power_of(bytes & 255) * kKeyDown, power_of(bytes >> 8 & 255) * kKeyDown,
                        power_of(bytes >> 16 & 255) * kKeyDown, power_of(bytes >> 24) * kKeyDown);
        if (g >= 2 && !wait(bars->pv_done[t], (g >> 1 & 1) ^ 1)) goto done;   // of tile g - 2
        __syncwarp();
        tc_fence_after();
        if (elect_one()) {
          issue_qk_codes<D>(dcol, tmem + C::COL_Q8, cdesc0 + static_cast<uint64_t>(slot * (kHalf >> 4)));
          tc_commit(smem_u32(&bars->s_full[t]));
          tc_commit(smem_u32(&bars->k_empty[slot]));
          if (j == kv1 - 1) tc_commit(smem_u32(&bars->q_empty));
          mbar_arrive(smem_u32(&bars->s_full[t]));   // the factors
        }
        __syncwarp();
        next_slot();
        continue;
      }
      if (g >= 2 && !wait(bars->pv_done[t], (g >> 1 & 1) ^ 1)) goto done;
      for (int hf = 0; hf < D / 64; ++hf) {
        if (hf > 0 && !wait(bars->k_full[slot], parity)) goto done;
        tc_fence_after();
        if (elect_one()) {
          issue_qk_half(dcol, tmem + C::COL_Q + 32 * hf, kdesc0 + static_cast<uint64_t>(slot * (kHalf >> 4)), hf);
          tc_commit(smem_u32(&bars->k_empty[slot]));
          if (hf == D / 64 - 1) {
            tc_commit(smem_u32(&bars->s_full[t]));
            if (j == kv1 - 1) tc_commit(smem_u32(&bars->q_empty));
            mbar_arrive(smem_u32(&bars->s_full[t]));
          }
        }
        __syncwarp();
        next_slot();
      }
    }
  }
done:
  // All MMAs issued must finish before Tensor Memory is released.
  if (elect_one()) tc_commit(smem_u32(&bars->drain));
  __syncwarp();
  drain(smem_u32(&bars->drain), 0);
}

template <int D>
__device__ void flat_products(const PrefixParams &p, uint8_t *smem, FlatBars *bars, const int *table, uint32_t tmem_in) {
  using C = FlatCfg<D>;
  volatile int *abort_flag = &bars->abort;
  const uint32_t tmem = uniform(tmem_in);
  uint32_t g = 0;
  const uint64_t vdesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_V), kHalf, 1024);
  auto wait = [&](uint64_t &bar, uint32_t parity) { return wait_for<false>(smem_u32(&bar), parity, abort_flag, p); };
  PrefixWalk walk = bars->start.walk;
  PrefixItem item = bars->start.item;
  bool more = bars->start.any != 0;
  for (; more; more = next_item(&bars->start, table, &walk, &item)) {
    const int kv0 = uniform(item.kv0), kv1 = uniform(item.kv1);
    for (int j = kv0; j < kv1; ++j, ++g) {
      const uint32_t t = g & 1, vs = g % C::VS;
      if (!wait(bars->v_full[vs], g / C::VS & 1)) goto done;
      if (!wait(bars->p_full[t], g >> 1 & 1)) goto done;
      tc_fence_after();
      if (elect_one()) {
        issue_pv<D>(tmem + C::COL_O, tmem + t * 128, vdesc0 + static_cast<uint64_t>(vs * (C::TILE >> 4)), j > kv0 ? 1u : 0u);
        tc_commit(smem_u32(&bars->v_empty[vs]));
        tc_commit(smem_u32(&bars->pv_done[t]));
        if (j == kv1 - 1) tc_commit(smem_u32(&bars->o_full));
      }
      __syncwarp();
    }
  }
done:
  if (elect_one()) tc_commit(smem_u32(&bars->drain));
  __syncwarp();
  drain(smem_u32(&bars->drain), 0);
}

// ------------------------------------------------------------------ softmax and epilogue
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 9, 128;" ::: "memory"); }

// Bits [lo, hi) of a 32-bit word, both limits taken into [0, 32].
__device__ __forceinline__ uint32_t bits_of(int lo, int hi) {
  auto below = [](int x) { return x <= 0 ? 0u : x >= 32 ? ~0u : (1u << x) - 1u; };
  return below(hi) & ~below(lo);
}
// Maximum of 32 scores and of `m`.
__device__ __forceinline__ float max32(const uint32_t (&s)[32], float m) {
  float mp[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) mp[i] = max3(__uint_as_float(s[i]), __uint_as_float(s[i + 8]), __uint_as_float(s[i + 16]));
#pragma unroll
  for (int i = 0; i < 4; ++i) mp[i] = max3(mp[i], mp[i + 4], __uint_as_float(s[i + 24]));
#pragma unroll
  for (int i = 0; i < 2; ++i) mp[i] = max3(mp[i], mp[i + 2], __uint_as_float(s[i + 28]));
  m = max3(m, __uint_as_float(s[30]), __uint_as_float(s[31]));
  return max3(m, mp[0], mp[1]);
}
// Scores of N times 32 keys in Tensor Memory, times fac and back where fac is given, with those outside [lo, hi) -inf,
// whatever they were. (In place and out of line: the softmax's loop stays short.)
template <int N>
__device__ __noinline__ void mask_scores(uint32_t taddr, const float *fac, float back, int lo, int hi) {
#pragma unroll 1
  for (int c = 0; c < N; ++c) {
    uint32_t s[32];
    tmem_ld32(taddr + 32 * c, s);
    tmem_wait_ld_regs(s);
    const uint32_t keep = bits_of(lo - 32 * c, hi - 32 * c);
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      if (fac) s[k] = __float_as_uint(__uint_as_float(s[k]) * fac[32 * c + k] * back);
      s[k] = keep >> k & 1 ? s[k] : 0xff800000u;
    }
    tmem_st32(taddr + 32 * c, s);
  }
  tmem_wait_st();
}
// P of a tile to zeros.
__device__ __noinline__ void zero_weights(uint32_t taddr) {
  uint32_t zero[32];
#pragma unroll
  for (int k = 0; k < 32; ++k) zero[k] = 0;
  tmem_st32(taddr, zero);
  tmem_st32(taddr + 32, zero);
}
// Weights 2^(s * scale - m) of 32 scores as bf16 pairs (the type of V, as both operands of an MMA have one: off by at most
// 2^-8 of a weight, as the output's own rounding is of it), and their sums added to `sum`, in fp32 pairs: an add for two
// weights (in the tall kernel four images took 983 us with an add for each, 943 so).
__device__ __forceinline__ void weights32(const uint32_t (&s)[32], uint64_t scale2, uint64_t negm2, uint32_t (&pk)[16],
                                          uint64_t (&sum)[2]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint64_t x2 = f2_fma(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), scale2, negm2);
    float x0, x1;
    f2_unpack(x2, x0, x1);
    x0 = ex2_approx(x0);
    x1 = ex2_approx(x1);
    sum[i & 1] = f2_add(sum[i & 1], f2_pack(x0, x1));
    pk[i] = pack_bf16x2(x0, x1);
  }
}
__device__ __forceinline__ float total(const uint64_t (&sum)[2]) {
  float a, b;
  f2_unpack(f2_add(sum[0], sum[1]), a, b);
  return a + b;
}
// The factor 2^(a - b) of a maximum that moved from a to b; 0 where there was none.
__device__ __forceinline__ float shrink(float a, float b) { return a == -INFINITY ? 0.f : ex2_approx(a - b); }

// NC: 32-key chunks of a tile that a copy takes (4, 2 or 1 with one, two or four copies).
template <int D, int NC>
__device__ void flat_softmax(const PrefixParams &p, uint8_t *smem, FlatBars *bars, const int *table, uint32_t tmem) {
  using C = FlatCfg<D>;
  constexpr int COPIES = 4 / NC, RT = BM / COPIES;   // rows of a unit
  const int tid = threadIdx.x, wq = tid >> 5;
  const int in = tid % RT, copy = tid / RT;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(wq * 32) << 16), tO = lanes + C::COL_O;
  volatile int *abort_flag = &bars->abort;
  float2 *exch = reinterpret_cast<float2 *>(smem + C::OFF_STG);
  float *fin = reinterpret_cast<float *>(smem + C::OFF_FIN);
  uint32_t step = 0, items = 0;   // tiles, items so far
  bool dead = false;   // a wait gave up: go on without waiting, store nothing
  auto wait = [&](uint64_t &bar, uint32_t parity) {
    if (!dead && !wait_for<true>(smem_u32(&bar), parity, abort_flag, p)) dead = true;
  };
  PrefixWalk walk = bars->start.walk;
  PrefixItem item = bars->start.item;
  bool more = bars->start.any != 0;
  bool cut = false;   // a piece was this CTA's first of its unit
  for (; more; ++items, more = next_item(&bars->start, table, &walk, &item)) {
    const int row = item.row0 + in;
    const bool idle = item.row0 + (wq * 32) % RT >= p.rows;   // no row in this warp
    const PrefixRange own = range_of(p, table, row);
    wait(bars->q_full, items & 1);
    const float row_factor = reinterpret_cast<const float *>(smem + C::OFF_QF)[tid];   // (of rows in codes)
    float row_scale = row_factor * (1.f / kKeyDown) * p.scale_log2;
    int whole = NC * 32;   // a tile's keys from the first to here or further: no masking
    if (row_scale > FLT_MAX) {   // (not a NaN)
      whole = INT_MAX;
      row_scale = fminf(row_factor * p.scale_log2, FLT_MAX);   // (finite, so that a score of 0 stays one)
    }
    mbar_arrive(smem_u32(&bars->q_seen));
    float m = -INFINITY, l = 0.f;
    for (int j = item.kv0; j < item.kv1; ++j, ++step) {
      const uint32_t t = step & 1, tS = lanes + t * 128;
      wait(bars->s_full[t], step >> 1 & 1);
      if (idle) {
        mbar_arrive(smem_u32(&bars->p_full[t]));
        continue;
      }
      tc_fence_after();
      const int first = (j < p.n_prefix ? j * BN : own_pos(p, item, j)) + copy * (NC * 32);
      const int lo = (j < p.n_prefix ? 0 : own.lo) - first, hi = (j < p.n_prefix ? p.Np : own.hi) - first;
      // Two passes over the scores, as 128 of them would not fit the registers beside the rest: the
      // maximum, then the weights (each chunk of P covers scores that have been read).
      const uint32_t tC = tS + copy * (NC * 32);
      if (__all_sync(0xffffffffu, lo >= NC * 32 || hi <= 0)) {   // nothing for any row: no weight
        zero_weights(tS);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&bars->p_full[t]));
        continue;
      }
      // Scores of cached keys are times the key's factor, then times the row's and the scale of all scores.
      bool times = is_cached(p, j);
      const float scale = times ? row_scale : p.scale_log2;
      const float4 *fac = reinterpret_cast<const float4 *>(smem + C::OFF_FAC) + (step & 3) * (BN / 4) + copy * NC * 8;
      // Mostly a row sees all of the tile's keys or none: that takes no masking of scores.
      bool live = lo < NC * 32 && hi > 0;
      if (__any_sync(0xffffffffu, live && (lo > 0 || hi < whole))) {
        mask_scores<NC>(tC, times ? reinterpret_cast<const float *>(fac) : nullptr, whole == INT_MAX ? 1.f / kKeyDown : 1.f, lo, hi);
        times = false;
        live = true;
      }
      constexpr int W = NC > 1 ? 2 : 1;   // chunks loaded at a time
      uint32_t s[W][32];
      auto finish = [&](int c, int k0) {
        uint32_t (&x)[32] = s[k0];
        tmem_wait_ld_regs(x);
        if (times)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 f = fac[8 * c + k];
            const uint64_t a = f2_mul(f2_pack(__uint_as_float(x[4 * k]), __uint_as_float(x[4 * k + 1])), f2_pack(f.x, f.y));
            const uint64_t b = f2_mul(f2_pack(__uint_as_float(x[4 * k + 2]), __uint_as_float(x[4 * k + 3])), f2_pack(f.z, f.w));
            x[4 * k] = static_cast<uint32_t>(a);
            x[4 * k + 1] = static_cast<uint32_t>(a >> 32);
            x[4 * k + 2] = static_cast<uint32_t>(b);
            x[4 * k + 3] = static_cast<uint32_t>(b >> 32);
          }
      };
      float mx = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < NC; c += W) {
#pragma unroll
        for (int k = 0; k < W; ++k) tmem_ld32(tC + 32 * (c + k), s[k]);
#pragma unroll
        for (int k = 0; k < W; ++k) {
          finish(c + k, k);
          mx = max32(s[k], mx);
          if (NC == 4 && times) tmem_st32(tC + 32 * (c + k), s[k]);   // (shorter than to multiply twice)
        }
      }
      if (NC == 4 && times) tmem_wait_st();
      times = false;
      const float m_new = live ? fmaxf(m, mx * scale) : m;
      float alpha = 1.f;
      bool rescale = false;
      if (j == item.kv0) {
        m = m_new;
      } else {
        const bool need = m_new > m + kGrowth;
        if (__any_sync(0xffffffffu, need)) {
          rescale = true;
          if (need) {
            alpha = shrink(m, m_new);
            m = m_new;
          }
        }
      }
      // (Without any key so far the weights are 2^(-inf - 0) = 0.)
      const float neg = m == -INFINITY ? 0.f : -m;
      const uint64_t scale2 = f2_pack(scale, scale), negm2 = f2_pack(neg, neg);
      uint64_t sum[2] = {0, 0};
#pragma unroll 1
      for (int c = 0; c < NC; c += W) {
        if constexpr (NC == 4) {
#pragma unroll
          for (int k = 0; k < W; ++k) tmem_ld32(tC + 32 * (c + k), s[k]);
        }
#pragma unroll
        for (int k = 0; k < W; ++k) {
          if constexpr (NC == 4) finish(c + k, k);
          uint32_t pk[16];
          weights32(s[k], scale2, negm2, pk, sum);
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = live ? pk[i] : 0;
          tmem_st16(tS + 16 * (copy * NC + c + k), pk);
        }
      }
      if constexpr (NC < 4) {
        uint32_t zero[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) zero[k] = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c / NC != copy) tmem_st16(tS + 16 * c, zero);
      }
      if (live) l = fmaf(l, alpha, total(sum));
      if (rescale) {
        // (The products before the last are done, as these scores followed them.)
        wait(bars->pv_done[t ^ 1], (step - 1) >> 1 & 1);
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t o[16];
          tmem_ld16(tO + 16 * c, o);
          tmem_wait_ld16(o);
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
          tmem_st16(tO + 16 * c, o);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(smem_u32(&bars->p_full[t]));
    }
    wait(bars->o_full, items & 1);
    tc_fence_after();
    {
      const uint32_t *bad = reinterpret_cast<const uint32_t *>(smem + C::OFF_BAD) + (items & 1) * 2 * kFlatGroupWarps * kBadWords;
      const int b = p.by_entry.of(min(row, p.rows - 1));
      uint32_t any = 0;
#pragma unroll
      for (int w = 0; w < 2 * kFlatGroupWarps; ++w)
        any |= bad[w * kBadWords + (b >> 5)] >> (b & 31) | bad[w * kBadWords + kPrefixEntries / 32];
      if (any & 1) l = NAN;
    }
    if (item.piece) {
      // Every copy's sums as they are; the join adds the copies with the pieces.
      float *part = part_of<D>(p, blockIdx.x, item.kv0 == 0 ? 1 : 0, BM);
      if (item.kv0 == 0) cut = true;
      const bool live = row < p.rows && !dead;
      if (live) {
        __stcg(part + D * BM + tid, m);
        __stcg(part + (D + 1) * BM + tid, l);
      }
      if (tid == 0 && item.kv0 == 0)
        __stcg(cut_place(p, item.unit), make_int4(blockIdx.x, dead ? 0 : pieces_of(p, bars->start.plan, item.u0, item.n), item.hk, item.row0));
      if (!idle) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t a[32];
          tmem_ld32(tO + 32 * c, a);
          tmem_wait_ld_regs(a);
          if (live)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              __stcg(reinterpret_cast<float4 *>(part) + (8 * c + k) * BM + tid,
                     make_float4(__uint_as_float(a[4 * k]), __uint_as_float(a[4 * k + 1]),
                                 __uint_as_float(a[4 * k + 2]), __uint_as_float(a[4 * k + 3])));
        }
      }
      tc_fence_before();
      continue;
    }
    if (tid == 0 && item.u0 > 0 && cut_by_unit(p)) __stcg(cut_place(p, item.unit), make_int4(0, 0, 0, 0));
    // (m, l) of all copies of a row.
    float top = m, all = l, f = 1.f;
    if constexpr (COPIES > 1) {
      exch[tid] = make_float2(m, l);
      softmax_sync();
#pragma unroll
      for (int k = 0; k < COPIES; ++k) top = fmaxf(top, exch[k * RT + in].x);
      all = 0.f;
#pragma unroll
      for (int k = 0; k < COPIES; ++k) {
        const float2 e = exch[k * RT + in];
        all = fmaf(shrink(e.x, top), e.y, all);
      }
      f = shrink(m, top);
    }
    const float norm = all == 0.f ? 0.f : 1.f / all;
    if constexpr (COPIES == 1) {
      uint16_t *dst = dead ? nullptr : out_row(p, item.hk, row, D);
      if (!idle) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t a[32];
          tmem_ld32(tO + 32 * c, a);
          tmem_wait_ld_regs(a);
          if (dst) {
            float x[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = __uint_as_float(a[k]) * norm;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              reinterpret_cast<uint4 *>(dst + 32 * c)[k] =
                  make_uint4(pack_bf16x2(x[8 * k], x[8 * k + 1]), pack_bf16x2(x[8 * k + 2], x[8 * k + 3]),
                             pack_bf16x2(x[8 * k + 4], x[8 * k + 5]), pack_bf16x2(x[8 * k + 6], x[8 * k + 7]));
          }
        }
      }
      tc_fence_before();
    } else {
      // The copies of a row lie in other warps' lanes: 16 columns at a time through shared memory
      // (16-byte groups, moved by half the row's number against bank conflicts), then a thread adds the
      // copies of four columns.
      if (copy == 0) fin[in] = norm;
      softmax_sync();   // exch has been read, fin is written
      float4 *stg = reinterpret_cast<float4 *>(smem + C::OFF_STG);
#pragma unroll 1
      for (int c = 0; c < D / 16; ++c) {
        if (!idle) {
          uint32_t a[16];
          tmem_ld16(tO + 16 * c, a);
          tmem_wait_ld16(a);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            stg[tid * 4 + (k ^ (tid >> 1 & 3))] =
                make_float4(f * __uint_as_float(a[4 * k]), f * __uint_as_float(a[4 * k + 1]),
                            f * __uint_as_float(a[4 * k + 2]), f * __uint_as_float(a[4 * k + 3]));
        }
        softmax_sync();
#pragma unroll
        for (int k = 0; k < RT * 4 / 128; ++k) {
          const int r = (tid + 128 * k) / 4, q = tid & 3;
          if (item.row0 + r >= p.rows || dead) continue;
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int e = 0; e < COPIES; ++e) {
            const int at = e * RT + r;
            const float4 y = stg[at * 4 + (q ^ (at >> 1 & 3))];
            x.x += y.x;
            x.y += y.y;
            x.z += y.z;
            x.w += y.w;
          }
          if (uint16_t *to = out_row(p, item.hk, item.row0 + r, D)) {
            const float g = fin[r];
            *reinterpret_cast<uint2 *>(to + 16 * c + 4 * q) =
                make_uint2(pack_bf16x2(x.x * g, x.y * g), pack_bf16x2(x.z * g, x.w * g));
          }
        }
        softmax_sync();
      }
      tc_fence_before();
    }
  }
  if (p.split && tid == 0 && !cut && !cut_by_unit(p)) __stcg(p.cuts + blockIdx.x, make_int4(0, 0, 0, 0));
}

template <int D>
__global__ void __launch_bounds__(512, 1) prefix_flat_kernel(const __grid_constant__ PrefixParams p) {
  using C = FlatCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];   // the swizzle pattern repeats every 1024 bytes
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicExch(p.status, kDevBadPlan);
    return;
  }
  FlatBars *bars = reinterpret_cast<FlatBars *>(smem + C::OFF_BAR);
  int *table = reinterpret_cast<int *>(smem + C::OFF_TAB);
  const int warp = uniform(threadIdx.x / 32);
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars->q_full), 2 * BM);
    mbar_init(smem_u32(&bars->q_empty), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&bars->v_full[s]), kFlatGroupWarps);
      mbar_init(smem_u32(&bars->v_empty[s]), 1);
      mbar_init(smem_u32(&bars->raw[s]), 1);
      mbar_init(smem_u32(&bars->s_full[s]), 2);     // the scores, and the keys' factors
      mbar_init(smem_u32(&bars->p_full[s]), 128);
    }
    for (int s = 0; s < C::KN; ++s) {
      mbar_init(smem_u32(&bars->k_full[s]), 1 + BN / 16);   // the keys, and the lanes with scales
      mbar_init(smem_u32(&bars->k_empty[s]), 1);
    }
    for (int s = 0; s < 2 * C::FV; ++s) {
      mbar_init(smem_u32(&bars->f_full[s]), 1 + BN / 16);
      mbar_init(smem_u32(&bars->f_empty[s]), kFlatGroupWarps);
    }
    mbar_init(smem_u32(&bars->pv_done[0]), 1);
    mbar_init(smem_u32(&bars->pv_done[1]), 1);
    mbar_init(smem_u32(&bars->o_full), 1);
    mbar_init(smem_u32(&bars->drain), 2);   // one commit of each issuer
    mbar_init(smem_u32(&bars->q_seen), BM);
    bars->abort = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) begin_schedule(p, table, &bars->start);
  if (warp == kFlatScores) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (p.split) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join waits for this grid's end itself
  const uint32_t tmem = bars->tmem_base;
  if (warp < kFlatValues) {
    if (p.copies == 1)
      flat_softmax<D, 4>(p, smem, bars, table, tmem);
    else if (p.copies == 2)
      flat_softmax<D, 2>(p, smem, bars, table, tmem);
    else
      flat_softmax<D, 1>(p, smem, bars, table, tmem);
  } else if (warp < kFlatScores) {
    flat_values<D>(p, smem, bars, table, tmem, (warp - kFlatValues) / kFlatGroupWarps);
  } else if (warp == kFlatScores) {
    flat_scores<D>(p, smem, bars, table, tmem);
  } else if (warp == kFlatProducts) {
    flat_products<D>(p, smem, bars, table, tmem);
  } else if (warp == kFlatLoadKeys) {
    flat_load_keys<D>(p, smem, bars, table);
  } else {
    flat_load_values<D>(p, smem, bars, table);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kFlatScores) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}
