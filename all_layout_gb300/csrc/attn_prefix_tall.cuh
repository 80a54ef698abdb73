// The tall kernel of shared-prefix attention (included by attn_prefix.cu): pairs of 128-row tiles
// against bf16 keys and values in tensors, for calls with many rows for each k/v head, where the
// tensor cores are the bound. (Cached keys and values are read back to bf16 by a launch before:
// 6 bytes a value, against 4 flops for every row that meets it.)
//
// Both tiles of a unit go over the same KV tiles, each KV tile loaded once for the pair. Own keys
// and a request's rows are padded to multiples of 128, so a tile of rows and a KV tile are of one request
// each; a tile of rows takes the prefix and its own request's keys. (Its zero weights never meet another
// request's values, which might not be numbers.)
//
// Roles (320 threads, at d = 64 352, one CTA per SM):
//   warps 0-3, 4-7  softmax of row tile 0 and 1, row r of the tile = TMEM lane r
//   warp 8          MMA issuer, Tensor Memory allocation
//   warp 9          TMA loader
//   warp 10         d = 64: issuer of the products
// Tensor Memory: S0 [0,128) S1 [128,256) O0 [256,256+d) O1 [256+d,256+2d); P_t over S_t's first 64.
// Measured at d = 128: 4 x 24 heads of 4096 queries against 4096 + 4096 keys 943 us = 1749 TFLOP/s; the tensor pipe is
// busy 75% of the cycles, the rest is what a row tile's softmax takes longer than the other tile's MMAs.
// Issue order at KV tile j, for t = 0, 1: O_t += P_t(j-1) V(j-1), S_t = Q_t K(j)^T: one thread's
// order keeps S_t(j) from overwriting P_t(j-1) before its product, and the commit that signals
// S_t(j) covers O_t. One tile's softmax runs beside the other's products.
// At d = 64 P has columns of its own, P_t [384+64t,448+64t), and a warp of its own issues the products: the scores
// of the next tile are computed as soon as the softmax has loaded this one's, so it never waits for them (19 heads of
// 2048 queries against 16384 keys: 143 us = 1140 TFLOP/s; in d = 128's order 1.15 times as long).

template <int D>
struct TallCfg {
  static constexpr int THREADS = D == 64 ? 352 : 320;
  static constexpr uint32_t COL_P = D == 64 ? 384 : 0, P_STEP = D == 64 ? 64 : 128;   // P_t at COL_P + t * P_STEP
  static constexpr int TILE = BM * D * 2;
  static constexpr int KS = D == 128 ? 2 : 3, VS = KS;
  static constexpr int OFF_K = 2 * TILE, OFF_V = OFF_K + KS * TILE;
  static constexpr int OFF_STG = OFF_V + VS * TILE;            // a warp's 32 rows of 64 columns, bf16
  static constexpr int OFF_TAB = OFF_STG + 8 * 32 * 128;
  static constexpr int OFF_BAR = OFF_TAB + kTable * 4;
  static constexpr int SMEM = OFF_BAR + 416;
  static_assert(SMEM <= 232448, "shared memory per CTA");
};
constexpr int kTallMma = 8, kTallLoad = 9, kTallProducts = 10;

struct TallBars {
  uint64_t q_full, q_empty;
  uint64_t k_full[3], k_empty[3], v_full[3], v_empty[3];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t s_read[2], pv_done[2];   // d = 64
  uint64_t drain;
  PrefixStart start;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(TallBars) <= 416, "barrier block too large");

// The KV tiles of an item that row tile t of it takes: [kv0, prefix) and [own0, own1), the prefix's and
// those of its rows' requests.
struct TallTiles {
  int kv0, prefix, own0, own1;
  __device__ __forceinline__ bool has(int j) const { return j < prefix || (j >= own0 && j < own1); }
  __device__ __forceinline__ int count() const { return max(prefix - kv0, 0) + own1 - own0; }
  __device__ __forceinline__ int last() const { return own1 > own0 ? own1 - 1 : prefix - 1; }
};
__device__ __forceinline__ TallTiles tiles_of(const PrefixParams &p, const int *table, const PrefixItem &it, int t) {
  const int row0 = it.row0 + t * BM;
  if (row0 >= p.rows) return TallTiles{0, 0, 0, 0};
  TallTiles r;
  r.kv0 = it.kv0;
  r.prefix = min(it.kv1, p.n_prefix);
  int a = table[p.by_entry.of(row0)] / BN - it.t0 + p.n_prefix;
  int e = table[p.by_entry.of(min(row0 + BM, p.rows) - 1) + 1] / BN - it.t0 + p.n_prefix;
  if (p.n_prefix == 0 && table[it.b_hi + 1] == table[it.b_lo]) {   // no key in the unit: the masked tile
    a = 0;
    e = 1;
  }
  r.own0 = max(a, it.kv0);
  r.own1 = max(min(e, it.kv1), r.own0);
  return r;
}

// Where own tile j of an item lies, and how many of its keys count (0: nothing to load). `b` only grows.
struct TallOwn {
  int off, valid;
};
__device__ __forceinline__ TallOwn own_tile(const PrefixParams &p, const int *table, const PrefixItem &it, int j, int &b) {
  const int pos = own_pos(p, it, j);
  while (b < it.b_hi && table[b + 1] <= pos) ++b;
  const int off = pos - table[b];
  return TallOwn{off, min(max(len_of(table, b) - off, 0), BN)};
}

// ------------------------------------------------------------------ TMA loader
template <int D>
__device__ void tall_loader(const PrefixParams &p, uint8_t *smem, TallBars *bars, const int *table) {
  using C = TallCfg<D>;
  volatile int *abort_flag = &bars->abort;
  const int lane = threadIdx.x & 31;
  uint32_t use = 0, items = 0, uses[2] = {0, 0};
  const uint32_t q_full = smem_u32(&bars->q_full);
  PrefixWalk walk = bars->start.walk;
  PrefixItem item = bars->start.item;
  bool more = bars->start.any != 0;
  bool ok = true;
  for (; ok && more; ++items, more = next_item(&bars->start, table, &walk, &item)) {
    if (items > 0) ok = wait_for<true>(smem_u32(&bars->q_empty), (items - 1) & 1, abort_flag, p);
    if (!ok) break;
    {
      // Eight rows a lane (queries are padded to multiples of eight, so they are one head's).
      const int row = item.row0 + lane * 8;
      const PrefixRow r = row_of(p, item.hk, min(row, p.rows - 1));
      const bool live = row < p.rows && r.n < p.Nq && r.h < (item.hk + 1) * p.group;
      const unsigned bytes = __popc(__ballot_sync(0xffffffffu, live)) * 8u * D * 2;
      if (lane == 0) mbar_arrive_expect_tx(q_full, bytes);
      __syncwarp();
      if (live) {
        const uint32_t dst = smem_u32(smem) + (lane / 16) * C::TILE + (lane % 16) * 1024;
        for (int hf = 0; hf < D / 64; ++hf) tma_load_4d(dst + hf * kHalf, &p.tm_q, q_full, hf * 64, r.n, r.h, p.b0 + r.b);
      }
      __syncwarp();
    }
    int b = item.b_lo;
    for (int j = item.kv0; ok && j < item.kv1; ++j, ++use) {
      const bool prefix = j < p.n_prefix;
      TallOwn own{0, BN};
      if (!prefix) own = own_tile(p, table, item, j, b);
      for (int kv = 0; ok && kv < 2; ++kv) {
        const uint32_t n = kv ? C::VS : C::KS, slot = use % n;
        ok = wait_for<true>(smem_u32(kv ? &bars->v_empty[slot] : &bars->k_empty[slot]), (use / n & 1) ^ 1, abort_flag, p);
        if (!ok) break;
        const uint32_t full = smem_u32(kv ? &bars->v_full[slot] : &bars->k_full[slot]);
        if (elect_one()) {
          mbar_arrive_expect_tx(full, own.valid > 0 ? C::TILE : 0);
          const uint32_t dst = smem_u32(smem + (kv ? C::OFF_V : C::OFF_K) + slot * C::TILE);
          if (prefix)
            for (int hf = 0; hf < D / 64; ++hf)
              tma_load_4d(dst + hf * kHalf, kv ? &p.tm_pv : &p.tm_pk, full, hf * 64, j * BN, item.hk, 0);
          else if (own.valid > 0)
            for (int hf = 0; hf < D / 64; ++hf)
              tma_load_4d(dst + hf * kHalf, kv ? &p.tm_v : &p.tm_k, full, hf * 64, own.off, item.hk, p.b0 + b);
        }
        __syncwarp();
        ++uses[kv];
      }
    }
  }
  // Every load issued must land before the CTA releases its shared memory.
  for (uint32_t s = 0; s < C::KS; ++s) {
    if (uses[0] > s) drain(smem_u32(&bars->k_full[s]), ((uses[0] - 1 - s) / C::KS) & 1);
    if (uses[1] > s) drain(smem_u32(&bars->v_full[s]), ((uses[1] - 1 - s) / C::VS) & 1);
  }
  if (items > 0) drain(q_full, (items - 1) & 1);
}

// ------------------------------------------------------------------ MMA issuers
// A key behind a request's last one has weight 0, but what lies in its row of V may not be a number. By one warp.
template <int D>
__device__ __forceinline__ void clear_tail(uint8_t *tile, int valid) {
  for (int hf = 0; hf < D / 64; ++hf)
    for (int o = valid * 128 + (threadIdx.x & 31) * 16; o < kHalf; o += 512)
      *reinterpret_cast<uint4 *>(tile + hf * kHalf + o) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

// d = 64: the scores, each row tile's as soon as its softmax has loaded the last ones.
template <int D>
__device__ void tall_scores(const PrefixParams &p, uint8_t *smem, TallBars *bars, const int *table, uint32_t tmem_in) {
  using C = TallCfg<D>;
  volatile int *abort_flag = &bars->abort;
  const uint32_t tmem = uniform(tmem_in);
  uint32_t use = 0, items = 0, done[2] = {0, 0};   // uses of the ring; scores issued of each row tile
  const uint64_t qdesc = smem_desc_sw128(smem_u32(smem), 16, 1024);
  const uint64_t kdesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
  auto wait = [&](uint64_t &bar, uint32_t parity) { return wait_for<false>(smem_u32(&bar), parity, abort_flag, p); };
  PrefixWalk walk = bars->start.walk;
  PrefixItem item = bars->start.item;
  bool more = bars->start.any != 0;
  for (; more; ++items, more = next_item(&bars->start, table, &walk, &item)) {
    const int kv0 = uniform(item.kv0), kv1 = uniform(item.kv1);
    TallTiles tiles[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const TallTiles x = tiles_of(p, table, item, t);
      tiles[t] = TallTiles{uniform(x.kv0), uniform(x.prefix), uniform(x.own0), uniform(x.own1)};
    }
    if (!wait(bars->q_full, items & 1)) goto done;
    for (int j = kv0; j < kv1; ++j, ++use) {
      const uint32_t ks = use % C::KS;
      if (!wait(bars->k_full[ks], use / C::KS & 1)) goto done;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (tiles[t].has(j)) {
          if (done[t] > 0 && !wait(bars->s_read[t], (done[t] - 1) & 1)) goto done;
          ++done[t];
          tc_fence_after();
          if (elect_one()) {
            issue_qk<D>(tmem + t * 128, qdesc + static_cast<uint64_t>(t * (C::TILE >> 4)), kdesc0 + static_cast<uint64_t>(ks * (C::TILE >> 4)));
            tc_commit(smem_u32(&bars->s_full[t]));
          }
          __syncwarp();
        }
      }
      if (elect_one()) {
        tc_commit(smem_u32(&bars->k_empty[ks]));
        if (j == kv1 - 1) tc_commit(smem_u32(&bars->q_empty));
      }
      __syncwarp();
    }
  }
done:
  // All MMAs issued must finish before Tensor Memory is released.
  if (elect_one()) tc_commit(smem_u32(&bars->drain));
  __syncwarp();
  drain(smem_u32(&bars->drain), 0);
}

// d = 64: the products with V.
template <int D>
__device__ void tall_products(const PrefixParams &p, uint8_t *smem, TallBars *bars, const int *table, uint32_t tmem_in) {
  using C = TallCfg<D>;
  volatile int *abort_flag = &bars->abort;
  const uint32_t tmem = uniform(tmem_in);
  uint32_t use = 0, pc = 0;   // uses of the ring; parities of p_full, a bit a row tile
  const uint64_t vdesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_V), kHalf, 1024);
  auto wait = [&](uint64_t &bar, uint32_t parity) { return wait_for<false>(smem_u32(&bar), parity, abort_flag, p); };
  PrefixWalk walk = bars->start.walk;
  PrefixItem item = bars->start.item;
  bool more = bars->start.any != 0;
  for (; more; more = next_item(&bars->start, table, &walk, &item)) {
    const int kv0 = uniform(item.kv0), kv1 = uniform(item.kv1);
    TallTiles tiles[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const TallTiles x = tiles_of(p, table, item, t);
      tiles[t] = TallTiles{uniform(x.kv0), uniform(x.prefix), uniform(x.own0), uniform(x.own1)};
    }
    int b = item.b_lo;
    bool fresh[2] = {true, true};   // no product of this item yet
    for (int j = kv0; j < kv1; ++j, ++use) {
      const uint32_t vs = use % C::VS;
      if (!wait(bars->v_full[vs], use / C::VS & 1)) goto done;
      if (j >= p.n_prefix) {
        const int valid = uniform(own_tile(p, table, item, j, b).valid);
        if (valid < BN) clear_tail<D>(smem + C::OFF_V + vs * C::TILE, valid);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (tiles[t].has(j)) {
          if (!wait(bars->p_full[t], pc >> t & 1)) goto done;
          pc ^= 1u << t;
          tc_fence_after();
          if (elect_one()) {
            issue_pv<D>(tmem + 256 + t * D, tmem + C::COL_P + t * C::P_STEP, vdesc0 + static_cast<uint64_t>(vs * (C::TILE >> 4)), fresh[t] ? 0u : 1u);
            tc_commit(smem_u32(&bars->pv_done[t]));
            if (j == tiles[t].last()) tc_commit(smem_u32(&bars->o_full[t]));
          }
          __syncwarp();
          fresh[t] = false;
        }
      }
      if (elect_one()) tc_commit(smem_u32(&bars->v_empty[vs]));
      __syncwarp();
    }
  }
done:
  if (elect_one()) tc_commit(smem_u32(&bars->drain));
  __syncwarp();
  drain(smem_u32(&bars->drain), 0);
}

// d = 128: both.
template <int D>
__device__ void tall_mma(const PrefixParams &p, uint8_t *smem, TallBars *bars, const int *table, uint32_t tmem_in) {
  using C = TallCfg<D>;
  volatile int *abort_flag = &bars->abort;
  const uint32_t tmem = uniform(tmem_in);
  uint32_t use = 0, items = 0, pc = 0;   // uses of the rings; parities of p_full, a bit a row tile
  const uint64_t qdesc = smem_desc_sw128(smem_u32(smem), 16, 1024);
  const uint64_t kdesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
  const uint64_t vdesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_V), kHalf, 1024);
  auto wait = [&](uint64_t &bar, uint32_t parity) { return wait_for<false>(smem_u32(&bar), parity, abort_flag, p); };
  PrefixWalk walk = bars->start.walk;
  PrefixItem item = bars->start.item;
  bool more = bars->start.any != 0;
  for (; more; ++items, more = next_item(&bars->start, table, &walk, &item)) {
    const int kv0 = uniform(item.kv0), kv1 = uniform(item.kv1);
    TallTiles tiles[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const TallTiles x = tiles_of(p, table, item, t);
      tiles[t] = TallTiles{uniform(x.kv0), uniform(x.prefix), uniform(x.own0), uniform(x.own1)};
    }
    int b = item.b_lo;
    if (!wait(bars->q_full, items & 1)) goto done;
    bool active[2] = {false, false}, fresh[2] = {true, true};   // at the tile before; no product of this item yet
    // Tiles before `plain`: both row tiles take them, and no V but the last has rows to clear.
    const int plain = uniform(item.row0 + BM >= p.rows ? 0 : item.b_lo == item.b_hi ? kv1 : min(kv1, p.n_prefix));
    for (int j = kv0; j <= kv1; ++j, ++use) {
      // Between two of them both row tiles have a product and scores.
      if (j > kv0 && j < plain) {
        for (; j < plain; ++j, ++use) {
          const uint32_t vs = (use - 1) % C::VS, ks = use % C::KS;
          const uint64_t vd = vdesc0 + static_cast<uint64_t>(vs * (C::TILE >> 4)), kd = kdesc0 + static_cast<uint64_t>(ks * (C::TILE >> 4));
          if (!wait(bars->v_full[vs], (use - 1) / C::VS & 1)) goto done;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!wait(bars->p_full[t], pc >> t & 1)) goto done;
            tc_fence_after();
            if (elect_one()) {
              issue_pv<D>(tmem + 256 + t * D, tmem + t * 128, vd, fresh[t] ? 0u : 1u);
              if (t == 1) tc_commit(smem_u32(&bars->v_empty[vs]));
            }
            __syncwarp();
            // (K is waited for after the first product, which does not need it.)
            if (t == 0) {
              if (!wait(bars->k_full[ks], use / C::KS & 1)) goto done;
              tc_fence_after();
            }
            if (elect_one()) {
              issue_qk<D>(tmem + t * 128, qdesc + static_cast<uint64_t>(t * (C::TILE >> 4)), kd);
              tc_commit(smem_u32(&bars->s_full[t]));
              if (t == 1) {
                tc_commit(smem_u32(&bars->k_empty[ks]));
                if (j == kv1 - 1) tc_commit(smem_u32(&bars->q_empty));
              }
            }
            __syncwarp();
            fresh[t] = false;
          }
          pc ^= 3u;
        }
      }
      const uint32_t vs = (use - 1) % C::VS, ks = use % C::KS;   // the last tile's V, this one's K
      const bool now[2] = {j < kv1 && tiles[0].has(j), j < kv1 && tiles[1].has(j)};
      if (j > kv0) {
        if (!wait(bars->v_full[vs], (use - 1) / C::VS & 1)) goto done;
        if (j - 1 >= p.n_prefix) {
          const int valid = uniform(own_tile(p, table, item, j - 1, b).valid);
          if (valid < BN) clear_tail<D>(smem + C::OFF_V + vs * C::TILE, valid);
        }
      }
      const uint64_t vd = vdesc0 + static_cast<uint64_t>(vs * (C::TILE >> 4)), kd = kdesc0 + static_cast<uint64_t>(ks * (C::TILE >> 4));
      if (active[0]) {
        if (!wait(bars->p_full[0], pc & 1)) goto done;
        pc ^= 1u;
        tc_fence_after();
        if (elect_one()) {
          issue_pv<D>(tmem + 256, tmem, vd, fresh[0] ? 0u : 1u);
          if (j - 1 == tiles[0].last()) tc_commit(smem_u32(&bars->o_full[0]));
        }
        __syncwarp();
        fresh[0] = false;
      }
      // (K is waited for after the first product, which does not need it.)
      if (j < kv1) {
        if (!wait(bars->k_full[ks], use / C::KS & 1)) goto done;
        tc_fence_after();
        if (now[0] && elect_one()) {
          issue_qk<D>(tmem, qdesc, kd);
          tc_commit(smem_u32(&bars->s_full[0]));
        }
        __syncwarp();
      }
      if (active[1]) {
        if (!wait(bars->p_full[1], pc >> 1 & 1)) goto done;
        pc ^= 2u;
        tc_fence_after();
      }
      if (elect_one()) {
        if (active[1]) {
          issue_pv<D>(tmem + 256 + D, tmem + 128, vd, fresh[1] ? 0u : 1u);
          if (j - 1 == tiles[1].last()) tc_commit(smem_u32(&bars->o_full[1]));
        }
        if (now[1]) {
          issue_qk<D>(tmem + 128, qdesc + static_cast<uint64_t>(C::TILE >> 4), kd);
          tc_commit(smem_u32(&bars->s_full[1]));
        }
        if (j > kv0) tc_commit(smem_u32(&bars->v_empty[vs]));
        if (j < kv1) tc_commit(smem_u32(&bars->k_empty[ks]));
        if (j == kv1 - 1) tc_commit(smem_u32(&bars->q_empty));
      }
      __syncwarp();
      if (active[1]) fresh[1] = false;
      active[0] = now[0];
      active[1] = now[1];
    }
    --use;   // (the step past the last tile has no K)
  }
done:
  // All MMAs issued must finish before Tensor Memory is released.
  if (elect_one()) tc_commit(smem_u32(&bars->drain));
  __syncwarp();
  drain(smem_u32(&bars->drain), 0);
}

// ------------------------------------------------------------------ softmax and epilogue
template <int D>
__device__ void tall_softmax(const PrefixParams &p, uint8_t *smem, TallBars *bars, const int *table, uint32_t tmem) {
  using C = TallCfg<D>;
  const int tid = threadIdx.x, t = tid >> 7, in = tid & 127, wq = in >> 5, lane = tid & 31;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(wq * 32) << 16);
  const uint32_t tS = lanes + t * 128, tP = lanes + C::COL_P + t * C::P_STEP, tO = lanes + 256 + t * D;
  const uint32_t s_full = smem_u32(&bars->s_full[t]), p_full = smem_u32(&bars->p_full[t]);
  const uint32_t o_full = smem_u32(&bars->o_full[t]);
  volatile int *abort_flag = &bars->abort;
  const float scale = p.scale_log2;
  uint32_t step = 0, outs = 0;
  PrefixWalk walk = bars->start.walk;
  PrefixItem item = bars->start.item;
  bool more = bars->start.any != 0;
  bool cut = false, ok = true;   // a piece was this CTA's first of its unit
  for (; ok && more; more = next_item(&bars->start, table, &walk, &item)) {
    const int row = item.row0 + t * BM + in;
    const TallTiles tiles = tiles_of(p, table, item, t);
    const PrefixRange own = range_of(p, table, row);
    const int n = tiles.count();
    float m = -INFINITY, l = 0.f;
    // The keys [lo, hi) of a tile that the row sees: first the prefix's tiles, then its own.
    const int n_own = n - (tiles.own1 - tiles.own0), own_lo = own.lo - own_pos(p, item, tiles.own0), own_len = own.hi - own.lo;
    int lo = -tiles.kv0 * BN, hi = p.Np - tiles.kv0 * BN;
    for (int i = 0; i < n; ++i, ++step, lo -= BN, hi -= BN) {
      if (i == n_own) {
        lo = own_lo;
        hi = own_lo + own_len;
      }
      const bool masked = __any_sync(0xffffffffu, lo > 0 || hi < BN);
      if (!wait_for<true>(s_full, step & 1, abort_flag, p)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // d = 64: the scores have been loaded; the last product, whose weights lie where the next ones go, is done.
      auto scores_read = [&] {
        if constexpr (D == 64) {
          tc_fence_before();
          mbar_arrive(smem_u32(&bars->s_read[t]));
        }
      };
      auto product_done = [&] {
        if constexpr (D == 64) {
          if (step == 0) return true;
          const bool done = wait_for<true>(smem_u32(&bars->pv_done[t]), (step - 1) & 1, abort_flag, p);
          tc_fence_after();
          return done;
        }
        return true;
      };
      if (masked) {
        if (__all_sync(0xffffffffu, lo >= BN || hi <= 0)) {   // nothing for any row: no weight
          scores_read();
          ok = product_done();
          if (!ok) break;
          zero_weights(tP);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(p_full);
          continue;
        }
        mask_scores<4>(tS, nullptr, 1.f, lo, hi);
      }
      uint32_t s[4][32];
      tmem_ld32(tS, s[0]);
      tmem_ld32(tS + 32, s[1]);
      tmem_ld32(tS + 64, s[2]);
      tmem_ld32(tS + 96, s[3]);
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_wait_ld_regs(s[c]);
      scores_read();
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) mx = max32(s[c], mx);
      const float m_new = fmaxf(m, mx * scale);
      float alpha = 1.f;
      bool rescale = false;
      if (i == 0) {
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
      ok = product_done();
      if (!ok) break;
      const uint64_t scale2 = f2_pack(scale, scale), negm2 = f2_pack(neg, neg);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
        weights32(s[c], scale2, negm2, pk, sum);
        tmem_st16(tP + 16 * c, pk);
      }
      l = fmaf(l, alpha, total(sum));
      if (rescale) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + 32 * c, o);
          tmem_wait_ld_regs(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
          tmem_st32(tO + 32 * c, o);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(p_full);
    }
    if (ok && n > 0) {
      ok = wait_for<true>(o_full, outs & 1, abort_flag, p);
      ++outs;
    }
    if (!ok) break;
    tc_fence_after();
    if (item.piece) {
      float *part = part_of<D>(p, blockIdx.x, item.kv0 == 0 ? 1 : 0, 2 * BM);
      const int at = t * BM + in;
      if (item.kv0 == 0) cut = true;
      if (row < p.rows) {
        __stcg(part + D * 2 * BM + at, m);
        __stcg(part + (D + 1) * 2 * BM + at, l);
      }
      if (tid == 0 && item.kv0 == 0) {
        __stcg(cut_place(p, item.unit), make_int4(blockIdx.x, pieces_of(p, bars->start.plan, item.u0, item.n), item.hk, item.row0));
      }
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * c, o);
        tmem_wait_ld_regs(o);
        if (row < p.rows)
#pragma unroll
          for (int k = 0; k < 8; ++k)   // (without a tile there is nothing in O)
            __stcg(reinterpret_cast<float4 *>(part) + (8 * c + k) * 2 * BM + at,
                   n == 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                          : make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                        __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3])));
      }
      tc_fence_before();
      continue;
    }
    if (tid == 0 && item.u0 > 0 && cut_by_unit(p)) __stcg(cut_place(p, item.unit), make_int4(0, 0, 0, 0));
    // Rows lie across the lanes: through shared memory, 64 columns at a time (16-byte chunks, each row's
    // permuted by its number against bank conflicts), so that eight lanes store a row's 128 bytes together.
    const float norm = l == 0.f ? 0.f : 1.f / l;
    const unsigned long long dst = reinterpret_cast<unsigned long long>(out_row(p, item.hk, row, D));
    uint4 *stg = reinterpret_cast<uint4 *>(smem + C::OFF_STG) + (tid / 32) * 32 * 8;
#pragma unroll 1
    for (int c = 0; c < D / 64; ++c) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t o[32];
        tmem_ld32(tO + 64 * c + 32 * hf, o);
        tmem_wait_ld_regs(o);
        float x[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] = n == 0 ? 0.f : __uint_as_float(o[k]) * norm;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          stg[lane * 8 + ((4 * hf + k) ^ (lane & 7))] =
              make_uint4(pack_bf16x2(x[8 * k], x[8 * k + 1]), pack_bf16x2(x[8 * k + 2], x[8 * k + 3]),
                         pack_bf16x2(x[8 * k + 4], x[8 * k + 5]), pack_bf16x2(x[8 * k + 6], x[8 * k + 7]));
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = 4 * k + lane / 8, ch = lane & 7;
        const unsigned long long to = __shfl_sync(0xffffffffu, dst, r);
        const uint4 v = stg[r * 8 + (ch ^ (r & 7))];
        if (to) reinterpret_cast<uint4 *>(to)[8 * c + ch] = v;
      }
      __syncwarp();   // the staged rows have been read
    }
    tc_fence_before();
  }
  if (p.split && tid == 0 && !cut && !cut_by_unit(p)) __stcg(p.cuts + blockIdx.x, make_int4(0, 0, 0, 0));
}

template <int D>
__global__ void __launch_bounds__(TallCfg<D>::THREADS, 1) prefix_tall_kernel(const __grid_constant__ PrefixParams p) {
  using C = TallCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];   // the swizzle pattern repeats every 1024 bytes
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicExch(p.status, kDevBadPlan);
    return;
  }
  TallBars *bars = reinterpret_cast<TallBars *>(smem + C::OFF_BAR);
  int *table = reinterpret_cast<int *>(smem + C::OFF_TAB);
  const int warp = uniform(threadIdx.x / 32);
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars->q_full), 1);
    mbar_init(smem_u32(&bars->q_empty), 1);
    for (int s = 0; s < C::KS; ++s) {
      mbar_init(smem_u32(&bars->k_full[s]), 1);
      mbar_init(smem_u32(&bars->k_empty[s]), 1);
      mbar_init(smem_u32(&bars->v_full[s]), 1);
      mbar_init(smem_u32(&bars->v_empty[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&bars->s_full[t]), 1);
      mbar_init(smem_u32(&bars->p_full[t]), BM);
      mbar_init(smem_u32(&bars->o_full[t]), 1);
      mbar_init(smem_u32(&bars->s_read[t]), BM);
      mbar_init(smem_u32(&bars->pv_done[t]), 1);
    }
    mbar_init(smem_u32(&bars->drain), D == 64 ? 2 : 1);   // a commit of each issuer
    bars->abort = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) begin_schedule(p, table, &bars->start);
  if (warp == kTallMma) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (p.split) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join waits for this grid's end itself
  const uint32_t tmem = bars->tmem_base;
  if (warp < kTallMma)
    tall_softmax<D>(p, smem, bars, table, tmem);
  else if (warp == kTallLoad)
    tall_loader<D>(p, smem, bars, table);
  else if constexpr (D == 64) {
    if (warp == kTallMma)
      tall_scores<D>(p, smem, bars, table, tmem);
    else
      tall_products<D>(p, smem, bars, table, tmem);
  } else {
    tall_mma<D>(p, smem, bars, table, tmem);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kTallMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}
