// Differential attention at d = 256: two maps of 128 columns over 256 columns of v.
//
// Included by attn_diff.cu inside its anonymous namespace (it uses that file's schedule, waits
// and softmax helpers).
//
// O of one map takes 256 of Tensor Memory's 512 columns, so the two maps of a query tile do not
// fit beside their scores. A unit (one query tile of one head) therefore runs map 1 over all its
// keys, leaves its unnormalised O in the workspace (fp32, 128 KB a CTA, which stay in L2), runs
// map 2, and combines the two. Scores are double-buffered: those of the next tile are computed
// while the softmax works on this one. Per KV tile and map the tensor pipe has 1536 cycles of
// work (512 for the scores, 1024 for the products), the softmax of four warps about as much.
// Bound: at 2.0 us a tile of both maps (2070 cycles a map) neither is full. Each SM reads 96 KB a
// tile and map from L2, about as fast as it gives them, and a unit costs 7.4 us beside its tiles
// (the loads of Q and the first K, O through the workspace, the stores). Measured (GB300): 12 heads
// of 4096 queries and keys 218 us = 1418 TFLOP/s, 76% of the cuBLAS rate. Map 2 reads V again: from L2
// while query tiles of a head run side by side, from HBM with few queries and long keys (one query of
// 8 heads against 65536 keys 136 us, 1.7 times what its bytes take once). Tried: both maps at once
// on halves of v's columns (half of the scores' work twice) 317-331 us; two places for Q and one
// tile of V 241 us.
//
// Roles (224 threads, one CTA per SM): warps 0-3 softmax and epilogue (a thread per row), warp 4
// the scores' issuer, warp 5 the products' issuer, warp 6 the TMA loader.
// Tensor Memory: S of even tiles [0,128), of odd ones [128,256); P (bf16 pairs) overwrites the
// first 64 columns of its S; O [256,512).
// Shared memory: Q of the map | K ring (2 tiles of a map's 128 columns) | V ring (2 tiles, as 4
// halves of 128 columns) | barriers | the norm's weights. (The other map's Q comes in while the
// epilogue of the map before runs; a second place for it in V's stead left every tile waiting for V.)
struct WideCfg {
  static constexpr int DH = 128, DV = 256, DQ = 256;
  static constexpr int SLOT = BN * 128 * 2;
  static constexpr int KS = 2, VS = 4;
  static constexpr int OFF_K = SLOT, OFF_V = OFF_K + KS * SLOT;
  static constexpr int OFF_BAR = OFF_V + VS * SLOT, OFF_W = OFF_BAR + 768;
  static constexpr int SMEM = OFF_W + 4 * DV;
  static constexpr int THREADS = 224;
  static constexpr uint32_t COL_O = 256;
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

// fp32 values of a piece's partial result: O and (m, l) of both maps, `rows` rows each.
__host__ __device__ constexpr int wide_part_floats(int rows) { return 2 * WideCfg::DV * rows + 4 * rows; }

struct WideBars {
  static constexpr int kScore = 4, kProduct = 5, kLoad = 6;   // warps
  uint64_t q_full, q_empty;
  uint64_t k_full[WideCfg::KS], k_empty[WideCfg::KS], v_full[WideCfg::VS], v_empty[WideCfg::VS];
  uint64_t s_full[2], p_full[2][2], pv_done[2];   // [S buffer], P by halves of 64 keys
  uint64_t o_full, drain[2];
  uint64_t item_full[4];
  DPlan plan;
  DTask task[4];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(WideBars) <= 768, "barrier block too large");

// A slot and the parity of its use, stepped by one role.
template <int N>
struct WideRing {
  uint32_t slot = 0, parity = 0;
  __device__ __forceinline__ void advance() {
    if (++slot == N) {
      slot = 0;
      parity ^= 1;
    }
  }
};

__device__ void wide_loader(const DiffParams &p, uint8_t *smem, WideBars *bars) {
  using C = WideCfg;
  uint32_t passes = 0, published = 0, k_uses = 0, v_uses = 0;   // passes: Q loads
  WideRing<C::KS> kr;
  WideRing<C::VS> vr;
  // 128 columns from x of 128 rows, as two 64-column halves.
  auto load = [&](uint32_t dst, const CUtensorMap *m, uint32_t full, int x, int row, int h, int b) {
    if (elect_one()) {
      mbar_arrive_expect_tx(full, C::SLOT);
      tma_load_4d(dst, m, full, x, row, h, b);
      tma_load_4d(dst + kDiffHalf, m, full, x + 64, row, h, b);
    }
    __syncwarp();
  };
  // Item i's record is written once the scores of item i - 1 are done: the softmax has then begun
  // the last tile but two of item i - 1 at least, and four records are enough.
  auto publish = [&](const DTask &task) {
    if (elect_one()) {
      bars->task[published & 3] = task;
      mbar_arrive(smem_u32(&bars->item_full[published & 3]));
    }
    __syncwarp();
    ++published;
  };
  DWalk walk;
  walk.start(p, bars->plan);
  DItem item;
  bool ok = true;
  while (ok && walk.next(p, item)) {
    const DPlace at = place_of(p, item);
    const int hk = at.h / p.group;
    for (int t = 0; ok && t < 2; ++t) {
      ok = diff_wait(smem_u32(&bars->q_empty), (passes & 1) ^ 1, bars, p);
      if (!ok) break;
      if (t == 0)
        publish(DTask{item.u0, item.b, item.keys, item.kv0, item.kv1, item.nk, at.h, at.q0, 0,
                      static_cast<short>(item.piece ? 2 : 1)});
      load(smem_u32(smem), &p.tm_q, smem_u32(&bars->q_full), t * C::DH, at.q0, at.h, item.b);
      ++passes;
      // K runs a tile ahead of V: a K slot is free as soon as its scores are done, a V slot only
      // when the products are, and the scores behind them should not wait for a load.
      for (int j = item.kv0 - 1; ok && j < item.kv1; ++j) {
        if (j + 1 < item.kv1) {
          ok = diff_wait(smem_u32(&bars->k_empty[kr.slot]), kr.parity ^ 1, bars, p);
          if (!ok) break;
          load(smem_u32(smem + C::OFF_K + kr.slot * C::SLOT), &p.tm_k, smem_u32(&bars->k_full[kr.slot]),
               t * C::DH, (j + 1) * BN, hk, item.b);
          kr.advance();
          ++k_uses;
        }
        for (int c = 0; ok && j >= item.kv0 && c < 2; ++c) {
          ok = diff_wait(smem_u32(&bars->v_empty[vr.slot]), vr.parity ^ 1, bars, p);
          if (!ok) break;
          load(smem_u32(smem + C::OFF_V + vr.slot * C::SLOT), &p.tm_v, smem_u32(&bars->v_full[vr.slot]),
               c * 128, j * BN, hk, item.b);
          vr.advance();
          ++v_uses;
        }
      }
    }
  }
  publish(DTask{0, 0, 0, 0, 0, 0, 0, 0, 0, 0});
  // Every load issued must land before the CTA releases its shared memory.
  for (uint32_t s = 0; s < C::KS; ++s)
    if (k_uses > s) diff_drain(smem_u32(&bars->k_full[s]), ((k_uses - 1 - s) / C::KS) & 1);
  for (uint32_t s = 0; s < C::VS; ++s)
    if (v_uses > s) diff_drain(smem_u32(&bars->v_full[s]), ((v_uses - 1 - s) / C::VS) & 1);
  if (passes > 0) diff_drain(smem_u32(&bars->q_full), (passes - 1) & 1);
}

// S of tile g into buffer g & 1, once the products of tile g - 2 have read P there.
__device__ void wide_score_issuer(const DiffParams &p, uint8_t *smem, WideBars *bars, uint32_t tmem_in) {
  using C = WideCfg;
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, 0);
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_in, 0);
  uint32_t q_parity = 0, buf = 0, parity = 0;   // S buffer and the parity of its use
  WideRing<C::KS> kr;
  const uint64_t qdesc = smem_desc_sw128(smem_u32(smem), 16, 1024);
  const uint64_t kdesc = smem_desc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
  DWalk walk;
  walk.start(p, bars->plan);
  DItem item;
  while (walk.next(p, item)) {
    const int nk = uniform(item.kv1 - item.kv0);
#pragma unroll 1
    for (int t = 0; t < 2; ++t, q_parity ^= 1) {
      if (!diff_wait(smem_u32(&bars->q_full), q_parity, bars, p)) goto drain;
#pragma unroll 1
      for (int j = 0; j < nk; ++j) {
        if (!diff_wait(smem_u32(&bars->k_full[0]) + 8 * kr.slot, kr.parity, bars, p)) goto drain;
        if (!diff_wait(smem_u32(&bars->pv_done[0]) + 8 * buf, parity ^ 1, bars, p)) goto drain;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t kd = kdesc + static_cast<uint64_t>(kr.slot * (C::SLOT >> 4));
#pragma unroll
          for (int kk = 0; kk < C::DH / 16; ++kk) {
            const uint64_t o = static_cast<uint64_t>(((kk / 4) * kDiffHalf + (kk % 4) * 32) >> 4);
            tc_mma_ss(tmem + buf * 128, qdesc + o, kd + o, idesc, kk > 0 ? 1u : 0u);
          }
          tc_commit(smem_u32(&bars->s_full[0]) + 8 * buf);
          tc_commit(smem_u32(&bars->k_empty[0]) + 8 * kr.slot);
          if (j == nk - 1) tc_commit(smem_u32(&bars->q_empty));
        }
        __syncwarp();
        kr.advance();
        buf ^= 1;
        if (buf == 0) parity ^= 1;
      }
    }
  }
drain:
  // All MMAs issued must finish before Tensor Memory is released.
  if (elect_one()) tc_commit(smem_u32(&bars->drain[0]));
  __syncwarp();
  diff_drain(smem_u32(&bars->drain[0]), 0);
}

// O += P V, by halves of 64 keys as their weights are written, each over two halves of 128 columns.
__device__ void wide_product_issuer(const DiffParams &p, uint8_t *smem, WideBars *bars, uint32_t tmem_in) {
  using C = WideCfg;
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, 1);
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_in, 0);
  const int lane = threadIdx.x & 31;
  uint32_t buf = 0, parity = 0;
  WideRing<C::VS> vr;
  const uint64_t vdesc = smem_desc_sw128(smem_u32(smem + C::OFF_V), kDiffHalf, 1024);
  DWalk walk;
  walk.start(p, bars->plan);
  DItem item;
  while (walk.next(p, item)) {
    const int nk = uniform(item.kv1 - item.kv0);
    // Rows of V behind the batch entry's last key are cleared (see diff_product_issuer).
    const int last_valid = uniform(item.keys >= p.Nk || item.kv1 < item.nk ? BN : item.keys - (item.nk - 1) * BN);
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
#pragma unroll 1
      for (int j = 0; j < nk; ++j) {
        WideRing<C::VS> v[2] = {vr, vr};
        v[1].advance();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (!diff_wait(smem_u32(&bars->v_full[0]) + 8 * v[c].slot, v[c].parity, bars, p)) goto drain;
          if (j == nk - 1 && last_valid < BN) {
            uint8_t *tile = smem + C::OFF_V + v[c].slot * C::SLOT;
            for (int hf = 0; hf < 2; ++hf)
              for (int o = last_valid * 128 + lane * 16; o < kDiffHalf; o += 512)
                *reinterpret_cast<uint4 *>(tile + hf * kDiffHalf + o) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!diff_wait(smem_u32(&bars->p_full[0][0]) + 16 * buf + 8 * half, parity, bars, p)) goto drain;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint64_t vd = vdesc + static_cast<uint64_t>(v[c].slot * (C::SLOT >> 4)) +
                                  (half == 0 ? 0 : kChunkRows);
#pragma unroll
              for (int kk = 0; kk < BC / 16; ++kk)
                tc_mma_ts(tmem + C::COL_O + c * 128, tmem + buf * 128 + half * 32 + kk * 8,
                          vd + static_cast<uint64_t>((kk * 2048) >> 4), idesc,
                          j > 0 || half > 0 || kk > 0 ? 1u : 0u);
              if (half == 1) tc_commit(smem_u32(&bars->v_empty[0]) + 8 * v[c].slot);
            }
            if (half == 1) {
              tc_commit(smem_u32(&bars->pv_done[0]) + 8 * buf);
              if (j == nk - 1) tc_commit(smem_u32(&bars->o_full));
            }
          }
          __syncwarp();
        }
        vr = v[1];
        vr.advance();
        buf ^= 1;
        if (buf == 0) parity ^= 1;
      }
    }
  }
drain:
  if (elect_one()) tc_commit(smem_u32(&bars->drain[1]));
  __syncwarp();
  diff_drain(smem_u32(&bars->drain[1]), 0);
}

// scaled_squares of a row whose 256 combined columns lie in O's Tensor Memory columns; all lanes take part.
__device__ __noinline__ float wide_squares(uint32_t tO, float ss) {
  float big = 0.f, sum = 0.f;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    const float s = near_one(big);   // (2^126 in the first pass, which does not use the sum)
    sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < WideCfg::DV / 32; ++c) {
      uint32_t x[32];
      tmem_ld32(tO + 32 * c, x);
      tmem_wait_ld_regs(x);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float y = __uint_as_float(x[i]);
        big = fmaxf(big, fabsf(y));
        sum = fmaf(y * s, y * s, sum);
      }
    }
  }
  return !squares_fit(ss) && has_root(big, ss) ? minus_root(sum, big) : ss;
}

// The final row, whose 256 combined columns lie in O's Tensor Memory columns: norm, factor, store.
__device__ __forceinline__ void wide_finish(const DiffParams &p, const float *weight, int b, int h, int n,
                                            bool live, uint32_t tO, float ss) {
  using C = WideCfg;
  float f = p.out_scale;
  if (p.weight) {
    if (__any_sync(0xffffffffu, !squares_fit(ss))) ss = wide_squares(tO, ss);
    f *= norm_factor(ss, C::DQ, p.eps);
  }
  uint4 *dst = live ? reinterpret_cast<uint4 *>(out_row(p, b, h, n, C::DQ)) : nullptr;
#pragma unroll 1
  for (int c = 0; c < C::DV / 32; ++c) {
    uint32_t x[32];
    tmem_ld32(tO + 32 * c, x);
    tmem_wait_ld_regs(x);
    if (live) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = __uint_as_float(x[8 * i + k]) * f;
        if (p.weight) {
          const float4 w0 = reinterpret_cast<const float4 *>(weight + 32 * c)[2 * i];
          const float4 w1 = reinterpret_cast<const float4 *>(weight + 32 * c)[2 * i + 1];
          y[0] *= w0.x, y[1] *= w0.y, y[2] *= w0.z, y[3] *= w0.w;
          y[4] *= w1.x, y[5] *= w1.y, y[6] *= w1.z, y[7] *= w1.w;
        }
        dst[4 * c + i] = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                    pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
      }
    }
    __syncwarp();
  }
}

// O of a row to the workspace, as float4 groups [col/4][row][4].
__device__ __forceinline__ void wide_leave(uint32_t tO, float4 *to, int stride, bool live) {
#pragma unroll 1
  for (int c = 0; c < WideCfg::DV / 32; ++c) {
    uint32_t o[32];
    tmem_ld32(tO + 32 * c, o);
    tmem_wait_ld_regs(o);
    if (live) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        __stcg(to + (8 * c + i) * stride,
               make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                           __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3])));
    }
    __syncwarp();
  }
}

// The pieces' common reference: 0 where no piece has a score above -inf, whose factors 2^(-inf - 0)
// are then 0 as the weights were (neg2), and the row's map gives 0 as it does in a whole unit.
__device__ __forceinline__ float finite_ref(float m) { return m == -INFINITY ? 0.f : m; }

// The end of a piece, per warp (its 32 rows): both maps' O, m and l are in the workspace. The
// warp that counts the last piece of these rows merges all of them in piece order.
__device__ __noinline__ void wide_merge(const DiffParams &p, const WideBars *bars, const float *weight,
                                        const DTask item, uint32_t tO, float lambda) {
  using C = WideCfg;
  const int lane = threadIdx.x & 31, wq = threadIdx.x / 32, row = threadIdx.x;
  const int R = p.part_rows, rows = min(BM, p.Nq - item.q0);
  const DSpan span = span_of(bars->plan, item);
  const int c0 = span.first, S = span.pieces;
  auto part = [&](int k) { return p.parts + (static_cast<size_t>(c0 + k) * 2 + (k == 0 ? 1 : 0)) * wide_part_floats(R); };
  auto stat_of = [&](int k) { return reinterpret_cast<const float4 *>(part(k) + 2 * C::DV * R); };
  __threadfence();
  __syncwarp();
  int last = 0;
  int *count = p.count + c0 * 4 + wq;
  if (lane == 0) {
    last = atomicAdd(count, 1) == S - 1;
    if (last) *count = 0;   // ready for the next launch
  }
  if (!__shfl_sync(0xffffffffu, last, 0)) return;
  __threadfence();
  if (rows > kFewRows) {
    const bool live = row < rows;
    const int r = live ? row : wq * 32;   // rows that are not there read one that is
    float m1 = -INFINITY, m2 = -INFINITY, l1 = 0.f, l2 = 0.f;
#pragma unroll 4
    for (int k = 0; k < S; ++k) {
      const float4 s = __ldcg(stat_of(k) + r);
      m1 = fmaxf(m1, s.x);
      m2 = fmaxf(m2, s.z);
    }
    m1 = finite_ref(m1), m2 = finite_ref(m2);
#pragma unroll 4
    for (int k = 0; k < S; ++k) {
      const float4 s = __ldcg(stat_of(k) + r);
      l1 = fmaf(ex2_approx(s.x - m1), s.y, l1);
      l2 = fmaf(ex2_approx(s.z - m2), s.w, l2);
    }
    const float f1 = map_factor(0, lambda, l1), f2 = map_factor(1, lambda, l2);
    float ss = 0.f;
#pragma unroll 1
    for (int c = 0; c < C::DV / 32; ++c) {
      float x[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = 0.f;
      // Two pieces' loads in flight at a time; the sum still runs in piece order.
#pragma unroll 1
      for (int k = 0; k < S; k += 2) {
        const int k2 = k + 1 < S ? k + 1 : k;
        const float4 s = __ldcg(stat_of(k) + r), s2 = __ldcg(stat_of(k2) + r);
        const float4 *a = reinterpret_cast<const float4 *>(part(k)) + 8 * c * R + r;
        const float4 *b = reinterpret_cast<const float4 *>(part(k2)) + 8 * c * R + r;
        float4 u[8], v[8], u2[8], v2[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          u[i] = __ldcg(a + i * R);
          v[i] = __ldcg(a + (C::DV / 4 + i) * R);
          u2[i] = __ldcg(b + i * R);
          v2[i] = __ldcg(b + (C::DV / 4 + i) * R);
        }
        const float g1 = f1 * ex2_approx(s.x - m1), g2 = f2 * ex2_approx(s.z - m2);
        const float h1 = k2 > k ? f1 * ex2_approx(s2.x - m1) : 0.f;
        const float h2 = k2 > k ? f2 * ex2_approx(s2.z - m2) : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          add_piece(x + 4 * i, g1, u[i], g2, v[i]);
          if (k2 > k) add_piece(x + 4 * i, h1, u2[i], h2, v2[i]);
        }
      }
      uint32_t o[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        ss = fmaf(x[i], x[i], ss);
        o[i] = __float_as_uint(x[i]);
      }
      __syncwarp();
      tmem_st32(tO + 32 * c, o);
    }
    tmem_wait_st();
    wide_finish(p, weight, item.b, item.h, item.q0 + row, live, tO, ss);
    return;
  }
  // Few rows: row by row, a lane takes columns 4 * lane and 128 + 4 * lane.
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
    m1 = finite_ref(m1), m2 = finite_ref(m2);
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
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < S; ++k) {
      const float4 s = __ldcg(stat_of(k) + r);
      const float g1 = f1 * ex2_approx(s.x - m1), g2 = f2 * ex2_approx(s.z - m2);
      const float4 *a = reinterpret_cast<const float4 *>(part(k)) + lane * R + r;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 u = __ldcg(a + i * 32 * R), v = __ldcg(a + (C::DV / 4 + i * 32) * R);
        add_piece(x + 4 * i, g1, u, g2, v);
      }
    }
    float f = p.out_scale;
    if (p.weight) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      ss = lanes_squares(x, ss, 32);
      f *= norm_factor(ss, C::DQ, p.eps);
    }
    uint2 *dst = reinterpret_cast<uint2 *>(out_row(p, item.b, item.h, item.q0 + r, C::DQ));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float4 w = make_float4(1.f, 1.f, 1.f, 1.f);
      if (p.weight) w = reinterpret_cast<const float4 *>(weight)[lane + 32 * i];
      dst[lane + 32 * i] = make_uint2(pack_bf16x2(x[4 * i] * f * w.x, x[4 * i + 1] * f * w.y),
                                      pack_bf16x2(x[4 * i + 2] * f * w.z, x[4 * i + 3] * f * w.w));
    }
  }
}

__device__ void wide_softmax(const DiffParams &p, uint8_t *smem, WideBars *bars, uint32_t tmem) {
  using C = WideCfg;
  const int row = threadIdx.x, wq = row / 32;
  const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
  const uint32_t tO = tmem + lane_base + C::COL_O;
  const uint32_t s_full = smem_u32(&bars->s_full[0]), p_full = smem_u32(&bars->p_full[0][0]);
  const uint32_t pv_done = smem_u32(&bars->pv_done[0]), o_full = smem_u32(&bars->o_full);
  const float *weight = reinterpret_cast<const float *>(smem + C::OFF_W);
  const uint64_t scale2 = f2_pack(p.scale_log2, p.scale_log2);
  const int R = p.part_rows;
  uint32_t buf = 0, parity = 0;   // S buffer and the parity of its use
  for (uint32_t items = 0;; ++items) {
    if (!diff_wait_inline(smem_u32(&bars->item_full[items & 3]), (items >> 2) & 1, bars, p)) return;
    const DTask &item = bars->task[items & 3];
    if (item.kind == 0) return;
    const bool idle = item.q0 + wq * 32 >= p.Nq;   // no query in this warp's rows
    const bool live = item.q0 + row < p.Nq;
    const float lambda = __ldg(p.lambda + item.h);
    const int nk = item.kv1 - item.kv0;
    // Where this item's O and sums go: a piece's place, or (map 1 of a whole unit) the CTA's own.
    float *place = p.stash + static_cast<size_t>(blockIdx.x) * C::DV * R;
    if (item.kind == 2) {
      const DSpan span = span_of(bars->plan, item);
      place = p.parts + (static_cast<size_t>(blockIdx.x) * 2 + (static_cast<int>(blockIdx.x) == span.first ? 1 : 0)) *
                            wide_part_floats(R);
    }
    float l1 = 0.f;
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      int valid = item.keys - item.kv0 * BN;
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int j = 0; j < nk; ++j, valid -= BN) {
        if (!diff_wait_inline(s_full + 8 * buf, parity, bars, p)) return;
        const uint32_t tS = tmem + lane_base + buf * 128;
        if (!idle) {
          tc_fence_after();
          if (valid < BN) {
            mask64(tS, valid);
            mask64(tS + BC, valid - BC);
          }
          uint32_t s[4][32];
          tmem_ld32(tS, s[0]);
          tmem_ld32(tS + 32, s[1]);
          tmem_wait_ld_regs(s[0]);
          tmem_wait_ld_regs(s[1]);
          tmem_ld32(tS + 64, s[2]);
          tmem_ld32(tS + 96, s[3]);
          float mx = max64(s[0], s[1]);
          tmem_wait_ld_regs(s[2]);
          tmem_wait_ld_regs(s[3]);
          mx = fmaxf(mx, max64(s[2], s[3])) * p.scale_log2;
          const float before = m;
          if (j == 0 || mx > m + kDiffRescale) m = mx;
          const uint64_t negm2 = neg2(m);
          uint32_t pk[4][16];
          weights32(s[0], scale2, negm2, pk[0]);
          weights32(s[1], scale2, negm2, pk[1]);
          tmem_st16(tS, pk[0]);
          tmem_st16(tS + 16, pk[1]);
          float alpha = 1.f;
          if (j > 0 && __any_sync(0xffffffffu, m != before)) {
            alpha = shrink(before, m);
            // O holds the sum through the last tile once its products are done, and this tile's
            // wait for this thread. The parity is exact: the phase before, of tile g - 3, was
            // waited for before the scores of tile g - 1 were issued.
            const uint32_t pb = buf ^ 1, pp = buf == 1 ? parity : parity ^ 1;
            if (!diff_wait_inline(pv_done + 8 * pb, pp, bars, p)) return;
            tc_fence_after();
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
          mbar_arrive(p_full + 16 * buf);
          weights32(s[2], scale2, negm2, pk[2]);
          weights32(s[3], scale2, negm2, pk[3]);
          tmem_st16(tS + 32, pk[2]);
          tmem_st16(tS + 48, pk[3]);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(p_full + 16 * buf + 8);
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 4; ++i) add_weights(pk[i], sum);
          l = fmaf(l, alpha, (sum[0] + sum[1]) + (sum[2] + sum[3]));
        } else {
          mbar_arrive(p_full + 16 * buf);
          mbar_arrive(p_full + 16 * buf + 8);
        }
        buf ^= 1;
        if (buf == 0) parity ^= 1;
      }
      if (!diff_wait_inline(o_full, t, bars, p)) return;   // two phases an item
      tc_fence_after();
      if (idle) continue;
      if (item.kind == 2) {
        wide_leave(tO, reinterpret_cast<float4 *>(place) + t * (C::DV / 4) * R + row, R, live);
        if (live) __stcg(reinterpret_cast<float2 *>(place + 2 * C::DV * R) + row * 2 + t, make_float2(m, l));
        __syncwarp();
        if (t == 1) wide_merge(p, bars, weight, item, tO, lambda);
      } else if (t == 0) {
        wide_leave(tO, reinterpret_cast<float4 *>(place) + row, R, live);
        l1 = l;
      } else {
        // x = O1 / l1 - lambda O2 / l2, back into O's columns, then the norm over the whole row.
        const float f1 = map_factor(0, lambda, l1), f2 = map_factor(1, lambda, l);
        const float4 *src = reinterpret_cast<const float4 *>(place) + (live ? row : wq * 32);
        float ss = 0.f;
        float4 u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = __ldcg(src + i * R);
#pragma unroll 1
        for (int c = 0; c < C::DV / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + 32 * c, o);
          float4 next[8];
          const int nc = c + 1 < C::DV / 32 ? c + 1 : 0;   // the next chunk's loads run meanwhile
#pragma unroll
          for (int i = 0; i < 8; ++i) next[i] = __ldcg(src + (8 * nc + i) * R);
          tmem_wait_ld_regs(o);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x[4] = {fmaf(f1, u[i].x, f2 * __uint_as_float(o[4 * i])),
                                fmaf(f1, u[i].y, f2 * __uint_as_float(o[4 * i + 1])),
                                fmaf(f1, u[i].z, f2 * __uint_as_float(o[4 * i + 2])),
                                fmaf(f1, u[i].w, f2 * __uint_as_float(o[4 * i + 3]))};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              ss = fmaf(x[k], x[k], ss);
              o[4 * i + k] = __float_as_uint(x[k]);
            }
            u[i] = next[i];
          }
          tmem_st32(tO + 32 * c, o);
        }
        tmem_wait_st();
        wide_finish(p, weight, item.b, item.h, item.q0 + row, live, tO, ss);
      }
      tc_fence_before();   // O has been read: the next P may let new products overwrite it
    }
  }
}

__global__ void __launch_bounds__(WideCfg::THREADS, 1) attn_diff_wide_kernel(const __grid_constant__ DiffParams p) {
  using C = WideCfg;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicExch(p.status, kDevBadPlan);
    return;
  }
  WideBars *bars = reinterpret_cast<WideBars *>(smem + C::OFF_BAR);
  const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->s_full[i]), 1);
      mbar_init(smem_u32(&bars->p_full[i][0]), 128);
      mbar_init(smem_u32(&bars->p_full[i][1]), 128);
      mbar_init(smem_u32(&bars->pv_done[i]), 1);
      mbar_init(smem_u32(&bars->drain[i]), 1);
    }
    for (int i = 0; i < C::KS; ++i) {
      mbar_init(smem_u32(&bars->k_full[i]), 1);
      mbar_init(smem_u32(&bars->k_empty[i]), 1);
    }
    for (int i = 0; i < C::VS; ++i) {
      mbar_init(smem_u32(&bars->v_full[i]), 1);
      mbar_init(smem_u32(&bars->v_empty[i]), 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&bars->item_full[i]), 1);
    mbar_init(smem_u32(&bars->q_full), 1);
    mbar_init(smem_u32(&bars->q_empty), 1);
    mbar_init(smem_u32(&bars->o_full), 1);
    bars->abort = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1 && p.split) plan_split(p, bars);
  if (p.weight)
    for (int i = threadIdx.x; i < C::DV; i += C::THREADS)
      reinterpret_cast<float *>(smem + C::OFF_W)[i] = __ldg(p.weight + i);
  if (warp == WideBars::kScore) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  if (warp == WideBars::kLoad && lane == 0) {
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  if (warp == WideBars::kLoad) {
    wide_loader(p, smem, bars);
  } else if (warp == WideBars::kScore) {
    wide_score_issuer(p, smem, bars, tmem);
  } else if (warp == WideBars::kProduct) {
    wide_product_issuer(p, smem, bars, tmem);
  } else {
    wide_softmax(p, smem, bars, tmem);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == WideBars::kScore) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}
