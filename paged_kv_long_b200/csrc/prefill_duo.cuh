// prefill_duo.cuh — windowed batch prefill at head dim 64 and 128: one CTA for two packed Q tiles
// (2t, 2t + 1) of a KV head, as the CTA pair does at head dim 256. Included by pa_kernels.cu.
//
// With one Q tile a CTA (prefill_kernel) an SM has one softmax warp per scheduler: its exponentials
// take 128 x 128 / 16 = 1,024 cycles a tile on the special-function unit, and while it waits for
// them, reads S or stores P the unit idles; measured 2,450 cycles a tile at head dim 128, of
// which its two products need 1,024. Here two softmax groups (warps 0-3 and 4-7, a thread a row)
// run on two tiles that share every K/V tile, so one's exponentials fill the other's gaps and the K/V copies
// are halved. Warps 8 and 9 issue the MMAs of tile A and of tile B, warps 10 and 11 the copies
// (kv_copy_role, and Q by tensor copy where G divides 128).
//
// Tensor memory (512 columns): O of both tiles (D each), S of both (128 each). P (16-bit pairs, 64
// columns) goes over the lower half of its S: a thread works through its row in chunks of 32
// scores, and chunk k's 16 columns of P end below the scores not yet read. A row's maximum is
// taken in a first pass over S, the exponentials in a second, so a thread holds 64 scores at a
// time and 384 threads fit (168 registers each; ptxas spills 84-88 bytes of them). P is rounded to
// the input type (see prefill_kernel).
//
// Each issuing warp runs PV(j), QK(j+1) of its tile: while one group's softmax works, the other
// tile's two products do. A thread that issues for both tiles loses ~950 cycles a tile to its
// commits and waits (4,850 cycles a pair of tiles, 4,000 as it is; see prefill_pair.cuh on issuing
// threads). P is announced in two halves, so that the first 64 keys' PV overlaps the second half's exponentials.
// The two groups take turns: left alone they fall into step whenever both wait for a K/V tile, and
// then share the special-function unit and the tensor cores by turns of 3,000 and 2,000 cycles.
// The commit that announces S(j) covers every MMA its thread issued before, PV(j - 1) among them,
// so a softmax that has S(j) may rescale O without another wait. V rows that no row of the unit
// sees are zeroed by the issuing warps before their PV (each has waited for every earlier fill of
// the ring itself; the other's zeros are the same).

constexpr int kDuoThreads = 384;
constexpr int kDuoMmaWarp = 8;   // and 9: one per tile
constexpr int kDuoCopyWarp = 10;  // and 11
constexpr int kDuoCopyWarps = 2;

template <int D>
struct DuoCfg {
  static constexpr int NP = D / 64;
  static constexpr int NSLOT = D == 128 ? 10 : 12;
  static constexpr int Q_OFF = 0;                                 // two tiles, NP panels each
  static constexpr int RING_OFF = 2 * NP * kPanel;
  static constexpr int BAR_OFF = RING_OFF + NSLOT * kPanel;
  static constexpr int B_FULL = 0, B_EMPTY = NSLOT, B_QFULL = 2 * NSLOT, B_SFULL = 2 * NSLOT + 1,
                       B_PFULL = 2 * NSLOT + 3,  // [tile][half of the keys]
                       B_TURN = 2 * NSLOT + 7,   // [tile]: its softmax may start the next tile
                       B_DONE = 2 * NSLOT + 9, N_BARS = 2 * NSLOT + 10;
  static constexpr int MISC_OFF = BAR_OFF + 8 * N_BARS;
  static constexpr int SMEM = MISC_OFF + 16;
  static constexpr int LAUNCH_SMEM = SMEM + 1024;
  static constexpr int PANEL_LOG = NP == 2 ? 8 : 7;
  static constexpr uint32_t S_COL = 256;
  static_assert(D == 64 || D == 128, "two Q tiles a CTA at head dim 64 and 128");
  static_assert(LAUNCH_SMEM <= 232448, "exceeds 227 KB of shared memory per CTA");
  static_assert(NSLOT * kPanel >= 2 * kTileRows * (D * 4 + 16), "staging needs the ring");
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kDuoThreads, 1)
    prefill_duo_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_q, const PrefillArgs a_in,
                       const __grid_constant__ ItemTable items) {
  PrefillArgs a = a_in;  // rebased on the item's sequence
  using C = DuoCfg<D>;
  constexpr int NP = C::NP, NSLOT = C::NSLOT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  int64_t tp;
  int g;
  const PaItem it = items.item[blockIdx.x];
  const int32_t rb = batch_rebase<D, true>(a, items, it.rb);
  rb_coords(rb, (a.q_tiles + 1) / 2, a.Hkv, &tp, &g);
  const int64_t kt0 = it.kt0;
  const int n = it.kt1 - it.kt0;
  {
    const int64_t last = 2 * tp + 1 < a.q_tiles ? 2 * tp + 1 : a.q_tiles - 1;
    set_window(a, a.hist_len + tile_first_token(2 * tp, a.G),
               a.hist_len + tile_last_token(last, a.R, a.G));
  }

  int32_t pre_row0 = a.oob_row, pre_row1 = a.oob_row;
  if (warp >= kDuoCopyWarp) {
    const bool report = warp == kDuoCopyWarp;
    pre_row0 = tile_page_row<true, true>(a, kt0, n, 0, lane, report);
    pre_row1 = tile_page_row<true, true>(a, kt0, n, 1, lane, report);
  }
  auto bar = [&](int i) -> uint32_t { return sb + C::BAR_OFF + 8u * (uint32_t)i; };
  auto slot_addr = [&](uint32_t slot) -> uint32_t { return sb + C::RING_OFF + slot * kPanel; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF + 4);
  if (threadIdx.x == 0) {
    for (int i = 0; i < NSLOT; ++i) {
      mbar_init(bar(C::B_FULL + i), 1);
      mbar_init(bar(C::B_EMPTY + i), 2);  // both tiles' products have read it
    }
    mbar_init(bar(C::B_QFULL), a.q_tma ? 1 : 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::B_SFULL + i), 1);
      mbar_init(bar(C::B_TURN + i), 4);
    }
    for (int i = 0; i < 4; ++i) mbar_init(bar(C::B_PFULL + i), 4);
    mbar_init(bar(C::B_DONE), 2);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == kDuoCopyWarp && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    if (a.q_tma) tma_prefetch_desc(&tm_q);
  }
  if (warp == kDuoMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint64_t tmo = a.timeout_ns;

  if (warp < kDuoMmaWarp) {
    // ============================================================ softmax + epilogue
    const int grp = warp >> 2, r = threadIdx.x & 127;  // the tile, the row = tensor-memory lane
    const int64_t qt = 2 * tp + grp;
    const int64_t grow = qt * kTileRows + r;
    const int64_t tok = grow / a.G;
    const bool valid = tok < a.R;
    const int head = g * a.G + (int)(grow % a.G);
    if (!a.q_tma) {
      const uint4* src =
          reinterpret_cast<const uint4*>(a.q + (valid ? (tok * a.Hq + head) * (int64_t)D : 0));
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 v = valid ? __ldg(src + p * 8 + c) : make_uint4(0u, 0u, 0u, 0u);
          st_shared_v4(sb + C::Q_OFF + (grp * NP + p) * kPanel + r * 128 + ((c ^ (r & 7)) << 4),
                       v.x, v.y, v.z, v.w);
        }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::B_QFULL));
    }
    const int64_t limit = valid ? a.hist_len + tok : -1;  // last key this row may see
    const int64_t low = row_low(a, limit);
    const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_s = t_lane + C::S_COL + 128u * grp, t_o = t_lane + (uint32_t)(D * grp);
    const uint32_t sfull = bar(C::B_SFULL + grp), pfull = bar(C::B_PFULL + 2 * grp);
    const uint32_t turn = bar(C::B_TURN + grp), other_turn = bar(C::B_TURN + (grp ^ 1));
    const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int64_t key0 = kv_tile<true>(a, kt0 + j) * kTileKeys;
      uint32_t vis[4];
      const bool masked = visible_bits(a, limit, low, key0, vis);
      // Tile A goes first; B's tile j starts when A's is half done, A's j + 1 when B's j is.
      if (!warp_wait(sfull, (uint32_t)j & 1u, abort_flag, tmo) ||
          ((grp == 1 || j > 0) &&
           !warp_wait(turn, (uint32_t)(grp == 1 ? j : j - 1) & 1u, abort_flag, tmo))) {
        ok = false;
        break;
      }
      tc_fence_after();
      auto mask = [&](float (&s)[32], uint32_t v) {
#pragma unroll
        for (int c = 0; c < 32; ++c) s[c] = (v >> c) & 1u ? s[c] : -INFINITY;
      };
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float s0[32], s1[32];
        tmem_ld32(t_s + 64u * h, s0);
        tmem_ld32(t_s + 64u * h + 32u, s1);
        tmem_wait_ld();
        if (masked) {
          mask(s0, vis[2 * h]);
          mask(s1, vis[2 * h + 1]);
        }
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          mx[0] = fmaxf(mx[0], s0[c]);
          mx[1] = fmaxf(mx[1], s0[c + 1]);
          mx[2] = fmaxf(mx[2], s1[c]);
          mx[3] = fmaxf(mx[3], s1[c + 1]);
        }
      }
      const float m_new =
          fmaxf(m_run, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2);
      const bool need = m_new > m_run + kRescaleLog2;
      if (j > 0 && __any_sync(0xffffffffu, need)) {
        const float f = need ? ex2(m_run - m_new) : 1.0f;
        l_run *= f;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tmem_ld32(t_o + 32u * c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= f;
          tmem_st32(t_o + 32u * c, o);
        }
        tmem_wait_st();
      }
      if (need) m_run = m_new;
      const float m_use = m_run == -INFINITY ? 0.f : m_run;
      const float2 nm2 = make_float2(-m_use, -m_use);
      float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      float cur[32], nxt[32];
      tmem_ld32(t_s, cur);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        tmem_wait_ld();
        if (k < 3) tmem_ld32(t_s + 32u * (k + 1), nxt);  // above what the stores below reach
        if (masked) mask(cur, vis[k]);
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float2 x = ffma2(make_float2(cur[c], cur[c + 1]), sc2, nm2);
          const float2 p = make_float2(ex2(x.x), ex2(x.y));
          ls[(c >> 1) & 1] = fadd2(ls[(c >> 1) & 1], p);
          pk[c >> 1] = pack2<BF16>(p.x, p.y);
        }
        tmem_st16u(t_s + 16u * k, pk);
        if (k == 1) {  // the first 64 keys
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(pfull);
            mbar_arrive(other_turn);
          }
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) cur[c] = nxt[c];
      }
      l_run += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pfull + 8u);
    }
    // Both tiles' last products: the rows below go through the ring's memory.
    if (ok) ok = warp_wait(bar(C::B_DONE), 0, abort_flag, tmo);
    if (ok) {
      tc_fence_after();
      SoftmaxCtx x;
      x.sb = sb;
      x.s = 0;
      x.slot = it.slot;
      x.row0 = kTileRows * grp;
      x.stage_off = C::RING_OFF + (uint32_t)(grp * kTileRows * (D * 4 + 16));
      write_row<D, true, false, BF16>(a, x, r, valid, tok, head, m_run, l_run, t_o);
    }
  } else if (warp >= kDuoCopyWarp) {
    // ============================================================ TMA issuers (two warps)
    if (a.q_tma && warp == kDuoCopyWarp && lane == 0) {
      // both tiles' panels: 128 / G whole tokens each; tokens past the sequence are other rows
      // (or zeros past the batch), whose scores are masked
      mbar_arrive_expect_tx(bar(C::B_QFULL), 2u * NP * kPanel);
      for (int t = 0; t < 2; ++t)
        for (int p = 0; p < NP; ++p)
          tma_load_4d(sb + C::Q_OFF + (t * NP + p) * kPanel, &tm_q, bar(C::B_QFULL), p * 64, 0, g,
                      a.q_row0 + (int32_t)((2 * tp + t) * (kTileRows / a.G)));
    }
    __syncwarp();
    kv_copy_role<NP, NSLOT, C::PANEL_LOG, true, true, kDuoCopyWarps>(
        a, &tm_k, &tm_v, g, kt0, n, warp - kDuoCopyWarp, sb + C::RING_OFF, bar(C::B_FULL),
        bar(C::B_EMPTY), pre_row0, pre_row1, abort_flag, tmo);
    if (a.q_tma && warp == kDuoCopyWarp && lane == 0)
      drain_wait(bar(C::B_QFULL), 0, abort_flag, tmo);
    __syncwarp();
  } else {
    // ============================================================ MMA issuers (lane 0 each)
    const int grp = warp - kDuoMmaWarp;
    constexpr uint32_t idesc_qk = umma_idesc_f16(128, kTileKeys, BF16, false);
    constexpr uint32_t idesc_pv = umma_idesc_f16(128, D, BF16, true);
    constexpr uint32_t kSlotDesc = kPanel >> 4;
    const uint64_t q_desc =
        smem_desc_sw128(sb + C::Q_OFF, 16, 1024) + (uint32_t)(grp * NP) * kSlotDesc;
    const uint64_t k_desc = smem_desc_sw128(sb + C::RING_OFF, 16, 1024);
    const uint64_t v_desc = smem_desc_sw128(sb + C::RING_OFF, (uint32_t)a.v_rows * 128u, 1024);
    const uint32_t t_s = tmem + C::S_COL + 128u * grp, t_o = tmem + (uint32_t)(D * grp);
    auto k_fill = [&](int j) -> uint32_t { return (j == 0 ? 0u : 2u * j - 1u) * NP; };
    auto wait_fills = [&](uint32_t q0) -> bool {
      bool w_ok = true;
#pragma unroll
      for (int p = 0; p < NP; ++p)
        if (w_ok)
          w_ok = warp_wait(bar(C::B_FULL + (q0 + p) % NSLOT), ((q0 + p) / NSLOT) & 1, abort_flag,
                           tmo);
      tc_fence_after();
      return w_ok;
    };
    auto release = [&](uint32_t q0) {
#pragma unroll
      for (int p = 0; p < NP; ++p) umma_commit(bar(C::B_EMPTY + (q0 + p) % NSLOT));
    };
    // S(j) over S(j - 1) and its P, which the PV issued before has read (tcgen05.mma executes in
    // issue order). The slots' descriptors are worked out before the wait that the products hang
    // on: an issuing lane's index arithmetic measured ~100 cycles an MMA.
    uint64_t kd[NP], vd[kTileKeys / 16];
    auto k_descs = [&](int j) {
#pragma unroll
      for (int p = 0; p < NP; ++p) kd[p] = k_desc + ((k_fill(j) + p) % NSLOT) * kSlotDesc;
    };
    auto qk = [&](int j) {
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const uint64_t ad = q_desc + p * kSlotDesc;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_ss(t_s, ad + 2 * kk, kd[p] + 2 * kk, idesc_qk, (p | kk) != 0 ? 1u : 0u);
      }
      umma_commit(bar(C::B_SFULL + grp));
      release(k_fill(j));
    };
    bool ok = warp_wait(bar(C::B_QFULL), 0, abort_flag, tmo) && wait_fills(k_fill(0));
    k_descs(0);
    if (ok && lane == 0) qk(0);
    __syncwarp();
    for (int j = 0; j < n && ok; ++j) {
      const uint32_t v0 = v_item(j, n) * NP;
      if (!(ok = wait_fills(v0))) break;
      const int64_t key0 = kv_tile<true>(a, kt0 + j) * kTileKeys;
      if (tile_unseen<true>(a, key0)) {
        // Unseen rows of pages that were loaded (the others arrived as zeros): behind the sinks
        // and before the window to their pages' ends, and behind the sequence.
        auto zero_rows = [&](int64_t from, int64_t to) {  // keys [from, to) of this tile
          const int r0 = clamp_tile(from - key0), r1 = clamp_tile(to - key0);
          for (int i = lane; i < (r1 - r0) * 8 * NP; i += 32) {
            const uint32_t k = r0 + i / (8 * NP), c = i % (8 * NP);
            const uint32_t off = v_offset<NP, C::PANEL_LOG>(k, c >> 3, a.v_shift);
            st_shared_v4(slot_addr((v0 + (off >> 14)) % NSLOT) + (off & (kPanel - 1)) +
                             (c & 7) * 16,
                         0u, 0u, 0u, 0u);
          }
        };
        const int64_t ps1 = a.page_rows - 1;
        if (a.sinks < a.win_lo) {
          const int64_t page_end = (a.sinks + ps1) & ~ps1, page0 = a.win_lo & ~ps1;
          zero_rows(a.sinks, page_end < a.win_lo ? page_end : a.win_lo);
          zero_rows(page0 > a.sinks ? page0 : a.sinks, a.win_lo);
        }
        zero_rows(a.total_keys, (a.total_keys + ps1) & ~ps1);
        fence_proxy_async_smem();
        __syncwarp();
      }
      {
        const uint32_t s0 = v0 % NSLOT;
#pragma unroll
        for (int ks = 0; ks < kTileKeys / 16; ++ks) {
          const uint32_t off = v_offset<NP, C::PANEL_LOG>(16u * ks, 0, a.v_shift);
          uint32_t sl = s0 + (off >> 14);
          if (sl >= (uint32_t)NSLOT) sl -= NSLOT;
          vd[ks] = v_desc + sl * kSlotDesc + ((off & (kPanel - 1)) >> 4);
        }
        if (j + 1 < n) k_descs(j + 1);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && ok && j + 1 < n) ok = wait_fills(k_fill(j + 1));
        if (ok)
          ok = warp_wait(bar(C::B_PFULL + 2 * grp + h), (uint32_t)j & 1u, abort_flag, tmo);
        tc_fence_after();
        if (ok && lane == 0) {
#pragma unroll
          for (int ks = 4 * h; ks < 4 * h + 4; ++ks)
            umma_ts(t_o, t_s + 8u * ks, vd[ks], idesc_pv, (j > 0 || ks > 0) ? 1u : 0u);
        }
      }
      if (ok && j + 1 < n && lane == 0) qk(j + 1);
      if (ok && lane == 0) release(v0);
      __syncwarp();
    }
    // Every issued MMA must finish before tensor memory is freed.
    if (lane == 0) {
      umma_commit(bar(C::B_DONE));
      drain_wait(bar(C::B_DONE), 0, abort_flag, tmo);
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kDuoMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}
