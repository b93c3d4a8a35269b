// decode_stream.cuh — one query token per sequence over part of its keys (a window and sinks, or
// the keys past a shared prefix), device lengths, groups of G <= 8 heads at head dim 128 or 256:
// the products and the softmax of decode_kernel.cuh (keys on the MMA's M side) in a kernel that
// stays for the whole step. Included by pa_kernels.cu.
//
// A unit is (sequence b, KV head g) with its list of n_b KV tiles (kv_tile). The units are laid
// end to end, b-major, each n_b + 1 slots long (its start, worth about a tile: measured 2.6 us
// at D 128 and 5 us at D 256 for the epilogue and the first loads, against 2.9 and 5 us a tile
// with all CTAs streaming; then its tiles), T slots in all, and CTA c of C takes the c-th of C
// equal runs of slots: a list of segments, each a unit or a part of one. Every CTA gets the same
// work whatever the lengths are, and its copy warps go on into the next segment while the softmax
// warps finish the last one. (One CTA per unit and split pays each unit's start and end in full
// and fills its last wave in part: 32 sequences, window 4,096, D 256: 71 us at 10 splits, 54 us
// at the best count, 4, against 40 us of K/V traffic.)
//
// Each CTA finds its run by itself: a block scan of the units' slots over runs of sequences (one
// each up to 256), then a walk. A segment that is a whole unit writes its output rows; a part of
// a unit leaves its rows and base-2 LSE in the CTA's workspace slot 0 (the CTA's first segment)
// or 1 (its last), which merge_stream_kernel joins after the same scan. Roundings: P to the input
// type (see prefill_kernel) and a whole unit's or merged row's output; partials, their LSEs and all
// sums are fp32.

constexpr int kStreamRuns = 256;  // runs of sequences in the scan (= threads of both kernels)
static_assert(kStreamRuns == kThreads, "one run a thread");

template <int D>
struct StreamCfg {
  static constexpr int NP = D / 64;
  static constexpr int NSLOT = kDecSlots;
  static constexpr int Q_OFF = 0;                          // 2 buffers x NP atoms of 8 rows
  static constexpr int P_OFF = Q_OFF + 2 * NP * 1024;      // 2 buffers x 2 panels x 1 KB
  static constexpr int RING_OFF = P_OFF + 2 * 2 * 1024;
  static constexpr int BAR_OFF = RING_OFF + NSLOT * kPanel;
  static constexpr int B_FULL = 0, B_EMPTY = NSLOT, B_QFULL = 2 * NSLOT, B_SFULL = 2 * NSLOT + 2,
                       B_PFULL = 2 * NSLOT + 4, B_PVDONE = 2 * NSLOT + 6,
                       B_MMADONE = 2 * NSLOT + 8, N_BARS = 2 * NSLOT + 9;
  static constexpr int RED_OFF = BAR_OFF + 8 * (N_BARS + 1);  // [2][4 warps][8 heads]
  static constexpr int SUM_OFF = RED_OFF + 2 * 4 * 8 * 4;     // [4 warps][8 heads]
  static constexpr int RUN_OFF = SUM_OFF + 4 * 8 * 4;         // [kStreamRuns + 1] slots
  static constexpr int MISC_OFF = RUN_OFF + 4 * (kStreamRuns + 1);
  static constexpr int SMEM = MISC_OFF + 16;
  static constexpr int LAUNCH_SMEM = SMEM + 1024;
  static constexpr int PANEL_LOG = (NP == 4) ? 9 : 8;
  static_assert(BAR_OFF % 8 == 0 && RED_OFF % 16 == 0 && MISC_OFF % 4 == 0, "alignment");
  static_assert(kDecCtasPerSm * (LAUNCH_SMEM + 1024) <= 233472, "two CTAs per SM");
};

// Keys, tiles and slots fit 32 bits here (the host sees to it: seq_cap, and the most slots below
// 2^31): a CTA's start is a few hundred instructions that no cache holds yet, and 64-bit
// arithmetic doubles them.

// One sequence's keys and its tile list: tile v of the list is KV tile v for v < head, else
// v + gap; the row sees key k < keys when k >= lo or k < sinks.
struct StreamSeq {
  int32_t keys, lo, head, gap;
};
__device__ __forceinline__ int32_t stream_tile(const StreamSeq& q, int32_t v) {
  return v < q.head ? v : v + q.gap;
}
__device__ __forceinline__ bool stream_unseen(const StreamSeq& q, int32_t sinks, int32_t key) {
  return key >= q.keys || (key < q.lo && key >= sinks);
}

// Sequence b's view (its length clamped into the table row; *bad: it was outside) and the number
// of its tiles: none when it ends before first_key.
__device__ __forceinline__ int32_t stream_seq(const PrefillArgs& a, int32_t b, StreamSeq& q,
                                              bool* bad) {
  int32_t len = __ldg(a.seq_lens + b);
  if ((uint32_t)len > (uint32_t)a.seq_cap) {
    *bad = true;
    len = len < 0 ? 0 : a.seq_cap;
  }
  q.keys = len;
  if (len <= a.first_key32) return 0;
  q.lo = max(max(len - a.window32, 0), a.first_key32);
  const int32_t w0 = q.lo / kTileKeys;
  q.head = (int32_t)(((uint32_t)min(a.sinks32, len) + kTileKeys - 1) / kTileKeys);
  q.gap = max(w0 - q.head, 0);
  return (len - 1) / kTileKeys + 1 - q.gap;
}

// Slots of a unit of n tiles (none without tiles), and sequences of a run of the scan.
__device__ __forceinline__ int32_t stream_slots(int32_t n) { return n > 0 ? n + 1 : 0; }
__device__ __forceinline__ int32_t stream_per(const PrefillArgs& a) {
  return (int32_t)(((uint32_t)a.batch + kStreamRuns - 1) / kStreamRuns);
}

// Slots before every run of sequences (run i: sequences [i per, (i + 1) per)), in all heads, into
// run[0 .. kStreamRuns]; `wsum`: a word per warp. Every thread of the block (kStreamRuns of
// them). Reports bad lengths when `report`.
__device__ __forceinline__ void stream_scan(const PrefillArgs& a, int32_t* run, int32_t* wsum,
                                            bool report) {
  const int t = threadIdx.x, lane = t & 31, wid = t >> 5;
  const int32_t per = stream_per(a);
  bool bad = false;
  int32_t sum = 0;
  StreamSeq q;
  for (int32_t i = 0; i < per; ++i) {
    const int64_t b = (int64_t)t * per + i;
    if (b < a.batch) sum += stream_slots(stream_seq(a, (int32_t)b, q, &bad));
  }
  sum *= a.Hkv;
  if (bad && report) atomicOr(&g_pa_error_flags, kFlagPage);
  int32_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) wsum[wid] = incl;
  __syncthreads();
  int32_t before = 0;
  for (int w = 0; w < wid; ++w) before += wsum[w];
  run[t + 1] = before + incl;
  if (t == 0) run[0] = 0;
  __syncthreads();
}

// The equal runs: C CTAs (two slots at least each: one tile a CTA adds more to the merge than it
// saves; one sequence at window 4,096 measured 16.5 us at two, 18.6 us at one) of q slots, the
// first r of them q + 1.
struct StreamShare {
  uint32_t C, q, r;
  __device__ __forceinline__ StreamShare(int32_t T, int64_t ctas) {
    const uint32_t most = (uint32_t)ctas;
    C = (uint32_t)T / 2 < most ? (uint32_t)T / 2 : most;
    q = C > 0 ? (uint32_t)T / C : 0;
    r = (uint32_t)T - q * C;
  }
  __device__ __forceinline__ int32_t first(uint32_t c) const {
    return (int32_t)(c * q + (c < r ? c : r));
  }
  __device__ __forceinline__ int32_t owner(int32_t x) const {
    const uint32_t big = r * (q + 1), y = (uint32_t)x;
    return (int32_t)(y < big ? y / (q + 1) : r + (y - big) / q);
  }
};

// A CTA's walk along its segments.
struct StreamWalk {
  StreamSeq q;      // the sequence
  int32_t b, g;     // which, and the KV head
  int32_t n_b;      // tiles of the unit
  int32_t t0;       // first tile of the segment in the unit
  int32_t left;     // slots of the CTA's run behind this segment
  int32_t n;        // tiles of the segment
  int32_t index;    // segments before this one
};

// The segment at slot x of the whole list, of a run of `slots`.
__device__ __forceinline__ StreamWalk stream_start(const PrefillArgs& a, const int32_t* run,
                                                   int32_t x, int32_t slots) {
  StreamWalk s;
  int lo = 0;
#pragma unroll 1
  for (int step = kStreamRuns / 2; step > 0; step >>= 1)  // the last run that begins at or before x
    if (run[lo + step] <= x) lo += step;
  bool bad;
  s.b = lo * stream_per(a);
  int32_t off = x - run[lo];
  for (;; ++s.b) {
    s.n_b = stream_seq(a, s.b, s.q, &bad);
    const int32_t all = stream_slots(s.n_b) * a.Hkv;
    if (off < all || s.b + 1 >= a.batch) break;
    off -= all;
  }
  s.g = (int32_t)((uint32_t)off / (uint32_t)(s.n_b + 1));
  off -= s.g * (s.n_b + 1);
  const int32_t mine = min(s.n_b + 1 - off, slots);
  s.left = slots - mine;
  s.t0 = off > 0 ? off - 1 : 0;
  s.n = off > 0 ? mine : mine - 1;  // >= 1: a run has two slots at least
  s.index = 0;
  return s;
}
__device__ __forceinline__ bool stream_next(const PrefillArgs& a, StreamWalk& s) {
  if (s.left <= 1) return false;  // one slot: the start of a unit that the next CTA has
  s.t0 = 0;
  ++s.index;
  if (++s.g == a.Hkv) {
    s.g = 0;
    bool bad;
    do {
      if (s.b + 1 >= a.batch) return false;
      s.n_b = stream_seq(a, ++s.b, s.q, &bad);
    } while (s.n_b == 0);
  }
  const int32_t mine = min(s.n_b + 1, s.left);
  s.left -= mine;
  s.n = mine - 1;
  return true;
}

// Copy warp w of kIssuers: the K/V tiles of all segments through the ring, as kv_copy_role does
// for one unit (K0, K1, V0, K2, V1, ..., V_{n-1} within a segment, fill numbers running on).
template <int NP, int NSLOT, int PANEL_LOG>
__device__ __forceinline__ void stream_copy_role(const PrefillArgs& a, const CUtensorMap* tm_k,
                                                 const CUtensorMap* tm_v, const int32_t* run,
                                                 int32_t x0, int32_t slots, int w, uint32_t ring,
                                                 uint32_t bar_full, uint32_t bar_empty,
                                                 volatile int* abort_flag, uint64_t tmo) {
  const int lane = threadIdx.x & 31;
  auto slot_addr = [&](uint32_t slot) -> uint32_t { return ring + slot * kPanel; };
  auto full = [&](uint32_t slot) -> uint32_t { return bar_full + 8u * slot; };
  const int ppt = a.pages_per_tile, prow = a.page_rows;
  const int vsub = prow >> a.v_shift;             // V boxes per page
  const int vbytes_log = a.v_shift + PANEL_LOG;   // log2 of a V box's bytes
  const int vbox_per_slot = 1 << (14 - vbytes_log);
  bool ok = true;
  // Key-row coordinate in the pool of page `lane` of the segment's tile jt (tile_page_row): pages
  // that the row does not see arrive as zeros.
  auto fetch = [&](const StreamWalk& seg, int jt) -> int32_t {
    int32_t row = a.oob_row;
    const int32_t lp = stream_tile(seg.q, seg.t0 + jt) * ppt + lane, page0 = lp << a.page_shift;
    if (jt < seg.n && lane < ppt && page0 < seg.q.keys &&
        (page0 < a.sinks32 || page0 + prow > seg.q.lo)) {
      const int32_t e = __ldg(a.page_table + (int64_t)seg.b * a.table_stride + lp);
      if (e >= 0 && e < a.num_pages)
        row = e << a.page_shift;
      else if (w == 0)
        atomicOr(&g_pa_error_flags, kFlagPage);
    }
    return row;
  };
  auto acquire = [&](uint32_t q) -> bool {
    const uint32_t slot = q % NSLOT;
    const bool r_ok = q < (uint32_t)NSLOT ||
                      warp_wait(bar_empty + 8u * slot, ((q / NSLOT) - 1) & 1, abort_flag, tmo);
    if (r_ok && lane == 0) mbar_arrive_expect_tx(full(slot), kPanel);
    __syncwarp();
    return r_ok;
  };
  uint32_t base = 0, issued_end = 0;  // fills of the segments before; one past the last issued
  StreamWalk s = stream_start(a, run, x0, slots);
  int32_t row_cur = fetch(s, 0), row_next = fetch(s, 1);
  for (bool more = true; more && ok;) {
    const int n = s.n;
    // the next segment's first table entries are read a segment ahead
    StreamWalk nx = s;
    more = stream_next(a, nx);
    int32_t next_0 = a.oob_row, next_1 = a.oob_row;
    if (more) {
      next_0 = fetch(nx, 0);
      next_1 = fetch(nx, 1);
    }
    int32_t row_prev = a.oob_row;
    for (int j = 0; j <= n && ok; ++j) {
      if (j < n) {
        const uint32_t item = j == 0 ? 0u : 2u * j - 1u;
        for (int k = 0; k < NP && ok; ++k) {
          const uint32_t q = base + item * NP + k;
          if ((int)(q % kIssuers) != w) continue;
          if (!(ok = acquire(q))) break;
          const uint32_t slot = q % NSLOT;
          if (lane < ppt)
            tma_load_3d(slot_addr(slot) + lane * prow * 128, tm_k, full(slot), k * 64, s.g,
                        row_cur);
          issued_end = q + 1;
        }
      }
      if (ok && j >= 1) {
        const uint32_t item = v_item(j - 1, n);
        for (int k = 0; k < NP && ok; ++k) {
          const uint32_t q = base + item * NP + k;
          if ((int)(q % kIssuers) != w) continue;
          if (!(ok = acquire(q))) break;
          const uint32_t slot = q % NSLOT;
          const int bx = k * vbox_per_slot + lane;
          const int pg = bx / vsub, sub = bx - pg * vsub;
          const int32_t prow_b = __shfl_sync(0xffffffffu, row_prev, pg & 31);
          if (lane < vbox_per_slot)
            tma_load_4d(slot_addr(slot) + (lane << vbytes_log), tm_v, full(slot), 0,
                        prow_b + (sub << a.v_shift), 0, s.g);
          issued_end = q + 1;
        }
      }
      row_prev = row_cur;
      row_cur = row_next;
      row_next = fetch(s, j + 2);
    }
    base += 2u * (uint32_t)n * NP;
    s = nx;
    row_cur = next_0;
    row_next = next_1;
  }
  // every copy must land before the CTA may exit (see kv_copy_role)
  for (uint32_t q = base > (uint32_t)NSLOT ? base - NSLOT : 0; q < issued_end; ++q)
    if ((int)(q % kIssuers) == w)
      drain_wait(full(q % NSLOT), (q / NSLOT) & 1, abort_flag, tmo);
  __syncwarp();
}

// WHOLE: the result of a whole unit is the output (16-bit); else a partial too (its row and LSE at
// row b Hq + head of the workspace's first batch * Hq rows, before the part slots), and the
// kernel is launched while the prefix's kernel before it ends.
template <int D, bool BF16, bool WHOLE>
__global__ void __launch_bounds__(kThreads, kDecCtasPerSm)
    decode_stream_kernel(const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const PrefillArgs a) {
  using C = StreamCfg<D>;
  constexpr int NP = C::NP, NSLOT = C::NSLOT, NH = D / 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t* run = reinterpret_cast<int32_t*>(smem + C::RUN_OFF);
  auto bar = [&](int i) -> uint32_t { return sb + C::BAR_OFF + 8u * (uint32_t)i; };
  auto slot_addr = [&](uint32_t r) -> uint32_t { return sb + C::RING_OFF + r * kPanel; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF + 4);

  if (threadIdx.x == 0) {
    for (int i = 0; i < NSLOT; ++i) {
      mbar_init(bar(C::B_FULL + i), 1);
      mbar_init(bar(C::B_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::B_QFULL + i), 4);
      mbar_init(bar(C::B_SFULL + i), 1);
      mbar_init(bar(C::B_PFULL + i), 4);
      mbar_init(bar(C::B_PVDONE + i), 1);
    }
    mbar_init(bar(C::B_MMADONE), 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == kMmaWarp + 1 && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), kDecTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  // its barriers also publish the set-up above; `red` is not in use yet
  stream_scan(a, run, reinterpret_cast<int32_t*>(smem + C::RED_OFF), blockIdx.x == 0);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const StreamShare share(run[kStreamRuns], gridDim.x);
  if (blockIdx.x >= share.C) {
    if (warp == kMmaWarp) tmem_dealloc(tmem, kDecTmemCols);
    if constexpr (!WHOLE) wait_dependencies();
    return;
  }
  const int32_t x0 = share.first(blockIdx.x);
  const int32_t slots = share.first(blockIdx.x + 1) - x0;
  const uint64_t tmo = a.timeout_ns;

  if (warp < 4) {
    // ============================================================ softmax + epilogue
    const int t = threadIdx.x;  // key t of each tile (S^T lane); dim t of each half (O^T lane)
    const int G = a.G;          // <= 8
    const uint32_t t_lane = tmem + ((uint32_t)(warp * 32) << 16);
    // Q rows 0..7 of a segment (zeros past G) in its buffer, 128-byte swizzle, one atom per
    // panel: 8 x D/8 pieces of 16 bytes, NP / 2 a thread. The next segment's are loaded at the
    // start of a segment and stored after its first tile: by then the segment before, the
    // buffer's last reader, has all its S.
    uint4 qv[NP / 2];
    auto q_load = [&](int64_t b, int g) {
#pragma unroll
      for (int i = 0; i < NP / 2; ++i) {
        const int p = t + 128 * i, row = p / (D / 8), col = p % (D / 8);
        qv[i] = row < G ? __ldg(reinterpret_cast<const uint4*>(
                              a.q + (b * a.Hq + g * G + row) * (int64_t)D) + col)
                        : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    auto q_store = [&](int buf) {
#pragma unroll
      for (int i = 0; i < NP / 2; ++i) {
        const int p = t + 128 * i, row = p / (D / 8), col = p % (D / 8);
        st_shared_v4(sb + C::Q_OFF + buf * (NP * 1024) + (col >> 3) * 1024 + row * 128 +
                         (((col & 7) ^ row) << 4),
                     qv[i].x, qv[i].y, qv[i].z, qv[i].w);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::B_QFULL + buf));
    };
    float* red = reinterpret_cast<float*>(smem + C::RED_OFF);
    float* sums = reinterpret_cast<float*>(smem + C::SUM_OFF);
    bool ok = true;
    uint32_t jj = 0;       // tiles of the segments before
    uint32_t fills = 0;    // ring fills of the segments before
    StreamWalk s = stream_start(a, run, x0, slots);
    q_load(s.b, s.g);
    q_store(0);
    for (bool more = true; more && ok;) {
      const int n = s.n;
      const StreamSeq seq = s.q;
      StreamWalk nx = s;
      more = stream_next(a, nx);
      if (more) q_load(nx.b, nx.g);
      float m_run[8], l_part[8];
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        m_run[h] = -INFINITY;
        l_part[h] = 0.f;
      }
      // PV of tile i (counted over all segments) completes phase i/2 of pv_done[i % 2]; the waits
      // below observe every one, the two last of a segment at its end.
      auto wait_pv = [&](uint32_t i) -> bool {
        return warp_wait(bar(C::B_PVDONE + (i & 1)), (i >> 1) & 1, abort_flag, tmo);
      };
      for (int j = 0; j < n; ++j) {
        const uint32_t i = jj + j;
        const int sbuf = i & 1;
        const int32_t key0 = stream_tile(seq, s.t0 + j) * kTileKeys;
        const bool live = !stream_unseen(seq, a.sinks32, key0 + t);
        float sv[8];
        if (ok) ok = warp_wait(bar(C::B_SFULL + sbuf), (i >> 1) & 1, abort_flag, tmo);
        if (ok) {
          tc_fence_after();
          tmem_ld8(t_lane + kDecSCol + 16u * sbuf, sv);
          tmem_wait_ld();
        }
        float mx[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) mx[h] = warp_max(ok && live ? sv[h] : -INFINITY);
        if (lane == 0) {
          float* r = red + sbuf * 32 + warp * 8;
          *reinterpret_cast<float4*>(r) = make_float4(mx[0], mx[1], mx[2], mx[3]);
          *reinterpret_cast<float4*>(r + 4) = make_float4(mx[4], mx[5], mx[6], mx[7]);
        }
        if (named_bar_or(kDecBarSoftmax, 128, !ok)) {
          ok = false;
          break;
        }
        float m_new[8];
        bool need[8], any = false;
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          const float* r = red + sbuf * 32 + h;
          const float tm = fmaxf(fmaxf(r[0], r[8]), fmaxf(r[16], r[24]));
          m_new[h] = fmaxf(m_run[h], tm * a.scale_log2);
          need[h] = m_new[h] > m_run[h] + kRescaleLog2;
          any |= need[h];
        }
        if (j == 0) {
#pragma unroll
          for (int h = 0; h < 8; ++h)
            if (need[h]) m_run[h] = m_new[h];
        } else if (any) {
          ok = wait_pv(i - 1);  // O^T must not change under a running MMA
          if (ok) {
            tc_fence_after();
            float f[8];
#pragma unroll
            for (int h = 0; h < 8; ++h) {
              f[h] = need[h] ? ex2(m_run[h] - m_new[h]) : 1.0f;
              l_part[h] *= f[h];
              if (need[h]) m_run[h] = m_new[h];
            }
#pragma unroll
            for (int hf = 0; hf < NH; ++hf) {
              float o[8];
              tmem_ld8(t_lane + kDecOCol + 16u * hf, o);
              tmem_wait_ld();
#pragma unroll
              for (int h = 0; h < 8; ++h) o[h] *= f[h];
              tmem_st8(t_lane + kDecOCol + 16u * hf, o);
            }
            tmem_wait_st();
          }
        }
        float p[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          const float mu = m_run[h] == -INFINITY ? 0.f : m_run[h];
          p[h] = ok && live ? ex2(fmaf(sv[h], a.scale_log2, -mu)) : 0.f;
          l_part[h] += p[h];
        }
        if (ok && i >= 2) ok = wait_pv(i - 2);  // the last reader of P's buffer
        if (ok && (key0 + kTileKeys > seq.keys ||
                   max(key0, a.sinks32) < min(key0 + kTileKeys, seq.lo))) {
          // V rows of keys that the row does not see may hold any bits; P is 0 there, but
          // 0 * NaN is NaN inside the MMA, so those rows are zeroed. Once S(j+1) and PV(i-1)
          // are done, every earlier fill of V(j)'s slots has landed (K up to K(j+1), V up to
          // V(i-1); a segment's last tile follows K(j) directly), so the parity waits see
          // V(j)'s own fills. Neither wait needs this P.
          if (j + 1 < n)
            ok = warp_wait(bar(C::B_SFULL + ((i + 1) & 1)), ((i + 1) >> 1) & 1, abort_flag, tmo);
          if (ok && i >= 1) ok = wait_pv(i - 1);
          const uint32_t seq0 = fills + v_item(j, n) * NP;
          for (int q = 0; q < NP && ok; ++q)
            ok = warp_wait(bar(C::B_FULL + (seq0 + q) % NSLOT), ((seq0 + q) / NSLOT) & 1,
                           abort_flag, tmo);
          const int32_t page0 = (key0 + t) & ~(a.page_rows - 1);  // its page's first key
          if (ok && !live && page0 < seq.keys &&  // (pages not loaded arrived as zeros)
              (page0 < a.sinks32 || page0 + a.page_rows > seq.lo)) {
#pragma unroll
            for (int q = 0; q < NP; ++q) {
              const uint32_t off = v_offset<NP, C::PANEL_LOG>((uint32_t)t, q, a.v_shift);
              const uint32_t ra = slot_addr((seq0 + (off >> 14)) % NSLOT) + (off & (kPanel - 1));
#pragma unroll
              for (int c = 0; c < 8; ++c) st_shared_v4(ra + c * 16, 0u, 0u, 0u, 0u);
            }
          }
        }
        if (ok) {
          const uint32_t pb = sb + C::P_OFF + (uint32_t)sbuf * 2048u + (uint32_t)(t >> 6) * 1024u;
          const uint32_t chunk = (uint32_t)((t & 63) >> 3), sub = (uint32_t)(t & 7) * 2u;
#pragma unroll
          for (int h = 0; h < 8; ++h)
            st_shared_u16(pb + h * 128u + ((chunk ^ (uint32_t)h) << 4) + sub, to16<BF16>(p[h]));
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bar(C::B_PFULL + sbuf));
        if (j == 0 && more) q_store((s.index + 1) & 1);
      }

      const uint32_t last = jj + n - 1;
      if (ok && last >= 1) ok = wait_pv(last - 1);
      if (ok) ok = wait_pv(last);
      float ls[8];
#pragma unroll
      for (int h = 0; h < 8; ++h) ls[h] = warp_sum(l_part[h]);
      if (lane == 0) {
        *reinterpret_cast<float4*>(sums + warp * 8) = make_float4(ls[0], ls[1], ls[2], ls[3]);
        *reinterpret_cast<float4*>(sums + warp * 8 + 4) = make_float4(ls[4], ls[5], ls[6], ls[7]);
      }
      if (named_bar_or(kDecBarSoftmax, 128, !ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float inv_l[8];
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        ls[h] = (sums[h] + sums[8 + h]) + (sums[16 + h] + sums[24 + h]);
        inv_l[h] = ls[h] > 0.f ? __frcp_rn(ls[h]) : 0.f;
      }
      const bool whole = n == s.n_b;
      const int64_t out_row = (int64_t)s.b * a.Hq + s.g * G;  // heads g G .. g G + G - 1
      const int64_t row0 =
          whole ? out_row
                : (WHOLE ? 0 : (int64_t)a.batch * a.Hq) +
                      (2 * (int64_t)blockIdx.x + (s.index > 0 ? 1 : 0)) * G;
#pragma unroll
      for (int hf = 0; hf < NH; ++hf) {
        float o[8];
        tmem_ld8(t_lane + kDecOCol + 16u * hf, o);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          if (h >= G) continue;
          const int64_t at = (row0 + h) * D + 128 * hf + t;
          if (WHOLE && whole)
            reinterpret_cast<uint16_t*>(a.out)[at] = to16<BF16>(o[h] * inv_l[h]);
          else
            a.ws_o[at] = o[h] * inv_l[h];
        }
      }
      if (!(WHOLE && whole) && t < G) {
        float m = m_run[0], l = ls[0];
#pragma unroll
        for (int h = 1; h < 8; ++h)
          if (t == h) {
            m = m_run[h];
            l = ls[h];
          }
        a.ws_lse[row0 + t] = row_lse(m, l);
      }
      // O^T is read: the next segment's first PV waits for a P that comes after this.
      tc_fence_before();
      jj += n;
      fills += 2u * (uint32_t)n * NP;
      s = nx;
    }
  } else if (warp > kMmaWarp) {
    // ============================================================ TMA issuers (three warps)
    stream_copy_role<NP, NSLOT, C::PANEL_LOG>(a, &tm_k, &tm_v, run, x0, slots,
                                              warp - kMmaWarp - 1, sb + C::RING_OFF,
                                              bar(C::B_FULL), bar(C::B_EMPTY), abort_flag, tmo);
    // All data has landed: the merge starts, and reads the lengths, while the last tiles' products
    // and epilogues run (2 us a call less than from this grid's end).
    launch_dependents();
  } else {
    // ============================================================ MMA issuer (one lane)
    if (lane == 0) {
      constexpr uint32_t idesc_qk = umma_idesc_f16(128, kDecN, BF16, false, false);
      constexpr uint32_t idesc_pv = umma_idesc_f16(128, kDecN, BF16, false, true);
      constexpr uint32_t kSlotDesc = kPanel >> 4;
      const uint64_t q_desc0 = smem_desc_sw128(sb + C::Q_OFF, 16, 0);
      const uint64_t p_desc = smem_desc_sw128(sb + C::P_OFF, 16, 0);
      const uint64_t k_desc = smem_desc_sw128(sb + C::RING_OFF, 16, 1024);
      const uint64_t v_desc = smem_desc_sw128(sb + C::RING_OFF, (uint32_t)a.v_rows * 128u, 1024);
      uint32_t slot = 0, round = 0, jj = 0;
      bool ok = true;
      StreamWalk s = stream_start(a, run, x0, slots);
      do {
        const int n = s.n;
        const uint64_t q_desc = q_desc0 + (uint32_t)(s.index & 1) * (NP * 1024 >> 4);
        ok = thread_wait(bar(C::B_QFULL + (s.index & 1)), (s.index >> 1) & 1, abort_flag, tmo);
        tc_fence_after();
        for (int j = 0; j <= n && ok; ++j) {
          if (j < n) {
            // S^T of tile i is written over that of tile i - 2, which the softmax read before it
            // released P(i-2) (the PV MMA that read P(i-2) was issued before this one).
            const uint32_t i = jj + j;
            const uint32_t s_tmem = tmem + kDecSCol + 16u * (i & 1);
#pragma unroll
            for (int p = 0; p < NP; ++p) {
              ok = thread_wait(bar(C::B_FULL + slot), round & 1, abort_flag, tmo);
              if (!ok) break;
              tc_fence_after();
              const uint64_t ad = k_desc + slot * kSlotDesc, bd = q_desc + p * (1024 >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_ss(s_tmem, ad + 2 * kk, bd + 2 * kk, idesc_qk, (p | kk) != 0 ? 1u : 0u);
              umma_commit(bar(C::B_EMPTY + slot));
              if (++slot == (uint32_t)NSLOT) {
                slot = 0;
                ++round;
              }
            }
            if (!ok) break;
            umma_commit(bar(C::B_SFULL + (i & 1)));
          }
          if (j >= 1) {
            const uint32_t i = jj + j - 1;
            ok = thread_wait(bar(C::B_PFULL + (i & 1)), (i >> 1) & 1, abort_flag, tmo);
            const uint32_t vslot0 = slot;
#pragma unroll
            for (int k = 0; k < NP; ++k) {
              if (ok) ok = thread_wait(bar(C::B_FULL + slot), round & 1, abort_flag, tmo);
              if (++slot == (uint32_t)NSLOT) {
                slot = 0;
                ++round;
              }
            }
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < kTileKeys / 16; ++ks) {
              const uint64_t bd = p_desc + (i & 1) * (2048 >> 4) + (ks >> 2) * (1024 >> 4) +
                                  (ks & 3) * 2;
#pragma unroll
              for (int hf = 0; hf < NH; ++hf) {
                const uint32_t off = v_offset<NP, C::PANEL_LOG>(16u * ks, 2u * hf, a.v_shift);
                uint32_t vs = vslot0 + (off >> 14);
                if (vs >= (uint32_t)NSLOT) vs -= NSLOT;
                umma_ss(tmem + kDecOCol + 16u * hf,
                        v_desc + vs * kSlotDesc + ((off & (kPanel - 1)) >> 4), bd, idesc_pv,
                        (j > 1 || ks > 0) ? 1u : 0u);
              }
            }
#pragma unroll
            for (int k = 0; k < NP; ++k) {
              uint32_t vs = vslot0 + k;
              if (vs >= (uint32_t)NSLOT) vs -= NSLOT;
              umma_commit(bar(C::B_EMPTY + vs));
            }
            umma_commit(bar(C::B_PVDONE + (i & 1)));
          }
        }
        jj += n;
      } while (ok && stream_next(a, s));
      // Every issued MMA must finish before tensor memory is freed.
      umma_commit(bar(C::B_MMADONE));
      drain_wait(bar(C::B_MMADONE), 0, abort_flag, tmo);
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kDecTmemCols);
  }
  // Nothing here needs the prefix's kernel, beside which this one may run; but this grid ends
  // after it, so that the merge, which waits for this grid, has both.
  if constexpr (!WHOLE) wait_dependencies();
}

// The units that the stream kernel cut, and the sequences without a key (zeros): an output row
// (b, head) at a time by WPR warps (1, or all 8 of a block, which take every 8th part: with 30 to
// 40 parts a row one warp's loads came to 18 us, 64 blocks of them leaving the GPU idle). The
// row's parts sit in the slots of CTAs c0 .. c1, those whose runs hold tiles of the unit: slot 0
// of each, or slot 1 of c0 when the unit is not the first of its run. PREFIX: n_pre partials of
// the shared prefix ([n_pre][batch * Hq] rows before the rest of the workspace) join, and a whole
// unit's partial is read from its own row.
constexpr int kMergeWarps = kStreamRuns / 32;

template <int D, int OUT, bool PREFIX, int WPR>
__global__ void __launch_bounds__(kStreamRuns, WPR > 1 ? 4 : 1)
    merge_stream_kernel(const PrefillArgs a, int64_t grid_ctas, const float* pre_o,
                        const float* pre_lse, int n_pre) {
  static_assert(WPR == 1 || WPR == kMergeWarps, "a row takes a warp or the block");
  constexpr int NV = D / 128;  // float4 columns a lane holds
  __shared__ int32_t run[kStreamRuns + 1], wsum[kMergeWarps];
  __shared__ float wpart[WPR > 1 ? kMergeWarps : 1][2];               // M and W of a warp's parts
  __shared__ float4 opart[WPR > 1 ? kMergeWarps : 1][NV][32];         // their weighted rows
  stream_scan(a, run, wsum, false);
  // Launched while the stream kernel ends (programmatic launch): its results are complete past
  // wait_dependencies, which every thread has to pass. The lengths were there before it, so the
  // first row's place is worked out ahead of the wait.
  bool waited = false;
  const StreamShare share(run[kStreamRuns], grid_ctas);
  const int lane = threadIdx.x & 31, wid = threadIdx.x / 32;
  const int64_t rows = (int64_t)a.batch * a.Hq;
  const int32_t per = stream_per(a);
  const int first = WPR > 1 ? wid : 0;  // this warp's first part
  constexpr int64_t kRows = kMergeWarps / WPR;  // rows of a block
  for (int64_t row = (int64_t)blockIdx.x * kRows + wid / WPR; row < rows;
       row += (int64_t)gridDim.x * kRows) {
    // rows < 2^31 (as the sequences' Q tiles are counted in 32 bits)
    const int32_t b = (int32_t)((uint32_t)row / (uint32_t)a.Hq), in_run = b / per;
    const int head = (int)(row - (int64_t)b * a.Hq), g = head / a.G;
    bool bad;
    StreamSeq q;
    int32_t off = run[in_run];  // the unit's first slot (its start; its tiles follow)
    for (int32_t c = in_run * per; c < b; ++c)
      off += stream_slots(stream_seq(a, c, q, &bad)) * a.Hkv;
    const int32_t n_b = stream_seq(a, b, q, &bad);
    off += g * (n_b + 1);
    int32_t c0 = 0, np = 0;  // parts of the unit
    bool whole = false, late = false;
    if (n_b > 0) {
      c0 = share.owner(off + 1);
      np = share.owner(off + n_b) - c0 + 1;
      whole = np == 1;
      late = share.first(c0) < off;  // the run begins in an earlier unit
    }
    if (!PREFIX && whole) continue;  // the stream kernel wrote the output
    if (!waited) wait_dependencies();
    waited = true;
    // Part p: of the prefix (p < n_pre), else of the unit.
    const int64_t unit0 = PREFIX ? rows : 0;  // rows of the workspace before the part slots
    const int64_t total = (PREFIX ? n_pre : 0) + np;
    auto place = [&](int64_t p, const float** o, const float** lse) {
      if (PREFIX && p < n_pre) {
        *o = pre_o + (p * rows + row) * D;
        *lse = pre_lse + p * rows + row;
        return;
      }
      const int64_t i = p - (PREFIX ? n_pre : 0);
      const int64_t r = whole ? row
                              : unit0 + (2 * (c0 + i) + (i == 0 && late ? 1 : 0)) * a.G +
                                    (head - g * a.G);
      *o = a.ws_o + r * D;
      *lse = a.ws_lse + r;
    };
    // This warp's parts: first, first + WPR, ... (lane i holds the LSE of the i-th of 32).
    const int64_t mine = total > first ? (total - first + WPR - 1) / WPR : 0;
    auto lse_of = [&](int64_t i) -> float {
      if (i >= mine) return -INFINITY;
      const float *o, *lse;
      place(first + i * WPR, &o, &lse);
      return *lse;
    };
    const float lse0 = lse_of(lane);
    float M = lse0;
    for (int64_t i = 32 + lane; i < mine; i += 32) M = max_nan(M, lse_of(i));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
    float W = 0.f;
    float4 acc[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kGroup = 8 / NV;  // parts loaded together
    for (int64_t i32 = 0; M != -INFINITY && i32 < mine; i32 += 32) {
      const float lse = i32 == 0 ? lse0 : lse_of(i32 + lane);
      const float wl = lse == -INFINITY ? 0.f : exp2f(lse - M);
      const int n32 = mine - i32 < 32 ? (int)(mine - i32) : 32;
      for (int i0 = 0; i0 < n32; i0 += kGroup) {
        float4 x[kGroup][NV];
#pragma unroll
        for (int k = 0; k < kGroup; ++k) {
          if (i0 + k >= n32) continue;
          const float *o, *l;
          place(first + (i32 + i0 + k) * WPR, &o, &l);
#pragma unroll
          for (int v = 0; v < NV; ++v)
            x[k][v] = *reinterpret_cast<const float4*>(o + lane * 4 + 128 * v);
        }
#pragma unroll
        for (int k = 0; k < kGroup; ++k) {
          const float w = __shfl_sync(0xffffffffu, wl, (i0 + k) & 31);
          if (i0 + k >= n32 || w == 0.f) continue;
          W += w;
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            acc[v].x = fmaf(w, x[k][v].x, acc[v].x);
            acc[v].y = fmaf(w, x[k][v].y, acc[v].y);
            acc[v].z = fmaf(w, x[k][v].z, acc[v].z);
            acc[v].w = fmaf(w, x[k][v].w, acc[v].w);
          }
        }
      }
    }
    if constexpr (WPR > 1) {  // the warps' sums join (their weights brought to one maximum)
      if (lane == 0) {
        wpart[wid][0] = M;
        wpart[wid][1] = W;
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) opart[wid][v][lane] = acc[v];
      __syncthreads();
      if (wid < NV) {  // warp v: the 128 columns from 128 v on
        float Mt = -INFINITY;
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) Mt = max_nan(Mt, wpart[w][0]);
        W = 0.f;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) {
          const float f = wpart[w][0] == -INFINITY ? 0.f : exp2f(wpart[w][0] - Mt);
          const float4 x = opart[w][wid][lane];
          W = fmaf(f, wpart[w][1], W);
          sum.x = fmaf(f, x.x, sum.x);
          sum.y = fmaf(f, x.y, sum.y);
          sum.z = fmaf(f, x.z, sum.z);
          sum.w = fmaf(f, x.w, sum.w);
        }
        acc[0] = sum;
      }
      __syncthreads();  // before the next row's sums
      if (wid >= NV) continue;
    }
    const float inv = W > 0.f ? 1.f / W : 0.f;
    uint16_t* dst = reinterpret_cast<uint16_t*>(a.out) + row * D;
#pragma unroll
    for (int v = 0; v < (WPR > 1 ? 1 : NV); ++v)
      *reinterpret_cast<uint2*>(dst + lane * 4 + 128 * (WPR > 1 ? wid : v)) =
          make_uint2(pack2<OUT == kOutBf16>(acc[v].x * inv, acc[v].y * inv),
                     pack2<OUT == kOutBf16>(acc[v].z * inv, acc[v].w * inv));
  }
  if (!waited) wait_dependencies();
}
