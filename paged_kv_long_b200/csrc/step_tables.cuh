// step_tables.cuh — the bookkeeping of a serving step on the device: page-table entries for the
// pages that the step's new rows need, and every new row's position and pool slot. Included by
// pa_kernels.cu.
//
// Request b brings r_b new rows after h_b cached keys. With old_b = ceil(h_b / PS) pages owned
// and new_b = ceil((h_b + r_b) / PS) - old_b pages to add,
//   R_b = sum of r over the requests before b, N_b = sum of new over them,
//   page(b, i) = table[b][i] for i < old_b, else free[used + N_b + i - old_b],
//   row R_b + i: position p = h_b + i, slot page(b, p / PS) * PS + p % PS.
//
// One launch: every block scans the lengths itself (8 bytes a request out of L2) and keeps both
// prefix sums in shared memory, so no block waits for another. A row whose page is new reads the
// free list, not the table entry that some block of this launch writes; the entries of owned
// pages are only read. Rows and new pages find their request by binary search in the prefix sums.
// Latency-bound at a decode step: a chain of three dependent loads and the scan's barriers.

constexpr int kStepThreads = 256;
constexpr int kStepMaxSeqs = PA_STEP_MAX_SEQS;

// Sum that stays at INT32_MAX once it gets there (lengths that no pool could hold).
__device__ __forceinline__ int32_t sat_add(int32_t a, int32_t b) {
  const uint32_t s = (uint32_t)a + (uint32_t)b;  // both >= 0: no wrap
  return s > 0x7fffffffu ? 0x7fffffff : (int32_t)s;
}

// A request's lengths, negative ones read as 0 and the sum kept below 2^31 (*bad is set).
struct StepSeq {
  int32_t hist, rows, old_pages, new_pages;
};
__device__ __forceinline__ StepSeq step_seq(const int32_t* q_lens, const int32_t* hist_lens,
                                            int b, int page_shift, int32_t stride, bool* bad) {
  StepSeq s;
  s.hist = __ldg(hist_lens + b);
  s.rows = __ldg(q_lens + b);
  if (s.hist < 0 || s.rows < 0) *bad = true;
  s.hist = max(s.hist, 0);
  s.rows = max(s.rows, 0);
  if (s.rows > 0x7fffffff - s.hist) {
    *bad = true;
    s.rows = 0x7fffffff - s.hist;
  }
  const uint32_t ps1 = (1u << page_shift) - 1u;
  s.old_pages = (int32_t)(((uint32_t)s.hist + ps1) >> page_shift);
  const int32_t all = (int32_t)(((uint32_t)(s.hist + s.rows) + ps1) >> page_shift);
  s.new_pages = max(0, min(all, stride) - s.old_pages);  // pages past the table row: not taken
  if (s.rows > 0 && all > stride) *bad = true;
  return s;
}

// Index of the last entry <= x of the ascending pre[0 .. n) (pre[0] = 0 <= x).
__device__ __forceinline__ int last_le(const int32_t* pre, int n, int32_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kStepThreads) block_tables_kernel(
    int B, const int32_t* __restrict__ q_lens, const int32_t* __restrict__ hist_lens,
    int page_shift, int32_t num_pages, const int32_t* __restrict__ free_pages, int32_t n_free,
    const int32_t* __restrict__ used_in, int32_t* __restrict__ used_out, int32_t* table,
    int32_t stride, int32_t max_rows, int32_t* __restrict__ slots,
    int32_t* __restrict__ positions, int32_t* __restrict__ cu_q_lens,
    int32_t* __restrict__ seq_lens) {
  extern __shared__ int32_t step_smem[];
  int32_t* pre_rows = step_smem;           // [B + 1]
  int32_t* pre_pages = step_smem + B + 1;  // [B + 1]
  __shared__ int32_t wsum[2][kStepThreads / 32];
  const int t = threadIdx.x, lane = t & 31, wid = t >> 5;
  const bool first = blockIdx.x == 0;
  bool bad = false;
  int32_t used = __ldg(used_in);
  if (used < 0 || used > n_free) {
    bad = true;
    used = used < 0 ? 0 : n_free;
  }

  // Prefix sums over the requests: thread t sums its run, a warp and then a block scan of the
  // runs' sums, and the run again from its start.
  const int per = (B + kStepThreads - 1) / kStepThreads;
  const int b0 = min(B, t * per), b1 = min(B, b0 + per);
  int32_t rows = 0, pages = 0;
  for (int b = b0; b < b1; ++b) {
    const StepSeq s = step_seq(q_lens, hist_lens, b, page_shift, stride, &bad);
    if (first) seq_lens[b] = s.hist + s.rows;
    pre_rows[b] = rows;
    pre_pages[b] = pages;
    rows = sat_add(rows, s.rows);
    pages = sat_add(pages, s.new_pages);
  }
  int32_t ir = rows, ip = pages;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t vr = __shfl_up_sync(0xffffffffu, ir, o);
    const int32_t vp = __shfl_up_sync(0xffffffffu, ip, o);
    if (lane >= o) {
      ir = sat_add(ir, vr);
      ip = sat_add(ip, vp);
    }
  }
  if (lane == 31) {
    wsum[0][wid] = ir;
    wsum[1][wid] = ip;
  }
  int32_t er = __shfl_up_sync(0xffffffffu, ir, 1), ep = __shfl_up_sync(0xffffffffu, ip, 1);
  if (lane == 0) er = ep = 0;
  __syncthreads();
  for (int w = 0; w < wid; ++w) {
    er = sat_add(er, wsum[0][w]);
    ep = sat_add(ep, wsum[1][w]);
  }
  for (int b = b0; b < b1; ++b) {
    pre_rows[b] = sat_add(pre_rows[b], er);
    pre_pages[b] = sat_add(pre_pages[b], ep);
  }
  if (t == kStepThreads - 1) {
    pre_rows[B] = sat_add(er, rows);
    pre_pages[B] = sat_add(ep, pages);
  }
  __syncthreads();
  const int32_t total = pre_rows[B], taken = pre_pages[B];
  if (first) {
    for (int b = t; b <= B; b += kStepThreads) cu_q_lens[b] = pre_rows[b];
    if (t == 0) {
      *used_out = min(sat_add(used, taken), n_free);
      if (total > max_rows || taken > n_free - used) bad = true;
    }
  }

  // Entry k of the step's free pages; -1 where the list is at its end or holds no page.
  auto fresh = [&](int32_t k) -> int32_t {
    if (k >= n_free - used) return -1;
    const int32_t e = __ldg(free_pages + used + k);
    if (e >= 0 && e < num_pages) return e;
    bad = true;
    return -1;
  };
  const int64_t tid = (int64_t)blockIdx.x * kStepThreads + t;
  const int64_t step = (int64_t)gridDim.x * kStepThreads;
  for (int64_t i = tid; i < max_rows; i += step) {
    int32_t slot = -1, pos = -1;  // rows behind the last request
    if (i < total) {
      const int b = last_le(pre_rows, B, (int32_t)i);
      const int32_t h = max(__ldg(hist_lens + b), 0);
      pos = h + ((int32_t)i - pre_rows[b]);
      const int32_t lp = pos >> page_shift;
      const int32_t old = (int32_t)(((uint32_t)h + (1u << page_shift) - 1u) >> page_shift);
      int32_t e = -1;
      if (lp < stride) {
        if (lp < old) {
          e = table[(int64_t)b * stride + lp];
          if (e < 0 || e >= num_pages) {
            bad = true;
            e = -1;
          }
        } else {
          e = fresh(pre_pages[b] + (lp - old));
        }
      }
      if (e >= 0) slot = (e << page_shift) + (pos & ((1 << page_shift) - 1));
    }
    slots[i] = slot;
    positions[i] = pos;
  }
  for (int64_t k = tid; k < taken; k += step) {
    const int b = last_le(pre_pages, B, (int32_t)k);
    const int32_t h = max(__ldg(hist_lens + b), 0);
    const int32_t old = (int32_t)(((uint32_t)h + (1u << page_shift) - 1u) >> page_shift);
    table[(int64_t)b * stride + old + ((int32_t)k - pre_pages[b])] = fresh((int32_t)k);
  }
  if (bad) atomicOr(&g_pa_error_flags, kFlagPage);
}
