// pa_schedule.h — host side of the balanced schedule: the item list of a plan made with the
// balanced policy, rebuilt deterministically from the plan's fields (and, for a batch, the
// sequences' lengths) by the planner, the prefill launch and the combine launch.
#pragma once
#include <vector>

#include "pa.h"
#include "pa_geometry.h"

namespace pa {

// f's status; PA_ERR_CUDA when host memory runs out (nothing throws across the ABI).
template <class F>
int no_throw(F&& f) {
  try {
    return f();
  } catch (...) {
    return PA_ERR_CUDA;
  }
}

struct Schedule {
  std::vector<PaItem> items;          // in launch order
  std::vector<PaSplitBlock> split;    // row blocks with more than one item
  int32_t n_slots = 0;                // workspace slots (partials)
  int32_t rows_per_block = 0;         // packed rows of a row block (per * 128)
  int32_t max_parts = 1;
  double makespan_us = 0.0;           // simulated
};

// Fills `out` for the piece described by `p` (its shape fields; the policy is not read).
// Returns false when the schedule would exceed the kernel's item or split-block tables.
bool build_balanced(const pa_plan_t& p, Schedule* out);

// A batch of sequences: sequence b has q_lens[b] query rows after hist_lens[b] keys.
struct Batch {
  std::vector<PaSeq> seq;   // q_row0, rows, hist, rb0 of every sequence
  int64_t total_rows = 0;   // sum of q_lens
  int64_t row_blocks = 0;   // sum of the sequences' row blocks
  int64_t max_hist = 0;
};
// Validates the lengths and lays the sequences out (rows packed in order). Returns a pa_status.
int describe_batch(int batch, const int32_t* q_lens, const int64_t* hist_lens, int G, int Hkv,
                   int per, Batch* out);
// CTAs per row block of a batch: 2 (CTA pairs, head dim 256) only when some sequence has two
// or more Q tiles; a batch of one-tile sequences (decode) would leave half of every pair idle.
int batch_ctas_per_unit(int head_dim, int G, int batch, const int32_t* q_lens);
// Q tiles per row block of a windowed batch: 2 when some sequence has two or more (a CTA pair at
// head dim 256, one CTA below), else 1.
int window_q_tiles_per_unit(int G, int batch, const int32_t* q_lens);
// The balanced schedule of a batch (row blocks of all sequences, longest first). With a window
// (win non-null) a row block's tiles are those its rows' windows and the sinks reach, and its
// items' [kt0, kt1) count along that list (window_tiles).
struct Window {
  int64_t window, sinks;
};
bool build_batch(int num_sms, int head_dim, int per, int G, int Hkv, const Batch& bt,
                 Schedule* out, const Window* win = nullptr);

// Most KV tiles that a window and sinks reach in a sequence of up to max_len keys.
int64_t window_most_tiles(int64_t max_len, int64_t window, int64_t sinks);

// How the decode entry points with a 16-bit output share their (sequence, KV head) units, of up
// to `tiles` KV tiles each: groups of up to 8 heads at head dim 128 or 256 on the stream kernel
// (`units` CTAs, equal shares of the tiles, two part slots of G rows each), the others in uniform
// splits of the single-CTA kernel (`units` = batch * Hkv * splits).
struct DecodeWork {
  bool stream;
  int32_t splits;
  int64_t units;
  // Workspace rows (D + 1 fp32 each) of the partials; `rows` = batch * Hq output rows.
  int64_t ws_rows(int G, int64_t rows) const {
    return stream ? 2 * units * G : splits > 1 ? splits * rows : 0;
  }
  uint64_t ws_bytes(int D, int G, int64_t rows) const {
    return (uint64_t)ws_rows(G, rows) * (D + 1) * 4ull;
  }
};
DecodeWork decode_work(int num_sms, int D, int G, int Hkv, int64_t batch, int64_t tiles);

// A decode step over a shared prefix: the prefix's packed (sequence, head) rows in `q_tiles` tiles
// a KV head, on `per` CTAs a unit, `splits` uniform splits of its keys; the sequences' own keys as
// decode_work shares them, on `own.units` CTAs beside the prefix's where that is the shorter.
// Workspace rows: the prefix's partials [splits][rows], then the own part's: [rows] of whole units
// and the part slots (stream kernel), or its uniform partials.
struct PrefixWork {
  int32_t per, q_tiles, splits;
  DecodeWork own;
  int64_t ws_rows(int G, int64_t rows) const {
    return splits * rows + (own.stream ? rows : 0) + own.ws_rows(G, rows);
  }
  uint64_t ws_bytes(int D, int G, int64_t rows) const {
    return (uint64_t)ws_rows(G, rows) * (D + 1) * 4ull;
  }
};
PrefixWork prefix_work(int num_sms, int D, int G, int Hkv, int64_t batch, int64_t prefix_len,
                       int64_t max_len);

}  // namespace pa
